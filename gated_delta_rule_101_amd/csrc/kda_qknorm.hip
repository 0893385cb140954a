// Norm of each query and key head with the rotation by position in the same
// pass, forward and backward, for gfx950:
//   n = x r, r = 1 / sqrt(mean x^2 + eps),  y = R (n w)
//   g = R^T dy,  dx = r (g w - n mean(g w n)),  dw = sum g n over tokens and heads
// with R turning pairs of the first R channels by their angles: (a, b) ->
// (a cos - b sin, a sin + b cos), pairs being (i, i + R / 2) or neighbours.
//
// One read and one write of each element, bound by HBM bandwidth.  A wave has
// one token; a head is LPH of its lanes, each with two blocks of V channels that
// hold whole pairs between them: blocks R / 2 apart in the rotated part, half
// of the rest apart behind it.  So the rotation stays inside a lane, and the
// token's cosines and sines are read once for all its heads.  Head groups are
// read BATCH at a time, so that their loads are in flight together; a group is all
// queries or all keys, so that weights and their gradients are named by it.  Where few
// tokens would leave the device empty, a token's head groups are dealt to
// several waves.  Backward: a lane's channels are the same for every head, so
// the weights' gradients add up in registers, meet in LDS and go to the
// workspace once a workgroup, to be summed by column.
// 16384 tokens of 32 + 8 heads x 128, bfloat16: forward 68 us, 5.0 TB/s; backward
// 101 us, 5.1 TB/s, and 5 us of column sums.  256 tokens: 8.7 us.
#include "kda_attn.h"
#include "kda_block.h"
#include "kda_block_device.h"

namespace kda {
namespace {

// One lane's channels: block j of a head's halves at a[j] and b[j], none (-1)
// beyond the head's end; angle indexes for the two.
template <int V, int NV, bool NEIGH> struct Channels {
    int a[NV], b[NV];
    int turned[NV];
    __device__ __forceinline__ Channels(int l, int lanes, int D, int R)
    {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (l + lanes * j);       // place among the D / 2 first halves
            turned[j] = 2 * c < R;
            if (2 * c >= D) a[j] = b[j] = -1;
            else if (turned[j]) {
                a[j] = NEIGH && V == 1 ? 2 * c : c;
                b[j] = NEIGH && V == 1 ? 2 * c + 1 : R / 2 + c;
            } else {
                a[j] = R / 2 + c;                    // R + (c - R / 2)
                b[j] = R / 2 + c + (D - R) / 2;
            }
        }
    }
};

template <int V, int NV, bool NEIGH> struct Angles {
    float cos[NV][V], sin[NV][V];                    // of the pairs (a, b), or of a's pairs, then b's
    __device__ __forceinline__ void load(const float *row, const Channels<V, NV, NEIGH> &ch, int R)
    {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                int i;
                if (NEIGH && V > 1) i = (e < V / 2 ? ch.a[j] : ch.b[j] - V) / 2 + e;
                else i = NEIGH ? ch.a[j] / 2 : ch.a[j] + e;
                const bool on = ch.turned[j] && ch.a[j] >= 0;
                cos[j][e] = on ? row[i] : 1.f;
                sin[j][e] = on ? row[R / 2 + i] : 0.f;
            }
    }
    // x and y: the blocks a and b; SIGN -1 turns back
    template <int SIGN> __device__ __forceinline__ void turn(float (&x)[NV][V], float (&y)[NV][V]) const
    {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (NEIGH && V > 1) {
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    pair<SIGN>(x[j][2 * e], x[j][2 * e + 1], cos[j][e], sin[j][e]);
                    pair<SIGN>(y[j][2 * e], y[j][2 * e + 1], cos[j][V / 2 + e], sin[j][V / 2 + e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) pair<SIGN>(x[j][e], y[j][e], cos[j][e], sin[j][e]);
            }
        }
    }
    template <int SIGN> static __device__ __forceinline__ void pair(float &a, float &b, float c, float s)
    {
        const float t = SIGN * s, u = a * c - b * t;
        b = a * t + b * c;
        a = u;
    }
};

template <typename T, int V, int NV, bool NEIGH> struct Head {
    typedef Channels<V, NV, NEIGH> Ch;
    Pack<T, V> a[NV], b[NV];
    __device__ __forceinline__ void load(const T *p, const Ch &ch)
    {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            a[j].zero();
            b[j].zero();
            if (p && ch.a[j] >= 0) {
                a[j].stream(p + ch.a[j]);
                b[j].stream(p + ch.b[j]);
            }
        }
    }
    __device__ __forceinline__ void to_f32(float (&x)[NV][V], float (&y)[NV][V]) const
    {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            a[j].to_f32(x[j]);
            b[j].to_f32(y[j]);
        }
    }
    static __device__ __forceinline__ void store(T *p, const float (&x)[NV][V], const float (&y)[NV][V], const Ch &ch)
    {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (ch.a[j] >= 0) {
                Pack<T, V>::unstream(p + ch.a[j], x[j]);
                Pack<T, V>::unstream(p + ch.b[j], y[j]);
            }
    }
};

template <int V, int NV> struct Weights {
    float a[2][NV][V], b[2][NV][V];                  // queries', keys'
};


template <typename T, int V, int NV, bool NEIGH, bool BWD>
__global__ void __launch_bounds__(256) kda_qk_norm_kernel(QkNormArgs a, int lanes, int parts)
{
    typedef Head<T, V, NV, NEIGH> H;
    constexpr int BATCH = BWD ? 3 : 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63, l = lane & (lanes - 1), sub = lane / lanes;
    const int per_wave = 64 / lanes, q_groups = (a.Hq + per_wave - 1) / per_wave, groups = q_groups + (a.Hk + per_wave - 1) / per_wave;
    const Channels<V, NV, NEIGH> ch(l, lanes, a.D, a.R);
    Weights<V, NV> w, dw;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float *p = s ? a.wk : a.wq;
                const bool on = p && ch.a[j] >= 0;
                w.a[s][j][e] = on ? p[ch.a[j] + e] : 1.f;
                w.b[s][j][e] = on ? p[ch.b[j] + e] : 1.f;
                dw.a[s][j][e] = dw.b[s][j][e] = 0.f;
            }
    const float inv_d = 1.f / a.D;
    const int64_t units = a.T * parts;
    for (int64_t u = (int64_t)blockIdx.x * 4 + wave; u < units; u += (int64_t)gridDim.x * 4) {
        const int64_t t = u / parts;
        const int part = (int)(u - t * parts);
        const int pos = a.positions ? a.positions[t] : 0;
        const bool real = pos >= 0, beyond = a.rotary && pos >= a.longest;
        Angles<V, NV, NEIGH> angles;
        angles.load(a.rotary + (real && !beyond ? (int64_t)pos * a.R : 0), ch, a.rotary ? a.R : 0);
        const float poison = beyond ? __builtin_nanf("") : 0.f;
        for (int g0 = part; g0 < groups; g0 += parts * BATCH) {
            H x[BATCH], gy[BWD ? BATCH : 1];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int g = g0 + i * parts;
                const bool is_q = g < q_groups;
                const int h = (is_q ? g : g - q_groups) * per_wave + sub;
                const bool on = g < groups && h < (is_q ? a.Hq : a.Hk) && real;
                const int64_t head = (int64_t)h * a.D;
                x[i].load(on ? (is_q ? (const T *)a.q + t * a.q_stride : (const T *)a.k + t * a.k_stride) + head : nullptr, ch);
                if constexpr (BWD)
                    gy[i].load(on ? (is_q ? (const T *)a.gq + t * a.gq_stride : (const T *)a.gk + t * a.gk_stride) + head : nullptr, ch);
            }
            // a group of heads, all queries or all keys
            const auto work = [&](auto keys, const H &xi, const H &gi, int h) {
                constexpr int S = decltype(keys)::value;
                const bool mine = h < (S ? a.Hk : a.Hq);
                float p[NV][V], q[NV][V], ss = 0.f, sd = 0.f;
                xi.to_f32(p, q);
                float gp[NV][V], gq[NV][V];
                if constexpr (BWD) {
                    gi.to_f32(gp, gq);
                    angles.template turn<-1>(gp, gq);
                }
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        ss += p[j][e] * p[j][e];
                        ss += q[j][e] * q[j][e];
                        if constexpr (BWD) {
                            sd += gp[j][e] * w.a[S][j][e] * p[j][e];
                            sd += gq[j][e] * w.b[S][j][e] * q[j][e];
                        }
                    }
                for (int m = 1; m < lanes; m <<= 1) {
                    ss += __shfl_xor(ss, m, 64);
                    if constexpr (BWD) sd += __shfl_xor(sd, m, 64);
                }
                // lanes of no head and rows of no token add nothing, also where eps is 0
                const float r = mine && real ? __builtin_amdgcn_rsqf(ss * inv_d + a.eps) + poison : 0.f;
                const float back = BWD ? sd * inv_d * r * r : 0.f;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        if constexpr (BWD) {
                            dw.a[S][j][e] += gp[j][e] * (p[j][e] * r);
                            dw.b[S][j][e] += gq[j][e] * (q[j][e] * r);
                            p[j][e] = r * (gp[j][e] * w.a[S][j][e] - p[j][e] * back);
                            q[j][e] = r * (gq[j][e] * w.b[S][j][e] - q[j][e] * back);
                        } else {
                            p[j][e] = p[j][e] * r * w.a[S][j][e];
                            q[j][e] = q[j][e] * r * w.b[S][j][e];
                        }
                    }
                if constexpr (!BWD) angles.template turn<1>(p, q);
                if (!real) {                          // a row of no token
#pragma unroll
                    for (int j = 0; j < NV; ++j)
#pragma unroll
                        for (int e = 0; e < V; ++e) p[j][e] = q[j][e] = 0.f;
                }
                if (mine)
                    H::store((S ? (T *)a.k_out + t * a.ko_stride : (T *)a.q_out + t * a.qo_stride) + (int64_t)h * a.D, p, q, ch);
            };
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int g = g0 + i * parts;
                if (g >= groups) break;
                if (g < q_groups) work(Const<0>{}, x[i], gy[BWD ? i : 0], g * per_wave + sub);
                else work(Const<1>{}, x[i], gy[BWD ? i : 0], (g - q_groups) * per_wave + sub);
            }
        }
    }
    if constexpr (BWD) {
        if (!a.ws) return;
        extern __shared__ float sums[];              // [2][D], filled wave after wave
        const auto add = [&](float &v) {             // over the heads side by side in the wave
            for (int m = lanes; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
        };
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    add(dw.a[s][j][e]);
                    add(dw.b[s][j][e]);
                }
        for (int v = 0; v < 4; ++v) {
            if (v == wave && sub == 0)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int j = 0; j < NV; ++j)
                        if (ch.a[j] >= 0)
#pragma unroll
                            for (int e = 0; e < V; ++e) {
                                float &x = sums[s * a.D + ch.a[j] + e], &y = sums[s * a.D + ch.b[j] + e];
                                x = v ? x + dw.a[s][j][e] : dw.a[s][j][e];
                                y = v ? y + dw.b[s][j][e] : dw.b[s][j][e];
                            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < 2 * a.D; i += 256) a.ws[(int64_t)blockIdx.x * 2 * a.D + i] = sums[i];
    }
}

struct Shape {
    int vec;                             // V
    int lanes, parts;
    int64_t blocks;
};
// Lanes a head: as many as its pairs of blocks, a power of two.
int head_lanes(int D, int V)
{
    int n = 1;
    while (n < 64 && n * 2 * V < D) n *= 2;
    return n;
}

constexpr int64_t FILL = 4096;           // waves that fill the device
// Workgroups: all resident (the backward's two a CU, a row of the workspace each:
// 101 us at 16384 tokens of 32 + 8 heads x 128, 110 with 1024, 123 with 768).  By
// elements a wave has fewer bytes in flight, and four a CU serve better (the same of
// 100 channels, bfloat16 / float32: 282 / 203 us, 483 / 292 with 512), but for long
// float32 rows (250 channels 449 us, 489 with 1024).
constexpr int64_t FWD_BLOCKS = 1024, BWD_BLOCKS = 512, BWD_NARROW = 1024;

Shape shape_of(const QkNormArgs &a, bool bwd)
{
    Shape s;
    // The widest V in which blocks are whole and rows aligned: 16 bytes, 8 of
    // bfloat16 (16384 tokens of 40 heads x 120: 198 us by elements, 88 so), or elements.
    const size_t e = a.bf16 ? 2 : 4;
    const auto fits = [&](int V) {
        const auto whole = [&](int64_t stride, const void *p) { return stride % V == 0 && ((uintptr_t)p & (V * e - 1)) == 0; };
        return a.D % (2 * V) == 0 && a.R % (2 * V) == 0 && whole(a.q_stride, a.q) && whole(a.k_stride, a.k) &&
               whole(a.qo_stride, a.q_out) && whole(a.ko_stride, a.k_out) &&
               (!bwd || (whole(a.gq_stride, a.gq) && whole(a.gk_stride, a.gk)));
    };
    s.vec = a.bf16 && fits(8) ? 8 : fits(4) ? 4 : 1;
    s.lanes = head_lanes(a.D, s.vec);
    const int per_wave = 64 / s.lanes, groups = (a.Hq + per_wave - 1) / per_wave + (a.Hk + per_wave - 1) / per_wave;
    const int64_t want = a.T > 0 ? FILL / a.T : 1;
    s.parts = (int)(want < 1 ? 1 : want > groups ? groups : want);
    const int64_t units = a.T * s.parts;
    s.blocks = (units + 3) / 4;
    const int64_t most = !bwd ? FWD_BLOCKS : s.vec > 1 || (!a.bf16 && a.D > 128) ? BWD_BLOCKS : BWD_NARROW;
    if (s.blocks > most) s.blocks = most;
    return s;
}

template <typename T, int V, int NV, bool BWD>
hipError_t launch(const QkNormArgs &a, const Shape &s, hipStream_t stream)
{
    const size_t lds = BWD && a.ws ? (size_t)2 * a.D * sizeof(float) : 0;
    if (a.neighbours)
        hipLaunchKernelGGL((kda_qk_norm_kernel<T, V, NV, true, BWD>), dim3((unsigned)s.blocks), dim3(256), lds, stream, a, s.lanes, s.parts);
    else
        hipLaunchKernelGGL((kda_qk_norm_kernel<T, V, NV, false, BWD>), dim3((unsigned)s.blocks), dim3(256), lds, stream, a, s.lanes, s.parts);
    return hipGetLastError();
}
template <typename T, bool BWD> hipError_t launch_v(const QkNormArgs &a, const Shape &s, hipStream_t stream)
{
    if (s.vec == WIDE<T>) return launch<T, WIDE<T>, 1, BWD>(a, s, stream);
    if constexpr (sizeof(T) == 2)
        if (s.vec == 4) return launch<T, 4, 1, BWD>(a, s, stream);
    if (a.D <= 128) return launch<T, 1, 1, BWD>(a, s, stream);
    return a.D <= 256 ? launch<T, 1, 2, BWD>(a, s, stream) : launch<T, 1, 4, BWD>(a, s, stream);
}

}  // namespace

hipError_t launch_qk_norm_fwd(const QkNormArgs &a, hipStream_t stream)
{
    const Shape s = shape_of(a, false);
    return a.bf16 ? launch_v<uint16_t, false>(a, s, stream) : launch_v<float, false>(a, s, stream);
}

int64_t qk_norm_bwd_workspace_floats(int64_t T, int Hq, int Hk, int D)
{
    // as many rows as any shape of these sizes has workgroups: a wave at least a head group
    const int64_t units = T * (Hq + Hk), blocks = (units + 3) / 4;
    return (blocks < BWD_NARROW ? blocks : BWD_NARROW) * 2 * D;
}

hipError_t launch_qk_norm_bwd(const QkNormArgs &a, hipStream_t stream)
{
    const Shape s = shape_of(a, true);
    ColumnSum jobs[2];
    int n = 0;
    if (a.dwq) jobs[n++] = {a.ws, a.dwq, a.T > 0 ? s.blocks : 0, a.D, 2 * (int64_t)a.D, false};
    if (a.dwk) jobs[n++] = {a.ws + a.D, a.dwk, a.T > 0 ? s.blocks : 0, a.D, 2 * (int64_t)a.D, false};
    if (n && !column_sums_fit(jobs, n)) return hipErrorNotSupported;
    if (s.blocks > 0) {
        const hipError_t e = a.bf16 ? launch_v<uint16_t, true>(a, s, stream) : launch_v<float, true>(a, s, stream);
        if (e != hipSuccess) return e;
    }
    return n ? launch_column_sums(jobs, n, stream) : hipSuccess;
}

}  // namespace kda
