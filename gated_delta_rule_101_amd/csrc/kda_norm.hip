// Layer norm for gfx950, forward and backward, over rows of D channels:
//   y = n w + b with n = (x - mean) r, r = 1 / sqrt(var + eps)
//   dx = r (g - mean(g) - n mean(g n)) with g = dy w,   dw = sum dy n,  db = sum dy.
//
// One read and one write of each element, bound by HBM bandwidth.  A group of
// TPR threads holds a whole row in registers (8 to 32 elements a thread),
// so the mean and then the centred sum of squares are taken without reading
// the row again, and the variance does not cancel.  TPR grows with D: above
// a wavefront the waves' sums also pass through LDS.
// Groups walk rows with a stride, keeping their channels' weights and, in the
// backward, their partial dw and db in registers; those meet in LDS, go to the
// workspace once a workgroup and are summed by column afterwards.
// Measured (bfloat16): 65536 x 4096 forward 0.197 ms, 5.4 TB/s; 16384 x 4096
// backward 0.091 ms, 4.4 TB/s with its column sums; 8192 x 16384 0.102 and 0.174
// ms, 5.3 and 4.6 TB/s (1024 threads a row, 16 elements each, without the next
// row's request for want of registers, took 0.17 ms for 0.04 and 0.28 for 0.07 at
// 3587 x 10272).
#include "kda_block.h"
#include "kda_block_device.h"

namespace kda {
namespace {

// Threads of a workgroup: whole groups, at least 256.
template <int TPR> constexpr int BLOCK = TPR > 256 ? TPR : 256;

// Sums of M values over 16 lanes (TPR = 16) or the wavefront, in every lane:
// pairs, quads, then halves and rows mirrored (all lanes of a quad hold its sum by
// then), rows by swaps.  Against shuffles, which go through LDS: 8192 x 16384 102
// us for 127, 65536 x 1024 55 for 56.5; but 65536 x 4096 212 for 206, so groups of 256
// threads keep the shuffles.
template <int TPR, int M> __device__ __forceinline__ void lane_sums(float (&x)[M])
{
    if constexpr (TPR == 256) {
#pragma unroll
        for (int m = 1; m < 64; m <<= 1)
#pragma unroll
            for (int i = 0; i < M; ++i) x[i] += __shfl_xor(x[i], m, 64);
    } else {
        constexpr int HALF_MIRROR = 0x141, MIRROR = 0x140;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            x[i] = quad_add<0x4E>(quad_add<0xB1>(x[i]));
            x[i] = quad_add<MIRROR>(quad_add<HALF_MIRROR>(x[i]));
            if constexpr (TPR > 16) {
                const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[i]), __float_as_uint(x[i]), false, false);
                x[i] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
                const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x[i]), __float_as_uint(x[i]), false, false);
                x[i] = __uint_as_float(q[0]) + __uint_as_float(q[1]);
            }
        }
    }
}

// Sums of M values over a group.  Above a wavefront the waves' sums meet in
// `part`, whose `slot` no later call may take before another barrier has
// passed: callers alternate slots.
template <int M> struct Part {
    float v[M];
};
template <int TPR, int M>
__device__ __forceinline__ void group_sums(float (&x)[M], Part<M> (*part)[BLOCK<TPR> / 64], int slot)
{
    lane_sums<TPR>(x);
    if constexpr (TPR > 64) {
        constexpr int WAVES = TPR / 64;
        const int wave = threadIdx.x / 64;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int m = 0; m < M; ++m) part[slot][wave].v[m] = x[m];
        __syncthreads();
#pragma unroll
        for (int m = 0; m < M; ++m) x[m] = 0.f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i)
#pragma unroll
            for (int m = 0; m < M; ++m) x[m] += part[slot][wave / WAVES * WAVES + i].v[m];
    }
}

// Channels of vector j of thread l: V j TPR + V l ..; live while below D.
template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(BLOCK<TPR>) kda_layer_norm_fwd_kernel(NormArgs a)
{
    constexpr int GROUPS = BLOCK<TPR> / TPR;
    __shared__ Part<1> part[4][BLOCK<TPR> / 64];
    const int l = threadIdx.x % TPR, D = a.D;
    float w[NV][V], b[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int d = V * (j * TPR + l) + c;
            w[j][c] = a.weight && d < D ? a.weight[d] : 1.f;
            b[j][c] = a.bias && d < D ? a.bias[d] : 0.f;
        }
    const float inv_d = 1.f / D;
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    // The next row is requested while this one is reduced.  Groups past the
    // last row repeat it (they take part in the barriers) and store nothing.
    int64_t row = (int64_t)blockIdx.x * GROUPS + threadIdx.x / TPR;
    Pack<T, V> raw[NV];
    const auto fetch = [&](int64_t r) {
        const T *x = (const T *)a.x + (r < a.rows ? r : a.rows - 1) * D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = V * (j * TPR + l);
            if (d < D) raw[j].stream(x + d);
            else raw[j].zero();
        }
    };
    fetch(row);
    int slot = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows; r0 += step, row += step) {
        float v[NV][V], s[1] = {0.f}, ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            raw[j].to_f32(v[j]);
#pragma unroll
            for (int c = 0; c < V; ++c) s[0] += v[j][c];
        }
        if (r0 + step < a.rows) fetch(row + step);
        group_sums<TPR>(s, part, slot);
        const float mean = s[0] * inv_d;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (V * (j * TPR + l) < D)
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    v[j][c] -= mean;
                    ss[0] = __builtin_fmaf(v[j][c], v[j][c], ss[0]);
                }
        group_sums<TPR>(ss, part, slot + 1);
        slot ^= 2;
        const float r = rsqrtf(__builtin_fmaf(ss[0], inv_d, a.eps));
        if (row < a.rows) {
            T *y = (T *)a.y + row * D;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int d = V * (j * TPR + l);
                if (d < D) {
                    float o[V];
#pragma unroll
                    for (int c = 0; c < V; ++c) o[c] = __builtin_fmaf(v[j][c] * r, w[j][c], b[j][c]);
                    Pack<T, V>::unstream(y + d, o);
                }
            }
        }
    }
}

template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(BLOCK<TPR>) kda_layer_norm_bwd_kernel(NormBwdArgs a)
{
    constexpr int GROUPS = BLOCK<TPR> / TPR;
    __shared__ Part<2> part[4][BLOCK<TPR> / 64];
    const int l = threadIdx.x % TPR, D = a.D;
    // Above 16 elements a thread the weights lie in LDS: with them in registers as
    // well the widest rows spilled.
    constexpr bool IN_LDS = NV * V > 16;
    constexpr bool AHEAD = !IN_LDS || V == 8;   // registers for the next row as well
    __shared__ __attribute__((aligned(16))) float ws[IN_LDS ? NV * V * TPR : 1];
    float wr[IN_LDS ? 1 : NV][V], dw[NV][V] = {}, db[NV][V] = {};
    constexpr int K = IN_LDS ? 0 : 1;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int d = V * (j * TPR + l) + c;
            wr[K * j][c] = a.weight && d < D ? a.weight[d] : 1.f;
            if (IN_LDS) ws[d] = wr[0][c];   // read back by this thread alone
        }
    const float inv_d = 1.f / D;
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    int64_t row = (int64_t)blockIdx.x * GROUPS + threadIdx.x / TPR;   // rows and idle groups as in the forward
    Pack<T, V> xr[NV], gr[NV];
    const auto fetch = [&](int64_t r) {
        const int64_t at = (r < a.rows ? r : a.rows - 1) * D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = V * (j * TPR + l);
            if (d < D) {
                xr[j].stream((const T *)a.x + at + d);
                gr[j].stream((const T *)a.dy + at + d);
            } else {
                xr[j].zero();
                gr[j].zero();
            }
        }
    };
    if (AHEAD) fetch(row);
    int slot = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows; r0 += step, row += step) {
        if (!AHEAD) fetch(row);
        float v[NV][V], g[NV][V];
        float s[2] = {0.f, 0.f}, ss[2] = {0.f, 0.f};   // of x, g; of (x - mean)^2, g (x - mean)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            xr[j].to_f32(v[j]);
            gr[j].to_f32(g[j]);
#pragma unroll
            for (int c = 0; c < V; ++c) {
                s[0] += v[j][c];
                s[1] = __builtin_fmaf(g[j][c], (IN_LDS ? ws[V * (j * TPR + l) + c] : wr[K * j][c]), s[1]);
            }
        }
        if (AHEAD && r0 + step < a.rows) fetch(row + step);
        group_sums<TPR>(s, part, slot);
        const float mean = s[0] * inv_d;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (V * (j * TPR + l) < D)
    #pragma unroll
                for (int c = 0; c < V; ++c) {
                    v[j][c] -= mean;
                    ss[0] = __builtin_fmaf(v[j][c], v[j][c], ss[0]);
                    ss[1] = __builtin_fmaf(g[j][c] * (IN_LDS ? ws[V * (j * TPR + l) + c] : wr[K * j][c]), v[j][c], ss[1]);
                }
        group_sums<TPR>(ss, part, slot + 1);
        slot ^= 2;
        const float r = rsqrtf(__builtin_fmaf(ss[0], inv_d, a.eps));
        const float c1 = s[1] * inv_d, c2 = ss[1] * r * inv_d;   // mean g, mean g n
        if (row < a.rows) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int d = V * (j * TPR + l);
                if (d < D) {
                    float o[V];
        #pragma unroll
                    for (int c = 0; c < V; ++c) {
                        const float n = v[j][c] * r;
                        dw[j][c] = __builtin_fmaf(g[j][c], n, dw[j][c]);
                        db[j][c] += g[j][c];
                        o[c] = r * (__builtin_fmaf(g[j][c], (IN_LDS ? ws[V * (j * TPR + l) + c] : wr[K * j][c]), -c1) - n * c2);
                    }
                    Pack<T, V>::unstream((T *)a.dx + row * D + d, o);
                }
            }
        }
    }
    if (!a.ws) return;
    float *p = a.ws + (int64_t)blockIdx.x * 2 * D;
    if constexpr (GROUPS == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const int d = V * (j * TPR + l) + c;
                if (d < D) {
                    p[d] = dw[j][c];
                    p[D + d] = db[j][c];
                }
            }
    } else {   // the groups' sums meet in LDS, in order
        constexpr int WIDTH = NV * V * TPR;
        __shared__ float sums[GROUPS][2][WIDTH];
        const int grp = threadIdx.x / TPR;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const int d = V * (j * TPR + l) + c;
                sums[grp][0][d] = dw[j][c];
                sums[grp][1][d] = db[j][c];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += BLOCK<TPR>) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < GROUPS; ++q) s += sums[q][i >= D][i >= D ? i - D : i];
            p[i] = s;
        }
    }
}

int threads_per_row(int D) { return D <= 256 ? 16 : D <= 1024 ? 64 : D <= 4096 ? 256 : 512; }
int groups_per_block(int tpr) { return tpr < 256 ? 256 / tpr : 1; }

// Workgroups: one round of rows if there are few, else a number that walks
// the rows in a loop and keeps weights and partial sums in registers.
int64_t fwd_blocks(int64_t rows, int tpr, int D)
{
    const int64_t need = (rows + groups_per_block(tpr) - 1) / groups_per_block(tpr);
    // all resident; 65536 x 4096: 208 us, 211 at 2048, 334 at 16384
    const int64_t most = tpr < 512 ? 1024 : D <= 16 * tpr ? 512 : 256;
    return need < most ? need : most;
}
int64_t bwd_blocks(int64_t rows, int tpr)
{
    const int64_t need = (rows + groups_per_block(tpr) - 1) / groups_per_block(tpr);
    const int64_t most = tpr == 512 ? 256 : 768;   // all resident; 16384 x 4096: 91 us, 97 at 512, 113 at 1024
    return need < most ? need : most;
}

// f(integral constants V, NV, TPR): 16 / sizeof(T) elements an access where
// D allows it; 8 or 16 elements a thread, 16 or 32 above 4096 channels.
template <int N> struct Int { static constexpr int value = N; };
template <typename T, int V, typename F> hipError_t by_size(int D, int tpr, F f)
{
    const bool half = D <= 8 * tpr;
    if (tpr == 16) return half ? f(Int<8 / V>{}, Int<16>{}) : f(Int<16 / V>{}, Int<16>{});
    if (tpr == 64) return half ? f(Int<8 / V>{}, Int<64>{}) : f(Int<16 / V>{}, Int<64>{});
    if (tpr == 256) return half ? f(Int<8 / V>{}, Int<256>{}) : f(Int<16 / V>{}, Int<256>{});
    return D <= 16 * tpr ? f(Int<16 / V>{}, Int<512>{}) : f(Int<32 / V>{}, Int<512>{});
}

template <typename T, int V> hipError_t fwd_v(const NormArgs &a, hipStream_t s)
{
    const int tpr = threads_per_row(a.D);
    return by_size<T, V>(a.D, tpr, [&](auto nv, auto t) {
        constexpr int NV = decltype(nv)::value, TPR = decltype(t)::value;
        kda_layer_norm_fwd_kernel<T, V, NV, TPR><<<(unsigned)fwd_blocks(a.rows, TPR, a.D), BLOCK<TPR>, 0, s>>>(a);
        return hipGetLastError();
    });
}

template <typename T, int V> hipError_t bwd_v(const NormBwdArgs &a, hipStream_t s)
{
    const int tpr = threads_per_row(a.D);
    return by_size<T, V>(a.D, tpr, [&](auto nv, auto t) {
        constexpr int NV = decltype(nv)::value, TPR = decltype(t)::value;
        kda_layer_norm_bwd_kernel<T, V, NV, TPR><<<(unsigned)bwd_blocks(a.rows, TPR), BLOCK<TPR>, 0, s>>>(a);
        return hipGetLastError();
    });
}

}  // namespace

int64_t norm_bwd_workspace_floats(int64_t rows, int D)
{
    const int tpr = threads_per_row(D);
    return bwd_blocks(rows, tpr) * 2 * D;
}

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t s)
{
    (void)hipGetLastError();
    if (a.bf16) return a.D % 8 == 0 ? fwd_v<uint16_t, 8>(a, s) : a.D % 4 == 0 ? fwd_v<uint16_t, 4>(a, s) : fwd_v<uint16_t, 1>(a, s);
    return a.D % 4 == 0 ? fwd_v<float, 4>(a, s) : fwd_v<float, 1>(a, s);
}

hipError_t launch_norm_bwd(const NormBwdArgs &args, hipStream_t s)
{
    (void)hipGetLastError();
    NormBwdArgs a = args;
    const bool sums = a.dweight || a.dbias;
    if (!sums) a.ws = nullptr;
    if (a.rows > 0) {
        const hipError_t e = a.bf16 ? (a.D % 8 == 0 ? bwd_v<uint16_t, 8>(a, s) : a.D % 4 == 0 ? bwd_v<uint16_t, 4>(a, s) : bwd_v<uint16_t, 1>(a, s))
                                    : (a.D % 4 == 0 ? bwd_v<float, 4>(a, s) : bwd_v<float, 1>(a, s));
        if (e != hipSuccess || !sums) return e;
    }
    const int tpr = threads_per_row(a.D);
    const int64_t n = a.rows > 0 ? bwd_blocks(a.rows, tpr) : 0;
    const ColumnSum jobs[] = {{a.ws, a.dweight, n, a.D, 2 * (int64_t)a.D, false},
                              {n ? a.ws + a.D : nullptr, a.dbias, n, a.D, 2 * (int64_t)a.D, false}};
    return launch_column_sums(jobs, 2, s);
}

}  // namespace kda
