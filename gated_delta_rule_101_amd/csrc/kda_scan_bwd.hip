// Gradients of the selective state space scan for gfx950.
//
// Forward, per channel d and state n (s: time step after bias and softplus):
//   h_t = a_t h_{t-1} + s_t x_t B_t,  a_t = exp(s_t A),  r_t = C_t . h_t,
//   y_t = (r_t + D x_t) silu(z_t)
// With gy = dy silu(z), q_t the gradient of h_t and g_t = a_t q_t:
//   q_t = C_t gy_t + g_{t+1}          (g past the end: dh_final)
//   dC_t = sum_d gy_t h_t             dB_t = sum_d s_t x_t q_t
//   p1_t = B_t . q_t                  p2_t = A . (g_t h_{t-1})
//   dx = s p1 + D gy                  ds = x p1 + p2,  ddt = ds * softplus'
//   dA = sum_t s_t g_t h_{t-1}        dD = sum gy x,   dz = dy (r + D x) silu'(z)
//
// Four kernels.
//  1. Segments of SEG tokens side by side, a lane a channel as in the forward:
//     the state a segment adds (from zero) and, with the running decay
//     P_t = prod a, the gradient it adds in front of itself, sum_t P_t C_t gy_t.
//     Both directions share each exp.
//  2. The true state in front of every segment and the true gradient behind it,
//     one thread per (d, n) over the segments.
//  3. The gradients.  A workgroup owns 64 channels and one segment.  Here a lane
//     owns ONE state of one channel (16 lanes a channel, 4 channels a
//     wavefront), so a whole chunk of 16 tokens keeps its decays and states in
//     registers between the forward and the reverse walk, and the sums over
//     channels of dB and dC are plain accumulators while the wavefront goes
//     through its channels.  The sums over n (r, p1, p2) reduce 16 tokens over
//     16 lanes by a butterfly that halves the values at each step (2 additions
//     a value), leaving lane i with token i.  Per-token values enter as DPP row
//     broadcasts of a register that holds token i in lane i.  First the
//     segment's states at every chunk start are recomputed into LDS, then the
//     chunks run backwards.
//  4. Column sums of the workgroups' partial dA, dD, dbias, dB, dC.
// Bound by vector instructions (about 22 issue slots per token, channel and
// state in kernel 3, 7 for its recomputation, 9 in kernel 1).
#include "kda_block.h"
#include "kda_block_device.h"

namespace kda {
namespace {

constexpr int CHUNK = 16;        // tokens a chunk: one per lane of a DPP row
constexpr int CH = 64;           // channels a workgroup
constexpr int WAVES = 4, QUADS = CH / WAVES / 4;

// Blocks of 16 states, and chunks a segment (LDS: a chunk's start states take
// 4 KiB per block).
int state_blocks(int N) { return N <= 16 ? 1 : N <= 32 ? 2 : 4; }
constexpr int seg_chunks(int nb) { return nb <= 2 ? 8 : 4; }

// Workspace, in floats.
struct Layout {
    int nseg, tiles, np;             // segments, 64-channel tiles a group, padded states
    float *h, *g, *sum;              // [B][nseg][D][np] states in front / gradients behind; [B][nseg][D]
    float *dA, *dD, *db;             // [B nseg][D][N], [B nseg][D] twice
    float *dB, *dC;                  // [tiles][B][T][G][N]
    int64_t floats;
};
Layout layout(float *p, int B, int T, int D, int N, int G)
{
    Layout w;
    const int nb = state_blocks(N), seg = CHUNK * seg_chunks(nb);
    w.nseg = T > 0 ? (T + seg - 1) / seg : 0;
    w.tiles = (D / G + CH - 1) / CH;
    w.np = 16 * nb;
    const auto r4 = [](int64_t n) { return (n + 3) / 4 * 4; };   // 16-byte aligned parts
    const int64_t bs = (int64_t)B * w.nseg;
    const int64_t state = bs * D * w.np, chan = r4(bs * D), rows = r4((int64_t)w.tiles * B * T * G * N);
    const int64_t a = r4(bs * D * N);
    int64_t o = 0;
    const auto take = [&](int64_t n) { float *q = p ? p + o : nullptr; o += n; return q; };
    w.h = take(state);
    w.g = take(state);
    w.sum = take(chan);
    w.dA = take(a);
    w.dD = take(chan);
    w.db = take(chan);
    w.dB = take(rows);
    w.dC = take(rows);
    w.floats = o;
    return w;
}

// --------------------------------------------------- 1. what a segment adds

template <typename T, int NP>
__device__ __forceinline__ void row_uniform(float (&o)[NP], const T *p, int N)
{
#pragma unroll
    for (int i = 0; i < NP; ++i) o[i] = i < N ? to_f32(p[i]) : 0.f;
}

template <typename T, int NB>
__global__ void __launch_bounds__(64) kda_scan_bwd_segment_kernel(ScanBwdArgs a, const T *__restrict__ Bm,
                                                                  const T *__restrict__ Cm, Layout w, int seg_tokens)
{
    constexpr int NP = 16 * NB;
    unsigned id = blockIdx.x;
    const int tile = id % w.tiles;
    id /= w.tiles;
    const int grp = id % a.G;
    id /= a.G;
    const int seg = id % w.nseg, b = id / w.nseg;
    const int D = a.D, N = a.N, Dg = D / a.G;
    const int c = tile * CH + threadIdx.x;
    const bool ok = c < Dg;
    const int d = grp * Dg + (ok ? c : Dg - 1);
    const int len = seq_length(a.lengths, b, a.T);
    const int t0 = seg * seg_tokens, te = min(t0 + seg_tokens, len);

    float A2[NP], h[NP], r[NP], P[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        A2[n] = n < N ? a.A[(int64_t)d * N + n] * LOG2E : 0.f;
        h[n] = r[n] = 0.f;
        P[n] = 1.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const int64_t base = (int64_t)b * a.T * D + d;
    const T *xp = (const T *)a.x + base, *tp = (const T *)a.dt + base, *gp = (const T *)a.dy + base;
    const T *zp = a.z ? (const T *)a.z + base : nullptr;
    const int64_t row0 = ((int64_t)b * a.T * a.G + grp) * N, row = (int64_t)a.G * N;
    float sum = 0.f;
    for (int t = t0; t < te; ++t) {
        const int64_t o = (int64_t)t * D;
        const float x = to_f32(xp[o]);
        float s = to_f32(tp[o]) + bias, gy = to_f32(gp[o]);
        if (a.softplus) s = softplus_f32(s);
        if (zp) {
            const float z = to_f32(zp[o]);
            gy *= z * sigmoid_f32(z);
        }
        sum += s;
        const float u = s * x;
        float Bv[NP], Cv[NP];
        row_uniform<T, NP>(Bv, Bm + row0 + t * row, N);
        row_uniform<T, NP>(Cv, Cm + row0 + t * row, N);
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const float e = fast_exp2(s * A2[n]);
            h[n] = __builtin_fmaf(e, h[n], u * Bv[n]);
            P[n] *= e;
            r[n] = __builtin_fmaf(P[n], gy * Cv[n], r[n]);
        }
    }
    if (!ok) return;
    const int64_t at = (((int64_t)b * w.nseg + seg) * D + d);
#pragma unroll
    for (int n = 0; n < NP; n += 4) {
        const float hv[4] = {h[n], h[n + 1], h[n + 2], h[n + 3]}, rv[4] = {r[n], r[n + 1], r[n + 2], r[n + 3]};
        store4(w.h + at * NP + n, hv);
        store4(w.g + at * NP + n, rv);
    }
    w.sum[at] = sum;
}

// --------------------------------- 2. states in front, gradients behind

// In place: h[seg] becomes the state in front of segment seg, g[seg] the
// gradient behind it.  A segment's decay is exp(A sum s).
__global__ void __launch_bounds__(256) kda_scan_bwd_join_kernel(ScanBwdArgs a, Layout w)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t per = (int64_t)a.D * w.np;
    if (id >= a.B * per) return;
    const int b = (int)(id / per);
    const int64_t dn = id % per;
    const int d = (int)(dn / w.np), n = (int)(dn % w.np);
    const bool in = n < a.N;
    const float A2 = in ? a.A[(int64_t)d * a.N + n] * LOG2E : 0.f;
    const int64_t st = ((int64_t)b * a.D + d) * a.N + n;
    float *hp = w.h + (int64_t)b * w.nseg * per + dn, *gp = w.g + (int64_t)b * w.nseg * per + dn;
    const float *sp = w.sum + (int64_t)b * w.nseg * a.D + d;
    float h = in && a.h0 ? a.h0[st] : 0.f;
#pragma unroll 4
    for (int s = 0; s < w.nseg; ++s) {
        const float add = hp[s * per], e = fast_exp2(A2 * sp[(int64_t)s * a.D]);
        hp[s * per] = h;
        h = __builtin_fmaf(e, h, add);
    }
    float g = in && a.dh_final ? a.dh_final[st] : 0.f;
#pragma unroll 4
    for (int s = w.nseg - 1; s >= 0; --s) {
        const float add = gp[s * per], e = fast_exp2(A2 * sp[(int64_t)s * a.D]);
        gp[s * per] = g;
        g = __builtin_fmaf(e, g, add);
    }
    if (in && a.dh0) a.dh0[st] = g;
}

// ------------------------------------------------------- 3. the gradients

// Sums v[t] over the 16 lanes of each DPP row for 16 tokens t at once; lane i
// returns token i's sum.  Each step adds a partner lane's half of the values
// to the own half: lanes 8..15 keep tokens 8..15, then lanes with bit 2 set
// the upper four, and so on.
template <int CTRL, int BANKS>
__device__ __forceinline__ float dpp_add(float keep, float x)
{
    // lanes of the selected banks: x + x of the partner lane; others: keep
    const int p = __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true);
    const float s = x + __int_as_float(p);
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(keep), __float_as_int(s), 0xE4, 0xF, BANKS, false));
}
__device__ __forceinline__ float row_sum_tokens(const float (&v)[16])
{
    constexpr int ROR8 = 0x128, SHL4 = 0x104, SHR4 = 0x114, SWAP2 = 0x4E, SWAP1 = 0xB1;
    const int lane = threadIdx.x & 15;
    float a[8], b[4], c[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = dpp_add<ROR8, 0xC>(dpp_add<ROR8, 0xF>(0.f, v[i]), v[i + 8]);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = dpp_add<SHR4, 0xA>(dpp_add<SHL4, 0xF>(0.f, a[i]), a[i + 4]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float p = dpp_add<SWAP2, 0xF>(0.f, b[i]), q = dpp_add<SWAP2, 0xF>(0.f, b[i + 2]);
        c[i] = lane & 2 ? q : p;
    }
    const float p = dpp_add<SWAP1, 0xF>(0.f, c[0]), q = dpp_add<SWAP1, 0xF>(0.f, c[1]);
    return lane & 1 ? q : p;
}

// f(integral constant t) for t = 0 .. 15, or 15 .. 0.
template <int I> struct At { static constexpr int value = I; };
template <int I = 0, typename F> __device__ __forceinline__ void each_token(F &&f)
{
    f(At<I>{});
    if constexpr (I + 1 < CHUNK) each_token<I + 1>(f);
}
template <int I = CHUNK - 1, typename F> __device__ __forceinline__ void each_token_back(F &&f)
{
    f(At<I>{});
    if constexpr (I > 0) each_token_back<I - 1>(f);
}

// [channel][16 tokens] tiles in LDS.  Threads that stage and finish tokens
// access 4 tokens of one channel (16 bytes), 64 channels a wavefront; those
// that compute access 4 channels' 16 tokens.  The 4-token pieces of a channel
// are permuted by its index so that neither has bank conflicts.
__device__ __forceinline__ int piece(int ch, int p) { return ch * 16 + 4 * (p ^ ((ch >> 2) & 3)); }
__device__ __forceinline__ int token_at(int ch, int t) { return piece(ch, t >> 2) + (t & 3); }

template <typename T, int NB>
__global__ void __launch_bounds__(256) kda_scan_bwd_kernel(ScanBwdArgs a, Layout w)
{
    constexpr int K = NB <= 2 ? 8 : 4, SEG = K * CHUNK;
    static_assert(QUADS == 4 && WAVES * QUADS * 4 == CH, "a wavefront's channels");
    __shared__ __attribute__((aligned(16))) float t_s[CH * 16], t_u[CH * 16], t_g[CH * 16];   // s, s x, gy
    __shared__ __attribute__((aligned(16))) float t_r[CH * 16], t_p1[CH * 16], t_p2[CH * 16];
    __shared__ float start[K][NB][CH * 16];               // states at the chunks' starts, [channel][16]
    __shared__ float l_A[NB][CH * 16], l_g[NB][CH * 16], l_dA[NB][CH * 16];
    __shared__ float flush[WAVES][8][64];                 // dB, dC of a chunk, per wavefront

    const int tid = threadIdx.x, wave = tid / 64, lane = tid & 63;
    const int ch4 = lane / 16, n = lane & 15;             // compute: channel of the quad, state or token
    unsigned id = blockIdx.x;
    const int tile = id % w.tiles;
    id /= w.tiles;
    const int grp = id % a.G;
    id /= a.G;
    const int seg = id % w.nseg, b = id / w.nseg;
    const int D = a.D, N = a.N, Dg = D / a.G;
    const int len = seq_length(a.lengths, b, a.T);
    const int t0 = seg * SEG, t1 = min(t0 + SEG, a.T), nch = (t1 - t0 + CHUNK - 1) / CHUNK;
    const int64_t bseg = (int64_t)b * w.nseg + seg;

    // staging role: channel `lane` of the tile, tokens 4 wave .. 4 wave + 3 of a chunk
    const bool ok = tile * CH + lane < Dg;
    const int d = grp * Dg + (ok ? tile * CH + lane : Dg - 1);
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f, skip = a.Dskip ? a.Dskip[d] : 0.f;
    const int64_t base = (int64_t)b * a.T * D + d;
    const int64_t row0 = ((int64_t)b * a.T * a.G + grp) * N, row = (int64_t)a.G * N;

    for (int i = tid; i < NB * CH * 16; i += 256) {
        const int nb = i / (CH * 16), c = i / 16 % CH, st = nb * 16 + (i & 15);
        const bool in = tile * CH + c < Dg;
        const int dd = grp * Dg + (in ? tile * CH + c : Dg - 1);
        const int64_t at = (bseg * D + dd) * w.np + st;
        l_A[nb][i % (CH * 16)] = st < N ? a.A[(int64_t)dd * N + st] : 0.f;
        start[0][nb][i % (CH * 16)] = w.h[at];
        l_g[nb][i % (CH * 16)] = w.g[at];
        l_dA[nb][i % (CH * 16)] = 0.f;
    }

    // B or C of a chunk's tokens for the lane's state; zero behind the end
    const auto load_rows = [&](float (&o)[CHUNK], const void *p, int tc, int nb) {
        const int st = nb * 16 + n;
#pragma unroll
        for (int t = 0; t < CHUNK; ++t)
            o[t] = tc + t < len && st < N ? to_f32(((const T *)p)[row0 + (tc + t) * row + st]) : 0.f;
    };

    // states at the chunks' starts
    for (int c = 0; c + 1 < nch; ++c) {
        const int tc = t0 + c * CHUNK;
        float s4[4], u4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = tc + 4 * wave + i;
            s4[i] = u4[i] = 0.f;
            if (t < len) {
                const int64_t o = base + (int64_t)t * D;
                const float v = to_f32(((const T *)a.dt)[o]) + bias;
                s4[i] = a.softplus ? softplus_f32(v) : v;
                u4[i] = s4[i] * to_f32(((const T *)a.x)[o]);
            }
        }
        store4(t_s + piece(lane, wave), s4);
        store4(t_u + piece(lane, wave), u4);
        __syncthreads();
        for (int nb = 0; nb < NB; ++nb) {
            float Bv[CHUNK];
            load_rows(Bv, a.Bm, tc, nb);
#pragma unroll 1
            for (int q = 0; q < QUADS; ++q) {
                const int cc = wave * 16 + q * 4 + ch4, at = cc * 16 + n;
                const float A2 = l_A[nb][at] * LOG2E;
                const float sv = t_s[token_at(cc, n)], uv = t_u[token_at(cc, n)];
                float h = start[c][nb][at];
                each_token([&](auto tt) {
                    constexpr int t = decltype(tt)::value;
                    h = __builtin_fmaf(fast_exp2(row_bcast<t>(sv) * A2), h, row_bcast<t>(uv) * Bv[t]);
                });
                start[c + 1][nb][at] = h;
            }
        }
        __syncthreads();
    }

    float dD = 0.f, db = 0.f;
    for (int c = nch - 1; c >= 0; --c) {
        const int tc = t0 + c * CHUNK;
        float x4[4], s4[4], u4[4], g4[4], ds4[4], dz4[4];   // ds4: ds/ddt; dz4: dy silu'(z)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = tc + 4 * wave + i;
            x4[i] = s4[i] = u4[i] = g4[i] = ds4[i] = dz4[i] = 0.f;
            if (ok && t < len) {   // idle lanes stay zero: their channel is another's
                const int64_t o = base + (int64_t)t * D;
                const float v = to_f32(((const T *)a.dt)[o]) + bias, dy = to_f32(((const T *)a.dy)[o]);
                x4[i] = to_f32(((const T *)a.x)[o]);
                s4[i] = a.softplus ? softplus_f32(v) : v;
                ds4[i] = a.softplus ? sigmoid_f32(v) : 1.f;
                u4[i] = s4[i] * x4[i];
                g4[i] = dy;
                if (a.z) {
                    const float z = to_f32(((const T *)a.z)[o]), sg = sigmoid_f32(z);
                    g4[i] = dy * z * sg;
                    dz4[i] = dy * sg * __builtin_fmaf(z, 1.f - sg, 1.f);
                }
            }
        }
        store4(t_s + piece(lane, wave), s4);
        store4(t_u + piece(lane, wave), u4);
        store4(t_g + piece(lane, wave), g4);
        __syncthreads();

        for (int nb = 0; nb < NB; ++nb) {
            float Bv[CHUNK], Cv[CHUNK], accB[CHUNK] = {}, accC[CHUNK] = {};
            load_rows(Bv, a.Bm, tc, nb);
            load_rows(Cv, a.Cm, tc, nb);
#pragma unroll 1
            for (int q = 0; q < QUADS; ++q) {
                const int cc = wave * 16 + q * 4 + ch4, at = cc * 16 + n, tok = token_at(cc, n);
                const float A = l_A[nb][at], A2 = A * LOG2E;
                const float sv = t_s[tok], uv = t_u[tok], gv = t_g[tok];
                float h = start[c][nb][at], g = l_g[nb][at], dA = l_dA[nb][at];
                float e[CHUNK], hp[CHUNK], v[CHUNK], v2[CHUNK];
                each_token([&](auto tt) {
                    constexpr int t = decltype(tt)::value;
                    e[t] = fast_exp2(row_bcast<t>(sv) * A2);
                    hp[t] = h;
                    h = __builtin_fmaf(e[t], h, row_bcast<t>(uv) * Bv[t]);
                    v[t] = h * Cv[t];
                    accC[t] = __builtin_fmaf(row_bcast<t>(gv), h, accC[t]);
                });
                float r = row_sum_tokens(v);
                each_token_back([&](auto tt) {
                    constexpr int t = decltype(tt)::value;
                    const float qt = __builtin_fmaf(row_bcast<t>(gv), Cv[t], g);
                    accB[t] = __builtin_fmaf(row_bcast<t>(uv), qt, accB[t]);
                    v[t] = qt * Bv[t];
                    g = e[t] * qt;
                    const float k = g * hp[t];
                    dA = __builtin_fmaf(row_bcast<t>(sv), k, dA);
                    v2[t] = A * k;
                });
                float p1 = row_sum_tokens(v), p2 = row_sum_tokens(v2);
                l_g[nb][at] = g;
                l_dA[nb][at] = dA;
                if (nb > 0) {
                    r += t_r[tok];
                    p1 += t_p1[tok];
                    p2 += t_p2[tok];
                }
                t_r[tok] = r;
                t_p1[tok] = p1;
                t_p2[tok] = p2;
            }
            // sums over the quad's four channels, tokens dealt out over the rows:
            // row 0 dB of tokens 0..7, row 1 of 8..15, rows 2 and 3 dC
            if (nb > 0) __syncthreads();   // the last block's sums have been read
            float k[CHUNK];
#pragma unroll
            for (int t = 0; t < CHUNK; ++t) {
                const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(accB[t]), __float_as_uint(accC[t]), false, false);
                k[t] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(k[t]), __float_as_uint(k[t + 8]), false, false);
                flush[wave][t][lane] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t8 = i * 4 + wave, t = tc + t8 + 8 * ((lane >> 4) & 1), st = nb * 16 + n;
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < WAVES; ++j) s += flush[j][t8][lane];
                if (t < a.T && st < N) {
                    float *p = lane < 32 ? w.dB : w.dC;
                    p[(int64_t)tile * a.B * a.T * row + row0 + t * row + st] = s;
                }
            }
        }

        float r4[4], p1[4], p2[4];
        Raw4<float> f;
        f.load(t_r + piece(lane, wave));
        f.to_f32(r4);
        f.load(t_p1 + piece(lane, wave));
        f.to_f32(p1);
        f.load(t_p2 + piece(lane, wave));
        f.to_f32(p2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = tc + 4 * wave + i;
            const float ddt = __builtin_fmaf(x4[i], p1[i], p2[i]) * ds4[i];
            dD = __builtin_fmaf(g4[i], x4[i], dD);
            db += ddt;
            if (ok && t < t1) {
                const int64_t o = base + (int64_t)t * D;
                ((T *)a.dx)[o] = from_f32<T>(__builtin_fmaf(s4[i], p1[i], skip * g4[i]));
                ((T *)a.ddt)[o] = from_f32<T>(ddt);
                if (a.dz) ((T *)a.dz)[o] = from_f32<T>(dz4[i] * __builtin_fmaf(skip, x4[i], r4[i]));
            }
        }
        // the next chunk's staging writes only what this chunk no longer reads
        // (t_s, t_u, t_g); its results wait behind the barrier after it
    }

    __syncthreads();
    for (int i = tid; i < NB * CH * 16; i += 256) {
        const int nb = i / (CH * 16), c = i / 16 % CH, st = nb * 16 + (i & 15);
        if (tile * CH + c < Dg && st < N)
            w.dA[(bseg * D + grp * Dg + tile * CH + c) * N + st] = l_dA[nb][i % (CH * 16)];
    }
    t_s[wave * 64 + lane] = dD;
    t_u[wave * 64 + lane] = db;
    __syncthreads();
    if (wave == 0 && ok) {
        float s = 0.f, u = 0.f;
#pragma unroll
        for (int j = 0; j < WAVES; ++j) {
            s += t_s[j * 64 + lane];
            u += t_u[j * 64 + lane];
        }
        w.dD[bseg * D + d] = s;
        w.db[bseg * D + d] = u;
    }
}

// Without tokens the state's gradient passes through.
__global__ void __launch_bounds__(256) kda_scan_bwd_pass_kernel(const float *in, float *out, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) out[i] = in ? in[i] : 0.f;
}

template <typename T, int NB> hipError_t run(const ScanBwdArgs &a, const Layout &w, hipStream_t s)
{
    const int seg = CHUNK * seg_chunks(NB);
    const int64_t blocks = (int64_t)a.B * w.nseg * a.G * w.tiles;
    const int64_t join = ((int64_t)a.B * a.D * w.np + 255) / 256;
    if (blocks >= ((int64_t)1 << 31) || join >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    kda_scan_bwd_segment_kernel<T, NB><<<(unsigned)blocks, 64, 0, s>>>(a, (const T *)a.Bm, (const T *)a.Cm, w, seg);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    kda_scan_bwd_join_kernel<<<(unsigned)join, 256, 0, s>>>(a, w);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    kda_scan_bwd_kernel<T, NB><<<(unsigned)blocks, 256, 0, s>>>(a, w);
    return hipGetLastError();
}

template <typename T> hipError_t dispatch(const ScanBwdArgs &a, const Layout &w, hipStream_t s)
{
    switch (state_blocks(a.N)) {
    case 1: return run<T, 1>(a, w, s);
    case 2: return run<T, 2>(a, w, s);
    default: return run<T, 4>(a, w, s);
    }
}

}  // namespace

int64_t scan_bwd_workspace_floats(int B, int T, int D, int N, int G) { return layout(nullptr, B, T, D, N, G).floats; }

hipError_t launch_scan_bwd(const ScanBwdArgs &a, hipStream_t s)
{
    (void)hipGetLastError();
    const Layout w = layout(a.ws, a.B, a.T, a.D, a.N, a.G);
    hipError_t e;
    if (a.B > 0 && a.T > 0) {
        e = a.bf16 ? dispatch<uint16_t>(a, w, s) : dispatch<float>(a, w, s);
        if (e != hipSuccess) return e;
    } else if (a.dh0 && a.B > 0) {
        const int64_t n = (int64_t)a.B * a.D * a.N, blocks = (n + 255) / 256;
        if (blocks >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
        kda_scan_bwd_pass_kernel<<<(unsigned)blocks, 256, 0, s>>>(a.dh_final, a.dh0, n);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t parts = (int64_t)a.B * w.nseg, DN = (int64_t)a.D * a.N, rows = (int64_t)a.B * a.T * a.G * a.N;
    const ColumnSum params[] = {{w.dA, a.dA, parts, DN, DN, false},
                                {w.dD, a.dDskip, parts, a.D, a.D, false},
                                {w.db, a.ddt_bias, parts, a.D, a.D, false}};
    if ((e = launch_column_sums(params, 3, s)) != hipSuccess) return e;
    const ColumnSum bc[] = {{w.dB, a.dBm, w.tiles, rows, rows, a.bf16}, {w.dC, a.dCm, w.tiles, rows, rows, a.bf16}};
    return launch_column_sums(bc, 2, s);
}

}  // namespace kda
