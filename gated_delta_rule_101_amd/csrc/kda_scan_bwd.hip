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
//  1. Segments of 32 to 256 tokens side by side, a quad of lanes a channel as in
//     the forward: the states it adds (from zero), stored at every chunk of 16 tokens, and,
//     with the running decay P_t = prod a, the gradient it adds in front of
//     itself, sum_t P_t C_t gy_t.  Both directions share each exp.
//  2. The true state in front of every segment and the true gradient behind it,
//     one thread per (d, n) over the segments.
//  3. The gradients.  A workgroup owns 64 channels and one segment, and walks
//     its chunks backwards (those behind the sequence's end only get zeros).
//     Here a lane owns ONE state of one channel (16 lanes a channel, 4 channels
//     a wavefront), so a chunk keeps its decays and states in registers between
//     its forward and its reverse walk, and the sums over channels of dB and dC
//     are plain accumulators while the wavefront goes through its channels.  The
//     sums over n (r, p1, p2) reduce 16 tokens over 16 lanes by a butterfly that
//     halves the values at each step (2 additions a value), leaving lane i with
//     token i.  Per-token values sit in a register that holds token i in lane i
//     and enter the arithmetic as DPP row
//     broadcasts, without instructions of their own.
//  4. Column sums of the workgroups' partial dA, dD, dbias, dB, dC.
// Bound by vector instructions, 26 per token, channel and state in kernel 3 and 10
// in kernel 1.  Measured: B4 T4096 D4096 N16 bfloat16 1.24 ms (kernels 1 to 4 under
// a trace, at lower clocks: 0.36, 0.015, 0.94 and 0.03).
#include "kda_block.h"
#include "kda_block_device.h"

namespace kda {
namespace {

constexpr int CHUNK = 16;        // tokens a chunk: one per lane of a DPP row
constexpr int CH = 64;           // channels a workgroup
constexpr int WAVES = 4, QUADS = CH / WAVES / 4;


int state_blocks(int N) { return N <= 16 ? 1 : N <= 32 ? 2 : 4; }   // of 16

// Workspace, in floats.
struct Layout {
    int seg, nseg, nchunk;           // tokens a segment; segments, chunks
    int tiles, np;                   // 64-channel tiles a group, room for the states (16, 32 or 64)
    float *h, *g, *sum;              // [B][nseg][D][np] states in front / gradients behind; [B][nseg][D]
    float *hc, *sc;                  // [B][nchunk][D][np] states a segment adds up to a chunk; [B][nchunk][D]
    float *dA, *dD, *db;             // [B nseg][D][N], [B nseg][D] twice
    float *dB, *dC;                  // [tiles][B][T][G][N]
    int64_t floats;
};
Layout layout(float *p, int B, int T, int D, int N, int G)
{
    Layout w;
    w.tiles = (D / G + CH - 1) / CH;
    // Segments of 256 tokens, halved down to 32 where there would be under 2048 of
    // them (two workgroups a compute unit, several rounds).
    w.seg = 256;
    while (w.seg > 32 && (int64_t)B * ((T + w.seg - 1) / w.seg) * G * w.tiles < 2048) w.seg /= 2;
    w.nseg = (T + w.seg - 1) / w.seg;
    w.nchunk = (T + CHUNK - 1) / CHUNK;
    w.np = 16 * state_blocks(N);
    const auto r4 = [](int64_t n) { return (n + 3) / 4 * 4; };   // 16-byte aligned parts
    const int64_t bs = (int64_t)B * w.nseg;
    const int64_t state = bs * D * w.np, chan = r4(bs * D), rows = r4((int64_t)w.tiles * B * T * G * N);
    const int64_t a = r4(bs * D * N);
    int64_t o = 0;
    const auto take = [&](int64_t n) { float *q = p ? p + o : nullptr; o += n; return q; };
    w.h = take(state);
    w.g = take(state);
    w.sum = take(chan);
    w.hc = take((int64_t)B * w.nchunk * D * w.np);
    w.sc = take(r4((int64_t)B * w.nchunk * D));
    w.dA = take(a);
    w.dD = take(chan);
    w.db = take(chan);
    w.dB = take(rows);
    w.dC = take(rows);
    w.floats = o;
    return w;
}

// --------------------------------------------------- 1. what a segment adds

// Lanes, staging and order as in the forward's kernel (kda_scan.hip).
template <typename T, int NB>
__global__ void __launch_bounds__(256) kda_scan_bwd_segment_kernel(ScanBwdArgs a, Layout w)
{
    constexpr int NP = 16 * NB;
    static_assert(CH * 4 == 256, "a quad per channel");
    __shared__ __attribute__((aligned(16))) float rows[2][2][CHUNK * NP];   // [buffer][B, C][token][state]
    const int tid = threadIdx.x, j = tid & 3, n0 = 4 * j;   // lane of the quad; its first state of each 16
    unsigned id = blockIdx.x;
    const int tile = id % w.tiles;
    id /= w.tiles;
    const int grp = id % a.G;
    id /= a.G;
    const int seg = id % w.nseg, b = id / w.nseg;
    const int D = a.D, N = a.N, Dg = D / a.G;
    const int c = tile * CH + tid / 4;
    const bool ok = c < Dg;
    const int d = grp * Dg + (ok ? c : Dg - 1);   // idle lanes repeat the last channel
    const int len = seq_length(a.lengths, b, a.T);
    const int t0 = seg * w.seg, t1 = min(t0 + w.seg, a.T), te = min(t1, len);

    float A2[NB][4], h[NB][4], r[NB][4], P[NB][4];   // states n0 + 16 m + n
#pragma unroll
    for (int m = 0; m < NB; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int st = n0 + 16 * m + n;
            A2[m][n] = st < N ? finite_rate(a.A[(int64_t)d * N + st]) * LOG2E : 0.f;
            h[m][n] = r[m][n] = 0.f;
            P[m][n] = 1.f;
        }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const bool gated = a.z != nullptr, soft = a.softplus;   // without a gate z reads x, unused
    const int64_t base = (int64_t)b * a.T * D;
    const T *xb = (const T *)a.x + base, *tb = (const T *)a.dt + base, *gb = (const T *)a.dy + base;
    const T *zb = (const T *)(gated ? a.z : a.x) + base;
    const unsigned dl = (unsigned)d * sizeof(T), rb = (unsigned)D * sizeof(T);   // lane, row: bytes
    unsigned off[4];   // of the lane's tokens in a chunk
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i] = (unsigned)(4 * i + j) * rb + dl;
    const int64_t row = (int64_t)a.G * N, row0 = ((int64_t)b * a.T * a.G + grp) * N;
    const int rt = tid / 16, rn = tid & 15;   // staging of B and C: token, state of a block

    float sum = 0.f;   // of this lane's tokens
    const auto quad_sum = [&] { return quad_add<0xB1>(quad_add<0x4E>(sum)); };
    const auto store_chunk = [&](int tc, float s) {   // a segment's first chunk has nothing in front of it
        if (tc > t0 && ok) {
            const int64_t at = ((int64_t)b * w.nchunk + tc / CHUNK) * D + d;
#pragma unroll
            for (int m = 0; m < NB; ++m) store4(w.hc + at * NP + 16 * m + n0, h[m]);
            if (j == 0) w.sc[at] = s;
        }
    };
    T xr[4], tr[4], gr[4], zr[4], Br[NB], Cr[NB];
    const auto fetch = [&](int tc) {      // tokens past the end: the last one again, masked later
        const int tf = min(tc, te - 1);
        const int64_t at = (int64_t)tf * D;
        const Rows<T> xs(xb + at), ts(tb + at), gs(gb + at), zs(zb + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned o = tf + CHUNK <= te ? off[i] : (unsigned)min(4 * i + j, te - 1 - tf) * rb + dl;
            xr[i] = xs.load(o, 0);
            tr[i] = ts.load(o, 0);
            gr[i] = gs.load(o, 0);
            zr[i] = zs.load(o, 0);
        }
        const int64_t o = row0 + (int64_t)min(tc + rt, te - 1) * row;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int st = min(16 * nb + rn, N - 1);
            Br[nb] = ((const T *)a.Bm)[o + st];
            Cr[nb] = ((const T *)a.Cm)[o + st];
        }
    };
    if (t0 < te) fetch(t0);
    int tc = t0;
    for (; tc < te; tc += CHUNK) {
        store_chunk(tc, quad_sum());
        float (&Bs)[CHUNK * NP] = rows[(tc / CHUNK) & 1][0], (&Cs)[CHUNK * NP] = rows[(tc / CHUNK) & 1][1];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const bool in = 16 * nb + rn < N && tc + rt < te;
            Bs[rt * NP + 16 * nb + rn] = in ? to_f32(Br[nb]) : 0.f;
            Cs[rt * NP + 16 * nb + rn] = in ? to_f32(Cr[nb]) : 0.f;
        }
        float s[4], u[4], gy[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = to_f32(tr[i]) + bias, sp = softplus_f32(v), z = to_f32(zr[i]);
            const bool in = tc + 4 * i + j < te;   // behind the end: a token that changes nothing
            s[i] = in ? (soft ? sp : v) : 0.f;
            u[i] = in ? s[i] * to_f32(xr[i]) : 0.f;
            gy[i] = in ? to_f32(gr[i]) * (gated ? z * sigmoid_f32(z) : 1.f) : 0.f;
            sum += s[i];
        }
        // one barrier a chunk: the buffer written next was last read a chunk earlier
        lds_barrier();
        fetch(tc + CHUNK);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int m = 0; m < NB; ++m) {
                float4 Bv[4], Cv[4];
                float e[4][4];
                const int at = 4 * i * NP + 16 * m + n0;
#pragma unroll
                for (int k = 0; k < 4; ++k) Bv[k] = *reinterpret_cast<const float4 *>(Bs + at + k * NP);
#pragma unroll
                for (int k = 0; k < 4; ++k) Cv[k] = *reinterpret_cast<const float4 *>(Cs + at + k * NP);
                each4([&](auto k) {
                    constexpr int K = decltype(k)::value;
#pragma unroll
                    for (int n = 0; n < 4; ++n) e[K][n] = quad_bcast<K>(s[i]) * A2[m][n];
                });
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < 4; ++n) e[k][n] = fast_exp2(e[k][n]);
                __builtin_amdgcn_sched_barrier(0);
                each4([&](auto k) {
                    constexpr int K = decltype(k)::value;
                    const float ub[4] = {quad_bcast<K>(u[i]) * Bv[K].x, quad_bcast<K>(u[i]) * Bv[K].y,
                                         quad_bcast<K>(u[i]) * Bv[K].z, quad_bcast<K>(u[i]) * Bv[K].w};
                    const float gc[4] = {quad_bcast<K>(gy[i]) * Cv[K].x, quad_bcast<K>(gy[i]) * Cv[K].y,
                                         quad_bcast<K>(gy[i]) * Cv[K].z, quad_bcast<K>(gy[i]) * Cv[K].w};
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        h[m][n] = __builtin_fmaf(e[K][n], h[m][n], ub[n]);
                        P[m][n] *= e[K][n];
                        r[m][n] = __builtin_fmaf(P[m][n], gc[n], r[m][n]);
                    }
                });
            }
        }
    }
    sum = quad_sum();
    for (; tc < t1; tc += CHUNK) store_chunk(tc, sum);
    if (!ok) return;
    const int64_t at = ((int64_t)b * w.nseg + seg) * D + d;
#pragma unroll
    for (int m = 0; m < NB; ++m) {
        store4(w.h + at * NP + 16 * m + n0, h[m]);
        store4(w.g + at * NP + 16 * m + n0, r[m]);
    }
    if (j == 0) w.sum[at] = sum;
}

// --------------------------------- 2. states in front, gradients behind

// In place: h[seg] becomes the state in front of segment seg, g[seg] the
// gradient behind it.  A segment's decay is exp(A sum s).  A thread walks one
// (sequence, channel, state) in one direction, the loads of JOIN segments out
// together and a batch ahead of the chain.
constexpr int JOIN = 8;
template <bool BACK>
__device__ __forceinline__ float join_walk(float *p, const float *sums, int64_t per, int64_t D, int nseg, float A2, float v)
{
    const auto at = [&](int i) { return BACK ? nseg - 1 - i : i; };
    float add[JOIN], s[JOIN];
    const auto fetch = [&](int i0) {
#pragma unroll
        for (int k = 0; k < JOIN; ++k) {
            const int seg = at(min(i0 + k, nseg - 1));
            add[k] = p[seg * per];
            s[k] = sums[seg * D];
        }
    };
    fetch(0);
    for (int i = 0; i < nseg; i += JOIN) {
        float e[JOIN], a[JOIN];
#pragma unroll
        for (int k = 0; k < JOIN; ++k) {
            e[k] = fast_exp2(A2 * s[k]);
            a[k] = add[k];
        }
        if (i + JOIN < nseg) fetch(i + JOIN);
#pragma unroll
        for (int k = 0; k < JOIN; ++k)
            if (i + k < nseg) {
                p[at(i + k) * per] = v;
                v = __builtin_fmaf(e[k], v, a[k]);
            }
    }
    return v;
}

__global__ void __launch_bounds__(256) kda_scan_bwd_join_kernel(ScanBwdArgs a, Layout w)
{
    const int64_t id = (int64_t)(blockIdx.x >> 1) * 256 + threadIdx.x;
    const int64_t per = (int64_t)a.D * w.np;
    if (id >= a.B * per) return;
    const int b = (int)(id / per);
    const int64_t dn = id % per;
    const int d = (int)(dn / w.np), n = (int)(dn % w.np);
    const bool in = n < a.N;
    const float A2 = in ? finite_rate(a.A[(int64_t)d * a.N + n]) * LOG2E : 0.f;
    const int64_t st = ((int64_t)b * a.D + d) * a.N + n, first = (int64_t)b * w.nseg * per + dn;
    const float *sums = w.sum + (int64_t)b * w.nseg * a.D + d;
    if (blockIdx.x & 1) {
        const float g = join_walk<true>(w.g + first, sums, per, a.D, w.nseg, A2, in && a.dh_final ? a.dh_final[st] : 0.f);
        if (in && a.dh0) a.dh0[st] = g;
    } else {
        join_walk<false>(w.h + first, sums, per, a.D, w.nseg, A2, in && a.h0 ? a.h0[st] : 0.f);
    }
}

// ------------------------------------------------------- 3. the gradients

// Sums v[t] over the 16 lanes of each DPP row for 16 tokens t at once; lane i
// returns token i's sum.  Each step adds a partner lane's half of the values
// to the own half: lanes 8..15 keep tokens 8..15, then lanes with bit 2 set
// the upper four, and so on.
//
// A DPP source must not come from a vector instruction within the two before.
// The compiler keeps that rule for its own instructions but does not look into
// assembly, hence the s_nop in front of each block (its inputs) and behind the
// last (its outputs).
template <int CTRL> __device__ __forceinline__ float add_partner(float x)
{
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ void row_sum_halves(float (&b)[4], const float (&v)[16])
{
    float a[8];
    // a[i]: v[i] of lanes l and l ^ 8 in lanes 0..7, v[i + 8] in lanes 8..15
#define KDA_ROR8(i, j) "v_add_f32_dpp %" #i ", %" #j ", %" #j " row_ror:8 row_mask:0xf bank_mask:0xf\n"
#define KDA_ROR8H(i, j) "v_add_f32_dpp %" #i ", %" #j ", %" #j " row_ror:8 row_mask:0xf bank_mask:0xc\n"
    asm("s_nop 1\n" KDA_ROR8(0, 8) KDA_ROR8(1, 9) KDA_ROR8(2, 10) KDA_ROR8(3, 11) KDA_ROR8(4, 12) KDA_ROR8(5, 13)
        KDA_ROR8(6, 14) KDA_ROR8(7, 15) KDA_ROR8H(0, 16) KDA_ROR8H(1, 17) KDA_ROR8H(2, 18) KDA_ROR8H(3, 19)
        KDA_ROR8H(4, 20) KDA_ROR8H(5, 21) KDA_ROR8H(6, 22) KDA_ROR8H(7, 23)
        : "=&v"(a[0]), "=&v"(a[1]), "=&v"(a[2]), "=&v"(a[3]), "=&v"(a[4]), "=&v"(a[5]), "=&v"(a[6]), "=&v"(a[7])
        : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]), "v"(v[8]),
          "v"(v[9]), "v"(v[10]), "v"(v[11]), "v"(v[12]), "v"(v[13]), "v"(v[14]), "v"(v[15]));
#undef KDA_ROR8
#undef KDA_ROR8H
    // b[i]: lanes without bit 2 add lane l + 4 of a[i], lanes with it lane l - 4 of a[i + 4]
#define KDA_SHL4(i, j) "v_add_f32_dpp %" #i ", %" #j ", %" #j " row_shl:4 row_mask:0xf bank_mask:0x5\n"
#define KDA_SHR4(i, j) "v_add_f32_dpp %" #i ", %" #j ", %" #j " row_shr:4 row_mask:0xf bank_mask:0xa\n"
    asm("s_nop 1\n" KDA_SHL4(0, 4) KDA_SHL4(1, 5) KDA_SHL4(2, 6) KDA_SHL4(3, 7) KDA_SHR4(0, 8) KDA_SHR4(1, 9)
        KDA_SHR4(2, 10) KDA_SHR4(3, 11) "s_nop 1"
        : "=&v"(b[0]), "=&v"(b[1]), "=&v"(b[2]), "=&v"(b[3])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(a[4]), "v"(a[5]), "v"(a[6]), "v"(a[7]));
#undef KDA_SHL4
#undef KDA_SHR4
}
// The last two steps, of three sums in turn: each has instructions of the others
// between one that writes and the DPP that reads it.
__device__ __forceinline__ void row_sum_quads(const float (&x)[4], const float (&y)[4], const float (&z)[4], float &sx,
                                              float &sy, float &sz)
{
    constexpr int SWAP2 = 0x4E, SWAP1 = 0xB1;   // quad_perm [2,3,0,1], [1,0,3,2]
    const bool up2 = threadIdx.x & 2, up1 = threadIdx.x & 1;
    const float x0 = add_partner<SWAP2>(x[0]), x1 = add_partner<SWAP2>(x[1]), x2 = add_partner<SWAP2>(x[2]), x3 = add_partner<SWAP2>(x[3]);
    const float y0 = add_partner<SWAP2>(y[0]), y1 = add_partner<SWAP2>(y[1]), y2 = add_partner<SWAP2>(y[2]), y3 = add_partner<SWAP2>(y[3]);
    const float z0 = add_partner<SWAP2>(z[0]), z1 = add_partner<SWAP2>(z[1]), z2 = add_partner<SWAP2>(z[2]), z3 = add_partner<SWAP2>(z[3]);
    const float xa = up2 ? x2 : x0, xb = up2 ? x3 : x1;
    const float ya = up2 ? y2 : y0, yb = up2 ? y3 : y1;
    const float za = up2 ? z2 : z0, zb = up2 ? z3 : z1;
    const float xp = add_partner<SWAP1>(xa), xq = add_partner<SWAP1>(xb);
    const float yp = add_partner<SWAP1>(ya), yq = add_partner<SWAP1>(yb);
    const float zp = add_partner<SWAP1>(za), zq = add_partner<SWAP1>(zb);
    sx = up1 ? xq : xp;
    sy = up1 ? yq : yp;
    sz = up1 ? zq : zp;
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

// acc += (row's lane t of x) * y.  The DPP source x must not come from a
// vector instruction within the two before: callers pass values read from LDS.
template <int t> __device__ __forceinline__ void fma_bcast(float &acc, float x, float y)
{
    asm("v_fmac_f32_dpp %0, %1, %2 row_newbcast:%3 row_mask:0xf bank_mask:0xf" : "+v"(acc) : "v"(x), "v"(y), "i"(t));
}

// [channel][16 tokens] tiles in LDS.  Threads that stage and finish tokens
// access 4 tokens of one channel (16 bytes), 64 channels a wavefront; those
// that compute access 4 channels' 16 tokens.  The 4-token pieces of a channel
// are permuted by its index so that neither has bank conflicts.
__device__ __forceinline__ int piece(int ch, int p) { return ch * 16 + 4 * (p ^ ((ch >> 2) & 3)); }
__device__ __forceinline__ int token_at(int ch, int t) { return piece(ch, t >> 2) + (t & 3); }

// A workgroup's tiles in LDS, arrays of their own (of one struct's parts the
// compiler cannot tell that they do not overlap).
template <int NB> struct Tiles {
    float (&s)[CH * 16], (&u)[CH * 16], (&g)[CH * 16];             // s, s x, gy
    float (&r)[CH * 16], (&p1)[CH * 16], (&p2)[CH * 16];
    float (&B)[NB][CHUNK * 16], (&C)[NB][CHUNK * 16];              // [token][16 states]
    float (&h)[NB][CH * 16];                                       // state in front of the chunk
    float (&A)[NB][CH * 16], (&gb)[NB][CH * 16], (&dA)[NB][CH * 16];   // [channel][16 states]; gb: gradient behind it
    float (&flush)[WAVES][8][64];                                  // dB, dC of a chunk, per wavefront
};

// One segment of a tile's channels.  TAIL: it has places behind the sequence's last
// token.  Chunks of such places only get zeros.  In the chunk of the last token
// they carry on a state and a gradient that may be infinite, so what they would
// add is chosen to be 0 and not multiplied by 0.
//
// FILL: N is below NP, and states have several places (see Places).  Here the
// gradients of the states, linear in C and in the gradient behind the segment,
// carry the places' shares: with both times the share, the sums over places of
// r, p1 and p2 are those over states, and dA, dB and dh0 of a place are divided
// by it again.
template <typename T, int NB, bool TAIL, bool FILL>
__device__ __forceinline__ void bwd_segment(const ScanBwdArgs &a, const Layout &w, const Tiles<NB> &m, int tile, int grp,
                                            int seg, int b)
{
    static_assert(QUADS == 4 && WAVES * QUADS * 4 == CH, "a wavefront's channels");
    static_assert(CHUNK == 16, "a token per lane of a DPP row");
    auto &t_s = m.s, &t_u = m.u, &t_g = m.g, &t_r = m.r, &t_p1 = m.p1, &t_p2 = m.p2;
    auto &t_B = m.B, &t_C = m.C;
    auto &l_h = m.h, &l_A = m.A, &l_g = m.gb, &l_dA = m.dA;
    auto &flush = m.flush;

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid & 63;
    const int ch4 = lane / 16, n = lane & 15;             // compute: channel of the quad, state or token
    const int D = a.D, N = a.N, Dg = D / a.G;
    const int len = seq_length(a.lengths, b, a.T);
    const int t0 = seg * w.seg, t1 = min(t0 + w.seg, a.T), nch = (t1 - t0 + CHUNK - 1) / CHUNK;
    const int64_t bseg = (int64_t)b * w.nseg + seg;

    // staging role: channel `lane` of the tile, tokens 4 wave .. 4 wave + 3 of a
    // chunk; and token tid / 16, state tid % 16 of B and C
    const bool ok = tile * CH + lane < Dg;
    const int d = grp * Dg + (ok ? tile * CH + lane : Dg - 1);
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f, skip = a.Dskip ? a.Dskip[d] : 0.f;
    // without a gate z reads x, unused; without a skip nothing is added, not 0 times something
    const bool gated = a.z != nullptr, skips = a.Dskip != nullptr, soft = a.softplus;
    const int64_t base = (int64_t)b * a.T * D;              // uniform; a lane adds its channel
    const T *xb = (const T *)a.x + base, *tb = (const T *)a.dt + base, *gb = (const T *)a.dy + base;
    const T *zb = (const T *)(gated ? a.z : a.x) + base;
    T *dxb = (T *)a.dx + base, *dtb = (T *)a.ddt + base, *dzb = (T *)a.dz + base;
    const unsigned dl = (unsigned)d * sizeof(T), rb = (unsigned)D * sizeof(T);   // lane, row: bytes
    const int64_t row0 = ((int64_t)b * a.T * a.G + grp) * N, row = (int64_t)a.G * N;

    // Slots of the [channel][16] tiles: slot k of a thread is element k 256 + tid.
    // Channels behind the group's last read it, but hold states and gradients of 0
    // (0 times infinite ones would make NaN of dB and dC).
    constexpr int SLOTS = NB * CH * 16 / 256, NP = 16 * NB;
    const int c0 = grp * Dg + tile * CH, cmax = Dg - 1 - tile * CH;   // the tile's first channel; last one in it
    const auto chan = [&](int k) { return (unsigned)min((k * 256 + tid) / 16 % CH, cmax); };
    const auto live = [&](int k) { return (k * 256 + tid) / 16 % CH <= cmax; };
    const Places<FILL> places(N, NP);
    const auto place = [&](int k) { return (k * 256 + tid) / (CH * 16) * 16 + (tid & 15); };
    const auto state = [&](int k) { return (unsigned)places.state(place(k)); };
    const bool joined = w.nchunk > 1;   // otherwise the segment is the sequence, and its chunk the only one
    const auto seg_start = [&](int k) -> float {   // state in front of the segment
        const unsigned c = chan(k), st = state(k);
        if (joined) return w.h[(bseg * D + c0 + c) * NP + st];
        return a.h0 ? a.h0[((int64_t)b * D + c0 + c) * N + st] : 0.f;
    };
    // one block of states keeps its segment's start in registers and loads the
    // chunks' a chunk ahead; more of them would cost a wavefront a SIMD
    constexpr bool AHEAD = NB == 1;
    float h_seg[AHEAD ? SLOTS : 1], hr[AHEAD ? SLOTS : 1], sr[AHEAD ? SLOTS : 1];
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
        const unsigned c = chan(k), st = state(k);
        const int64_t own = ((int64_t)b * D + c0 + c) * N + st;   // in dh_final
        const float behind = joined ? w.g[(bseg * D + c0 + c) * NP + st] : a.dh_final ? a.dh_final[own] : 0.f;
        (&l_A[0][0])[k * 256 + tid] = finite_rate(a.A[(int64_t)(c0 + c) * N + st]);
        (&l_g[0][0])[k * 256 + tid] = live(k) ? behind * places.share(place(k)) : 0.f;
        (&l_dA[0][0])[k * 256 + tid] = 0.f;
        if constexpr (AHEAD) h_seg[k] = seg_start(k);
    }
    // dB and dC of token 8 (row & 1) of a chunk's first wave-share, this lane's state
    float *const dBC = (lane < 32 ? w.dB : w.dC) + (int64_t)tile * a.B * a.T * row + row0 + 8 * ((lane >> 4) & 1) * row + n;

    // raw inputs of one chunk, loaded a chunk ahead
    T xr[4], tr[4], gr[4], zr[4], Br[NB], Cr[NB];
    const auto fetch = [&](int c) {
        const int tc = t0 + c * CHUNK;
        const int tf = max(min(tc + 4 * wave, len - 1), 0);   // past the end: the last token, masked later
        const int64_t rf = (int64_t)tf * D;
        const Rows<T> xs(xb + rf), ts(tb + rf), gs(gb + rf), zs(zb + rf);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned o = (unsigned)max(min(i, len - 1 - tf), 0) * rb;
            xr[i] = xs.load(dl, o);
            tr[i] = ts.load(dl, o);
            gr[i] = gs.load(dl, o);
            zr[i] = zs.load(dl, o);
        }
        __builtin_amdgcn_sched_barrier(0);   // the order in which they are used
        const int tr0 = max(min(tc, len - 1), 0);
        const T *Bp = (const T *)a.Bm + row0 + tr0 * row, *Cp = (const T *)a.Cm + row0 + tr0 * row;
        const unsigned o = (unsigned)max(min(tid / 16, len - 1 - tr0), 0) * (unsigned)row;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const unsigned st = places.state(nb * 16 + (tid & 15));
            Br[nb] = Bp[o + st];
            Cr[nb] = Cp[o + st];
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (AHEAD) {   // (the segment's first chunk has nothing in front of it: its values go unused)
            const int64_t at = ((int64_t)b * w.nchunk + tc / CHUNK) * D + c0;
            const float *hp = w.hc + at * NP, *sp = w.sc + at;
#pragma unroll
            for (int k = 0; k < SLOTS; ++k) {
                hr[k] = hp[chan(k) * NP + state(k)];
                sr[k] = sp[chan(k)];
            }
        }
    };
    const int own = TAIL ? max((min(t1, len) - t0 + CHUNK - 1) / CHUNK, 0) : nch;   // chunks with tokens
    if constexpr (TAIL)
        for (int c = own; c < nch; ++c) {
            const int tc = t0 + c * CHUNK;
            const int64_t rw = (int64_t)(tc + 4 * wave) * D;
            const Rows<T> dxs(dxb + rw), dts(dtb + rw), dzs(dzb + rw);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (ok && tc + 4 * wave + i < t1) {
                    dxs.store(from_f32<T>(0.f), dl, i * rb);
                    dts.store(from_f32<T>(0.f), dl, i * rb);
                    if (gated) dzs.store(from_f32<T>(0.f), dl, i * rb);
                }
            for (int k = 0; k < 2 * NB; ++k) {
                const int t8 = (k & 1) * 4 + wave, st = k / 2 * 16;
                if (tc + t8 + 8 * ((lane >> 4) & 1) < t1 && st + n < N) dBC[(tc + t8) * row + st] = 0.f;
            }
        }
    fetch(max(own - 1, 0));

    float dD = 0.f, db = 0.f;
    for (int c = own - 1; c >= 0; --c) {
        const int tc = t0 + c * CHUNK, nv = TAIL ? len - tc : CHUNK;   // first token; how many are the sequence's
        float x4[4], s4[4], u4[4], g4[4], ds4[4], dz4[4];   // ds4: ds/ddt; dz4: dy silu'(z)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = ok && 4 * wave + i < nv;   // idle lanes stay zero: their channel is another's
            const float v = to_f32(tr[i]) + bias, dy = in ? to_f32(gr[i]) : 0.f, z = in ? to_f32(zr[i]) : 0.f;
            const float sg = sigmoid_f32(z), sp = softplus_f32(v), sv = sigmoid_f32(v);
            x4[i] = in ? to_f32(xr[i]) : 0.f;
            s4[i] = in ? (soft ? sp : v) : 0.f;
            ds4[i] = in ? (soft ? sv : 1.f) : 0.f;
            u4[i] = s4[i] * x4[i];
            g4[i] = dy * (gated ? z * sg : 1.f);
            dz4[i] = dy * (sg * __builtin_fmaf(z, 1.f - sg, 1.f));
        }
        store4(t_s + piece(lane, wave), s4);
        store4(t_u + piece(lane, wave), u4);
        store4(t_g + piece(lane, wave), g4);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const bool in = tid / 16 < nv;
            t_B[nb][tid] = in ? to_f32(Br[nb]) : 0.f;
            t_C[nb][tid] = in ? to_f32(Cr[nb]) * places.share(nb * 16 + (tid & 15)) : 0.f;
        }
        // a chunk's start: what the segment added so far, and the rest of its own start
        const int64_t ca = ((int64_t)b * w.nchunk + tc / CHUNK) * D + c0;
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) {
            float start, add = 0.f, sum = 0.f;
            if constexpr (AHEAD) {
                start = h_seg[k];
                add = hr[k];
                sum = sr[k];
            } else {
                start = seg_start(k);
                if (c > 0) {
                    add = w.hc[(ca + chan(k)) * NP + state(k)];
                    sum = w.sc[ca + chan(k)];
                }
            }
            const float A2 = (&l_A[0][0])[k * 256 + tid] * LOG2E;
            const float front = c > 0 ? __builtin_fmaf(fast_exp2(A2 * sum), start, add) : start;
            (&l_h[0][0])[k * 256 + tid] = live(k) ? front : 0.f;
        }
        __syncthreads();
        fetch(max(c - 1, 0));

#pragma unroll 1
        for (int nb = 0; nb < NB; ++nb) {
            float Bv[CHUNK], Cv[CHUNK], accB[CHUNK] = {}, accC[CHUNK] = {};
#pragma unroll
            for (int t = 0; t < CHUNK; ++t) {
                Bv[t] = t_B[nb][t * 16 + n];
                Cv[t] = t_C[nb][t * 16 + n];
            }
#pragma unroll 1
            for (int q = 0; q < QUADS; ++q) {
                const int cc = wave * 16 + q * 4 + ch4, at = cc * 16 + n, tok = token_at(cc, n);
                const float A = l_A[nb][at], A2 = A * LOG2E;
                const float sv = t_s[tok], uv = t_u[tok], gv = t_g[tok];
                float h = l_h[nb][at], g = l_g[nb][at], dA = l_dA[nb][at];
                __builtin_amdgcn_sched_barrier(0);   // all reads out here, not in front of their uses
                float e[CHUNK], hp[CHUNK], v[CHUNK], v2[CHUNK];
                each_token([&](auto tt) {
                    constexpr int t = decltype(tt)::value;
                    e[t] = fast_exp2(row_bcast<t>(sv) * A2);
                    hp[t] = h;
                    h = __builtin_fmaf(e[t], h, row_bcast<t>(uv) * Bv[t]);
                    v[t] = h * Cv[t];
                    fma_bcast<t>(accC[t], gv, h);
                });
                float rh[4], p1h[4], p2h[4], r, p1, p2;
                row_sum_halves(rh, v);
                each_token_back([&](auto tt) {
                    constexpr int t = decltype(tt)::value;
                    fma_bcast<t>(g, gv, Cv[t]);          // q_t
                    fma_bcast<t>(accB[t], uv, g);
                    v[t] = g * Bv[t];
                    g *= e[t];                           // g_t
                    const float k = TAIL && t >= nv ? 0.f : g * hp[t];
                    fma_bcast<t>(dA, sv, k);
                    v2[t] = A * k;
                });
                row_sum_halves(p1h, v);
                row_sum_halves(p2h, v2);
                row_sum_quads(rh, p1h, p2h, r, p1, p2);
                l_g[nb][at] = g;
                l_dA[nb][at] = dA;
                if (NB > 1 && nb > 0) {
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
            if (NB > 1 && nb > 0) __syncthreads();   // the last block's sums have been read
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
                const int t8 = i * 4 + wave;
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < WAVES; ++j) s += flush[j][t8][lane];
                const int t = t8 + 8 * ((lane >> 4) & 1);
                if (FILL && lane < 32) s *= places.places_of(nb * 16 + n);   // dB
                if ((!TAIL || tc + t < a.T) && (!FILL || nb * 16 + n < N)) dBC[(tc + t8) * row + nb * 16] = t < nv ? s : 0.f;
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
        const int64_t rw = (int64_t)(tc + 4 * wave) * D;
        const Rows<T> dxs(dxb + rw), dts(dtb + rw), dzs(dzb + rw);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = 4 * wave + i < nv;
            const float ddt = in ? __builtin_fmaf(x4[i], p1[i], p2[i]) * ds4[i] : 0.f;
            const float dx = in ? __builtin_fmaf(s4[i], p1[i], skips ? skip * g4[i] : 0.f) : 0.f;
            const float dz = in ? dz4[i] * (skips ? __builtin_fmaf(skip, x4[i], r4[i]) : r4[i]) : 0.f;
            dD = __builtin_fmaf(g4[i], x4[i], dD);
            db += ddt;
            if (ok && (!TAIL || tc + 4 * wave + i < t1)) {
                dxs.store(from_f32<T>(dx), dl, i * rb);
                dts.store(from_f32<T>(ddt), dl, i * rb);
                if (gated) dzs.store(from_f32<T>(dz), dl, i * rb);
            }
        }
        // the next chunk's staging writes only what no wavefront reads any more
        // (t_s, t_u, t_g, t_B, t_C, l_h); its results wait behind the next barrier
    }

    __syncthreads();
    for (int i = tid; i < NB * CH * 16; i += 256) {
        const int nb = i / (CH * 16), c = i / 16 % CH, st = nb * 16 + (i & 15);
        if (tile * CH + c < Dg && (!FILL || st < N)) {
            const float f = places.places_of(st);
            w.dA[(bseg * D + grp * Dg + tile * CH + c) * N + st] = l_dA[nb][i % (CH * 16)] * f;
            if (a.dh0 && w.nchunk == 1) a.dh0[((int64_t)b * D + grp * Dg + tile * CH + c) * N + st] = l_g[nb][i % (CH * 16)] * f;
        }
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

template <typename T, int NB, bool FILL>
__global__ void __launch_bounds__(256, NB <= 2 ? 2 : 1) kda_scan_bwd_kernel(ScanBwdArgs a, Layout w)
{
    __shared__ __attribute__((aligned(16))) float t_s[CH * 16], t_u[CH * 16], t_g[CH * 16];
    __shared__ __attribute__((aligned(16))) float t_r[CH * 16], t_p1[CH * 16], t_p2[CH * 16];
    __shared__ float t_B[NB][CHUNK * 16], t_C[NB][CHUNK * 16];
    __shared__ float l_h[NB][CH * 16];
    __shared__ float l_A[NB][CH * 16], l_g[NB][CH * 16], l_dA[NB][CH * 16];
    __shared__ float flush[WAVES][8][64];
    const Tiles<NB> m{t_s, t_u, t_g, t_r, t_p1, t_p2, t_B, t_C, l_h, l_A, l_g, l_dA, flush};
    unsigned id = blockIdx.x;
    const int tile = id % w.tiles;
    id /= w.tiles;
    const int grp = id % a.G;
    id /= a.G;
    const int seg = id % w.nseg, b = id / w.nseg;
    const int t0 = seg * w.seg, chunks = (min(w.seg, a.T - t0) + CHUNK - 1) / CHUNK;
    // (Two bodies: with the choices of the second in one, B4 T4096 D4096 N16 took 5% longer.)
    if (t0 + chunks * CHUNK <= seq_length(a.lengths, b, a.T)) bwd_segment<T, NB, false, FILL>(a, w, m, tile, grp, seg, b);
    else bwd_segment<T, NB, true, FILL>(a, w, m, tile, grp, seg, b);
}

// Without tokens the state's gradient passes through.
__global__ void __launch_bounds__(256) kda_scan_bwd_pass_kernel(const float *in, float *out, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) out[i] = in ? in[i] : 0.f;
}

template <typename T, int NB> hipError_t run(const ScanBwdArgs &a, const Layout &w, hipStream_t s)
{
    const int64_t blocks = (int64_t)a.B * w.nseg * a.G * w.tiles;
    const int64_t join = ((int64_t)a.B * a.D * w.np + 255) / 256 * 2;
    if (!grid_fits(blocks, 256) || !grid_fits(join, 256)) return hipErrorNotSupported;
    hipError_t e;
    if (w.nchunk > 1) {   // a single chunk has nothing in front of it or behind it
        kda_scan_bwd_segment_kernel<T, NB><<<(unsigned)blocks, 256, 0, s>>>(a, w);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        kda_scan_bwd_join_kernel<<<(unsigned)join, 256, 0, s>>>(a, w);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    (a.N == w.np ? kda_scan_bwd_kernel<T, NB, false> : kda_scan_bwd_kernel<T, NB, true>)<<<(unsigned)blocks, 256, 0, s>>>(a, w);
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
    const int64_t parts = (int64_t)a.B * w.nseg, DN = (int64_t)a.D * a.N, rows = (int64_t)a.B * a.T * a.G * a.N;
    const ColumnSum jobs[] = {{w.dA, a.dA, parts, DN, DN, false},
                              {w.dD, a.dDskip, parts, a.D, a.D, false},
                              {w.db, a.ddt_bias, parts, a.D, a.D, false},
                              {w.dB, a.dBm, w.tiles, rows, rows, a.bf16},
                              {w.dC, a.dCm, w.tiles, rows, rows, a.bf16}};
    if (!column_sums_fit(jobs, 5)) return hipErrorNotSupported;
    hipError_t e;
    if (a.B > 0 && a.T > 0) {
        e = a.bf16 ? dispatch<uint16_t>(a, w, s) : dispatch<float>(a, w, s);
        if (e != hipSuccess) return e;
    } else if (a.dh0 && a.B > 0) {
        const int64_t n = (int64_t)a.B * a.D * a.N, blocks = (n + 255) / 256;
        if (!grid_fits(blocks, 256)) return hipErrorNotSupported;
        kda_scan_bwd_pass_kernel<<<(unsigned)blocks, 256, 0, s>>>(a.dh_final, a.dh0, n);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return launch_column_sums(jobs, 5, s);
}

}  // namespace kda
