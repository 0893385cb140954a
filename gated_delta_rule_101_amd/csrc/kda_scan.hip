// Selective state space scan for gfx950, forward over a sequence and one token.
//
// Per channel d with N states (in NP = 16 NB places; where N is smaller, some states
// have more than one, see Places):
//   s = softplus(dt + bias),  h[n] <- exp(s A[n]) h[n] + s x B[n],
//   y = (sum_n C[n] h[n] + D x) silu(z)
//
// A quad of lanes owns a channel, lane j of it places 4 j .. 4 j + 3 of each 16
// in registers.  What a channel's token costs once
// (softplus, gate, conversions) is dealt out over the quad: lane j takes every
// fourth token and hands its s and s x to the others by DPP quad broadcasts,
// which ride on the multiplications, and the partial outputs of four tokens meet
// so that lane j keeps token j's.  B and C rows go through LDS as float32, CHUNK
// tokens at a time, read as one 16-byte broadcast per token and row.  A state
// costs 6 issue slots a token (multiply, exp2 at half rate, two products, two
// sums) and a channel's token about 14 slots a lane besides: the vector units
// bound it, not HBM.
//
// The recurrence is a chain over tokens, and few channels leave the device idle
// (B D / 16 wavefronts for 1024 SIMDs).  With a workspace the tokens are then
// cut into segments: a first pass runs all but the last from a zero state (the
// first from h0) and stores end states and sums of s, a second pass forms each
// segment's true starting state from those (the decay of a whole segment is
// exp(A sum s)) and runs it again with the outputs.
//
// Measured (bfloat16, N = 16): B4 T4096 D4096, one chain of 1024 wavefronts, 0.432
// ms (8.1 vector instructions a state and token; four wavefronts a SIMD would
// take 0.31); B1 T16384 D4096, 32 segments, 0.464 ms; one token of B256 D12288 0.076
// ms, 5.7 TB/s.
#include "kda_block.h"
#include "kda_block_device.h"

#include <algorithm>

namespace kda {
namespace {

constexpr int CHUNK = 16;

// Segments of the forward and their workspace: slot 0 is a copy of h0 (h_final
// may be h0 itself, and other wavefronts write it while segment 0 still
// starts), slot s the state at the end of segment s - 1, [B][count][D][NP], and
// sums[s] that segment's sum of time steps, [B][count][D].
struct Segments {
    int count, tokens;   // segments, tokens each (a multiple of CHUNK)
    float *slots, *sums;
};

// Sums of four values over a quad, lane j's the j-th: lanes with bit 1 keep values
// 2 and 3, then lanes with bit 0 the odd one (every lane takes part in both sums
// before it chooses).
__device__ __forceinline__ float quad_sums(const float (&y)[4])
{
    constexpr int SWAP2 = 0x4E, SWAP1 = 0xB1;   // quad_perm [2,3,0,1], [1,0,3,2]
    const int j = threadIdx.x & 3;
    const float a0 = quad_add<SWAP2>(y[0]), a1 = quad_add<SWAP2>(y[1]);
    const float a2 = quad_add<SWAP2>(y[2]), a3 = quad_add<SWAP2>(y[3]);
    const float p0 = j & 2 ? a2 : a0, p1 = j & 2 ? a3 : a1;
    const float q0 = quad_add<SWAP1>(p0), q1 = quad_add<SWAP1>(p1);
    return j & 1 ? q1 : q0;
}

template <typename T, int NB, bool STATES_ONLY, bool FILL>
__global__ void __launch_bounds__(256) kda_scan_kernel(ScanArgs a, Segments sg, int tiles)
{
    constexpr int NP = 16 * NB, CHANNELS = 64;
    __shared__ __attribute__((aligned(16))) float rows[2][2][CHUNK * NP];   // [buffer][B, C][token][place]
    const int tid = threadIdx.x, j = tid & 3, n0 = 4 * j;   // lane of the quad; its first place of each 16
    unsigned id = blockIdx.x;
    const int tile = id % tiles;
    id /= tiles;
    const int g = id % a.G;
    id /= a.G;
    const int runs = STATES_ONLY ? sg.count - 1 : sg.count;
    const int seg = id % runs, b = id / runs;
    const int D = a.D, N = a.N, Dg = D / a.G;
    const int c = tile * CHANNELS + tid / 4;
    const bool ok = c < Dg;
    const int d = g * Dg + (ok ? c : Dg - 1);   // idle lanes repeat the last channel
    const int len = seq_length(a.lengths, b, a.T);
    const int t0 = seg * sg.tokens, t1 = min(t0 + sg.tokens, a.T), te = min(t1, len);

    // places n0 + 16 m + n: their states' rates in base 2, values
    float A2[NB][4], h[NB][4];
    const Places<FILL> places(N, NP);
    const auto each_place = [&](auto f) {
#pragma unroll
        for (int m = 0; m < NB; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n) f(m, n, n0 + 16 * m + n);
    };
    each_place([&](int m, int n, int s) { A2[m][n] = finite_rate(a.A[(int64_t)d * N + places.state(s)]) * LOG2E; });
    const int64_t at_state = ((int64_t)b * D + d) * N;
    float *slots = sg.slots + ((int64_t)b * sg.count * D + d) * NP + n0, *sums = sg.sums + (int64_t)b * sg.count * D + d;
    const int64_t next_slot = (int64_t)D * NP;
    const auto load_slot = [&](int s, int m, float (&v)[4]) {
        const float4 q = *reinterpret_cast<const float4 *>(slots + s * next_slot + 16 * m);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    };
    const auto store_slot = [&](int s) {
#pragma unroll
        for (int m = 0; m < NB; ++m) store4(slots + s * next_slot + 16 * m, h[m]);
    };
    if (seg == 0 && (STATES_ONLY || sg.count == 1)) {
        each_place([&](int m, int n, int s) { h[m][n] = a.h0 ? a.h0[at_state + places.state(s)] : 0.f; });
        if (STATES_ONLY && ok) store_slot(0);
    } else if (STATES_ONLY) {
        each_place([&](int m, int n, int) { h[m][n] = 0.f; });
    } else {
#pragma unroll
        for (int m = 0; m < NB; ++m) load_slot(min(seg, 1), m, h[m]);
        // a few segments' loads together: the chain itself is one multiply-add each
        constexpr int JOIN = NB == 1 ? 16 : 8 / NB;
        for (int i = 2; i <= seg; i += JOIN) {
            float v[JOIN][NB][4], s[JOIN];
#pragma unroll
            for (int k = 0; k < JOIN; ++k) {
#pragma unroll
                for (int m = 0; m < NB; ++m) load_slot(min(i + k, seg), m, v[k][m]);
                s[k] = sums[(int64_t)min(i + k, seg) * D];
            }
#pragma unroll
            for (int k = 0; k < JOIN; ++k)
                if (i + k <= seg)
                    each_place([&](int m, int n, int) {
                        h[m][n] = __builtin_fmaf(fast_exp2(A2[m][n] * s[k]), h[m][n], v[k][m][n]);
                    });
        }
    }

    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f, skip = a.Dskip ? a.Dskip[d] : 0.f;
    // without a gate z reads x, unused; without a skip nothing is added, not 0 times x
    const bool gated = a.z != nullptr, skips = a.Dskip != nullptr, soft = a.softplus;
    const int64_t base = (int64_t)b * a.T * D;
    const T *xb = (const T *)a.x + base, *tb = (const T *)a.dt + base, *zb = (const T *)(gated ? a.z : a.x) + base;
    T *yb = (T *)a.y + base;
    const unsigned dl = (unsigned)d * sizeof(T), rb = (unsigned)D * sizeof(T);   // lane, row: bytes
    unsigned off[4];   // of the lane's tokens in a chunk
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i] = (unsigned)(4 * i + j) * rb + dl;
    const int64_t row = (int64_t)a.G * N, row0 = ((int64_t)b * a.T * a.G + g) * N;
    const int rt = tid / 16, rn = tid & 15;   // staging of B and C: token, place of a block
    int from[NB];                             // the states there, and their shares
    float share[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        from[nb] = places.state(16 * nb + rn);
        share[nb] = places.share(16 * nb + rn);
    }

    float sum = 0.f;   // of this lane's tokens
    if (t0 < te) {
        T xr[4], tr[4], zr[4], Br[NB], Cr[NB];
        const auto fetch = [&](int tc) {      // tokens past the end: the last one again, masked later
            const int tf = min(tc, te - 1);
            const int64_t at = (int64_t)tf * D;
            const Rows<T> xs(xb + at), ts(tb + at), zs(zb + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned o = tf + CHUNK <= te ? off[i] : (unsigned)min(4 * i + j, te - 1 - tf) * rb + dl;
                xr[i] = xs.load(o, 0);
                tr[i] = ts.load(o, 0);
                if (!STATES_ONLY) zr[i] = zs.load(o, 0);
            }
            __builtin_amdgcn_sched_barrier(0);   // the order in which they are used
            const int64_t o = row0 + (int64_t)min(tc + rt, te - 1) * row;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                Br[nb] = ((const T *)a.Bm)[o + from[nb]];
                if (!STATES_ONLY) Cr[nb] = ((const T *)a.Cm)[o + from[nb]];
            }
        };
        fetch(t0);
        for (int tc = t0; tc < te; tc += CHUNK) {
            float (&Bs)[CHUNK * NP] = rows[(tc / CHUNK) & 1][0], (&Cs)[CHUNK * NP] = rows[(tc / CHUNK) & 1][1];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const bool in = tc + rt < te;
                Bs[rt * NP + 16 * nb + rn] = in ? to_f32(Br[nb]) : 0.f;
                if (!STATES_ONLY) Cs[rt * NP + 16 * nb + rn] = in ? to_f32(Cr[nb]) * share[nb] : 0.f;
            }
            float x[4], s[4], z[4], u[4], r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = to_f32(xr[i]);
                s[i] = to_f32(tr[i]) + bias;
                if (!STATES_ONLY) z[i] = to_f32(zr[i]);
            }
            // one barrier a chunk: the buffer written next was last read a chunk earlier
            lds_barrier();
            fetch(tc + CHUNK);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float sp = softplus_f32(s[i]);
                s[i] = soft ? sp : s[i];
                u[i] = s[i] * x[i];
            }
            // Tokens behind the end change nothing: no step and no input.  (Their
            // B rows are zeros and every rate is finite, so 0 times them is 0.)
            if (tc + CHUNK > te)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (tc + 4 * i + j >= te) s[i] = u[i] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += s[i];
            // Four tokens and states of a lane at a time: all their rows and decays
            // first, then the chain.  Few wavefronts share a SIMD here, so the order
            // has to give each instruction independent neighbours; the barrier keeps it.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y[4];
#pragma unroll
                for (int m = 0; m < NB; ++m) {
                    float4 Bv[4], Cv[4];
                    float e[4][4];
                    const int at = 4 * i * NP + 16 * m + n0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) Bv[k] = *reinterpret_cast<const float4 *>(Bs + at + k * NP);
                    if (!STATES_ONLY)
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
#pragma unroll
                        for (int n = 0; n < 4; ++n) e[K][n] = h[m][n] = __builtin_fmaf(e[K][n], h[m][n], ub[n]);
                    });
                    if constexpr (!STATES_ONLY) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) y[k] = m ? __builtin_fmaf(Cv[k].x, e[k][0], y[k]) : Cv[k].x * e[k][0];
#pragma unroll
                        for (int k = 0; k < 4; ++k) y[k] = __builtin_fmaf(Cv[k].y, e[k][1], y[k]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) y[k] = __builtin_fmaf(Cv[k].z, e[k][2], y[k]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) y[k] = __builtin_fmaf(Cv[k].w, e[k][3], y[k]);
                    }
                }
                if constexpr (!STATES_ONLY) {
                    r[i] = quad_sums(y);
                }
            }
            if constexpr (!STATES_ONLY) {
                const Rows<T> ys(yb + (int64_t)tc * D);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float gate = z[i] * sigmoid_f32(z[i]);
                    r[i] = (skips ? __builtin_fmaf(skip, x[i], r[i]) : r[i]) * (gated ? gate : 1.f);
                }
                if (ok) {
                    if (tc + CHUNK <= te) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) ys.store(from_f32<T>(r[i]), off[i], 0);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (tc + 4 * i + j < te) ys.store(from_f32<T>(r[i]), off[i], 0);
                    }
                }
            }
        }
    }
    if constexpr (STATES_ONLY) {
        sum = quad_add<0xB1>(quad_add<0x4E>(sum));   // the quad's tokens
        if (!ok) return;
        store_slot(seg + 1);
        if (j == 0) sums[(int64_t)(seg + 1) * D] = sum;
    } else {
        if (!ok) return;
        for (int t = max(t0, te) + j; t < t1; t += 4) yb[(int64_t)t * D + d] = from_f32<T>(0.f);
        if (a.h_final && seg == sg.count - 1)
            each_place([&](int m, int n, int s) {
                if (!FILL || s < N) a.h_final[at_state + s] = h[m][n];
            });
    }
}

// One token.  L lanes (a power of two with 4 L >= N) have a channel of four
// sequences, lane l of them states 4 l .. 4 l + 3 and, for what a channel costs
// once, sequence l % 4 (l and l + 2, or all four, where L is 2 or 1): as in the
// forward with sequences in the place of tokens, so rates and positions are shared
// by the four.  The read and write of the states bound it; all their loads are out
// before the first is used, and as they pass once they are non-temporal.
//
// A workgroup takes 256 / L channels; where there are fewer, sequences lie side by
// side in it, 1 << shift threads each.  Measured (bfloat16): B256 D12288 N16 0.076
// ms, 5.7 TB/s; 0.101 with four channels of one sequence a thread, each with its
// own rates, positions and softplus (twice the vector instructions).
template <int L, int I, int K> __device__ __forceinline__ float of_sequence(const float (&v)[K])
{
    constexpr int PAIR = I & 1 ? 0xF5 : 0xA0;   // quad_perm [1,1,3,3] or [0,0,2,2]
    if constexpr (L == 1) return v[I];
    else if constexpr (L == 2)
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v[I / 2]), PAIR, 0xF, 0xF, true));
    else return quad_bcast<I>(v[0]);
}
template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(256) kda_scan_step_kernel(ScanArgs a, int tiles, int shift)
{
    constexpr int K = L < 4 ? 4 / L : 1;   // sequences of which a lane does the channel's own part
    const int tid = threadIdx.x, l = tid % L, n0 = 4 * l;
    const int tile = blockIdx.x % tiles, per = 256 >> shift, side = tid >> shift;
    const int64_t first = (int64_t)(blockIdx.x / tiles) * 4 * per;   // sequence
    const int B = a.B, D = a.D, N = a.N;
    const int c = tile * (256 / L) + (tid & ((1 << shift) - 1)) / L, d = min(c, D - 1);
    const bool ok = c < D, in4 = n0 < N;
    const unsigned row = (unsigned)a.G * N, g = a.G == 1 ? 0 : d / (D / a.G);

    // states and rows of B and C of sequences first + i per + side, i < 4
    Pack<float, 4> hr[4];
    Raw4<T> Br[4], Cr[4];
    float hs[4][4], Bs[4][4], Cs[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t q = first + i * per < B ? first + i * per : B - 1;   // behind the last sequence: it again, not stored
        const unsigned sd = min(side, (int)(B - 1 - q));
        const float *hp = a.h_final + q * D * N;
        const T *Bp = (const T *)a.Bm + q * row, *Cp = (const T *)a.Cm + q * row;
        const unsigned at = (sd * D + d) * N + n0, rat = sd * row + g * N + n0;
        if constexpr (VEC) {
            hr[i].zero();
            Br[i].zero();
            Cr[i].zero();
            if (in4) {
                hr[i].stream(hp + at);
                Br[i].load(Bp + rat);
                Cr[i].load(Cp + rat);
            }
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                hs[i][n] = n0 + n < N ? hp[at + n] : 0.f;
                Bs[i][n] = n0 + n < N ? to_f32(Bp[rat + n]) : 0.f;
                Cs[i][n] = n0 + n < N ? to_f32(Cp[rat + n]) : 0.f;
            }
        }
    }
    float A2[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) A2[n] = n0 + n < N ? finite_rate(a.A[(int64_t)d * N + n0 + n]) * LOG2E : 0.f;
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f, skip = a.Dskip ? a.Dskip[d] : 0.f;
    const auto own = [&](int k) { return first + (int64_t)(l % 4 + k * L) * per + side; };
    const auto token = [&](int k) { return (own(k) < B ? own(k) : B - 1) * D + d; };
    float x[K], z[K], s[K], u[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        x[k] = to_f32(((const T *)a.x)[token(k)]);
        z[k] = a.z ? to_f32(((const T *)a.z)[token(k)]) : 0.f;
        s[k] = to_f32(((const T *)a.dt)[token(k)]) + bias;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (a.softplus) s[k] = softplus_f32(s[k]);
        u[k] = s[k] * x[k];
    }

    float y[4] = {};
    each4([&](auto i) {
        constexpr int I = decltype(i)::value;
        const int64_t q = first + I * per;
        float *hp = a.h_final + q * D * N + ((unsigned)side * D + d) * N + n0;
        if constexpr (VEC) {
            hr[I].to_f32(hs[I]);
            Br[I].to_f32(Bs[I]);
            Cr[I].to_f32(Cs[I]);
        }
        float (&h)[4] = hs[I];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float v = __builtin_fmaf(fast_exp2(of_sequence<L, I>(s) * A2[n]), h[n], of_sequence<L, I>(u) * Bs[I][n]);
            h[n] = VEC || n0 + n < N ? v : 0.f;   // (with an infinite s x not 0 by itself)
            y[I] = __builtin_fmaf(Cs[I][n], h[n], y[I]);
        }
        if (VEC && !in4) y[I] = 0.f;
        if (ok && q + side < B) {
            if constexpr (VEC) {
                if (in4) Pack<float, 4>::unstream(hp, h);
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    if (n0 + n < N) hp[n] = h[n];
            }
        }
    });
    float r[K];
    if constexpr (L == 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) r[k] = y[k];
    } else if constexpr (L == 2) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float p = quad_add<0xB1>(y[2 * k]), q = quad_add<0xB1>(y[2 * k + 1]);   // quad_perm [1,0,3,2]
            r[k] = l ? q : p;
        }
    } else {
        r[0] = quad_sums(y);
#pragma unroll
        for (int m = 4; m < L; m <<= 1) r[0] += __shfl_xor(r[0], m, L);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (ok && l < 4 && own(k) < B) {
            const float v = a.Dskip ? __builtin_fmaf(skip, x[k], r[k]) : r[k];
            ((T *)a.y)[token(k)] = from_f32<T>(a.z ? v * (z[k] * sigmoid_f32(z[k])) : v);
        }
}

int state_blocks(int N) { return N <= 16 ? 1 : N <= 32 ? 2 : 4; }   // NB
int channel_tiles(int D, int G) { return (D / G + 63) / 64; }   // of a workgroup's channels

// Segments: of the powers of two, the one with the smallest estimated time, in
// microseconds from timings on MI355X (bfloat16).  At N = 16, with w wavefronts
// a SIMD, a token takes max(0.104, 0.03 + 0.067 w) with outputs and max(0.06,
// 0.02 + 0.05 w) without; a second launch 6; and every segment reads the end
// states in front of it, in total states x n^2 / 2 at about 20 MB/us.  One
// segment and the choice measure: B1 T2048 D1024 218 and 28 (32 segments), B1
// T16384 D4096 1725 and 467 (32), B2 T2048 D4096 215 and 126 (16), B4 T2048 D4096
// 218 and 230 (8: one is kept); N = 64: B1 T2048 D1024 551 and 73 (32).
Segments plan(int B, int T, int D, int N, int G)
{
    const int nb = state_blocks(N);
    const double waves = 4.0 * B * G * channel_tiles(D, G) / 1024.0;   // a SIMD, in one segment
    const double states = 64.0 * nb * B * D / 2.0 / 20e6;              // bytes of all states / 2 / rate
    const double out = 0.4 + 0.6 * nb, in = 0.3 + 0.7 * nb;            // a token's time over that with 16 states
    Segments s{};
    double least = 0.0;
    for (int n = 1; n <= 128 && (n == 1 || n * CHUNK <= T); n *= 2) {
        const int tokens = (T + n * CHUNK - 1) / (n * CHUNK) * CHUNK, count = tokens > 0 ? (T + tokens - 1) / tokens : 1;
        const double w = waves * count;
        double us = tokens * out * std::max(0.104, 0.03 + 0.067 * w);
        if (count > 1) us += tokens * in * std::max(0.06, 0.02 + 0.05 * w) + 6.0 + 0.03 * count + states * count * count;
        if (n == 1 || us < least) {
            s.tokens = tokens;
            s.count = count;
            least = us;
        }
    }
    return s;
}

template <typename T, int NB> hipError_t fwd_launch(const ScanArgs &a, hipStream_t stream)
{
    const int tiles = channel_tiles(a.D, a.G);
    Segments s = plan(a.B, a.T, a.D, a.N, a.G);
    if (!a.ws) {
        s.count = 1;
        s.tokens = a.T;
    }
    const int64_t blocks = (int64_t)a.B * a.G * tiles;
    if (!grid_fits(blocks * s.count, 256)) return hipErrorNotSupported;
    if (s.count > 1) {
        s.slots = a.ws;
        s.sums = a.ws + (int64_t)a.B * s.count * 16 * NB * a.D;
        (a.N == 16 * NB ? kda_scan_kernel<T, NB, true, false> : kda_scan_kernel<T, NB, true, true>)
            <<<(unsigned)(blocks * (s.count - 1)), 256, 0, stream>>>(a, s, tiles);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    (a.N == 16 * NB ? kda_scan_kernel<T, NB, false, false> : kda_scan_kernel<T, NB, false, true>)
        <<<(unsigned)(blocks * s.count), 256, 0, stream>>>(a, s, tiles);
    return hipGetLastError();
}

template <typename T> hipError_t fwd_dispatch(const ScanArgs &a, hipStream_t s)
{
    switch (state_blocks(a.N)) {
    case 1: return fwd_launch<T, 1>(a, s);
    case 2: return fwd_launch<T, 2>(a, s);
    default: return fwd_launch<T, 4>(a, s);
    }
}

template <typename T, int L> hipError_t step_launch(const ScanArgs &a, hipStream_t stream)
{
    int shift = 0;   // threads of a sequence in a workgroup
    while (shift < 8 && (1 << shift) < (int64_t)L * a.D) ++shift;
    const int tiles = (a.D + 256 / L - 1) / (256 / L), group = 4 * (256 >> shift);
    const int64_t blocks = (int64_t)tiles * (((int64_t)a.B + group - 1) / group);
    if (!grid_fits(blocks, 256)) return hipErrorNotSupported;
    (a.N % 4 == 0 ? kda_scan_step_kernel<T, L, true> : kda_scan_step_kernel<T, L, false>)
        <<<(unsigned)blocks, 256, 0, stream>>>(a, tiles, shift);
    return hipGetLastError();
}

template <typename T> hipError_t step_dispatch(const ScanArgs &a, hipStream_t s)
{
    if (a.N <= 4) return step_launch<T, 1>(a, s);
    if (a.N <= 8) return step_launch<T, 2>(a, s);
    if (a.N <= 16) return step_launch<T, 4>(a, s);
    if (a.N <= 32) return step_launch<T, 8>(a, s);
    return step_launch<T, 16>(a, s);
}

}  // namespace

int64_t scan_fwd_workspace_floats(int B, int T, int D, int N, int G)
{
    const Segments s = plan(B, T, D, N, G);
    return s.count > 1 ? (int64_t)B * s.count * D * (16 * state_blocks(N) + 1) : 0;
}

hipError_t launch_scan_fwd(const ScanArgs &a, hipStream_t s)
{
    (void)hipGetLastError();
    return a.bf16 ? fwd_dispatch<uint16_t>(a, s) : fwd_dispatch<float>(a, s);
}

hipError_t launch_scan_step(const ScanArgs &a, hipStream_t s)
{
    (void)hipGetLastError();
    return a.bf16 ? step_dispatch<uint16_t>(a, s) : step_dispatch<float>(a, s);
}

}  // namespace kda
