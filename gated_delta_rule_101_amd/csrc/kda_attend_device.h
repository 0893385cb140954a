// Device pieces of attention over the 8-bit paged cache, shared by the kernel
// for few queries a sequence and the one for prompts.
#pragma once

#include "kda_attend_line.h"
#include "kda_attn.h"
#include "kda_code8.h"

namespace kda {

__device__ __forceinline__ float fast_log2(float x) { return __builtin_amdgcn_logf(x); }

__device__ __forceinline__ Sequence sequence(const AttendArgs &a, int b)
{
    int from = b, to = b + 1;                // without row starts, one row each
    if (a.q_start) {
        from = a.q_start[b];
        to = a.q_start[b + 1];
    }
    return sequence_of(from, to, a.tokens, a.context[b], a.room);
}

// The page of a token, -1 where there is none: behind the last token, or an
// entry that names no page of the cache.
__device__ __forceinline__ int page_of(const AttendArgs &a, const int *table, int token, int context, int shift)
{
    if (token >= context) return -1;
    const int id = table[token >> shift];
    return (unsigned)id < (unsigned)a.pages ? id : -1;
}

// Over the four lanes that hold one query (m, m + 16, m + 32, m + 48).
__device__ __forceinline__ float quarters_max(float x)
{
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float quarters_sum(float x)
{
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// 8 values as SPLIT float16 parts: nearest, then nearest of what is left.
template <int SPLIT, typename F> __device__ __forceinline__ void split_f16(const float *x, F part)
{
    f16x8 y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (_Float16)x[i];
    part(0) = y;
    if constexpr (SPLIT == 2) {
        f16x8 z;
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = (_Float16)(x[i] - (float)y[i]);
        part(1) = z;
    }
}

// e with most 2^e in [2^14, 2^15), by the exponent's bits; 0 where most is 0 or not finite.
__device__ __forceinline__ int range_exponent(float most)
{
    const int ex = (int)(__float_as_uint(most) >> 23);
    return ex == 0 || ex == 255 ? 0 : 127 + 14 - ex;
}

// One query row (zeros unless `real`) as the second operand of the score products,
// scaled into float16's range; returns what the products are to be multiplied
// by.  A lane's channels are 64 c + 16 quarter + 0 .. 15 for each c, which are
// inner steps 2 c and 2 c + 1: the order in which it reads keys.
template <typename T, int D, int SPLIT, int KS, typename F>
__device__ __forceinline__ float load_query(const T *p, bool real, int quarter, F part)
{
    float x[D / 64][16], most = 0.f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
            Raw8<T> raw;
            raw.load(p + 64 * c + 16 * quarter + e);
            float v[8];
            raw.to_f32(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[c][e + i] = real ? v[i] : 0.f;
                most = fmaxf(most, fabsf(x[c][e + i]));
            }
        }
    most = quarters_max(most);
    const int e = range_exponent(most);
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __builtin_ldexpf(x[c][8 * k + i], e);
            split_f16<SPLIT>(v, [&](int s) -> f16x8 & { return part(s, 2 * c + k); });
        }
    return __builtin_ldexpf(1.f, -e);
}

// The same for 32x32x16 products: a lane's channels are 16 k + 8 half + 0 .. 7.
// The sign of the softmax's scale goes with the query, so that maxima of the
// products are maxima of the scores.
template <typename T, int D, int SPLIT>
__device__ __forceinline__ float load_row(const T *p, bool real, int half, bool negative, f16x8 (&q)[SPLIT][D / 16])
{
    float x[D / 16][8], most = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        Raw8<T> raw;
        raw.load(p + 16 * k + 8 * half);
        raw.to_f32(x[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[k][i] = !real ? 0.f : negative ? -x[k][i] : x[k][i];
            most = fmaxf(most, fabsf(x[k][i]));
        }
    }
    const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(most), __float_as_uint(most), false, false);
    most = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
    const int e = range_exponent(most);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = __builtin_ldexpf(x[k][i], e);
        split_f16<SPLIT>(x[k], [&](int s) -> f16x8 & { return q[s][k]; });
    }
    return __builtin_ldexpf(1.f, -e);
}

// Value scales go into the weights' exponents: a place of score z (in base 2) on a
// page of value scale 2^lv has weight 2^(z + lv - top - lift + 13), with `top` the
// base of the row's scores and `lift` that of its (z - top + lv), each up to SLACK
// below its largest value so far.  So a row's largest weight x scale stands between
// 2^13 and 2^15, below float16's 65504, whatever pages others see, and what is up to
// 2^27 times smaller keeps all bits.  The sum of the weights alone, in units of 2^top,
// takes the scale back, 2^-rel.
constexpr float VALUE_REST = 0x1p-13f, SLACK = 2.f;
// held: a base, 0 where there is none yet.  rel = lv - lift + 13: a scale 2^64 below
// what the row holds, or zero, adds nothing (float16 ends at 2^-25), but its weights
// still count in the sum.  Scales that are not finite pass as zero here: the weights of
// their tokens are made NaN behind the sum.
__device__ __forceinline__ float held(float base) { return base == -__builtin_inff() ? 0.f : base; }
// Scores beyond FAR are first taken relative to their base, both as rounded (a fused
// product would differ by its rounding): added to rel, the base would take bits from it, as
// many as weights past float16 from 2^24 on.
constexpr float FAR = 0x1p20f;
__device__ __forceinline__ float from_base(float score, float base)
{
#pragma clang fp contract(off)
    return score - base;
}
__device__ __forceinline__ float relative_level(float lv, float lift) { return fmaxf(lv - lift, -64.f) + 13.f; }
__device__ __forceinline__ bool is_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// 16 bytes with those from place n on cleared.
__device__ __forceinline__ uint4 keep_bytes(uint4 x, int n)
{
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = n - 4 * i;
        w[i] = k >= 4 ? w[i] : k <= 0 ? 0u : w[i] & ((1u << (8 * k)) - 1u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A call's pieces in its workspace: one record a workgroup, then two pieces each.
struct Record {      // a row of units that is cut: its first piece is this workgroup's
    int b, h, block, last;                   // last: the workgroup of its last piece, -1: none
};
constexpr int SHARES = 1024;                 // workgroups that share the line of units, at most
// Floats of one piece: output rows, then maxima and sums.
template <int D, int ROWS> constexpr int PIECE = ROWS * (D + 2);

// Four channels of a finished row (index i G + g): o / l, 0 where nothing was
// seen; with the first, the row's log of the weights' sum.
template <typename T>
__device__ __forceinline__ void write_row(const AttendArgs &a, const Sequence &s, int h, int G, int r, int d, int D,
                                          const float (&y)[4], float best, float l)
{
    const int i = r / G, g = r - i * G;
    const int64_t at = (int64_t)(s.first + i) * a.Hq + h * G + g;
    const bool none = l == 0.f;                // a row that saw something has its maximum's weight, 1, in l
    const float inv = 1.f / l;
    const float z[4] = {none ? 0.f : y[0] * inv, none ? 0.f : y[1] * inv, none ? 0.f : y[2] * inv, none ? 0.f : y[3] * inv};
    store4((T *)a.out + at * D + d, z);
    if (a.lse && d == 0) a.lse[at] = none ? -__builtin_inff() : (best + fast_log2(l)) * LN2;
}

// A value that all lanes hold, as the scalar it is.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A workgroup's share of the line of units.
struct Line {
    int b;                                   // sequence of the next unit
    int u;                                   // the unit's place among its sequence's
    int left, at, share;                     // units to do, place on the line, units a workgroup
    bool single;                             // shares begin with the rows of units
    // the workgroup that ends a row of units of which this one has the first, but not all
    __device__ __forceinline__ int last(int tiles) const
    {
        return single ? blockIdx.x + last_share(0, tiles, share) : last_share(at, tiles, share);
    }
};
template <int WAVES> __device__ __forceinline__ unsigned workgroup_sum(unsigned x, unsigned *part)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) x = units_add(x, __shfl_xor(x, m, 64));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) x = units_add(x, part[w]);
    __syncthreads();
    return x;
}
// `at_least`: a share's least units, where rows of units are that long; short
// rows stay whole.  part: [WAVES] in LDS.
template <int WAVES>
__device__ __forceinline__ Line cut_line(const AttendArgs &a, int G, int rows_of_block, int at_least, unsigned *part)
{
    const int lane = threadIdx.x & 63;
    if (a.B == 1) {
        // all rows of units are alike: equal parts of each, of `at_least` units where that leaves enough workgroups
        const Sequence s = sequence(a, 0);
        const unsigned tiles = tiles_of(s), rows = blocks_of(s, G, rows_of_block) * a.Hk;
        if (rows > 0 && rows <= gridDim.x) {
            const unsigned parts = min((tiles + at_least - 1) / at_least, gridDim.x / rows);
            const unsigned share = (tiles + parts - 1) / parts, row = blockIdx.x / parts, part_of = blockIdx.x - row * parts;
            const int left = row < rows ? (int)(tiles - part_of * share) : 0;
            return Line{0, (int)(row * tiles + part_of * share), max(min(left, (int)share), 0), 0, (int)share, true};
        }
    }
    unsigned units = 0, rows = 0, upto = 0, mine = 0;
    const auto of_lane = [&](int b) {            // units of sequence b, and of those up to it among 64
        mine = 0;
        if (b < a.B) {
            const Sequence s = sequence(a, b);
            mine = (unsigned)blocks_of(s, G, rows_of_block) * a.Hk;
            rows = units_add(rows, mine);
            mine *= tiles_of(s);                 // of one sequence alone: below LINE_LIMIT
        }
        upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const unsigned y = __shfl_up(upto, d, 64);
            if (lane >= d) upto = units_add(upto, y);
        }
    };
    if (a.B <= 64) {                             // a wave sees them all
        of_lane(lane);
        units = uniform(__shfl(upto, 63, 64));
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) rows = units_add(rows, __shfl_xor(rows, m, 64));
        rows = uniform(rows);
    } else {
        for (int b = threadIdx.x; b < a.B; b += 64 * WAVES) {
            const Sequence s = sequence(a, b);
            const unsigned r = (unsigned)blocks_of(s, G, rows_of_block) * a.Hk;
            rows = units_add(rows, r);
            units = units_add(units, r * tiles_of(s));
        }
        units = uniform(workgroup_sum<WAVES>(units, part));
        rows = uniform(workgroup_sum<WAVES>(rows, part));
    }
    Line l = {0, 0, 0, 0, 1, false};
    if (units == 0 || units >= LINE_LIMIT) return l;
    l.share = share_of(units, rows, gridDim.x, at_least);
    const int64_t at = (int64_t)l.share * blockIdx.x;
    if (at >= units) return l;
    l.at = (int)at;
    l.left = min(l.share, (int)units - l.at);
    unsigned before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        if (a.B > 64) of_lane(b0 + lane);
        const uint64_t past = __ballot(before + upto > (unsigned)l.at);
        if (past) {
            const int f = __builtin_ctzll(past);
            l.b = b0 + f;
            l.u = uniform(l.at - before - __shfl(upto - mine, f, 64));
            break;
        }
        before = uniform(before + __shfl(upto, 63, 64));
    }
    return l;
}

// The launcher for many query rows a sequence (kda_cache_attend_rows.hip), and
// floats of workspace it may need.
hipError_t launch_attend_rows(const AttendArgs &a, hipStream_t stream);
int64_t attend_rows_workspace_floats(int tokens, int B, int Hq, int Hk, int D, int page, int per, int most);
// The second launch of a line with blocks of ROWS query rows.
template <int ROWS> hipError_t launch_attend_join(const AttendArgs &a, int workgroups, int rows, hipStream_t stream);

}  // namespace kda
