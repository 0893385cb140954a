// Attention over the 8-bit paged cache for gfx950, for few queries a sequence:
//   s = scale (q . K) k_scale, o = sum softmax(s) V v_scale, query i of n at
// position context - n + i seeing places up to its own.
//
// Bound by HBM bandwidth: every code is read once for the G = Hq / Hk heads and
// the queries that share it, which make the columns of the products.  With
// 16x16x32 float16 products and the score tile transposed (tokens x queries), a
// lane holds 16 neighbouring tokens' scores of one query.  Which token a tile's
// row is, and which channel an inner index, is free as long as both operands
// agree; chosen so that a lane's codes are 16 neighbouring bytes: of a key's
// row, and of a channel's row in the values' pages, which hold tokens innermost
// for this.  So codes go from memory to registers to float16 (exact for either
// code), and weights from scores to the second product, with neither LDS nor
// exchanges between lanes.
//
// Work is counted in units: 64 tokens of one sequence, key head and block of
// 16 rows (query, head of the group).  All units of the call lie on one line which is cut into equal
// shares, one a workgroup, whatever the lengths are; its waves take turns at a
// share's units.  A share that ends inside a row of units leaves its running
// maximum, sum and output in the workspace, and a second launch joins them.
//
// Float16: queries are scaled by a power of two that puts their row's largest
// channel at 2^14 .. 2^15 (bfloat16 fits exactly, what is lost of a channel is
// under 2^-39 of the largest).  Weights carry their page's value scale, in the
// exponent, over the largest weight x scale that their row has met, so that they
// are in float16's range whatever the pages' scales are, and stand 2^13 times larger.
// They are rounded to 11 bits, three more than a bfloat16 output has: over many
// places these roundings average out, and the error against float64 stays that of the
// output's own rounding (1.67e-3 of its size, 1.66e-3 with float32 weights), where
// a second part would double the second product.  The sum of the weights is of
// float32 ones.  Float32 queries and weights are taken in two float16 parts.
//
// 256 sequences of 4096 to 8192 tokens, 32 query and 8 key heads x 128, e4m3: 0.57
// ms, 5.7 TB/s; one sequence of 777: 7.7 us.
#include "kda_attn.h"
#include "kda_block.h"
#include "kda_attend_device.h"

namespace kda {
namespace {

template <int D, bool BF, bool INT8>
__global__ void __launch_bounds__(256, D <= 128 ? 2 : 1) kda_cache_attend_kernel(AttendArgs a, int shift)
{
    constexpr int SPLIT = BF ? 1 : 2, KS = D / 32, DT = D / 16, ROWS = 16;
    typedef typename Store<BF>::type T;
    __shared__ unsigned part[4];
    __shared__ __align__(16) float merge[4][16][D + 4];
    __shared__ float stat[4][2][ROWS];
    const int wave = uniform((int)threadIdx.x / 64), lane = threadIdx.x & 63, m = lane & 15, quarter = lane >> 4;
    const int G = a.Hq / a.Hk;
    Line line = cut_line<4>(a, G, ROWS, 4, part);    // a unit for each wave
    Record mine = {0, 0, 0, -1};
    float *const pieces = a.ws + (sizeof(Record) / 4) * gridDim.x;
    while (line.left > 0) {
        const Sequence s = sequence(a, line.b);
        const int tiles = tiles_of(s), blocks = blocks_of(s, G, ROWS);
        const unsigned u = line.u;
        if (u >= (unsigned)tiles * blocks * a.Hk) {
            line.u = 0;
            if (++line.b >= a.B) break;         // the line ends with the last sequence
            continue;
        }
        const int b = line.b;
        const int row = u / (unsigned)tiles, t_begin = u - row * tiles;
        const int t_end = min(tiles, t_begin + line.left);
        const int h = row / blocks, block = row - h * blocks;
        const int r0 = block * ROWS, active = min(ROWS, s.queries * G - r0);
        // Pages of a tile: of this lane's key rows (group m / 4), of its scores' tokens (group = quarter); looked up
        // a tile ahead.
        const int *table = a.table + (int64_t)b * a.per;
        const int gk = m >> 2;
        const auto look_up = [&](int t, int &pk, int &pv) {
            pk = page_of(a, table, t * 64 + 16 * gk, s.context, shift);
            pv = page_of(a, table, t * 64 + 16 * quarter, s.context, shift);
        };
        int pk, pv;
        look_up(t_begin + wave, pk, pv);

        // queries: lane m is row r0 + m
        f16x8 q[SPLIT][KS];
        const int at_row = r0 + min(m, active - 1), qi = at_row / G, qg = at_row - qi * G;
        const int limit = m < active ? s.context - s.queries + qi + 1 : 0x7fffffff;
        const float factor = load_query<T, D, SPLIT, KS>((const T *)a.q + ((int64_t)(s.first + qi) * a.Hq + h * G + qg) * D,
                                                         m < active, quarter,
                                                         [&](int x, int k) -> f16x8 & { return q[x][k]; }) * a.scale * LOG2E;
        // tiles with every place seen by every row need no mask
        const int whole = min(s.context - s.queries + r0 / G + 1, s.context);
        const int furthest = min(s.context, s.context - s.queries + (r0 + active - 1) / G + 1);

        f32x4 o[DT];
        float top = -__builtin_inff(), sum = 0.f, lift = -__builtin_inff();
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};

        for (int t = t_begin + wave; t < t_end; t += 4) {
            const int t0 = t * 64;
            if (t0 >= furthest) break;
            const int64_t ak = (int64_t)max(pk, 0) * a.Hk + h, av = (int64_t)max(pv, 0) * a.Hk + h;
            const uint8_t *kp = a.k_codes + (ak * a.page + ((t0 + 16 * gk) & (a.page - 1)) + (m & 3)) * D + 16 * quarter;
            const uint8_t *vp = a.v_codes + (av * D + m) * a.page + ((t0 + 16 * quarter) & (a.page - 1));
            uint4 kr[4][D / 64], vr[DT];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    kr[i][c] = *reinterpret_cast<const uint4 *>(kp + 4 * i * D + 64 * c);
            const float ks = a.k_scale[av], vs = a.v_scale[av];
#pragma unroll
            for (int d = 0; d < DT; ++d) vr[d] = *reinterpret_cast<const uint4 *>(vp + (int64_t)16 * d * a.page);

            const bool gone = pv < 0, masked = t0 + 64 > whole || __any(gone);
            look_up(t + 4, pk, pv);
            f16x8 ka[4][KS];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    ka[i][2 * c] = codes_f16<INT8>(kr[i][c].x, kr[i][c].y);
                    ka[i][2 * c + 1] = codes_f16<INT8>(kr[i][c].z, kr[i][c].w);
                }
            const int tb = t0 + 16 * quarter;                  // this lane's first token
            const bool broken = !gone && !is_finite(vs);
            const float lv = gone || broken ? -__builtin_inff() : fast_log2(vs);
            f16x8 w[SPLIT][2];
            const float c = factor * (gone ? 0.f : is_finite(ks) ? ks : __builtin_nanf(""));
            const int seen = gone ? 0 : min(limit, s.context) - tb;     // of this lane's 16 tokens
            float v[16], own = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int p = 0; p < SPLIT; ++p)
                        x = __builtin_amdgcn_mfma_f32_16x16x32_f16(ka[i][k], q[p][k], x, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * i + j] = x[j] * c;
            }
            if (masked) {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = i < seen ? v[i] : -__builtin_inff();
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) own = fmaxf(own, v[i]);
            const float best = quarters_max(own);
            if (__any(best > top + SLACK)) {     // rare after the first tiles
                const float now = fmaxf(top, best), back = now == -__builtin_inff() ? 0.f : top - now;
                top = now;
                sum *= fast_exp2(back);
                lift += back;                    // the outputs' unit, 2^(top + lift), stays
            }
            float base = held(top);
            if (__any(fabsf(base) > FAR)) {
                const float far = fabsf(base) > FAR ? base : 0.f;        // other rows stay as they are
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = from_base(v[i], far);
                own = from_base(own, far);
                base -= far;
            }
            const float most = quarters_max(own - base + lv);
            if (__any(most > lift + SLACK)) {
                const float now = fmaxf(lift, most), fade = now == -__builtin_inff() ? 1.f : fast_exp2(lift - now);
                lift = now;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[d][i] *= fade;
            }
            const float rel = relative_level(lv, held(lift)), offset = rel - base;
            float total = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                v[i] = fast_exp2(v[i] + offset);
                total += v[i];
            }
            sum = __builtin_fmaf(total, fast_exp2(-rel), sum);
            if (__any(broken)) {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = broken && i < seen ? __builtin_nanf("") : v[i];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) split_f16<SPLIT>(v + 8 * k, [&](int p) -> f16x8 & { return w[p][k]; });
            if (masked && !INT8) {
                // weights of places that hold no token are zero; their codes must not be NaN
                const int there = gone ? 0 : s.context - tb;
#pragma unroll
                for (int d = 0; d < DT; ++d) vr[d] = keep_bytes(vr[d], there);
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const f16x8 lo = codes_f16<INT8>(vr[d].x, vr[d].y), hi = codes_f16<INT8>(vr[d].z, vr[d].w);
#pragma unroll
                for (int p = 0; p < SPLIT; ++p) {
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, w[p][0], o[d], 0, 0, 0);
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, w[p][1], o[d], 0, 0, 0);
                }
            }
        }

        // The four waves' parts meet: scaled to the common maximum, in units of the values.
        sum = quarters_sum(sum);
        if (quarter == 0) {
            stat[wave][0][m] = top;
            stat[wave][1][m] = sum;
        }
        const bool whole_row = t_begin == 0 && t_end == tiles;
        float *piece = pieces + (int64_t)(2 * blockIdx.x + (t_begin == 0)) * PIECE<D, ROWS>;
        if (t_begin == 0 && !whole_row) mine = {b, h, block, line.last(tiles)};
        line.u += t_end - t_begin;
        line.left -= t_end - t_begin;
        line.at += t_end - t_begin;
        __syncthreads();
        float best = -__builtin_inff();
#pragma unroll
        for (int v = 0; v < 4; ++v) best = fmaxf(best, stat[v][0][m]);
        const float f = fast_exp2(lift == -__builtin_inff() ? lift : top - best + lift);      // 0 where every value was
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) merge[wave][m][16 * d + 4 * quarter + i] = o[d][i] * VALUE_REST * f;
        __syncthreads();
        for (int e = threadIdx.x; e < 16 * (D / 4); e += 256) {
            const int rr = e / (D / 4), d = 4 * (e % (D / 4));
            if (rr >= active) continue;
            float hi = -__builtin_inff(), l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int v = 0; v < 4; ++v) hi = fmaxf(hi, stat[v][0][rr]);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                l += stat[v][1][rr] * (hi == -__builtin_inff() ? 1.f : fast_exp2(stat[v][0][rr] - hi));
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] += merge[v][rr][d + i];
            }
            if (whole_row) {
                write_row<T>(a, s, h, G, r0 + rr, d, D, y, hi, l);
            } else {
                *reinterpret_cast<float4 *>(piece + rr * D + d) = make_float4(y[0], y[1], y[2], y[3]);
                if (d == 0) {
                    piece[ROWS * D + rr] = hi;
                    piece[ROWS * D + ROWS + rr] = l;
                }
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) reinterpret_cast<Record *>(a.ws)[blockIdx.x] = mine;
}

// Joins the pieces of cut rows: blocks (first piece's workgroup, query rows).  A
// group of D / 4 lanes has a row where pieces are few; where they are many (one
// long sequence), the groups share each row's pieces and meet in LDS.
template <int D> constexpr int JOIN_ROWS = 1024 / D;         // groups of a workgroup
template <int D, int ROWS, bool BF>
__global__ void __launch_bounds__(256) kda_cache_attend_join_kernel(AttendArgs a)
{
    constexpr int L = D / 4, GROUPS = JOIN_ROWS<D>, ALONE = 16;
    typedef typename Store<BF>::type T;
    __shared__ __align__(16) float acc[GROUPS][L][4];
    __shared__ float best_of[GROUPS], sum_of[GROUPS];
    const int first = blockIdx.x, tid = threadIdx.x, l = tid % L, g = tid / L, d = 4 * l;
    const Record rec = reinterpret_cast<const Record *>(a.ws)[first];
    if (rec.last < 0) return;
    const Sequence s = sequence(a, rec.b);
    const int G = a.Hq / a.Hk, r0 = rec.block * ROWS, active = min(ROWS, s.queries * G - r0);
    const float *pieces = a.ws + (sizeof(Record) / 4) * gridDim.x;
    const int n = rec.last - first + 1, row0 = blockIdx.y * GROUPS;
    const auto piece = [&](int i) { return pieces + (int64_t)(2 * (first + i) + (i == 0)) * PIECE<D, ROWS>; };
    // pieces i, i + step, ... of a row: the running maximum, sum and output
    const auto gather = [&](int rr, int i, int step, float &best, float &sum, float (&y)[4]) {
        best = -__builtin_inff();
        sum = y[0] = y[1] = y[2] = y[3] = 0.f;
#pragma unroll 4
        for (; i < n; i += step) {
            const float *p = piece(i);
            const float top = p[ROWS * D + rr], part = p[ROWS * D + ROWS + rr];
            const float4 x = *reinterpret_cast<const float4 *>(p + rr * D + d);
            const float now = fmaxf(best, top);
            const float f = best == now ? 1.f : fast_exp2(best - now), w = top == now ? 1.f : fast_exp2(top - now);
            best = now;
            sum = sum * f + part * w;
            y[0] = y[0] * f + x.x * w;
            y[1] = y[1] * f + x.y * w;
            y[2] = y[2] * f + x.z * w;
            y[3] = y[3] * f + x.w * w;
        }
    };
    float best, sum, y[4];
    if (n <= ALONE) {
        const int rr = row0 + g;
        if (rr >= active) return;
        gather(rr, 0, 1, best, sum, y);
        write_row<T>(a, s, rec.h, G, r0 + rr, d, D, y, best, sum);
        return;
    }
    for (int rr = row0; rr < min(row0 + GROUPS, active); ++rr) {
        gather(rr, g, GROUPS, best, sum, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[g][l][i] = y[i];
        if (l == 0) {
            best_of[g] = best;
            sum_of[g] = sum;
        }
        __syncthreads();
        if (g == 0) {
            for (int k = 0; k < GROUPS; ++k) best = fmaxf(best, best_of[k]);
            sum = y[0] = y[1] = y[2] = y[3] = 0.f;
            for (int k = 0; k < GROUPS; ++k) {
                const float w = best_of[k] == best ? 1.f : fast_exp2(best_of[k] - best);
                sum += sum_of[k] * w;
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] += acc[k][l][i] * w;
            }
            write_row<T>(a, s, rec.h, G, r0 + rr, d, D, y, best, sum);
        }
        __syncthreads();
    }
}

// Which kernel: this one for up to 16 rows of a sequence and key head, and, as
// blocks of 16, for up to 64 while the line is short enough that latency counts
// (at most FEW units): its waves keep more bytes in flight.  Beyond, reading the
// cache once for all rows wins.  32 / 8 heads x 128, 4096 to 8192 tokens, e4m3, us
// here and there: 4 queries of 64 sequences 170 / 202, 8 of them 308 / 194; of 4
// sequences 8 queries 32 / 44, 16 queries 39 / 57.  Not for float32 rows of 256
// channels, which do not fit the other's registers.
constexpr int64_t FEW = 16384;
int64_t units_of(int B, int Hk, int64_t tiles, int64_t rows)
{
    return times((int64_t)B * Hk, times(tiles > 0 ? tiles : 1, (rows + 15) / 16));
}
bool is_few(int D, bool bf16, int64_t rows, int64_t units)
{
    return rows <= 16 || (D == 256 && !bf16) || (rows <= 64 && units <= FEW);
}

template <int D, bool BF, bool INT8> hipError_t launch(const AttendArgs &a, int n, hipStream_t stream)
{
    hipLaunchKernelGGL((kda_cache_attend_kernel<D, BF, INT8>), dim3(n), dim3(256), 0, stream, a, __builtin_ctz(a.page));
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_attend_join<16>(a, n, a.most * (a.Hq / a.Hk), stream);
}
template <int D, bool BF, bool INT8> hipError_t launch_rows(const AttendArgs &a, hipStream_t s)
{
    const int64_t rows = (int64_t)a.most * (a.Hq / a.Hk), tiles = ((int64_t)a.per * a.page + 63) / 64;
    if (!line_fits(tiles, (int64_t)a.tokens * (a.Hq / a.Hk), 16, a.B, a.Hk)) return hipErrorNotSupported;
    return launch<D, BF, INT8>(a, shares(units_of(a.B, a.Hk, tiles, rows), 512), s);
}
template <bool BF, bool INT8> hipError_t launch_d(const AttendArgs &a, hipStream_t s)
{
    return a.D == 64 ? launch_rows<64, BF, INT8>(a, s) : a.D == 128 ? launch_rows<128, BF, INT8>(a, s)
                                                                    : launch_rows<256, BF, INT8>(a, s);
}
template <int D, int ROWS> hipError_t join(const AttendArgs &a, int n, int rows, hipStream_t stream)
{
    const int used = rows < ROWS ? rows : ROWS;
    const dim3 grid((unsigned)n, (unsigned)((used + JOIN_ROWS<D> - 1) / JOIN_ROWS<D>));
    if (a.bf16) hipLaunchKernelGGL((kda_cache_attend_join_kernel<D, ROWS, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((kda_cache_attend_join_kernel<D, ROWS, false>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

template <int ROWS> hipError_t launch_attend_join(const AttendArgs &a, int n, int rows, hipStream_t stream)
{
    // `rows` is what the caller says that a sequence has: where the device knows of more, every row of a block may be in use
    if (a.q_start) rows = ROWS;
    return a.D == 64 ? join<64, ROWS>(a, n, rows, stream) : a.D == 128 ? join<128, ROWS>(a, n, rows, stream)
                                                                       : join<256, ROWS>(a, n, rows, stream);
}
template hipError_t launch_attend_join<64>(const AttendArgs &, int, int, hipStream_t);
template hipError_t launch_attend_join<128>(const AttendArgs &, int, int, hipStream_t);

int64_t cache_attend_workspace_floats(int tokens, int B, int Hq, int Hk, int D, int page, int per, int most)
{
    const int64_t rows = (int64_t)most * (Hq / Hk), tiles = ((int64_t)per * page + 63) / 64, units = units_of(B, Hk, tiles, rows);
    int64_t need = 0;
    for (const bool bf16 : {false, true}) {          // the size does not depend on the type
        int64_t x;
        if (is_few(D, bf16, rows, units)) x = shares(units, 512) * (int64_t)(sizeof(Record) / 4 + 2 * 16 * (D + 2));
        else x = attend_rows_workspace_floats(tokens, B, Hq, Hk, D, page, per, most);
        need = x > need ? x : need;
    }
    return need;
}

hipError_t launch_cache_attend(const AttendArgs &a, hipStream_t s)
{
    const int64_t rows = (int64_t)a.most * (a.Hq / a.Hk), tiles = ((int64_t)a.per * a.page + 63) / 64;
    if (!is_few(a.D, a.bf16, rows, units_of(a.B, a.Hk, tiles, rows))) return launch_attend_rows(a, s);
    if (a.bf16) return a.int8 ? launch_d<true, true>(a, s) : launch_d<true, false>(a, s);
    return a.int8 ? launch_d<false, true>(a, s) : launch_d<false, false>(a, s);
}

}  // namespace kda
