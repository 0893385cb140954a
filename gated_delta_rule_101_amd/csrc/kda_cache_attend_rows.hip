// Attention over the 8-bit paged cache for gfx950, for many query rows a
// sequence: prompts, and drafts of grouped heads.  The formulas and float16
// forms are those of kda_cache_attend.hip.
//
// A workgroup has 32 rows (query, head of the group) a wave, of one sequence and
// key head, and walks the tokens 64 at a time.  Bound by the matrix cores and,
// as much, by the softmax between its two products, so codes are turned into
// float16 once a workgroup: the next tile's bytes are requested before this
// tile's products and go to the other half of LDS, as float16, behind them.
//
// 32x32x16 products of the transposed score tile: a lane holds scores of one row
// (its column) and, by the order in which LDS holds the keys, 8 neighbouring
// tokens of each 16, which are the second product's inner index as they stand.
// Values are innermost in tokens in their pages, so that product's other operand
// is 16 bytes of a channel's row.  LDS rows are padded by 16 bytes: lanes read
// down the rows.
//
// Where blocks of rows are many, each is a workgroup, the last ones (the
// longest) first, heads innermost so that workgroups of one head share an L2.
// Where they are few, the line of units is cut into shares as for single
// queries.
//
// 3 prompt chunks of up to 4096 tokens behind as many, 32 and 8 heads x 128, e4m3:
// 0.99 ms, 0.89 PFLOP/s (float32 2.1 ms); 16 drafts of 24 sequences of 8192 to 16384 tokens, integers:
// 0.17 ms, 3.6 TB/s.
#include "kda_attn.h"
#include "kda_block.h"
#include "kda_attend_device.h"

namespace kda {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int D> struct Tile {
    static constexpr int KSTRIDE = 2 * D + 16, VSTRIDE = 2 * 64 + 16;      // bytes
    uint8_t k[64 * KSTRIDE], v[D * VSTRIDE];
};

__device__ __forceinline__ float halves_max(float x)
{
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float halves_sum(float x)
{
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// The LDS row of a tile's token: the score product's row whose result a lane
// half h holds as the (4 b + c)th value is 8 b + 4 h + c, and is to be token
// 16 (b / 2) + 8 h + 4 (b & 1) + c.
__device__ __forceinline__ int key_row(int t) { return (t & 0x33) | (t & 8) >> 1 | (t & 4) << 1; }

// A tile's bytes on their way from memory to LDS: each thread 16-byte parts.  A
// wave's keys of one part are of one 16-token group, so their page is a scalar;
// values' groups, the scales and the pages' numbers go by lane & 3.  Pages are
// looked up a tile ahead of the codes.
template <int D, int WAVES, bool INT8> struct Loader {
    static constexpr int THREADS = 64 * WAVES, PARTS = 4 * D / THREADS;    // of keys, and of values
    uint4 k[PARTS], v[PARTS];
    float ks, lv;                            // key scale, log2 of the value scale
    int there, broken;                       // by group: has a page, its value scale is not finite
    int page, ahead;                         // of the tile whose codes are next to be requested, of the one behind
    // thread's part i of the keys: token, 16 channels from c; of the values: channel, group of 16 tokens
    static __device__ __forceinline__ int key_token(int i) { return (threadIdx.x + i * THREADS) / (D / 16); }
    static __device__ __forceinline__ int key_part(int i) { return (threadIdx.x + i * THREADS) % (D / 16); }
    static __device__ __forceinline__ int key_group(int i) { return uniform(key_token(i) / 16); }
    static __device__ __forceinline__ int channel(int i) { return (threadIdx.x + i * THREADS) / 4; }
    __device__ __forceinline__ void look_up(const AttendArgs &a, const int *table, int t0, int context, int shift)
    {
        page = ahead;
        ahead = page_of(a, table, t0 + 16 * (threadIdx.x & 3), context, shift);
    }
    __device__ __forceinline__ void load(const AttendArgs &a, int h, int t0, int context)
    {
        const int in = a.page - 1, id = max(page, 0);
        const int64_t at = (int64_t)id * a.Hk + h, bytes = (int64_t)a.page * D;
        ks = a.k_scale[at];
        lv = a.v_scale[at];
        if (a.page >= 64) {                  // the tile is of one page: scalar bases
            const int64_t from = ((int64_t)uniform(id) * a.Hk + h) * bytes;
            const uint8_t *kb = a.k_codes + from + (t0 & in) * D, *vb = a.v_codes + from + (t0 & in);
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
                k[i] = *reinterpret_cast<const uint4 *>(kb + (uint32_t)(key_token(i) * D + 16 * key_part(i)));
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
                v[i] = *reinterpret_cast<const uint4 *>(vb + (uint32_t)(channel(i) * a.page + 16 * (threadIdx.x & 3)));
        } else {
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                const int g = key_group(i);
                const uint8_t *kb = a.k_codes + ((int64_t)__builtin_amdgcn_readlane(id, g) * a.Hk + h) * bytes + ((t0 + 16 * g) & in) * D;
                k[i] = *reinterpret_cast<const uint4 *>(kb + (uint32_t)((key_token(i) & 15) * D + 16 * key_part(i)));
            }
            const uint8_t *vb = a.v_codes + at * bytes + ((t0 + 16 * (threadIdx.x & 3)) & in);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) v[i] = *reinterpret_cast<const uint4 *>(vb + (uint32_t)(channel(i) * a.page));
        }
        there = (int)__ballot(page >= 0) & 15;
        if (!INT8 && (t0 + 64 > context || there != 15)) {
            // no NaN where the weight is zero
            const int n = page < 0 ? 0 : context - (t0 + 16 * (threadIdx.x & 3));
#pragma unroll
            for (int i = 0; i < PARTS; ++i) v[i] = keep_bytes(v[i], n);
        }
    }
    // behind the loads' arrival
    __device__ __forceinline__ void scales()
    {
        const bool fine = is_finite(lv);
        const bool has = there >> (threadIdx.x & 3) & 1;
        broken = (int)__ballot(has && !fine) & 15;
        lv = fine && has ? fast_log2(lv) : -__builtin_inff();
        ks = !has ? 0.f : is_finite(ks) ? ks : __builtin_nanf("");   // infinite: not a weight of 0 where the product is negative
    }
    __device__ __forceinline__ void put(Tile<D> &tile) const
    {
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
            uint8_t *to = tile.k + key_row(key_token(i)) * Tile<D>::KSTRIDE + 32 * key_part(i);
            *reinterpret_cast<f16x8 *>(to) = codes_f16<INT8>(k[i].x, k[i].y);
            *reinterpret_cast<f16x8 *>(to + 16) = codes_f16<INT8>(k[i].z, k[i].w);
        }
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
            uint8_t *to = tile.v + channel(i) * Tile<D>::VSTRIDE + 32 * (threadIdx.x & 3);
            *reinterpret_cast<f16x8 *>(to) = codes_f16<INT8>(v[i].x, v[i].y);
            *reinterpret_cast<f16x8 *>(to + 16) = codes_f16<INT8>(v[i].z, v[i].w);
        }
    }
};
__device__ __forceinline__ float lane_value(float x, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

// Tiles of a workgroup's LDS: two, and one barrier a tile; one where workgroups
// are of two waves, so that four of them fit a CU.
template <int WAVES> constexpr int TILES = WAVES == 2 ? 1 : 2;

// LINE: shares of the line of units; otherwise a workgroup a block of rows.
template <int D, int WAVES, bool BF, bool INT8, bool LINE>
__global__ void __launch_bounds__(64 * WAVES, D == 256 || (D == 128 && !BF) ? 1 : 2) kda_cache_attend_rows_kernel(AttendArgs a, int shift)
{
    constexpr int SPLIT = BF ? 1 : 2, KS = D / 16, DT = D / 32, ROWS = 32 * WAVES, BUFFERS = TILES<WAVES>;
    typedef typename Store<BF>::type T;
    extern __shared__ __align__(16) uint8_t lds[];
    Tile<D> *const tiles_lds = reinterpret_cast<Tile<D> *>(lds);
    __shared__ unsigned part[WAVES];
    const int wave = uniform((int)threadIdx.x / 64), lane = threadIdx.x & 63, m = lane & 31, half = lane >> 5;
    const int G = a.Hq / a.Hk;
    Line line;
    int b, h, block, t_begin = 0, t_end;
    if constexpr (LINE) {
        line = cut_line<WAVES>(a, G, ROWS, 1, part);
    } else {
        // the block's place among all sequences' blocks, sequence b's being counted from q_start[b] G / ROWS + b
        const int64_t blocks = gridDim.x / a.Hk, at = blocks - 1 - blockIdx.x / a.Hk;
        h = blockIdx.x % a.Hk;
        int n = 0;
        for (int b0 = 0; b0 < a.B; b0 += 64) {
            const bool upto = b0 + lane < a.B && (int64_t)sequence(a, min(b0 + lane, a.B - 1)).first * G / ROWS + b0 + lane <= at;
            const uint64_t past = ~__ballot(upto);
            n = b0 + (past ? __builtin_ctzll(past) : 64);
            if (past) break;
        }
        if (n == 0) return;                              // rows in front of the first sequence
        b = uniform(min(n, a.B) - 1);
        const Sequence s = sequence(a, b);
        block = (int)(at - ((int64_t)s.first * G / ROWS + b));
        if (block >= blocks_of(s, G, ROWS)) return;
    }
    Record mine = {0, 0, 0, -1};
    while (!LINE || line.left > 0) {
        Sequence s;
        int tiles;
        if constexpr (LINE) {
            s = sequence(a, line.b);
            tiles = tiles_of(s);
            const int blocks = blocks_of(s, G, ROWS);
            if ((unsigned)line.u >= (unsigned)tiles * blocks * a.Hk) {
                line.u = 0;
                if (++line.b >= a.B) break;         // the line ends with the last sequence
                continue;
            }
            b = line.b;
            const int row = (unsigned)line.u / (unsigned)tiles;
            t_begin = line.u - row * tiles;
            t_end = min(tiles, t_begin + line.left);
            h = row / blocks;
            block = row - h * blocks;
        } else {
            s = sequence(a, b);
            tiles = t_end = tiles_of(s);
        }
        const int r0 = block * ROWS, active = min(ROWS, s.queries * G - r0);
        const int furthest = min(s.context, s.context - s.queries + (r0 + active - 1) / G + 1);
        const int t_stop = min(t_end, (furthest + 63) / 64);       // tiles behind it are seen by no row

        // this wave's rows
        const int w0 = 32 * wave, r = w0 + m, qi = (r0 + min(r, active - 1)) / G, qg = (r0 + min(r, active - 1)) - qi * G;
        const int limit = r < active ? min(s.context - s.queries + qi + 1, s.context) : 0x7fffffff;
        const int whole = min(s.context - s.queries + (r0 + min(w0, active - 1)) / G + 1, s.context);
        f16x8 q[SPLIT][KS];
        const float factor = load_row<T, D, SPLIT>((const T *)a.q + ((int64_t)(s.first + qi) * a.Hq + h * G + qg) * D,
                                                   r < active, half, a.scale < 0.f, q) * fabsf(a.scale) * LOG2E;
        f32x16 o[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
        float top = -__builtin_inff(), sum = 0.f, lift = -__builtin_inff(), spoiled = 0.f;

        const int *table = a.table + (int64_t)b * a.per;
        Loader<D, WAVES, INT8> next;
        if (t_begin < t_stop) {
            next.look_up(a, table, t_begin * 64, s.context, shift);
            next.look_up(a, table, t_begin * 64 + 64, s.context, shift);
            next.load(a, h, t_begin * 64, s.context);
            next.put(tiles_lds[0]);
        }
        __syncthreads();
        for (int t = t_begin; t < t_stop; ++t) {
            const Tile<D> &tile = tiles_lds[BUFFERS == 2 ? (t - t_begin) & 1 : 0];
            const int t0 = t * 64;
            // this tile's scales, by group
            next.scales();
            float ks[4], lv[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                ks[g] = lane_value(next.ks, g);
                lv[g] = lane_value(next.lv, g);
            }
            const int there = next.there, broken = next.broken;
            if (t + 1 < t_stop) {
                next.look_up(a, table, t0 + 128, s.context, shift);
                next.load(a, h, t0 + 64, s.context);
            }

            f32x16 x[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[j][i] = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const f16x8 c = *reinterpret_cast<const f16x8 *>(tile.k + (32 * j + m) * Tile<D>::KSTRIDE + 32 * k + 16 * half);
#pragma unroll
                    for (int p = 0; p < SPLIT; ++p) x[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(c, q[p][k], x[j], 0, 0, 0);
                }
            }
            // scores to weights, in place
            float c[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) c[g] = factor * ks[g];
            if (t0 + 64 > whole || there != 15) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int seen = there >> g & 1 ? limit - (t0 + 16 * g + 8 * half) : 0;       // of 8 tokens
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[g >> 1][8 * (g & 1) + i] = i < seen ? x[g >> 1][8 * (g & 1) + i] * c[g] : -__builtin_inff();
                    c[g] = 1.f;
                }
            }
            float best = -__builtin_inff(), most = -__builtin_inff();     // of the scores, and with the value scales
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float y = x[g >> 1][8 * (g & 1)];
#pragma unroll
                for (int i = 1; i < 8; ++i) y = fmaxf(y, x[g >> 1][8 * (g & 1) + i]);
                y *= c[g];
                best = fmaxf(best, y);
                most = fmaxf(most, y + lv[g]);
            }
            best = halves_max(best);
            most = halves_max(most);
            // A base that is up to SLACK below the maximum serves as well: outputs then move rarely.
            if (__any(best > top + SLACK)) {
                const float now = fmaxf(top, best), back = now == -__builtin_inff() ? 0.f : top - now;
                top = now;
                sum *= fast_exp2(back);
                lift += back;                    // the outputs' unit, 2^(top + lift), stays
            }
            float base = held(top);
            if (__any(fabsf(base) > FAR)) {
                const bool far = fabsf(base) > FAR;                      // other rows stay as they are
                float from = -__builtin_inff();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float was = x[g >> 1][8 * (g & 1) + i], z = from_base(was * c[g], base);
                        x[g >> 1][8 * (g & 1) + i] = far ? z : was;
                        from = fmaxf(from, z + lv[g]);
                    }
                    c[g] = far ? 1.f : c[g];
                }
                from = halves_max(from);
                most = far ? from : most;
                base = far ? 0.f : base;
            }
            most -= base;
            if (__any(most > lift + SLACK)) {
                const float now = fmaxf(lift, most), fade = now == -__builtin_inff() ? 1.f : fast_exp2(lift - now);
                lift = now;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[d][i] *= fade;
            }
            const float lift_of = held(lift);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float rel = relative_level(lv[g], lift_of), offset = rel - base;
                float total = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = fast_exp2(__builtin_fmaf(x[g >> 1][8 * (g & 1) + i], c[g], offset));
                    x[g >> 1][8 * (g & 1) + i] = v;
                    total += v;
                }
                sum = __builtin_fmaf(total, fast_exp2(-rel), sum);
            }
            if (broken) {                        // a value scale that is not finite: NaN for the rows that see its tokens
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    spoiled = broken >> g & 1 && limit > t0 + 16 * g + 8 * half ? __builtin_nanf("") : spoiled;
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = x[g >> 1][8 * (g & 1) + i];
                f16x8 w[SPLIT];
                split_f16<SPLIT>(v, [&](int p) -> f16x8 & { return w[p]; });
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const f16x8 c = *reinterpret_cast<const f16x8 *>(tile.v + (32 * d + m) * Tile<D>::VSTRIDE + 32 * g + 16 * half);
#pragma unroll
                    for (int p = 0; p < SPLIT; ++p) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(c, w[p], o[d], 0, 0, 0);
                }
            }
            if (BUFFERS == 1) __syncthreads();
            if (t + 1 < t_stop) next.put(tiles_lds[BUFFERS == 2 ? (t + 1 - t_begin) & 1 : 0]);
            __syncthreads();
        }

        sum = halves_sum(sum);
        const bool whole_row = t_begin == 0 && t_end == tiles;
        const float f = fast_exp2(lift) + halves_sum(spoiled);           // 0 where every value was
        float *piece = nullptr;
        if constexpr (LINE) {
            piece = a.ws + (sizeof(Record) / 4) * gridDim.x + (int64_t)(2 * blockIdx.x + (t_begin == 0)) * PIECE<D, ROWS>;
            if (t_begin == 0 && !whole_row) mine = {b, h, block, line.last(tiles)};
            line.u += t_end - t_begin;
            line.left -= t_end - t_begin;
            line.at += t_end - t_begin;
        }
        if (r < active) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = 32 * d + 8 * i + 4 * half;
                    const float y[4] = {o[d][4 * i] * VALUE_REST * f, o[d][4 * i + 1] * VALUE_REST * f,
                                        o[d][4 * i + 2] * VALUE_REST * f, o[d][4 * i + 3] * VALUE_REST * f};
                    if (!LINE || whole_row) write_row<T>(a, s, h, G, r0 + r, at, D, y, top, sum);
                    else *reinterpret_cast<float4 *>(piece + (int64_t)r * D + at) = make_float4(y[0], y[1], y[2], y[3]);
                }
            if (LINE && !whole_row && half == 0) {
                piece[ROWS * D + r] = top;
                piece[ROWS * D + ROWS + r] = sum;
            }
        }
        if constexpr (!LINE) return;
        __syncthreads();
    }
    if (LINE && threadIdx.x == 0) reinterpret_cast<Record *>(a.ws)[blockIdx.x] = mine;
}

// How a call is run: waves a workgroup, and whether its line is cut.
struct Shape {
    int waves, workgroups;
    bool line;
};
Shape shape_of(int tokens, int B, int Hq, int Hk, int D, int page, int per, int most)
{
    Shape s;
    const int64_t rows = (int64_t)most * (Hq / Hk), tiles = ((int64_t)per * page + 63) / 64;
    s.waves = D == 256 ? 4 : rows <= 64 ? 2 : 4;
    // blocks of all sequences, at most (as the kernel counts them)
    const int64_t blocks = ((int64_t)tokens * (Hq / Hk) / (32 * s.waves) + B) * Hk;
    // A line where blocks are few and the table holds several times the queries: its
    // rows of units are taken as equally long, so a prompt's causal corner is better
    // left to the hardware's order (32 / 8 heads x 128, us as a line and by blocks:
    // 512 new of 512 tokens 36 / 22, 1000 of 1000 46 / 37, twice 1000 of 3000 132 /
    // 125; 256 of 4096 65 / 118, 512 of 16384 200 / 494, 8 x 500 of 4000 249 / 254).
    s.line = blocks < 1024 && tiles * 64 >= 4 * (int64_t)most && line_fits(tiles, (int64_t)tokens * (Hq / Hk), 32 * s.waves, B, Hk);
    s.workgroups = s.line ? shares(blocks * (tiles > 0 ? tiles : 1), s.waves == 2 ? 1024 : D == 256 ? 256 : 512) : blocks < ((int64_t)1 << 24) ? (int)blocks : 0;
    return s;
}

template <int D, int WAVES, bool BF, bool INT8> hipError_t launch(const AttendArgs &a, const Shape &s, hipStream_t stream)
{
    const int shift = __builtin_ctz(a.page);
    const size_t bytes = TILES<WAVES> * sizeof(Tile<D>);
    const dim3 grid((unsigned)s.workgroups), threads(64 * WAVES);
    const auto set = [&](const void *k) { return hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes); };
    if (!s.line) {
        const auto k = kda_cache_attend_rows_kernel<D, WAVES, BF, INT8, false>;
        const hipError_t e = set(reinterpret_cast<const void *>(k));
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k, grid, threads, bytes, stream, a, shift);
        return hipGetLastError();
    }
    const auto k = kda_cache_attend_rows_kernel<D, WAVES, BF, INT8, true>;
    hipError_t e = set(reinterpret_cast<const void *>(k));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, grid, threads, bytes, stream, a, shift);
    e = hipGetLastError();
    return e != hipSuccess ? e : launch_attend_join<32 * WAVES>(a, s.workgroups, 32 * WAVES, stream);
}
template <bool BF, bool INT8> hipError_t launch_d(const AttendArgs &a, const Shape &s, hipStream_t stream)
{
    if (a.D == 64) return s.waves == 2 ? launch<64, 2, BF, INT8>(a, s, stream) : launch<64, 4, BF, INT8>(a, s, stream);
    if (a.D == 128) return s.waves == 2 ? launch<128, 2, BF, INT8>(a, s, stream) : launch<128, 4, BF, INT8>(a, s, stream);
    if constexpr (BF) return launch<256, 4, BF, INT8>(a, s, stream);
    return hipErrorNotSupported;             // those rows are the other kernel's
}

}  // namespace

int64_t attend_rows_workspace_floats(int tokens, int B, int Hq, int Hk, int D, int page, int per, int most)
{
    const Shape s = shape_of(tokens, B, Hq, Hk, D, page, per, most);
    return s.line ? (int64_t)s.workgroups * (int64_t)(sizeof(Record) / 4 + 2 * 32 * s.waves * (D + 2)) : 0;
}

hipError_t launch_attend_rows(const AttendArgs &a, hipStream_t stream)
{
    const Shape s = shape_of(a.tokens, a.B, a.Hq, a.Hk, a.D, a.page, a.per, a.most);
    if (s.workgroups == 0) return hipErrorNotSupported;
    if (a.bf16) return a.int8 ? launch_d<true, true>(a, s, stream) : launch_d<true, false>(a, s, stream);
    return a.int8 ? launch_d<false, true>(a, s, stream) : launch_d<false, false>(a, s, stream);
}

}  // namespace kda
