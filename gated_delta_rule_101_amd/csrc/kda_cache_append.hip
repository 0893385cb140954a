// Appending keys and values to the 8-bit paged cache for gfx950.
//
// For a page and head that tokens of the call go to, with m the largest
// magnitude among them and Q the largest code:
//   scale' = max(scale if the page goes on, m / Q),  code = round(x / scale'),
//   codes that were there: round(code scale / scale'), where the scale grew.
// A page goes on where the first place written is not its first.
//
// A workgroup has one head's keys or values and a run of `chunk` tokens; runs
// of tokens that share a page (neighbours in the call) belong to the chunk that
// holds their first token.  A run of up to SHORT tokens is a wave's: a decoding
// step has one token a page.  A longer one is the whole workgroup's: the rows
// stay in registers between the maximum and the codes, and values, whose pages
// hold tokens innermost, pass through LDS so that both are read and written in
// whole lines.  Each place takes the last of the call's tokens that name it.
// Bound by latency: 256 tokens of 8 heads x 128, a page each, 9.7 us; prompts of
// 19472 tokens 42 us, 2.8 TB/s (float32 51 us, 3.9).  At 256 channels and pages of 128
// the kernel of float32 rows and integers spills 84 bytes a lane.
#include "kda_attn.h"
#include "kda_block.h"
#include "kda_code8.h"

namespace kda {
namespace {

constexpr int SHORT = 8, MAX_PAGE = 128;

// Magnitudes are compared by their bits, where NaN stands above infinity.
__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ unsigned wave_max(unsigned x)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) x = max(x, (unsigned)__shfl_xor((int)x, m, 64));
    return x;
}

// The largest magnitude of a thread's values, as packed where they are bfloat16.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ unsigned most_of(const Pack<uint16_t, 8> &x, unsigned most)
{
    const uint32_t w[4] = {x.a.x, x.a.y, x.a.z, x.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        most = __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2, most),
                                                                      __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu)));
    return most;
}
__device__ __forceinline__ unsigned most_of(const Pack<float, 4> &x, unsigned most)
{
    most = max(max(most, magnitude(x.a.x)), magnitude(x.a.y));
    return max(max(most, magnitude(x.a.z)), magnitude(x.a.w));
}
template <typename T> __device__ __forceinline__ unsigned unpacked(unsigned most)
{
    return sizeof(T) == 4 ? most : max(most << 16, most & 0xffff0000u);
}

// The page's scale, and what its earlier codes are multiplied by (1: nothing).
struct Scale {
    float now, grown;
};
template <bool INT8> __device__ __forceinline__ Scale next_scale(float old, int first, unsigned most)
{
    if (first == 0) old = 0.f;
    const float m = __uint_as_float(most) * CODE_UNIT<INT8>;
    Scale s;
    s.now = __uint_as_float(max(__float_as_uint(old), __float_as_uint(m)));
    const float r = old / s.now;
    s.grown = first > 0 && fabsf(r) <= 3.4028235e38f ? r : 1.f;
    return s;
}
template <bool INT8> __device__ __forceinline__ uint32_t regrown(uint32_t byte, float grown)
{
    return to_code<INT8>(from_code<INT8>(byte) * grown);
}

// A run of few tokens in one page, by one wave: channels in the lanes.
template <typename T, int D, bool INT8, bool INNERMOST>
__device__ void append_short(const T *x, int64_t stride, const int *slots, int n, int page, uint8_t *codes, float *scale)
{
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    float v[SHORT][E];
    int at[SHORT];
    unsigned most = 0;
    int first = page;
#pragma unroll
    for (int t = 0; t < SHORT; ++t) {
        at[t] = -1;
        if (t < n) {
            at[t] = slots[t] & (page - 1);
            first = min(first, at[t]);
#pragma unroll
            for (int e = 0; e < E; ++e) v[t][e] = to_f32(x[(int64_t)t * stride + lane + 64 * e]);
        }
    }
#pragma unroll
    for (int t = 0; t < SHORT; ++t) {
        bool last = t < n;                     // no later token of the run names this place
#pragma unroll
        for (int u = t + 1; u < SHORT; ++u) last = last && at[u] != at[t];
        if (!last) at[t] = -1;
        if (at[t] >= 0)
#pragma unroll
            for (int e = 0; e < E; ++e) most = max(most, magnitude(v[t][e]));
    }
    const Scale s = next_scale<INT8>(*scale, first, wave_max(most));
    if (s.grown != 1.f) {
        if constexpr (!INNERMOST) {
            for (int i = 4 * lane; i < first * D; i += 256) {
                uint32_t w = *reinterpret_cast<const uint32_t *>(codes + i), r = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) r |= regrown<INT8>((w >> (8 * j)) & 0xff, s.grown) << (8 * j);
                *reinterpret_cast<uint32_t *>(codes + i) = r;
            }
        } else {
            // 16 places of a channel at once; only places in front of `first` are written
            const int parts = (first + 15) / 16;
            for (int i = lane; i < D * parts; i += 64) {
                const int d = i / parts, p0 = 16 * (i % parts);
                uint8_t *row = codes + d * page + p0;
                const uint4 w = *reinterpret_cast<const uint4 *>(row);
                uint32_t r[4] = {w.x, w.y, w.z, w.w};
                const int m = min(first - p0, 16);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < m) {
                        const int sh = 8 * (j & 3);
                        r[j / 4] = (r[j / 4] & ~(0xffu << sh)) | regrown<INT8>((r[j / 4] >> sh) & 0xff, s.grown) << sh;
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (4 * j + 4 <= m) reinterpret_cast<uint32_t *>(row)[j] = r[j];
                    else
                        for (int k = 4 * j; k < m; ++k) row[k] = (uint8_t)(r[j] >> (8 * (k & 3)));
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < SHORT; ++t)
        if (at[t] >= 0)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = lane + 64 * e;
                codes[INNERMOST ? d * page + at[t] : at[t] * D + d] = (uint8_t)to_code<INT8>(v[t][e] / s.now);
            }
    if (lane == 0) *scale = s.now;
}

// Codes of 4 values at one scale, a word.  The quotients are rounded as the
// division is: q = x r with r = 1 / s rounded, then one step on the exact
// remainder; none is beyond the largest code by more than its rounding.  Plain
// division and checked codes where r or a remainder would leave the normal
// numbers, or the scale is none.
template <bool INT8> struct Coder {
    float s, r;
    bool easy;
    __device__ __forceinline__ explicit Coder(float s_) : s(s_), r(1.f / s_), easy(s_ > 0x1p-90f && s_ < 0x1p90f) {}
    __device__ __forceinline__ uint32_t word(const float *x) const
    {
        uint32_t k[4];
        if (!easy) {
#pragma unroll
            for (int i = 0; i < 4; ++i) k[i] = to_code<INT8>(x[i] / s);
            return k[0] | k[1] << 8 | k[2] << 16 | k[3] << 24;
        }
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = x[i] * r;
            q[i] = __builtin_fmaf(__builtin_fmaf(-q[i], s, x[i]), r, q[i]);
        }
        if constexpr (INT8) {
            // at 1.5 * 2^23 an integer is in the low bits, rounded to even
#pragma unroll
            for (int i = 0; i < 4; ++i) k[i] = __float_as_uint(q[i] + 12582912.f);
            const uint32_t a = __builtin_amdgcn_perm(k[1], k[0], 0x0c0c0400u), b = __builtin_amdgcn_perm(k[3], k[2], 0x0c0c0400u);
            return a | b << 16;
        } else {
            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
            return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
        }
    }
};

// A longer run, by the workgroup: a thread has V channels of 4 neighbouring
// places.  LDS: source[place], the maximum's parts and, for values, the page's
// new codes, a word of 4 places at a time.  next: the first token's place where
// the tokens stand one after the other, as a sequence's do, -1 otherwise: only
// then are their places looked up.
template <typename T, int D, bool INT8, bool INNERMOST, int MOST>
__device__ void append_long(const T *x, int64_t stride, const int *slots, int n, int page, uint8_t *codes, float *scale,
                            int next, int *source, unsigned *part, uint32_t *tile)
{
    constexpr int V = WIDE<T>, L = D / V, PLACES = 4 * (256 / L), ITERS = (MOST + PLACES - 1) / PLACES;
    const int tid = threadIdx.x, lane = tid & 63, d0 = V * (tid % L), q0 = 4 * (tid / L);
    const int pitch = page / 4 + 1;          // words of a channel's row in the tile: odd, for the banks
    const bool wide = !(stride % V) && !((uintptr_t)x & 15);
    const float old = *scale;
    uint64_t lo, hi;                         // the places written, as bits
    if (next >= 0) {
        const auto ones = [](int k) { return k >= 64 ? ~0ull : k <= 0 ? 0ull : (1ull << k) - 1; };
        lo = ones(next + n) & ~ones(next);
        hi = ones(next + n - 64) & ~ones(next - 64);
    } else {
        if (tid < MAX_PAGE) source[tid] = -1;
        __syncthreads();
        for (int t = tid; t < n; t += 256) atomicMax(&source[slots[t] & (page - 1)], t);
        __syncthreads();
        lo = __ballot(lane < page && source[lane] >= 0);
        hi = __ballot(64 + lane < page && source[64 + lane] >= 0);
    }
    const int first = lo ? __builtin_ctzll(lo) : 64 + __builtin_ctzll(hi);
    Pack<T, V> raw[ITERS][4];
    unsigned most = 0;
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int p = i * PLACES + q0 + j;
            raw[i][j].zero();
            if (p < page && ((p < 64 ? lo >> p : hi >> (p - 64)) & 1)) {
                const int from = next >= 0 ? p - next : source[p];
                const T *row = x + (int64_t)from * stride + d0;
                if (wide) {
                    raw[i][j].stream(row);
                } else {
                    T e[V];
#pragma unroll
                    for (int c = 0; c < V; ++c) e[c] = row[c];
                    __builtin_memcpy(&raw[i][j], e, sizeof(e));
                }
            }
        }
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) most = most_of(raw[i][j], most);
    most = wave_max(unpacked<T>(most));
    if (lane == 0) part[tid / 64] = most;
    __syncthreads();
    most = max(max(part[0], part[1]), max(part[2], part[3]));
    const Scale s = next_scale<INT8>(old, first, most);
    const Coder<INT8> by(s.now);
    if (tid == 0) *scale = s.now;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int p = i * PLACES + q0;
        const unsigned fresh = (unsigned)((p < 64 ? lo >> p : hi >> (p - 64)) & 15);
        if (p >= page || !fresh) continue;
        uint32_t w[4][V / 4];                // by place, 4 channels a word
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[V];
            raw[i][j].to_f32(v);
#pragma unroll
            for (int c = 0; c < V; c += 4) w[j][c / 4] = by.word(v + c);
        }
        if constexpr (INNERMOST) {
            // 4 x 4 bytes turned: a channel's 4 places in a word
#pragma unroll
            for (int c = 0; c < V; c += 4) {
                const uint32_t a0 = w[0][c / 4], a1 = w[1][c / 4], a2 = w[2][c / 4], a3 = w[3][c / 4];
                const uint32_t b0 = __builtin_amdgcn_perm(a1, a0, 0x05010400u), b1 = __builtin_amdgcn_perm(a1, a0, 0x07030602u);
                const uint32_t b2 = __builtin_amdgcn_perm(a3, a2, 0x05010400u), b3 = __builtin_amdgcn_perm(a3, a2, 0x07030602u);
                uint32_t *to = tile + (d0 + c) * pitch + p / 4;
                to[0] = __builtin_amdgcn_perm(b2, b0, 0x05040100u);
                to[pitch] = __builtin_amdgcn_perm(b2, b0, 0x07060302u);
                to[2 * pitch] = __builtin_amdgcn_perm(b3, b1, 0x05040100u);
                to[3 * pitch] = __builtin_amdgcn_perm(b3, b1, 0x07060302u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (fresh >> j & 1) {
                    uint32_t *to = reinterpret_cast<uint32_t *>(codes + (p + j) * D + d0);
#pragma unroll
                    for (int c = 0; c < V / 4; ++c) to[c] = w[j][c];
                }
        }
    }
    if constexpr (!INNERMOST) {
        if (s.grown != 1.f)
            for (int i = 4 * tid; i < first * D; i += 1024) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + i);
                uint32_t r = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) r |= regrown<INT8>((w >> (8 * j)) & 0xff, s.grown) << (8 * j);
                *reinterpret_cast<uint32_t *>(codes + i) = r;
            }
    } else {
        __syncthreads();
        // 16 places of a channel at once, merged with what is there unless all are new
        const int parts = page / 16, bits = __builtin_ctz(parts);
        for (int i = tid; i < D * parts; i += 256) {
            const int d = i >> bits, p0 = 16 * (i & (parts - 1));
            uint8_t *row = codes + d * page + p0;
            const unsigned fresh = (unsigned)((p0 < 64 ? lo >> p0 : hi >> (p0 - 64)) & 0xffff);
            if (!fresh && (p0 >= first || s.grown == 1.f)) continue;
            uint32_t now[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) now[j] = tile[d * pitch + p0 / 4 + j];
            if (fresh != 0xffffu) {
                const uint4 w = *reinterpret_cast<const uint4 *>(row);
                const uint32_t was[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (fresh >> j & 1) continue;
                    const int sh = 8 * (j & 3);
                    uint32_t b = (was[j / 4] >> sh) & 0xff;
                    if (p0 + j < first && s.grown != 1.f) b = regrown<INT8>(b, s.grown);
                    now[j / 4] = (now[j / 4] & ~(0xffu << sh)) | b << sh;
                }
            }
            *reinterpret_cast<uint4 *>(row) = make_uint4(now[0], now[1], now[2], now[3]);
        }
    }
    __syncthreads();   // source, part and tile are the next run's
}

// Blocks: chunks of tokens x heads x {keys, values}.  MOST: tokens a page, at
// most, for which a thread has registers.
template <typename T, int D, bool INT8, int MOST>
__global__ void __launch_bounds__(256, D <= 128 && MOST <= 64 ? 4 : 1) kda_cache_append_kernel(AppendArgs a, int chunk)
{
    extern __shared__ __align__(16) uint32_t tile[];
    __shared__ int source[MAX_PAGE];
    __shared__ unsigned part[4];
    const int h = blockIdx.y >> 1, wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    const bool values = blockIdx.y & 1;
    const int t0 = blockIdx.x * chunk;
    const int shift = __builtin_ctz(a.page);
    const unsigned places = (unsigned)a.pages * (unsigned)a.page;     // below 2^31
    const auto slot_of = [&](int t) {
        const int s = t >= 0 && t < a.tokens ? a.slots[t] : -1;
        return (unsigned)s < places ? s : -1;
    };
    const auto page_of = [&](int t) { return slot_of(t) >> shift; };        // -1 stays
    // lane i looks at token t0 - 1 + i: runs of this chunk start where the page is another than the token's before
    const int slot = slot_of(t0 - 1 + lane), id = slot >> shift, before = __shfl_up(id, 1, 64);
    uint64_t starts = __ballot(lane > 0 && lane <= chunk && id >= 0 && id != before);
    const uint64_t breaks = __ballot(lane > 0 && id != before);
    const T *const x = (const T *)(values ? a.v : a.k) + (int64_t)h * D;
    const int64_t stride = values ? a.v_stride : a.k_stride;
    for (int runs = 0; starts; starts &= starts - 1) {
        const int at = __builtin_ctzll(starts), t = t0 - 1 + at, page = __builtin_amdgcn_readlane(id, at);
        // the run's length: to the next break in sight, or further
        const uint64_t rest = at < 63 ? breaks >> (at + 1) : 0;
        int n = rest ? 1 + __builtin_ctzll(rest) : 64 - at;
        if (!rest)
            while (true) {
                const uint64_t other = __ballot(page_of(t + n + lane) != page);
                n += other ? __builtin_ctzll(other) : 64;
                if (other) break;
            }
        // slots one after the other, as far as the lanes see all of the run
        const uint64_t run = at + n <= 64 ? (n >= 64 ? ~0ull : (1ull << n) - 1) << at : 0;
        const int at_slot = __builtin_amdgcn_readlane(slot, at);
        const bool orderly = run && !(__ballot(slot - lane != at_slot - at) & run);
        const T *from = x + (int64_t)t * stride;
        const int64_t head = (int64_t)page * a.Hk + h;
        uint8_t *codes = (values ? a.v_codes : a.k_codes) + head * a.page * D;
        float *scale = (values ? a.v_scale : a.k_scale) + head;
        if (n <= SHORT) {
            if ((runs++ & 3) == wave) {
                if (values) append_short<T, D, INT8, true>(from, stride, a.slots + t, n, a.page, codes, scale);
                else append_short<T, D, INT8, false>(from, stride, a.slots + t, n, a.page, codes, scale);
            }
        } else {
            if (values) append_long<T, D, INT8, true, MOST>(from, stride, a.slots + t, n, a.page, codes, scale, orderly ? at_slot & (a.page - 1) : -1, source, part, tile);
            else append_long<T, D, INT8, false, MOST>(from, stride, a.slots + t, n, a.page, codes, scale, orderly ? at_slot & (a.page - 1) : -1, source, part, tile);
        }
    }
}

template <typename T, int D, bool INT8> hipError_t launch(const AppendArgs &a, hipStream_t stream)
{
    // Chunks of 4 to 62 tokens for 4096 workgroups or more: a decoding step's tokens
    // are a page each, and a wave takes one after the other; of a prompt's chunks
    // those that begin no page have nothing to do (19472 tokens of 8 heads, us with
    // chunks of up to 8, 16, 48 and 62: pages of 64 47, 45, 38 and 42, of 16 91, 83,
    // 75 and 74).
    const int64_t lanes = 2 * (int64_t)a.Hk, even = a.tokens * lanes / 4096;
    const int chunk = (int)(even < 4 ? 4 : even > 62 ? 62 : even);
    const int64_t blocks = ((int64_t)a.tokens + chunk - 1) / chunk;
    if (!grid_fits(blocks, 256) || lanes > 65535) return hipErrorNotSupported;
    const dim3 grid((unsigned)blocks, (unsigned)lanes);
    const size_t lds = (size_t)D * (a.page + 4);
    if (a.page <= 64) hipLaunchKernelGGL((kda_cache_append_kernel<T, D, INT8, 64>), grid, dim3(256), lds, stream, a, chunk);
    else hipLaunchKernelGGL((kda_cache_append_kernel<T, D, INT8, 128>), grid, dim3(256), lds, stream, a, chunk);
    return hipGetLastError();
}
template <typename T, bool INT8> hipError_t launch_d(const AppendArgs &a, hipStream_t s)
{
    return a.D == 64 ? launch<T, 64, INT8>(a, s) : a.D == 128 ? launch<T, 128, INT8>(a, s) : launch<T, 256, INT8>(a, s);
}

}  // namespace

hipError_t launch_cache_append(const AppendArgs &a, hipStream_t s)
{
    if (a.bf16) return a.int8 ? launch_d<uint16_t, true>(a, s) : launch_d<uint16_t, false>(a, s);
    return a.int8 ? launch_d<float, true>(a, s) : launch_d<float, false>(a, s);
}

}  // namespace kda
