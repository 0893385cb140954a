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
// Bound by HBM bandwidth for prompts, by latency for single tokens.
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

// A longer run, by the workgroup.  LDS: source[place], the maximum's parts, and
// for values the page's new codes.
template <typename T, int D, bool INT8, bool INNERMOST>
__device__ void append_long(const T *x, int64_t stride, const int *slots, int n, int page, uint8_t *codes, float *scale,
                            int *source, unsigned *part, uint8_t *tile)
{
    constexpr int V = WIDE<T>, L = D / V, ROWS = 256 / L, ITERS = MAX_PAGE / ROWS;
    const int tid = threadIdx.x, d0 = V * (tid % L);
    const bool wide = !(stride % V) && !((uintptr_t)x & 15);
    if (tid < MAX_PAGE) source[tid] = -1;
    __syncthreads();
    int first = page;
    for (int t = tid; t < n; t += 256) atomicMax(&source[slots[t] & (page - 1)], t);
    __syncthreads();
    // the first place written, and the rows' largest magnitude
    Pack<T, V> raw[ITERS];
    unsigned most = 0;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int p = i * ROWS + tid / L;
        raw[i].zero();
        if (p < page && source[p] >= 0) {
            const T *row = x + (int64_t)source[p] * stride + d0;
            if (wide) {
                raw[i].load(row);
            } else {
                T e[V];
#pragma unroll
                for (int c = 0; c < V; ++c) e[c] = row[c];
                __builtin_memcpy(&raw[i], e, sizeof(e));
            }
        }
    }
    for (int p = tid & 63; p < page; p += 64)
        if (source[p] >= 0) {
            first = p;
            break;
        }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) first = min(first, __shfl_xor(first, m, 64));
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        float v[V];
        raw[i].to_f32(v);
#pragma unroll
        for (int c = 0; c < V; ++c) most = max(most, magnitude(v[c]));
    }
    most = wave_max(most);
    if ((tid & 63) == 0) part[tid / 64] = most;
    const float old = *scale;
    __syncthreads();
    most = max(max(part[0], part[1]), max(part[2], part[3]));
    const Scale s = next_scale<INT8>(old, first, most);
    if (tid == 0) *scale = s.now;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int p = i * ROWS + tid / L;
        if (p >= page || source[p] < 0) continue;
        float v[V];
        raw[i].to_f32(v);
        uint32_t w[(V + 3) / 4] = {};
#pragma unroll
        for (int c = 0; c < V; ++c) w[c / 4] |= to_code<INT8>(v[c] / s.now) << (8 * (c & 3));
        if constexpr (INNERMOST) {
#pragma unroll
            for (int c = 0; c < V; ++c) tile[(d0 + c) * page + p] = (uint8_t)(w[c / 4] >> (8 * (c & 3)));
        } else {
            uint32_t *to = reinterpret_cast<uint32_t *>(codes + (int64_t)p * D + d0);
#pragma unroll
            for (int j = 0; j < V / 4; ++j) to[j] = w[j];
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
        const int parts = page / 16;
        for (int i = tid; i < D * parts; i += 256) {
            const int d = i / parts, p0 = 16 * (i % parts);
            uint8_t *row = codes + d * page + p0;
            const uint4 t = *reinterpret_cast<const uint4 *>(tile + d * page + p0);
            uint32_t now[4] = {t.x, t.y, t.z, t.w};
            unsigned fresh = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) fresh |= source[p0 + j] >= 0 ? 1u << j : 0u;
            if (!fresh && (p0 >= first || s.grown == 1.f)) continue;
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

// Blocks: chunks of tokens x heads x {keys, values}.
template <typename T, int D, bool INT8>
__global__ void __launch_bounds__(256) kda_cache_append_kernel(AppendArgs a, int chunk)
{
    extern __shared__ __align__(16) uint8_t tile[];
    __shared__ int source[MAX_PAGE];
    __shared__ unsigned part[4];
    const int h = blockIdx.y >> 1, wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    const bool values = blockIdx.y & 1;
    const int t0 = blockIdx.x * chunk, t1 = min(t0 + chunk, a.tokens);
    const int shift = __builtin_ctz(a.page);
    const unsigned places = (unsigned)a.pages * (unsigned)a.page;     // below 2^31
    const auto page_of = [&](int t) {
        const int s = a.slots[t];
        return (unsigned)s < places ? s >> shift : -1;
    };
    int before = t0 > 0 ? page_of(t0 - 1) : -2, runs = 0;
    for (int t = t0; t < t1;) {
        const int id = page_of(t);
        const bool starts = id >= 0 && id != before;
        before = id;
        if (!starts) {
            ++t;
            continue;
        }
        // the run's length: each wave looks at 64 tokens at once
        int n = 0;
        while (true) {
            const int u = t + n + lane;
            const uint64_t other = __ballot(u >= a.tokens || page_of(u) != id);
            n += other ? __builtin_ctzll(other) : 64;
            if (other) break;
        }
        const T *x = (const T *)(values ? a.v : a.k);
        const int64_t stride = values ? a.v_stride : a.k_stride;
        x += (int64_t)t * stride + (int64_t)h * D;
        const int64_t at = (int64_t)id * a.Hk + h;
        uint8_t *codes = (values ? a.v_codes : a.k_codes) + at * a.page * D;
        float *scale = (values ? a.v_scale : a.k_scale) + at;
        if (n <= SHORT) {
            if ((runs++ & 3) == wave) {
                if (values) append_short<T, D, INT8, true>(x, stride, a.slots + t, n, a.page, codes, scale);
                else append_short<T, D, INT8, false>(x, stride, a.slots + t, n, a.page, codes, scale);
            }
        } else {
            if (values) append_long<T, D, INT8, true>(x, stride, a.slots + t, n, a.page, codes, scale, source, part, tile);
            else append_long<T, D, INT8, false>(x, stride, a.slots + t, n, a.page, codes, scale, source, part, tile);
        }
        t += n;
    }
}

template <typename T, int D, bool INT8> hipError_t launch(const AppendArgs &a, hipStream_t stream)
{
    // Short chunks while they are few enough to run at once: a decoding step's
    // tokens are a page each, and a wave takes one after the other.
    const int64_t lanes = 2 * (int64_t)a.Hk;
    const int chunk = a.tokens * lanes <= 4 * 4096 ? 4 : 16;
    const int64_t blocks = ((int64_t)a.tokens + chunk - 1) / chunk;
    if (!grid_fits(blocks, 256) || lanes > 65535) return hipErrorNotSupported;
    hipLaunchKernelGGL((kda_cache_append_kernel<T, D, INT8>), dim3((unsigned)blocks, (unsigned)lanes), dim3(256),
                       (size_t)D * a.page, stream, a, chunk);
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
