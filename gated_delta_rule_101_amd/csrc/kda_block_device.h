// Device helpers of the short convolution, the selective scan and layer norm.
#pragma once

#include "kda_device.h"

namespace kda {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// V consecutive storage elements in one access: V = 16 / sizeof(T) takes a
// 16-byte load, V = 1 a scalar one (rows whose length leaves them unaligned).
// stream / unstream are the non-temporal forms, for data that passes once.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <typename T, int V> struct Pack;
template <typename T> struct Pack<T, 1> {
    T a;
    __device__ __forceinline__ void load(const T *p) { a = *p; }
    __device__ __forceinline__ void stream(const T *p) { a = __builtin_nontemporal_load(p); }
    __device__ __forceinline__ void zero() { a = T(0); }
    __device__ __forceinline__ void to_f32(float (&x)[1]) const { x[0] = kda::to_f32(a); }
    static __device__ __forceinline__ void store(T *p, const float (&x)[1]) { *p = from_f32<T>(x[0]); }
    static __device__ __forceinline__ void unstream(T *p, const float (&x)[1]) {
        __builtin_nontemporal_store(from_f32<T>(x[0]), p);
    }
};
template <> struct Pack<uint16_t, 8> : Raw8<uint16_t> {
    __device__ __forceinline__ void stream(const uint16_t *p) {
        const u32x4 t = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
        a = make_uint4(t[0], t[1], t[2], t[3]);
    }
    static __device__ __forceinline__ u32x4 bits(const float (&x)[8]) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)f32_to_bf16(x[2 * i]) | ((uint32_t)f32_to_bf16(x[2 * i + 1]) << 16);
        return w;
    }
    static __device__ __forceinline__ void store(uint16_t *p, const float (&x)[8]) { *reinterpret_cast<u32x4 *>(p) = bits(x); }
    static __device__ __forceinline__ void unstream(uint16_t *p, const float (&x)[8]) {
        __builtin_nontemporal_store(bits(x), reinterpret_cast<u32x4 *>(p));
    }
};
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <> struct Pack<uint16_t, 4> : Raw4<uint16_t> {
    __device__ __forceinline__ void stream(const uint16_t *p) {
        const u32x2 t = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
        a = make_uint2(t[0], t[1]);
    }
    static __device__ __forceinline__ u32x2 bits(const float (&x)[4]) {
        return u32x2{(uint32_t)f32_to_bf16(x[0]) | ((uint32_t)f32_to_bf16(x[1]) << 16),
                     (uint32_t)f32_to_bf16(x[2]) | ((uint32_t)f32_to_bf16(x[3]) << 16)};
    }
    static __device__ __forceinline__ void store(uint16_t *p, const float (&x)[4]) { *reinterpret_cast<u32x2 *>(p) = bits(x); }
    static __device__ __forceinline__ void unstream(uint16_t *p, const float (&x)[4]) {
        __builtin_nontemporal_store(bits(x), reinterpret_cast<u32x2 *>(p));
    }
};
template <> struct Pack<float, 4> : Raw4<float> {
    __device__ __forceinline__ void stream(const float *p) {
        const f32x4 t = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
        a = make_float4(t[0], t[1], t[2], t[3]);
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[4]) { store4(p, x); }
    static __device__ __forceinline__ void unstream(float *p, const float (&x)[4]) {
        __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4 *>(p));
    }
};
template <typename T> constexpr int WIDE = 16 / (int)sizeof(T);

// A few rows of a token tensor behind a pointer that is the same for the whole
// wavefront, accessed at a lane's byte offset plus a uniform one, both 32 bits:
// buffer instructions take all three as they are, where a global access pays a
// 64-bit vector addition each.  The row pointer must be rebuilt often enough
// that the uniform offset stays below 2^31.
template <typename T> struct Rows {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ explicit Rows(const T *p)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(p), (short)0, (int)0xFFFFFFFF, 0x00020000)) {}
    __device__ __forceinline__ T load(unsigned lane, unsigned uniform) const {
        if constexpr (sizeof(T) == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, lane, uniform, 0);
        else return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, lane, uniform, 0));
    }
    __device__ __forceinline__ void store(T v, unsigned lane, unsigned uniform) const {
        if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(v, r, lane, uniform, 0);
        else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, lane, uniform, 0);
    }
};

// log(1 + e) for e in [0, 1]: 2 artanh(r) with r = e / (2 + e) <= 1/3, whose
// series in r^2 <= 1/9 is cut after r^13 (the rest is below 2e-8 of the sum).
// log2(1 + e) directly would lose the small e, where softplus itself is e.
__device__ __forceinline__ float log1p_unit(float e) {
    const float r = e * fast_rcp(2.f + e), q = r * r;
    float p = __builtin_fmaf(q, 1.f / 13, 1.f / 11);
    p = __builtin_fmaf(q, p, 1.f / 9);
    p = __builtin_fmaf(q, p, 1.f / 7);
    p = __builtin_fmaf(q, p, 1.f / 5);
    p = __builtin_fmaf(q, p, 1.f / 3);
    p = __builtin_fmaf(q, p, 1.f);
    return 2.f * r * p;
}
// softplus(v) = max(v, 0) + log(1 + exp(-|v|)).
__device__ __forceinline__ float softplus_f32(float v) {
    return fmaxf(v, 0.f) + log1p_unit(fast_exp2(-fabsf(v) * LOG2E));
}

// ------------------------------------------------------------ quads of lanes
//
// A value that lane K of each quad holds, for all four; as an operand it rides
// on the instruction that uses it.
template <int K> struct Const { static constexpr int value = K; };
template <typename F> __device__ __forceinline__ void each4(F f)
{
    f(Const<0>{});
    f(Const<1>{});
    f(Const<2>{});
    f(Const<3>{});
}
template <int K> __device__ __forceinline__ float quad_bcast(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), K * 0x55, 0xF, 0xF, true));
}
template <int CTRL> __device__ __forceinline__ float quad_add(float x)
{
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}

// Rates are used in base 2, and held where that is finite.  A lower one, -infinity
// (-exp of a large number) among them, then still forgets at every positive step,
// and leaves a token of step 0, such as those behind a sequence's end, a token
// that changes nothing.
__device__ __forceinline__ float finite_rate(float A) {
    constexpr float LOWEST = -2.3586e38f;   // times LOG2E: -3.4027e38
    return A < LOWEST ? LOWEST : A;
}

// ----------------------------------------------------- states and places
//
// N states of a channel in NP places of registers, NP (a power of two) >= N.  Where
// places are left they hold a state once more: a place that held none would
// take part in the arithmetic with zeros, and 0 times an infinite s x is NaN.
// With G the power of two in [N, 2 N), place p holds state p mod G, or that
// less N; so a state has NP / G places, those in front of G - N twice as many,
// each with the same values.  Sums over the states take each place's share of
// its state, one over their number: exact, as that is a power of two.
template <bool FILL> struct Places {
    int n, g, places;
    __device__ __forceinline__ Places(int N, int NP) : n(N), g(NP), places(NP) {
        if (FILL)
            while (g >= 2 * n) g >>= 1;
    }
    __device__ __forceinline__ int state(int p) const {
        const int q = p & (g - 1);
        return !FILL ? p : q < n ? q : q - n;
    }
    __device__ __forceinline__ float places_of(int p) const {   // of p's state
        return !FILL ? 1.f : (float)(places / g * (state(p) < g - n ? 2 : 1));
    }
    __device__ __forceinline__ float share(int p) const { return 1.f / places_of(p); }
};

// Tokens of sequence b: lengths[b] clamped to [0, T], or T.
__device__ __forceinline__ int seq_length(const int *lengths, int b, int T) {
    return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace kda
