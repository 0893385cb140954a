// The cache's 8-bit codes on the device: e4m3 floats (largest 448) or integers
// (-127 .. 127), a value being its code times the scale of its page and head.
#pragma once

#include "kda_block_device.h"

namespace kda {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// 8 codes as float16, which holds every one exactly.
template <bool INT8> __device__ __forceinline__ f16x8 codes_f16(uint32_t lo, uint32_t hi)
{
    f16x2 p[4];
    if constexpr (INT8) {
        // a byte x + 128 under 0x64 is the float16 1024 + x + 128
        const uint32_t w[2] = {lo ^ 0x80808080u, hi ^ 0x80808080u};
        const f16x2 off = {(_Float16)1152.f, (_Float16)1152.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            p[2 * i] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w[i], 0x04010400u)) - off;
            p[2 * i + 1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w[i], 0x04030402u)) - off;
        }
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
    }
    return f16x8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

template <bool INT8> constexpr float CODE_MAX = INT8 ? 127.f : 448.f;
template <bool INT8> constexpr float CODE_UNIT = INT8 ? 1.f / 127.f : 1.f / 448.f;

// The code nearest to v, ties to even; 0 where v is not finite, which is where
// the scale is zero or not finite itself.
template <bool INT8> __device__ __forceinline__ uint32_t to_code(float v)
{
    constexpr float M = CODE_MAX<INT8>;
    v = fabsf(v) <= 3.4028235e38f ? fminf(fmaxf(v, -M), M) : 0.f;
    if constexpr (INT8) return (uint32_t)(int)__builtin_rintf(v) & 0xffu;
    else return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xffu;
}
template <bool INT8> __device__ __forceinline__ float from_code(uint32_t byte)
{
    if constexpr (INT8) return (float)(int8_t)byte;
    else return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
}

}  // namespace kda
