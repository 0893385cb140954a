// Host-side checks that the C ABI's entry points share: argument buffers,
// element types, a launcher's result.
#pragma once

#include "../../include/kda.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {

constexpr int64_t MAX_DIM = (int64_t)1 << 24, MAX_COUNT = (int64_t)1 << 40;

// One argument buffer: its bytes, whether it may be NULL, and how it is aligned.
struct Buffer {
    const void *p;
    size_t bytes;
    bool required;
    size_t align = 16;
};

inline bool overlap(const Buffer &a, const Buffer &b)
{
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

// Every required buffer present, all aligned, no output over an input or over
// another output.  `same_in`/`same_out` name one output that may be exactly
// one input (in place).
template <int NI, int NO>
kda_status_t check_buffers(const Buffer (&in)[NI], const Buffer (&out)[NO], int same_in = -1, int same_out = -1)
{
    const auto bad = [](const Buffer &b) {
        return b.bytes && ((b.required && !b.p) || ((uintptr_t)b.p & (b.align - 1)));
    };
    for (const Buffer &b : in)
        if (bad(b)) return KDA_ERR_INVALID_ARG;
    for (const Buffer &b : out)
        if (bad(b)) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i], in[j]) && !(i == same_out && j == same_in && out[i].p == in[j].p))
                return KDA_ERR_INVALID_ARG;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j])) return KDA_ERR_INVALID_ARG;
    }
    return KDA_OK;
}

inline bool valid_dtype(kda_dtype_t d) { return d == KDA_F32 || d == KDA_BF16; }
inline size_t dsize(kda_dtype_t d) { return d == KDA_BF16 ? 2 : 4; }

// A launcher's own refusal (a grid too large) and the runtime's.
inline kda_status_t launched(hipError_t e)
{
    return e == hipSuccess ? KDA_OK : e == hipErrorNotSupported ? KDA_ERR_UNSUPPORTED : KDA_ERR_LAUNCH;
}

}  // namespace
