// Interface between the C ABI of the attention layer's operators
// (kda_attn_api.hip) and their launchers.  Arguments arrive validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

struct PlanArgs {
    const int *cached, *added;
    int *table;                              // [B][per], entries of new pages written
    const int *free_pages, *free_count;      // [capacity], [1]
    int *q_start, *context, *positions, *slots, *free_left;
    int B, per, capacity, tokens, page;
};

struct QkNormArgs {
    const void *q, *k;
    const float *wq = nullptr, *wk = nullptr;        // nullable: ones
    const int *positions = nullptr;                  // with rotary; without, their sign alone counts
    const float *rotary = nullptr;                   // [longest][R]: R / 2 cosines, then the sines
    const void *gq = nullptr, *gk = nullptr;         // backward: upstream gradients
    void *q_out, *k_out;                             // or the gradients of q and k
    float *dwq = nullptr, *dwk = nullptr, *ws = nullptr;
    int64_t T;
    int64_t q_stride, k_stride, gq_stride = 0, gk_stride = 0, qo_stride, ko_stride;   // elements between tokens
    int Hq, Hk, D, R, longest;
    float eps;
    bool neighbours, bf16;
};

struct AppendArgs {
    const void *k, *v;
    const int *slots;
    uint8_t *k_codes, *v_codes;              // [pages][Hk][page][D], [pages][Hk][D][page]
    float *k_scale, *v_scale;                // [pages][Hk]
    int64_t k_stride, v_stride;
    int tokens, Hk, D, pages, page;
    bool int8, bf16;
};

struct AttendArgs {
    const void *q;
    const uint8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    const int *table, *context, *q_start = nullptr;  // q_start nullable: one query a sequence
    void *out;
    float *lse = nullptr, *ws;
    int tokens, B, Hq, Hk, D, pages, page, per, most;
    int64_t room;                            // tokens that a context may have: 0 without pages
    float scale;
    bool int8, bf16;
};

// As in kda_block.h: hipErrorNotSupported, with nothing enqueued, where a grid
// cannot be launched.
hipError_t launch_cache_plan(const PlanArgs &a, hipStream_t stream);
hipError_t launch_qk_norm_fwd(const QkNormArgs &a, hipStream_t stream);
hipError_t launch_qk_norm_bwd(const QkNormArgs &a, hipStream_t stream);
int64_t qk_norm_bwd_workspace_floats(int64_t T, int Hq, int Hk, int D);
hipError_t launch_cache_append(const AppendArgs &a, hipStream_t stream);
hipError_t launch_cache_attend(const AttendArgs &a, hipStream_t stream);
int64_t cache_attend_workspace_floats(int tokens, int B, int Hq, int Hk, int D, int page, int per, int most);

}  // namespace kda
