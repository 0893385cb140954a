// Interface between the C ABI of the short convolution, the selective scan and
// layer norm (kda_block_api.hip) and their launchers.  Arguments arrive
// validated; element counts fit 64 bits, B, T and D fit 24.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

struct ConvArgs {
    const void *x;
    const float *w, *bias = nullptr;         // [D][W]; nullable bias
    const void *state0 = nullptr;            // nullable: zeros
    const int *lengths = nullptr;            // nullable: all T
    void *y;
    void *state_final = nullptr;             // nullable: not written; may be state0
    int B, T, D, W;
    bool silu, bf16;
};

struct ConvBwdArgs {
    const void *dy, *x;
    const float *w, *bias = nullptr;
    const void *state0 = nullptr, *dstate_final = nullptr;
    const int *lengths = nullptr;
    void *dx;
    float *dw, *dbias = nullptr;
    void *dstate0 = nullptr;
    float *ws;                               // partial sums: dw [runs][D][W], then dbias [runs][D]
    int B, T, D, W;
    bool silu, bf16;
};

struct ScanArgs {
    const void *x, *dt;
    const float *A;
    const void *Bm, *Cm;
    const float *Dskip = nullptr;
    const void *z = nullptr;
    const float *dt_bias = nullptr, *h0 = nullptr;
    const int *lengths = nullptr;
    void *y;
    float *h_final = nullptr;                // or, for a step, the states (in place)
    float *ws = nullptr;                     // nullable: one segment
    int B, T, D, N, G;
    bool softplus, bf16;
};

struct ScanBwdArgs {
    const void *dy, *x, *dt;
    const float *A;
    const void *Bm, *Cm;
    const float *Dskip = nullptr;
    const void *z = nullptr;
    const float *dt_bias = nullptr, *h0 = nullptr, *dh_final = nullptr;
    const int *lengths = nullptr;
    void *dx, *ddt;
    float *dA;
    void *dBm, *dCm;
    float *dDskip = nullptr;
    void *dz = nullptr;
    float *ddt_bias = nullptr, *dh0 = nullptr;
    float *ws = nullptr;
    int B, T, D, N, G;
    bool softplus, bf16;
};

struct NormArgs {
    const void *x;
    const float *weight = nullptr, *bias = nullptr;
    void *y;
    int64_t rows;
    int D;
    float eps;
    bool bf16;
};

struct NormBwdArgs {
    const void *dy, *x;
    const float *weight = nullptr;
    void *dx;
    float *dweight = nullptr, *dbias = nullptr;
    float *ws = nullptr;                     // [blocks][2][D]
    int64_t rows;
    int D;
    float eps;
    bool bf16;
};

// Column sums out[m] = sum_r in[r * stride + m], m < cols, of up to five
// matrices; rows == 0 gives zeros.  The matrices may be overwritten.
struct ColumnSum {
    float *in;
    void *out;
    int64_t rows, cols, stride;
    bool out_bf16;
};
hipError_t launch_column_sums(const ColumnSum *jobs, int n, hipStream_t stream);
bool column_sums_fit(const ColumnSum *jobs, int n);      // its grids can be launched

// HIP launches fewer than 2^32 threads along an axis.  Every launcher below
// checks all its grids before the first of them and returns
// hipErrorNotSupported, with nothing enqueued, where one is larger.
inline bool grid_fits(int64_t blocks, int threads) { return blocks < ((int64_t)1 << 32) / threads; }

hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs &a, hipStream_t stream);      // state_final is the state, T unused
hipError_t launch_conv_bwd(const ConvBwdArgs &a, hipStream_t stream);
int64_t conv_bwd_workspace_floats(int B, int T, int D, int W);
hipError_t launch_scan_fwd(const ScanArgs &a, hipStream_t stream);
int64_t scan_fwd_workspace_floats(int B, int T, int D, int N, int G);
hipError_t launch_scan_step(const ScanArgs &a, hipStream_t stream);
hipError_t launch_scan_bwd(const ScanBwdArgs &a, hipStream_t stream);
int64_t scan_bwd_workspace_floats(int B, int T, int D, int N, int G);
hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t stream);
hipError_t launch_norm_bwd(const NormBwdArgs &a, hipStream_t stream);
int64_t norm_bwd_workspace_floats(int64_t rows, int D);

}  // namespace kda
