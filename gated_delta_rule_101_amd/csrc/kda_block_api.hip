// C ABI of the short convolution, the selective scan and layer norm: host-side
// validation, then the launches on the caller's stream.  Declarations and the
// full contract are in include/kda.h.
#include "kda_block.h"
#include "kda_check.h"

namespace {

// Sizes that are not negative and whose products fit: KDA_OK, or the error.
kda_status_t check_sizes(int B, int T, int D)
{
    if (B < 0 || T < 0 || D < 0) return KDA_ERR_INVALID_ARG;
    if (B >= MAX_DIM || T >= MAX_DIM || D >= MAX_DIM) return KDA_ERR_UNSUPPORTED;
    if (T > 0 && (int64_t)B * T >= MAX_COUNT) return KDA_ERR_UNSUPPORTED;
    if (D > 0 && (int64_t)B * (T > 0 ? T : 1) >= MAX_COUNT / D) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status_t check_conv(int B, int T, int D, int W, kda_dtype_t dtype)
{
    const kda_status_t st = check_sizes(B, T, D);
    if (st != KDA_OK) return st;
    if (W <= 0 || !valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    return W < 2 || W > 4 ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

kda_status_t check_scan(int B, int T, int D, int N, int G, kda_dtype_t dtype)
{
    const kda_status_t st = check_sizes(B, T, D);
    if (st != KDA_OK) return st;
    if (N <= 0 || G <= 0 || D % G || !valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    if (N > 64) return KDA_ERR_UNSUPPORTED;
    // the states' elements and the rows of B and C stay countable as well
    if ((int64_t)G * N >= MAX_DIM) return KDA_ERR_UNSUPPORTED;
    if (D > 0 && (int64_t)B >= MAX_COUNT / ((int64_t)D * N)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)B * (T > 0 ? T : 1) >= MAX_COUNT / ((int64_t)G * N)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------- short convolution

kda_status_t kda_short_conv_fwd(const void *x, const float *w, const float *bias, const void *state0,
                                const int *lengths, void *y, void *state_final,
                                int B, int T, int D, int W, int silu, kda_dtype_t dtype, void *stream)
{
    const kda_status_t st = check_conv(B, T, D, W, dtype);
    if (st != KDA_OK) return st;
    if (B == 0 || D == 0 || (T == 0 && !state_final)) return KDA_OK;
    const size_t e = dsize(dtype), tok = (size_t)B * T * D * e, state = (size_t)B * (W - 1) * D * e;
    const Buffer in[] = {{x, tok, true}, {w, (size_t)D * W * 4, true}, {bias, (size_t)D * 4, false},
                         {state0, state, false}, {lengths, (size_t)B * 4, false, 4}};
    const Buffer out[] = {{y, tok, true}, {state_final, state, false}};
    const kda_status_t ok = check_buffers(in, out, 3, 1);
    if (ok != KDA_OK) return ok;
    kda::ConvArgs a;
    a.x = x; a.w = w; a.bias = bias; a.state0 = state0; a.lengths = lengths; a.y = y; a.state_final = state_final;
    a.B = B; a.T = T; a.D = D; a.W = W; a.silu = silu != 0; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_conv_fwd(a, (hipStream_t)stream));
}

kda_status_t kda_short_conv_step(const void *x, const float *w, const float *bias, void *state, void *y,
                                 int B, int D, int W, int silu, kda_dtype_t dtype, void *stream)
{
    const kda_status_t st = check_conv(B, 1, D, W, dtype);
    if (st != KDA_OK) return st;
    if (B == 0 || D == 0) return KDA_OK;
    const size_t e = dsize(dtype), tok = (size_t)B * D * e;
    const Buffer in[] = {{x, tok, true}, {w, (size_t)D * W * 4, true}, {bias, (size_t)D * 4, false}};
    const Buffer out[] = {{y, tok, true}, {state, (W - 1) * tok, true}};
    const kda_status_t ok = check_buffers(in, out, 0, 0);
    if (ok != KDA_OK) return ok;
    kda::ConvArgs a;
    a.x = x; a.w = w; a.bias = bias; a.y = y; a.state_final = state;
    a.B = B; a.T = 1; a.D = D; a.W = W; a.silu = silu != 0; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_conv_step(a, (hipStream_t)stream));
}

size_t kda_short_conv_bwd_workspace_bytes(int B, int T, int D, int W)
{
    if (check_conv(B, T, D, W, KDA_F32) != KDA_OK || B == 0 || D == 0) return 0;
    return (size_t)kda::conv_bwd_workspace_floats(B, T, D, W) * sizeof(float);
}

kda_status_t kda_short_conv_bwd(const void *dy, const void *x, const float *w, const float *bias,
                                const void *state0, const void *dstate_final, const int *lengths,
                                void *dx, float *dw, float *dbias, void *dstate0,
                                void *workspace, size_t workspace_bytes,
                                int B, int T, int D, int W, int silu, kda_dtype_t dtype, void *stream)
{
    const kda_status_t st = check_conv(B, T, D, W, dtype);
    if (st != KDA_OK) return st;
    if (D == 0) return KDA_OK;
    const size_t e = dsize(dtype), tok = (size_t)B * T * D * e, state = (size_t)B * (W - 1) * D * e;
    const size_t need = kda_short_conv_bwd_workspace_bytes(B, T, D, W);
    if (workspace_bytes < need) return KDA_ERR_INVALID_ARG;
    const Buffer in[] = {{dy, tok, true}, {x, tok, true}, {w, (size_t)D * W * 4, true}, {bias, (size_t)D * 4, false},
                         {state0, state, false}, {dstate_final, state, false}, {lengths, (size_t)B * 4, false, 4}};
    const Buffer out[] = {{dx, tok, true}, {dw, (size_t)D * W * 4, true}, {dbias, (size_t)D * 4, false},
                          {dstate0, state, false}, {workspace, need, true}};
    const kda_status_t ok = check_buffers(in, out);
    if (ok != KDA_OK) return ok;
    kda::ConvBwdArgs a;
    a.dy = dy; a.x = x; a.w = w; a.bias = bias; a.state0 = state0; a.dstate_final = dstate_final;
    a.lengths = lengths; a.dx = dx; a.dw = dw; a.dbias = dbias; a.dstate0 = dstate0; a.ws = (float *)workspace;
    a.B = B; a.T = T; a.D = D; a.W = W; a.silu = silu != 0; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_conv_bwd(a, (hipStream_t)stream));
}

// ---------------------------------------------------------- selective scan

size_t kda_selective_scan_fwd_workspace_bytes(int B, int T, int D, int N, int G)
{
    if (check_scan(B, T, D, N, G, KDA_F32) != KDA_OK || B == 0 || T == 0 || D == 0) return 0;
    return (size_t)kda::scan_fwd_workspace_floats(B, T, D, N, G) * sizeof(float);
}

kda_status_t kda_selective_scan_fwd(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                                    const float *Dskip, const void *z, const float *dt_bias, const float *h0,
                                    const int *lengths, void *y, float *h_final,
                                    void *workspace, size_t workspace_bytes,
                                    int B, int T, int D, int N, int G, int softplus, kda_dtype_t dtype, void *stream)
{
    const kda_status_t st = check_scan(B, T, D, N, G, dtype);
    if (st != KDA_OK) return st;
    if (B == 0 || D == 0 || (T == 0 && !h_final)) return KDA_OK;
    const size_t e = dsize(dtype), tok = (size_t)B * T * D * e, rows = (size_t)B * T * G * N * e;
    const size_t state = (size_t)B * D * N * 4, need = kda_selective_scan_fwd_workspace_bytes(B, T, D, N, G);
    if (workspace && workspace_bytes < need) return KDA_ERR_INVALID_ARG;
    const Buffer in[] = {{x, tok, true}, {dt, tok, true}, {A, (size_t)D * N * 4, true}, {Bm, rows, true},
                         {Cm, rows, true}, {Dskip, (size_t)D * 4, false}, {z, tok, false},
                         {dt_bias, (size_t)D * 4, false}, {h0, state, false}, {lengths, (size_t)B * 4, false, 4}};
    const Buffer out[] = {{y, tok, true}, {h_final, state, false}, {workspace, need, false}};
    const kda_status_t ok = check_buffers(in, out, 8, 1);
    if (ok != KDA_OK) return ok;
    kda::ScanArgs a;
    a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.dt_bias = dt_bias; a.h0 = h0;
    a.lengths = lengths; a.y = y; a.h_final = h_final; a.ws = (float *)workspace;
    a.B = B; a.T = T; a.D = D; a.N = N; a.G = G; a.softplus = softplus != 0; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_scan_fwd(a, (hipStream_t)stream));
}

kda_status_t kda_selective_scan_step(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                                     const float *Dskip, const void *z, const float *dt_bias, float *h, void *y,
                                     int B, int D, int N, int G, int softplus, kda_dtype_t dtype, void *stream)
{
    const kda_status_t st = check_scan(B, 1, D, N, G, dtype);
    if (st != KDA_OK) return st;
    if (B == 0 || D == 0) return KDA_OK;
    const size_t e = dsize(dtype), tok = (size_t)B * D * e, rows = (size_t)B * G * N * e;
    const Buffer in[] = {{x, tok, true}, {dt, tok, true}, {A, (size_t)D * N * 4, true}, {Bm, rows, true},
                         {Cm, rows, true}, {Dskip, (size_t)D * 4, false}, {z, tok, false},
                         {dt_bias, (size_t)D * 4, false}};
    const Buffer out[] = {{y, tok, true}, {h, (size_t)B * D * N * 4, true}};
    const kda_status_t ok = check_buffers(in, out);
    if (ok != KDA_OK) return ok;
    kda::ScanArgs a;
    a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.dt_bias = dt_bias;
    a.y = y; a.h_final = h;
    a.B = B; a.T = 1; a.D = D; a.N = N; a.G = G; a.softplus = softplus != 0; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_scan_step(a, (hipStream_t)stream));
}

size_t kda_selective_scan_bwd_workspace_bytes(int B, int T, int D, int N, int G)
{
    if (check_scan(B, T, D, N, G, KDA_F32) != KDA_OK || B == 0 || T == 0 || D == 0) return 0;
    return (size_t)kda::scan_bwd_workspace_floats(B, T, D, N, G) * sizeof(float);
}

kda_status_t kda_selective_scan_bwd(const void *dy, const void *x, const void *dt, const float *A, const void *Bm,
                                    const void *Cm, const float *Dskip, const void *z, const float *dt_bias,
                                    const float *h0, const float *dh_final, const int *lengths,
                                    void *dx, void *ddt, float *dA, void *dBm, void *dCm, float *dDskip, void *dz,
                                    float *ddt_bias, float *dh0, void *workspace, size_t workspace_bytes,
                                    int B, int T, int D, int N, int G, int softplus, kda_dtype_t dtype, void *stream)
{
    const kda_status_t st = check_scan(B, T, D, N, G, dtype);
    if (st != KDA_OK) return st;
    if (D == 0) return KDA_OK;   // as declared: dBm and dCm, the only outputs with elements, are the caller's
    const size_t e = dsize(dtype), tok = (size_t)B * T * D * e, rows = (size_t)B * T * G * N * e;
    const size_t state = (size_t)B * D * N * 4, need = kda_selective_scan_bwd_workspace_bytes(B, T, D, N, G);
    if (workspace_bytes < need) return KDA_ERR_INVALID_ARG;
    // a gradient goes with its input; without tokens dz has no bytes to write
    if ((!Dskip) != (!dDskip) || (!dt_bias) != (!ddt_bias) || (tok > 0 && (!z) != (!dz))) return KDA_ERR_INVALID_ARG;
    const Buffer in[] = {{dy, tok, true}, {x, tok, true}, {dt, tok, true}, {A, (size_t)D * N * 4, true},
                         {Bm, rows, true}, {Cm, rows, true}, {Dskip, (size_t)D * 4, false}, {z, tok, false},
                         {dt_bias, (size_t)D * 4, false}, {h0, state, false}, {dh_final, state, false},
                         {lengths, (size_t)B * 4, false, 4}};
    const Buffer out[] = {{dx, tok, true}, {ddt, tok, true}, {dA, (size_t)D * N * 4, true}, {dBm, rows, true},
                          {dCm, rows, true}, {dDskip, (size_t)D * 4, false}, {dz, tok, false},
                          {ddt_bias, (size_t)D * 4, false}, {dh0, state, false}, {workspace, need, true}};
    const kda_status_t ok = check_buffers(in, out);
    if (ok != KDA_OK) return ok;
    kda::ScanBwdArgs a;
    a.dy = dy; a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.dt_bias = dt_bias;
    a.h0 = h0; a.dh_final = dh_final; a.lengths = lengths;
    a.dx = dx; a.ddt = ddt; a.dA = dA; a.dBm = dBm; a.dCm = dCm; a.dDskip = dDskip; a.dz = dz;
    a.ddt_bias = ddt_bias; a.dh0 = dh0; a.ws = (float *)workspace;
    a.B = B; a.T = T; a.D = D; a.N = N; a.G = G; a.softplus = softplus != 0; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_scan_bwd(a, (hipStream_t)stream));
}

// -------------------------------------------------------------- layer norm

static kda_status_t check_norm(int64_t rows, int D, float eps, kda_dtype_t dtype)
{
    if (rows < 0 || D <= 0 || !valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    if (!(eps >= 0.f && eps <= 3.0e38f)) return KDA_ERR_INVALID_ARG;   // NaN and inf too
    return D > 16384 || rows >= MAX_COUNT / D ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

kda_status_t kda_layer_norm_fwd(const void *x, const float *weight, const float *bias, float eps, void *y,
                                int64_t rows, int D, kda_dtype_t dtype, void *stream)
{
    const kda_status_t st = check_norm(rows, D, eps, dtype);
    if (st != KDA_OK) return st;
    if (rows == 0) return KDA_OK;
    const size_t bytes = (size_t)rows * D * dsize(dtype);
    const Buffer in[] = {{x, bytes, true}, {weight, (size_t)D * 4, false}, {bias, (size_t)D * 4, false}};
    const Buffer out[] = {{y, bytes, true}};
    const kda_status_t ok = check_buffers(in, out, 0, 0);
    if (ok != KDA_OK) return ok;
    kda::NormArgs a;
    a.x = x; a.weight = weight; a.bias = bias; a.y = y;
    a.rows = rows; a.D = D; a.eps = eps; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_norm_fwd(a, (hipStream_t)stream));
}

size_t kda_layer_norm_bwd_workspace_bytes(int64_t rows, int D)
{
    if (check_norm(rows, D, 0.f, KDA_F32) != KDA_OK || rows == 0) return 0;
    return (size_t)kda::norm_bwd_workspace_floats(rows, D) * sizeof(float);
}

kda_status_t kda_layer_norm_bwd(const void *dy, const void *x, const float *weight, float eps, void *dx,
                                float *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                                int64_t rows, int D, kda_dtype_t dtype, void *stream)
{
    const kda_status_t st = check_norm(rows, D, eps, dtype);
    if (st != KDA_OK) return st;
    const size_t bytes = (size_t)rows * D * dsize(dtype);
    const size_t need = dweight || dbias ? kda_layer_norm_bwd_workspace_bytes(rows, D) : 0;
    if (workspace_bytes < need) return KDA_ERR_INVALID_ARG;
    const Buffer in[] = {{dy, bytes, true}, {x, bytes, true}, {weight, (size_t)D * 4, false}};
    const Buffer out[] = {{dx, bytes, true}, {dweight, (size_t)D * 4, false}, {dbias, (size_t)D * 4, false},
                          {workspace, need, true}};
    const kda_status_t ok = check_buffers(in, out, 0, 0);
    if (ok != KDA_OK) return ok;
    if (rows == 0 && !dweight && !dbias) return KDA_OK;
    kda::NormBwdArgs a;
    a.dy = dy; a.x = x; a.weight = weight; a.dx = dx; a.dweight = dweight; a.dbias = dbias;
    a.ws = (float *)workspace; a.rows = rows; a.D = D; a.eps = eps; a.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_norm_bwd(a, (hipStream_t)stream));
}

}  // extern "C"
