// Short causal depthwise convolution for gfx950: forward over a sequence, one
// token, and the gradients.
//
//   pre[t] = bias + sum_{j < W} w[j] x[t - W + 1 + j],   y = silu(pre) or pre
//
// Every element is touched once, so all three are bound by HBM bandwidth.  A
// thread owns V neighbouring channels (16 bytes of a token's row) and walks a
// run of tokens with the last W - 1 inputs in registers, so that a run reads
// its tokens once plus W - 1 tokens in front (which its neighbour run brings
// into the cache as well).  Rows whose length is no multiple of V are walked
// one channel a thread.  Measured (bfloat16, W = 4): forward of B4 T16384 D4096
// 0.209 ms, 5.1 TB/s; backward of B4 T4096 D4096 0.085 ms, 4.7 TB/s (0.003 more without
// the non-temporal loads, the same with 8 tokens requested together).
#include "kda_block.h"
#include "kda_block_device.h"

namespace kda {
namespace {

constexpr int THREADS = 256;
constexpr int BATCH = 4;   // tokens whose loads are issued together; a run is a multiple of them
template <bool B> struct Flag { static constexpr bool value = B; };

template <typename T, int W, int V>
__device__ __forceinline__ void load_taps(float (&w)[W][V], float (&bias)[V], const float *wp, const float *bp, int d)
{
#pragma unroll
    for (int c = 0; c < V; ++c) {
        bias[c] = bp ? bp[d + c] : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][c] = wp[(int64_t)(d + c) * W + j];
    }
}

// Input row p of a sequence whose first W - 1 rows are its state: p < 0 reads
// state row p + W - 1 (zeros without a state).
template <typename T, int W, int V>
__device__ __forceinline__ void load_row(Pack<T, V> &r, const T *x, const T *state, int p, int D)
{
    if (p >= 0) r.load(x + (int64_t)p * D);
    else if (state) r.load(state + (int64_t)(p + W - 1) * D);
    else r.zero();
}

// ------------------------------------------------------------------ forward

// Run `run` covers tokens [run RT, (run + 1) RT).  The thread of run 0 also
// writes the final state: only it reads the initial one, so the two may be
// one buffer.
template <typename T, int W, int V, bool SILU>
__global__ void __launch_bounds__(THREADS) kda_conv_fwd_kernel(ConvArgs a, int RT, int nruns, int ncg, int64_t total)
{
    const int64_t id = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (id >= total) return;
    const int cg = (int)(id % ncg);
    const int64_t rest = id / ncg;
    const int run = (int)(rest % nruns), b = (int)(rest / nruns);
    const int D = a.D, d = cg * V;
    const int len = seq_length(a.lengths, b, a.T);
    const T *x = (const T *)a.x + (int64_t)b * a.T * D + d;
    T *y = (T *)a.y + (int64_t)b * a.T * D + d;
    const T *state = a.state0 ? (const T *)a.state0 + (int64_t)b * (W - 1) * D + d : nullptr;
    const int t0 = run * RT, t1 = min(t0 + RT, a.T), tv = min(t1, len);

    Pack<T, V> last[W - 1];
    if (run == 0 && a.state_final)
#pragma unroll
        for (int r = 0; r < W - 1; ++r) load_row<T, W, V>(last[r], x, state, len - (W - 1) + r, D);

    if (t0 < tv) {
        float w[W][V], bias[V], win[W][V];   // win[j]: input t - (W - 1) + j
        load_taps<T, W, V>(w, bias, a.w, a.bias, d);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            Pack<T, V> r;
            load_row<T, W, V>(r, x, state, t0 - (W - 1) + j, D);
            r.to_f32(win[j]);
        }
        for (int t = t0; t < tv; t += BATCH) {
            Pack<T, V> in[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) in[i].load(x + (int64_t)min(t + i, tv - 1) * D);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                in[i].to_f32(win[W - 1]);
                float o[V];
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    float p = bias[c];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = __builtin_fmaf(w[j][c], win[j][c], p);
                    o[c] = SILU ? p * sigmoid_f32(p) : p;
                }
                if (t + i < tv) Pack<T, V>::unstream(y + (int64_t)(t + i) * D, o);
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int c = 0; c < V; ++c) win[j][c] = win[j + 1][c];
            }
        }
    }
    const float zero[V] = {};
    for (int t = max(tv, t0); t < t1; ++t) Pack<T, V>::store(y + (int64_t)t * D, zero);

    if (run == 0 && a.state_final) {
        T *f = (T *)a.state_final + (int64_t)b * (W - 1) * D + d;
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            float v[V];
            last[r].to_f32(v);   // exact both ways: the state holds inputs in their own type
            Pack<T, V>::store(f + (int64_t)r * D, v);
        }
    }
}

// ---------------------------------------------------------------- one token

template <typename T, int W, int V>
__global__ void __launch_bounds__(THREADS) kda_conv_step_kernel(ConvArgs a, int ncg, int64_t total)
{
    const int64_t id = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (id >= total) return;
    const int d = (int)(id % ncg) * V, b = (int)(id / ncg), D = a.D;
    T *state = (T *)a.state_final + (int64_t)b * (W - 1) * D + d;
    Pack<T, V> r[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j].load(state + (int64_t)j * D);
    r[W - 1].load((const T *)a.x + (int64_t)b * D + d);
    float w[W][V], p[V];
    load_taps<T, W, V>(w, p, a.w, a.bias, d);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float v[V];
        r[j].to_f32(v);
        if (j > 0) Pack<T, V>::store(state + (int64_t)(j - 1) * D, v);
#pragma unroll
        for (int c = 0; c < V; ++c) p[c] = __builtin_fmaf(w[j][c], v[c], p[c]);
    }
#pragma unroll
    for (int c = 0; c < V; ++c) p[c] = a.silu ? p[c] * sigmoid_f32(p[c]) : p[c];
    Pack<T, V>::store((T *)a.y + (int64_t)b * D + d, p);
}

// ----------------------------------------------------------------- backward

// With dpre[t] = dy[t] silu'(pre[t]):
//   dx[t] = sum_j w[j] dpre[t + W - 1 - j],   dw[j] = sum_t dpre[t] x[t - W + 1 + j].
// A run walks its tokens and W - 1 tokens behind them (their dpre reaches back
// into the run) and writes dx of token t - (W - 1) at token t; run 0 starts
// W - 1 positions early, where dx is the state's gradient.  Only the run's
// own tokens enter dw and dbias, which stay in registers and go to the
// workspace once a run.
template <typename T, int W, int V, bool SILU>
__global__ void __launch_bounds__(THREADS) kda_conv_bwd_kernel(ConvBwdArgs a, int RT, int nruns, int ncg, int64_t total)
{
    const int64_t id = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (id >= total) return;
    const int cg = (int)(id % ncg);
    const int64_t rest = id / ncg;   // b nruns + run: the row of the partial sums
    const int run = (int)(rest % nruns), b = (int)(rest / nruns);
    const int D = a.D, d = cg * V;
    const int len = seq_length(a.lengths, b, a.T);
    const T *x = (const T *)a.x + (int64_t)b * a.T * D + d;
    const T *dy = (const T *)a.dy + (int64_t)b * a.T * D + d;
    T *dx = (T *)a.dx + (int64_t)b * a.T * D + d;
    const int64_t so = (int64_t)b * (W - 1) * D + d;
    const T *state = a.state0 ? (const T *)a.state0 + so : nullptr;
    const T *dsf = a.dstate_final ? (const T *)a.dstate_final + so : nullptr;
    T *ds0 = a.dstate0 ? (T *)a.dstate0 + so : nullptr;
    const int t0 = run * RT, t1 = min(t0 + RT, a.T);

    float w[W][V], bias[V], win[W][V], dp[W][V];   // dp[j]: dpre of token t - (W - 1) + j
    float dw[W][V] = {}, db[V] = {};
    load_taps<T, W, V>(w, bias, a.w, a.bias, d);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int c = 0; c < V; ++c) dp[j][c] = 0.f;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        Pack<T, V> r;
        const int p = t0 - (W - 1) + j;
        if (p < len) load_row<T, W, V>(r, x, state, p, D);
        else r.zero();
        r.to_f32(win[j]);
    }
    Pack<T, V> xn[BATCH], gn[BATCH];   // the next batch, requested while this one is computed
    const auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (t + i < min(len, t1 + W - 1)) {
                xn[i].stream(x + (int64_t)(t + i) * D);
                gn[i].stream(dy + (int64_t)(t + i) * D);
            } else {
                xn[i].zero();
                gn[i].zero();
            }
        }
    };
    // One batch of tokens from t.  OWN: they belong to the run and enter dw and
    // dbias; otherwise they are the W - 1 behind it.  A token past the sequence
    // has no share of anything: its g is 0, but the inputs in its window may be
    // infinite, so unless all are known to be INSIDE its dpre is chosen to be 0
    // and dw takes nothing of it.
    const auto batch = [&](int t, auto own, auto inside) {
        Pack<T, V> xi[BATCH], gi[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            xi[i] = xn[i];
            gi[i] = gn[i];
        }
        if constexpr (decltype(own)::value) fetch(t + BATCH);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const bool in = decltype(inside)::value || t + i < len;
            float g[V], out[V];
            xi[i].to_f32(win[W - 1]);
            gi[i].to_f32(g);
#pragma unroll
            for (int c = 0; c < V; ++c) {
                float v = g[c];
                if constexpr (SILU) {
                    float p = bias[c];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = __builtin_fmaf(w[j][c], win[j][c], p);
                    const float sg = sigmoid_f32(p);
                    v = in ? v * (sg * __builtin_fmaf(p, 1.f - sg, 1.f)) : 0.f;
                }
                dp[W - 1][c] = v;
                float s = w[0][c] * v;
#pragma unroll
                for (int j = 1; j < W; ++j) s = __builtin_fmaf(w[j][c], dp[W - 1 - j][c], s);
                out[c] = s;
            }
            if (decltype(own)::value && in)
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    db[c] += dp[W - 1][c];
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j][c] = __builtin_fmaf(dp[W - 1][c], win[j][c], dw[j][c]);
                }
            const int to = t + i - (W - 1);
            if (to < t1 && (to >= t0 || run == 0)) {
                const int r = to - len + (W - 1);   // row of the final state that this input is
                if (dsf && r >= 0 && r < W - 1) {
                    Pack<T, V> q;
                    float f[V];
                    q.load(dsf + (int64_t)r * D);
                    q.to_f32(f);
#pragma unroll
                    for (int c = 0; c < V; ++c) out[c] += f[c];
                }
                if (to >= 0) {
                    if (to >= len)
#pragma unroll
                        for (int c = 0; c < V; ++c) out[c] = 0.f;
                    Pack<T, V>::unstream(dx + (int64_t)to * D, out);
                } else if (ds0) {
                    Pack<T, V>::store(ds0 + (int64_t)(to + W - 1) * D, out);
                }
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    win[j][c] = win[j + 1][c];
                    dp[j][c] = dp[j + 1][c];
                }
        }
    };
    fetch(t0);
    int t = t0;
    // The loops end at the last token that has a share of a gradient, W - 1 behind
    // the run's or the sequence's last.  (A run's length is a multiple of BATCH
    // unless the sequence ends in it.)
    for (; t + BATCH <= min(t1, len); t += BATCH) batch(t, Flag<true>{}, Flag<true>{});
    for (; t < min(t1, len + W - 1); t += BATCH) batch(t, Flag<true>{}, Flag<false>{});
    if (t < min(t1, len) + W - 1) {
        batch(t, Flag<false>{}, Flag<false>{});
        t += BATCH;
    }
    const float zero[V] = {};
    for (t = max(t - (W - 1), t0); t < t1; ++t) Pack<T, V>::unstream(dx + (int64_t)t * D, zero);
    float *pw = a.ws + rest * ((int64_t)D * W) + (int64_t)d * W;
    float *pb = a.ws + (int64_t)a.B * nruns * D * W + rest * D + d;
#pragma unroll
    for (int c = 0; c < V; ++c) {
#pragma unroll
        for (int j = 0; j < W; ++j) pw[c * W + j] = dw[j][c];
        pb[c] = db[c];
    }
}

// Tokens a run: as many as leave `want` threads, so that the halo (and the
// backward's partial sums) stay small against the run; at least 4, more than
// the W - 1 tokens of the halo.  (A grid too large to launch is the launcher's
// to refuse: with many channels no length of run makes it small.)
int run_tokens(int B, int T, int64_t ncg, int most, int64_t want)
{
    int rt = most;
    while (rt > 4 && (int64_t)B * ((T + rt - 1) / rt) * ncg < want) rt >>= 1;
    return rt;
}
// (Forward of B4 T16384 D4096 in runs of 16, 32, 64, 128 and 256 tokens: 261, 227,
// 217, 215 and 211 us.)
int fwd_run(int B, int T, int64_t ncg) { return run_tokens(B, T, ncg, 256, 1 << 17); }
int bwd_run(int B, int T, int64_t ncg) { return run_tokens(B, T, ncg, 256, 1 << 17); }

// The backward holds taps, windows and sums of every channel it walks: four
// channels a thread for either type (with eight the registers leave one
// wavefront a SIMD).
constexpr int BWD_WIDE = 4;
int64_t bwd_runs(int B, int T, int D)
{
    const int rt = bwd_run(B, T, D % BWD_WIDE ? D : D / BWD_WIDE);
    return T > 0 ? (T + rt - 1) / rt : 1;
}

template <typename T, int W>
hipError_t fwd_w(const ConvArgs &a, hipStream_t s)
{
    constexpr int V = WIDE<T>;
    const bool wide = a.D % V == 0;
    const int ncg = wide ? a.D / V : a.D;
    const int rt = fwd_run(a.B, a.T, ncg), nruns = a.T > 0 ? (a.T + rt - 1) / rt : 1;
    const int64_t total = (int64_t)a.B * nruns * ncg, blocks = (total + THREADS - 1) / THREADS;
    if (!grid_fits(blocks, THREADS)) return hipErrorNotSupported;
    if (wide) (a.silu ? kda_conv_fwd_kernel<T, W, V, true> : kda_conv_fwd_kernel<T, W, V, false>)<<<(unsigned)blocks, THREADS, 0, s>>>(
        a, rt, nruns, ncg, total);
    else (a.silu ? kda_conv_fwd_kernel<T, W, 1, true> : kda_conv_fwd_kernel<T, W, 1, false>)<<<(unsigned)blocks, THREADS, 0, s>>>(
        a, rt, nruns, ncg, total);
    return hipGetLastError();
}

template <typename T, int W>
hipError_t step_w(const ConvArgs &a, hipStream_t s)
{
    constexpr int V = WIDE<T>;
    const bool wide = a.D % V == 0;
    const int ncg = wide ? a.D / V : a.D;
    const int64_t total = (int64_t)a.B * ncg, blocks = (total + THREADS - 1) / THREADS;
    if (!grid_fits(blocks, THREADS)) return hipErrorNotSupported;
    if (wide) kda_conv_step_kernel<T, W, V><<<(unsigned)blocks, THREADS, 0, s>>>(a, ncg, total);
    else kda_conv_step_kernel<T, W, 1><<<(unsigned)blocks, THREADS, 0, s>>>(a, ncg, total);
    return hipGetLastError();
}

template <typename T, int W>
hipError_t bwd_w(const ConvBwdArgs &a, hipStream_t s)
{
    constexpr int V = BWD_WIDE;
    const bool wide = a.D % V == 0;
    const int ncg = wide ? a.D / V : a.D;
    const int rt = bwd_run(a.B, a.T, ncg), nruns = a.T > 0 ? (a.T + rt - 1) / rt : 1;
    const int64_t total = (int64_t)a.B * nruns * ncg, blocks = (total + THREADS - 1) / THREADS;
    const int64_t rows = (int64_t)a.B * nruns, cols = (int64_t)a.D * W;
    const ColumnSum jobs[] = {{a.ws, a.dw, rows, cols, cols, false},
                              {a.ws + rows * cols, a.dbias, rows, a.D, a.D, false}};
    if (!grid_fits(blocks, THREADS) || !column_sums_fit(jobs, 2)) return hipErrorNotSupported;
    if (total > 0) {
        (wide ? a.silu ? kda_conv_bwd_kernel<T, W, V, true> : kda_conv_bwd_kernel<T, W, V, false>
              : a.silu ? kda_conv_bwd_kernel<T, W, 1, true> : kda_conv_bwd_kernel<T, W, 1, false>)
            <<<(unsigned)blocks, THREADS, 0, s>>>(a, rt, nruns, ncg, total);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_column_sums(jobs, 2, s);
}

template <typename F2, typename F3, typename F4>
hipError_t by_width(int W, F2 f2, F3 f3, F4 f4)
{
    (void)hipGetLastError();
    return W == 2 ? f2() : W == 3 ? f3() : W == 4 ? f4() : hipErrorInvalidValue;
}

}  // namespace

int64_t conv_bwd_workspace_floats(int B, int T, int D, int W) { return (int64_t)B * bwd_runs(B, T, D) * D * (W + 1); }

hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t s)
{
    if (a.bf16)
        return by_width(a.W, [&] { return fwd_w<uint16_t, 2>(a, s); }, [&] { return fwd_w<uint16_t, 3>(a, s); },
                        [&] { return fwd_w<uint16_t, 4>(a, s); });
    return by_width(a.W, [&] { return fwd_w<float, 2>(a, s); }, [&] { return fwd_w<float, 3>(a, s); },
                    [&] { return fwd_w<float, 4>(a, s); });
}

hipError_t launch_conv_step(const ConvArgs &a, hipStream_t s)
{
    if (a.bf16)
        return by_width(a.W, [&] { return step_w<uint16_t, 2>(a, s); }, [&] { return step_w<uint16_t, 3>(a, s); },
                        [&] { return step_w<uint16_t, 4>(a, s); });
    return by_width(a.W, [&] { return step_w<float, 2>(a, s); }, [&] { return step_w<float, 3>(a, s); },
                    [&] { return step_w<float, 4>(a, s); });
}

hipError_t launch_conv_bwd(const ConvBwdArgs &a, hipStream_t s)
{
    if (a.bf16)
        return by_width(a.W, [&] { return bwd_w<uint16_t, 2>(a, s); }, [&] { return bwd_w<uint16_t, 3>(a, s); },
                        [&] { return bwd_w<uint16_t, 4>(a, s); });
    return by_width(a.W, [&] { return bwd_w<float, 2>(a, s); }, [&] { return bwd_w<float, 3>(a, s); },
                    [&] { return bwd_w<float, 4>(a, s); });
}

}  // namespace kda
