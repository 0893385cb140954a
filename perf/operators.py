"""The workloads by which the state-space operators and layer norm are measured.

Three families, each with its direction for prompts, for training and, where
it serves single tokens, its step:

* short convolution: y[t] = silu(bias + sum_j w[:, j] x[t - W + 1 + j]), per channel
* selective scan:    h[t] = exp(dt[t] A) h[t-1] + dt[t] x[t] B[t],
                     y[t] = (C[t] . h[t] + D x[t]) silu(z[t]), per channel, N states each
* layer norm:        y = (x - mean) / sqrt(var + eps) * w + b, per row

`own` selects the library's kernels; otherwise `run` computes the same with
elementary torch operations in float32.  `exact` computes them in float64,
written apart from the float32 form.
"""

import math

import torch

own = False

EPS = 1e-5
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a short chat turn through one layer of 1024 channels: latency decides
        dict(name="scan_fwd_short_prompt", op="scan_fwd", B=1, T=77, D=1024, N=16, G=1, dtype="bf16", h0=False,
             ragged=False),
        # a long document continued from an earlier state, one sequence: time has to be split to fill the device
        dict(name="scan_fwd_long_prompt", op="scan_fwd", B=1, T=16384, D=4096, N=16, G=1, dtype="bf16", h0=True,
             ragged=False),
        # the forward of a training step, 32 heads x 128 channels
        dict(name="scan_fwd_train", op="scan_fwd", B=4, T=4096, D=4096, N=16, G=1, dtype="bf16", h0=False,
             ragged=False),
        # fine-tuning in float32 on a right-padded batch, channels and tokens off every tile size, two B/C groups
        dict(name="scan_bwd_ragged_f32", op="scan_bwd", B=3, T=1001, D=1000, N=16, G=2, dtype="f32", h0=True,
             ragged=True),
        # the backward of the training step above
        dict(name="scan_bwd_train", op="scan_bwd", B=4, T=4096, D=4096, N=16, G=1, dtype="bf16", h0=False,
             ragged=False),
        # one token for each of 256 sequences, 96 x 128 channels: the serving batch
        dict(name="scan_step_batch", op="scan_step", B=256, D=12288, N=16, G=1, dtype="bf16"),
        # the convolution in front of the mixing layer, training shape
        dict(name="conv_fwd_train", op="conv_fwd", B=4, T=16384, D=4096, W=4, dtype="bf16", s0=False, ragged=False),
        # its backward
        dict(name="conv_bwd_train", op="conv_bwd", B=4, T=4096, D=4096, W=4, dtype="bf16", s0=False, ragged=False),
        # one token of one sequence: the smallest call there is
        dict(name="conv_step_single", op="conv_step", B=1, D=4096, W=4, dtype="bf16"),
        # the norm in front of a layer over a training batch's tokens
        dict(name="norm_fwd_train", op="norm_fwd", rows=65536, D=4096, dtype="bf16"),
        # its backward, with the weight's gradient reduced over the rows
        dict(name="norm_bwd_train", op="norm_bwd", rows=16384, D=4096, dtype="bf16"),
        # a few tokens in float32, an odd row length
        dict(name="norm_fwd_small_odd", op="norm_fwd", rows=37, D=1111, dtype="f32"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "conv_fwd", "conv_bwd",
                     "conv_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan_fwd", "scan_bwd"):
        B = _logint(rng, 1, 8)
        N = rng.choice([16, 16, 16, rng.randint(1, 64)])
        G = rng.choice([1, 1, 2])
        D = G * _logint(rng, 16, 4096 // G)
        cap = (1 << 28) // (B * D * N)                       # elements of the state's history
        T = _logint(rng, 1, max(1, min(8192, cap)))
        return dict(op=op, B=B, T=T, D=D, N=N, G=G, dtype=dtype, h0=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "scan_step":
        return dict(op=op, B=_logint(rng, 1, 256), D=2 * _logint(rng, 32, 6144),
                    N=rng.choice([16, 16, rng.randint(1, 64)]), G=rng.choice([1, 2]), dtype=dtype)
    if op in ("conv_fwd", "conv_bwd"):
        B = _logint(rng, 1, 8)
        D = _logint(rng, 16, 4096)
        T = _logint(rng, 1, max(1, min(16384, (1 << 26) // (B * D))))
        return dict(op=op, B=B, T=T, D=D, W=rng.choice([2, 3, 4, 4]), dtype=dtype, s0=rng.random() < 0.5,
                    ragged=rng.random() < 0.5)
    if op == "conv_step":
        return dict(op=op, B=_logint(rng, 1, 256), D=_logint(rng, 64, 12288), W=rng.choice([2, 3, 4, 4]),
                    dtype=dtype)
    D = _logint(rng, 8, 16384)
    return dict(op=op, rows=_logint(rng, 1, max(1, min(65536, (1 << 26) // D))), D=D, dtype=dtype)


def _lengths(case):
    """Tokens of each sequence of a right-padded batch: from T down to just above T / 2."""
    B, T = case["B"], case["T"]
    return [T - (b * T) // (2 * B) if case["ragged"] else T for b in range(B)]


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype="f32", scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(_DT[dtype])


def _scan_params(g, D, N):
    """Decay rates -1 .. -N spread per channel, and the bias whose softplus is a
    time step between 0.001 and 0.1: how such layers are initialised."""
    base = torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
    A = -base * torch.exp(0.2 * torch.randn((D, N), generator=g, device="cuda"))
    u = torch.rand((D,), generator=g, device="cuda")
    step = torch.exp(math.log(1e-3) + u * (math.log(0.1) - math.log(1e-3)))
    bias = step + torch.log(-torch.expm1(-step))             # softplus(bias) = step
    skip = 1.0 + 0.1 * torch.randn((D,), generator=g, device="cuda")
    return A.contiguous(), bias, skip


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], case["dtype"]
    s = {"op": op}
    if op in ("scan_fwd", "scan_bwd"):
        B, T, D, N, G = (case[k] for k in "BTDNG")
        s["A"], s["dt_bias"], s["D"] = _scan_params(g, D, N)
        s["x"] = _randn(g, (B, T, D), dt)
        s["dt"] = _randn(g, (B, T, D), dt, 0.5)
        s["Bm"] = _randn(g, (B, T, G, N), dt)
        s["Cm"] = _randn(g, (B, T, G, N), dt)
        s["z"] = _randn(g, (B, T, D), dt)
        s["h0"] = _randn(g, (B, D, N)) if case["h0"] else None
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        if op == "scan_bwd":
            s["dy"] = _randn(g, (B, T, D), dt)
            s["dh_final"] = _randn(g, (B, D, N)) if case["h0"] else None
    elif op == "scan_step":
        B, D, N, G = (case[k] for k in "BDNG")
        s["A"], s["dt_bias"], s["D"] = _scan_params(g, D, N)
        s["x"] = _randn(g, (B, D), dt)
        s["dt"] = _randn(g, (B, D), dt, 0.5)
        s["Bm"] = _randn(g, (B, G, N), dt)
        s["Cm"] = _randn(g, (B, G, N), dt)
        s["z"] = _randn(g, (B, D), dt)
        s["h"] = _randn(g, (B, D, N))
    elif op in ("conv_fwd", "conv_bwd"):
        B, T, D, W = (case[k] for k in "BTDW")
        s["x"] = _randn(g, (B, T, D), dt)
        s["w"] = _randn(g, (D, W), scale=W ** -0.5)
        s["bias"] = _randn(g, (D,), scale=0.1)
        s["s0"] = _randn(g, (B, W - 1, D), dt) if case["s0"] else None
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        if op == "conv_bwd":
            s["dy"] = _randn(g, (B, T, D), dt)
            s["ds_final"] = _randn(g, (B, W - 1, D), dt) if case["s0"] else None
    elif op == "conv_step":
        B, D, W = (case[k] for k in "BDW")
        s["x"] = _randn(g, (B, D), dt)
        s["w"] = _randn(g, (D, W), scale=W ** -0.5)
        s["bias"] = _randn(g, (D,), scale=0.1)
        s["state"] = _randn(g, (B, W - 1, D), dt)
    else:
        rows, D = case["rows"], case["D"]
        s["x"] = _randn(g, (rows, D), dt) + 0.5
        s["w"] = 1.0 + _randn(g, (D,), scale=0.1)
        s["b"] = _randn(g, (D,), scale=0.1)
        if op == "norm_bwd":
            s["dy"] = _randn(g, (rows, D), dt)
    return s


# -------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import gated_delta_rule_101_amd as kda
    op = s["op"]
    if op == "scan_fwd":
        y, h = kda.kda_selective_scan_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["h0"], D=s["D"], z=s["z"],
                                          dt_bias=s["dt_bias"], softplus=True, lengths=s["lengths"])
        return [y, h]
    if op == "scan_bwd":
        r = kda.kda_selective_scan_bwd(s["dy"], s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["h0"], D=s["D"],
                                       z=s["z"], dt_bias=s["dt_bias"], softplus=True, dh_final=s["dh_final"],
                                       lengths=s["lengths"], want_dh0=s["h0"] is not None)
        return [r[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")] + \
               ([r["dh0"]] if s["h0"] is not None else [])
    if op == "scan_step":
        y = kda.kda_selective_scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["h"], D=s["D"], z=s["z"],
                                        dt_bias=s["dt_bias"], softplus=True)
        return [y, s["h"]]
    if op == "conv_fwd":
        y, f = kda.kda_short_conv_fwd(s["x"], s["w"], s["bias"], s["s0"], silu=True, lengths=s["lengths"])
        return [y, f]
    if op == "conv_bwd":
        r = kda.kda_short_conv_bwd(s["dy"], s["x"], s["w"], s["bias"], s["s0"], silu=True,
                                   dstate_final=s["ds_final"], lengths=s["lengths"],
                                   want_dstate0=s["s0"] is not None)
        return [r[k] for k in ("dx", "dw", "dbias")] + ([r["dstate0"]] if s["s0"] is not None else [])
    if op == "conv_step":
        y = kda.kda_short_conv_step(s["x"], s["w"], s["bias"], s["state"], silu=True)
        return [y, s["state"]]
    if op == "norm_fwd":
        return [kda.kda_layer_norm_fwd(s["x"], s["w"], s["b"], EPS)]
    dx, dw, db = kda.kda_layer_norm_bwd(s["dy"], s["x"], s["w"], EPS)
    return [dx, dw, db]


# ----------------------------------------------------- plain form, float32

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _valid(lengths, B, T, device):
    """[B, T, 1] truth values: tokens inside their sequence (None: all)."""
    if lengths is None:
        return None
    return (torch.arange(T, device=device)[None, :] < lengths[:, None])[:, :, None]


def _scan_terms(s):
    """float32 time steps (0 behind a sequence's end), inputs and per-channel B, C rows."""
    x, dt = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    B, T, D = x.shape
    ok = _valid(s["lengths"], B, T, x.device)
    if ok is not None:
        x = torch.where(ok, x, torch.zeros_like(x))
        dt = torch.where(ok, dt, torch.zeros_like(dt))
    G = s["Bm"].shape[2]
    return x, dt, s["Bm"].float(), s["Cm"].float(), ok, B, T, D, G, D // G


def _states(s, x, dt, Bm, B, D, G, Dg, t0, t1, h):
    """States of tokens t0 .. t1 - 1 from the state h before them: [t1 - t0, B, D, N], and the decays."""
    N = s["A"].shape[1]
    d = dt[:, t0:t1].transpose(0, 1)
    decay = torch.exp(d[..., None] * s["A"])
    u = (d * x[:, t0:t1].transpose(0, 1)).reshape(t1 - t0, B, G, Dg, 1)
    hs = (u * Bm[:, t0:t1].transpose(0, 1).reshape(t1 - t0, B, G, 1, N)).reshape(t1 - t0, B, D, N)
    for i in range(t1 - t0):
        h = hs[i].addcmul_(decay[i], h)
    return hs, decay


_BLOCK = 512    # tokens whose states the plain form holds at once


def _plain_scan_fwd(s):
    x, dt, Bm, Cm, ok, B, T, D, G, Dg = _scan_terms(s)
    N = s["A"].shape[1]
    h = torch.zeros((B, D, N), device=x.device) if s["h0"] is None else s["h0"]
    y = torch.empty_like(x)
    for t0 in range(0, T, _BLOCK):
        t1 = min(T, t0 + _BLOCK)
        hs, _ = _states(s, x, dt, Bm, B, D, G, Dg, t0, t1, h)
        c = Cm[:, t0:t1].transpose(0, 1).reshape(t1 - t0, B, G, 1, N)
        y[:, t0:t1] = (hs.reshape(t1 - t0, B, G, Dg, N) * c).sum(-1).reshape(t1 - t0, B, D).transpose(0, 1)
        h = hs[-1].clone()
    z = s["z"].float()
    y = (y + s["D"] * x) * (z * _sigmoid(z))
    if ok is not None:
        y = torch.where(ok, y, torch.zeros_like(y))
    return [y.to(s["x"].dtype), h.clone()]


def _plain_scan_bwd(s):
    x, dt, Bm, Cm, ok, B, T, D, G, Dg = _scan_terms(s)
    N, A = s["A"].shape[1], s["A"]
    z, dy = s["z"].float(), s["dy"].float()
    if ok is not None:
        dy, z = (torch.where(ok, v, torch.zeros_like(v)) for v in (dy, z))
    sg = _sigmoid(z)
    gate = z * sg
    gy = dy * gate                                            # gradient of the ungated output
    h0 = torch.zeros((B, D, N), device=x.device) if s["h0"] is None else s["h0"]
    # states at the blocks' starts
    starts, h = [], h0
    for t0 in range(0, T, _BLOCK):
        starts.append(h)
        hs, _ = _states(s, x, dt, Bm, B, D, G, Dg, t0, min(T, t0 + _BLOCK), h)
        h = hs[-1].clone()
    carry = torch.zeros_like(h0) if s["dh_final"] is None else s["dh_final"].clone()
    dA = torch.zeros_like(A)
    dx, ddt, ypre = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dB, dC = torch.empty_like(Bm), torch.empty_like(Cm)
    for k in range(len(starts) - 1, -1, -1):
        t0, t1 = k * _BLOCK, min(T, (k + 1) * _BLOCK)
        n = t1 - t0
        hs, decay = _states(s, x, dt, Bm, B, D, G, Dg, t0, t1, starts[k])
        h5 = hs.reshape(n, B, G, Dg, N)
        b5 = Bm[:, t0:t1].transpose(0, 1).reshape(n, B, G, 1, N)
        c5 = Cm[:, t0:t1].transpose(0, 1).reshape(n, B, G, 1, N)
        g5 = gy[:, t0:t1].transpose(0, 1).reshape(n, B, G, Dg, 1)
        ypre[:, t0:t1] = (h5 * c5).sum(-1).reshape(n, B, D).transpose(0, 1)
        dC[:, t0:t1] = (h5 * g5).sum(3).transpose(0, 1)
        dh = (g5 * c5).reshape(n, B, D, N)
        for i in range(n - 1, -1, -1):
            carry = decay[i] * dh[i].add_(carry)
        d5 = dh.reshape(n, B, G, Dg, N)
        x5 = x[:, t0:t1].transpose(0, 1).reshape(n, B, G, Dg, 1)
        t5 = dt[:, t0:t1].transpose(0, 1).reshape(n, B, G, Dg, 1)
        dB[:, t0:t1] = (d5 * (t5 * x5)).sum(3).transpose(0, 1)
        du = (d5 * b5).sum(-1).reshape(n, B, D).transpose(0, 1)
        # gradient of the exponent dt A: dh * decay * (state before the token)
        prev = torch.cat([starts[k][None], hs[:-1]])
        e = dh.mul_(decay).mul_(prev)
        dA += (e * t5.reshape(n, B, D, 1)).sum((0, 1))
        ddt[:, t0:t1] = (e * A).sum(-1).transpose(0, 1) + du * x[:, t0:t1]
        dx[:, t0:t1] = du * dt[:, t0:t1]
    dx = dx + s["D"] * gy
    dD = (gy * x).sum((0, 1))
    dz = dy * (ypre + s["D"] * x) * (sg * (1.0 + z * (1.0 - sg)))
    ddt = ddt * _sigmoid(s["dt"].float() + s["dt_bias"])
    if ok is not None:
        dx, ddt, dz = (torch.where(ok, v, torch.zeros_like(v)) for v in (dx, ddt, dz))
    t = s["x"].dtype
    out = [dx.to(t), ddt.to(t), dA, dB.to(t), dC.to(t), dD, dz.to(t), ddt.sum((0, 1))]
    return out + ([carry] if s["h0"] is not None else [])


def _plain_scan_step(s):
    x, z = s["x"].float(), s["z"].float()
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    B, D = x.shape
    G, N = s["Bm"].shape[1:]
    u = (dt * x).reshape(B, G, D // G, 1)
    new = torch.exp(dt[..., None] * s["A"]) * s["h"] + (u * s["Bm"].float()[:, :, None, :]).reshape(B, D, N)
    y = (new.reshape(B, G, D // G, N) * s["Cm"].float()[:, :, None, :]).sum(-1).reshape(B, D)
    s["h"].copy_(new)
    y = (y + s["D"] * x) * (z * _sigmoid(z))
    return [y.to(s["x"].dtype), s["h"]]


def _conv_padded(s):
    """float32 inputs behind the state in front of them, [B, W - 1 + T, D]."""
    x = s["x"].float()
    B, T, D = x.shape
    W = s["w"].shape[1]
    front = torch.zeros((B, W - 1, D), device=x.device) if s["s0"] is None else s["s0"].float()
    ok = _valid(s["lengths"], B, T, x.device)
    if ok is not None:
        x = torch.where(ok, x, torch.zeros_like(x))
    return torch.cat([front, x], 1), ok, B, T, D, W


def _last_rows(xp, s, B, T, W):
    """Index [B, W - 1] of the last W - 1 rows of each sequence in the padded rows."""
    n = torch.full((B,), T, device=xp.device) if s["lengths"] is None else s["lengths"].long()
    return n[:, None] + torch.arange(W - 1, device=xp.device)[None, :]


def _plain_conv_fwd(s):
    xp, ok, B, T, D, W = _conv_padded(s)
    pre = s["bias"] + sum(xp[:, j:j + T] * s["w"][:, j] for j in range(W))
    y = pre * _sigmoid(pre)
    if ok is not None:
        y = torch.where(ok, y, torch.zeros_like(y))
    idx = _last_rows(xp, s, B, T, W)
    last = torch.gather(xp, 1, idx[:, :, None].expand(B, W - 1, D))
    return [y.to(s["x"].dtype), last.to(s["x"].dtype)]


def _plain_conv_bwd(s):
    xp, ok, B, T, D, W = _conv_padded(s)
    pre = s["bias"] + sum(xp[:, j:j + T] * s["w"][:, j] for j in range(W))
    sg = _sigmoid(pre)
    dpre = s["dy"].float() * (sg * (1.0 + pre * (1.0 - sg)))
    if ok is not None:
        dpre = torch.where(ok, dpre, torch.zeros_like(dpre))
    dxp = torch.zeros_like(xp)
    for j in range(W):
        dxp[:, j:j + T] += dpre * s["w"][:, j]
    if s["ds_final"] is not None:
        idx = _last_rows(xp, s, B, T, W)
        for j in range(W - 1):
            rows = torch.arange(B, device=xp.device)
            dxp[rows, idx[:, j]] += s["ds_final"][:, j].float()
    dw = torch.stack([(dpre * xp[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)
    t = s["x"].dtype
    out = [dxp[:, W - 1:].to(t), dw, dpre.sum((0, 1))]
    return out + ([dxp[:, :W - 1].to(t)] if s["s0"] is not None else [])


def _plain_conv_step(s):
    rows = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = s["bias"] + (rows.float() * s["w"].t()).sum(1)
    s["state"].copy_(rows[:, 1:])
    return [(pre * _sigmoid(pre)).to(s["x"].dtype), s["state"]]


def _plain_norm_fwd(s):
    x = s["x"].float()
    c = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    return [(c * r * s["w"] + s["b"]).to(s["x"].dtype)]


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    c = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    n = c * r
    g = dy * s["w"]
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    return [dx.to(s["x"].dtype), (dy * n).sum(0), dy.sum(0)]


_PLAIN = {"scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
          "conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
          "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}


def _run_plain(s):
    return _PLAIN[s["op"]](s)


# ------------------------------------------------------------------- work

def work(case):
    e, op = _SIZE[case["dtype"]], case["op"]
    if op in ("scan_fwd", "scan_bwd"):
        B, T, D, N, G = (case[k] for k in "BTDNG")
        tok, out = sum(_lengths(case)), B * T                 # padded tokens are not read, their outputs are written
        params = 4 * (D * N + 2 * D)
        state = 4 * B * D * N
        if op == "scan_fwd":
            nbytes = e * (3 * tok * D + 2 * tok * G * N + out * D) + params + state * (1 + case["h0"])
            flops = tok * D * (7 * N + 16)
        else:
            # x, dt, z, dy, B, C in; dx, ddt, dz, dB, dC and the parameters' gradients out
            nbytes = e * (4 * tok * D + 2 * tok * G * N + 3 * out * D + 2 * out * G * N) + 2 * params + \
                state * 3 * case["h0"]
            flops = tok * D * (24 * N + 40)
        return {"bytes": nbytes, "flops": flops}
    if op == "scan_step":
        B, D, N, G = (case[k] for k in "BDNG")
        return {"bytes": e * (4 * B * D + 2 * B * G * N) + 4 * (D * N + 2 * D) + 8 * B * D * N,
                "flops": B * D * (7 * N + 16)}
    if op in ("conv_fwd", "conv_bwd"):
        B, T, D, W = (case[k] for k in "BTDW")
        tok, out = sum(_lengths(case)), B * T
        state = e * B * (W - 1) * D
        if op == "conv_fwd":
            return {"bytes": e * (tok + out) * D + 4 * D * (W + 1) + state * (1 + case["s0"]),
                    "flops": tok * D * (2 * W + 6)}
        return {"bytes": e * (2 * tok + out) * D + 8 * D * (W + 1) + state * 3 * case["s0"],
                "flops": tok * D * (6 * W + 12)}
    if op == "conv_step":
        B, D, W = (case[k] for k in "BDW")
        return {"bytes": e * 2 * B * D + 2 * e * B * (W - 1) * D + 4 * D * (W + 1), "flops": B * D * (2 * W + 6)}
    rows, D = case["rows"], case["D"]
    if op == "norm_fwd":
        return {"bytes": 2 * e * rows * D + 8 * D, "flops": 8 * rows * D}
    return {"bytes": 3 * e * rows * D + 12 * D, "flops": 18 * rows * D}


# ------------------------------------------------------- float64 reference

def exact(case, seed):
    s = {k: (v.double() if torch.is_tensor(v) and v.is_floating_point() else v)
         for k, v in prepare(case, seed).items()}
    return _EXACT[case["op"]](case, s)


def _silu64(v):
    return v * torch.special.expit(v)


def _softplus64(v):
    return torch.logaddexp(v, torch.zeros((), dtype=v.dtype, device=v.device))


def _mask64(case, device):
    n = torch.tensor(_lengths(case), device=device)
    return (torch.arange(case["T"], device=device) < n[:, None]).double()


def _group(m, D):
    """[B, G, N] rows of B or C as [B, D, N], one per channel."""
    return m.repeat_interleave(D // m.shape[1], 1)


def _exact_scan_fwd(case, s):
    B, T, D, N = (case[k] for k in "BTDN")
    ok = _mask64(case, s["x"].device)
    step = _softplus64(s["dt"] + s["dt_bias"]) * ok[:, :, None]
    h = torch.zeros((B, D, N), dtype=torch.float64, device=step.device) if s["h0"] is None else s["h0"]
    y = torch.zeros_like(s["x"])
    for t in range(T):
        w = step[:, t] * s["x"][:, t]
        h = torch.exp(step[:, t, :, None] * s["A"]) * h + w[:, :, None] * _group(s["Bm"][:, t], D)
        y[:, t] = (_group(s["Cm"][:, t], D) * h).sum(2)
    y = (y + s["x"] * s["D"]) * _silu64(s["z"]) * ok[:, :, None]
    return [y, h]


def _exact_scan_bwd(case, s):
    """The reverse recurrence of the definition, token by token: with q_t the
    gradient of token t's state, q_t = C_t gy_t + exp(dt_{t+1} A) q_{t+1}."""
    B, T, D, N, G = (case[k] for k in "BTDNG")
    if 8 * B * T * D * N > 60e9:
        return None
    dev = s["x"].device
    ok = _mask64(case, dev)[:, :, None]
    raw = s["dt"] + s["dt_bias"]
    step = _softplus64(raw) * ok
    sig = torch.special.expit(s["z"])
    gy = s["dy"] * s["z"] * sig * ok
    zero = torch.zeros((B, D, N), dtype=torch.float64, device=dev)
    h = torch.empty((T + 1, B, D, N), dtype=torch.float64, device=dev)
    h[0] = zero if s["h0"] is None else s["h0"]
    read = torch.zeros_like(s["x"])
    for t in range(T):
        w = step[:, t] * s["x"][:, t]
        h[t + 1] = torch.exp(step[:, t, :, None] * s["A"]) * h[t] + w[:, :, None] * _group(s["Bm"][:, t], D)
        read[:, t] = (_group(s["Cm"][:, t], D) * h[t + 1]).sum(2)
    dA = torch.zeros_like(s["A"])
    dx, ddt = torch.zeros_like(s["x"]), torch.zeros_like(s["x"])
    dB, dC = torch.zeros_like(s["Bm"]), torch.zeros_like(s["Cm"])
    back = zero if s["dh_final"] is None else s["dh_final"]
    for t in range(T - 1, -1, -1):
        xt, dtt = s["x"][:, t], step[:, t]
        q = back + _group(s["Cm"][:, t], D) * gy[:, t, :, None]
        dC[:, t] = (gy[:, t, :, None] * h[t + 1]).reshape(B, G, D // G, N).sum(2)
        dB[:, t] = ((dtt * xt)[:, :, None] * q).reshape(B, G, D // G, N).sum(2)
        into = (_group(s["Bm"][:, t], D) * q).sum(2)
        back = torch.exp(dtt[:, :, None] * s["A"]) * q
        e = back * h[t]
        dA += (dtt[:, :, None] * e).sum(0)
        ddt[:, t] = (s["A"] * e).sum(2) + into * xt
        dx[:, t] = into * dtt
    dx = (dx + gy * s["D"]) * ok
    dz = s["dy"] * (read + s["x"] * s["D"]) * (sig + s["z"] * sig * (1 - sig)) * ok
    ddt = ddt * torch.special.expit(raw) * ok
    out = [dx, ddt, dA, dB, dC, (gy * s["x"]).sum((0, 1)), dz, ddt.sum((0, 1))]
    return out + ([back] if s["h0"] is not None else [])


def _exact_scan_step(case, s):
    D = case["D"]
    step = _softplus64(s["dt"] + s["dt_bias"])
    h = torch.exp(step[:, :, None] * s["A"]) * s["h"] + (step * s["x"])[:, :, None] * _group(s["Bm"], D)
    y = (_group(s["Cm"], D) * h).sum(2) + s["D"] * s["x"]
    return [y * _silu64(s["z"]), h]


def _exact_rows(case, s):
    """Every sequence's rows with its state in front, cut at its length: a list of [n + W - 1, D]."""
    out = []
    for b, n in enumerate(_lengths(case)):
        front = s["x"].new_zeros((case["W"] - 1, case["D"])) if s["s0"] is None else s["s0"][b]
        out.append(torch.cat([front, s["x"][b, :n]]))
    return out


def _exact_conv_fwd(case, s):
    W = case["W"]
    y = torch.zeros_like(s["x"])
    last = []
    for b, rows in enumerate(_exact_rows(case, s)):
        pre = (rows.unfold(0, W, 1) * s["w"]).sum(2) + s["bias"]
        y[b, :pre.shape[0]] = _silu64(pre)
        last.append(rows[rows.shape[0] - (W - 1):])
    return [y, torch.stack(last)]


def _exact_conv_bwd(case, s):
    W = case["W"]
    dx = torch.zeros_like(s["x"])
    dw, dbias, dfront = torch.zeros_like(s["w"]), torch.zeros_like(s["bias"]), []
    for b, rows in enumerate(_exact_rows(case, s)):
        n = rows.shape[0] - (W - 1)
        win = rows.unfold(0, W, 1)                            # [n, D, W]
        pre = (win * s["w"]).sum(2) + s["bias"]
        sig = torch.special.expit(pre)
        g = s["dy"][b, :n] * (sig + pre * sig * (1 - sig))
        dw += (g[:, :, None] * win).sum(0)
        dbias += g.sum(0)
        full = torch.nn.functional.pad(g, (0, 0, W - 1, W - 1))
        d = (full.unfold(0, W, 1) * s["w"].flip(1)).sum(2)    # [n + W - 1, D]
        if s["ds_final"] is not None:
            d[d.shape[0] - (W - 1):] += s["ds_final"][b]
        dfront.append(d[:W - 1])
        dx[b, :n] = d[W - 1:]
    return [dx, dw, dbias] + ([torch.stack(dfront)] if s["s0"] is not None else [])


def _exact_conv_step(case, s):
    rows = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = (rows.transpose(1, 2) * s["w"]).sum(2) + s["bias"]
    return [_silu64(pre), rows[:, 1:]]


def _exact_norm_fwd(case, s):
    var, mean = torch.var_mean(s["x"], -1, correction=0, keepdim=True)
    return [(s["x"] - mean) / torch.sqrt(var + EPS) * s["w"] + s["b"]]


def _exact_norm_bwd(case, s):
    D = case["D"]
    var, mean = torch.var_mean(s["x"], -1, correction=0, keepdim=True)
    sd = torch.sqrt(var + EPS)
    n = (s["x"] - mean) / sd
    g = s["dy"] * s["w"]
    dx = (g - g.sum(-1, keepdim=True) / D - n * ((g * n).sum(-1, keepdim=True) / D)) / sd
    return [dx, (s["dy"] * n).sum(0), s["dy"].sum(0)]


_EXACT = {"scan_fwd": _exact_scan_fwd, "scan_bwd": _exact_scan_bwd, "scan_step": _exact_scan_step,
          "conv_fwd": _exact_conv_fwd, "conv_bwd": _exact_conv_bwd, "conv_step": _exact_conv_step,
          "norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd}
