"""GPU parity of the short convolution, the selective scan and layer norm with
their plain float64 forms, each value within the bound that those carry along
(tests/block_reference.py).  Tokens behind a sequence's end hold NaN: they enter
no result, and their outputs and gradients are zeros."""

import pytest
import torch

import block_reference as ref
from block_reference import f64
from gpu_support import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_101_amd as m
    m.load_library()
    return m


def _dev(t):
    return None if t is None else t.cuda()


def _rand(g, shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def _ragged(B, T):
    """Full, empty, one token, and in between; out-of-range values are clamped."""
    return torch.tensor(([T + 5, 0, min(1, T), (T + 1) // 2, -3] * B)[:B], dtype=torch.int32)


def _poison(lengths, *tensors):
    if lengths is None:
        return
    for t in tensors:
        if t is not None:
            for b, n in enumerate(ref.lengths_of(lengths, t.shape[0], t.shape[1])):
                t[b, n:] = float("nan")


# ------------------------------------------------------------ convolution

CONV = [  # B, T, D, W, dtype, state, ragged, silu
    (1, 1, 1, 2, F32, False, False, True), (2, 1, 8, 4, BF, True, False, True),
    (5, 2, 7, 4, BF, True, True, True), (5, 3, 12, 3, F32, True, True, False),
    (2, 5, 100, 4, BF, True, False, True), (1, 64, 64, 4, BF, False, False, True),
    (5, 67, 40, 3, BF, True, True, True), (3, 300, 33, 2, F32, True, True, True),
    (2, 513, 256, 4, BF, True, False, True), (1, 1000, 1000, 4, F32, False, False, True),
    (3, 1500, 5, 4, F32, True, True, True),   # more runs than one pass of the column sums takes
]
CONV_IDS = [f"B{c[0]}_T{c[1]}_D{c[2]}_W{c[3]}_{'bf16' if c[4] == BF else 'f32'}{'_s0' * c[5]}{'_len' * c[6]}"
            for c in CONV]


def _conv_case(c, seed=0):
    B, T, D, W, dt, state, ragged, silu = c
    g = torch.Generator().manual_seed(100 * T + D + seed)
    x = _rand(g, (B, T, D), dt)
    w, bias = _rand(g, (D, W), scale=W ** -0.5), _rand(g, (D,), scale=0.2)
    s0 = _rand(g, (B, W - 1, D), dt) if state else None
    dy, dsf = _rand(g, (B, T, D), dt), (_rand(g, (B, W - 1, D), dt) if state else None)
    lengths = _ragged(B, T) if ragged else None
    _poison(lengths, x, dy)
    return x, w, bias, s0, dy, dsf, lengths, silu


@pytest.mark.parametrize("c", CONV, ids=CONV_IDS)
def test_conv_forward(kda, c):
    x, w, bias, s0, _, _, lengths, silu = _conv_case(c)
    say(f"[conv fwd] {c}")
    y, last = kda.kda_short_conv_fwd(_dev(x), _dev(w), _dev(bias), _dev(s0), silu=silu, lengths=_dev(lengths))
    torch.cuda.synchronize()
    ry, rlast, E = ref.conv_fwd(f64(x), f64(w), f64(bias), f64(s0), lengths, silu)
    ref.check(y, ry, E, x.dtype, "y")
    assert torch.equal(f64(last), rlast)   # inputs in their own type, moved


@pytest.mark.parametrize("c", CONV, ids=CONV_IDS)
def test_conv_backward(kda, c):
    x, w, bias, s0, dy, dsf, lengths, silu = _conv_case(c)
    say(f"[conv bwd] {c}")
    got = kda.kda_short_conv_bwd(_dev(dy), _dev(x), _dev(w), _dev(bias), _dev(s0), silu=silu,
                                 dstate_final=_dev(dsf), lengths=_dev(lengths), want_dstate0=True)
    torch.cuda.synchronize()
    want = ref.conv_bwd(f64(dy), f64(x), f64(w), f64(bias), f64(s0), f64(dsf), lengths, silu)
    for k, (r, E) in want.items():
        ref.check(got[k], r, E, F32 if k in ("dw", "dbias") else x.dtype, k)


def test_conv_without_bias_and_in_place_states(kda):
    c = (3, 9, 24, 4, BF, True, True, True)
    x, w, _, s0, dy, _, lengths, _ = _conv_case(c)
    s = _dev(s0)
    y, last = kda.kda_short_conv_fwd(_dev(x), _dev(w), None, s, lengths=_dev(lengths), state_final=s)
    torch.cuda.synchronize()
    ry, rlast, E = ref.conv_fwd(f64(x), f64(w), None, f64(s0), lengths, True)
    ref.check(y, ry, E, BF, "y")
    assert last.data_ptr() == s.data_ptr() and torch.equal(f64(s), rlast)
    y2, none = kda.kda_short_conv_fwd(_dev(x), _dev(w), None, _dev(s0), lengths=_dev(lengths),
                                      output_final_state=False)
    assert none is None and torch.equal(y2, y)


@pytest.mark.parametrize("D,W,dt", [(1, 2, F32), (8, 4, BF), (36, 3, F32), (37, 4, BF), (1024, 4, BF)])
def test_conv_steps_continue_a_prompt(kda, D, W, dt):
    """A prompt, then tokens one at a time, equal the whole sequence at once."""
    B, T, more = 3, 6, 5
    g = torch.Generator().manual_seed(D)
    x = _rand(g, (B, T + more, D), dt)
    w, bias = _rand(g, (D, W)), _rand(g, (D,))
    say(f"[conv step] D={D} W={W}")
    ry, rlast, E = ref.conv_fwd(f64(x), f64(w), f64(bias), None, None, True)
    y, s = kda.kda_short_conv_fwd(_dev(x[:, :T].contiguous()), _dev(w), _dev(bias))
    ref.check(y, ry[:, :T], E[:, :T], dt, "prompt")
    for t in range(T, T + more):
        xt = _dev(x[:, t].contiguous())
        yt = kda.kda_short_conv_step(xt, _dev(w), _dev(bias), s, y=xt if t % 2 else None)   # in place every other token
        torch.cuda.synchronize()
        ref.check(yt, ry[:, t], E[:, t], dt, f"token {t}")
    assert torch.equal(f64(s), rlast)


# ------------------------------------------------------------------- scan

SCAN = [  # B, T, D, N, G, dtype, states, ragged, gated, softplus
    (1, 1, 1, 1, 1, F32, False, False, False, True), (2, 1, 64, 16, 1, BF, True, False, True, True),
    (5, 7, 10, 5, 2, F32, True, True, True, True), (1, 16, 65, 16, 1, BF, False, False, True, True),
    (5, 33, 48, 16, 3, BF, True, True, True, True), (2, 130, 96, 16, 1, F32, True, False, True, False),
    (3, 257, 40, 17, 1, BF, True, True, True, True), (1, 300, 128, 32, 2, F32, True, False, False, True),
    (2, 100, 24, 33, 2, BF, True, True, True, True), (1, 150, 70, 64, 1, BF, True, False, True, True),
    (5, 385, 72, 16, 1, BF, True, True, True, True), (1, 1000, 130, 16, 1, F32, False, False, True, True),
    (2, 700, 20, 53, 1, BF, True, True, True, True), (3, 40, 5, 16, 5, F32, True, True, True, True),
    (9, 4000, 3, 2, 1, F32, True, True, True, True),      # parameters' gradients over more than 1024 segments
    (2, 4100, 8, 16, 1, BF, False, False, True, True),    # B and C rows by the wide column sum
]
SCAN_IDS = [f"B{c[0]}_T{c[1]}_D{c[2]}_N{c[3]}_G{c[4]}_{'bf16' if c[5] == BF else 'f32'}{'_h0' * c[6]}{'_len' * c[7]}"
            for c in SCAN]


def _scan_case(c, seed=0):
    B, T, D, N, G, dt, states, ragged, gated, softplus = c
    g = torch.Generator().manual_seed(1000 * N + T + seed)
    p = dict(x=_rand(g, (B, T, D), dt), dt=_rand(g, (B, T, D), dt, 0.5),
             A=-torch.arange(1, N + 1, dtype=F32) * torch.exp(0.2 * torch.randn((D, N), generator=g)),
             Bm=_rand(g, (B, T, G, N), dt), Cm=_rand(g, (B, T, G, N), dt),
             h0=_rand(g, (B, D, N)) if states else None, D=_rand(g, (D,)) if gated else None,
             z=_rand(g, (B, T, D), dt) if gated else None, dt_bias=_rand(g, (D,)) - 2.0 if softplus else None)
    if not softplus:
        p["dt"] = p["dt"].abs() * 0.2
    dy, dh = _rand(g, (B, T, D), dt), (_rand(g, (B, D, N)) if states else None)
    lengths = _ragged(B, T) if ragged else None
    _poison(lengths, p["x"], p["dt"], p["z"], p["Bm"], p["Cm"], dy)
    return p, dy, dh, lengths, softplus


def _scan_ref(p):
    return [f64(p[k]) for k in ("x", "dt", "A", "Bm", "Cm", "h0", "D", "z", "dt_bias")]


def _scan_call(kda, p, softplus, lengths, **kw):
    d = {k: _dev(v) for k, v in p.items()}
    return kda.kda_selective_scan_fwd(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], kw.pop("h0", d["h0"]), D=d["D"],
                                      z=d["z"], dt_bias=d["dt_bias"], softplus=softplus, lengths=_dev(lengths), **kw)


@pytest.mark.parametrize("c", SCAN, ids=SCAN_IDS)
def test_scan_forward(kda, c):
    p, _, _, lengths, softplus = _scan_case(c)
    say(f"[scan fwd] {c}")
    y, h = _scan_call(kda, p, softplus, lengths)
    torch.cuda.synchronize()
    (ry, Ey), (rh, Eh), _ = ref.scan_fwd(*_scan_ref(p), softplus, lengths)
    ref.check(y, ry, Ey, p["x"].dtype, "y")
    ref.check(h, rh, Eh, F32, "h_final")


@pytest.mark.parametrize("c", SCAN, ids=SCAN_IDS)
def test_scan_backward(kda, c):
    p, dy, dh, lengths, softplus = _scan_case(c)
    say(f"[scan bwd] {c}")
    d = {k: _dev(v) for k, v in p.items()}
    got = kda.kda_selective_scan_bwd(_dev(dy), d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["h0"], D=d["D"], z=d["z"],
                                     dt_bias=d["dt_bias"], softplus=softplus, dh_final=_dev(dh),
                                     lengths=_dev(lengths), want_dh0=True)
    torch.cuda.synchronize()
    want = ref.scan_bwd(f64(dy), *_scan_ref(p), softplus, f64(dh), lengths)
    for k, v in (("dD", "D"), ("dz", "z"), ("ddt_bias", "dt_bias")):
        if p[v] is None:
            assert k not in got
            del want[k]
    assert set(got) == set(want)
    for k, (r, E) in want.items():
        ref.check(got[k], r, E, p["x"].dtype if k in ("dx", "ddt", "dz", "dB", "dC") else F32, k)


def test_scan_one_chain_equals_segments(kda):
    """Without a workspace each channel runs in one chain; the same bound holds."""
    import gated_delta_rule_101_amd.kda as K
    c = (2, 333, 80, 16, 1, F32, True, False, True, True)
    p, _, _, _, softplus = _scan_case(c)
    B, T, D, N = 2, 333, 80, 16
    assert kda.kda_selective_scan_fwd_workspace_bytes(B, T, D, N, 1) > 0
    d = {k: _dev(v) for k, v in p.items()}
    y, h = torch.empty_like(d["x"]), torch.empty_like(d["h0"])
    st = K.load_library().kda_selective_scan_fwd(
        *(K._ptr(d[k]) for k in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0")), None, K._ptr(y), K._ptr(h),
        None, 0, B, T, D, N, 1, 1, K.KDA_F32, torch.cuda.current_stream().cuda_stream)
    assert st == K.KDA_OK
    torch.cuda.synchronize()
    (ry, Ey), (rh, Eh), _ = ref.scan_fwd(*_scan_ref(p), True, None)
    ref.check(y, ry, Ey, F32, "y")
    ref.check(h, rh, Eh, F32, "h_final")


def test_scan_state_in_place(kda):
    """h_final may be h0 itself, cut into segments or not."""
    for T in (5, 700):
        c = (2, T, 100, 16, 1, BF, True, False, True, True)
        p, _, _, _, softplus = _scan_case(c)
        h = _dev(p["h0"])
        y, hf = _scan_call(kda, p, softplus, None, h0=h, h_final=h)
        y2, h2 = _scan_call(kda, p, softplus, None)
        torch.cuda.synchronize()
        assert hf.data_ptr() == h.data_ptr()
        assert torch.equal(y, y2) and torch.equal(h, h2), T


@pytest.mark.parametrize("N,G,dt", [(1, 1, F32), (4, 1, BF), (7, 2, BF), (16, 1, BF), (16, 4, F32), (18, 1, BF),
                                    (32, 2, BF), (64, 1, F32)])
def test_scan_steps_continue_a_prompt(kda, N, G, dt):
    B, T, more, D = 3, 20, 4, 36
    c = (B, T + more, D, N, G, dt, True, False, True, True)
    p, _, _, _, _ = _scan_case(c)
    say(f"[scan step] N={N} G={G}")
    (ry, Ey), (rh, Eh), _ = ref.scan_fwd(*_scan_ref(p), True, None)
    cut = {k: v[:, :T].contiguous() if v is not None and v.dim() >= 3 and k != "h0" else v for k, v in p.items()}
    y, h = _scan_call(kda, cut, True, None)
    ref.check(y, ry[:, :T], Ey[:, :T], dt, "prompt")
    d = {k: _dev(v) for k, v in p.items()}
    for t in range(T, T + more):
        one = {k: d[k][:, t].contiguous() for k in ("x", "dt", "Bm", "Cm", "z")}
        yt = kda.kda_selective_scan_step(one["x"], one["dt"], d["A"], one["Bm"], one["Cm"], h, D=d["D"], z=one["z"],
                                         dt_bias=d["dt_bias"])
        torch.cuda.synchronize()
        ref.check(yt, ry[:, t], Ey[:, t], dt, f"token {t}")
    ref.check(h, rh, Eh, F32, "h")


@pytest.mark.parametrize("B,D,N,G,dt", [(1, 300, 16, 1, BF), (4, 65, 16, 5, F32), (9, 70, 13, 2, BF), (40, 3, 64, 1, F32),
                                        (1030, 1, 3, 1, BF), (5, 600, 5, 3, F32), (130, 7, 8, 7, BF), (6, 260, 2, 1, F32),
                                        (7, 33, 32, 1, BF), (19, 17, 40, 1, BF)])
def test_scan_step_batches(kda, B, D, N, G, dt):
    """Batches of any size over channels of any number, with nothing written
    behind the last sequence's state and output."""
    c = (B, 1, D, N, G, dt, True, False, True, True)
    p, _, _, _, _ = _scan_case(c)
    d = {k: _dev(v) for k, v in p.items()}
    h = torch.full((B + 3, D, N), 7.0, device="cuda")
    y = torch.full((B + 3, D), 7.0, device="cuda", dtype=dt)
    h[:B] = d["h0"]
    kda.kda_selective_scan_step(d["x"][:, 0], d["dt"][:, 0], d["A"], d["Bm"][:, 0], d["Cm"][:, 0], h[:B], D=d["D"],
                                z=d["z"][:, 0], dt_bias=d["dt_bias"], y=y[:B])
    torch.cuda.synchronize()
    (ry, Ey), (rh, Eh), _ = ref.scan_fwd(*_scan_ref(p), True, None)
    ref.check(y[:B], ry[:, 0], Ey[:, 0], dt, "y")
    ref.check(h[:B], rh, Eh, F32, "h")
    assert (h[B:] == 7).all() and (y[B:] == 7).all()


def test_scan_without_tokens(kda):
    g = torch.Generator().manual_seed(1)
    D, N = 20, 16
    h0 = _dev(_rand(g, (2, D, N)))
    x, bc = torch.empty((2, 0, D), device="cuda"), torch.empty((2, 0, 1, N), device="cuda")
    A = -torch.ones((D, N), device="cuda")
    y, h = kda.kda_selective_scan_fwd(x, x, A, bc, bc, h0)
    assert y.shape == (2, 0, D) and torch.equal(h, h0)
    r = kda.kda_selective_scan_bwd(x, x, x, A, bc, bc, h0, dh_final=h0, want_dh0=True)
    torch.cuda.synchronize()
    assert torch.equal(r["dh0"], h0) and not r["dA"].any()
    _, s = kda.kda_short_conv_fwd(x, torch.ones((D, 3), device="cuda"), None, h0[:, :, :2].transpose(1, 2).contiguous())
    assert torch.equal(s, h0[:, :, :2].transpose(1, 2))
    e = torch.empty((0, 4, D), device="cuda")
    r = kda.kda_selective_scan_bwd(e, e, e, A, torch.empty((0, 4, 1, N), device="cuda"),
                                   torch.empty((0, 4, 1, N), device="cuda"))
    assert not r["dA"].any()
    r = kda.kda_short_conv_bwd(e, e, torch.ones((D, 3), device="cuda"))
    assert not r["dw"].any() and not r["dbias"].any()
    _, dw, db = kda.kda_layer_norm_bwd(torch.empty((0, D), device="cuda"), torch.empty((0, D), device="cuda"))
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


def test_scan_extreme_steps_and_rates(kda):
    """Time steps whose softplus is linear or underflows, rates that wipe the
    state in one token, and a rate of zero that keeps it for ever."""
    B, T, D, N = 1, 40, 8, 16
    g = torch.Generator().manual_seed(9)
    p = dict(x=_rand(g, (B, T, D)), dt=torch.linspace(-110, 60, B * T * D).reshape(B, T, D),
             A=-torch.tensor([0.0, 1e-4, 1.0, 100.0] * 4).repeat(D, 1), Bm=_rand(g, (B, T, 1, N)),
             Cm=_rand(g, (B, T, 1, N)), h0=_rand(g, (B, D, N)), D=None, z=_rand(g, (B, T, D), scale=30.0), dt_bias=None)
    y, h = _scan_call(kda, p, True, None)
    torch.cuda.synchronize()
    (ry, Ey), (rh, Eh), _ = ref.scan_fwd(*_scan_ref(p), True, None)
    ref.check(y, ry, Ey, F32, "y")
    ref.check(h, rh, Eh, F32, "h")


@pytest.mark.parametrize("T", [21, 700])
@pytest.mark.parametrize("ragged", [False, True])
def test_scan_infinite_last_token_and_rate(kda, T, ragged):
    """The places behind a sequence's last token, which share a chunk with it,
    multiply nothing into the state: an infinite input stays infinite there, and a
    rate of -infinity forgets and leaves the last token's own part."""
    c = (2, T, 40, 16, 1, F32, True, ragged, True, True)
    p, _, _, _, _ = _scan_case(c)
    last = [T - 1, T - 7] if ragged else [T - 1, T - 1]
    lengths = torch.tensor([n + 1 for n in last], dtype=torch.int32) if ragged else None
    for k in ("x", "dt", "z", "Bm", "Cm"):
        p[k] = torch.nan_to_num(p[k], nan=0.5)
    for b, t in enumerate(last):
        p["x"][b, t, 3] = float("inf")
    p["A"][5] = float("-inf")
    if ragged:
        for k in ("x", "dt", "z", "Bm", "Cm"):
            p[k][1, last[1] + 1:] = float("nan")
    y, h = _scan_call(kda, p, True, _dev(lengths))
    torch.cuda.synchronize()
    for b, t in enumerate(last):
        assert torch.equal(h[b, 3].cpu(), torch.sign(p["Bm"][b, t, 0]) * float("inf"))
    # the other channels: a rate that every positive step turns into a factor 0
    p["A"][5] = -1e30
    for b, t in enumerate(last):
        p["x"][b, t, 3] = 0.0
    (ry, Ey), (rh, Eh), _ = ref.scan_fwd(*_scan_ref(p), True, lengths)
    keep = [d for d in range(40) if d != 3]
    ref.check(y[..., keep], ry[..., keep], Ey[..., keep], F32, "y")
    ref.check(h[:, keep], rh[:, keep], Eh[:, keep], F32, "h_final")


# ------------------------------------------------------------- layer norm

NORM = [(1, 1, F32), (3, 7, BF), (37, 1111, F32), (5, 16, BF), (17, 64, BF), (9, 256, F32), (300, 257, BF),
        (33, 1024, BF), (5, 1025, F32), (600, 4096, BF), (7, 4100, F32), (3, 8200, BF), (5, 16384, F32),
        (2, 16383, BF), (2500, 24, F32)]


@pytest.mark.parametrize("rows,D,dt", NORM, ids=[f"r{r}_D{d}_{'bf16' if t == BF else 'f32'}" for r, d, t in NORM])
def test_norm_forward_and_backward(kda, rows, D, dt):
    g = torch.Generator().manual_seed(rows + D)
    x = (_rand(g, (rows, D)) * (1 + torch.arange(rows)[:, None] % 3) + 2.0).to(dt)
    dy = _rand(g, (rows, D), dt)
    w, b = 1 + _rand(g, (D,), scale=0.2), _rand(g, (D,))
    say(f"[norm] rows={rows} D={D}")
    y = kda.kda_layer_norm_fwd(_dev(x), _dev(w), _dev(b), 1e-5)
    dx, dw, db = kda.kda_layer_norm_bwd(_dev(dy), _dev(x), _dev(w), 1e-5)
    torch.cuda.synchronize()
    ry, E = ref.norm_fwd(f64(x), f64(w), f64(b), 1e-5)
    ref.check(y, ry, E, dt, "y")
    for got, (r, E), t, k in zip((dx, dw, db), ref.norm_bwd(f64(dy), f64(x), f64(w), 1e-5), (dt, F32, F32),
                                 ("dx", "dw", "db")):
        ref.check(got, r, E, t, k)


@pytest.mark.parametrize("rows,D,dt", [(700, 5120, BF), (600, 12288, F32), (520, 9000, BF), (300, 8194, BF), (280, 16381, F32),
                                       (1100, 600, F32), (2000, 200, BF)])
def test_norm_rows_of_many_workgroups(kda, rows, D, dt):
    """More rows than the workgroups take in one round."""
    test_norm_forward_and_backward(kda, rows, D, dt)


def test_norm_in_place_without_parameters_and_offset_rows(kda):
    g = torch.Generator().manual_seed(2)
    x = (_rand(g, (4, 3, 96)) + 300.0).to(F32)   # a mean far above the spread
    dy = _rand(g, (4, 3, 96))
    xd = _dev(x)
    y = kda.kda_layer_norm_fwd(xd.clone(), eps=1e-3)
    xi = xd.clone()
    assert kda.kda_layer_norm_fwd(xi, eps=1e-3, y=xi).data_ptr() == xi.data_ptr()
    dyi = _dev(dy)
    dx, dw, db = kda.kda_layer_norm_bwd(dyi, xd, eps=1e-3, want_dweight=False, want_dbias=False, dx=dyi)
    torch.cuda.synchronize()
    assert dw is None and db is None and dx.data_ptr() == dyi.data_ptr() and torch.equal(y, xi)
    ry, E = ref.norm_fwd(f64(x).reshape(12, 96), None, None, 1e-3)
    ref.check(y.reshape(12, 96), ry, E, F32, "y")
    (r, E), _, _ = ref.norm_bwd(f64(dy).reshape(12, 96), f64(x).reshape(12, 96), None, 1e-3)
    ref.check(dx.reshape(12, 96), r, E, F32, "dx")
    # one of the parameters' gradients alone
    _, dw1, none = kda.kda_layer_norm_bwd(_dev(dy), xd, eps=1e-3, want_dbias=False)
    _, none2, db1 = kda.kda_layer_norm_bwd(_dev(dy), xd, eps=1e-3, want_dweight=False)
    _, dw2, db2 = kda.kda_layer_norm_bwd(_dev(dy), xd, eps=1e-3)
    assert none is None and none2 is None and torch.equal(dw1, dw2) and torch.equal(db1, db2)


# --------------------------------------------------------- used together

def _block(kda, p, x, lengths, h0=None, s0=None):
    """norm -> convolution -> scan, as in a state-space block."""
    n = kda.kda_layer_norm_fwd(x, p["nw"], p["nb"])
    c, s = kda.kda_short_conv_fwd(n, p["cw"], p["cb"], s0, lengths=lengths)
    y, h = kda.kda_selective_scan_fwd(c, p["dt"], p["A"], p["Bm"], p["Cm"], h0, D=p["D"], z=p["z"],
                                      dt_bias=p["bias"], lengths=lengths)
    return n, c, s, y, h


def _block_params(B, T, D, N, dt):
    g = torch.Generator().manual_seed(77)
    return {k: _dev(v) for k, v in dict(
        nw=1 + _rand(g, (D,), scale=0.1), nb=_rand(g, (D,)), cw=_rand(g, (D, 4), scale=0.5), cb=_rand(g, (D,)),
        dt=_rand(g, (B, T, D), dt), A=-torch.arange(1, N + 1, dtype=F32).repeat(D, 1), Bm=_rand(g, (B, T, 1, N), dt),
        Cm=_rand(g, (B, T, 1, N), dt), D=_rand(g, (D,)), z=_rand(g, (B, T, D), dt), bias=_rand(g, (D,)) - 2,
        x=_rand(g, (B, T, D), dt), dy=_rand(g, (B, T, D), dt)).items()}


def test_block_forward_backward_and_step(kda):
    """A right-padded batch through the three operators and back, each stage
    against float64 on the values it was given; then one more token."""
    B, T, D, N, dt = 3, 150, 88, 16, BF
    p = _block_params(B, T, D, N, dt)
    lengths = torch.tensor([150, 61, 1], dtype=torch.int32)
    n, c, s, y, h = _block(kda, p, p["x"], _dev(lengths))
    scan = kda.kda_selective_scan_bwd(p["dy"], c, p["dt"], p["A"], p["Bm"], p["Cm"], D=p["D"], z=p["z"],
                                      dt_bias=p["bias"], lengths=_dev(lengths))
    conv = kda.kda_short_conv_bwd(scan["dx"], n, p["cw"], p["cb"], lengths=_dev(lengths))
    dx, dw, db = kda.kda_layer_norm_bwd(conv["dx"], p["x"], p["nw"])
    torch.cuda.synchronize()
    flat = lambda t: f64(t).reshape(B * T, D)  # noqa: E731
    r, E = ref.norm_fwd(flat(p["x"]), f64(p["nw"]), f64(p["nb"]), 1e-5)
    ref.check(n.reshape(B * T, D), r, E, dt, "norm")
    r, last, E = ref.conv_fwd(f64(n), f64(p["cw"]), f64(p["cb"]), None, lengths, True)
    ref.check(c, r, E, dt, "conv")
    assert torch.equal(f64(s), last)
    args = [f64(t) for t in (c, p["dt"], p["A"], p["Bm"], p["Cm"], None, p["D"], p["z"], p["bias"])]
    (r, E), (rh, Eh), _ = ref.scan_fwd(*args, True, lengths)
    ref.check(y, r, E, dt, "scan")
    ref.check(h, rh, Eh, F32, "state")
    for k, (r, E) in ref.scan_bwd(f64(p["dy"]), *args, True, None, lengths).items():
        if k in scan:
            ref.check(scan[k], r, E, scan[k].dtype, k)
    for k, (r, E) in ref.conv_bwd(f64(scan["dx"]), f64(n), f64(p["cw"]), f64(p["cb"]), None, None, lengths,
                                  True).items():
        if k in conv:
            ref.check(conv[k], r, E, conv[k].dtype, k)
    for got, (r, E), k in zip((dx.reshape(B * T, D), dw, db),
                              ref.norm_bwd(flat(conv["dx"]), flat(p["x"]), f64(p["nw"]), 1e-5), ("dx", "dw", "db")):
        ref.check(got, r, E, got.dtype, k)
    # one more token of every sequence, from the states the prompt left
    h_before, s_before = h.clone(), s.clone()
    one = {k: p[k][:, 0].contiguous() for k in ("x", "dt", "Bm", "Cm", "z")}
    n1 = kda.kda_layer_norm_fwd(one["x"], p["nw"], p["nb"])
    c1 = kda.kda_short_conv_step(n1, p["cw"], p["cb"], s)
    y1 = kda.kda_selective_scan_step(c1, one["dt"], p["A"], one["Bm"], one["Cm"], h, D=p["D"], z=one["z"],
                                     dt_bias=p["bias"])
    torch.cuda.synchronize()
    r, last, E = ref.conv_fwd(f64(n1)[:, None], f64(p["cw"]), f64(p["cb"]), f64(s_before), None, True)
    ref.check(c1, r[:, 0], E[:, 0], dt, "conv step")
    assert torch.equal(f64(s), last)
    (r, E), (rh, Eh), _ = ref.scan_fwd(f64(c1)[:, None], f64(one["dt"])[:, None], f64(p["A"]), f64(one["Bm"])[:, None],
                                       f64(one["Cm"])[:, None], f64(h_before), f64(p["D"]), f64(one["z"])[:, None],
                                       f64(p["bias"]), True, None)
    ref.check(y1, r[:, 0], E[:, 0], dt, "scan step")
    ref.check(h, rh, Eh, F32, "state after the step")


def _everything(kda, p, lengths):
    n, c, s, y, h = _block(kda, p, p["x"], lengths)
    scan = kda.kda_selective_scan_bwd(p["dy"], c, p["dt"], p["A"], p["Bm"], p["Cm"], D=p["D"], z=p["z"],
                                      dt_bias=p["bias"], lengths=lengths, want_dh0=True)
    conv = kda.kda_short_conv_bwd(scan["dx"], n, p["cw"], p["cb"], lengths=lengths, want_dstate0=True)
    norm = kda.kda_layer_norm_bwd(conv["dx"], p["x"], p["nw"])
    return [n, c, s, y, h, *scan.values(), *conv.values(), *norm]


def test_repeated_streams_and_graph(kda):
    """The same bits on a second call, on another stream, and from a captured
    graph replayed several times with eager work in between and other inputs."""
    p = _block_params(2, 300, 200, 16, BF)
    lengths = _dev(torch.tensor([300, 123], dtype=torch.int32))
    first = _everything(kda, p, lengths)
    again = _everything(kda, p, lengths)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _everything(kda, p, lengths)
    torch.cuda.synchronize()
    explicit = kda.kda_selective_scan_fwd(first[1], p["dt"], p["A"], p["Bm"], p["Cm"], D=p["D"], z=p["z"],
                                          dt_bias=p["bias"], lengths=lengths, stream=side)
    side.synchronize()
    for a, b, c in zip(first, again, other):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert torch.equal(explicit[0], first[3]) and torch.equal(explicit[1], first[4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _everything(kda, p, lengths)
    x0 = p["x"].clone()
    for i in range(3):
        p["x"].copy_(x0 * (1 + i))
        want = _everything(kda, p, lengths)
        torch.cuda.synchronize()
        for t in captured:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(a, b), i


def test_largest_rows_pass_32_bit_offsets(kda):
    """A convolution and a norm over 2^31 + elements: the last rows are right."""
    T, D = 600000, 4096   # 2.46e9 elements, 4.9 GB in bfloat16
    x = torch.zeros((1, T, D), dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(5)
    tail = _rand(g, (1, 8, D), BF)
    x[:, -8:] = _dev(tail)
    w, bias = _rand(g, (D, 4)), _rand(g, (D,))
    y, last = kda.kda_short_conv_fwd(x, _dev(w), _dev(bias))
    torch.cuda.synchronize()
    r, rl, E = ref.conv_fwd(f64(tail), f64(w), f64(bias), None, None, True)
    ref.check(y[:, -8:], r, E, BF, "conv")
    assert torch.equal(f64(last), rl)
    del y
    n = kda.kda_layer_norm_fwd(x.reshape(T, D), _dev(bias), None, y=x.reshape(T, D))
    torch.cuda.synchronize()
    r, E = ref.norm_fwd(f64(tail)[0], f64(bias), None, 1e-5)
    ref.check(n[-8:], r, E, BF, "norm")
