"""The block operators where a value overflows, a sequence ends inside a chunk
or states are padded: what does not belong to a sequence or does not exist must
not reach a sum, not even as 0 times infinity.

Expectations come from the formulas.  Most results do not depend on the one
value that is infinite here; those are compared with the float64 form of the
same inputs with that value 0, in the bounds of tests/block_reference.py."""

import pytest
import torch

import block_reference as ref
from block_reference import f64
from gpu_support import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_101_amd as m
    m.load_library()
    return m


def _dev(t):
    return None if t is None else t.cuda()


def _scan_params(B, T, D, N, G, dt, seed):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, scale=1.0, dtype=F32):
        return (torch.randn(shape, generator=g) * scale).to(dtype)

    return dict(x=r(B, T, D, dtype=dt), dt=r(B, T, D, scale=0.5, dtype=dt), A=-torch.rand((D, N), generator=g) - 0.1,
                Bm=r(B, T, G, N, dtype=dt), Cm=r(B, T, G, N, dtype=dt), h0=r(B, D, N), D=r(D), z=r(B, T, D, dtype=dt),
                dt_bias=r(D) - 2.0, dy=r(B, T, D, dtype=dt), dh=r(B, D, N))


def _scan_bwd(kda, p, lengths):
    d = {k: _dev(v) for k, v in p.items()}
    got = kda.kda_selective_scan_bwd(d["dy"], d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["h0"], D=d["D"], z=d["z"],
                                     dt_bias=d["dt_bias"], dh_final=d["dh"], lengths=_dev(lengths), want_dh0=True)
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in got.items()}


def _scan_ref(p, lengths):
    args = [f64(p[k]) for k in ("x", "dt", "A", "Bm", "Cm", "h0", "D", "z", "dt_bias")]
    return ref.scan_bwd(f64(p["dy"]), *args, True, f64(p["dh"]), lengths)


def _scan_fwd(kda, p, lengths=None):
    d = {k: _dev(v) for k, v in p.items()}
    y, h = kda.kda_selective_scan_fwd(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["h0"], D=d["D"], z=d["z"],
                                      dt_bias=d["dt_bias"], lengths=_dev(lengths))
    torch.cuda.synchronize()
    return y.cpu(), h.cpu()


def _check(got, want, where, name):
    r, E = want
    ref.check(got[where], r[where], E[where], got.dtype, name)


# ------------------------------------------- behind a sequence's last token

@pytest.mark.parametrize("T,short,N,dt", [(21, 0, 16, F32), (21, 6, 16, F32), (21, 17, 16, BF), (37, 20, 20, F32), (64, 1, 16, F32),
                                          (700, 0, 16, F32), (700, 7, 16, BF), (700, 333, 40, F32), (700, 1, 17, F32)])
def test_scan_backward_infinite_last_token(kda, T, short, N, dt):
    """An infinite last input x of one channel enters that token's ddt, dz, dB and dC
    and the sums dD and ddt_bias; dx, dA and dh0 do not depend on it, and neither
    do the other tokens, which behind the end are zeros."""
    B, D, ch = 2, 40, 3
    p = _scan_params(B, T, D, N, 1, dt, T + short)
    last = T - 1 - short
    lengths = torch.tensor([T, last + 1], dtype=torch.int32) if short else None
    for k in ("x", "dt", "z", "Bm", "Cm", "dy"):
        p[k][1, last + 1:] = float("nan")
    p["x"][1, last, ch] = 0.0
    want = _scan_ref(p, lengths)
    p["x"][1, last, ch] = INF
    say(f"[scan bwd, infinite last token] T={T} length={last + 1} N={N}")
    got = _scan_bwd(kda, p, lengths)
    for k in ("dx", "dA", "dh0"):
        _check(got[k], want[k], (slice(None),), k)
    others = [d for d in range(D) if d != ch]
    for k in ("dD", "ddt_bias"):
        _check(got[k], want[k], others, k)
        assert torch.isinf(got[k][ch]), k
    for k in ("ddt", "dz"):
        _check(got[k], want[k], (slice(None), slice(None), others), k)
        assert not torch.isfinite(got[k][1, last, ch]), k   # (dz takes infinities of both signs)
    for k in ("ddt", "dz", "dB", "dC"):
        _check(got[k], want[k], (0,), k)
        _check(got[k], want[k], (1, slice(0, last)), k)
        assert (got[k][1, last + 1:] == 0).all(), k
    assert torch.isinf(got["dB"][1, last]).all() and torch.isinf(got["dC"][1, last]).all()


@pytest.mark.parametrize("T,short,W", [(5, 0, 4), (9, 3, 4), (14, 1, 3), (300, 0, 2), (301, 40, 4)])
@pytest.mark.parametrize("value", [INF, float("nan")])
def test_conv_backward_infinite_last_token(kda, T, short, W, value):
    """Without the SiLU only dw's last tap takes the last input."""
    B, D, ch = 2, 12, 5
    g = torch.Generator().manual_seed(T)
    x, dy = torch.randn((B, T, D), generator=g), torch.randn((B, T, D), generator=g)
    w, s0, dsf = (torch.randn(s, generator=g) for s in ((D, W), (B, W - 1, D), (B, W - 1, D)))
    last = T - 1 - short
    lengths = torch.tensor([T, last + 1], dtype=torch.int32) if short else None
    x[1, last + 1:] = dy[1, last + 1:] = float("nan")
    x[1, last, ch] = 0.0
    want = ref.conv_bwd(f64(dy), f64(x), f64(w), None, f64(s0), f64(dsf), lengths, False)
    x[1, last, ch] = value
    say(f"[conv bwd, {value} last token] T={T} length={last + 1} W={W}")
    got = kda.kda_short_conv_bwd(_dev(dy), _dev(x), _dev(w), None, _dev(s0), silu=False, dstate_final=_dev(dsf),
                                 lengths=_dev(lengths), want_dstate0=True)
    torch.cuda.synchronize()
    got = {k: v.cpu() for k, v in got.items()}
    assert not torch.isfinite(got["dw"][ch, W - 1])
    got["dw"][ch, W - 1] = want["dw"][0][ch, W - 1].float()
    for k in want:
        _check(got[k], want[k], (slice(None),), k)


# ------------------------------------------------------------ padded states

def _positive(p):
    """Signs for which no two infinities meet with opposite ones; rates that keep a state."""
    for k in ("x", "Bm", "Cm", "z", "dy", "h0", "D", "dh"):
        p[k] = p[k].abs() + 0.1
    p["A"] = p["A"] * 1e-4
    return p


@pytest.mark.parametrize("T", [3, 40, 700])
@pytest.mark.parametrize("N", [1, 5, 16, 17, 33, 53])
def test_scan_forward_infinite_input(kda, N, T):
    """One infinite input makes its channel's outputs infinite from there on, for
    any number of states; the other channels do not see it."""
    B, D, ch, at = 2, 40, 2, T // 2
    p = _positive(_scan_params(B, T, D, N, 1, F32, N + T))
    p["x"][0, at, ch] = 0.0
    args = [f64(p[k]) for k in ("x", "dt", "A", "Bm", "Cm", "h0", "D", "z", "dt_bias")]
    want_y, want_h, _ = ref.scan_fwd(*args, True, None)
    p["x"][0, at, ch] = INF
    say(f"[scan fwd, infinite input] T={T} N={N}")
    y, h = _scan_fwd(kda, p)
    assert (y[0, at:, ch] == INF).all() and (h[0, ch] == INF).all()
    others = [d for d in range(D) if d != ch]
    _check(y, want_y, (slice(None), slice(None), others), "y")
    _check(y, want_y, (1,), "y")
    _check(y, want_y, (0, slice(0, at)), "y")
    _check(h, want_h, (slice(None), others), "h_final")
    _check(h, want_h, (1,), "h_final")


@pytest.mark.parametrize("T", [21, 700])
def test_scan_forward_infinite_time_step(kda, T):
    """An infinite time step forgets the state; its own infinite input stays."""
    B, D, N, ch, at = 1, 20, 5, 2, T // 2
    p = _positive(_scan_params(B, T, D, N, 1, F32, T))
    p["dt"][0, at, ch] = INF
    say(f"[scan fwd, infinite step] T={T}")
    y, h = _scan_fwd(kda, p)
    assert (y[0, at:, ch] == INF).all() and (h[0, ch] == INF).all()
    assert torch.isfinite(y[:, :, [d for d in range(D) if d != ch]]).all()


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N", [1, 3, 5, 6, 12, 16, 20, 33, 48])
def test_scan_step_infinite_input(kda, N, dt):
    B, D, ch = 5, 36, 2
    p = _positive(_scan_params(B, 1, D, N, 1, dt, N))
    p["x"][1, 0, ch] = 0.0
    args = [f64(p[k]) for k in ("x", "dt", "A", "Bm", "Cm", "h0", "D", "z", "dt_bias")]
    (ry, Ey), (rh, Eh), _ = ref.scan_fwd(*args, True, None)
    p["x"][1, 0, ch] = INF
    d = {k: _dev(v) for k, v in p.items()}
    say(f"[scan step, infinite input] N={N}")
    y = kda.kda_selective_scan_step(d["x"][:, 0], d["dt"][:, 0], d["A"], d["Bm"][:, 0], d["Cm"][:, 0], d["h0"],
                                    D=d["D"], z=d["z"][:, 0], dt_bias=d["dt_bias"])
    torch.cuda.synchronize()
    y, h = y.cpu(), d["h0"].cpu()
    assert y[1, ch] == INF and (h[1, ch] == INF).all()
    y[1, ch], h[1, ch] = ry[1, 0, ch].to(dt), rh[1, ch].float()
    _check(y, (ry[:, 0], Ey[:, 0]), (slice(None),), "y")
    _check(h, (rh, Eh), (slice(None),), "h")


@pytest.mark.parametrize("T", [7, 40, 700])
@pytest.mark.parametrize("N", [1, 5, 16, 17, 33, 53])
def test_scan_backward_infinite_upstream(kda, N, T):
    """One infinite dy makes its channel's dx and that token's dB and dC infinite from
    there backwards, and that token's dz; the other channels do not see it."""
    B, D, ch, at = 2, 40, 2, T // 2
    p = _positive(_scan_params(B, T, D, N, 1, F32, N + T))
    p["dy"][0, at, ch] = 0.0
    want = _scan_ref(p, None)
    p["dy"][0, at, ch] = INF
    say(f"[scan bwd, infinite upstream] T={T} N={N}")
    got = _scan_bwd(kda, p, None)
    assert (got["dx"][0, :at + 1, ch] == INF).all() and got["dz"][0, at, ch] == INF
    assert (got["dB"][0, :at + 1] == INF).all() and (got["dC"][0, at] == INF).all()
    assert (got["dA"][ch] == INF).all() and (got["dh0"][0, ch] == INF).all() and got["dD"][ch] == INF
    others = [d for d in range(D) if d != ch]
    for k in ("dx", "ddt", "dz"):
        _check(got[k], want[k], (slice(None), slice(None), others), k)
    for k in ("dx", "ddt", "dz", "dB"):
        _check(got[k], want[k], (0, slice(at + 1, T)), k)
        _check(got[k], want[k], (1,), k)
    _check(got["dC"], want["dC"], (0, [t for t in range(T) if t != at]), "dC")
    _check(got["dC"], want["dC"], (1,), "dC")
    for k in ("dA", "dD", "ddt_bias"):
        _check(got[k], want[k], others, k)
    _check(got["dh0"], want["dh0"], (slice(None), others), "dh0")


@pytest.mark.parametrize("N", [1, 5, 17, 33])
def test_scan_backward_infinite_input_and_padded_states(kda, N):
    """dz takes the read of the infinite state, which is infinite and not NaN."""
    B, T, D, ch = 1, 32, 20, 2
    p = _positive(_scan_params(B, T, D, N, 1, F32, N))
    p["x"][0, T - 1, ch] = INF
    say(f"[scan bwd, infinite input] N={N}")
    got = _scan_bwd(kda, p, None)
    assert got["dz"][0, T - 1, ch] == INF and got["ddt"][0, T - 1, ch] == INF
    for k in ("dx", "dA", "dh0"):
        assert torch.isfinite(got[k]).all(), k


@pytest.mark.parametrize("T", [5, 32, 300])
@pytest.mark.parametrize("D,G,N", [(1, 1, 16), (40, 1, 16), (65, 1, 16), (100, 2, 5), (130, 1, 33)])
def test_scan_backward_infinite_last_channel(kda, D, G, N, T):
    """Lanes behind a group's last channel repeat it; what is infinite in it enters the
    rows of B and C once, as infinity."""
    p = _positive(_scan_params(2, T, D, N, G, F32, D + T))
    say(f"[scan bwd, infinite last channel] D={D} G={G} T={T}")
    at = T // 2
    p["x"][0, at, D - 1] = INF                 # from there on the state is infinite
    p["dy"][1, at, D - 1] = INF                # back from there its gradient is
    got = _scan_bwd(kda, p, None)
    assert (got["dB"][0, at, G - 1] == INF).all() and (got["dC"][0, at:, G - 1] == INF).all()
    assert (got["dB"][1, :at + 1, G - 1] == INF).all() and (got["dC"][1, at, G - 1] == INF).all()
    for t in [t for t in range(T) if t != at]:
        assert torch.isfinite(got["dB"][0, t]).all() and torch.isfinite(got["dC"][1, t]).all(), t
    assert torch.isfinite(got["dB"][1, at + 1:]).all() and torch.isfinite(got["dC"][0, :at]).all()
    for g in range(G - 1):
        assert torch.isfinite(got["dB"][:, :, g]).all() and torch.isfinite(got["dC"][:, :, g]).all()


# ------------------------------------------------------ without skip and gate

@pytest.mark.parametrize("N", [1, 16, 20])
@pytest.mark.parametrize("gated", [False, True])
def test_scan_infinite_input_without_skip(kda, gated, N):
    """No D: nothing is added to the read, not 0 times an infinite input; nor is anything to dx and dz."""
    B, T, D, ch, at = 2, 40, 24, 2, 20
    p = _positive(_scan_params(B, T, D, N, 1, F32, N))
    p["D"] = None
    if not gated:
        p["z"] = None
    p["x"][0, at, ch] = INF
    say(f"[scan without D, infinite input] N={N} gated={gated}")
    y, h = _scan_fwd(kda, p)
    assert (y[0, at:, ch] == INF).all() and (h[0, ch] == INF).all()
    assert torch.isfinite(y[1]).all() and torch.isfinite(y[0, :at]).all()
    d = {k: _dev(v) for k, v in p.items()}
    h = d["h0"].clone()
    one = {k: None if d[k] is None else d[k][:, at].contiguous() for k in ("x", "dt", "Bm", "Cm", "z")}
    y = kda.kda_selective_scan_step(one["x"], one["dt"], d["A"], one["Bm"], one["Cm"], h, z=one["z"],
                                    dt_bias=d["dt_bias"])
    torch.cuda.synchronize()
    assert y[0, ch] == INF and torch.isfinite(y[1]).all()


@pytest.mark.parametrize("gated", [False, True])
def test_scan_backward_infinite_upstream_without_skip(kda, gated):
    B, T, D, N, ch, at = 2, 40, 24, 16, 2, 20
    p = _positive(_scan_params(B, T, D, N, 1, F32, 3))
    p["D"] = None
    if not gated:
        p["z"] = None
    p["dy"][0, at, ch] = INF
    p["x"][1, T - 1, ch] = INF
    say(f"[scan bwd without D, infinite upstream and input] gated={gated}")
    got = _scan_bwd(kda, p, None)
    assert (got["dx"][0, :at + 1, ch] == INF).all() and torch.isfinite(got["dx"][1]).all()
    if gated:
        assert got["dz"][0, at, ch] == INF and got["dz"][1, T - 1, ch] == INF
    else:
        assert "dz" not in got
    assert "dD" not in got


# -------------------------------------------------------------------- rates

@pytest.mark.parametrize("T,short", [(1, 0), (21, 0), (21, 6), (700, 0), (700, 400)])
def test_scan_backward_lowest_finite_rates(kda, T, short):
    """A finite rate whose base-2 form is not finite forgets at every positive step and
    changes nothing in the places without one."""
    B, D, N = 2, 20, 16
    p = _scan_params(B, T, D, N, 1, F32, T + short)
    p["A"][4] = -3e38
    p["A"][7, ::3] = torch.finfo(F32).min
    lengths = torch.tensor([T, T - short], dtype=torch.int32) if short else None
    say(f"[scan bwd, lowest rates] T={T} length={T - short}")
    got, want = _scan_bwd(kda, p, lengths), _scan_ref(p, lengths)
    for k in want:
        _check(got[k], want[k], (slice(None),), k)


@pytest.mark.parametrize("T", [21, 300])
def test_scan_backward_infinite_rates(kda, T):
    """-infinity, which forgets at once: the gradients of the lowest finite rate."""
    p = _scan_params(2, T, 20, 16, 1, F32, T)
    lengths = torch.tensor([T, T - 6], dtype=torch.int32)
    p["A"][4] = -3e38
    want = _scan_ref(p, lengths)
    p["A"][4] = -INF
    say(f"[scan bwd, infinite rates] T={T}")
    got = _scan_bwd(kda, p, lengths)
    for k in want:
        _check(got[k], want[k], (slice(None),), k)


# ----------------------------------------------------------- nothing to sum

@pytest.mark.parametrize("G", [1, 3])
def test_scan_backward_without_channels(kda, G):
    """dB and dC have rows without any channel: zeros."""
    x, A = torch.empty((2, 3, 0), device="cuda"), torch.empty((0, 4), device="cuda")
    bc = torch.ones((2, 3, G, 4), device="cuda")
    stale = [torch.full_like(bc, 7.0) for _ in range(8)]   # what fresh allocations would find
    torch.cuda.synchronize()
    del stale
    got = kda.kda_selective_scan_bwd(x, x, x, A, bc, bc, want_dh0=True)
    torch.cuda.synchronize()
    assert got["dB"].shape == bc.shape and not got["dB"].any() and not got["dC"].any()
    assert got["dx"].shape == x.shape and got["dA"].shape == A.shape and got["dh0"].shape == (2, 0, 4)
