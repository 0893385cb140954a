"""Refusals of the short convolution, the selective scan and layer norm on the
host (no GPU needed): every call here fails validation or has nothing to do, so
none reaches a launch.  The addresses are never dereferenced."""

import ctypes
import os

import pytest
import torch

BIG = 1 << 32   # apart enough that the buffers do not overlap


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_101_amd import kda
    if not os.path.exists(kda.LIBRARY):
        from gated_delta_rule_101_amd.build_lib import build_library
        build_library()
    return kda.load_library()


@pytest.fixture(scope="module")
def st():
    from gated_delta_rule_101_amd import kda
    return kda


def _caller(fn, names, ints, sizes=None):
    """fn(*pointers, [workspace_bytes], *ints) with distinct addresses by default."""
    base = {n: (i + 1) * BIG for i, n in enumerate(names)}

    def call(**kw):
        p = {**base, **{k: v for k, v in kw.items() if k in base}}
        s = {**ints, **{k: v for k, v in kw.items() if k in ints}}
        ws = [kw.get("size", sizes(s))] if sizes else []
        return fn(*p.values(), *ws, *s.values(), None)
    call.base = base
    return call


def test_conv_refusals(lib, st):
    INV, UNS, OK = st.KDA_ERR_INVALID_ARG, st.KDA_ERR_UNSUPPORTED, st.KDA_OK
    ints = dict(B=2, T=10, D=24, W=4, silu=1, dtype=1)
    fwd = _caller(lib.kda_short_conv_fwd, ("x", "w", "bias", "s0", "lengths", "y", "sf"), ints)
    b = fwd.base
    for k in ("x", "w", "y"):
        assert fwd(**{k: None}) == INV, k
    for k in ("x", "w", "bias", "s0", "y", "sf"):
        assert fwd(**{k: b[k] + 4}) == INV, k            # misaligned
    assert fwd(lengths=b["lengths"] + 2) == INV
    assert fwd(y=b["x"]) == INV and fwd(y=b["w"] + 16) == INV
    assert fwd(sf=b["s0"] + 16) == INV                    # partial overlap; exact is allowed
    assert fwd(sf=b["y"]) == INV and fwd(sf=b["x"]) == INV
    for k in ("B", "T", "D"):
        assert fwd(**{k: -1}) == INV, k
        assert fwd(**{k: 1 << 24}) == UNS, k
    assert fwd(B=1 << 20, T=1 << 20) == UNS and fwd(B=1 << 12, T=1 << 16, D=1 << 12) == UNS
    assert fwd(W=0) == INV and fwd(W=1) == UNS and fwd(W=5) == UNS
    assert fwd(dtype=2) == INV and fwd(dtype=-1) == INV
    assert fwd(B=0) == OK and fwd(D=0) == OK and fwd(T=0, sf=None) == OK

    step = _caller(lib.kda_short_conv_step, ("x", "w", "bias", "s", "y"), dict(B=2, D=24, W=4, silu=1, dtype=1))
    b = step.base
    for k in ("x", "w", "s", "y"):
        assert step(**{k: None}) == INV, k
    assert step(y=b["x"] + 16) == INV and step(y=b["s"]) == INV and step(s=b["x"]) == INV
    assert step(W=5) == UNS and step(B=0) == OK

    need = lambda s: lib.kda_short_conv_bwd_workspace_bytes(s["B"], s["T"], s["D"], s["W"])  # noqa: E731
    assert need(dict(ints, B=2)) > 0 and need(dict(ints, W=9)) == 0 and need(dict(ints, B=0)) == 0
    bwd = _caller(lib.kda_short_conv_bwd, ("dy", "x", "w", "bias", "s0", "dsf", "lengths", "dx", "dw", "db", "ds0", "ws"),
                  ints, need)
    b = bwd.base
    for k in ("dy", "x", "w", "dx", "dw", "ws"):
        assert bwd(**{k: None}) == INV, k
    assert bwd(size=need(ints) - 1) == INV
    assert bwd(dx=b["dy"]) == INV and bwd(dw=b["w"]) == INV and bwd(ws=b["dx"] + 64) == INV
    assert bwd(ds0=b["s0"]) == INV and bwd(D=0) == OK


def test_scan_refusals(lib, st):
    INV, UNS, OK = st.KDA_ERR_INVALID_ARG, st.KDA_ERR_UNSUPPORTED, st.KDA_OK
    ints = dict(B=2, T=640, D=96, N=16, G=2, softplus=1, dtype=1)
    wsb = lambda f: (lambda s: f(s["B"], s["T"], s["D"], s["N"], s["G"]))  # noqa: E731
    need = wsb(lib.kda_selective_scan_fwd_workspace_bytes)
    assert need(ints) > 0 and need(dict(ints, T=8)) == 0 and need(dict(ints, N=65)) == 0 and need(dict(ints, G=5)) == 0
    assert need(dict(ints, B=128, D=4096)) == 0           # enough channels: no segments
    fwd = _caller(lib.kda_selective_scan_fwd, ("x", "dt", "A", "Bm", "Cm", "D_", "z", "bias", "h0", "lengths", "y", "hf",
                                               "ws"), ints, need)
    b = fwd.base
    for k in ("x", "dt", "A", "Bm", "Cm", "y"):
        assert fwd(**{k: None}) == INV, k
    for k in b:
        assert fwd(**{k: b[k] + 2}) == INV, k             # misaligned
    assert fwd(size=need(ints) - 1) == INV                # too small for a workspace that is given
    assert fwd(y=b["x"]) == INV and fwd(y=b["z"]) == INV and fwd(hf=b["h0"] + 64) == INV and fwd(hf=b["y"]) == INV
    assert fwd(ws=b["h0"]) == INV and fwd(ws=b["y"] + 256) == INV
    for k in ("B", "T", "D"):
        assert fwd(**{k: -2}) == INV and fwd(**{k: 1 << 24}) == UNS, k
    assert fwd(N=0) == INV and fwd(N=65) == UNS and fwd(G=0) == INV and fwd(G=5) == INV
    assert fwd(B=1 << 23, T=1, D=1 << 14, G=1) == UNS     # states past 2^40 elements
    assert fwd(D=1 << 21, G=1 << 20, B=1, T=1) == UNS     # rows of B and C past 2^24 elements
    assert fwd(dtype=3) == INV
    assert fwd(B=0) == OK and fwd(D=0) == OK and fwd(T=0, hf=None) == OK

    step = _caller(lib.kda_selective_scan_step, ("x", "dt", "A", "Bm", "Cm", "D_", "z", "bias", "h", "y"),
                   dict(B=2, D=96, N=16, G=2, softplus=1, dtype=0))
    b = step.base
    for k in ("x", "dt", "A", "Bm", "Cm", "h", "y"):
        assert step(**{k: None}) == INV, k
    assert step(y=b["x"]) == INV and step(y=b["h"] + 64) == INV and step(h=b["A"]) == INV
    assert step(N=65) == UNS and step(G=7) == INV and step(B=0) == OK

    need = wsb(lib.kda_selective_scan_bwd_workspace_bytes)
    assert need(ints) > 0 and need(dict(ints, T=0)) == 0
    bwd = _caller(lib.kda_selective_scan_bwd,
                  ("dy", "x", "dt", "A", "Bm", "Cm", "D_", "z", "bias", "h0", "dhf", "lengths", "dx", "ddt", "dA", "dB",
                   "dC", "dD", "dz", "dbias", "dh0", "ws"), ints, need)
    b = bwd.base
    for k in ("dy", "x", "dt", "A", "Bm", "Cm", "dx", "ddt", "dA", "dB", "dC", "ws"):
        assert bwd(**{k: None}) == INV, k
    for given, grad in (("D_", "dD"), ("z", "dz"), ("bias", "dbias")):
        assert bwd(**{given: None}) == INV and bwd(**{grad: None}) == INV   # one without the other
    assert bwd(size=need(ints) - 1) == INV
    assert bwd(dx=b["dy"]) == INV and bwd(dB=b["dC"]) == INV and bwd(dh0=b["h0"]) == INV and bwd(ws=b["dz"]) == INV
    assert bwd(D=0, G=1) == OK


def test_norm_refusals(lib, st):
    INV, UNS, OK = st.KDA_ERR_INVALID_ARG, st.KDA_ERR_UNSUPPORTED, st.KDA_OK

    def fwd(x=BIG, w=2 * BIG, b=3 * BIG, eps=1e-5, y=4 * BIG, rows=10, D=100, dtype=1):
        return lib.kda_layer_norm_fwd(x, w, b, eps, y, rows, D, dtype, None)
    assert fwd(x=None) == INV and fwd(y=None) == INV and fwd(w=2 * BIG + 4) == INV and fwd(x=BIG + 2) == INV
    assert fwd(y=BIG + 16) == INV and fwd(y=2 * BIG) == INV
    for eps in (-1.0, float("nan"), float("inf")):
        assert fwd(eps=eps) == INV
    assert fwd(rows=-1) == INV and fwd(D=0) == INV and fwd(D=16385) == UNS and fwd(rows=1 << 40) == UNS
    assert fwd(dtype=9) == INV and fwd(rows=0) == OK
    need = lib.kda_layer_norm_bwd_workspace_bytes(10, 100)
    assert need > 0 and lib.kda_layer_norm_bwd_workspace_bytes(0, 100) == 0

    def bwd(dy=BIG, x=2 * BIG, w=3 * BIG, dx=4 * BIG, dw=5 * BIG, db=6 * BIG, ws=7 * BIG, size=need, rows=10, D=100):
        return lib.kda_layer_norm_bwd(dy, x, w, 1e-5, dx, dw, db, ws, size, rows, D, 1, None)
    for k in ("dy", "x", "dx", "ws"):
        assert bwd(**{k: None}) == INV, k
    assert bwd(size=need - 4) == INV and bwd(dx=2 * BIG) == INV and bwd(dx=BIG + 16) == INV and bwd(dw=6 * BIG) == INV
    assert bwd(ws=5 * BIG) == INV and bwd(D=16385) == UNS
    assert bwd(rows=0, dw=None, db=None, ws=None, size=0) == OK


def test_binding_refuses_before_the_library(st):
    """Shapes and dtypes are errors of the binding; CPU tensors never launch."""
    import gated_delta_rule_101_amd as kda
    x = torch.zeros((2, 5, 8))
    w = torch.zeros((8, 4))
    with pytest.raises(ValueError):
        kda.kda_short_conv_fwd(x, w)                       # not on the GPU
    with pytest.raises(ValueError):
        kda.kda_short_conv_fwd(x[0], w)
    with pytest.raises(ValueError):
        kda.kda_short_conv_fwd(x, w.t())
    with pytest.raises(TypeError):
        kda.kda_short_conv_fwd(x, w.double())
    with pytest.raises(ValueError):
        kda.kda_short_conv_step(x[:, 0], w, None, torch.zeros((2, 2, 8)))
    with pytest.raises(TypeError):
        kda.kda_short_conv_bwd(x.bfloat16(), x, w)
    A, bc = torch.zeros((8, 3)), torch.zeros((2, 5, 1, 3))
    with pytest.raises(ValueError):
        kda.kda_selective_scan_fwd(x, x, A, bc, bc)        # not on the GPU
    with pytest.raises(ValueError):
        kda.kda_selective_scan_fwd(x, x, A, bc[:, :, 0], bc)
    with pytest.raises(ValueError):
        kda.kda_selective_scan_fwd(x, x[:, :4], A, bc, bc)
    with pytest.raises(TypeError):
        kda.kda_selective_scan_fwd(x, x, A, bc, bc, torch.zeros((2, 8, 3)).bfloat16())
    with pytest.raises(TypeError):
        kda.kda_selective_scan_fwd(x, x, A, bc, bc, lengths=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        kda.kda_selective_scan_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], torch.zeros((2, 8, 4)))
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x, torch.zeros(7))
    with pytest.raises(TypeError):
        kda.kda_layer_norm_bwd(x.bfloat16(), x)


def test_workspace_sizes_are_ints_of_the_shape(lib):
    """Sizes past 32 bits come back whole."""
    n = lib.kda_selective_scan_bwd_workspace_bytes(8, 16384, 12288, 64, 1)
    assert n > (1 << 32) and ctypes.c_size_t(n).value == n
