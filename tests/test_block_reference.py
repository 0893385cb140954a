"""The float64 forms of tests/block_reference.py against differences: the
directional derivative of sum(outputs * upstream) along a random direction,
(L(p + e v) - L(p - e v)) / 2e, equals <gradient, v>.  With e = 1e-5 the
truncation is e^2 times a third derivative and the rounding 1e-16 |L| / e; both
stay below 1e-7 of the terms' magnitude."""

import pytest
import torch

import block_reference as ref

E = 1e-5


def _rand(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, dtype=torch.float64) * scale


def _directional(loss, inputs, grads, g):
    for name, x in inputs.items():
        if x is None:
            continue
        v = _rand(g, *x.shape)
        hi, lo = dict(inputs), dict(inputs)
        hi[name], lo[name] = x + E * v, x - E * v
        num = (loss(hi) - loss(lo)) / (2 * E)
        ana = (grads[name] * v).sum()
        scale = float((grads[name] * v).abs().sum()) + 1.0
        assert abs(float(num - ana)) <= 1e-7 * scale, name


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 7])
def test_conv_gradients_equal_differences(W, T, silu):
    g = torch.Generator().manual_seed(10 * W + T)
    B, D = 3, 5
    lengths = [T, T // 2, 0]
    inputs = {"x": _rand(g, B, T, D), "w": _rand(g, D, W), "bias": _rand(g, D), "state0": _rand(g, B, W - 1, D)}
    dy, dsf = _rand(g, B, T, D), _rand(g, B, W - 1, D)

    def loss(p):
        y, last, _ = ref.conv_fwd(p["x"], p["w"], p["bias"], p["state0"], lengths, silu)
        return (y * dy).sum() + (last * dsf).sum()

    r = ref.conv_bwd(dy, *inputs.values(), dsf, lengths, silu)
    _directional(loss, inputs, {"x": r["dx"][0], "w": r["dw"][0], "bias": r["dbias"][0], "state0": r["dstate0"][0]}, g)


@pytest.mark.parametrize("softplus,gated", [(True, True), (False, False)])
@pytest.mark.parametrize("T,N,G", [(1, 1, 1), (9, 3, 2), (17, 16, 1)])
def test_scan_gradients_equal_differences(T, N, G, softplus, gated):
    g = torch.Generator().manual_seed(T)
    B, D = 3, 4
    lengths = [T, (T + 1) // 2, 0]
    inputs = {"x": _rand(g, B, T, D), "dt": _rand(g, B, T, D, scale=0.5), "A": -_rand(g, D, N).abs() - 0.1,
              "Bm": _rand(g, B, T, G, N), "Cm": _rand(g, B, T, G, N), "h0": _rand(g, B, D, N), "D": _rand(g, D),
              "z": _rand(g, B, T, D) if gated else None, "dt_bias": _rand(g, D)}
    if not softplus:
        inputs["dt"], inputs["dt_bias"] = inputs["dt"].abs() * 0.1, inputs["dt_bias"].abs() * 0.1
    dy, dh = _rand(g, B, T, D), _rand(g, B, D, N)

    def loss(p):
        (y, _), (h, _), _ = ref.scan_fwd(p["x"], p["dt"], p["A"], p["Bm"], p["Cm"], p["h0"], p["D"], p["z"],
                                         p["dt_bias"], softplus, lengths)
        return (y * dy).sum() + (h * dh).sum()

    r = ref.scan_bwd(dy, inputs["x"], inputs["dt"], inputs["A"], inputs["Bm"], inputs["Cm"], inputs["h0"],
                     inputs["D"], inputs["z"], inputs["dt_bias"], softplus, dh, lengths)
    names = {"x": "dx", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "h0": "dh0", "D": "dD", "z": "dz",
             "dt_bias": "ddt_bias"}
    _directional(loss, inputs, {k: r[n][0] for k, n in names.items()}, g)


def test_norm_gradients_equal_differences():
    g = torch.Generator().manual_seed(3)
    inputs = {"x": _rand(g, 5, 13), "w": _rand(g, 13), "b": _rand(g, 13)}
    dy = _rand(g, 5, 13)
    (dx, _), (dw, _), (db, _) = ref.norm_bwd(dy, inputs["x"], inputs["w"], 1e-5)
    _directional(lambda p: (ref.norm_fwd(p["x"], p["w"], p["b"], 1e-5)[0] * dy).sum(), inputs,
                 {"x": dx, "w": dw, "b": db}, g)


def test_bounds_hold_for_float32_and_catch_a_wrong_token():
    """The plain recurrence in float32 stays inside its bound, and dropping one
    token's input leaves it."""
    g = torch.Generator().manual_seed(4)
    B, T, D, N = 1, 40, 6, 16
    x, dt = (torch.randn((B, T, D), generator=g) for _ in range(2))
    A = -torch.arange(1, N + 1, dtype=torch.float32).repeat(D, 1)
    Bm, Cm = (torch.randn((B, T, 1, N), generator=g) for _ in range(2))
    args = [t.double() for t in (x, dt, A, Bm, Cm)]
    (y, Ey), (h, Eh), _ = ref.scan_fwd(*args, None, None, None, None, True, None)

    def plain(x):
        h, out = torch.zeros((B, D, N)), torch.empty_like(x)
        for t in range(T):
            s = torch.nn.functional.softplus(dt[:, t])
            h = torch.exp(s[..., None] * A) * h + (s * x[:, t])[..., None] * Bm[:, t]
            out[:, t] = (h * Cm[:, t]).sum(-1)
        return out, h

    got, hg = plain(x)
    ref.check(got, y, Ey, torch.float32, "y")
    ref.check(hg, h, Eh, torch.float32, "h")
    x[0, 20, 3] = 0.0
    with pytest.raises(AssertionError):
        ref.check(plain(x)[0], y, Ey, torch.float32, "y")
