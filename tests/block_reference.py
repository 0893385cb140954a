"""Plain float64 forms of the short convolution, the selective scan and layer
norm with their gradients, each with a bound on what float32 arithmetic may
lose, carried along the same formulas to first order.

Notation: U = 2^-24, half a float32 step relative to the value.  A bound Eq
is what the float32 value of q may be off.  Each elementary operation adds U
times its result; a sum of k terms k U times the sum of their magnitudes,
whatever its order; exp2 and reciprocal two steps; exp(w) formed as
exp2(w log2 e) carries the rounding of its argument, 2 U |w|.  A stored
output adds half a step of its type.  `bound` doubles the first-order sum for
the products of errors that it leaves out.
"""

from __future__ import annotations

import torch

U = 2.0 ** -24
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # eps / 2


def f64(t):
    return None if t is None else t.detach().cpu().double()


def bound(E, ref, dtype):
    return 2.0 * E + STEP[dtype] * (ref.abs() + 2.0 * E)


def check(got, ref, E, dtype, what):
    """got (any device) against ref within the bound; both finite."""
    assert got.dtype == dtype, what
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    if g.numel() == 0:
        return
    assert torch.isfinite(g).all(), what
    over = (g - ref).abs() - bound(E, ref, dtype) - 1e-37   # below float32's normal range
    worst = float(over.max())
    assert worst <= 0, f"{what}: off by {float((g - ref).abs().max()):.3e}, {worst:.3e} past its bound"


def lengths_of(lengths, B, T):
    if lengths is None:
        return [T] * B
    return [min(max(int(n), 0), T) for n in lengths]


def _silu(p):
    s = torch.sigmoid(p)
    return p * s, s * (1 + p * (1 - s)), s


def _silu_loss(p):
    """Relative loss of sigmoid, and so of silu, at p."""
    return U * (2 * p.abs() + 8)


# ------------------------------------------------------------ convolution

def conv_fwd(x, w, bias, state0, lengths, silu):
    """y, state_final and E of y."""
    B, T, D = x.shape
    W = w.shape[1]
    bias = torch.zeros(D, dtype=torch.float64) if bias is None else bias
    y, E = torch.zeros_like(x), torch.zeros_like(x)
    last = torch.zeros((B, W - 1, D), dtype=torch.float64)
    for b, n in enumerate(lengths_of(lengths, B, T)):
        front = torch.zeros((W - 1, D), dtype=torch.float64) if state0 is None else state0[b]
        rows = torch.cat([front, x[b, :n]])
        last[b] = rows[n:]
        p, m = bias.expand(n, D).clone(), bias.abs().expand(n, D).clone()
        for j in range(W):
            p = p + rows[j:j + n] * w[:, j]
            m = m + (rows[j:j + n] * w[:, j]).abs()
        Ep = U * (W + 2) * m
        if silu:
            y[b, :n] = _silu(p)[0]
            E[b, :n] = 1.1 * Ep + y[b, :n].abs() * _silu_loss(p)   # |silu'| < 1.1
        else:
            y[b, :n], E[b, :n] = p, Ep
    return y, last, E


def conv_bwd(dy, x, w, bias, state0, dstate_final, lengths, silu):
    """dict name -> (gradient, E)."""
    B, T, D = x.shape
    W = w.shape[1]
    bias = torch.zeros(D, dtype=torch.float64) if bias is None else bias
    dx, Edx = torch.zeros_like(x), torch.zeros_like(x)
    dw, Edw, mdw = (torch.zeros_like(w) for _ in range(3))
    db, Edb, mdb = (torch.zeros(D, dtype=torch.float64) for _ in range(3))
    ds, Eds = (torch.zeros((B, W - 1, D), dtype=torch.float64) for _ in range(2))
    for b, n in enumerate(lengths_of(lengths, B, T)):
        front = torch.zeros((W - 1, D), dtype=torch.float64) if state0 is None else state0[b]
        rows = torch.cat([front, x[b, :n]])
        p, m = bias.expand(n, D).clone(), bias.abs().expand(n, D).clone()
        for j in range(W):
            p = p + rows[j:j + n] * w[:, j]
            m = m + (rows[j:j + n] * w[:, j]).abs()
        g = dy[b, :n]
        if silu:
            _, der, sg = _silu(p)
            dp = g * der
            # |silu''| <= 1/2; silu' = sg (1 + p (1 - sg)) loses by its terms' magnitudes
            Edp = g.abs() * (0.5 * U * (W + 2) * m + sg * (1 + p.abs()) * (_silu_loss(p) + 4 * U))
        else:
            dp, Edp = g, torch.zeros_like(g)
        drows, Er = torch.zeros_like(rows), torch.zeros_like(rows)
        for j in range(W):
            drows[j:j + n] += dp * w[:, j]
            Er[j:j + n] += w[:, j].abs() * (Edp + U * (W + 2) * dp.abs())
            dw[:, j] += (dp * rows[j:j + n]).sum(0)
            mdw[:, j] += (dp * rows[j:j + n]).abs().sum(0)
            Edw[:, j] += (Edp * rows[j:j + n].abs()).sum(0)
        db += dp.sum(0)
        mdb += dp.abs().sum(0)
        Edb += Edp.sum(0)
        if dstate_final is not None:
            drows[n:] += dstate_final[b]
            Er[n:] += U * (drows[n:].abs() + dstate_final[b].abs())
        dx[b, :n], Edx[b, :n] = drows[W - 1:], Er[W - 1:]
        ds[b], Eds[b] = drows[:W - 1], Er[:W - 1]
    terms = U * (B * T + 32)
    return {"dx": (dx, Edx), "dw": (dw, Edw + terms * mdw), "dbias": (db, Edb + terms * mdb), "dstate0": (ds, Eds)}


# ------------------------------------------------------------------- scan

def _scan_inputs(x, dt, dt_bias, z, softplus, lengths):
    B, T, D = x.shape
    ok = torch.zeros((B, T, 1), dtype=torch.float64)
    for b, n in enumerate(lengths_of(lengths, B, T)):
        ok[b, :n] = 1
    keep = ok > 0
    x = torch.where(keep, x, 0.0)
    v = torch.where(keep, dt if dt_bias is None else dt + dt_bias, 0.0)
    if softplus:
        s = torch.where(keep, torch.logaddexp(v, torch.zeros_like(v)), 0.0)
        ds = torch.where(keep, torch.sigmoid(v), 0.0)
        Es = U * (8 + 4 * v.abs()) * (s + ds)
    else:
        s, ds, Es = v, ok.expand_as(v), U * v.abs()
    if z is None:
        gate, dgate, sg, Eg = ok.expand_as(x), torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    else:
        zz = torch.where(keep, z, 0.0)
        gate, dgate, sg = _silu(zz)
        Eg = gate.abs() * _silu_loss(zz)
    return x, v, s, ds, Es, gate, dgate, sg, Eg, keep


def _decay(s, Es, A, T):
    """a, and its relative loss; the joins of segments take a segment's decay
    from its summed time steps, a sum of at most T terms."""
    sA = (s[:, :, None] * A).abs()
    return torch.exp(s[:, :, None] * A), A.abs() * Es[:, :, None] + (4 + T) * U * sA + 3 * U


def _rows(m, D):
    return m.repeat_interleave(D // m.shape[1], 1)


def scan_fwd(x, dt, A, Bm, Cm, h0, Dskip, z, dt_bias, softplus, lengths):
    """(y, E), (h_final, E), and what the gradients need."""
    B, T, D = x.shape
    N = A.shape[1]
    x, v, s, ds, Es, gate, dgate, sg, Eg, keep = _scan_inputs(x, dt, dt_bias, z, softplus, lengths)
    skip = torch.zeros(D, dtype=torch.float64) if Dskip is None else Dskip
    h = torch.zeros((B, D, N), dtype=torch.float64) if h0 is None else h0
    Eh = torch.zeros_like(h)
    hs, Ehs, r, Er = [h], [Eh], torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T):
        k = keep[:, t, :, None]
        bb = torch.where(k, _rows(Bm[:, t], D), 0.0)
        cc = torch.where(k, _rows(Cm[:, t], D), 0.0)
        a, ra = _decay(s[:, t], Es[:, t], A, T)
        u = (s[:, t] * x[:, t])[:, :, None]
        Eu = (x[:, t].abs() * Es[:, t])[:, :, None] + U * u.abs()
        new = a * h + u * bb
        Eh = torch.where(k, a * Eh + a * ra * h.abs() + bb.abs() * Eu + U * (2 * (u * bb).abs() + new.abs()), Eh)
        h = torch.where(k, new, h)
        hs.append(h)
        Ehs.append(Eh)
        r[:, t] = (cc * h).sum(2)
        Er[:, t] = (cc.abs() * Eh).sum(2) + U * (N + 2) * (cc * h).abs().sum(2)
    pre = r + skip * x
    y = pre * gate
    Epre = Er + 2 * U * (r.abs() + (skip * x).abs())
    E = gate.abs() * Epre + pre.abs() * Eg + U * y.abs()
    return (y, E), (h, Eh), (hs, Ehs, pre, Epre)


def scan_bwd(dy, x, dt, A, Bm, Cm, h0, Dskip, z, dt_bias, softplus, dh_final, lengths):
    """dict name -> (gradient, E)."""
    B, T, D = x.shape
    N, G = A.shape[1], Bm.shape[2]
    _, _, (hs, Ehs, pre, Epre) = scan_fwd(x, dt, A, Bm, Cm, h0, Dskip, z, dt_bias, softplus, lengths)
    x, v, s, ds, Es, gate, dgate, sg, Eg, keep = _scan_inputs(x, dt, dt_bias, z, softplus, lengths)
    skip = torch.zeros(D, dtype=torch.float64) if Dskip is None else Dskip
    dy = torch.where(keep, dy, 0.0)
    gy = dy * gate
    Egy = dy.abs() * Eg + U * gy.abs()
    zz = torch.zeros_like(x) if z is None else torch.where(keep, z, 0.0)
    dz = dy * dgate * pre
    Edz = dy.abs() * (dgate.abs() * Epre + pre.abs() * sg * (1 + zz.abs()) * (_silu_loss(zz) + 6 * U))
    g = torch.zeros((B, D, N), dtype=torch.float64) if dh_final is None else dh_final
    Egr = torch.zeros_like(g)
    dx, Edx, ddt, Eddt = (torch.zeros_like(x) for _ in range(4))
    dA, EdA, mdA = (torch.zeros_like(A) for _ in range(3))
    dB, EdB, dC, EdC = (torch.zeros_like(Bm) for _ in range(4))
    # sums over the channels of a group: a few per lane, lanes, wavefronts, then the workgroups
    terms = U * (D // G / 16 + 32)

    def channels(m):
        return m.reshape(B, G, D // G, N).sum(2)

    for t in range(T - 1, -1, -1):
        k = keep[:, t, :, None]
        bb = torch.where(k, _rows(Bm[:, t], D), 0.0)
        cc = torch.where(k, _rows(Cm[:, t], D), 0.0)
        a, ra = _decay(s[:, t], Es[:, t], A, T)
        h, Eh, hp, Ehp = hs[t + 1], Ehs[t + 1], hs[t], Ehs[t]
        gt, Egt = gy[:, t, :, None], Egy[:, t, :, None]
        q = torch.where(k, cc * gt + g, 0.0)
        Eq = torch.where(k, cc.abs() * Egt + Egr + U * ((cc * gt).abs() + q.abs()), 0.0)
        dC[:, t] = channels(gt * h)
        EdC[:, t] = channels(gt.abs() * Eh + h.abs() * Egt + terms * (gt * h).abs())
        u = (s[:, t] * x[:, t])[:, :, None]
        Eu = (x[:, t].abs() * Es[:, t])[:, :, None] + U * u.abs()
        dB[:, t] = channels(u * q)
        EdB[:, t] = channels(u.abs() * Eq + q.abs() * Eu + terms * (u * q).abs())
        p1 = (bb * q).sum(2)
        Ep1 = (bb.abs() * Eq + U * (N + 2) * (bb * q).abs()).sum(2)
        Egr = torch.where(k, a * Eq + a * ra * q.abs() + U * (a * q).abs(), Egr)
        g = torch.where(k, a * q, g)
        e = torch.where(k, g * hp, 0.0)
        Ee = torch.where(k, g.abs() * Ehp + hp.abs() * Egr + U * e.abs(), 0.0)
        p2 = (A * e).sum(2)
        Ep2 = (A.abs() * Ee + U * (N + 2) * (A * e).abs()).sum(2)
        st, xt = s[:, t], x[:, t]
        dA += (st[:, :, None] * e).sum(0)
        mdA += (st[:, :, None] * e).abs().sum(0)
        EdA += (st[:, :, None].abs() * Ee + e.abs() * Es[:, t, :, None]).sum(0)
        dx[:, t] = st * p1 + skip * gy[:, t]
        Edx[:, t] = st.abs() * Ep1 + p1.abs() * Es[:, t] + skip.abs() * Egy[:, t] + \
            2 * U * ((st * p1).abs() + (skip * gy[:, t]).abs())
        raw = xt * p1 + p2
        ddt[:, t] = raw * ds[:, t]
        Eddt[:, t] = ds[:, t] * (xt.abs() * Ep1 + Ep2 + 2 * U * ((xt * p1).abs() + p2.abs())
                                 + raw.abs() * U * (2 * v[:, t].abs() + 8))
    many = U * (B * T + 32)
    out = {"dx": (dx, Edx), "ddt": (ddt, Eddt), "dA": (dA, EdA + many * mdA), "dB": (dB, EdB), "dC": (dC, EdC),
           "dz": (dz, Edz), "dh0": (g, Egr),
           "dD": ((gy * x).sum((0, 1)), (x.abs() * Egy + many * (gy * x).abs()).sum((0, 1))),
           "ddt_bias": (ddt.sum((0, 1)), (Eddt + many * ddt.abs()).sum((0, 1)))}
    return out


# ------------------------------------------------------------- layer norm

# Terms of a row sum that meet one another in turn: 16 a thread, then lanes
# (6 halvings) and wavefronts (16); 64 covers them and the scaling by 1 / D.
ROW = 64


def _norm_parts(x, eps):
    D = x.shape[-1]
    m = x.mean(-1, keepdim=True)
    c = x - m
    Ec = U * (ROW * x.abs().mean(-1, keepdim=True) + c.abs())
    var = (c * c).mean(-1, keepdim=True)
    Evar = (2 * c.abs() * Ec).mean(-1, keepdim=True) + U * ROW * var
    r = 1 / torch.sqrt(var + eps)
    rr = 0.5 * (Evar + U * (var + eps)) * r * r + 4 * U      # relative
    n = c * r
    return c, Ec, r, rr, n, Ec * r + n.abs() * (rr + U)


def norm_fwd(x, w, b, eps):
    _, _, _, _, n, En = _norm_parts(x, eps)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w
    b = torch.zeros(x.shape[-1], dtype=torch.float64) if b is None else b
    y = n * w + b
    return y, w.abs() * En + U * ((n * w).abs() + y.abs())


def norm_bwd(dy, x, w, eps):
    """(dx, E), (dw, E), (db, E)."""
    rows, D = x.shape
    c, Ec, r, rr, n, En = _norm_parts(x, eps)
    w = torch.ones(D, dtype=torch.float64) if w is None else w
    g = dy * w
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    c1, c2 = mean(g), mean(g * n)
    E1 = U * ROW * mean(g.abs())
    E2 = mean(g.abs() * En) + U * ROW * mean((g * n).abs()) + c2.abs() * (rr + 3 * U)
    dx = r * (g - c1 - n * c2)
    Edx = r * (U * g.abs() + E1 + n.abs() * E2 + c2.abs() * En + 4 * U * (g.abs() + c1.abs() + (n * c2).abs())) + \
        dx.abs() * (rr + U)
    many = U * (rows + 32)
    dw, db = (dy * n).sum(0), dy.sum(0)
    return (dx, Edx), (dw, (dy.abs() * En + many * (dy * n).abs()).sum(0)), (db, many * dy.abs().sum(0))
