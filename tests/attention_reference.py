"""Plain float64 forms of the attention layer's operators, with the errors that
float32 arithmetic, float16 parts and one final rounding allow.  They share no
code with the library.

Half a step of rounding, relative: float32 2^-24, bfloat16 2^-8, float16 2^-11,
e4m3 2^-4.
"""

import math

import torch

QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


# ------------------------------------------------------------------------ plan

def plan(cached, added, table, free, free_count, page, tokens):
    """Lists in, a dict of lists out; `table` (list of lists) is changed in place."""
    per = len(table[0]) if table else 0
    free_count = min(max(free_count, 0), len(free))
    left, wanted, row = free_count, 0, 0
    out = {"q_start": [], "context": [], "positions": [-1] * tokens, "slots": [-1] * tokens}
    for b, (c, a) in enumerate(zip(cached, added)):
        out["q_start"].append(min(row, tokens))
        have, want = -(-c // page), -(-(c + a) // page)
        ok = c >= 0 and a >= 0 and want <= per
        wanted += want - have if ok else 0
        end = row + max(a, 0)
        if ok and wanted <= free_count and end <= tokens:
            first = free_count - (wanted - (want - have))
            for j in range(have, want):
                table[b][j] = free[first - 1 - (j - have)]
            left -= want - have
            for i in range(a):
                p = c + i
                out["positions"][row + i] = p
                id_ = table[b][p // page]
                out["slots"][row + i] = -1 if id_ < 0 else id_ * page + p % page
            out["context"].append(c + a)
        else:
            out["context"].append(0)
        row = end
    out["q_start"].append(min(row, tokens))
    out["free_count"] = [left]
    return out


# ------------------------------------------------------------- query, key norm

def _turn(x, cos, sin, neighbours):
    R = 2 * cos.shape[-1]
    y = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if neighbours else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _angles(rotary, positions, shape):
    if rotary is None:
        return torch.ones(shape[:-2] + (1, 0)).double(), torch.zeros(shape[:-2] + (1, 0)).double()
    half = rotary.shape[1] // 2
    p = positions.long().clamp(0, max(rotary.shape[0] - 1, 0))
    rows = rotary.double()[p].unsqueeze(-2)
    return rows[..., :half], rows[..., half:]


def _kinds(rotary, positions, shape):
    """Rows of no token, rows beyond the table."""
    if rotary is None:
        none = torch.zeros(shape[:-2] + (1, 1), dtype=torch.bool)
        return none, none
    p = positions[..., None, None]
    return p < 0, p >= rotary.shape[0]


def qk_fwd(x, w, eps, positions, rotary, neighbours):
    """One of the two, on the CPU: y in float64 and how far a float32 result, rounded to x's type, may be."""
    v = x.double()
    D = v.shape[-1]
    w = torch.ones(D).double() if w is None else w.double()
    none, beyond = _kinds(rotary, positions, x.shape)
    v = torch.where(none, 1.0, v)
    n = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    cos, sin = _angles(rotary, positions, x.shape)
    y = _turn(n * w, cos, sin, neighbours)
    # the mean's D additions and the root, two factors, the turn's two products and sum
    size = _turn((n * w).abs(), cos.abs(), -sin.abs(), neighbours).abs() + (n * w).abs()
    tol = HALF[x.dtype] * y.abs() + (D / 2 + 8) * 2.0 ** -24 * size + 1e-37
    y = torch.where(beyond, math.nan, torch.where(none, 0.0, y))
    return y, tol


def qk_bwd(dy, x, w, eps, positions, rotary, neighbours):
    """(dx, its tolerance, dw, its tolerance)."""
    v, dy = x.double(), dy.double()
    D = v.shape[-1]
    w = torch.ones(D).double() if w is None else w.double()
    none, beyond = _kinds(rotary, positions, x.shape)
    dy, v = torch.where(none, 0.0, dy), torch.where(none, 1.0, v)
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    n = v * r
    cos, sin = _angles(rotary, positions, x.shape)
    g = _turn(dy, cos, -sin, neighbours)
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    ga = _turn(dy.abs(), cos.abs(), -sin.abs(), neighbours).abs() + dy.abs()
    size = r * (ga * w.abs() + n.abs() * (ga * w.abs() * n.abs()).mean(-1, keepdim=True))
    tol = HALF[x.dtype] * dx.abs() + (D + 12) * 2.0 ** -24 * size + 1e-37
    dx = torch.where(beyond, math.nan, torch.where(none, 0.0, dx))
    lead = tuple(range(dx.dim() - 1))
    dw = torch.where(beyond, math.nan, torch.where(none, 0.0, g * n))
    terms = dw.numel() // D
    wtol = (D / 2 + 12 + math.sqrt(terms) + min(terms, 64)) * 2.0 ** -24 * (ga * n.abs()).sum(lead) + 1e-37
    return dx, tol, dw.sum(lead), wtol


# ----------------------------------------------------------------------- cache

def code(v, kind):
    """float32 values to codes: the nearest, 0 for what is not finite."""
    v = torch.where(torch.isfinite(v), v, torch.zeros_like(v)).clamp(-QMAX[kind], QMAX[kind])
    return v.round().to(torch.int8) if kind is torch.int8 else v.to(kind)


def append(x, slots, codes, scales, innermost):
    """One of the two, on the CPU, in place, token by token in float32 as the formula has it."""
    pages, Hk, page = codes.shape[0], codes.shape[1], codes.shape[3 if innermost else 2]
    unit = torch.tensor(1.0) / QMAX[codes.dtype]
    by_page = {}
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            by_page.setdefault(s // page, {})[s % page] = t
    for p, places in by_page.items():
        first = min(places)
        rows = codes[p].transpose(1, 2) if innermost else codes[p]          # [Hk, page, D]
        rows = rows.contiguous().clone()
        ts = list(places.values())
        most = x[ts].float().abs().amax((0, 2)) * unit
        old = scales[p].clone() if first else torch.zeros(Hk)
        new = torch.maximum(old, most)
        grown = old / new
        if first:
            again = code(rows[:, :first].float() * grown[:, None, None], codes.dtype)
            keep = ~(torch.isfinite(grown) & (grown != 1))
            for h in range(Hk):
                if not keep[h]:
                    rows[h, :first] = again[h]
        for o, t in places.items():
            rows[:, o] = code(x[t].float() / new[:, None], codes.dtype)
        codes[p] = rows.transpose(1, 2) if innermost else rows
        scales[p] = new


def fill(kv, kind, innermost):
    """Pages [pages, Hk, page, D] of float32 values as codes and scales."""
    scale = kv.abs().amax((2, 3)) / QMAX[kind]
    c = code(kv / scale[:, :, None, None], kind)
    return (c.transpose(2, 3).contiguous() if innermost else c.contiguous()), scale


def attention(q, k_codes, v_codes, k_scale, v_scale, table, context, q_start, scale):
    """(out, tolerance, lse, tolerance) on the CPU; rows of no sequence are NaN in out's tolerance."""
    N, Hq, D = q.shape
    pages, Hk, page, _ = k_codes.shape
    G, half = Hq // Hk, HALF[q.dtype]
    out = torch.full((N, Hq, D), math.nan).double()
    lse = torch.full((N, Hq), math.nan).double()
    tol, ltol = torch.full_like(out, math.nan), torch.full_like(lse, math.nan)
    per = table.shape[1]
    for b in range(table.shape[0]):
        r0, r1 = int(q_start[b]), int(q_start[b + 1])
        ctx = min(max(int(context[b]), 0), per * page)
        n = r1 - r0
        if n <= 0:
            continue
        ids = table[b, :-(-ctx // page)].long()
        there = ((ids >= 0) & (ids < pages)).repeat_interleave(page)[:ctx]
        ids = ids.clamp(0, max(pages - 1, 0))
        k = (k_codes[ids].double() * k_scale.double()[ids][..., None, None]).transpose(0, 1).reshape(Hk, -1, D)[:, :ctx]
        v = (v_codes[ids].double() * v_scale.double()[ids][..., None, None]).permute(1, 0, 3, 2).reshape(Hk, -1, D)[:, :ctx]
        v_raw = v_codes[ids].double().permute(1, 0, 3, 2).reshape(Hk, -1, D)[:, :ctx]
        pos = ctx - n + torch.arange(n)
        seen = (torch.arange(ctx)[None] <= pos[:, None]) & there[None]      # [n, ctx]
        for hq in range(Hq):
            h = hq // G
            x = q[r0:r1, hq].double()
            z = scale * (x @ k[h].t())
            size = abs(scale) * (x.abs() @ torch.nan_to_num(k[h]).abs().t())
            z = torch.where(seen, z, -math.inf)
            L = torch.where(seen, size, 0.0).amax(-1, keepdim=True) if ctx else torch.zeros(n, 1).double()
            m = z.amax(-1, keepdim=True) if ctx else torch.full((n, 1), -math.inf).double()
            p = torch.where(seen, torch.exp(z - torch.where(torch.isfinite(m), m, 0.0)), 0.0)
            l = p.sum(-1, keepdim=True)
            w = torch.where(l != 0, p / l, 0.0)
            vv = torch.where(seen.any(0)[:, None], v[h], 0.0) if ctx else v[h]
            # a place that a row does not see adds nothing to it, whatever it holds
            bad = torch.isnan(vv).any(-1)
            y = w @ torch.nan_to_num(vv)
            y = torch.where((seen & bad[None]).any(-1, keepdim=True), math.nan, y)
            A = w @ torch.nan_to_num(vv).abs()
            # float16 loses up to 2^-25 of a weight, which stands there times 2^14 / (2 largest value scale seen)
            codes = torch.nan_to_num(torch.where(seen.any(0)[:, None], v_raw[h], 0.0)).abs()
            lost = 2.0 ** -38 * v_scale[ids, h].nan_to_num(0, 0, 0).max() * (seen.double() @ codes) if ctx else 0.0
            parts = 2.0 ** -11 if q.dtype is torch.bfloat16 else 2.0 ** -21
            # scores: float32 sums of D products (float16 parts of float32 queries: 2^-22 each), the exponent's
            # rounding at their size; weights: their parts, exp2 and log2, the sums over the places
            dz = (D + 24) * 2.0 ** -24 * L + (2.0 ** -21 * L if q.dtype is torch.float32 else 0.0) + 2.0 ** -20
            out[r0:r1, hq] = y
            tol[r0:r1, hq] = half * y.abs() + (parts + 2 * dz + (ctx / 8 + 64) * 2.0 ** -24) * A + lost + 1e-30
            lse[r0:r1, hq] = (torch.where(torch.isfinite(m), m, 0.0) + torch.log(l))[:, 0]
            ltol[r0:r1, hq] = (dz + (ctx / 8 + 64) * 2.0 ** -24)[:, 0] + 2.0 ** -22 * lse[r0:r1, hq].nan_to_num(0, 0, 0).abs()
    return out, tol, lse, ltol
