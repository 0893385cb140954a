"""The workloads by which the attention layer's operators are measured: what
serves and trains a softmax attention layer between the recurrent ones.

* plan:    block tables, row starts, positions and cache slots of a step from
           the requests' lengths and a list of free pages
* qk:      y = R(position) (x / sqrt(mean x^2 + eps) * w) for each query and key
           head, R a rotation of pairs of channels; forward and backward
* append:  keys and values into a paged cache of 8-bit codes, one scale for each
           page and head, which grows (and the codes with it) as tokens come
* attend:  softmax(scale q.K) V over that cache, causal, for one query a
           sequence, a few drafts or a whole prompt

`own` selects the library's kernels; otherwise `run` computes the same with
elementary torch operations in float32.  `exact` computes them in float64,
written apart from the float32 form.
"""

import math

import torch

own = False

EPS = 1e-6
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a serving step: one token for each of 256 requests, lengths as they come
        dict(name="plan_decode", op="plan", B=256, page=64, longest=8192, new=1),
        # many short requests admitted at once with their prompts, a few hundred tokens each
        dict(name="plan_admit", op="plan", B=2000, page=16, longest=300, new=250),
        # the serving step's queries and keys: 32 and 8 heads of 128 channels
        dict(name="qk_fwd_decode", op="qk_fwd", T=256, Hq=32, Hk=8, D=128, R=128, pairs="halves", dtype="bf16"),
        # the same layer over a prompt of 16384 tokens
        dict(name="qk_fwd_prompt", op="qk_fwd", T=16384, Hq=32, Hk=8, D=128, R=128, pairs="halves", dtype="bf16"),
        # its backward in a training step
        dict(name="qk_bwd_train", op="qk_bwd", T=16384, Hq=32, Hk=8, D=128, R=128, pairs="halves", dtype="bf16"),
        # float32 fine-tuning, odd token count, a quarter of the channels rotated, neighbours as pairs
        dict(name="qk_bwd_partial_f32", op="qk_bwd", T=1037, Hq=6, Hk=2, D=96, R=24, pairs="neighbours", dtype="f32"),
        # the serving step's token of 256 sequences, each in a page of its own that goes on
        dict(name="append_decode", op="append", B=256, new=1, ragged=False, Hk=8, D=128, page=64, code="e4m3",
             dtype="bf16"),
        # prompts of up to 4096 tokens of 6 sequences, of odd lengths
        dict(name="append_prompt", op="append", B=6, new=4096, ragged=True, Hk=8, D=128, page=64, code="e4m3",
             dtype="bf16"),
        # one chat turn's next token: latency decides
        dict(name="attend_decode_single", op="attend", B=1, longest=777, new=1, Hq=32, Hk=8, D=128, page=64,
             code="e4m3", dtype="bf16", ragged=False),
        # one token for each of 256 sequences of 4096 to 8192 tokens: the serving batch
        dict(name="attend_decode_batch", op="attend", B=256, longest=8192, new=1, Hq=32, Hk=8, D=128, page=64,
             code="e4m3", dtype="bf16", ragged=True),
        # 16 drafts verified for each of 24 sequences, small pages of integers
        dict(name="attend_verify", op="attend", B=24, longest=16384, new=16, Hq=32, Hk=8, D=128, page=16, code="int8",
             dtype="bf16", ragged=True),
        # prompts' next chunks of 2048 to 4096 tokens behind what the cache holds
        dict(name="attend_prompt", op="attend", B=3, longest=8192, new=4096, Hq=32, Hk=8, D=128, page=64, code="e4m3",
             dtype="bf16", ragged=True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["plan", "qk_fwd", "qk_bwd", "append", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _logint(rng, 1, 4000)
        return dict(op=op, B=B, page=page, longest=_logint(rng, 1, 1 << 14), new=_logint(rng, 1, max(1, 500000 // B)))
    if op in ("qk_fwd", "qk_bwd"):
        D = rng.choice([64, 128, 128, 256, 2 * rng.randint(8, 128)])
        R = rng.choice([D, D, 2 * rng.randint(1, D // 2)])
        Hk = _logint(rng, 1, 16)
        Hq = Hk * _logint(rng, 1, 8)
        T = _logint(rng, 1, max(1, min(20000, (1 << 26) // (D * (Hq + Hk)))))
        return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, R=R, pairs=rng.choice(["halves", "halves", "neighbours"]),
                    dtype=dtype)
    D, code, Hk = rng.choice([64, 128, 128, 256]), rng.choice(["e4m3", "int8"]), _logint(rng, 1, 16)
    if op == "append":
        B = _logint(rng, 1, 256)
        new = _logint(rng, 1, max(1, min(8192, (1 << 24) // (B * Hk * D))))
        return dict(op=op, B=B, new=new, ragged=rng.random() < 0.5, Hk=Hk, D=D, page=page, code=code, dtype=dtype)
    Hq = Hk * rng.choice([1, 2, 4, 4, 8, 6])
    new = rng.choice([1, 1, _logint(rng, 2, 32), _logint(rng, 33, 3000)])
    B = _logint(rng, 1, max(1, min(256, 4096 // new)))
    # elements of the cache, and pairs of the plain form's products
    cap = min((1 << 30) // (B * Hk * D), (1 << 29) // (B * new * Hq))
    longest = max(new, _logint(rng, 1, max(1, min(32768, cap))))
    return dict(op=op, B=B, longest=longest, new=new, Hq=Hq, Hk=Hk, D=D, page=page, code=code, dtype=dtype,
                ragged=rng.random() < 0.7)


def _lengths(case):
    """Tokens of each request with its new ones, and the new ones: from the longest down to just above a half."""
    B, top, new = case["B"], case["longest"], case["new"]
    if not case["ragged"]:
        return [top] * B, [new] * B
    total = [top - (b * top) // (2 * B) for b in range(B)]
    return total, [min(t, new - (b * (new // 2)) // B) for b, t in enumerate(total)]


def _plan_tokens(case):
    return sum(1 + b * case["new"] // case["B"] for b in range(case["B"]))


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype="f32", scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(_DT[dtype])


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _rotary(longest, R):
    """[longest, R] float32: R/2 cosines, then R/2 sines, of position * 10000^(-2i/R), angles in float64."""
    i = torch.arange(R // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(longest, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / R)
    return torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()


def _codes(g, pages, Hk, rows, cols, code):
    """Random pages [pages, Hk, rows, cols] as an append leaves them: each page and head scaled by its own largest
    value.  Heads and pages differ in size by a few times, as layers' keys and values do."""
    qmax = _QMAX[_CODE[code]]
    out = torch.empty((pages, Hk, rows, cols), dtype=_CODE[code], device="cuda")
    scale = torch.empty((pages, Hk), device="cuda")
    for p0 in range(0, pages, 4096):
        p1 = min(pages, p0 + 4096)
        x = torch.randn((p1 - p0, Hk, rows, cols), generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn((p1 - p0, Hk, 1, 1), generator=g, device="cuda"))
        s = x.abs().amax((2, 3)) / qmax
        x = (x / s[:, :, None, None]).clamp(-qmax, qmax)
        out[p0:p1] = (x.round() if code == "int8" else x).to(_CODE[code])
        scale[p0:p1] = s
    return out, scale


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op}
    if op == "plan":
        B, page = case["B"], case["page"]
        cached = torch.randint(0, case["longest"] + 1, (B,), generator=g, device="cuda")
        # from one new token to all of a prompt, in any order; the step's buffers hold a multiple of 64 tokens
        lengths = 1 + torch.arange(B, device="cuda") * case["new"] // B
        added = lengths[torch.randperm(B, generator=g, device="cuda")]
        per = -(-(case["longest"] + case["new"]) // page)
        order = torch.randperm(2 * B * per, generator=g, device="cuda")
        have = (cached + page - 1) // page
        table = order[:B * per].reshape(B, per)
        s["table"] = torch.where(torch.arange(per, device="cuda") < have[:, None], table, -1).int().contiguous()
        s["free"] = order[B * per:].int().contiguous()
        s["free_count"] = _int([B * per])
        s["cached"], s["added"] = cached.int(), added.int()
        s["page"], s["tokens"] = page, -(-_plan_tokens(case) // 64) * 64
    elif op in ("qk_fwd", "qk_bwd"):
        T, Hq, Hk, D, R, dt = (case[k] for k in ("T", "Hq", "Hk", "D", "R", "dtype"))
        rows = _randn(g, (T, (Hq + 2 * Hk) * D), dt)          # one projection's output: queries, keys and values
        s["q"] = rows[:, :Hq * D].view(T, Hq, D)
        s["k"] = rows[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["wq"] = 1.0 + _randn(g, (D,), scale=0.1)
        s["wk"] = 1.0 + _randn(g, (D,), scale=0.1)
        longest = max(2 * T, 4096)
        s["rotary"] = _rotary(longest, R)
        first = torch.randint(0, longest - T + 1, (1,), generator=g, device="cuda")
        s["positions"] = (first + torch.arange(T, device="cuda")).int()
        s["neighbours"] = case["pairs"] == "neighbours"
        if op == "qk_bwd":
            s["dq"], s["dk"] = _randn(g, (T, Hq, D), dt), _randn(g, (T, Hk, D), dt)
    elif op == "append":
        B, Hk, D, page, dt = (case[k] for k in ("B", "Hk", "D", "page", "dtype"))
        total, new = _lengths(dict(case, longest=case["new"]))
        # each sequence goes on somewhere inside its page
        at = torch.randint(0, page, (B,), generator=g, device="cuda")
        cap = -(-(case["new"] + page) // page)
        table = torch.randperm(B * cap, generator=g, device="cuda").reshape(B, cap)
        n, start = torch.tensor(new, device="cuda"), torch.tensor(_starts(new)[:-1], device="cuda")
        b = torch.repeat_interleave(torch.arange(B, device="cuda"), n)
        pos = at[b] + torch.arange(b.numel(), device="cuda") - start[b]
        s["slots"] = (table[b, pos // page] * page + pos % page).int()
        N = s["slots"].numel()
        rows = _randn(g, (N, 2 * Hk * D), dt)                 # one projection's output: keys and values
        s["k"], s["v"] = rows[:, :Hk * D].view(N, Hk, D), rows[:, Hk * D:].view(N, Hk, D)
        s["kc"], s["ks"] = _codes(g, B * cap, Hk, page, D, case["code"])
        s["vc"], s["vs"] = _codes(g, B * cap, Hk, D, page, case["code"])
    else:
        B, Hq, Hk, D, page, dt = (case[k] for k in ("B", "Hq", "Hk", "D", "page", "dtype"))
        total, new = _lengths(case)
        per = -(-case["longest"] // page)
        pages = sum(-(-t // page) for t in total)
        order = torch.randperm(pages, generator=g, device="cuda")
        first = torch.tensor(_starts([-(-t // page) for t in total])[:-1], device="cuda")
        have = torch.tensor([-(-t // page) for t in total], device="cuda")
        i = torch.arange(per, device="cuda")
        table = order[(first[:, None] + i).clamp(max=pages - 1)]
        s["table"] = torch.where(i < have[:, None], table, -1).int().contiguous()
        s["context"], s["starts"] = _int(total), _int(_starts(new))
        s["q"] = _randn(g, (sum(new), Hq, D), dt, 2.0)
        s["kc"], s["ks"] = _codes(g, pages, Hk, page, D, case["code"])
        s["vc"], s["vs"] = _codes(g, pages, Hk, D, page, case["code"])
        s["scale"], s["most"] = D ** -0.5, max(new)
    return s


# -------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import gated_delta_rule_101_amd as kda
    op = s["op"]
    if op == "plan":
        p = kda.kda_cache_plan(s["cached"], s["added"], s["table"], s["free"], s["free_count"], page_size=s["page"],
                               tokens=s["tokens"])
        return [s["table"], p["q_start"], p["context"], p["positions"], p["slots"], p["free_count"]]
    if op == "qk_fwd":
        return list(kda.kda_qk_norm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], EPS, positions=s["positions"],
                                             rotary=s["rotary"], neighbours=s["neighbours"]))
    if op == "qk_bwd":
        r = kda.kda_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], EPS,
                                     positions=s["positions"], rotary=s["rotary"], neighbours=s["neighbours"])
        return [r[k] for k in ("dq", "dk", "dq_weight", "dk_weight")]
    if op == "append":
        kda.kda_cache_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
        return [s["kc"], s["vc"], s["ks"], s["vs"]]
    one = s["most"] == 1
    o, lse = kda.kda_cache_attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["context"],
                                     q_start=None if one else s["starts"], max_queries=s["most"], scale=s["scale"],
                                     want_lse=True)
    return [o, lse]


# ----------------------------------------------------- plain form, float32

def _plain_plan(s):
    page, N = s["page"], s["tokens"]
    c, a, table = s["cached"].long(), s["added"].long(), s["table"]
    B, per = table.shape
    have, want = (c + page - 1) // page, (c + a + page - 1) // page
    ok = (c >= 0) & (a >= 0) & (want <= per)
    need = torch.where(ok, want - have, 0)
    taken, rows = torch.cumsum(need, 0), torch.cumsum(a.clamp(min=0), 0)
    served = ok & (taken <= s["free_count"]) & (rows <= N)
    context = torch.where(served, c + a, 0)
    t = torch.arange(N, device=c.device)
    b = torch.searchsorted(rows, t, right=True).clamp(max=B - 1)
    live = served[b] & (t < rows[b])
    pos = torch.where(live, c[b] + t - (rows[b] - a[b]), -1)
    i = pos.clamp(min=0) // page
    fresh = (i >= have[b]) & live
    at = s["free_count"] - 1 - (taken[b] - need[b] + i - have[b])
    taken_page = s["free"][at.clamp(min=0, max=s["free"].numel() - 1)].long()
    old = table[b, i].long()
    own_page = torch.where(fresh, taken_page, old)
    slots = torch.where(live, own_page * page + pos % page, -1)
    # a page's entry is the same for each of its tokens; tokens of no request write to a row of their own
    entries = torch.cat([table, table[:1]])
    entries[torch.where(live, b, B), i] = own_page.int()
    table.copy_(entries[:B])
    starts = torch.cat([torch.zeros_like(rows[:1]), rows]).clamp(max=N)
    left = s["free_count"] - torch.where(served, need, 0).sum()
    return [table, starts.int(), context.int(), pos.int(), slots.int(), left.int()]


def _turn(x, cos, sin, neighbours, back=False):
    """The first R channels' pairs turned by their angles (back: by the opposite ones)."""
    R = 2 * cos.shape[-1]
    cos, sin = cos[:, None], -sin[:, None] if back else sin[:, None]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if neighbours else (x[..., :R // 2], x[..., R // 2:R])
    p, q = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([p, q], -1).flatten(-2) if neighbours else torch.cat([p, q], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _angles(s):
    rows = s["rotary"][s["positions"].long()]
    half = rows.shape[1] // 2
    return rows[:, :half], rows[:, half:]


def _plain_qk_fwd(s):
    cos, sin = _angles(s)

    def one(x, w):
        v = x.float()
        n = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
        return _turn(n * w, cos, sin, s["neighbours"]).to(x.dtype)

    return [one(s["q"], s["wq"]), one(s["k"], s["wk"])]


def _plain_qk_bwd(s):
    cos, sin = _angles(s)

    def one(x, w, dy):
        v = x.float()
        r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
        n, g = v * r, _turn(dy.float(), cos, sin, s["neighbours"], back=True)
        dn = g * w
        dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        return dx.to(x.dtype), (g * n).sum((0, 1))

    dq, dwq = one(s["q"], s["wq"], s["dq"])
    dk, dwk = one(s["k"], s["wk"], s["dk"])
    return [dq, dk, dwq, dwk]


def _plain_append(s):
    pages, Hk, page, D = s["kc"].shape
    slots = s["slots"].long()
    p, off = slots // page, slots % page
    first = torch.full((pages,), page, device=p.device).scatter_reduce(0, p, off, "amin")
    touched = first < page
    goes_on = torch.arange(page, device=p.device) < first[:, None]          # tokens that were there before
    goes_on = goes_on & touched[:, None]

    def one(x, codes, scales, innermost):
        x, qmax = x.float(), _QMAX[codes.dtype]

        def code(v):
            v = torch.where(torch.isfinite(v), v, torch.zeros_like(v)).clamp(-qmax, qmax)
            return (v.round() if codes.dtype == torch.int8 else v).to(codes.dtype).view(torch.uint8)

        most = torch.zeros((pages, Hk), device=x.device).scatter_reduce(
            0, p[:, None].expand(-1, Hk), x.abs().amax(-1), "amax")
        unit = torch.ones((), device=x.device) / qmax
        old = torch.where(goes_on[:, :1], scales, torch.zeros_like(scales))
        new = torch.maximum(old, most * unit)
        # codes that were there, at the scale that the page has now
        grown = old / new
        at = goes_on[:, None, None, :] if innermost else goes_on[:, None, :, None]
        again = at & (torch.isfinite(grown) & (grown != 1))[:, :, None, None]
        raw = codes.view(torch.uint8)
        raw.copy_(torch.where(again, code(codes.float() * grown[:, :, None, None]), raw))
        rows = code(x / new[p][:, :, None])
        if innermost:
            raw[p, :, :, off] = rows
        else:
            raw[p, :, off] = rows
        scales.copy_(torch.where(touched[:, None], new, scales))

    one(s["k"], s["kc"], s["ks"], False)
    one(s["v"], s["vc"], s["vs"], True)
    return [s["kc"], s["vc"], s["ks"], s["vs"]]


def _plain_attend(s):
    q, table, context, starts = s["q"].float(), s["table"].long().clamp(min=0), s["context"].long(), s["starts"].long()
    N, Hq, D = q.shape
    B, per = table.shape
    _, Hk, page, _ = s["kc"].shape
    G, most, T = Hq // Hk, s["most"], per * page
    kind = s["kc"].dtype
    k = s["kc"].view(torch.uint8)[table].view(kind).float() * s["ks"][table][..., None, None]
    k = k.permute(0, 2, 1, 3, 4).reshape(B * Hk, T, D)
    v = s["vc"].view(torch.uint8)[table].view(kind).float() * s["vs"][table][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(B * Hk, T, D)
    i = torch.arange(most, device=q.device)
    n = starts[1:] - starts[:-1]
    rows = (starts[:-1, None] + i).clamp(max=N - 1)                         # [B, most]
    pos = context[:, None] - n[:, None] + i
    qb = q[rows].reshape(B, most, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B * Hk, most * G, D)
    x = torch.bmm(qb, k.transpose(1, 2)) * s["scale"]
    seen = torch.arange(T, device=q.device) <= pos[..., None]               # [B, most, T]
    x = x.reshape(B, Hk, most, G, T).masked_fill_(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.bmm(x.reshape(B * Hk, most * G, T), v).reshape(B, Hk, most, G, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + torch.log(total))[..., 0]
    # each row's place among the padded ones
    t = torch.arange(N, device=q.device)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    at = t - starts[b]
    return [o[b, :, at].reshape(N, Hq, D).to(s["q"].dtype), lse[b, :, at].reshape(N, Hq)]


_PLAIN = {"plan": _plain_plan, "qk_fwd": _plain_qk_fwd, "qk_bwd": _plain_qk_bwd, "append": _plain_append,
          "attend": _plain_attend}


def _run_plain(s):
    return _PLAIN[s["op"]](s)


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "plan":
        # lengths in, row starts and contexts out; two numbers a token; a page's number read and written
        B, tokens = case["B"], _plan_tokens(case)
        return {"bytes": 16 * B + 8 * tokens + 8 * tokens / case["page"], "flops": 8 * tokens}
    e = _SIZE[case["dtype"]]
    if op in ("qk_fwd", "qk_bwd"):
        T, Hq, Hk, D, R = (case[k] for k in ("T", "Hq", "Hk", "D", "R"))
        n = T * (Hq + Hk) * D
        if op == "qk_fwd":
            return {"bytes": 2 * e * n + T * (4 * R + 4) + 8 * D, "flops": 8 * n}
        return {"bytes": 3 * e * n + T * (4 * R + 4) + 16 * D, "flops": 18 * n}
    if op == "append":
        n = sum(_lengths(dict(case, longest=case["new"]))[1])
        pages = -(-n // case["page"]) if case["new"] > case["page"] else case["B"]
        return {"bytes": 2 * n * case["Hk"] * case["D"] * (e + 1) + 4 * n + 16 * pages * case["Hk"],
                "flops": 6 * n * case["Hk"] * case["D"]}
    total, new = _lengths(case)
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    pairs = sum(n * t - n * (n - 1) // 2 for t, n in zip(total, new))
    rows = sum(new)
    return {"bytes": sum(total) * Hk * 2 * D + 8 * Hk * sum(-(-t // case["page"]) for t in total) +
            rows * Hq * (2 * e * D + 4), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------- float64 reference

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_plan(case, s):
    """From the lists, request by request, on the host."""
    page, N = s["page"], s["tokens"]
    table, free = s["table"].cpu().clone(), s["free"].tolist()
    left, starts, context, pos, slots = int(s["free_count"]), [0], [], [-1] * N, [-1] * N
    wanted, full = left, False
    for b, (c, a) in enumerate(zip(s["cached"].tolist(), s["added"].tolist())):
        have, want = -(-c // page), -(-(c + a) // page)
        row = starts[-1]
        starts.append(row + a)
        wanted -= want - have if want <= table.shape[1] else 0
        served = want <= table.shape[1] and wanted >= 0 and row + a <= N
        context.append(c + a if served else 0)
        if served:
            for j in range(have, want):
                left -= 1
                table[b, j] = free[left]
            entries = table[b].tolist()
            pos[row:row + a] = range(c, c + a)
            slots[row:row + a] = [entries[p // page] * page + p % page for p in range(c, c + a)]
    ints = [torch.tensor(v, dtype=torch.int32) for v in ([min(x, N) for x in starts], context, pos, slots, [left])]
    return [table, *ints]


def _exact_qk(case, s):
    T, D, R = case["T"], case["D"], case["R"]
    table = s["rotary"].double()[s["positions"].long()]
    # each head's rotation as a matrix's action: y[i] = c[i] x[i] + t[i] x[mate(i)]
    i = torch.arange(D, device="cuda")
    if s["neighbours"]:
        mate, pair, sign = i ^ 1, i // 2, 2.0 * (i % 2) - 1.0
    else:
        mate, pair, sign = (i + R // 2) % max(R, 1), i % max(R // 2, 1), torch.where(i < R // 2, -1.0, 1.0).double()
    turned = i < R
    mate, pair = torch.where(turned, mate, i), torch.where(turned, pair, 0)
    c = torch.where(turned, table[:, pair], 1.0)[:, None]
    t = torch.where(turned, table[:, R // 2 + pair] * sign, 0.0)[:, None]
    out = [[], []]
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x, w = x.double(), w.double()
        norm = (x.square().sum(-1, keepdim=True) / D + EPS).sqrt()
        if dy is None:
            y = x / norm * w
            out[0].append(c * y + t * y[..., mate])
            continue
        dy = dy.double()
        g = c * dy + (t * dy)[..., mate]
        out[0].append((g * w - x * ((g * w * x).sum(-1, keepdim=True) / (D * norm.square()))) / norm)
        out[1].append((g * x / norm).sum((0, 1)))
    return out[0] + out[1]


def _exact_append(case, s):
    """Page by page, over the pages that tokens go to."""
    pages, Hk, page, D = s["kc"].shape
    slots = s["slots"].long()
    order = torch.argsort(slots)
    where = (slots[order] // page).tolist()
    runs, i = [], 0
    while i < len(where):
        j = i
        while j < len(where) and where[j] == where[i]:
            j += 1
        runs.append((where[i], i, j))
        i = j
    off = (slots[order] % page).tolist()
    out = []
    for x, codes, scales, innermost in ((s["k"], s["kc"], s["ks"], False), (s["v"], s["vc"], s["vs"], True)):
        x, qmax, whole = x.double()[order], _QMAX[codes.dtype], codes.dtype == torch.int8
        values = codes.float().double()
        values = values.transpose(2, 3).contiguous() if innermost else values
        scale = scales.double()
        for p, i, j in runs:
            first = off[i]
            before = scale[p] if first else torch.zeros_like(scale[p])
            now = torch.maximum(before, (x[i:j].abs().amax((0, 2)) / qmax))
            stored = now.float().double()
            if first:
                old = values[p, :, :first] * (before / stored)[:, None, None]
                same = (before == now)[:, None, None]
                old = torch.where(same, values[p, :, :first], old.round() if whole else old)
                values[p, :, :first] = old if whole else old.float().to(codes.dtype).double()
            new = (x[i:j] / stored[:, None]).clamp(-qmax, qmax)
            new = new.round() if whole else new.float().to(codes.dtype).double()
            values[p, :, first:first + j - i] = new.transpose(0, 1)
            scale[p] = now
        out.append((values.transpose(2, 3).contiguous() if innermost else values, scale))
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


def _exact_attend(case, s):
    total, new = _lengths(case)
    Hq, Hk, D, page = case["Hq"], case["Hk"], case["D"], case["page"]
    G, kind = Hq // Hk, s["kc"].dtype
    o, lse, row = [], [], 0
    for b, (t, n) in enumerate(zip(total, new)):
        ids = s["table"][b, :-(-t // page)].long()
        k = s["kc"].view(torch.uint8)[ids].view(kind).double() * s["ks"].double()[ids][..., None, None]
        v = s["vc"].view(torch.uint8)[ids].view(kind).double() * s["vs"].double()[ids][..., None, None]
        k = k.transpose(0, 1).reshape(Hk, -1, D)[:, :t]
        v = v.permute(1, 0, 3, 2).reshape(Hk, -1, D)[:, :t]
        q = s["q"][row:row + n].double()
        hidden = torch.arange(t, device="cuda") > torch.arange(t - n, t, device="cuda")[:, None]
        ob, lb = torch.empty_like(q), torch.empty((n, Hq), dtype=torch.float64, device="cuda")
        for h in range(Hq):
            z = (q[:, h] @ k[h // G].t()) * s["scale"]
            z = z.masked_fill(hidden, -math.inf)
            lb[:, h] = torch.logsumexp(z, -1)
            ob[:, h] = torch.exp(z - lb[:, h, None]) @ v[h // G]
        o.append(ob)
        lse.append(lb)
        row += n
    return [torch.cat(o), torch.cat(lse)]


_EXACT = {"plan": _exact_plan, "qk_fwd": _exact_qk, "qk_bwd": _exact_qk, "append": _exact_append,
          "attend": _exact_attend}
