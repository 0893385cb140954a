"""The attention layer's operators on the GPU against float64 (tests/attention_reference.py)."""

import math

import pytest
import torch

import attention_reference as ref
from gpu_support import say

pytestmark = pytest.mark.gpu

E4M3, INT8, BF16, F32 = torch.float8_e4m3fn, torch.int8, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_101_amd as m
    m.load_library()
    return m


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def close(got, want, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    over = ((got - want).abs() / tol)[fine]
    if over.numel():
        say(f"[{what}] worst error / tolerance {over.max():.3f}")
        assert over.max() <= 1, f"{what}: {over.max():.3f} of the tolerance"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------ plan

def run_plan(kda, cached, added, table, free, free_count, page, tokens):
    t = torch.tensor(table, dtype=torch.int32, device="cuda").reshape(len(cached), -1)
    p = kda.kda_cache_plan(i32(cached), i32(added), t, i32(free), i32([free_count]), page_size=page, tokens=tokens)
    return t, p


@pytest.mark.parametrize("B,page,longest,new,room,spare", [
    (1, 16, 5, 1, 0, 9), (1, 64, 0, 1, 3, 9), (3, 16, 40, 17, 64, 99), (256, 64, 900, 1, 0, 300),
    (1024, 16, 50, 3, 10, 3000), (1025, 32, 70, 9, 1, 3000), (5000, 128, 300, 4, 100, 9000),
    (70, 16, 64, 40, 0, 60), (300, 16, 100, 20, -500, 900)])
def test_plan(kda, B, page, longest, new, room, spare):
    """room: rows behind the last request (negative: too few); spare: free pages, at times too few."""
    g = gen(B + page)
    cached = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    added = torch.randint(0, new + 1, (B,), generator=g).tolist()
    per = -(-(longest + new) // page)
    ids = torch.randperm(B * per + spare, generator=g).tolist()
    table = [[ids[b * per + j] if j < -(-c // page) else -1 for j in range(per)] for b, c in enumerate(cached)]
    free = ids[B * per:]
    tokens = sum(added) + room
    got_table, p = run_plan(kda, cached, added, table, free, len(free), page, tokens)
    want = ref.plan(cached, added, table, free, len(free), page, tokens)
    for name in want:
        assert p[name].tolist() == want[name], name
    assert got_table.tolist() == table


def test_plan_refuses_requests_that_cannot_be_served(kda):
    # negative lengths, too many pages for the table, pages that run out, a free count beyond the list
    cached, added = [-1, 5, 0, 30, 3, 0], [4, -2, 100, 4, 1, 40]
    table = [[7, 8, 9, -1] for _ in cached]
    for free_count in (9, -3, 1, 3):
        t = [row[:] for row in table]
        got, p = run_plan(kda, cached, added, t, [20, 21, 22, 23], free_count, 16, 160)
        want = ref.plan(cached, added, t, [20, 21, 22, 23], free_count, 16, 160)
        for name in want:
            assert p[name].tolist() == want[name], (free_count, name)
        assert got.tolist() == t


def test_plan_without_requests_or_rows(kda):
    t = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    p = kda.kda_cache_plan(none, none, t, i32([3, 4]), i32([2]), page_size=16, tokens=5)
    assert p["q_start"].tolist() == [0] and p["positions"].tolist() == [-1] * 5 and p["slots"].tolist() == [-1] * 5
    assert p["free_count"].tolist() == [2]
    p = kda.kda_cache_plan(i32([5]), i32([0]), i32([[1]]), none, i32([0]), page_size=16, tokens=0)
    assert p["q_start"].tolist() == [0, 0] and p["context"].tolist() == [5] and p["free_count"].tolist() == [0]


# ------------------------------------------------------------- query, key norm

def rotary_table(rows, R):
    i = torch.arange(R // 2).double()
    angle = torch.arange(rows).double()[:, None] * 10000.0 ** (-2 * i / max(R, 1))
    return torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()


QK = [  # T, Hq, Hk, D, R, neighbours, dtype, fused
    (1, 1, 1, 64, 64, False, BF16, True), (1, 32, 8, 128, 128, False, BF16, True), (7, 5, 3, 128, 128, True, F32, True),
    (300, 4, 2, 96, 32, False, BF16, False), (33, 3, 1, 80, 80, True, BF16, True), (65, 2, 2, 256, 64, False, F32, True),
    (19, 3, 2, 6, 4, False, F32, True), (21, 3, 2, 10, 10, True, BF16, True), (17, 2, 1, 2, 2, False, BF16, False),
    (9, 3, 2, 202, 100, False, BF16, True), (9, 2, 2, 510, 254, True, F32, True), (5, 2, 1, 512, 512, False, BF16, True),
    (5, 2, 1, 512, 512, True, F32, False), (40, 4, 4, 128, 0, False, BF16, True), (2000, 9, 3, 64, 16, True, BF16, True),
    (3, 6, 0, 128, 128, False, BF16, False), (3, 0, 2, 64, 64, False, F32, False), (5000, 2, 1, 128, 128, False, F32, True),
    (1, 1, 1, 62, 30, True, BF16, True), (50, 5, 2, 120, 120, False, BF16, True), (31, 3, 2, 72, 24, True, BF16, True),
    (9, 2, 1, 504, 8, False, BF16, False), (700, 3, 2, 40, 0, False, BF16, True)]


def qk_inputs(T, Hq, Hk, D, R, dtype, fused, seed):
    g = gen(seed)
    if fused:      # parts of one projection's output, off its first columns
        rows = (torch.randn(T, 8 + (Hq + 2 * Hk) * D, generator=g) * 2).to(dtype).cuda()
        q = rows[:, 8:8 + Hq * D].view(T, Hq, D)
        k = rows[:, 8 + Hq * D:8 + (Hq + Hk) * D].view(T, Hk, D)
    else:
        q = (torch.randn(T, Hq, D, generator=g) * 2).to(dtype).cuda()
        k = (torch.randn(T, Hk, D, generator=g) * 2).to(dtype).cuda()
    wq, wk = (1 + 0.2 * torch.randn(2, D, generator=g)).cuda()
    if not R:
        return q, k, wq, wk, None, None
    rows = 3 * T + 5
    pos = torch.randint(0, rows, (T,), generator=g).int()
    if T > 8:
        pos[3], pos[5], pos[6] = -1, rows, 2 ** 31 - 1
    return q, k, wq, wk, pos.cuda(), rotary_table(rows, R).cuda()


def cpu(*ts):
    return [t.cpu() if torch.is_tensor(t) else t for t in ts]


@pytest.mark.parametrize("T,Hq,Hk,D,R,neighbours,dtype,fused", QK)
def test_qk_norm_rope(kda, T, Hq, Hk, D, R, neighbours, dtype, fused):
    q, k, wq, wk, pos, table = qk_inputs(T, Hq, Hk, D, R, dtype, fused, T + D)
    yq, yk = kda.kda_qk_norm_rope_fwd(q, k, wq, wk, 1e-6, positions=pos, rotary=table, neighbours=neighbours)
    for y, x, w, name in ((yq, q, wq, "q"), (yk, k, wk, "k")):
        want, tol = ref.qk_fwd(*cpu(x, w), 1e-6, *cpu(pos, table), neighbours)
        close(y, want, tol, "fwd " + name)
    g = gen(T * D)
    dq, dk = (torch.randn(t.shape, generator=g).to(dtype).cuda() for t in (q, k))
    r = kda.kda_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, 1e-6, positions=pos, rotary=table, neighbours=neighbours)
    for n, x, w, dy in (("q", q, wq, dq), ("k", k, wk, dk)):
        dx, tol, dw, wtol = ref.qk_bwd(*cpu(dy, x, w), 1e-6, *cpu(pos, table), neighbours)
        close(r["d" + n], dx, tol, "d" + n)
        close(r[f"d{n}_weight"], dw, wtol, f"d{n}_weight")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_qk_norm_rope_in_place_and_without_weights(kda, dtype):
    T, Hq, Hk, D = 37, 4, 2, 128
    q, k, _, _, pos, table = qk_inputs(T, Hq, Hk, D, 128, dtype, True, 5)
    rest = q.new_empty(0)
    want = kda.kda_qk_norm_rope_fwd(q, k, positions=pos, rotary=table)
    base = q._base.clone()
    q2, k2 = base[:, 8:8 + Hq * D].view(T, Hq, D), base[:, 8 + Hq * D:8 + (Hq + Hk) * D].view(T, Hk, D)
    got = kda.kda_qk_norm_rope_fwd(q2, k2, positions=pos, rotary=table, q_out=q2, k_out=k2)
    assert got[0] is q2 and got[1] is k2
    for a, b in zip(want, got):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
    v0 = 8 + (Hq + Hk) * D
    assert torch.equal(base[:, :8], q._base[:, :8]) and torch.equal(base[:, v0:], q._base[:, v0:])
    y, tol = ref.qk_fwd(*cpu(q, None), 1e-6, *cpu(pos, table), False)
    close(want[0], y, tol, "no weight")
    # gradients: written into a fused gradient's rows, or over the upstream ones
    g = gen(1)
    dq, dk = (torch.randn(t.shape, generator=g).to(dtype).cuda() for t in (q, k))
    r = kda.kda_qk_norm_rope_bwd(dq, dk, q, k, positions=pos, rotary=table)
    wide = torch.zeros_like(base)
    s = kda.kda_qk_norm_rope_bwd(dq, dk, q, k, positions=pos, rotary=table, dq=wide[:, 8:8 + Hq * D].view(T, Hq, D),
                                 dk=wide[:, 8 + Hq * D:v0].view(T, Hk, D))
    p = kda.kda_qk_norm_rope_bwd(dq, dk, q, k, positions=pos, rotary=table, dq=dq, dk=dk, want_dweights=False)
    assert p["dq"] is dq and "dq_weight" not in p
    for other in (s, p):
        for n in ("dq", "dk"):
            assert torch.equal(torch.nan_to_num(other[n].float()), torch.nan_to_num(r[n].float()))
    assert not wide[:, :8].any() and not wide[:, v0:].any()


def test_qk_norm_rope_batches_and_padding_without_eps(kda):
    """[B, T, H, D] inputs; rows of no token hold NaN and add nothing, also with eps 0 and lanes of no head."""
    B, T, Hq, Hk, D = 2, 13, 3, 2, 128
    g = gen(2)
    q, k = torch.randn(B, T, Hq, D, generator=g).cuda(), torch.randn(B, T, Hk, D, generator=g).cuda()
    dq, dk = torch.randn(B, T, Hq, D, generator=g).cuda(), torch.randn(B, T, Hk, D, generator=g).cuda()
    pos = torch.arange(T).repeat(B, 1).int()
    pos[1, 9:] = -1
    for t in (q, k, dq, dk):
        t[1, 9:] = math.nan
    table = rotary_table(T, D).cuda()
    yq, yk = kda.kda_qk_norm_rope_fwd(q, k, eps=0.0, positions=pos.cuda(), rotary=table)
    r = kda.kda_qk_norm_rope_bwd(dq, dk, q, k, eps=0.0, positions=pos.cuda(), rotary=table)
    for x, y, dy, n in ((q, yq, dq, "q"), (k, yk, dk, "k")):
        want, tol = ref.qk_fwd(*cpu(torch.nan_to_num(x), None), 0.0, pos, table.cpu(), False)
        close(y, want, tol, n)
        dx, tol, dw, wtol = ref.qk_bwd(*cpu(torch.nan_to_num(dy), torch.nan_to_num(x), None), 0.0, pos, table.cpu(), False)
        close(r["d" + n], dx, tol, "d" + n)
        close(r[f"d{n}_weight"], dw, wtol, f"d{n}_weight")


def test_qk_norm_rope_gradients_against_differences(kda):
    """Directional differences of the float32 forward: step h, error of order h^2 and 2^-24 / h."""
    T, Hq, Hk, D = 5, 2, 1, 64
    q, k, wq, wk, pos, table = qk_inputs(T, Hq, Hk, D, 32, F32, False, 11)
    g = gen(12)
    dq, dk = torch.randn(q.shape, generator=g).cuda(), torch.randn(k.shape, generator=g).cuda()
    r = kda.kda_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, positions=pos, rotary=table)

    def loss(q, k, wq, wk):
        a, b = kda.kda_qk_norm_rope_fwd(q, k, wq, wk, positions=pos, rotary=table)
        return (a.double() * dq).sum() + (b.double() * dk).sum()

    args, grads = [q, k, wq, wk], [r["dq"], r["dk"], r["dq_weight"], r["dk_weight"]]
    h = 2.0 ** -8
    for i in range(4):
        u = torch.randn(args[i].shape, generator=g).cuda()
        plus, minus = [*args], [*args]
        plus[i], minus[i] = args[i] + h * u, args[i] - h * u
        slope = (loss(*plus) - loss(*minus)) / (2 * h)
        want = (grads[i].double() * u).sum()
        # third derivatives of the norm are a few times 1 / |x|^3 with |x| around 16 a row; sums of 640 terms
        assert abs(slope - want) <= 640 * (h * h + 2.0 ** -22 / h), (i, float(slope), float(want))


# ---------------------------------------------------------------------- append

def cache(pages, Hk, page, D, kind, seed):
    """A cache of noise, as freed pages leave it: any byte, any scale."""
    g = gen(seed)
    k = torch.randint(-128, 128, (pages, Hk, page, D), generator=g).to(torch.int8)
    v = torch.randint(-128, 128, (pages, Hk, D, page), generator=g).to(torch.int8)
    ks, vs = torch.rand(2, pages, Hk, generator=g) * 0.02
    if kind is INT8:
        k, v = k.clamp(min=-127), v.clamp(min=-127)
    return k.view(kind), v.view(kind), ks.contiguous(), vs.contiguous()


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


def equal(a, b):
    """Float32 tensors alike, NaN with NaN."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def check_append(kda, k, v, slots, c, what):
    dev = [t.cuda() for t in c]
    want = [t.clone() for t in c]
    kda.kda_cache_append(k, v, i32(slots.tolist()), *dev)
    ref.append(k.cpu(), slots, want[0], want[2], False)
    ref.append(v.cpu(), slots, want[1], want[3], True)
    for i, n in ((2, "k_scale"), (3, "v_scale")):
        assert equal(dev[i].cpu(), want[i]), f"{what} {n}"
    for i, n in ((0, "k_codes"), (1, "v_codes")):
        assert torch.equal(bits(dev[i]), bits(want[i])), f"{what} {n}"
    return dev


def sequence_slots(lists, page):
    """Slots of runs (page ids, first place, tokens)."""
    out = []
    for ids, first, n in lists:
        out += [ids[p // page] * page + p % page for p in range(first, first + n)]
    return torch.tensor(out, dtype=torch.int32)


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("Hk,D,page,dtype,runs", [
    (1, 64, 16, BF16, [([0], 0, 1)]),
    (8, 128, 64, BF16, [([3], 5, 1), ([1], 0, 1), ([2], 63, 1)]),
    (2, 128, 64, BF16, [([5, 2, 4], 10, 170), ([1], 0, 64), ([3], 60, 4)]),
    (3, 64, 16, F32, [([5, 2, 4, 7], 3, 61), ([1], 7, 9), ([3], 8, 8), ([0], 0, 8)]),
    (1, 256, 128, F32, [([1, 0], 100, 150)]),
    (2, 256, 32, BF16, [([9, 4], 31, 2), ([1, 2, 3], 0, 96), ([7], 1, 12)]),
    (1, 64, 128, BF16, [([2], 0, 9), ([1], 1, 127), ([0], 100, 28)])])
def test_append(kda, kind, Hk, D, page, dtype, runs):
    slots = sequence_slots(runs, page)
    g = gen(D + page)
    # keys and values of one projection, values of pages' sizes and one of a few sizes
    rows = (torch.randn(len(slots), 3 + 2 * Hk * D, generator=g) * torch.exp(torch.randn(len(slots), 1, generator=g)))
    rows = rows.to(dtype).cuda()
    k, v = rows[:, 3:3 + Hk * D].view(-1, Hk, D), rows[:, 3 + Hk * D:].view(-1, Hk, D)
    c = cache(10, Hk, page, D, kind, page)
    c[2][3] *= 100                                            # a page whose scale stays
    check_append(kda, k, v, slots, c, str(kind))


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_append_special_values(kda, kind):
    """Zeros, infinities, NaN, tiny and huge values; scales that are zero, NaN or infinite before."""
    Hk, D, page = 2, 64, 16
    runs = [([i], 0 if i % 2 else 4, 3 if i < 6 else 12) for i in range(12)]
    slots = sequence_slots(runs, page)
    g = gen(3)
    k, v = torch.randn(2, len(slots), Hk, D, generator=g)
    starts = [0]
    for _, _, n in runs:
        starts.append(starts[-1] + n)
    for i, x in enumerate([0.0, math.inf, math.nan, 1e-40, 3e38, -math.inf] * 2):
        k[starts[i] + 1, 0, 5] = x
        v[starts[i] + 2, 1, 7] = x
    for i in (0, 3, 6, 9):
        k[starts[i]:starts[i + 1], 1] = 0 if i % 2 == 0 else 1e-42
        v[starts[i]:starts[i + 1], 0] = 0 if i % 2 == 0 else 1e-42
    c = cache(12, Hk, page, D, kind, 4)
    c[2][4, 1], c[3][4, 0], c[2][8, 0], c[3][8, 1], c[2][10, 0] = 0.0, 0.0, math.nan, math.inf, math.inf
    check_append(kda, k.cuda(), v.cuda(), slots, c, str(kind))


def test_append_slots_outside_the_cache_and_twice(kda):
    Hk, D, page, pages = 2, 128, 32, 3
    g = gen(6)
    slots = torch.tensor([-1, 5, 5, 6, 96, 2 ** 31 - 1, 33, 34, 33, -5] + [64 + i for i in range(20)] + [70, 64],
                         dtype=torch.int32)
    k, v = torch.randn(2, len(slots), Hk, D, generator=g).to(BF16).cuda()
    check_append(kda, k, v, slots, cache(pages, Hk, page, D, E4M3, 7), "twice")


def test_append_many_tokens(kda):
    """Longer chunks of tokens to a workgroup: over 16384 rows of keys and values together."""
    Hk, D, page = 4, 64, 64
    lengths = [1300, 1, 700, 64, 63, 190]
    ids = torch.randperm(60, generator=gen(8)).tolist()
    runs, at = [], 0
    for i, n in enumerate(lengths):
        first = 11 * i
        need = -(-(first + n) // page)
        runs.append((ids[at:at + need], first, n))
        at += need
    slots = sequence_slots(runs, page)
    k, v = torch.randn(2, len(slots), Hk, D, generator=gen(9)).to(BF16).cuda()
    check_append(kda, k, v, slots, cache(60, Hk, page, D, INT8, 10), "many")


# ------------------------------------------------------------------- attention

def layer(total, new, Hq, Hk, D, page, kind, dtype, seed, spread=0.5, q_scale=2.0, extra=2):
    """Inputs on the CPU: q, cache, table, context, q_start.  Places behind the contexts hold any byte."""
    g = gen(seed)
    need = [-(-max(t, 0) // page) for t in total]
    pages = sum(need) + extra
    size = torch.exp(spread * torch.randn(2, pages, Hk, 1, 1, generator=g))
    kv = torch.randn(2, pages, Hk, page, D, generator=g) * size
    kc, ks = ref.fill(kv[0], kind, False)
    vc, vs = ref.fill(kv[1], kind, True)
    ids = torch.randperm(pages, generator=g)
    per = max(need + [1]) + 1
    table = torch.full((len(total), per), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n].int()
        at += n
        if n:
            used = total[b] - (n - 1) * page
            last = int(table[b, n - 1])
            kc.view(torch.uint8)[last, :, used:] = 0x7f       # NaN in e4m3
            vc.view(torch.uint8)[last, :, :, used:] = 0xff if kind is E4M3 else 0x81
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    q = (q_scale * torch.randn(starts[-1], Hq, D, generator=g)).to(dtype)
    return q, [kc, vc, ks, vs], table, torch.tensor(total).int(), torch.tensor(starts).int()


def check_attention(kda, q, c, table, context, starts, what, most=None, scale=None, one=False):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    o, lse = kda.kda_cache_attention(q.cuda(), *[t.cuda() for t in c], table.cuda(), context.cuda(),
                                     q_start=None if one else starts.cuda(), max_queries=most, scale=scale,
                                     want_lse=True)
    want, tol, wl, wt = ref.attention(q, *c, table, context, starts, scale)
    close(o, want, tol, what + " out")
    close(lse, wl, wt, what + " lse")
    return o, lse


SINGLE = [  # contexts, Hq, Hk, D, page, kind, dtype
    ([1], 1, 1, 64, 16, E4M3, BF16), ([777], 32, 8, 128, 64, E4M3, BF16), ([0, 1, 63, 64, 65, 500], 4, 2, 128, 64, INT8, BF16),
    ([15, 16, 17, 31, 129], 6, 1, 64, 16, INT8, F32), ([300, 2, 90], 16, 1, 256, 128, E4M3, F32),
    ([1000, 31, 33], 40, 2, 256, 32, INT8, BF16), ([70] * 70, 8, 8, 64, 32, E4M3, F32),
    ([20000], 4, 2, 128, 128, E4M3, BF16), ([5000, 1], 3, 3, 128, 16, INT8, F32), ([90, 4096], 96, 1, 64, 64, E4M3, BF16)]


@pytest.mark.parametrize("total,Hq,Hk,D,page,kind,dtype", SINGLE)
def test_attention_one_query(kda, total, Hq, Hk, D, page, kind, dtype):
    x = layer(total, [1] * len(total), Hq, Hk, D, page, kind, dtype, sum(total) + Hq)
    check_attention(kda, *x, "one", one=True)


SEVERAL = [  # contexts, queries, Hq, Hk, D, page, kind, dtype
    ([5], [5], 1, 1, 64, 16, E4M3, BF16), ([40, 3, 0, 64, 130], [4, 7, 2, 0, 17], 4, 2, 128, 32, INT8, F32),
    ([1000, 200], [16, 16], 8, 2, 128, 16, E4M3, BF16), ([200, 64, 65], [16, 3, 9], 16, 2, 64, 64, INT8, BF16),
    ([129, 300, 1], [8, 8, 1], 32, 4, 256, 128, E4M3, F32), ([70, 4000], [2, 8], 6, 2, 256, 32, INT8, BF16),
    ([300], [300], 4, 2, 128, 64, E4M3, BF16), ([515, 100, 260], [500, 37, 1], 4, 1, 64, 64, E4M3, F32),
    ([700, 20], [130, 33], 6, 3, 256, 16, INT8, BF16), ([256, 1100], [256, 129], 2, 2, 128, 128, INT8, F32),
    ([90] * 20, [40] * 20, 3, 1, 128, 32, E4M3, BF16), ([2300], [1], 1, 1, 128, 64, E4M3, BF16)]


@pytest.mark.parametrize("total,new,Hq,Hk,D,page,kind,dtype", SEVERAL)
def test_attention_several_queries(kda, total, new, Hq, Hk, D, page, kind, dtype):
    x = layer(total, new, Hq, Hk, D, page, kind, dtype, sum(total) + Hq)
    check_attention(kda, *x, "several", most=max(new))
    check_attention(kda, *x, "any hint", most=1)
    check_attention(kda, *x, "no hint")


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("new", [1, 9, 150])
def test_attention_pages_of_no_cache(kda, kind, new):
    """Given-up pages (-1), numbers that name no page, whole sequences of them."""
    q, c, table, context, starts = layer([500, 400, 200], [new] * 3, 4, 2, 64, 16, kind, BF16, 21)
    table[0, :20] = -1
    table[1, 3], table[1, 7], table[1, 11] = 2 ** 30, -2 ** 31, c[0].shape[0]
    table[2] = -7
    check_attention(kda, q, c, table, context, starts, "pages", most=new)


@pytest.mark.parametrize("new", [1, 5, 100])
def test_attention_lengths_that_do_not_fit(kda, new):
    """Contexts shorter than their queries, negative, beyond the table; row starts beyond the rows."""
    q, c, table, context, starts = layer([200, 150, 90, 90], [new] * 4, 4, 2, 128, 32, E4M3, BF16, 22)
    context[0], context[1] = new - 1, -5
    table[3, 3:] = -1
    context[3] = 2 ** 31 - 1
    want, tol, wl, wt = ref.attention(q, *c, table, context, starts, 0.1)
    bad = starts.clone()
    bad[4] = 2 ** 31 - 1
    o, lse = kda.kda_cache_attention(q.cuda(), *[t.cuda() for t in c], table.cuda(), context.cuda(), q_start=bad.cuda(),
                                     max_queries=new, scale=0.1, want_lse=True)
    close(o, want, tol, "clamped out")
    close(lse, wl, wt, "clamped lse")


@pytest.mark.parametrize("new", [1, 12, 140])
def test_attention_rows_of_no_sequence_stay(kda, new):
    q, c, table, context, starts = layer([100, 60], [new, new], 4, 2, 128, 64, E4M3, BF16, 23)
    more = torch.cat([q, torch.full((9, 4, 128), math.nan, dtype=BF16)]).cuda()
    out = torch.full(more.shape, 7.0, dtype=BF16, device="cuda")
    lse = torch.full(more.shape[:2], 7.0, device="cuda")
    kda.kda_cache_attention(more, *[t.cuda() for t in c], table.cuda(), context.cuda(), q_start=starts.cuda(),
                            max_queries=new, out=out, lse=lse)
    n = q.shape[0]
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    want, tol, wl, wt = ref.attention(q, *c, table, context, starts, 128 ** -0.5)
    close(out[:n], want, tol, "rows")
    close(lse[:n], wl, wt, "rows lse")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 7, 130])
def test_attention_scales(kda, dtype, new):
    """Pages of very different sizes, zero pages, a page that is not finite: NaN for the rows that see it alone."""
    q, c, table, context, starts = layer([330, 200], [new, new], 4, 2, 64, 32, E4M3, dtype, 24, spread=0.0)
    size = 10.0 ** torch.linspace(-12, 8, c[0].shape[0])
    c[3] *= size[torch.randperm(len(size), generator=gen(5))][:, None]
    c[2][table[0, 2].long()] = 0
    c[3][table[0, 5].long()] = 0
    check_attention(kda, q, c, table, context, starts, "sizes", most=new)
    c[3][table[1, :7].long()] = 0                             # no value of the second sequence but zeros
    check_attention(kda, q, c, table, context, starts, "zeros", most=new)
    c[2][table[0, 10].long(), 0] = math.nan                   # tokens 320 .. 329: the last rows see them
    c[3][table[1, 6].long(), 1] = math.nan                    # tokens 192 .. 199
    check_attention(kda, q, c, table, context, starts, "NaN", most=new)
    c[2][table[1].long().clamp(min=0)] = math.nan             # everything
    check_attention(kda, q, c, table, context, starts, "all NaN", most=new)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 4, 130])
def test_attention_queries_of_any_size(kda, dtype, new):
    """Queries scaled by 1e-30 to 1e30 (with keys that bring the scores back): float16's range does not matter."""
    for power in (-30, -6, 6, 30):
        q, c, table, context, starts = layer([200, 150], [new, new], 4, 1, 128, 64, INT8, dtype, 25)
        q = (q.float() * 10.0 ** power).to(dtype)
        c[2] *= 10.0 ** -power
        check_attention(kda, q, c, table, context, starts, f"1e{power}", most=new)
    q, c, table, context, starts = layer([200, 150], [new, new], 4, 1, 128, 64, INT8, dtype, 26)
    q[0, 0] = 0
    check_attention(kda, q, c, table, context, starts, "zero query", most=new, scale=-0.3)
    check_attention(kda, q, c, table, context, starts, "scale 0", most=new, scale=0.0)


@pytest.mark.parametrize("new", [1, 64])
def test_attention_offsets_beyond_32_bits(kda, new):
    Hk, D, page, pages = 16, 256, 128, 9000                   # 4.7e9 bytes each of keys and values
    kc = torch.empty((pages, Hk, page, D), dtype=torch.int8, device="cuda")
    vc = torch.empty((pages, Hk, D, page), dtype=torch.int8, device="cuda")
    ks, vs = torch.zeros((2, pages, Hk), device="cuda")
    q, c, table, context, starts = layer([200], [new], 16, Hk, D, page, INT8, BF16, 27, extra=0)
    far = torch.tensor([8999, 8200])
    near = table[0, :2].long()
    for big, small in ((kc, c[0]), (vc, c[1]), (ks, c[2]), (vs, c[3])):
        big[far.cuda()] = small[near].cuda()
    slots = torch.tensor([8999 * page + 100], dtype=torch.int32)
    kv = torch.randn(2, 1, Hk, D, generator=gen(28)).to(BF16).cuda()
    kda.kda_cache_append(kv[0], kv[1], slots.cuda(), kc, vc, ks, vs)
    ref.append(kv[0].cpu(), near[0:1] * page + 100, c[0], c[2], False)
    ref.append(kv[1].cpu(), near[0:1] * page + 100, c[1], c[3], True)
    for big, small in ((kc, c[0]), (vc, c[1]), (ks, c[2]), (vs, c[3])):
        assert torch.equal(bits(big[far.cuda()]), bits(small[near]))
    want, tol, wl, wt = ref.attention(q, *c, table, context, starts, 1 / 16)
    t = table.clone()
    t[0, :2] = far.int()
    o = kda.kda_cache_attention(q.cuda(), kc, vc, ks, vs, t.cuda(), context.cuda(), q_start=starts.cuda(), max_queries=new)
    close(o, want, tol, "far")


def test_attention_empty_calls(kda):
    q, c, table, context, starts = layer([50], [3], 4, 2, 64, 16, E4M3, BF16, 29)
    d = [t.cuda() for t in c]
    o = kda.kda_cache_attention(q[:0].cuda(), *d, table[:0].cuda(), context[:0].cuda(), q_start=starts[:1].cuda())
    assert o.shape == (0, 4, 64)
    empty = [t[:0] for t in d]                                # a cache of no pages: nothing to see
    o, lse = kda.kda_cache_attention(q.cuda(), *empty, table.cuda(), context.cuda(), q_start=starts.cuda(), want_lse=True)
    assert not o.any() and (lse == -math.inf).all()
    kda.kda_cache_append(q[:, :2].contiguous().cuda(), q[:, :2].contiguous().cuda(), i32([0, 1, 2]), *empty)
    kda.kda_cache_append(q[:0, :2].cuda(), q[:0, :2].cuda(), i32([]), *d)
    a, b = kda.kda_qk_norm_rope_fwd(q[:0].cuda(), q[:0, :2].cuda())
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)
    r = kda.kda_qk_norm_rope_bwd(a, b, a, b)
    assert not r["dq_weight"].any() and not r["dk_weight"].any()


# ------------------------------------------------------------- runs of them all

class Server:
    """A layer's cache and its requests, stepped through the operators as a server does."""

    def __init__(self, kda, B, Hq, Hk, D, page, pages, kind, dtype):
        self.kda, self.shape, self.dtype, self.page = kda, (Hq, Hk, D), dtype, page
        self.table = torch.full((B, pages // B), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=gen(40)).int().cuda()
        self.count = i32([pages])
        self.cached = i32([0] * B)
        self.cache = [torch.zeros((pages, Hk, page, D), device="cuda").to(kind),
                      torch.zeros((pages, Hk, D, page), device="cuda").to(kind),
                      torch.zeros((pages, Hk), device="cuda"), torch.zeros((pages, Hk), device="cuda")]
        self.wq, self.wk = (1 + 0.1 * torch.randn(2, D, generator=gen(41))).cuda()
        self.rotary = rotary_table(self.table.shape[1] * page, D).cuda()

    def step(self, rows, added, tokens, most):
        Hq, Hk, D = self.shape
        p = self.kda.kda_cache_plan(self.cached, added, self.table, self.free, self.count, page_size=self.page,
                                    tokens=tokens)
        n = rows.shape[0]
        q, k, v = (t.view(n, -1, D) for t in rows.split([Hq * D, Hk * D, Hk * D], 1))
        q, k = self.kda.kda_qk_norm_rope_fwd(q, k, self.wq, self.wk, positions=p["positions"], rotary=self.rotary)
        self.kda.kda_cache_append(k, v, p["slots"], *self.cache)
        o = self.kda.kda_cache_attention(q, *self.cache, self.table, p["context"], q_start=p["q_start"], max_queries=most)
        self.cached.copy_(p["context"])
        self.count.copy_(p["free_count"])
        return q, k, v, o, p


@pytest.mark.parametrize("kind,dtype", [(E4M3, BF16), (INT8, F32)])
def test_steps_of_a_server(kda, kind, dtype):
    """Prompts, single tokens and drafts through all four, against attention over the values as they were: what 8
    bits take away is bounded from the codes' step, half of 2^-3 (e4m3) or 1/127 of the page's largest value."""
    B, Hq, Hk, D, page = 3, 8, 2, 64, 16
    s = Server(kda, B, Hq, Hk, D, page, 60, kind, dtype)
    kept = [([], []) for _ in range(B)]
    g = gen(42)
    for added in ([37, 5, 16], [1, 1, 1], [1, 0, 1], [4, 4, 4], [1, 1, 30], [1, 1, 1]):
        n = sum(added)
        rows = torch.randn(n + 3, (Hq + 2 * Hk) * D, generator=g).to(dtype).cuda()
        q, k, v, o, p = s.step(rows, i32(added), n + 3, max(added))
        starts = p["q_start"].tolist()
        for b in range(B):
            kept[b][0].append(k[starts[b]:starts[b + 1]].cpu().double())
            kept[b][1].append(v[starts[b]:starts[b + 1]].cpu().double())
        # as the cache has it: exactly the reference's attention over the codes
        c = [t.cpu() for t in s.cache]
        want, tol, _, _ = ref.attention(q[:n].cpu(), *c, s.table.cpu(), p["context"].cpu(), p["q_start"].cpu(), D ** -0.5)
        close(o[:n], want, tol, f"step {added}")
        for b in range(B):
            K, V = torch.cat(kept[b][0]), torch.cat(kept[b][1])
            T = K.shape[0]
            assert int(p["context"][b]) == T
            ids = s.table[b, :-(-T // page)].cpu().long()
            for x, codes, scales, inner in ((K, c[0], c[2], False), (V, c[1], c[3], True)):
                vals = codes[ids].double()
                vals = vals.transpose(2, 3) if inner else vals
                vals = (vals * scales.double()[ids][..., None, None]).permute(0, 2, 1, 3).reshape(-1, Hk, D)[:T]
                unit = scales.double()[ids].repeat_interleave(page, 0)[:T, :, None]
                # one rounding when it came, one for each of up to 5 later calls that moved the page's scale
                step = (2.0 ** -4 * x.abs() + 2.0 ** -10 * unit) if kind is E4M3 else 0.5 * unit
                assert ((vals - x).abs() <= 6.5 * step + 1e-6 * x.abs()).all(), (added, b)


def test_a_captured_step_replays(kda):
    """A decoding step of all four in one graph, replayed with eager work between, against a server without one."""
    B, Hq, Hk, D, page = 4, 8, 2, 64, 16
    two = [Server(kda, B, Hq, Hk, D, page, 64, E4M3, BF16) for _ in range(2)]
    g = gen(43)
    prompt = torch.randn(40, (Hq + 2 * Hk) * D, generator=g).to(BF16).cuda()
    for s in two:
        s.step(prompt, i32([10, 20, 3, 7]), 40, 20)
    ones, rows = i32([1] * B), torch.zeros((B, (Hq + 2 * Hk) * D), dtype=BF16, device="cuda")
    warm = torch.cuda.Stream()
    saved = [t.clone() for t in (*two[0].cache, two[0].table, two[0].cached, two[0].count)]
    with torch.cuda.stream(warm):
        two[0].step(rows, ones, B, 1)
    torch.cuda.synchronize()
    for t, u in zip((*two[0].cache, two[0].table, two[0].cached, two[0].count), saved):
        t.copy_(u)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = two[0].step(rows, ones, B, 1)[3]
    for t, u in zip((*two[0].cache, two[0].table, two[0].cached, two[0].count), saved):
        t.copy_(u)
    for i in range(20):
        x = torch.randn(rows.shape, generator=g).to(BF16).cuda()
        rows.copy_(x)
        graph.replay()
        want = two[1].step(x, ones, B, 1)[3]
        torch.cuda.synchronize()
        assert torch.equal(o, want), i
        assert torch.equal(two[0].table, two[1].table) and torch.equal(two[0].count, two[1].count)


@pytest.mark.parametrize("new,B", [(1, 3), (40, 2), (700, 2), (2500, 4)])
def test_captured_attention_replays(kda, new, B):
    """Each kernel in a graph of its own: one query, lines of 64 and of 128 rows, a workgroup a block of rows."""
    q, c, table, context, starts = layer([new + 900 - 300 * b for b in range(B)], [new] * B, 16 if new == 2500 else 4, 2, 64,
                                         32, E4M3, BF16, 45)
    d = [t.cuda() for t in c]
    q, t, n, s = q.cuda(), table.cuda(), context.cuda(), starts.cuda()
    kw = dict(q_start=s, max_queries=new, want_lse=True)
    want = kda.kda_cache_attention(q, *d, t, n, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kda.kda_cache_attention(q, *d, t, n, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = kda.kda_cache_attention(q, *d, t, n, **kw)
    for i in range(4):
        o.fill_(7)
        lse.fill_(7)
        graph.replay()
        other = kda.kda_cache_attention(q, *d, t, n, **kw)
        torch.cuda.synchronize()
        for x, y, z in zip((o, lse), want, other):
            assert torch.equal(x, y) and torch.equal(z, y), i
    n.copy_(n - 50)                                           # the graph reads the lengths of the time
    graph.replay()
    want = kda.kda_cache_attention(q, *d, t, n, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_captured_gradients_replay(kda):
    q, k, wq, wk, pos, table = qk_inputs(500, 4, 2, 128, 64, BF16, True, 46)
    g = gen(47)
    dq, dk = (torch.randn(t.shape, generator=g).to(BF16).cuda() for t in (q, k))
    args = (dq, dk, q, k, wq, wk)
    kw = dict(positions=pos, rotary=table)
    kda.kda_qk_norm_rope_bwd(*args, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = kda.kda_qk_norm_rope_bwd(*args, **kw)
    for i in range(4):
        dq.copy_(torch.randn(q.shape, generator=g))
        graph.replay()
        want = kda.kda_qk_norm_rope_bwd(*args, **kw)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(torch.nan_to_num(r[n].float()), torch.nan_to_num(want[n].float())), (i, n)


def test_queries_that_are_not_finite(kda):
    """A row that is not finite is NaN; the rows beside it, of the same products, are not."""
    for new in (1, 8, 100):
        q, c, table, context, starts = layer([300, 200], [new, new], 4, 2, 64, 32, INT8, BF16, 48)
        clean = check_attention(kda, q, c, table, context, starts, "clean", most=new)
        bad = q.clone()
        bad[0, 0, 3], bad[new, 3, 60], bad[2 * new - 1, 1, 0] = math.nan, math.inf, -math.inf
        o, lse = kda.kda_cache_attention(bad.cuda(), *[t.cuda() for t in c], table.cuda(), context.cuda(),
                                         q_start=starts.cuda(), max_queries=new, want_lse=True)
        hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
        hit[0, 0] = hit[new, 3] = hit[2 * new - 1, 1] = True
        assert torch.isnan(o[hit]).all()
        assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("most", [1, 12, 200])
def test_row_starts_of_any_kind_stay_inside(kda, most):
    """Row starts that descend, lengths and tables of any numbers: rows beside the call's stay as they are, and the
    next call is right."""
    q, c, table, context, starts = layer([300, 200, 100], [most] * 3, 4, 2, 64, 32, E4M3, BF16, 49)
    d, N = [t.cuda() for t in c], q.shape[0]
    room = torch.full((N + 64, 4, 64), 7.0, dtype=BF16, device="cuda")
    g = gen(50)
    for i in range(6):
        bad = torch.randint(-50, N + 50, (4,), generator=g).int() if i else torch.tensor([0, N, 0, N]).int()
        n = torch.randint(-100, 2000, (3,), generator=g).int()
        t = torch.randint(-3, c[0].shape[0] + 3, table.shape, generator=g).int()
        kda.kda_cache_attention(q.cuda(), *d, t.cuda(), n.cuda(), q_start=bad.cuda(), max_queries=most, out=room[32:N + 32])
    torch.cuda.synchronize()
    assert (room[:32] == 7).all() and (room[N + 32:] == 7).all()
    check_attention(kda, q, c, table, context, starts, "after", most=most)


def test_plan_pages_of_large_numbers(kda):
    t, p = run_plan(kda, [16, 0], [1, 1], [[2 ** 31 - 1, -1], [-1, -1]], [2 ** 27 - 1, 2 ** 30], 2, 16, 2)
    assert p["slots"].tolist() == [-1, (2 ** 27 - 1) * 16] and t.tolist() == [[2 ** 31 - 1, 2 ** 30], [2 ** 27 - 1, -1]]


def test_other_streams_and_repeatable(kda):
    """On a stream of the caller's, twice, bit for bit; two calls at once with workspaces of their own."""
    q, c, table, context, starts = layer([3000, 900, 64], [3, 1, 2], 8, 2, 128, 64, E4M3, BF16, 44)
    d = [t.cuda() for t in c]
    args = (q.cuda(), *d, table.cuda(), context.cuda())
    kw = dict(q_start=starts.cuda(), max_queries=3, want_lse=True)
    o, lse = kda.kda_cache_attention(*args, **kw)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        r = [kda.kda_cache_attention(*args, stream=s, **kw) for s in (a, b)]
        torch.cuda.synchronize()
        for x, y in r:
            assert torch.equal(x, o) and torch.equal(y, lse)
