"""Python binding of the softmax attention layers between recurrent ones
(libkda.so, include/kda.h): a serving step's plan, norm and rotation of queries
and keys, and a paged cache in 8 bits with the attention that reads it.
Argument marshalling only, as in kda.py.

    plan = kda_cache_plan(cached, added, block_table, free_pages, free_count, page_size=64, tokens=N)
    q, k = kda_qk_norm_rope_fwd(q, k, q_weight, k_weight, eps, positions=plan["positions"], rotary=rotary)
    kda_cache_append(k, v, plan["slots"], k_codes, v_codes, k_scale, v_scale)       # in place
    o = kda_cache_attention(q, k_codes, v_codes, k_scale, v_scale, block_table, plan["context"],
                            q_start=plan["q_start"], max_queries=longest)

and the gradients kda_qk_norm_rope_bwd.  The cache of a layer is k_codes
[pages, Hk, page, D] and v_codes [pages, Hk, D, page] (torch.float8_e4m3fn or
torch.int8) with k_scale and v_scale [pages, Hk] float32; page is 16, 32, 64 or
128 tokens, D is 64, 128 or 256.  Token rows are bfloat16 or float32, indices
int32.  Tensors lie on one GPU; where a token stride is allowed, heads and
channels still lie next to each other.  Outputs and workspaces that a call
allocates belong to the stream it runs on.
"""

from __future__ import annotations

from functools import lru_cache
from typing import Dict, Optional, Tuple, Union

import torch

from .block import _device, _on, _shape, _workspace
from .kda import KDA_CODE_E4M3, KDA_CODE_INT8, _dtype_code, _nbytes, _ptr, _raise, load_library

_CODES = {torch.float8_e4m3fn: KDA_CODE_E4M3, torch.int8: KDA_CODE_INT8}


def _heads(t: torch.Tensor, what: str) -> Tuple[int, int, int, int]:
    """(tokens, heads, channels, token stride) of rows [..., heads, channels]."""
    shape, strides = t.shape, t.stride()
    if len(shape) < 3:
        raise ValueError(f"{what} must be [..., heads, channels]")
    H, D = shape[-2:]
    width = H * D
    if len(shape) == 3 and strides[1:] == (D, 1) and shape[0] > 1 and width:     # the common case
        return shape[0], H, D, strides[0]
    lead = shape[:-2]
    T = lead.numel()
    if T == 0 or width == 0:
        return T, H, D, width
    if (D > 1 and strides[-1] != 1) or (H > 1 and strides[-2] != D):
        raise ValueError(f"{what}: heads and channels must be contiguous")
    # the leading axes as one: each that has more than one entry steps over the next
    stride = step = None
    for n, s in zip(reversed(lead), reversed(strides[:-2])):
        if n == 1:
            continue
        if stride is None:
            stride = s
        elif s != step:
            raise ValueError(f"{what}: tokens must lie at one stride")
        step = s * n
    return T, H, D, width if stride is None else stride


def _gpu(*ts: Optional[torch.Tensor]) -> torch.device:
    """_device of tensors of which the first is given, sooner where nothing is wrong."""
    index = ts[0].get_device()
    for t in ts:
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            return _device(*ts)
    return ts[0].device if index >= 0 else _device(*ts)


def _one_device(dev: torch.device, *ts: Optional[torch.Tensor]):
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on one device")


# ------------------------------------------------------------------------ plan

def kda_cache_plan(cached: torch.Tensor, added: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                   free_count: torch.Tensor, *, page_size: int, tokens: int,
                   stream: Optional[torch.cuda.Stream] = None) -> Dict[str, torch.Tensor]:
    """The plan of a serving step whose request b has cached[b] tokens and brings
    added[b] (int32 [B]).  New pages come from the end of free_pages int32, of
    whose entries the first free_count (int32 [1]) are free; block_table
    [B, max_pages] int32 gets their numbers IN PLACE.  Returns a dict of q_start
    [B+1], context [B], positions [tokens], slots [tokens] and free_count [1], the
    new one, all int32.  `tokens` is the step's room for rows; those behind the
    last request, and those of requests that are not served, have positions and
    slots -1, the latter's context is 0."""
    lib = load_library()
    if cached.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("cached must be [B], block_table [B,max_pages], free_pages [pages]")
    B, per = cached.shape[0], block_table.shape[1]
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    for t, shape, what in ((cached, (B,), "cached"), (added, (B,), "added"), (block_table, (B, per), "block_table"),
                           (free_pages, (free_pages.shape[0],), "free_pages"), (free_count, (1,), "free_count")):
        _shape(t, shape, what, torch.int32)
    dev = _gpu(cached, added, block_table, free_pages, free_count)
    with _on(dev, stream) as handle:
        # one allocation: the outputs are parts of it
        flat = torch.empty(2 * B + 2 + 2 * tokens, dtype=torch.int32, device=dev)
        q_start, context, left, positions, slots = flat.split([B + 1, B, 1, tokens, tokens])
        st = lib.kda_cache_plan(_ptr(cached), _ptr(added), _ptr(block_table), _ptr(free_pages), _ptr(free_count),
                                _ptr(q_start), _ptr(context), _ptr(positions), _ptr(slots), _ptr(left),
                                B, per, free_pages.shape[0], tokens, page_size, handle)
    _raise(st, "kda_cache_plan")
    return {"q_start": q_start, "context": context, "positions": positions, "slots": slots, "free_count": left}


# ------------------------------------------------------------- query, key norm

def _qk_shapes(q, k, q_weight, k_weight, positions, rotary):
    T, Hq, D, sq = _heads(q, "q")
    Tk, Hk, Dk, sk = _heads(k, "k")
    if q.shape[:-2] != k.shape[:-2] or Dk != D:
        raise ValueError("q [...,Hq,D] and k [...,Hk,D] must share tokens and channels")
    if k.dtype is not q.dtype:
        raise TypeError("q and k must have one dtype")
    _shape(q_weight, (D,), "q_weight", torch.float32)
    _shape(k_weight, (D,), "k_weight", torch.float32)
    rows = R = 0
    if rotary is not None:
        if positions is None:
            raise ValueError("rotary needs positions")
        if rotary.dim() != 2:
            raise ValueError("rotary must be [rows,rotary_dim]")
        rows, R = rotary.shape
        _shape(rotary, (rows, R), "rotary", torch.float32)
    _shape(positions, q.shape[:-2], "positions", torch.int32)
    return T, Hq, Hk, D, rows, R, sq, sk


def _like(t: Optional[torch.Tensor], x: torch.Tensor, width: int, what: str, dev) -> Tuple[torch.Tensor, int]:
    """An output of x's shape and type, `t` or a new one, and its token stride."""
    if t is None:
        return torch.empty(x.shape, dtype=x.dtype, device=dev), width
    _shape(t, x.shape, what, x.dtype)
    return t, _heads(t, what)[3]


def kda_qk_norm_rope_fwd(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                         k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
                         positions: Optional[torch.Tensor] = None, rotary: Optional[torch.Tensor] = None,
                         neighbours: bool = False, q_out: Optional[torch.Tensor] = None,
                         k_out: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Each head of q [...,Hq,D] and k [...,Hk,D] over the root of its mean square
    (+ eps), times q_weight or k_weight [D] float32, then the pairs of its first
    R channels turned by the angles in row positions[...] (int32) of rotary
    [rows,R] float32: R/2 cosines, then R/2 sines.  Pairs are (i, i + R/2), or
    neighbours.  q, k and the outputs may have a token stride (parts of a fused
    projection); q_out and k_out may be q and k themselves.  Returns (q_out,
    k_out): zeros where a position is negative, with a table or without one, NaN
    where it is not in the table."""
    lib = load_library()
    T, Hq, Hk, D, rows, R, sq, sk = _qk_shapes(q, k, q_weight, k_weight, positions, rotary)
    code = _dtype_code(q)
    dev = _device(q_weight, k_weight, positions, rotary) or q.device
    if dev.type != "cuda":
        raise ValueError("all tensors must be on the GPU")
    _one_device(dev, q, k, q_out, k_out)
    with _on(dev, stream) as handle:
        q_out, so = _like(q_out, q, Hq * D, "q_out", dev)
        k_out, sko = _like(k_out, k, Hk * D, "k_out", dev)
        st = lib.kda_qk_norm_rope_fwd(_ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), float(eps), _ptr(positions),
                                      _ptr(rotary) if R else None, _ptr(q_out), _ptr(k_out), T, Hq, Hk, D, R, rows,
                                      int(neighbours), sq, sk, so, sko, code, handle)
    _raise(st, "kda_qk_norm_rope_fwd")
    return q_out, k_out


def kda_qk_norm_rope_bwd_workspace_bytes(tokens: int, Hq: int, Hk: int, D: int) -> int:
    """Device bytes kda_qk_norm_rope_bwd needs where a weight's gradient is wanted."""
    return int(load_library().kda_qk_norm_rope_bwd_workspace_bytes(tokens, Hq, Hk, D))


def kda_qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                         q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                         eps: float = 1e-6, *, positions: Optional[torch.Tensor] = None,
                         rotary: Optional[torch.Tensor] = None, neighbours: bool = False, want_dweights: bool = True,
                         dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> Dict[str, torch.Tensor]:
    """Gradients of kda_qk_norm_rope_fwd(q, k, ...) for dq_out and dk_out: a dict of
    dq and dk (q's and k's shapes and type) and, unless want_dweights is False,
    dq_weight and dk_weight [D] float32, the sums over tokens and heads (with or
    without weights).  dq and dk may be passed, with a token stride, and may be
    dq_out and dk_out, or q and k, themselves."""
    lib = load_library()
    T, Hq, Hk, D, rows, R, sq, sk = _qk_shapes(q, k, q_weight, k_weight, positions, rotary)
    code = _dtype_code(q)
    _shape(dq_out, q.shape, "dq_out", q.dtype)
    _shape(dk_out, k.shape, "dk_out", k.dtype)
    sgq, sgk = _heads(dq_out, "dq_out")[3], _heads(dk_out, "dk_out")[3]
    dev = _device(q_weight, k_weight, positions, rotary, workspace) or q.device
    if dev.type != "cuda":
        raise ValueError("all tensors must be on the GPU")
    _one_device(dev, dq_out, dk_out, q, k, dq, dk)
    with _on(dev, stream) as handle:
        dq, sdq = _like(dq, q, Hq * D, "dq", dev)
        dk, sdk = _like(dk, k, Hk * D, "dk", dev)
        out = {"dq": dq, "dk": dk}
        need = 0
        if want_dweights:
            out["dq_weight"], out["dk_weight"] = torch.empty((2, D), dtype=torch.float32, device=dev).unbind()
            need = int(lib.kda_qk_norm_rope_bwd_workspace_bytes(T, Hq, Hk, D))
        ws = _workspace(workspace, need, dev)
        st = lib.kda_qk_norm_rope_bwd(_ptr(dq_out), _ptr(dk_out), _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
                                      float(eps), _ptr(positions), _ptr(rotary) if R else None, _ptr(out["dq"]),
                                      _ptr(out["dk"]), _ptr(out.get("dq_weight")), _ptr(out.get("dk_weight")),
                                      _ptr(ws), _nbytes(ws), T, Hq, Hk, D, R, rows, int(neighbours), sgq, sgk, sq, sk,
                                      sdq, sdk, code, handle)
    _raise(st, "kda_qk_norm_rope_bwd")
    return out


# ----------------------------------------------------------------------- cache

def _cache_shapes(k_codes, v_codes, k_scale, v_scale):
    if k_codes.dim() != 4:
        raise ValueError("k_codes must be [pages,Hk,page,D]")
    pages, Hk, page, D = k_codes.shape
    if k_codes.dtype not in _CODES:
        raise TypeError("the cache must be torch.float8_e4m3fn or torch.int8")
    _shape(v_codes, (pages, Hk, D, page), "v_codes", k_codes.dtype)
    _shape(k_scale, (pages, Hk), "k_scale", torch.float32)
    _shape(v_scale, (pages, Hk), "v_scale", torch.float32)
    return pages, Hk, page, D, _CODES[k_codes.dtype]


def kda_cache_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_codes: torch.Tensor,
                     v_codes: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, *,
                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """New keys and values k, v [...,Hk,D] (with a token stride, if need be) into
    the cache's places slots [...] int32, IN PLACE; slots outside the cache are
    skipped.  A page's scale for a head grows with its largest value, and the
    codes in front of the first place written with it; a page written from its
    first place starts anew.  The tokens that go to one page stand next to each
    other in the call, none that is skipped between them."""
    lib = load_library()
    pages, Hk, page, D, fmt = _cache_shapes(k_codes, v_codes, k_scale, v_scale)
    T, H, Dk, sk = _heads(k, "k")
    sv = _heads(v, "v")[3]
    if H != Hk or Dk != D:
        raise ValueError(f"k must be [...,{Hk},{D}]")
    _shape(v, k.shape, "v", k.dtype)
    _shape(slots, k.shape[:-2], "slots", torch.int32)
    code = _dtype_code(k)
    dev = _gpu(slots, k_codes, v_codes, k_scale, v_scale)
    _one_device(dev, k, v)
    with _on(dev, stream) as handle:
        st = lib.kda_cache_append(_ptr(k), _ptr(v), _ptr(slots), _ptr(k_codes), _ptr(v_codes), _ptr(k_scale),
                                  _ptr(v_scale), T, Hk, D, pages, page, sk, sv, fmt, code, handle)
    _raise(st, "kda_cache_append")


def kda_cache_attention_workspace_bytes(tokens: int, B: int, Hq: int, Hk: int, D: int, page: int, max_pages: int,
                                        max_queries: int = 1) -> int:
    """Device bytes kda_cache_attention needs."""
    return _attention_bytes(tokens, B, Hq, Hk, D, page, max_pages, max_queries)


@lru_cache(maxsize=1024)
def _attention_bytes(*sizes: int) -> int:
    """A function of the sizes alone: 0.2 us where a call of the library takes 2, of 18 for the smallest attention."""
    return int(load_library().kda_cache_attention_workspace_bytes(*sizes))


def kda_cache_attention(q: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                        v_scale: torch.Tensor, block_table: torch.Tensor, context: torch.Tensor, *,
                        q_start: Optional[torch.Tensor] = None, max_queries: Optional[int] = None,
                        scale: Optional[float] = None, want_lse: bool = False, out: Optional[torch.Tensor] = None,
                        lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None
                        ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """Causal attention of q [tokens,Hq,D] over the cache.  Sequence b's pages are
    block_table[b] (int32 [B,max_pages]), it has context[b] tokens, and its
    queries, the last of them, are the rows from q_start[b] to q_start[b+1]
    (int32 [B+1]; None: one row each).  max_queries is the most rows of a
    sequence, by which the kernel is chosen; None says one without q_start and
    with it that one sequence may have them all, so pass it for speed.  scale is
    D**-0.5 unless given.  Returns out (q's shape and type), or (out, lse) with
    lse [tokens,Hq] float32 if want_lse or lse is given.  A row that sees no
    token has out 0 and lse -inf; rows of no sequence are not written."""
    lib = load_library()
    pages, Hk, page, D, fmt = _cache_shapes(k_codes, v_codes, k_scale, v_scale)
    if q.dim() != 3 or q.shape[2] != D or q.shape[1] == 0 or q.shape[1] % max(Hk, 1):
        raise ValueError(f"q must be [tokens,Hq,{D}] with Hq a multiple of {Hk}")
    N, Hq = q.shape[:2]
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B,max_pages]")
    B, per = block_table.shape
    _shape(block_table, (B, per), "block_table", torch.int32)
    _shape(context, (B,), "context", torch.int32)
    _shape(q_start, (B + 1,), "q_start", torch.int32)
    if q_start is None and N != B:
        raise ValueError("without q_start there is one query a sequence")
    _shape(out, q.shape, "out", q.dtype)
    _shape(lse, (N, Hq), "lse", torch.float32)
    most = 1 if q_start is None else N if max_queries is None else int(max_queries)
    code = _dtype_code(q)
    dev = _gpu(q, k_codes, v_codes, k_scale, v_scale, block_table, context, q_start, out, lse, workspace)
    with _on(dev, stream) as handle:
        if out is None:
            out = torch.empty_like(q)
        if lse is None and want_lse:
            lse = torch.empty((N, Hq), dtype=torch.float32, device=dev)
        ws = _workspace(workspace, _attention_bytes(N, B, Hq, Hk, D, page, per, most), dev)
        st = lib.kda_cache_attention(_ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scale), _ptr(v_scale),
                                     _ptr(block_table), _ptr(context), _ptr(q_start), _ptr(out), _ptr(lse), _ptr(ws),
                                     _nbytes(ws), N, B, Hq, Hk, D, pages, page, per, most,
                                     float(D ** -0.5 if scale is None else scale), fmt, code, handle)
    _raise(st, "kda_cache_attention")
    return out if lse is None else (out, lse)
