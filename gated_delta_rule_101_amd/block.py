"""Python binding of the rest of a recurrent block around the KDA layer: the
short causal convolution, the selective state space scan and layer norm
(libkda.so, include/kda.h).  Argument marshalling only, as in kda.py.

    y, state = kda_short_conv_fwd(x, w, bias, state0)
    y = kda_short_conv_step(x, w, bias, state)              # state updated in place
    y, h = kda_selective_scan_fwd(x, dt, A, Bm, Cm, h0, D=D, z=z, dt_bias=dt_bias)
    y = kda_selective_scan_step(x, dt, A, Bm, Cm, h, D=D, z=z, dt_bias=dt_bias)   # h in place
    y = kda_layer_norm_fwd(x, weight, bias, eps)

and the gradients kda_short_conv_bwd, kda_selective_scan_bwd and
kda_layer_norm_bwd.  Per-token tensors of one call share one dtype (bfloat16 or
float32), which outputs and their gradients have too; parameters, scan states
and parameters' gradients are float32.  Tensors are contiguous and lie on one
GPU.  Outputs and workspaces that the call allocates belong to the stream it
runs on (`stream`, or the current one of the tensors' device).
"""

from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch

from .kda import _dtype_code, _nbytes, _ptr, _raise, load_library


def _stream_handle(index: int) -> int:
    """Handle of the current stream of a device."""
    return torch.cuda.current_stream(index).cuda_stream


# The same without a Stream object, where torch has it: 0.1 us against 1.1, in
# calls of 8 us for the smallest operators.
_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_handle)


class _on:
    """Makes the tensors' device, and `stream` if one is given, current inside
    the block (the launch goes there and what is allocated meanwhile belongs to
    that stream); enters with the stream's handle.  Nothing has to be switched
    in the common case, no stream given on the current device."""

    __slots__ = ("handle", "inner")

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        self.inner = None
        if stream is None:
            if torch.cuda.current_device() != device.index:
                self.inner = torch.cuda.device(device)
            self.handle = _stream_handle(device.index)
        else:
            if stream.device != device:
                raise ValueError("stream must be of the tensors' device")
            self.inner = torch.cuda.stream(stream)   # switches the device as well
            self.handle = stream.cuda_stream

    def __enter__(self) -> int:
        if self.inner is not None:
            self.inner.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)


def _device(*ts: Optional[torch.Tensor]) -> torch.device:
    """The GPU that holds all the tensors given, each contiguous."""
    dev = None
    for t in ts:
        if t is None:
            continue
        d = t.device
        if dev is None:
            if d.type != "cuda":
                raise ValueError("all tensors must be on the GPU")
            dev = d
        elif d != dev:
            raise ValueError("all tensors must be on one device")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    return dev


def _shape(t: Optional[torch.Tensor], shape, what: str, dtype: Optional[torch.dtype] = None):
    if t is None:
        return
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, not {list(t.shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")


def _workspace(workspace: Optional[torch.Tensor], need: int, device) -> Optional[torch.Tensor]:
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if _nbytes(workspace) < need:
        raise ValueError(f"workspace needs {need} bytes")
    return workspace


# ------------------------------------------------------------ short convolution

def _conv_shapes(x, w, bias, state, lengths, token: bool):
    if x.dim() != (2 if token else 3):
        raise ValueError("x must be [B,D]" if token else "x must be [B,T,D]")
    B, T, D = (x.shape[0], 1, x.shape[1]) if token else x.shape
    if w.dim() != 2 or w.shape[0] != D:
        raise ValueError("w must be [D,W]")
    W = w.shape[1]
    _shape(w, (D, W), "w", torch.float32)
    _shape(bias, (D,), "bias", torch.float32)
    _shape(state, (B, W - 1, D), "the state", x.dtype)
    _shape(lengths, (B,), "lengths", torch.int32)
    return B, T, D, W


def kda_short_conv_fwd(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                       state0: Optional[torch.Tensor] = None, *, silu: bool = True,
                       lengths: Optional[torch.Tensor] = None, output_final_state: bool = True,
                       y: Optional[torch.Tensor] = None, state_final: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None
                       ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Depthwise causal convolution of x [B,T,D] with w [D,W] float32 (W 2 to 4,
    the last tap the current token's), bias [D] float32, then SiLU unless
    silu=False.  state0 [B,W-1,D] holds the inputs in front (None: zeros);
    lengths [B] int32 cuts right-padded sequences.  Returns (y, state_final
    [B,W-1,D] or None); state_final may be passed and may be state0 itself."""
    lib = load_library()
    B, T, D, W = _conv_shapes(x, w, bias, state0, lengths, False)
    dev = _device(x, w, bias, state0, lengths, y, state_final)
    _shape(y, x.shape, "y", x.dtype)
    _shape(state_final, (B, W - 1, D), "state_final", x.dtype)
    with _on(dev, stream) as handle:
        if y is None:
            y = torch.empty_like(x)
        if state_final is None and output_final_state:
            state_final = torch.empty((B, W - 1, D), dtype=x.dtype, device=dev)
        st = lib.kda_short_conv_fwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(state0), _ptr(lengths), _ptr(y),
                                    _ptr(state_final), B, T, D, W, int(silu), _dtype_code(x), handle)
    _raise(st, "kda_short_conv_fwd")
    return y, state_final


def kda_short_conv_step(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor], state: torch.Tensor, *,
                        silu: bool = True, y: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token: x [B,D]; state [B,W-1,D] is shifted by it IN PLACE.  Returns
    y [B,D]; y may be passed and may be x itself."""
    lib = load_library()
    B, _, D, W = _conv_shapes(x, w, bias, state, None, True)
    _shape(y, x.shape, "y", x.dtype)
    dev = _device(x, w, bias, state, y)
    with _on(dev, stream) as handle:
        if y is None:
            y = torch.empty_like(x)
        st = lib.kda_short_conv_step(_ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(y), B, D, W, int(silu),
                                     _dtype_code(x), handle)
    _raise(st, "kda_short_conv_step")
    return y


def kda_short_conv_bwd_workspace_bytes(B: int, T: int, D: int, W: int) -> int:
    """Device bytes kda_short_conv_bwd needs."""
    return int(load_library().kda_short_conv_bwd_workspace_bytes(B, T, D, W))


def kda_short_conv_bwd(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                       state0: Optional[torch.Tensor] = None, *, silu: bool = True,
                       dstate_final: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                       want_dstate0: bool = False, workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> Dict[str, torch.Tensor]:
    """Gradients of kda_short_conv_fwd for dy [B,T,D] and dstate_final [B,W-1,D]:
    a dict of dx [B,T,D] (x's dtype), dw [D,W] and dbias [D] (float32, dbias
    with or without a bias) and, if want_dstate0, dstate0 [B,W-1,D]."""
    lib = load_library()
    B, T, D, W = _conv_shapes(x, w, bias, state0, lengths, False)
    _shape(dy, x.shape, "dy", x.dtype)
    _shape(dstate_final, (B, W - 1, D), "dstate_final", x.dtype)
    dev = _device(dy, x, w, bias, state0, dstate_final, lengths, workspace)
    with _on(dev, stream) as handle:
        out = {"dx": torch.empty_like(x), "dw": torch.empty_like(w),
               "dbias": torch.empty((D,), dtype=torch.float32, device=dev)}
        if want_dstate0:
            out["dstate0"] = torch.empty((B, W - 1, D), dtype=x.dtype, device=dev)
        ws = _workspace(workspace, int(lib.kda_short_conv_bwd_workspace_bytes(B, T, D, W)), dev)
        st = lib.kda_short_conv_bwd(_ptr(dy), _ptr(x), _ptr(w), _ptr(bias), _ptr(state0), _ptr(dstate_final),
                                    _ptr(lengths), _ptr(out["dx"]), _ptr(out["dw"]), _ptr(out["dbias"]),
                                    _ptr(out.get("dstate0")), _ptr(ws), _nbytes(ws), B, T, D, W, int(silu),
                                    _dtype_code(x), handle)
    _raise(st, "kda_short_conv_bwd")
    return out


# --------------------------------------------------------------- selective scan

def _scan_shapes(x, dt, A, Bm, Cm, h, D, z, dt_bias, lengths, token: bool):
    if x.dim() != (2 if token else 3):
        raise ValueError("x must be [B,D]" if token else "x must be [B,T,D]")
    B, T, C = (x.shape[0], 1, x.shape[1]) if token else x.shape
    if A.dim() != 2 or A.shape[0] != C:
        raise ValueError("A must be [D,N]")
    N = A.shape[1]
    lead = (B,) if token else (B, T)
    if Bm.dim() != len(lead) + 2:
        raise ValueError("Bm must be [B,G,N]" if token else "Bm must be [B,T,G,N]")
    G = Bm.shape[-2]
    _shape(A, (C, N), "A", torch.float32)
    _shape(dt, x.shape, "dt", x.dtype)
    _shape(Bm, lead + (G, N), "Bm", x.dtype)
    _shape(Cm, lead + (G, N), "Cm", x.dtype)
    _shape(z, x.shape, "z", x.dtype)
    _shape(D, (C,), "D", torch.float32)
    _shape(dt_bias, (C,), "dt_bias", torch.float32)
    _shape(h, (B, C, N), "the state", torch.float32)
    _shape(lengths, (B,), "lengths", torch.int32)
    return B, T, C, N, G


def kda_selective_scan_fwd_workspace_bytes(B: int, T: int, D: int, N: int, G: int = 1) -> int:
    """Device bytes with which kda_selective_scan_fwd cuts the sequence into segments (0: it would not)."""
    return int(load_library().kda_selective_scan_fwd_workspace_bytes(B, T, D, N, G))


def kda_selective_scan_fwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                           h0: Optional[torch.Tensor] = None, *, D: Optional[torch.Tensor] = None,
                           z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                           softplus: bool = True, lengths: Optional[torch.Tensor] = None,
                           output_final_state: bool = True, y: Optional[torch.Tensor] = None,
                           h_final: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None
                           ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Selective scan over x, dt, z [B,T,D] with rates A [D,N] float32 (N 1 to
    64), Bm, Cm [B,T,G,N], skip D and dt_bias [D] float32, states h0 [B,D,N]
    float32 (None: zeros), lengths [B] int32 of right-padded sequences.
    Returns (y [B,T,D], h_final [B,D,N] or None); h_final may be passed and may
    be h0 itself.  The workspace (device bytes) is allocated here when not given."""
    lib = load_library()
    B, T, C, N, G = _scan_shapes(x, dt, A, Bm, Cm, h0, D, z, dt_bias, lengths, False)
    _shape(y, x.shape, "y", x.dtype)
    _shape(h_final, (B, C, N), "h_final", torch.float32)
    dev = _device(x, dt, A, Bm, Cm, h0, D, z, dt_bias, lengths, y, h_final, workspace)
    with _on(dev, stream) as handle:
        if y is None:
            y = torch.empty_like(x)
        if h_final is None and output_final_state:
            h_final = torch.empty((B, C, N), dtype=torch.float32, device=dev)
        ws = _workspace(workspace, int(lib.kda_selective_scan_fwd_workspace_bytes(B, T, C, N, G)), dev)
        st = lib.kda_selective_scan_fwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z),
                                        _ptr(dt_bias), _ptr(h0), _ptr(lengths), _ptr(y), _ptr(h_final), _ptr(ws),
                                        _nbytes(ws), B, T, C, N, G, int(softplus), _dtype_code(x), handle)
    _raise(st, "kda_selective_scan_fwd")
    return y, h_final


def kda_selective_scan_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                            h: torch.Tensor, *, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                            dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                            y: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token: x, dt, z [B,D], Bm, Cm [B,G,N]; the states h [B,D,N] float32
    are advanced IN PLACE.  Returns y [B,D]."""
    lib = load_library()
    B, _, C, N, G = _scan_shapes(x, dt, A, Bm, Cm, h, D, z, dt_bias, None, True)
    _shape(y, x.shape, "y", x.dtype)
    dev = _device(x, dt, A, Bm, Cm, h, D, z, dt_bias, y)
    with _on(dev, stream) as handle:
        if y is None:
            y = torch.empty_like(x)
        st = lib.kda_selective_scan_step(_ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z),
                                         _ptr(dt_bias), _ptr(h), _ptr(y), B, C, N, G, int(softplus),
                                         _dtype_code(x), handle)
    _raise(st, "kda_selective_scan_step")
    return y


def kda_selective_scan_bwd_workspace_bytes(B: int, T: int, D: int, N: int, G: int = 1) -> int:
    """Device bytes kda_selective_scan_bwd needs."""
    return int(load_library().kda_selective_scan_bwd_workspace_bytes(B, T, D, N, G))


def kda_selective_scan_bwd(dy: torch.Tensor, x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor,
                           Cm: torch.Tensor, h0: Optional[torch.Tensor] = None, *,
                           D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                           dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                           dh_final: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                           want_dh0: bool = False, workspace: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> Dict[str, torch.Tensor]:
    """Gradients of kda_selective_scan_fwd for dy [B,T,D] and dh_final [B,D,N]
    float32: a dict of dx, ddt [B,T,D], dB, dC [B,T,G,N] (x's dtype), dA [D,N]
    float32, dD, ddt_bias [D] float32 and dz [B,T,D] where D, dt_bias and z are
    given, and, if want_dh0, dh0 [B,D,N] float32."""
    lib = load_library()
    B, T, C, N, G = _scan_shapes(x, dt, A, Bm, Cm, h0, D, z, dt_bias, lengths, False)
    _shape(dy, x.shape, "dy", x.dtype)
    _shape(dh_final, (B, C, N), "dh_final", torch.float32)
    dev = _device(dy, x, dt, A, Bm, Cm, h0, D, z, dt_bias, dh_final, lengths, workspace)
    with _on(dev, stream) as handle:
        out = {"dx": torch.empty_like(x), "ddt": torch.empty_like(x), "dA": torch.empty_like(A),
               "dB": torch.empty_like(Bm), "dC": torch.empty_like(Cm)}
        if C == 0:   # the library has nothing to launch; the rows of B and C still have gradients, of no channel
            out["dB"].zero_()
            out["dC"].zero_()
        if D is not None:
            out["dD"] = torch.empty_like(D)
        if z is not None:
            out["dz"] = torch.empty_like(z)
        if dt_bias is not None:
            out["ddt_bias"] = torch.empty_like(dt_bias)
        if want_dh0:
            out["dh0"] = torch.empty((B, C, N), dtype=torch.float32, device=dev)
        ws = _workspace(workspace, int(lib.kda_selective_scan_bwd_workspace_bytes(B, T, C, N, G)), dev)
        st = lib.kda_selective_scan_bwd(_ptr(dy), _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z),
                                        _ptr(dt_bias), _ptr(h0), _ptr(dh_final), _ptr(lengths), _ptr(out["dx"]),
                                        _ptr(out["ddt"]), _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dC"]),
                                        _ptr(out.get("dD")), _ptr(out.get("dz")), _ptr(out.get("ddt_bias")),
                                        _ptr(out.get("dh0")), _ptr(ws), _nbytes(ws), B, T, C, N, G, int(softplus),
                                        _dtype_code(x), handle)
    _raise(st, "kda_selective_scan_bwd")
    return out


# ------------------------------------------------------------------- layer norm

def kda_layer_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, eps: float = 1e-5, *,
                       y: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y = (x - mean) / sqrt(var + eps) * weight + bias over the last axis of x
    [..., D] (D up to 16384), weight and bias [D] float32 or None.  y may be
    passed and may be x itself."""
    lib = load_library()
    if x.dim() == 0:
        raise ValueError("x must be [..., D]")
    D = x.shape[-1]
    _shape(weight, (D,), "weight", torch.float32)
    _shape(bias, (D,), "bias", torch.float32)
    _shape(y, x.shape, "y", x.dtype)
    dev = _device(x, weight, bias, y)
    with _on(dev, stream) as handle:
        if y is None:
            y = torch.empty_like(x)
        st = lib.kda_layer_norm_fwd(_ptr(x), _ptr(weight), _ptr(bias), float(eps), _ptr(y),
                                    x.numel() // D if D else 0, D, _dtype_code(x), handle)
    _raise(st, "kda_layer_norm_fwd")
    return y


def kda_layer_norm_bwd_workspace_bytes(rows: int, D: int) -> int:
    """Device bytes kda_layer_norm_bwd needs where a parameter's gradient is wanted."""
    return int(load_library().kda_layer_norm_bwd_workspace_bytes(rows, D))


def kda_layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       eps: float = 1e-5, *, want_dweight: bool = True, want_dbias: bool = True,
                       dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None
                       ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of kda_layer_norm_fwd for dy (x's shape and dtype): (dx, dweight
    [D] float32 or None, dbias [D] float32 or None).  dx may be passed and may
    be dy itself."""
    lib = load_library()
    if x.dim() == 0:
        raise ValueError("x must be [..., D]")
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    _shape(dy, x.shape, "dy", x.dtype)
    _shape(weight, (D,), "weight", torch.float32)
    _shape(dx, x.shape, "dx", x.dtype)
    dev = _device(dy, x, weight, dx, workspace)
    with _on(dev, stream) as handle:
        if dx is None:
            dx = torch.empty_like(x)
        dw = torch.empty((D,), dtype=torch.float32, device=dev) if want_dweight else None
        db = torch.empty((D,), dtype=torch.float32, device=dev) if want_dbias else None
        need = int(lib.kda_layer_norm_bwd_workspace_bytes(rows, D)) if want_dweight or want_dbias else 0
        ws = _workspace(workspace, need, dev)
        st = lib.kda_layer_norm_bwd(_ptr(dy), _ptr(x), _ptr(weight), float(eps), _ptr(dx), _ptr(dw), _ptr(db),
                                    _ptr(ws), _nbytes(ws), rows, D, _dtype_code(x), handle)
    _raise(st, "kda_layer_norm_bwd")
    return dx, dw, db
