"""Binding of the gated delta rule and of layer normalisation (include/ccv.h).

As in ``binding.py``: argument checks that need tensors, allocation of missing
outputs and of the workspace, and the C call on the tensor's current stream.
The compute is in the library's kernels alone.

    gated_delta_rule_fwd    whole sequences         (ccv_gdr_fwd)
    gated_delta_rule_bwd    its backward pass       (ccv_gdr_bwd)
    gated_delta_rule_step   decode step             (ccv_gdr_step)
    layer_norm_fwd          layer normalisation     (ccv_ln_fwd)
    layer_norm_bwd          its backward pass       (ccv_ln_bwd)
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple, Union

import torch

from .binding import TORCH_DTYPE, CcvError, _arr, _i64p, load_library

_vp, _i64, _f32, _int, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_uint64
_T = [_vp, _i64p]  # a tensor: pointer, strides

_SIGNATURES = {
    "ccv_gdr_fwd": _T * 9 + [_vp, _u64] + [_i64] * 6 + [_f32, _int, _vp],
    "ccv_gdr_fwd_workspace_size": [_i64] * 6 + [_int, ctypes.POINTER(_u64)],
    "ccv_gdr_step": _T * 6 + [_i64, _vp, _i64] + _T + [_i64] * 6 + [_f32, _int, _vp],
    "ccv_gdr_bwd": _T * 15 + [_vp, _u64] + [_i64] * 6 + [_f32, _int, _vp],
    "ccv_gdr_bwd_workspace_size": [_i64] * 6 + [_int, ctypes.POINTER(_u64)],
    "ccv_ln_fwd": _T + [_vp, _i64] * 2 + _T + [_i64, _i64, _f32, _int, _int, _vp],
    "ccv_ln_bwd": _T + [_vp, _i64] + _T * 2 + [_vp, _i64] * 2 + [_vp, _u64, _i64, _i64, _f32, _int, _int, _vp],
    "ccv_ln_bwd_workspace_size": [_i64, _i64, ctypes.POINTER(_u64)],
}
_bound = {}


def _fn(name: str):
    f = _bound.get(name)
    if f is None:
        f = getattr(load_library(), name)
        f.argtypes = _SIGNATURES[name]
        f.restype = _int
        _bound[name] = f
    return f


def _call(name: str, *args) -> None:
    rc = (_bound.get(name) or _fn(name))(*args)
    if rc != 0:
        raise CcvError(rc, load_library().ccv_last_error().decode())


_strides = {}  # the C arrays of stride tuples seen: a decode step's are the same every time


def _st(strides):
    a = _strides.get(strides)
    if a is None:
        if len(_strides) > 4096:
            _strides.clear()
        a = _strides[strides] = _arr(strides)
    return a


def _t(x: Optional[torch.Tensor]):
    """(pointer, strides) of a tensor or of a missing one."""
    return (None, None) if x is None else (x.data_ptr() or None, _st(x.stride()))


def _v(x: Optional[torch.Tensor]):
    """(pointer, stride) of a vector."""
    return (None, 0) if x is None else (x.data_ptr() or None, x.stride(0))


def _ws(x: Optional[torch.Tensor]):
    """(pointer, bytes) of a workspace."""
    return (None, 0) if x is None else (x.data_ptr(), x.numel() * x.element_size())


def _check(dev: int, tensors) -> None:
    """(name, tensor, shape, dtype) each: None, or that shape and dtype on the device."""
    for name, t, shape, dtype in tensors:
        if t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0):
            continue
        if t.get_device() != dev or dev < 0:
            raise ValueError("all tensors must live on one CUDA device")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")


def _launch(dev: int, stream: Optional[torch.cuda.Stream], name: str, *args) -> None:
    """The call on `stream` (default: the device's current one), with the device current."""
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        _call(name, *args, raw)
    else:
        with torch.cuda.device(dev):
            _call(name, *args, raw)


def _gdr_sizes(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q and k must be [B, L, Hk, Dk] and v [B, L, Hv, Dv]")
    if v.dtype not in TORCH_DTYPE:
        raise ValueError(f"unsupported dtype {v.dtype}")
    B, L, Hk, Dk = q.shape
    _, _, Hv, Dv = v.shape
    return B, L, Hk, Hv, Dk, Dv


_sizes = {}  # workspace sizes by the sizes they follow from


def _need(name: str, *key: int) -> int:
    n = _sizes.get((name, key))
    if n is None:
        c = _u64(0)
        _call(name, *key, ctypes.byref(c))
        if len(_sizes) > 4096:
            _sizes.clear()
        n = _sizes[name, key] = int(c.value)
    return n


def _workspace(need: int, workspace: Optional[torch.Tensor], device) -> Optional[torch.Tensor]:
    if workspace is None:
        return torch.empty((need,), dtype=torch.uint8, device=device) if need > 0 else None
    if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' CUDA device")
    return workspace


def ccv_gdr_fwd_workspace_size(B: int, L: int, Hk: int, Hv: int, Dk: int, Dv: int, dtype: int) -> int:
    """Bytes of workspace ``ccv_gdr_fwd`` needs for these sizes."""
    return _need("ccv_gdr_fwd_workspace_size", B, L, Hk, Hv, Dk, Dv, dtype)


def ccv_gdr_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                scale: Optional[float] = None, seq_idx: Optional[torch.Tensor] = None,
                initial_state: Optional[torch.Tensor] = None, return_final_state: bool = False,
                final_state_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """Gated delta rule over whole sequences.

    q, k [B,L,Hk,Dk], v [B,L,Hv,Dv] (Hv a multiple of Hk, any strides),
    g FP32 [B,L,Hv] (log decay), beta [B,L,Hv], seq_idx int32 [B,L],
    initial_state FP32 [B,Hv,Dk,Dv]; scale defaults to Dk ** -0.5.  Returns
    ``out`` [B,L,Hv,Dv] or ``(out, final_state)`` when it is requested.
    """
    B, L, Hk, Hv, Dk, Dv = _gdr_sizes(q, k, v)
    dt, st = v.dtype, (B, Hv, Dk, Dv)
    if out is None:
        out = torch.empty((B, L, Hv, Dv), dtype=dt, device=v.device)
    if return_final_state and final_state_out is None:
        final_state_out = torch.empty(st, dtype=torch.float32, device=v.device)
    dev, qk, vo, gate, f32 = v.get_device(), (B, L, Hk, Dk), (B, L, Hv, Dv), (B, L, Hv), torch.float32
    _check(dev, (("q", q, qk, dt), ("k", k, qk, dt), ("v", v, vo, dt), ("g", g, gate, f32), ("beta", beta, gate, dt),
                 ("seq_idx", seq_idx, (B, L), torch.int32), ("initial_state", initial_state, st, f32),
                 ("out", out, vo, dt), ("final_state_out", final_state_out, st, f32)))
    need = ccv_gdr_fwd_workspace_size(B, L, Hk, Hv, Dk, Dv, TORCH_DTYPE[dt])
    ws = _workspace(need, workspace, v.device)
    _launch(dev, stream, "ccv_gdr_fwd", *_t(q), *_t(k), *_t(v), *_t(g), *_t(beta), *_t(seq_idx), *_t(initial_state),
            *_t(out), *_t(final_state_out), *_ws(ws), B, L, Hk, Hv, Dk, Dv, max(Dk, 1) ** -0.5 if scale is None else scale,
            TORCH_DTYPE[dt])
    return (out, final_state_out) if final_state_out is not None else out


def ccv_gdr_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                 state: torch.Tensor, scale: Optional[float] = None, state_indices: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Decode step of the gated delta rule: S new tokens per request against
    the cache ``state`` FP32 [n_slots,Hv,Dk,Dv], advanced in place.

    q, k [B,S,Hk,Dk], v [B,S,Hv,Dv], g, beta [B,S,Hv], or all without S for
    one token.  ``state_indices`` int32 [B] names each request's slot (default:
    request b uses slot b); negative or too large: a padding row, whose outputs
    are zero.  Returns out in v's shape.
    """
    one = v.dim() == 3
    if one:
        q, k, v, g, beta = q.unsqueeze(1), k.unsqueeze(1), v.unsqueeze(1), g.unsqueeze(1), beta.unsqueeze(1)
    B, S, Hk, Hv, Dk, Dv = _gdr_sizes(q, k, v)
    dt = v.dtype
    if state.dim() != 4:
        raise ValueError("state must be [n_slots, Hv, Dk, Dv]")
    if out is None:
        out = torch.empty((B, S, Hv, Dv), dtype=dt, device=v.device)
        res = out.squeeze(1) if one else out
    else:
        res, out = out, (out.unsqueeze(1) if one else out)
    dev, qk, vo, gate, f32 = v.get_device(), (B, S, Hk, Dk), (B, S, Hv, Dv), (B, S, Hv), torch.float32
    slots = state.shape[0]
    _check(dev, (("q", q, qk, dt), ("k", k, qk, dt), ("v", v, vo, dt), ("g", g, gate, f32), ("beta", beta, gate, dt),
                 ("state", state, (slots, Hv, Dk, Dv), f32), ("state_indices", state_indices, (B,), torch.int32),
                 ("out", out, vo, dt)))
    _launch(dev, stream, "ccv_gdr_step", *_t(q), *_t(k), *_t(v), *_t(g), *_t(beta), *_t(state), slots,
            *_v(state_indices), *_t(out), B, S, Hk, Hv, Dk, Dv, max(Dk, 1) ** -0.5 if scale is None else scale,
            TORCH_DTYPE[dt])
    return res


def ccv_gdr_bwd_workspace_size(B: int, L: int, Hk: int, Hv: int, Dk: int, Dv: int, dtype: int) -> int:
    """Bytes of workspace ``ccv_gdr_bwd`` needs for these sizes."""
    return _need("ccv_gdr_bwd_workspace_size", B, L, Hk, Hv, Dk, Dv, dtype)


def ccv_gdr_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                dout: torch.Tensor, scale: Optional[float] = None, seq_idx: Optional[torch.Tensor] = None,
                initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                dv: Optional[torch.Tensor] = None, dg: Optional[torch.Tensor] = None,
                dbeta: Optional[torch.Tensor] = None, dinitial_state: Optional[torch.Tensor] = None,
                return_dinitial_state: bool = False, workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """Backward pass of ``ccv_gdr_fwd``: returns (dq, dk, dv, dg, dbeta, dinitial_state).

    The forward's inputs plus dout [B,L,Hv,Dv] and dfinal_state FP32
    [B,Hv,Dk,Dv] (or None).  Gradients have their inputs' shapes and dtypes;
    dinitial_state is made when initial_state is given and
    ``return_dinitial_state`` is set (or the tensor is passed in).
    """
    B, L, Hk, Hv, Dk, Dv = _gdr_sizes(q, k, v)
    dt, st, dev = v.dtype, (B, Hv, Dk, Dv), v.device
    qk, vo, gate = (B, L, Hk, Dk), (B, L, Hv, Dv), (B, L, Hv)
    dq = torch.empty(qk, dtype=dt, device=dev) if dq is None else dq
    dk = torch.empty(qk, dtype=dt, device=dev) if dk is None else dk
    dv = torch.empty(vo, dtype=dt, device=dev) if dv is None else dv
    dg = torch.empty(gate, dtype=torch.float32, device=dev) if dg is None else dg
    dbeta = torch.empty(gate, dtype=dt, device=dev) if dbeta is None else dbeta
    if dinitial_state is None and return_dinitial_state and initial_state is not None:
        dinitial_state = torch.empty(st, dtype=torch.float32, device=dev)
    f32 = torch.float32
    _check(v.get_device(), (
        ("q", q, qk, dt), ("k", k, qk, dt), ("v", v, vo, dt), ("g", g, gate, f32), ("beta", beta, gate, dt),
        ("seq_idx", seq_idx, (B, L), torch.int32), ("initial_state", initial_state, st, f32), ("dout", dout, vo, dt),
        ("dfinal_state", dfinal_state, st, f32), ("dq", dq, qk, dt), ("dk", dk, qk, dt), ("dv", dv, vo, dt),
        ("dg", dg, gate, f32), ("dbeta", dbeta, gate, dt), ("dinitial_state", dinitial_state, st, f32)))
    need = ccv_gdr_bwd_workspace_size(B, L, Hk, Hv, Dk, Dv, TORCH_DTYPE[dt])
    ws = _workspace(need, workspace, dev)
    _launch(v.get_device(), stream, "ccv_gdr_bwd", *_t(q), *_t(k), *_t(v), *_t(g), *_t(beta), *_t(seq_idx),
            *_t(initial_state), *_t(dout), *_t(dfinal_state), *_t(dq), *_t(dk), *_t(dv), *_t(dg), *_t(dbeta),
            *_t(dinitial_state), *_ws(ws), B, L, Hk, Hv, Dk, Dv, max(Dk, 1) ** -0.5 if scale is None else scale,
            TORCH_DTYPE[dt])
    return dq, dk, dv, dg, dbeta, dinitial_state


def _rows(x: torch.Tensor) -> torch.Tensor:
    """[..., D] as [N, D] without a copy."""
    if x.dim() == 2:
        return x
    if x.dim() == 1:
        return x.unsqueeze(0)
    try:
        return x.view(-1, x.shape[-1])
    except RuntimeError as e:
        raise ValueError("the leading dimensions of a layer norm's tensor must collapse into one stride "
                         "(pass a 2-D view)") from e


def _ln_check(x, weight, bias):
    if x.dim() < 1 or x.dtype not in TORCH_DTYPE:
        raise ValueError(f"x must be [..., D] of a supported dtype, got {x.dtype}")
    D = x.shape[-1]
    par = weight if weight is not None else bias
    wdt = par.dtype if par is not None else x.dtype
    if wdt not in TORCH_DTYPE:
        raise ValueError(f"unsupported weight dtype {wdt}")
    _check(x.get_device(), (("x", x, x.shape, x.dtype), ("weight", weight, (D,), wdt), ("bias", bias, (D,), wdt)))
    return D, wdt


def ccv_ln_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Layer normalisation of x [..., D] over its last dimension; weight and
    bias [D] in a dtype of their own, or None."""
    D, wdt = _ln_check(x, weight, bias)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _check(x.get_device(), (("out", out, x.shape, x.dtype),))
    x2, o2 = (x, out) if x.numel() == 0 else (_rows(x), _rows(out))
    N = x.numel() // D if D else 0
    if N == 0:
        return out
    _launch(x.get_device(), stream, "ccv_ln_fwd", *_t(x2), *_v(weight), *_v(bias), *_t(o2), N, D, eps,
            TORCH_DTYPE[x.dtype], TORCH_DTYPE[wdt])
    return out


def ccv_ln_bwd_workspace_size(N: int, D: int) -> int:
    """Bytes of workspace ``ccv_ln_bwd`` needs."""
    return _need("ccv_ln_bwd_workspace_size", N, D)


def ccv_ln_bwd(x: torch.Tensor, weight: Optional[torch.Tensor], dout: torch.Tensor,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5, dx: Optional[torch.Tensor] = None,
               dweight: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Backward pass of ``ccv_ln_fwd``: returns (dx, dweight, dbias).

    x, weight, bias: the forward's inputs (bias only tells that dbias is
    wanted); dout [..., D].  dweight (dbias) is made when weight (bias) is
    given, in its dtype.
    """
    D, wdt = _ln_check(x, weight, bias)
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if dweight is None and weight is not None:
        dweight = torch.empty((D,), dtype=wdt, device=x.device)
    if dbias is None and bias is not None:
        dbias = torch.empty((D,), dtype=wdt, device=x.device)
    dev = x.get_device()
    _check(dev, (("dout", dout, x.shape, x.dtype), ("dx", dx, x.shape, x.dtype), ("dweight", dweight, (D,), wdt),
                 ("dbias", dbias, (D,), wdt)))
    N = x.numel() // D if D else 0
    x2, g2, d2 = (_rows(x), _rows(dout), _rows(dx)) if N else (x.new_empty((0, D)),) * 3
    need = ccv_ln_bwd_workspace_size(N, D) if dweight is not None or dbias is not None else 0
    ws = _workspace(need, workspace, x.device)
    _launch(dev, stream, "ccv_ln_bwd", *_t(x2), *_v(weight), *_t(g2), *_t(d2), *_v(dweight), *_v(dbias), *_ws(ws), N,
            D, eps, TORCH_DTYPE[x.dtype], TORCH_DTYPE[wdt])
    return dx, dweight, dbias


gated_delta_rule_fwd = ccv_gdr_fwd
gated_delta_rule_bwd = ccv_gdr_bwd
gated_delta_rule_step = ccv_gdr_step
layer_norm_fwd = ccv_ln_fwd
layer_norm_bwd = ccv_ln_bwd
