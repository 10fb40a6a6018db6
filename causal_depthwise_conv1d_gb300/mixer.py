"""Binding of the gated delta rule, the gated linear recurrence and the layer
and group norms (include/ccv.h).

As in ``binding.py``: argument checks that need tensors, allocation of missing
outputs and of the workspace, and the C call on the tensor's current stream.
These are made by a small C++ extension (``ext/mixer_ext.cpp``): in Python they
took 15-20 us a call, several times a decode step's kernel.  The compute is in
the library's kernels alone.

    gated_delta_rule_fwd    whole sequences         (ccv_gdr_fwd)
    gated_delta_rule_bwd    its backward pass       (ccv_gdr_bwd)
    gated_delta_rule_step   decode step             (ccv_gdr_step)
    layer_norm_fwd          layer normalisation     (ccv_ln_fwd)
    layer_norm_bwd          its backward pass       (ccv_ln_bwd)

    gated_linear_recurrence_fwd    whole sequences      (ccv_glr_fwd)
    gated_linear_recurrence_bwd    its backward pass    (ccv_glr_bwd)
    gated_linear_recurrence_step   decode step          (ccv_glr_step)
    group_norm_fwd                 group normalisation  (ccv_gn_fwd)
    group_norm_bwd                 its backward pass    (ccv_gn_bwd)
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional, Tuple, Union

import torch

from .binding import CcvError, _arr, _i64p, load_library  # noqa: F401

EXT_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_mixer_ext.so")

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
    "ccv_glr_fwd": _T * 3 + [_vp, _i64] + _T * 5 + [_vp, _u64] + [_i64] * 3 + [_int, _vp],
    "ccv_glr_fwd_workspace_size": [_i64] * 3 + [_int, ctypes.POINTER(_u64)],
    "ccv_glr_step": _T * 3 + [_vp, _i64] + _T + [_i64, _vp, _i64] + _T + [_i64] * 3 + [_int, _vp],
    "ccv_glr_bwd": _T * 3 + [_vp, _i64] + _T * 8 + [_vp, _i64] + _T + [_vp, _u64] + [_i64] * 3 + [_int, _vp],
    "ccv_glr_bwd_workspace_size": [_i64] * 3 + [_int, ctypes.POINTER(_u64)],
    "ccv_gn_fwd": _T + [_vp, _i64] * 2 + _T + [_vp, _u64] + [_i64] * 4 + [_f32, _int, _int, _int, _vp],
    "ccv_gn_fwd_workspace_size": [_i64] * 4 + [ctypes.POINTER(_u64)],
    "ccv_gn_bwd": _T + [_vp, _i64] * 2 + _T * 2 + [_vp, _i64] * 2 + [_vp, _u64] + [_i64] * 4 +
                  [_f32, _int, _int, _int, _vp],
    "ccv_gn_bwd_workspace_size": [_i64] * 4 + [ctypes.POINTER(_u64)],
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


_ext_module = None


def _ext():
    """The tensor front end (ext/mixer_ext.cpp), loaded with the library it calls."""
    global _ext_module
    if _ext_module is None:
        lib = load_library()
        if not os.path.exists(EXT_PATH):
            raise CcvError(-1, f"{EXT_PATH} is missing: build it with __graft_entry__.build() "
                               "or python causal_depthwise_conv1d_gb300/build.py")
        # the extension resolves the C ABI from the library that is already loaded
        ctypes.CDLL(lib._name, mode=ctypes.RTLD_GLOBAL)
        spec = importlib.util.spec_from_file_location("_mixer_ext", EXT_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _ext_module = module
    return _ext_module


def _raise(rc: int):
    raise CcvError(rc, load_library().ccv_last_error().decode())


def _need(name: str, *key: int) -> int:
    n = _u64(0)
    _call(name, *key, ctypes.byref(n))
    return int(n.value)


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
    rc, out, final = (_ext_module or _ext()).gdr_fwd(q, k, v, g, beta, scale, seq_idx, initial_state,
                                                     return_final_state, final_state_out, out, workspace,
                                                     None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return out if final is None else (out, final)


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
    rc, out = (_ext_module or _ext()).gdr_step(q, k, v, g, beta, state, scale, state_indices, out,
                                               None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return out


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
    rc, *grads = (_ext_module or _ext()).gdr_bwd(q, k, v, g, beta, dout, scale, seq_idx, initial_state, dfinal_state,
                                                 dq, dk, dv, dg, dbeta, dinitial_state, return_dinitial_state,
                                                 workspace, None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return tuple(grads)


def ccv_ln_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Layer normalisation of x [..., D] over its last dimension; weight and
    bias [D] in a dtype of their own, or None."""
    rc, out = (_ext_module or _ext()).ln_fwd(x, weight, bias, eps, out, None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
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
    rc, *grads = (_ext_module or _ext()).ln_bwd(x, weight, dout, bias, eps, dx, dweight, dbias, workspace,
                                                None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return tuple(grads)


def ccv_glr_fwd_workspace_size(B: int, L: int, C: int, dtype: int) -> int:
    """Bytes of workspace ``ccv_glr_fwd`` needs for these sizes."""
    return _need("ccv_glr_fwd_workspace_size", B, L, C, dtype)


def ccv_glr_fwd(x: torch.Tensor, decay_gate: torch.Tensor, input_gate: torch.Tensor, rate: torch.Tensor,
                seq_idx: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                return_final_state: bool = False, final_state_out: Optional[torch.Tensor] = None,
                return_chunk_states: bool = False, chunk_states_out: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """Gated linear recurrence over whole sequences: with
    a = exp(-rate sigmoid(decay_gate)), h_t = a h_{t-1} + sqrt(1 - a^2) sigmoid(input_gate) x.

    x, decay_gate, input_gate [B,L,C] (any strides; the gates before their
    sigmoid), rate FP32 [C] >= 0, seq_idx int32 [B,L], initial_state FP32 [B,C].
    Returns ``out`` [B,L,C], followed, where requested, by the final state FP32
    [B,C] and by the states before every 64th token FP32 [B,ceil(L/64),C],
    which ``ccv_glr_bwd`` takes.
    """
    rc, out, *extra = (_ext_module or _ext()).glr_fwd(x, decay_gate, input_gate, rate, seq_idx, initial_state,
                                                      return_final_state, final_state_out, return_chunk_states,
                                                      chunk_states_out, out, workspace,
                                                      None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    extra = [t for t in extra if t is not None]
    return (out, *extra) if extra else out


def ccv_glr_step(x: torch.Tensor, decay_gate: torch.Tensor, input_gate: torch.Tensor, rate: torch.Tensor,
                 state: torch.Tensor, state_indices: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Decode step of the gated linear recurrence: S new tokens per request
    against the cache ``state`` FP32 [n_slots,C], advanced in place.

    x, decay_gate, input_gate [B,S,C], or [B,C] for one token.
    ``state_indices`` int32 [B] names each request's slot (default: request b
    uses slot b); negative or too large: a padding row, whose outputs are zero.
    Returns out in x's shape.
    """
    rc, out = (_ext_module or _ext()).glr_step(x, decay_gate, input_gate, rate, state, state_indices, out,
                                               None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return out


def ccv_glr_bwd_workspace_size(B: int, L: int, C: int, dtype: int) -> int:
    """Bytes of workspace ``ccv_glr_bwd`` needs for these sizes."""
    return _need("ccv_glr_bwd_workspace_size", B, L, C, dtype)


def ccv_glr_bwd(x: torch.Tensor, decay_gate: torch.Tensor, input_gate: torch.Tensor, rate: torch.Tensor,
                dout: torch.Tensor, seq_idx: Optional[torch.Tensor] = None,
                initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                chunk_states: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                ddecay_gate: Optional[torch.Tensor] = None, dinput_gate: Optional[torch.Tensor] = None,
                drate: Optional[torch.Tensor] = None, dinitial_state: Optional[torch.Tensor] = None,
                return_dinitial_state: bool = False, workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """Backward pass of ``ccv_glr_fwd``: returns (dx, ddecay_gate, dinput_gate, drate, dinitial_state).

    The forward's inputs plus dout [B,L,C] and dfinal_state FP32 [B,C] (or
    None).  ``chunk_states`` is what the forward pass returned with
    ``return_chunk_states``; without it the states are computed once more.
    Gradients have their inputs' shapes and dtypes; dinitial_state is made when
    initial_state is given and ``return_dinitial_state`` is set (or the tensor
    is passed in).
    """
    rc, *grads = (_ext_module or _ext()).glr_bwd(x, decay_gate, input_gate, rate, dout, seq_idx, initial_state,
                                                 dfinal_state, chunk_states, dx, ddecay_gate, dinput_gate, drate,
                                                 dinitial_state, return_dinitial_state, workspace,
                                                 None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return tuple(grads)


def _silu(activation: Optional[str]) -> bool:
    if activation not in (None, "silu", "swish"):
        raise ValueError(f"activation must be None, 'silu' or 'swish', got {activation!r}")
    return activation is not None


def ccv_gn_fwd_workspace_size(N: int, S: int, C: int, groups: int) -> int:
    """Bytes of workspace ``ccv_gn_fwd`` needs."""
    return _need("ccv_gn_fwd_workspace_size", N, S, C, groups)


def ccv_gn_fwd(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5, activation: Optional[str] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Group normalisation of x [N, ..., C], channels last, then the activation (None, "silu" or "swish").

    Statistics of C / groups adjacent channels over all inner dimensions; with
    x [N, C] every row's groups on their own, as the norm of a token's heads.
    weight and bias [C] in a dtype of their own, or None.
    """
    rc, out = (_ext_module or _ext()).gn_fwd(x, groups, weight, bias, eps, _silu(activation), out, workspace,
                                             None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return out


def ccv_gn_bwd_workspace_size(N: int, S: int, C: int, groups: int) -> int:
    """Bytes of workspace ``ccv_gn_bwd`` needs."""
    return _need("ccv_gn_bwd_workspace_size", N, S, C, groups)


def ccv_gn_bwd(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor], dout: torch.Tensor,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5, activation: Optional[str] = None,
               dx: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
               dbias: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """Backward pass of ``ccv_gn_fwd``: returns (dx, dweight, dbias).

    x, groups, weight, bias, eps, activation: the forward's; dout in x's shape.
    dweight (dbias) is made when weight (bias) is given, in its dtype.
    """
    rc, *grads = (_ext_module or _ext()).gn_bwd(x, groups, weight, dout, bias, eps, _silu(activation), dx, dweight,
                                                dbias, workspace, None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return tuple(grads)


gated_delta_rule_fwd = ccv_gdr_fwd
gated_delta_rule_bwd = ccv_gdr_bwd
gated_delta_rule_step = ccv_gdr_step
layer_norm_fwd = ccv_ln_fwd
layer_norm_bwd = ccv_ln_bwd
gated_linear_recurrence_fwd = ccv_glr_fwd
gated_linear_recurrence_bwd = ccv_glr_bwd
gated_linear_recurrence_step = ccv_glr_step
group_norm_fwd = ccv_gn_fwd
group_norm_bwd = ccv_gn_bwd
