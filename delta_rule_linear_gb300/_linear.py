"""Binding of linear attention with a decay per head and of the block norms (include/kda.h).

Argument marshalling only, as ``_lib``: outputs and workspaces are torch tensors of the stream the
call runs on.  q, k, v and the other token arrays may be views with any batch, token and head strides
(16-byte multiples, last dimension contiguous), e.g. slices of one projection's output.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._lib import KDA_BF16, KDA_F32, KdaError, load, query_device_error

_DT = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}
_ACT = {None: 0, "silu": 1, "sigmoid": 2}
_NONE = contextlib.nullcontext()
_on = torch.cuda.stream


def _code(t, what="q/k/v"):
    c = _DT.get(t.dtype)
    if c is None:
        raise TypeError(f"{what} must be bfloat16 or float32, got {t.dtype}")
    return c


def _need(t, name, dtype, shape, dense=True):
    """Refuses a tensor that the call cannot take (dense: contiguous; else a strided view)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dense:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel():
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _strides(*ts):
    """None when every array is contiguous, else their strides without the last dimension."""
    if all(t.is_contiguous() for t in ts):
        return None
    s = [x for t in ts for x in t.stride()[:-1]]
    return (ctypes.c_longlong * len(s))(*s)


def _p(t):
    return None if t is None else t.data_ptr()


def _raw(stream):
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _ok(code, where, lib):
    if code:
        raise KdaError(code, where, lib)


def _ws(need, where, lib, device, workspace):
    if need == 0:
        raise KdaError(4, where, lib)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace too small")
    return workspace


def _heads(H, HV):
    if HV < H or HV % H:
        raise ValueError(f"the value heads ({HV}) must be a multiple of the q/k heads ({H})")


def _decay(decay, shape):
    """1 for a fixed decay per head ([HV]), 0 for one per token and head (or none)."""
    if decay is None:
        return 0
    if decay.dim() == 1:
        _need(decay, "decay", torch.float32, shape[-1:])
        return 1
    _need(decay, "decay", torch.float32, shape)
    return 0


def linear_chunk_fwd(q, k, v, decay=None, initial_state=None, *, scale=None, out=None, final_state=None,
                     workspace=None, stream=None, check_device=False):
    """kda_linear_chunk_fwd: chunked prefill of linear attention with a decay per head,
    h_t = exp(decay_t) h_{t-1} + k_t v_t^T, o_t = h_t^T (scale q_t).

    q, k [B,T,H,dk], v [B,T,HV,dv] (HV a multiple of H; value head hv reads q/k head hv // m), decay
    [B,T,HV] fp32, [HV] (the same at every token) or None; initial_state [B,HV,dk,dv] fp32 or None.
    Returns (o [B,T,HV,dv], final_state [B,HV,dk,dv] fp32).  check_device as in chunk_fwd.
    """
    lib = load()
    B, T, H, dk = q.shape
    HV, dv = v.shape[-2:]
    _heads(H, HV)
    dt = _code(q)
    _need(q, "q", q.dtype, q.shape, False)
    _need(k, "k", q.dtype, q.shape, False)
    _need(v, "v", q.dtype, (B, T, HV, dv), False)
    fixed = _decay(decay, (B, T, HV))
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (B, HV, dk, dv))
    with _NONE if stream is None else _on(stream):
        if out is None:
            out = torch.empty((B, T, HV, dv), dtype=q.dtype, device=q.device)
        else:
            _need(out, "out", q.dtype, (B, T, HV, dv), False)
        if final_state is None:
            final_state = torch.empty((B, HV, dk, dv), dtype=torch.float32, device=q.device)
        else:
            _need(final_state, "final_state", torch.float32, (B, HV, dk, dv))
        need = lib.kda_linear_chunk_fwd_workspace(B, T, H, HV, dk, dv, dt)
        ws = _ws(need, "kda_linear_chunk_fwd_workspace", lib, q.device, workspace)
        _ok(lib.kda_linear_chunk_fwd(_p(q), _p(k), _p(v), _p(decay), fixed, _p(initial_state), _p(out),
                                     _p(final_state), _strides(q, k, v, out), B, T, H, HV, dk, dv, dt, scale or 0.0,
                                     _p(ws), ws.numel() * ws.element_size(), _raw(stream)),
            "kda_linear_chunk_fwd", lib)
        if check_device:
            _ok(query_device_error(ws, stream), "kda_linear_chunk_fwd (device)", lib)
    return out, final_state


def linear_varlen_fwd(q, k, v, cu_seqlens, decay=None, initial_state=None, *, cu_seqlens_cpu=None, scale=None,
                      out=None, final_state=None, workspace=None, stream=None, check_device=False):
    """kda_linear_varlen_fwd: packed sequences [1,total,H,D] split by cu_seqlens [N+1] (int32, device);
    cu_seqlens_cpu, its host copy where there is one, is checked and tells how to split the work.
    Returns (o [1,total,HV,dv], final_state [N,HV,dk,dv] fp32)."""
    lib = load()
    one, total, H, dk = q.shape
    HV, dv = v.shape[-2:]
    _heads(H, HV)
    if one != 1:
        raise ValueError("packed sequences need token arrays with B == 1")
    dt = _code(q)
    N = cu_seqlens.numel() - 1
    _need(q, "q", q.dtype, q.shape, False)
    _need(k, "k", q.dtype, q.shape, False)
    _need(v, "v", q.dtype, (1, total, HV, dv), False)
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    fixed = _decay(decay, (1, total, HV))
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (N, HV, dk, dv))
    host = None
    if cu_seqlens_cpu is not None:
        host = cu_seqlens_cpu.to(torch.int32).contiguous()
        if host.is_cuda or host.numel() != N + 1:
            raise ValueError("cu_seqlens_cpu must be a host tensor of cu_seqlens' length")
    with _NONE if stream is None else _on(stream):
        if out is None:
            out = torch.empty((1, total, HV, dv), dtype=q.dtype, device=q.device)
        else:
            _need(out, "out", q.dtype, (1, total, HV, dv), False)
        if final_state is None:
            final_state = torch.empty((N, HV, dk, dv), dtype=torch.float32, device=q.device)
        else:
            _need(final_state, "final_state", torch.float32, (N, HV, dk, dv))
        need = lib.kda_linear_varlen_fwd_workspace(N, total, H, HV, dk, dv, dt)
        ws = _ws(need, "kda_linear_varlen_fwd_workspace", lib, q.device, workspace)
        _ok(lib.kda_linear_varlen_fwd(_p(q), _p(k), _p(v), _p(decay), fixed, _p(cu_seqlens), _p(host),
                                      _p(initial_state), _p(out), _p(final_state), _strides(q, k, v, out), N, total, H,
                                      HV, dk, dv, dt, scale or 0.0, _p(ws), ws.numel() * ws.element_size(),
                                      _raw(stream)),
            "kda_linear_varlen_fwd", lib)
        if check_device:
            _ok(query_device_error(ws, stream), "kda_linear_varlen_fwd (device)", lib)
    return out, final_state


def linear_decode_step(q, k, v, decay, state, *, scale=None, out=None, stream=None):
    """kda_linear_decode_step: one token per sequence; ``state`` [B,HV,dk,dv] fp32 is updated in place.
    q, k [B,1,H,dk] or [B,H,dk]; v [B,1,HV,dv] or [B,HV,dv]; decay [B,1,HV] or [B,HV] fp32, [HV] or None.
    Returns o with v's shape."""
    lib = load()
    B, HV, dk, dv = state.shape
    H = q.shape[-2]
    _heads(H, HV)
    dt = _code(q)
    mid = (1,) if q.dim() == 4 else ()
    _need(q, "q", q.dtype, (B, *mid, H, dk), False)
    _need(k, "k", q.dtype, (B, *mid, H, dk), False)
    _need(v, "v", q.dtype, (B, *mid, HV, dv), False)
    _need(state, "state", torch.float32, state.shape)
    fixed = 0
    if decay is not None:
        fixed = int(decay.dim() == 1)
        _need(decay, "decay", torch.float32, (HV,) if fixed else (B, *mid[:decay.dim() - 2], HV))
    with _NONE if stream is None else _on(stream):
        if out is None:
            out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        else:
            _need(out, "out", v.dtype, v.shape, False)
        s = None
        if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and out.is_contiguous()):
            s = (ctypes.c_longlong * 8)(*(x for t in (q, k, v, out) for x in (t.stride(0), t.stride(-2))))
        _ok(lib.kda_linear_decode_step(_p(q), _p(k), _p(v), _p(decay), fixed, _p(state), _p(out), s, B, H, HV, dk, dv,
                                       dt, scale or 0.0, _raw(stream)), "kda_linear_decode_step", lib)
    return out


def linear_chunk_bwd(q, k, v, decay, initial_state, d_o, dfinal_state=None, *, scale=None, workspace=None, stream=None,
                     check_device=False):
    """kda_linear_chunk_bwd: gradients of linear_chunk_fwd given dL/do (dtype of q) and dL/dfinal_state
    (fp32 or None).  Returns a dict dq, dk, dv (q's dtype), ddecay (fp32, decay's shape; absent without a
    decay) and dh0 (fp32; absent without an initial state)."""
    lib = load()
    B, T, H, dk = q.shape
    HV, dv = v.shape[-2:]
    _heads(H, HV)
    dt = _code(q)
    _need(q, "q", q.dtype, q.shape, False)
    _need(k, "k", q.dtype, q.shape, False)
    _need(v, "v", q.dtype, (B, T, HV, dv), False)
    _need(d_o, "d_o", q.dtype, (B, T, HV, dv), False)
    fixed = _decay(decay, (B, T, HV))
    for t, name in ((initial_state, "initial_state"), (dfinal_state, "dfinal_state")):
        if t is not None:
            _need(t, name, torch.float32, (B, HV, dk, dv))
    with _NONE if stream is None else _on(stream):
        dev = q.device
        dq = torch.empty((B, T, H, dk), dtype=q.dtype, device=dev)
        dkk = torch.empty((B, T, H, dk), dtype=q.dtype, device=dev)
        dvv = torch.empty((B, T, HV, dv), dtype=q.dtype, device=dev)
        out = dict(dq=dq, dk=dkk, dv=dvv)
        dg = dh0 = None
        if decay is not None:
            dg = out["ddecay"] = torch.empty(decay.shape, dtype=torch.float32, device=dev)
        if initial_state is not None:
            dh0 = out["dh0"] = torch.empty((B, HV, dk, dv), dtype=torch.float32, device=dev)
        need = lib.kda_linear_chunk_bwd_workspace(B, T, H, HV, dk, dv, dt)
        ws = _ws(need, "kda_linear_chunk_bwd_workspace", lib, dev, workspace)
        _ok(lib.kda_linear_chunk_bwd(_p(q), _p(k), _p(v), _p(decay), fixed, _p(initial_state), _p(d_o),
                                     _p(dfinal_state), _p(dq), _p(dkk), _p(dvv), _p(dg), _p(dh0),
                                     _strides(q, k, v, d_o, dq, dkk, dvv), B, T, H, HV, dk, dv, dt, scale or 0.0,
                                     _p(ws), ws.numel() * ws.element_size(), _raw(stream)),
            "kda_linear_chunk_bwd", lib)
        if check_device:
            _ok(query_device_error(ws, stream), "kda_linear_chunk_bwd (device)", lib)
    return out


def _token_strides(t):
    """(token, head) strides of [..., H, D] whose leading dimensions step evenly."""
    lead = t.dim() - 2
    if lead == 0:
        return 0, t.stride(-2)
    for i in range(lead - 1):
        if t.shape[i] > 1 and t.stride(i) != t.stride(i + 1) * t.shape[i + 1]:
            raise ValueError("the leading dimensions must step evenly (one stride from token to token)")
    return t.stride(lead - 1), t.stride(-2)


def _norm_args(x, gate, weight, activation, *more):
    act = _ACT.get(activation if gate is not None else None)
    if act is None:
        raise ValueError("activation must be 'silu' or 'sigmoid'")
    if x.dim() < 2:
        raise ValueError("x must be [..., H, D]")
    H, D = x.shape[-2:]
    dt = _code(x, "x")
    _need(weight, "weight", torch.float32, (D,))
    ts = [x, gate, *more]
    for t, name in zip(ts, ("x", "gate", "d_y")):
        if t is not None:
            _need(t, name, x.dtype, x.shape, False)
    return act, dt, H, D, x.numel() // max(1, H * D)


def gated_norm_fwd(x, gate, weight, *, eps=1e-6, activation="silu", out=None, stream=None):
    """kda_gated_norm_fwd: y = x (mean(x^2) + eps)^(-1/2) weight act(gate) over the last dimension.
    x, gate [..., H, D] (gate None: no gate), weight [D] fp32, activation "silu" or "sigmoid"."""
    lib = load()
    act, dt, H, D, N = _norm_args(x, gate, weight, activation)
    with _NONE if stream is None else _on(stream):
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            _need(out, "out", x.dtype, x.shape, False)
        s = None
        if not (x.is_contiguous() and out.is_contiguous() and (gate is None or gate.is_contiguous())):
            s = (ctypes.c_longlong * 6)(*_token_strides(x), *_token_strides(gate if gate is not None else x),
                                        *_token_strides(out))
        _ok(lib.kda_gated_norm_fwd(_p(x), _p(gate), _p(weight), _p(out), s, N, H, D, dt, act, eps, _raw(stream)),
            "kda_gated_norm_fwd", lib)
    return out


def gated_norm_bwd(d_y, x, gate, weight, *, eps=1e-6, activation="silu", workspace=None, stream=None):
    """kda_gated_norm_bwd: a dict dx, dgate (x's dtype; dgate absent without a gate) and dw [D] fp32."""
    lib = load()
    act, dt, H, D, N = _norm_args(x, gate, weight, activation, d_y)
    with _NONE if stream is None else _on(stream):
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dg = torch.empty(x.shape, dtype=x.dtype, device=x.device) if gate is not None else None
        dw = torch.empty(D, dtype=torch.float32, device=x.device)
        ws = _ws(lib.kda_gated_norm_bwd_workspace(D), "kda_gated_norm_bwd_workspace", lib, x.device, workspace)
        s = None
        if not (x.is_contiguous() and d_y.is_contiguous() and (gate is None or gate.is_contiguous())):
            s = (ctypes.c_longlong * 10)(*_token_strides(x), *_token_strides(gate if gate is not None else x),
                                         *_token_strides(d_y), H * D, D, H * D, D)
        _ok(lib.kda_gated_norm_bwd(_p(d_y), _p(x), _p(gate), _p(weight), _p(dx), _p(dg), _p(dw), s, N, H, D, dt, act, eps,
                                   _p(ws), ws.numel() * ws.element_size(), _raw(stream)), "kda_gated_norm_bwd", lib)
    return dict(dx=dx, dgate=dg, dw=dw) if dg is not None else dict(dx=dx, dw=dw)


def _rows(t, D):
    """Row stride of [..., D] whose leading dimensions step evenly."""
    lead = t.dim() - 1
    for i in range(lead - 1):
        if t.shape[i] > 1 and t.stride(i) != t.stride(i + 1) * t.shape[i + 1]:
            raise ValueError("the leading dimensions must step evenly (one stride from row to row)")
    return t.stride(lead - 1) if lead else D


def _scale(scale, D):
    if isinstance(scale, torch.Tensor):
        _need(scale, "scale", torch.float32, (D,))
        return scale.data_ptr(), 0.0
    return None, float(scale)


def residual_norm_fwd(x, y, weight, *, scale=1.0, eps=1e-6, out=None, out_norm=None, stream=None):
    """kda_residual_norm_fwd: x' = x + scale y and n = x' (mean(x'^2) + eps)^(-1/2) weight over the last
    dimension.  x [..., D] is the residual stream (bf16, or fp32 around bf16 blocks), y [..., D] the
    block's output, weight [D] fp32, scale a number or a [D] fp32 tensor.  Returns (x' in x's dtype, n in
    y's); out may be x."""
    lib = load()
    D = x.shape[-1]
    _need(x, "x", x.dtype, x.shape, False)
    _need(y, "y", y.dtype, x.shape, False)
    _need(weight, "weight", torch.float32, (D,))
    cv, c = _scale(scale, D)
    with _NONE if stream is None else _on(stream):
        for t, name, like in ((out, "out", x), (out_norm, "out_norm", y)):
            if t is not None:
                _need(t, name, like.dtype, x.shape)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if out_norm is None:
            out_norm = torch.empty(x.shape, dtype=y.dtype, device=x.device)
        _ok(lib.kda_residual_norm_fwd(_p(x), _p(y), _p(weight), cv, c, _p(out), _p(out_norm), _rows(x, D), _rows(y, D),
                                      x.numel() // max(1, D), D, _code(x, "x"), _code(y, "y"), eps, _raw(stream)),
            "kda_residual_norm_fwd", lib)
    return out, out_norm


def residual_norm_bwd(d_n, d_x, x, weight, y=None, *, scale=1.0, eps=1e-6, workspace=None, stream=None):
    """kda_residual_norm_bwd: gradients of residual_norm_fwd at its output x (= x'), given those of n and
    x' (d_x None: zeros).  Returns a dict dx (x's dtype; the gradient of the incoming residual), dy = scale
    dx (d_n's dtype), dw [D] fp32, and dscale [D] fp32 when y is given."""
    lib = load()
    D = x.shape[-1]
    _need(x, "x", x.dtype, x.shape)
    _need(d_n, "d_n", d_n.dtype, x.shape)
    _need(weight, "weight", torch.float32, (D,))
    if d_x is not None:
        _need(d_x, "d_x", x.dtype, x.shape)
    if y is not None:
        _need(y, "y", d_n.dtype, x.shape)
    cv, c = _scale(scale, D)
    with _NONE if stream is None else _on(stream):
        out = dict(dx=torch.empty(x.shape, dtype=x.dtype, device=x.device),
                   dy=torch.empty(x.shape, dtype=d_n.dtype, device=x.device),
                   dw=torch.empty(D, dtype=torch.float32, device=x.device))
        if y is not None:
            out["dscale"] = torch.empty(D, dtype=torch.float32, device=x.device)
        ws = _ws(lib.kda_residual_norm_bwd_workspace(D), "kda_residual_norm_bwd_workspace", lib, x.device, workspace)
        _ok(lib.kda_residual_norm_bwd(_p(d_n), _p(d_x), _p(x), _p(y), _p(weight), cv, c, _p(out["dx"]), _p(out["dy"]),
                                      _p(out["dw"]), _p(out.get("dscale")), x.numel() // max(1, D), D, _code(x, "x"),
                                      _code(d_n, "d_n"), eps, _p(ws), ws.numel() * ws.element_size(), _raw(stream)),
            "kda_residual_norm_bwd", lib)
    return out
