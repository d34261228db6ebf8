"""Binding of linear attention with a decay per head and of the block norms (include/kda.h).

Argument marshalling only, as ``_lib``: outputs and workspaces are torch tensors of the stream the
call runs on, and the tensors of a call are all on the current device.  q, k, v and the other token
arrays may be views with any batch, token and head strides (16-byte multiples, last dimension
contiguous), e.g. slices of one projection's output.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._lib import KDA_BF16, KDA_F32, KdaError, load, query_device_error

_DT = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}
_ACT = {"silu": 1, "sigmoid": 2}
_F32 = torch.float32
_empty = torch.empty
_like = torch.empty_like      # of contiguous tensors: cheaper than naming shape, type and device
# The calls below cost a few microseconds on the GPU for small inputs, so their checks are a handful of
# comparisons; what fails one goes through _need, which finds the words.


def _code(t, what="q/k/v"):
    c = _DT.get(t.dtype)
    if c is None:
        raise TypeError(f"{what} must be bfloat16 or float32, got {t.dtype}")
    return c


def _need(t, name, dtype, shape, dev, dense=True):
    """Refuses a tensor that the call on device `dev` cannot take (dense: contiguous; else a strided view)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on CUDA device {t.get_device()}, the call's other tensors on device {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dense:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif t.shape[-1] > 1 and t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _view(t, name, dtype, shape, dev):
    """Checks a strided view; True when it is contiguous."""
    if t.is_contiguous() and t.dtype is dtype and t.get_device() == dev and t.shape == shape:
        return True
    _need(t, name, dtype, shape, dev, False)
    return t.is_contiguous()


def _into(t, name, dtype, shape, dev):
    """_view of an output, whose elements have to be apart: through a broadcast dimension CTAs write over one another."""
    if _view(t, name, dtype, shape, dev):
        return True
    if any(s == 0 and n > 1 for s, n in zip(t.stride(), t.shape)) and t.numel():
        raise ValueError(f"{name} must not be a broadcast view")
    return False


def _dense(t, name, dtype, shape, dev):
    if not (t.is_contiguous() and t.dtype is dtype and t.get_device() == dev and t.shape == shape):
        _need(t, name, dtype, shape, dev)


# The current device, on which a call launches; the short way where this torch has it.
_here = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device(t, name):
    """The device of a call, named by its first tensor: the kernels run on the current one, so it has to be that."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev, here = t.get_device(), _here()
    if dev != here:
        raise ValueError(f"{name} is on CUDA device {dev}, but the current device is {here}: make the call under "
                         f"torch.cuda.device({dev})")
    return dev


def _strides(*ts):
    s = [x for t in ts for x in t.stride()[:-1]]
    return (ctypes.c_longlong * len(s))(*s)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle; the short way where this torch has it.
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw(dev):
    return _current(dev) if _current is not None else torch.cuda.current_stream().cuda_stream


def _on(stream, call, *args, **kw):
    """Runs a call on another stream than the current one: what it allocates belongs there too."""
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _ok(code, where, lib):
    if code:
        raise KdaError(code, where, lib)


@functools.lru_cache(maxsize=1024)
def _bytes(query, *sizes):
    return getattr(load(), query)(*sizes)


_HEADER = 256       # bytes of a workspace that is its header alone (the error word)
_headers = {}
_capturing = torch.cuda.is_current_stream_capturing


def _ws(query, sizes, t, stream, workspace, asked=False):
    """(workspace, its bytes) of a call on t's device.  A call that needs the header alone takes one that is kept per
    stream, whose calls follow one another; where its error word is asked for, a fresh one."""
    if workspace is not None:
        # its bytes are counted from here on: a cut or broadcast view has fewer of its own
        if workspace.get_device() != t.get_device() or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on the call's device")
        return workspace, workspace.numel() * workspace.element_size()
    need = _bytes(query, *sizes)
    if need == 0:
        raise KdaError(4, query, load())
    if need > _HEADER or asked:
        return _empty(need, dtype=torch.uint8, device=t.device), need
    key = (t.get_device(), stream)
    ws = _headers.get(key)
    if ws is None:
        ws = _empty(_HEADER, dtype=torch.uint8, device=t.device)
        if not _capturing():        # a capture's memory is its graph's: kept, it would be used beside and after the graph
            _headers[key] = ws
    return ws, _HEADER


def _heads(H, HV):
    if HV < H or HV % H:
        raise ValueError(f"the value heads ({HV}) must be a multiple of the q/k heads ({H})")


def _decay(decay, shape, dev):
    """1 for a fixed decay per head ([HV]), 0 for one per token and head (or none)."""
    if decay is None:
        return 0
    if decay.dim() == 1:
        _dense(decay, "decay", _F32, shape[-1:], dev)
        return 1
    _dense(decay, "decay", _F32, shape, dev)
    return 0


def _qkv(q, k, v, B, T, H, HV, dk, dv, dev):
    """Checks q, k and v; True when all are contiguous."""
    if HV != H:
        _heads(H, HV)
    dt = q.dtype
    return (_view(q, "q", dt, q.shape, dev) & _view(k, "k", dt, (B, T, H, dk), dev) &
            _view(v, "v", dt, (B, T, HV, dv), dev))


def linear_chunk_fwd(q, k, v, decay=None, initial_state=None, *, scale=None, out=None, final_state=None,
                     workspace=None, stream=None, check_device=False):
    """kda_linear_chunk_fwd: chunked prefill of linear attention with a decay per head,
    h_t = exp(decay_t) h_{t-1} + k_t v_t^T, o_t = h_t^T (scale q_t).

    q, k [B,T,H,dk], v [B,T,HV,dv] (HV a multiple of H; value head hv reads q/k head hv // m), decay
    [B,T,HV] fp32, [HV] (the same at every token) or None; initial_state [B,HV,dk,dv] fp32 or None.
    Returns (o [B,T,HV,dv], final_state [B,HV,dk,dv] fp32).  check_device as in chunk_fwd.
    """
    if stream is not None:
        return _on(stream, linear_chunk_fwd, q, k, v, decay, initial_state, scale=scale, out=out,
                   final_state=final_state, workspace=workspace, check_device=check_device)
    lib = load()
    B, T, H, dk = q.shape
    HV, dv = v.shape[-2:]
    dt, dev = _code(q), _device(q, "q")
    plain = _qkv(q, k, v, B, T, H, HV, dk, dv, dev)
    fixed = _decay(decay, (B, T, HV), dev)
    if initial_state is not None:
        _dense(initial_state, "initial_state", _F32, (B, HV, dk, dv), dev)
    if out is None:
        out = _like(v) if plain else _empty((B, T, HV, dv), dtype=q.dtype, device=q.device)
    else:
        plain &= _into(out, "out", q.dtype, (B, T, HV, dv), dev)
    if final_state is None:
        final_state = _empty((B, HV, dk, dv), dtype=_F32, device=q.device)
    else:
        _dense(final_state, "final_state", _F32, (B, HV, dk, dv), dev)
    st = _raw(dev)
    ws, n = _ws("kda_linear_chunk_fwd_workspace", (B, T, H, HV, dk, dv, dt), q, st, workspace, check_device)
    _ok(lib.kda_linear_chunk_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(decay), fixed, _ptr(initial_state),
                                 out.data_ptr(), final_state.data_ptr(), None if plain else _strides(q, k, v, out), B, T, H,
                                 HV, dk, dv, dt, scale or 0.0, ws.data_ptr(), n, st), "kda_linear_chunk_fwd", lib)
    if check_device and B:        # an empty batch launches nothing and leaves the header as it is
        _ok(query_device_error(ws), "kda_linear_chunk_fwd (device)", lib)
    return out, final_state


def linear_varlen_fwd(q, k, v, cu_seqlens, decay=None, initial_state=None, *, cu_seqlens_cpu=None, scale=None,
                      out=None, final_state=None, workspace=None, stream=None, check_device=False):
    """kda_linear_varlen_fwd: packed sequences [1,total,H,D] split by cu_seqlens [N+1] (int32, device);
    cu_seqlens_cpu, its host copy where there is one, is checked and tells how to split the work.
    Returns (o [1,total,HV,dv], final_state [N,HV,dk,dv] fp32)."""
    if stream is not None:
        return _on(stream, linear_varlen_fwd, q, k, v, cu_seqlens, decay, initial_state, cu_seqlens_cpu=cu_seqlens_cpu,
                   scale=scale, out=out, final_state=final_state, workspace=workspace, check_device=check_device)
    lib = load()
    one, total, H, dk = q.shape
    HV, dv = v.shape[-2:]
    if one != 1:
        raise ValueError("packed sequences need token arrays with B == 1")
    dt, dev = _code(q), _device(q, "q")
    N = cu_seqlens.numel() - 1
    plain = _qkv(q, k, v, 1, total, H, HV, dk, dv, dev)
    _dense(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    fixed = _decay(decay, (1, total, HV), dev)
    if initial_state is not None:
        _dense(initial_state, "initial_state", _F32, (N, HV, dk, dv), dev)
    host = None
    if cu_seqlens_cpu is not None:
        host = cu_seqlens_cpu.to(torch.int32).contiguous()
        if host.is_cuda or host.numel() != N + 1:
            raise ValueError("cu_seqlens_cpu must be a host tensor of cu_seqlens' length")
    if out is None:
        out = _like(v) if plain else _empty((1, total, HV, dv), dtype=q.dtype, device=q.device)
    else:
        plain &= _into(out, "out", q.dtype, (1, total, HV, dv), dev)
    if final_state is None:
        final_state = _empty((N, HV, dk, dv), dtype=_F32, device=q.device)
    else:
        _dense(final_state, "final_state", _F32, (N, HV, dk, dv), dev)
    st = _raw(dev)
    ws, n = _ws("kda_linear_varlen_fwd_workspace", (N, total, H, HV, dk, dv, dt), q, st, workspace, check_device)
    _ok(lib.kda_linear_varlen_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(decay), fixed, cu_seqlens.data_ptr(),
                                  _ptr(host), _ptr(initial_state), out.data_ptr(), final_state.data_ptr(),
                                  None if plain else _strides(q, k, v, out), N, total, H, HV, dk, dv, dt, scale or 0.0,
                                  ws.data_ptr(), n, st), "kda_linear_varlen_fwd", lib)
    if check_device and N:        # an empty batch launches nothing and leaves the header as it is
        _ok(query_device_error(ws), "kda_linear_varlen_fwd (device)", lib)
    return out, final_state


def linear_decode_step(q, k, v, decay, state, *, scale=None, out=None, stream=None):
    """kda_linear_decode_step: one token per sequence; ``state`` [B,HV,dk,dv] fp32 is updated in place.
    q, k [B,1,H,dk] or [B,H,dk]; v [B,1,HV,dv] or [B,HV,dv]; decay [B,1,HV] or [B,HV] fp32, [HV] or None.
    Returns o with v's shape."""
    if stream is not None:
        return _on(stream, linear_decode_step, q, k, v, decay, state, scale=scale, out=out)
    lib = load()
    B, HV, dk, dv = state.shape
    H = q.shape[-2]
    if HV != H:
        _heads(H, HV)
    dt, dtype, dev = _code(q), q.dtype, _device(q, "q")
    if q.dim() == 4:
        qs, vs = (B, 1, H, dk), (B, 1, HV, dv)
    else:
        qs, vs = (B, H, dk), (B, HV, dv)
    plain = _view(q, "q", dtype, qs, dev) & _view(k, "k", dtype, qs, dev) & _view(v, "v", dtype, vs, dev)
    _dense(state, "state", _F32, state.shape, dev)
    fixed = 0
    if decay is not None:
        if decay.dim() == 1:
            fixed = 1
            _dense(decay, "decay", _F32, (HV,), dev)
        else:
            _dense(decay, "decay", _F32, (B, 1, HV) if decay.dim() == 3 else (B, HV), dev)
    if out is None:
        out = _like(v) if plain else _empty(vs, dtype=dtype, device=q.device)
    else:
        plain &= _into(out, "out", dtype, vs, dev)
    s = None
    if not plain:
        s = (ctypes.c_longlong * 8)(*(x for t in (q, k, v, out) for x in (t.stride(0), t.stride(-2))))
    _ok(lib.kda_linear_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(decay), fixed, state.data_ptr(),
                                   out.data_ptr(), s, B, H, HV, dk, dv, dt, scale or 0.0, _raw(dev)),
        "kda_linear_decode_step", lib)
    return out


def linear_chunk_bwd(q, k, v, decay, initial_state, d_o, dfinal_state=None, *, scale=None, workspace=None, stream=None,
                     check_device=False):
    """kda_linear_chunk_bwd: gradients of linear_chunk_fwd given dL/do (dtype of q) and dL/dfinal_state
    (fp32 or None).  Returns a dict dq, dk, dv (q's dtype), ddecay (fp32, decay's shape; absent without a
    decay) and dh0 (fp32; absent without an initial state)."""
    if stream is not None:
        return _on(stream, linear_chunk_bwd, q, k, v, decay, initial_state, d_o, dfinal_state, scale=scale,
                   workspace=workspace, check_device=check_device)
    lib = load()
    B, T, H, dk = q.shape
    HV, dv = v.shape[-2:]
    dt, dtype, dev = _code(q), q.dtype, _device(q, "q")
    plain = _qkv(q, k, v, B, T, H, HV, dk, dv, dev) & _view(d_o, "d_o", dtype, (B, T, HV, dv), dev)
    fixed = _decay(decay, (B, T, HV), dev)
    if initial_state is not None:
        _dense(initial_state, "initial_state", _F32, (B, HV, dk, dv), dev)
    if dfinal_state is not None:
        _dense(dfinal_state, "dfinal_state", _F32, (B, HV, dk, dv), dev)
    if plain:
        dq, dkk, dvv = _like(q), _like(k), _like(v)
    else:
        dq = _empty((B, T, H, dk), dtype=dtype, device=q.device)
        dkk = _empty((B, T, H, dk), dtype=dtype, device=q.device)
        dvv = _empty((B, T, HV, dv), dtype=dtype, device=q.device)
    out = dict(dq=dq, dk=dkk, dv=dvv)
    dg = dh0 = None
    if decay is not None:
        dg = out["ddecay"] = _like(decay)
    if initial_state is not None:
        dh0 = out["dh0"] = _like(initial_state)
    st = _raw(dev)
    ws, n = _ws("kda_linear_chunk_bwd_workspace", (B, T, H, HV, dk, dv, dt), q, st, workspace, check_device)
    _ok(lib.kda_linear_chunk_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(decay), fixed, _ptr(initial_state),
                                 d_o.data_ptr(), _ptr(dfinal_state), dq.data_ptr(), dkk.data_ptr(), dvv.data_ptr(),
                                 _ptr(dg), _ptr(dh0), None if plain else _strides(q, k, v, d_o, dq, dkk, dvv), B, T, H, HV,
                                 dk, dv, dt, scale or 0.0, ws.data_ptr(), n, st), "kda_linear_chunk_bwd", lib)
    if check_device and B:        # an empty batch launches nothing and leaves the header as it is
        _ok(query_device_error(ws), "kda_linear_chunk_bwd (device)", lib)
    return out


def _step(t, lead, what, none):
    """The stride from one place of the first ``lead`` dimensions to the next, in order (``none``: there is one place
    or none).  Dimensions of size 1 are left out: their strides say nothing."""
    step = span = None
    for i in range(lead - 1, -1, -1):
        n, s = t.shape[i], t.stride(i)
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != span:
            raise ValueError(f"the leading dimensions must step evenly (one stride from {what} to {what})")
        span = s * n
    return none if step is None else step


def _token_strides(t):
    """(token, head) strides of [..., H, D] whose leading dimensions step evenly."""
    H, D = t.shape[-2:]
    return _step(t, t.dim() - 2, "token", H * D), t.stride(-2) if H > 1 else D


def _norm_args(x, gate, weight, activation):
    act = 0 if gate is None else _ACT.get(activation)
    if act is None:
        raise ValueError("a gate's activation must be 'silu' or 'sigmoid'")
    if x.dim() < 2:
        raise ValueError("x must be [..., H, D]")
    H, D = x.shape[-2:]
    dt, dev = _code(x, "x"), _device(x, "x")
    _dense(weight, "weight", _F32, (D,), dev)
    plain = _view(x, "x", x.dtype, x.shape, dev)
    if gate is not None:
        plain &= _view(gate, "gate", x.dtype, x.shape, dev)
    return act, dt, H, D, x.numel() // max(1, H * D), plain, dev


def gated_norm_fwd(x, gate, weight, *, eps=1e-6, activation="silu", out=None, stream=None):
    """kda_gated_norm_fwd: y = x (mean(x^2) + eps)^(-1/2) weight act(gate) over the last dimension.
    x, gate [..., H, D] (gate None: no gate, whatever the activation), weight [D] fp32, activation "silu" or "sigmoid"."""
    if stream is not None:
        return _on(stream, gated_norm_fwd, x, gate, weight, eps=eps, activation=activation, out=out)
    lib = load()
    act, dt, H, D, N, plain, dev = _norm_args(x, gate, weight, activation)
    if out is None:
        out = _like(x) if plain else _empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        plain &= _into(out, "out", x.dtype, x.shape, dev)
    s = None
    if not plain:
        s = (ctypes.c_longlong * 6)(*_token_strides(x), *_token_strides(gate if gate is not None else x),
                                    *_token_strides(out))
    _ok(lib.kda_gated_norm_fwd(x.data_ptr(), _ptr(gate), weight.data_ptr(), out.data_ptr(), s, N, H, D, dt, act, eps,
                               _raw(dev)), "kda_gated_norm_fwd", lib)
    return out


def gated_norm_bwd(d_y, x, gate, weight, *, eps=1e-6, activation="silu", workspace=None, stream=None):
    """kda_gated_norm_bwd: a dict dx, dgate (x's dtype; dgate absent without a gate) and dw [D] fp32."""
    if stream is not None:
        return _on(stream, gated_norm_bwd, d_y, x, gate, weight, eps=eps, activation=activation, workspace=workspace)
    lib = load()
    act, dt, H, D, N, plain, dev = _norm_args(x, gate, weight, activation)
    plain &= _view(d_y, "d_y", x.dtype, x.shape, dev)
    dx = _like(x) if plain else _empty(x.shape, dtype=x.dtype, device=x.device)
    dw = _like(weight)
    out = dict(dx=dx, dw=dw)
    dg = None
    if gate is not None:
        dg = out["dgate"] = _like(dx)
    st = _raw(dev)
    ws, n = _ws("kda_gated_norm_bwd_workspace", (D,), x, st, workspace)
    s = None
    if not plain:
        s = (ctypes.c_longlong * 10)(*_token_strides(x), *_token_strides(gate if gate is not None else x),
                                     *_token_strides(d_y), H * D, D, H * D, D)
    _ok(lib.kda_gated_norm_bwd(d_y.data_ptr(), x.data_ptr(), _ptr(gate), weight.data_ptr(), dx.data_ptr(), _ptr(dg),
                               dw.data_ptr(), s, N, H, D, dt, act, eps, ws.data_ptr(), n, st),
        "kda_gated_norm_bwd", lib)
    return out


def _rows(t, D):
    """Row stride of [..., D] whose leading dimensions step evenly."""
    return D if t.is_contiguous() else _step(t, t.dim() - 1, "row", D)


def _scale(scale, D, dev):
    if isinstance(scale, torch.Tensor):
        _dense(scale, "scale", _F32, (D,), dev)
        return scale.data_ptr(), 0.0
    return None, float(scale)


def residual_norm_fwd(x, y, weight, *, scale=1.0, eps=1e-6, out=None, out_norm=None, stream=None):
    """kda_residual_norm_fwd: x' = x + scale y and n = x' (mean(x'^2) + eps)^(-1/2) weight over the last
    dimension.  x [..., D] is the residual stream (bf16, or fp32 around bf16 blocks), y [..., D] the
    block's output, weight [D] fp32, scale a number or a [D] fp32 tensor.  Returns (x' in x's dtype, n in
    y's); out may be x."""
    if stream is not None:
        return _on(stream, residual_norm_fwd, x, y, weight, scale=scale, eps=eps, out=out, out_norm=out_norm)
    lib = load()
    shape = x.shape
    D = shape[-1]
    res, dt, dev = _code(x, "x"), _code(y, "y"), _device(x, "x")
    x_dense, y_dense = _view(x, "x", x.dtype, shape, dev), _view(y, "y", y.dtype, shape, dev)
    _dense(weight, "weight", _F32, (D,), dev)
    cv, c = _scale(scale, D, dev)
    if out is None:
        out = _like(x) if x_dense else _empty(shape, dtype=x.dtype, device=x.device)
    else:
        _dense(out, "out", x.dtype, shape, dev)
    if out_norm is None:
        out_norm = _like(y) if y_dense else _empty(shape, dtype=y.dtype, device=x.device)
    else:
        _dense(out_norm, "out_norm", y.dtype, shape, dev)
    _ok(lib.kda_residual_norm_fwd(x.data_ptr(), y.data_ptr(), weight.data_ptr(), cv, c, out.data_ptr(), out_norm.data_ptr(),
                                  _rows(x, D), _rows(y, D), x.numel() // max(1, D), D, res, dt, eps, _raw(dev)),
        "kda_residual_norm_fwd", lib)
    return out, out_norm


def residual_norm_bwd(d_n, d_x, x, weight, y=None, *, scale=1.0, eps=1e-6, workspace=None, stream=None):
    """kda_residual_norm_bwd: gradients of residual_norm_fwd at its output x (= x'), given those of n and
    x' (d_x None: zeros).  Returns a dict dx (x's dtype; the gradient of the incoming residual), dy = scale
    dx (d_n's dtype), dw [D] fp32, and dscale [D] fp32 when y is given."""
    if stream is not None:
        return _on(stream, residual_norm_bwd, d_n, d_x, x, weight, y, scale=scale, eps=eps, workspace=workspace)
    lib = load()
    shape = x.shape
    D = shape[-1]
    res, dt, dev = _code(x, "x"), _code(d_n, "d_n"), _device(x, "x")
    _dense(x, "x", x.dtype, shape, dev)
    _dense(d_n, "d_n", d_n.dtype, shape, dev)
    _dense(weight, "weight", _F32, (D,), dev)
    if d_x is not None:
        _dense(d_x, "d_x", x.dtype, shape, dev)
    cv, c = _scale(scale, D, dev)
    dx, dy, dw = _like(x), _like(d_n), _like(weight)
    out = dict(dx=dx, dy=dy, dw=dw)
    ds = None
    if y is not None:
        _dense(y, "y", d_n.dtype, shape, dev)
        ds = out["dscale"] = _like(weight)
    st = _raw(dev)
    ws, n = _ws("kda_residual_norm_bwd_workspace", (D,), x, st, workspace)
    _ok(lib.kda_residual_norm_bwd(d_n.data_ptr(), _ptr(d_x), x.data_ptr(), _ptr(y), weight.data_ptr(), cv, c, dx.data_ptr(),
                                  dy.data_ptr(), dw.data_ptr(), _ptr(ds), x.numel() // max(1, D), D, res, dt, eps,
                                  ws.data_ptr(), n, st), "kda_residual_norm_bwd", lib)
    return out
