"""Binding of the short convolution, the state space scan and beam search (include/kda.h).

Argument marshalling only, as ``_linear``: outputs and workspaces are torch tensors of the stream the call runs
on, and the tensors of a call are all on the current device.  Token arrays may be views with any strides (the last
dimension contiguous), e.g. slices of one projection's output.
"""
from __future__ import annotations

import ctypes

import torch

from . import _linear
from ._linear import _F32, _code, _dense, _empty, _into, _like, _need, _ok, _on, _ptr, _view  # noqa: F401

_CONV_ACT = {None: 0, "silu": 1}
_I32 = torch.int32


# The calls below cost the GPU a few microseconds where inputs are small, so what they check on the way is a handful of
# comparisons; what fails one goes through _need, which finds the words.  The library, the current device and stream and
# a call's workspace are _linear's.


def _longs(*xs):
    return (ctypes.c_longlong * len(xs))(*xs)


def _packed(x, what="token arrays"):
    if x.shape[0] != 1:
        raise ValueError(f"packed sequences need {what} with B == 1")


def _cu(cu_seqlens, cu_seqlens_cpu, dev):
    """Checks a packed batch's prefix array; (sequences, its host copy as int32 or None)."""
    N = cu_seqlens.numel() - 1
    if N < 0:
        raise ValueError("cu_seqlens must have one entry more than there are sequences")
    _dense(cu_seqlens, "cu_seqlens", _I32, (N + 1,), dev)
    if cu_seqlens_cpu is None:
        return N, None
    host = cu_seqlens_cpu.to(_I32).contiguous()
    if host.is_cuda or host.numel() != N + 1:
        raise ValueError("cu_seqlens_cpu must be a host tensor of cu_seqlens' length")
    return N, host


# ------------------------------------------------------------------------------ short convolution
def _conv_args(x, weight, bias, activation):
    act = _CONV_ACT.get(activation)
    if act is None:
        raise ValueError("a convolution's activation must be 'silu' or None")
    C, K = x.shape[-1], weight.shape[-1]
    dt, dev = _code(x, "x"), _linear._device(x, "x")
    plain = x.is_contiguous() or _view(x, "x", x.dtype, x.shape, dev)
    _dense(weight, "weight", _F32, (C, K), dev)
    if bias is not None:
        _dense(bias, "bias", _F32, (C,), dev)
    return act, dt, dev, plain, C, K


def _conv_call(x, weight, bias, initial_state, activation, out, final_state, cu, cu_cpu):
    lib = _linear.load()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    act, dt, dev, plain, C, K = _conv_args(x, weight, bias, activation)
    B, T = x.shape[:2]
    n, host = B, None
    if cu is not None:
        _packed(x)
        n, host = _cu(cu, cu_cpu, dev)
    window = (n, K - 1, C)
    if initial_state is not None:
        _dense(initial_state, "initial_state", x.dtype, window, dev)
    if out is None:
        out = _like(x) if plain else x.new_empty(x.shape)
    else:
        plain &= _into(out, "out", x.dtype, x.shape, dev)
    if final_state is None:
        final_state = x.new_empty(window) if initial_state is None else _like(initial_state)
    else:
        _dense(final_state, "final_state", x.dtype, window, dev)
    s = None if plain else _longs(x.stride(0), x.stride(1), out.stride(0), out.stride(1))
    a, z = (x.data_ptr(), weight.data_ptr(), _ptr(bias)), (_ptr(initial_state), out.data_ptr(), final_state.data_ptr(), s)
    if cu is None:
        _ok(lib.kda_conv_fwd(*a, *z, B, T, C, K, dt, act, _linear._raw(dev)), "kda_conv_fwd", lib)
    else:
        _ok(lib.kda_conv_varlen_fwd(*a, cu.data_ptr(), _ptr(host), *z, n, T, C, K, dt, act, _linear._raw(dev)), "kda_conv_varlen_fwd", lib)
    return out, final_state


def conv_fwd(x, weight, bias=None, initial_state=None, *, activation="silu", out=None, final_state=None, stream=None):
    """kda_conv_fwd: the short causal convolution, y_t = act(bias + sum_j weight[:, j] x_{t-K+1+j}) per channel.

    x [B,T,C]; weight [C,K] fp32, K in {2, 3, 4}; bias [C] fp32 or None; initial_state [B,K-1,C] in x's dtype, the last
    K - 1 tokens before x, or None (zeros); activation "silu" or None.  Returns (y [B,T,C], the next window [B,K-1,C])."""
    if stream is not None:
        return _on(stream, conv_fwd, x, weight, bias, initial_state, activation=activation, out=out, final_state=final_state)
    return _conv_call(x, weight, bias, initial_state, activation, out, final_state, None, None)


def conv_varlen_fwd(x, weight, cu_seqlens, bias=None, initial_state=None, *, cu_seqlens_cpu=None, activation="silu",
                    out=None, final_state=None, stream=None):
    """kda_conv_varlen_fwd: packed sequences [1,total,C] split by cu_seqlens [N+1] (int32, device); cu_seqlens_cpu, its
    host copy where there is one, is checked.  Returns (y [1,total,C], the windows [N,K-1,C])."""
    if stream is not None:
        return _on(stream, conv_varlen_fwd, x, weight, cu_seqlens, bias, initial_state, cu_seqlens_cpu=cu_seqlens_cpu,
                   activation=activation, out=out, final_state=final_state)
    return _conv_call(x, weight, bias, initial_state, activation, out, final_state, cu_seqlens, cu_seqlens_cpu)


def conv_decode_step(x, weight, state, bias=None, *, activation="silu", out=None, stream=None):
    """kda_conv_decode_step: one token per request; ``state`` [B,K-1,C], the window in x's dtype, moves on by one token
    in place.  x [B,C] or [B,1,C].  Returns y with x's shape."""
    if stream is not None:
        return _on(stream, conv_decode_step, x, weight, state, bias, activation=activation, out=out)
    lib = _linear.load()
    if x.dim() not in (2, 3) or (x.dim() == 3 and x.shape[1] != 1):
        raise ValueError("x must be [B, C] or [B, 1, C]")
    act, dt, dev, plain, C, K = _conv_args(x, weight, bias, activation)
    B = x.shape[0]
    _dense(state, "state", x.dtype, (B, K - 1, C), dev)
    if out is None:
        out = _like(x) if plain else x.new_empty(x.shape)
    else:
        plain &= _into(out, "out", x.dtype, x.shape, dev)
    s = None if plain else _longs(x.stride(0), out.stride(0))
    _ok(lib.kda_conv_decode_step(x.data_ptr(), weight.data_ptr(), _ptr(bias), state.data_ptr(), out.data_ptr(), s, B, C, K, dt,
                                 act, _linear._raw(dev)), "kda_conv_decode_step", lib)
    return out


def conv_bwd(d_y, x, weight, bias=None, initial_state=None, dfinal_state=None, *, cu_seqlens=None, activation="silu",
             workspace=None, stream=None):
    """kda_conv_bwd: gradients of conv_fwd (of conv_varlen_fwd with cu_seqlens) given dL/dy and dL/d(the next window) (None:
    zeros).  Returns a dict dx (x's dtype), dw [C,K] fp32, dbias [C] fp32 (absent without a bias) and dstate (the gradient
    of the initial window; absent without one)."""
    if stream is not None:
        return _on(stream, conv_bwd, d_y, x, weight, bias, initial_state, dfinal_state, cu_seqlens=cu_seqlens,
                   activation=activation, workspace=workspace)
    lib = _linear.load()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    act, dt, dev, plain, C, K = _conv_args(x, weight, bias, activation)
    B, T = x.shape[:2]
    n = B
    if cu_seqlens is not None:
        _packed(x)
        n, _ = _cu(cu_seqlens, None, dev)
    plain &= _view(d_y, "d_y", x.dtype, x.shape, dev)
    window = (n, K - 1, C)
    if initial_state is not None:
        _dense(initial_state, "initial_state", x.dtype, window, dev)
    if dfinal_state is not None:
        _dense(dfinal_state, "dfinal_state", x.dtype, window, dev)
    dx, dw = _like(x) if plain else x.new_empty(x.shape), _like(weight)
    out = dict(dx=dx, dw=dw)
    db = dh = None
    if bias is not None:
        db = out["dbias"] = _like(bias)
    if initial_state is not None:
        dh = out["dstate"] = _like(initial_state)
    st = _linear._raw(dev)
    ws, size = _linear._ws("kda_conv_bwd_workspace", (C, K), x, st, workspace)
    s = None if plain else _longs(x.stride(0), x.stride(1), d_y.stride(0), d_y.stride(1), T * C, C)
    _ok(lib.kda_conv_bwd(d_y.data_ptr(), x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state), _ptr(dfinal_state),
                         dx.data_ptr(), dw.data_ptr(), _ptr(db), _ptr(dh), _ptr(cu_seqlens), s, n, T, C, K, dt, act,
                         ws.data_ptr(), size, st), "kda_conv_bwd", lib)
    return out


# ------------------------------------------------------------------------------ state space scan
def _heads(t, name, dtype, lead, dev, N):
    """[..., G, N] (or [..., N], one group) as (G, whether it is contiguous)."""
    if t.dim() == len(lead) + 1:
        return 1, _view(t, name, dtype, (*lead, N), dev)
    if t.dim() != len(lead) + 2:
        raise ValueError(f"{name} must have the shape [..., G, N] or [..., N]")
    G = t.shape[-2]
    return G, _view(t, name, dtype, (*lead, G, N), dev)


def _scan_args(x, dt, A, B, C, skip, gate, dt_bias, dev):
    """Checks what every scan call has; (D, G, N, whether all is contiguous)."""
    shape, dtype = x.shape, x.dtype
    D = shape[-1]
    if A.dim() != 2:
        raise ValueError("A must be [D, N]")
    N = A.shape[1]
    heads = B.shape
    G = heads[-2] if len(heads) == len(shape) + 1 else 1
    plain = (x.is_contiguous() and dt.is_contiguous() and B.is_contiguous() and C.is_contiguous() and dt.dtype is dtype and
             B.dtype is dtype and C.dtype is dtype and dt.get_device() == dev and B.get_device() == dev and C.get_device() == dev and
             dt.shape == shape and C.shape == heads and heads[-1] == N and heads[:-1] == (shape[:-1] if G == 1 and len(heads) == len(shape)
                                                                                          else (*shape[:-1], G)))
    if not plain:
        plain = _view(x, "x", dtype, shape, dev) & _view(dt, "dt", dtype, shape, dev)
        G, p = _heads(B, "B", dtype, shape[:-1], dev, N)
        plain &= p
        G2, p = _heads(C, "C", dtype, shape[:-1], dev, N)
        plain &= p
        if G2 != G or B.dim() != C.dim():
            raise ValueError(f"C has shape {tuple(C.shape)}, expected B's {tuple(B.shape)}")
    _dense(A, "A", _F32, (D, N), dev)
    if G == 0 or D % G:
        raise ValueError(f"the channels ({D}) must be a multiple of the groups ({G})")
    if gate is not None:
        plain &= _view(gate, "gate", dtype, shape, dev)
    if skip is not None:
        _dense(skip, "skip", _F32, (D,), dev)
    if dt_bias is not None:
        _dense(dt_bias, "dt_bias", _F32, (D,), dev)
    return D, G, N, plain


def _scan_strides(*ts):
    """(batch, token, group) strides of [B,T,D] and [B,T,G,N] arrays (None: the first one's)."""
    out = []
    for t in ts:
        t = ts[0] if t is None else t
        out += [t.stride(0), t.stride(1), t.stride(2) if t.dim() == 4 else 0]
    return _longs(*out)


def _scan_call(x, dt, A, B, C, initial_state, skip, gate, dt_bias, softplus, out, final_state, workspace, check, cu, cu_cpu):
    lib = _linear.load()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    code, dev = _code(x, "x"), _linear._device(x, "x")
    D, G, N, plain = _scan_args(x, dt, A, B, C, skip, gate, dt_bias, dev)
    n, T, host = x.shape[0], x.shape[1], None
    if cu is not None:
        _packed(x)
        n, host = _cu(cu, cu_cpu, dev)
    if initial_state is not None:
        _dense(initial_state, "initial_state", _F32, (n, D, N), dev)
    if out is None:
        out = _like(x) if plain else x.new_empty(x.shape)
    else:
        plain &= _into(out, "out", x.dtype, x.shape, dev)
    if final_state is None:
        final_state = A.new_empty((n, D, N)) if initial_state is None else _like(initial_state)
    else:
        _dense(final_state, "final_state", _F32, (n, D, N), dev)
    st = _linear._raw(dev)
    s = None if plain else _scan_strides(x, dt, B, C, gate, out)
    a = (x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(skip), _ptr(gate), _ptr(dt_bias))
    if cu is None:
        ws, size = _linear._ws("kda_ssm_chunk_fwd_workspace", (n, T, D, G, N, code), x, st, workspace, check)
        _ok(lib.kda_ssm_chunk_fwd(*a, _ptr(initial_state), out.data_ptr(), final_state.data_ptr(), s, n, T, D, G, N, code,
                                  int(softplus), ws.data_ptr(), size, st), "kda_ssm_chunk_fwd", lib)
    else:
        ws, size = _linear._ws("kda_ssm_varlen_fwd_workspace", (n, T, D, G, N, code), x, st, workspace, check)
        _ok(lib.kda_ssm_varlen_fwd(*a, cu.data_ptr(), _ptr(host), _ptr(initial_state), out.data_ptr(), final_state.data_ptr(), s,
                                   n, T, D, G, N, code, int(softplus), ws.data_ptr(), size, st), "kda_ssm_varlen_fwd", lib)
    if check and n:        # an empty batch launches nothing and leaves the header as it is
        _ok(_linear.query_device_error(ws), "state space scan (device)", lib)
    return out, final_state


def ssm_chunk_fwd(x, dt, A, B, C, initial_state=None, *, skip=None, gate=None, dt_bias=None, softplus=True, out=None,
                  final_state=None, workspace=None, stream=None, check_device=False):
    """kda_ssm_chunk_fwd: the state space scan, dt_t = softplus(dt_t + dt_bias), h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,
    y_t = (C_t . h_t + skip x_t) silu(gate_t), with N states for each of D channels.

    x, dt, gate [B,T,D]; B, C [B,T,G,N] or [B,T,N] (channel d reads group d // (D // G)), N in {8, 16, 32, 64}; A [D,N] (finite,
    negative for a decay), skip [D], dt_bias [D] fp32; initial_state [B,D,N] fp32; skip, gate, dt_bias, initial_state may
    be None; softplus=False uses dt + dt_bias as it is.  Returns (y [B,T,D], final_state [B,D,N] fp32).  check_device as in
    chunk_fwd."""
    if stream is not None:
        return _on(stream, ssm_chunk_fwd, x, dt, A, B, C, initial_state, skip=skip, gate=gate, dt_bias=dt_bias,
                   softplus=softplus, out=out, final_state=final_state, workspace=workspace, check_device=check_device)
    return _scan_call(x, dt, A, B, C, initial_state, skip, gate, dt_bias, softplus, out, final_state, workspace, check_device,
                      None, None)


def ssm_varlen_fwd(x, dt, A, B, C, cu_seqlens, initial_state=None, *, cu_seqlens_cpu=None, skip=None, gate=None, dt_bias=None,
                   softplus=True, out=None, final_state=None, workspace=None, stream=None, check_device=False):
    """kda_ssm_varlen_fwd: packed sequences [1,total,..] split by cu_seqlens [N+1] (int32, device); cu_seqlens_cpu, its host
    copy where there is one, is checked and tells how to split the work.  Returns (y [1,total,D], final_state [N,D,N])."""
    if stream is not None:
        return _on(stream, ssm_varlen_fwd, x, dt, A, B, C, cu_seqlens, initial_state, cu_seqlens_cpu=cu_seqlens_cpu, skip=skip,
                   gate=gate, dt_bias=dt_bias, softplus=softplus, out=out, final_state=final_state, workspace=workspace,
                   check_device=check_device)
    return _scan_call(x, dt, A, B, C, initial_state, skip, gate, dt_bias, softplus, out, final_state, workspace, check_device,
                      cu_seqlens, cu_seqlens_cpu)


def ssm_decode_step(x, dt, A, B, C, state, *, skip=None, gate=None, dt_bias=None, softplus=True, out=None, stream=None):
    """kda_ssm_decode_step: one token per request; ``state`` [B,D,N] fp32 is updated in place.  x, dt, gate [B,D] (or
    [B,1,D]), B, C [B,G,N] or [B,N] ([B,1,G,N]).  Returns y with x's shape."""
    if stream is not None:
        return _on(stream, ssm_decode_step, x, dt, A, B, C, state, skip=skip, gate=gate, dt_bias=dt_bias, softplus=softplus,
                   out=out)
    lib = _linear.load()
    if x.dim() not in (2, 3) or (x.dim() == 3 and x.shape[1] != 1):
        raise ValueError("x must be [B, D] or [B, 1, D]")
    code, dev = _code(x, "x"), _linear._device(x, "x")
    D, G, N, plain = _scan_args(x, dt, A, B, C, skip, gate, dt_bias, dev)
    nb = x.shape[0]
    _dense(state, "state", _F32, (nb, D, N), dev)
    if out is None:
        out = _like(x) if plain else x.new_empty(x.shape)
    else:
        plain &= _into(out, "out", x.dtype, x.shape, dev)
    s = None
    if not plain:
        group = lambda t: t.stride(-2) if G > 1 else N  # noqa: E731
        s = _longs(x.stride(0), dt.stride(0), B.stride(0), group(B), C.stride(0), group(C),
                   (x if gate is None else gate).stride(0), out.stride(0))
    _ok(lib.kda_ssm_decode_step(x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(skip), _ptr(gate),
                                _ptr(dt_bias), state.data_ptr(), out.data_ptr(), s, nb, D, G, N, code, int(softplus), _linear._raw(dev)),
        "kda_ssm_decode_step", lib)
    return out


def ssm_chunk_bwd(d_y, x, dt, A, B, C, initial_state=None, dfinal_state=None, *, skip=None, gate=None, dt_bias=None,
                  softplus=True, cu_seqlens=None, workspace=None, stream=None):
    """kda_ssm_chunk_bwd: gradients of ssm_chunk_fwd (of ssm_varlen_fwd with cu_seqlens) given dL/dy (x's dtype) and
    dL/dfinal_state (fp32 or None).  Returns a dict dx, ddt, dB, dC, dgate (x's dtype), dA, dskip, ddt_bias, dh0 (fp32);
    dskip, dgate, ddt_bias and dh0 are absent where there is no such input."""
    if stream is not None:
        return _on(stream, ssm_chunk_bwd, d_y, x, dt, A, B, C, initial_state, dfinal_state, skip=skip, gate=gate,
                   dt_bias=dt_bias, softplus=softplus, cu_seqlens=cu_seqlens, workspace=workspace)
    lib = _linear.load()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    code, dev = _code(x, "x"), _linear._device(x, "x")
    D, G, N, plain = _scan_args(x, dt, A, B, C, skip, gate, dt_bias, dev)
    plain &= _view(d_y, "d_y", x.dtype, x.shape, dev)
    n, T = x.shape[:2]
    if cu_seqlens is not None:
        _packed(x)
        n, _ = _cu(cu_seqlens, None, dev)
    if initial_state is not None:
        _dense(initial_state, "initial_state", _F32, (n, D, N), dev)
    if dfinal_state is not None:
        _dense(dfinal_state, "dfinal_state", _F32, (n, D, N), dev)
    rows = _like if plain else lambda t: t.new_empty(t.shape)
    dx, dB = rows(x), rows(B)
    out = dict(dx=dx, ddt=_like(dx), dA=_like(A), dB=dB, dC=_like(dB))
    if skip is not None:
        out["dskip"] = _like(skip)
    if gate is not None:
        out["dgate"] = _like(dx)
    if dt_bias is not None:
        out["ddt_bias"] = _like(dt_bias)
    if initial_state is not None:
        out["dh0"] = _like(initial_state)
    st = _linear._raw(dev)
    ws, size = _linear._ws("kda_ssm_chunk_bwd_workspace", (n, T, int(cu_seqlens is not None), D, G, N, code), x, st, workspace)
    g = lambda name: _ptr(out.get(name))  # noqa: E731
    _ok(lib.kda_ssm_chunk_bwd(d_y.data_ptr(), x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(skip),
                              _ptr(gate), _ptr(dt_bias), _ptr(initial_state), _ptr(dfinal_state), g("dx"), g("ddt"), g("dA"),
                              g("dB"), g("dC"), g("dskip"), g("dgate"), g("ddt_bias"), g("dh0"), _ptr(cu_seqlens),
                              None if plain else _scan_strides(x, dt, B, C, gate, d_y), n, T, D, G, N, code, int(softplus),
                              ws.data_ptr(), size, st), "kda_ssm_chunk_bwd", lib)
    return out


# ------------------------------------------------------------------------------ beam search
def beam_select(logits, scores, k=None, *, finished=None, eos=None, out=None, workspace=None, stream=None):
    """kda_beam_select: the k best of all total[w, v] = scores[w] + log_softmax(logits[w])[v], in order, equal totals by
    the lowest w V + v.

    logits [B,W,V] (a view's rows may lie apart), scores [B,W] fp32, k <= 32 (None: W); finished [B,W] bool or None: such a
    beam has the one candidate ``eos``, with its score as it is.  out: a tuple of the three outputs.  Returns (scores [B,k]
    fp32, parents [B,k] int32, tokens [B,k] int32)."""
    if stream is not None:
        return _on(stream, beam_select, logits, scores, k, finished=finished, eos=eos, out=out, workspace=workspace)
    lib = _linear.load()
    if logits.dim() != 3:
        raise ValueError("logits must be [B, W, V]")
    B, W, V = logits.shape
    code, dev = _code(logits, "logits"), _linear._device(logits, "logits")
    plain = logits.is_contiguous() or _view(logits, "logits", logits.dtype, logits.shape, dev)
    _dense(scores, "scores", _F32, (B, W), dev)
    if finished is not None:
        _dense(finished, "finished", torch.bool, (B, W), dev)
        if eos is None:
            raise ValueError("finished beams need the token they go on with: eos")
    k = W if k is None else k
    if out is None:
        tokens = _empty((B, k), dtype=_I32, device=logits.device)
        out = (_like(scores) if k == W else scores.new_empty((B, k)), _like(tokens), tokens)
    else:
        for t, name, dtype in zip(out, ("out scores", "out parents", "out tokens"), (_F32, _I32, _I32)):
            _dense(t, name, dtype, (B, k), dev)
    st = _linear._raw(dev)
    ws, size = _linear._ws("kda_beam_select_workspace", (B, W, V, code), logits, st, workspace)
    _ok(lib.kda_beam_select(logits.data_ptr(), None if plain else _longs(logits.stride(0), logits.stride(1)), scores.data_ptr(),
                            _ptr(finished), eos or 0, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), B, W, V, k, code,
                            ws.data_ptr(), size, st), "kda_beam_select", lib)
    return tuple(out)


def beam_reorder(states, parents, *, stream=None):
    """kda_beam_reorder: the recurrent memories follow the beams, in place: row (b, w) becomes row (b, parents[b, w]).

    states: a tensor or a list of them, each contiguous, of any type, [B * W, ...] or [B, W, ...]; parents [B,W] int32,
    W <= 32 (a parent outside 0 .. W - 1 leaves its beam as it is).  Returns states."""
    if stream is not None:
        return _on(stream, beam_reorder, states, parents)
    lib = _linear.load()
    if parents.dim() != 2:
        raise ValueError("parents must be [B, W]")
    B, W = parents.shape
    dev = _linear._device(parents, "parents")
    _dense(parents, "parents", _I32, (B, W), dev)
    arrays = [states] if isinstance(states, torch.Tensor) else list(states)
    n, rows, ptrs, sizes = len(arrays), B * W, [], []
    for i, t in enumerate(arrays):
        if not (t.is_contiguous() and t.get_device() == dev):
            _need(t, f"states[{i}]", t.dtype, t.shape, dev)
        shape = t.shape
        if not (shape and (shape[0] == rows or tuple(shape[:2]) == (B, W))):
            raise ValueError(f"states[{i}] has shape {tuple(shape)}, expected [{rows}, ...] or [{B}, {W}, ...]")
        ptrs.append(t.data_ptr())
        sizes.append(t.nbytes // rows if rows else 0)
    ptrs, sizes = (ctypes.c_void_p * n)(*ptrs), (ctypes.c_longlong * n)(*sizes)
    _ok(lib.kda_beam_reorder(ptrs, sizes, n, parents.data_ptr(), B, W, _linear._raw(dev)), "kda_beam_reorder", lib)
    return states
