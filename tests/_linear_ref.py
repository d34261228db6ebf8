"""Plain fp64 numpy statements of linear attention with a decay per head, its gradients and the
block norms, token by token (test infrastructure; shares no code with the library).

Tolerances, derived from the number formats before any run:
  U8 = 2^-9, a bound on bf16 rounding errors over an array (each is at most 2^-8 of its value and
  2^-8 / sqrt(3) of the value's power of two in the mean square, 1.7e-3 normwise); U16 = 2^-17, the
  same of a value kept as a sum of two bf16s.
  fp32 arithmetic: sums of n rounded terms err like sqrt(n) 2^-24 on these random inputs; with at
  most ~600 tokens and 128 channels that is below 2e-5 normwise with a margin of ten.
  bf16 outputs of fp32 arithmetic round once: U8 (plus the above).
  Chunked bf16 forward: the score matrix, the memory operand and the output each round once to
  bf16: 3 U8 normwise.  Chunked bf16 gradients round one operand more: 4 U8.
  Chunked fp32 results of bf16 inputs (memories, the decay's gradient) use sums of two bf16s for
  every scaled operand: one such rounding per product for the memories (2 U16), at most three
  factors in the decay's gradient (each term a product of two of them and a weight): 6 U16.
"""
import numpy as np

U8 = 2.0 ** -9
U16 = 2.0 ** -17
F32 = 2e-5
BF16_O = 3 * U8
BF16_GRAD = 4 * U8
TC_STATE = 2 * U16
TC_DDECAY = 6 * U16


def frob(got, ref):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref))
    den = np.linalg.norm(ref)
    return float(np.linalg.norm(got - ref) / den) if den else float(np.linalg.norm(got))


def spread(x, m):
    return np.repeat(x, m, axis=2)


def forward(q, k, v, decay=None, h0=None, scale=None):
    """q, k [B,T,H,dk], v [B,T,HV,dv], decay [B,T,HV] or [HV] or None.  Returns o, h."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, T, H, dk = q.shape
    HV, dv = v.shape[2:]
    q, k = spread(q, HV // H), spread(k, HV // H)
    g = np.zeros((B, T, HV)) if decay is None else np.broadcast_to(np.asarray(decay, np.float64), (B, T, HV))
    s = dk ** -0.5 if scale is None else scale
    h = np.zeros((B, HV, dk, dv)) if h0 is None else np.array(h0, np.float64)
    o = np.zeros((B, T, HV, dv))
    for t in range(T):
        h = np.exp(g[:, t])[..., None, None] * h + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = s * np.einsum("bhi,bhij->bhj", q[:, t], h)
    return o, h


def backward(q, k, v, decay, h0, d_o, dhT=None, scale=None):
    """Gradients of sum(o . d_o) + sum(h_T . dhT): dq, dk, dv, ddecay [B,T,HV], dh0."""
    q, k, v, d_o = (np.asarray(x, np.float64) for x in (q, k, v, d_o))
    B, T, H, dk = q.shape
    HV, dv = v.shape[2:]
    m = HV // H
    qs, ks = spread(q, m), spread(k, m)
    g = np.zeros((B, T, HV)) if decay is None else np.broadcast_to(np.asarray(decay, np.float64), (B, T, HV))
    s = dk ** -0.5 if scale is None else scale
    h = np.zeros((B, HV, dk, dv)) if h0 is None else np.array(h0, np.float64)
    kept, dq = [h], np.zeros((B, T, HV, dk))
    for t in range(T):
        h = np.exp(g[:, t])[..., None, None] * h + ks[:, t, :, :, None] * v[:, t, :, None, :]
        kept.append(h)
        dq[:, t] = s * np.einsum("bhij,bhj->bhi", h, d_o[:, t])
    D = np.zeros((B, HV, dk, dv)) if dhT is None else np.array(dhT, np.float64)
    dkk, dvv, dg = np.zeros((B, T, HV, dk)), np.zeros((B, T, HV, dv)), np.zeros((B, T, HV))
    for t in range(T - 1, -1, -1):
        D = D + s * qs[:, t, :, :, None] * d_o[:, t, :, None, :]
        dkk[:, t] = np.einsum("bhij,bhj->bhi", D, v[:, t])
        dvv[:, t] = np.einsum("bhij,bhi->bhj", D, ks[:, t])
        D = np.exp(g[:, t])[..., None, None] * D
        dg[:, t] = np.einsum("bhij,bhij->bh", kept[t], D)
    fold = lambda x: x.reshape(B, T, H, m, dk).sum(3)  # noqa: E731
    return dict(dq=fold(dq), dk=fold(dkk), dv=dvv, ddecay=dg, dh0=D)


def _act(a, kind):
    s = 1.0 / (1.0 + np.exp(-a))
    return (a * s, s * (1 + a * (1 - s))) if kind == "silu" else (s, s * (1 - s))


def gated_norm(x, gate, w, eps, act):
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    a = _act(np.asarray(gate, np.float64), act)[0] if gate is not None else 1.0
    return x * r * np.asarray(w, np.float64) * a


def gated_norm_grad(dy, x, gate, w, eps, act):
    dy, x, w = (np.asarray(z, np.float64) for z in (dy, x, w))
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    a, da = _act(np.asarray(gate, np.float64), act) if gate is not None else (np.ones_like(x), np.zeros_like(x))
    xn, t = x * r, dy * a * w
    dx = r * (t - xn * (t * xn).mean(-1, keepdims=True))
    return dict(dx=dx, dgate=dy * xn * w * da, dw=(dy * a * xn).reshape(-1, x.shape[-1]).sum(0))


def residual_norm(x, y, w, c, eps):
    z = np.asarray(x, np.float64) + np.asarray(c, np.float64) * np.asarray(y, np.float64)
    return z, z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def residual_norm_grad(dn, dxo, z, y, w, c, eps):
    dn, z, w = (np.asarray(t, np.float64) for t in (dn, z, w))
    r = 1.0 / np.sqrt((z * z).mean(-1, keepdims=True) + eps)
    xn, t = z * r, dn * w
    dx = (0.0 if dxo is None else np.asarray(dxo, np.float64)) + r * (t - xn * (t * xn).mean(-1, keepdims=True))
    D = z.shape[-1]
    out = dict(dx=dx, dy=np.asarray(c, np.float64) * dx, dw=(dn * xn).reshape(-1, D).sum(0))
    if y is not None:
        out["dscale"] = (dx * np.asarray(y, np.float64)).reshape(-1, D).sum(0)
    return out
