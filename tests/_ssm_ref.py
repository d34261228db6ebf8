"""Plain fp64 numpy statements of the short convolution, the state space scan, their gradients and beam search's
selection (test infrastructure; shares no code with the library).

Tolerances, derived from the number formats before any run, relative in the Frobenius norm:
  U8 = 2^-8 bounds the rounding of an array to bf16: each value is off by at most half a step, 2^-8 of itself, and so
  is the array (a few values may all be off by that much; only large arrays come near the mean, 1.7e-3).
  conv: sums of up to 8 fp32 products and a sigmoid of approximate exp2 and reciprocal (2^-22 each): 1e-6; sums over
  rows (dw, dbias) of up to a few thousand fp32 terms err like sqrt(n) 2^-24 on random inputs: 1e-5 holds them.
  scan: a factor exp(dt A) errs by at most 2^-22.5 (approximate exp2) and 2^-24 of its exponent (which is below 2 where
  the factor counts): 3e-7.  A memory carries at most the product of T factors: T 3e-7.  dt itself (softplus) errs by 5e-7.
  scan(T) = 2e-6 + 3e-7 T; gradients run through two such chains: twice that.
  Scores of the selection are rounded once to fp32, 2^-24 of their size, from a log-sum-exp of fp32 terms: 1e-6.
"""
import numpy as np

U8 = 2.0 ** -8
CONV, CONV_SUMS = 1e-6, 1e-5


def scan_tol(T):
    return 2e-6 + 3e-7 * T


def frob(got, ref):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref))
    den = np.linalg.norm(ref)
    return float(np.linalg.norm(got - ref) / den) if den else float(np.linalg.norm(got))


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


def silu(x):
    s = 1.0 / (1.0 + np.exp(-x))
    return x * s, s * (1 + x * (1 - s))


# ------------------------------------------------------------------------------ convolution
def conv(x, w, bias=None, h0=None, act="silu"):
    """One sequence batch [B,T,C]: (y, next window)."""
    x, w, bias, h0 = _f(x), _f(w), _f(bias), _f(h0)
    B, T, C = x.shape
    K = w.shape[1]
    rows = np.concatenate([np.zeros((B, K - 1, C)) if h0 is None else h0, x], 1)
    p = np.zeros((B, T, C)) + (0.0 if bias is None else bias)
    for t in range(T):
        for j in range(K):
            p[:, t] += w[:, j] * rows[:, t + j]
    return (silu(p)[0] if act else p), rows[:, T:]


def conv_grad(dy, x, w, bias=None, h0=None, dhT=None, act="silu"):
    dy, x, w, bias, h0, dhT = (_f(t) for t in (dy, x, w, bias, h0, dhT))
    B, T, C = x.shape
    K = w.shape[1]
    rows = np.concatenate([np.zeros((B, K - 1, C)) if h0 is None else h0, x], 1)
    p = conv(x, w, bias, h0, None)[0]
    q = dy * (silu(p)[1] if act else 1.0)
    dr = np.zeros_like(rows)
    if dhT is not None:
        dr[:, T:] += dhT
    dw = np.zeros_like(w)
    for t in range(T):
        for j in range(K):
            dr[:, t + j] += q[:, t] * w[:, j]
            dw[:, j] += (q[:, t] * rows[:, t + j]).sum(0)
    return dict(dx=dr[:, K - 1:], dw=dw, dbias=q.sum((0, 1)), dstate=dr[:, :K - 1])


# ------------------------------------------------------------------------------ scan
def softplus(x):
    return np.logaddexp(x, 0.0)


def _spread(t, D):
    """[B,T,G,N] to channels [B,T,D,N]."""
    return np.repeat(t, D // t.shape[2], axis=2)


def scan(x, dt, A, Bm, Cm, h0=None, skip=None, gate=None, dt_bias=None, use_softplus=True, grad=None):
    """x, dt, gate [B,T,D], Bm, Cm [B,T,G,N]: (y, h), or with grad = (dy, dhT) the dict of gradients."""
    x, dt, A, Bm, Cm, h0, skip, gate, dt_bias = (_f(t) for t in (x, dt, A, Bm, Cm, h0, skip, gate, dt_bias))
    B, T, D = x.shape
    G, N = Bm.shape[2:]
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    step = softplus(raw) if use_softplus else raw
    Bs, Cs = _spread(Bm, D), _spread(Cm, D)
    sk = np.zeros(D) if skip is None else skip
    h = np.zeros((B, D, N)) if h0 is None else h0.copy()
    r, kept = np.zeros((B, T, D)), []
    for t in range(T):
        kept.append(h)
        h = np.exp(step[:, t, :, None] * A) * h + (step[:, t] * x[:, t])[..., None] * Bs[:, t]
        r[:, t] = (h * Cs[:, t]).sum(-1) + sk * x[:, t]
    act, dact = silu(gate) if gate is not None else (1.0, None)
    if grad is None:
        return r * act, h
    dy, dhT = _f(grad[0]), _f(grad[1])
    kept.append(h)
    p = dy * act
    g = np.zeros((B, D, N)) if dhT is None else dhT.copy()
    out = dict(dx=sk * p, ddt=np.zeros_like(x), dA=np.zeros_like(A), dB=np.zeros_like(Bm), dC=np.zeros_like(Cm),
               dskip=(p * x).sum((0, 1)))
    if gate is not None:
        out["dgate"] = dy * r * dact
    fold = lambda t: t.reshape(B, G, D // G, N).sum(2)  # noqa: E731
    for t in range(T - 1, -1, -1):
        a = np.exp(step[:, t, :, None] * A)
        g = g + p[:, t, :, None] * Cs[:, t]
        out["dC"][:, t] = fold(p[:, t, :, None] * kept[t + 1])
        out["dB"][:, t] = fold((step[:, t] * x[:, t])[..., None] * g)
        s = (g * Bs[:, t]).sum(-1)
        g = a * g
        e = g * kept[t]
        out["dx"][:, t] += step[:, t] * s
        out["ddt"][:, t] = (x[:, t] * s + (e * A).sum(-1)) * (1 / (1 + np.exp(-raw[:, t])) if use_softplus else 1.0)
        out["dA"] += (e * step[:, t, :, None]).sum(0)
    out["ddt_bias"], out["dh0"] = out["ddt"].sum((0, 1)), g
    return out


# ------------------------------------------------------------------------------ packed sequences
def packed(cu, call, rows, seqs):
    """Applies call(rows of one sequence [1,T,..], its part of seqs [1,..]) to every sequence; lists of what it returns."""
    out = []
    for n in range(len(cu) - 1):
        a, b = cu[n], cu[n + 1]
        out.append(call(*[None if t is None else t[:, a:b] for t in rows], *[None if t is None else t[n:n + 1] for t in seqs]))
    return out


# ------------------------------------------------------------------------------ beam search
def select(logits, scores, k, finished=None, eos=None):
    """The k best totals of [B,W,V] by sorting all of them: (scores fp64, parents, tokens)."""
    x, s = _f(logits), _f(scores)
    B, W, V = x.shape
    out = [np.zeros((B, k)), np.zeros((B, k), np.int64), np.zeros((B, k), np.int64)]
    for b in range(B):
        total = np.full((W, V), -np.inf)
        for w in range(W):
            if finished is not None and finished[b, w]:
                total[w, eos] = s[b, w]
                continue
            m = x[b, w].max()
            if not np.isfinite(m) or np.isnan(x[b, w]).any() or np.isnan(s[b, w]):
                continue
            total[w] = s[b, w] + x[b, w] - (m + np.log(np.exp(x[b, w] - m).sum()))
        flat = total.reshape(-1)
        at = np.lexsort((np.arange(flat.size), -flat))[:k]
        out[0][b], out[1][b], out[2][b] = flat[at], at // V, at % V
    return out
