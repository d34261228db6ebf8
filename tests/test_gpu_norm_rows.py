"""Gradients of the block norms element by element, in rows that one element dominates and in rows at the ends of the
range: norms over an array cannot see single small elements.

dx = r (t - xn mean(t xn)) cancels at an element that carries the row: there it is r (t u - xn w) with u = r^2 (eps + the
other elements' mean square) and w = r times the others' mean of t x.  Every element is held to ref.F32 of the two terms
that its value is the difference of, these two at a dominating element, t and xn mean(t xn) elsewhere: sums of up to
16,384 products of random signs err by some sqrt(2^14) 2^-24 = 8e-6 of their norm at most, and the few operations after
them by 2^-24 each."""
import numpy as np
import pytest

import _linear_ref as ref
from test_gpu_linear import _np, _t

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def kda():
    import delta_rule_linear_gb300 as m
    m.load()
    return m


def _rows(D, large, rows=48, seed=0):
    """Rows of which one element, somewhere, is `large` times the others; a few with two such, and a few plain ones."""
    r = np.random.default_rng(seed)
    x = r.normal(size=(rows, D))
    at = r.integers(0, D, size=rows)
    at[0], at[1] = 0, D - 1
    x[np.arange(rows), at] = large * r.choice([-1.0, 1.0], size=rows)
    if D > 1:
        x[5, (at[5] + 1) % D] = x[5, at[5]]
    x[7] = r.normal(size=D)
    return x.astype(np.float32)


def _bound(x, t):
    """dx in fp64, and the size of the terms it is the difference of."""
    x, t = x.astype(np.float64), t.astype(np.float64)
    ss, dot = (x * x).sum(-1, keepdims=True), (t * x).sum(-1, keepdims=True)
    D = x.shape[-1]
    r = 1 / np.sqrt(ss / D + EPS)
    top = x * x > 0.5 * ss
    one = np.ones_like(x)
    ss1 = np.where(top, ((~top) * x * x).sum(-1, keepdims=True) * one, ss * one)
    dot1 = np.where(top, ((~top) * t * x).sum(-1, keepdims=True) * one, dot * one)
    u = np.where(top, r * r * (EPS + ss1 / D), 1.0)
    w = r * dot1 / D
    size = np.sqrt(((t * x) ** 2 * ~top).sum(-1, keepdims=True)) * r / D        # what a sum's rounding is relative to
    return r * (t * u - x * r * w), r * (np.abs(t) * u + np.abs(x * r) * np.maximum(np.abs(w), size))


LARGE = [30.0, 1e3, 1e5, 1e6]


@pytest.mark.parametrize("large", LARGE)
@pytest.mark.parametrize("D", [1, 2, 32, 64, 77, 128, 250, 256, 512, 1000, 1024])
def test_gated_norm_gradient_at_a_dominating_element(kda, D, large):
    import torch
    x = _rows(D, large).reshape(-1, 3, D)
    r = np.random.default_rng(1)
    dy, w, a = r.normal(size=x.shape), 1 + 0.3 * r.normal(size=D), r.normal(size=x.shape)
    X, DY, W, A = (_t(z, torch.float32) for z in (x, dy, w, a))
    for gate, act in ((None, None), (A, "silu"), (A, "sigmoid")):
        got = kda.gated_norm_bwd(DY, X, gate, W, eps=EPS, activation=act)
        f = ref._act(_np(A), act)[0] if act else 1.0
        want, size = _bound(x, _np(DY) * f * _np(W))
        assert (np.abs(_np(got["dx"]) - want) <= ref.F32 * size).all(), (act, (np.abs(_np(got["dx"]) - want) / size).max())


@pytest.mark.parametrize("large", LARGE)
@pytest.mark.parametrize("D", [1, 2, 64, 256, 257, 512, 1000, 2048, 2049, 4096, 8192, 12000, 16384])
def test_residual_norm_gradient_at_a_dominating_element(kda, D, large):
    import torch
    x = _rows(D, large)
    r = np.random.default_rng(1)
    X, DN, W, DX = (_t(z, torch.float32) for z in (x, r.normal(size=x.shape), 1 + 0.3 * r.normal(size=D), r.normal(size=x.shape)))
    got = kda.residual_norm_bwd(DN, None, X, W, scale=2.0, eps=EPS)
    want, size = _bound(x, _np(DN) * _np(W))
    assert (np.abs(_np(got["dx"]) - want) <= ref.F32 * size).all(), (np.abs(_np(got["dx"]) - want) / size).max()
    assert torch.equal(got["dy"], 2 * got["dx"])
    both = kda.residual_norm_bwd(DN, DX, X, W, scale=2.0, eps=EPS)
    assert torch.equal(both["dx"], DX + got["dx"]) or \
        (np.abs(_np(both["dx"]) - (_np(DX) + want)) <= ref.F32 * (size + np.abs(_np(DX)))).all()


@pytest.mark.parametrize("large", [1e16, 1e18, 1e25])
def test_rows_at_the_end_of_the_range_have_finite_gradients(kda, large):
    """Their squares, or products with them, pass the largest fp32; the gradient itself is next to nothing."""
    import torch
    r = np.random.default_rng(2)
    x = _rows(128, large)
    x[9] = large
    X, DY, W = _t(x, torch.float32), 1e3 * _t(r.normal(size=x.shape), torch.float32), _t(1 + 0.3 * r.normal(size=128), torch.float32)
    plain = [i for i in range(len(x)) if i != 7]
    for dx in (kda.gated_norm_bwd(DY[:, None], X[:, None], None, W, eps=EPS)["dx"][:, 0], kda.residual_norm_bwd(DY, None, X, W, eps=EPS)["dx"]):
        assert torch.isfinite(dx).all() and float(dx[plain].abs().max()) <= 1e5 / large


def _gates(rows, D):
    """Every row the same x, so that y / act(gate) is one value, and gates over the whole range of a sigmoid."""
    return np.linspace(-80.0, 80.0, rows * D).astype(np.float32).reshape(rows, 1, D)


@pytest.mark.parametrize("D", [64, 77])
def test_the_gradient_of_a_closed_or_open_sigmoid_gate(kda, D):
    """Element by element: s (1 - s) has as many bits for a gate of 80 as for one of -80 (a difference taken from 1 has
    three digits at 10 and none above 17).  An exponential with an exponent rounded at 80 and some ten operations: ref.F32."""
    import torch
    a = _gates(300, D)
    x = np.broadcast_to(np.random.default_rng(3).normal(size=D).astype(np.float32), a.shape)
    w, dy = np.ones(D, np.float32), np.random.default_rng(4).normal(size=a.shape).astype(np.float32)
    f = a.astype(np.float64)
    r = 1 / np.sqrt((x.astype(np.float64) ** 2).mean(-1, keepdims=True) + EPS)
    want = dy * x * r / (1.0 + np.exp(-f)) / (1.0 + np.exp(f))
    got = kda.gated_norm_bwd(*(_t(z, torch.float32) for z in (dy, x, a, w)), eps=EPS, activation="sigmoid")["dgate"]
    err = np.abs(_np(got) - want) / np.abs(want)
    assert err.max() <= ref.F32, (err.max(), a.reshape(-1)[err.argmax()])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_infinite_and_nan_gates(kda, dtype):
    """The limits where there are any, NaN where the formula has one, and other elements unharmed."""
    import torch
    dt = getattr(torch, dtype)
    x, w = torch.ones(2, 1, 64, device="cuda", dtype=dt), torch.ones(64, device="cuda")
    a = torch.zeros_like(x)
    inf = float("inf")
    a[0, 0, :5] = torch.tensor([inf, -inf, float("nan"), 1e30, -1e30], device="cuda", dtype=dt)
    y = {act: kda.gated_norm_fwd(x, a, w, eps=0.0, activation=act)[0, 0].float() for act in ("silu", "sigmoid")}
    assert y["sigmoid"][0] == 1 and y["sigmoid"][1] == 0 and y["sigmoid"][2].isnan() and y["sigmoid"][3] == 1 and y["sigmoid"][4] == 0
    assert y["silu"][0] == inf and y["silu"][1].isnan() and y["silu"][2].isnan() and y["silu"][3] > 9e29 and y["silu"][4] == 0
    assert (y["sigmoid"][5:] == 0.5).all() and (y["silu"][5:] == 0).all()
    a[0, 0, :3] = 0
    for act, half in (("sigmoid", 0.25), ("silu", 0.5)):
        g = kda.gated_norm_bwd(x, x, a, w, eps=0.0, activation=act)
        d = g["dgate"][0, 0].float()
        assert d[3] == (0 if act == "sigmoid" else 1) and d[4] == 0 and (d[5:] == half).all()
        assert torch.isfinite(g["dx"][1]).all()


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("D", [64, 77])
def test_fp32_gates_over_the_whole_range(kda, D, act):
    """Element by element: an exponential of 2^-22, a reciprocal and a reciprocal root of 2^-22.4 and 2^-23, a sum of squares
    of up to eight terms a lane and some six roundings of 2^-24 are 1.2e-6 together; 1.5e-6 with what the exponent's own
    rounding leaves once its rest is taken along (left out, that alone is 2.6e-6 at 80)."""
    import torch
    a = _gates(300, D)
    x = np.broadcast_to(np.random.default_rng(3).normal(size=D).astype(np.float32), a.shape)
    w, dy = np.ones(D, np.float32), np.random.default_rng(4).normal(size=a.shape).astype(np.float32)
    X, A, W, DY = (_t(z, torch.float32) for z in (x, a, w, dy))
    want = ref.gated_norm(x, a, w, EPS, act)
    err = np.abs(_np(kda.gated_norm_fwd(X, A, W, eps=EPS, activation=act)) - want) / np.abs(want).clip(1e-300)
    assert err[a != 0].max() <= 1.5e-6, (err[a != 0].max(), a[a != 0][err[a != 0].argmax()])
    if act == "sigmoid":
        f = a.astype(np.float64)
        r = 1 / np.sqrt((x.astype(np.float64) ** 2).mean(-1, keepdims=True) + EPS)
        want = dy * x * r / (1.0 + np.exp(-f)) / (1.0 + np.exp(f))
        err = np.abs(_np(kda.gated_norm_bwd(DY, X, A, W, eps=EPS, activation=act)["dgate"]) - want) / np.abs(want)
        assert err.max() <= 2e-6, (err.max(), a.reshape(-1)[err.argmax()])
