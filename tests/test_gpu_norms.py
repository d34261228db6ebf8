"""The gated norm and the residual norm on the GPU against their fp64 statements."""
import numpy as np
import pytest

import _linear_ref as ref
from test_gpu_linear import _dt, _np, _t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import delta_rule_linear_gb300 as m
    m.load()
    return m


# one rounding of the output (bf16: a single value is off by up to 2^-8 of itself, half a unit in the
# last of its 8 bits) on top of fp32 arithmetic
def _tol(dtype):
    return ref.F32 if dtype == "f32" else 2.0 ** -8 + ref.F32


WIDTHS = [1, 32, 48, 64, 77, 96, 128, 200, 250, 256, 264, 512, 520, 1000, 1001, 1024]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_gated_norm(kda, D, dtype):
    import torch
    r = np.random.default_rng(D)
    act = ("silu", "sigmoid")[D % 2]
    dt = _dt(dtype)
    x, a, dy = (_t(2.0 * r.normal(size=(3, 7, 3, D)), dt) for _ in range(3))
    w = _t(1 + 0.3 * r.normal(size=D), torch.float32)
    y = kda.gated_norm_fwd(x, a, w, eps=1e-5, activation=act)
    assert ref.frob(_np(y), ref.gated_norm(_np(x), _np(a), _np(w), 1e-5, act)) <= _tol(dtype)
    got = kda.gated_norm_bwd(dy, x, a, w, eps=1e-5, activation=act)
    want = ref.gated_norm_grad(_np(dy), _np(x), _np(a), _np(w), 1e-5, act)
    for n in ("dx", "dgate"):
        assert ref.frob(_np(got[n]), want[n]) <= _tol(dtype), n
    assert ref.frob(_np(got["dw"]), want["dw"]) <= ref.F32


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 65])
def test_gated_norm_views_no_gate_and_in_place(kda, D, dtype):
    import torch
    r = np.random.default_rng(1)
    dt = _dt(dtype)
    z = _t(r.normal(size=(5, 2 * 4 * D)), dt)                 # value and gate of one projection
    x, a = (z[:, i * 4 * D:(i + 1) * 4 * D].unflatten(-1, (4, D)) for i in range(2))
    w = _t(r.normal(size=D), torch.float32)
    dy = _t(r.normal(size=(5, 4, D)), dt)
    assert torch.equal(kda.gated_norm_fwd(x, a, w), kda.gated_norm_fwd(x.contiguous(), a.contiguous(), w))
    g0, g1 = kda.gated_norm_bwd(dy, x, a, w), kda.gated_norm_bwd(dy, x.contiguous(), a.contiguous(), w)
    assert all(torch.equal(g0[n], g1[n]) for n in g0)
    y = kda.gated_norm_fwd(x, None, w)
    assert ref.frob(_np(y), ref.gated_norm(_np(x), None, _np(w), 1e-6, None)) <= _tol(dtype)
    got = kda.gated_norm_bwd(dy, x, None, w)
    want = ref.gated_norm_grad(_np(dy), _np(x), None, _np(w), 1e-6, None)
    assert "dgate" not in got and ref.frob(_np(got["dx"]), want["dx"]) <= _tol(dtype)
    want_y = kda.gated_norm_fwd(x, a, w)
    kda.gated_norm_fwd(x, a, w, out=x)
    assert torch.equal(x, want_y)


def test_gated_norm_many_rows_zero_rows_and_large_gates(kda):
    import torch
    r = np.random.default_rng(2)
    x = r.normal(size=(6000, 2, 64)).astype(np.float32)
    x[17], x[18] = 0.0, 1e-20
    a = r.normal(size=x.shape).astype(np.float32) * 40
    a[5, 0, :4] = [120.0, -120.0, 1e30, -1e30]
    w, dy = r.normal(size=64).astype(np.float32), r.normal(size=x.shape).astype(np.float32)
    X, A, W, DY = (_t(t, torch.float32) for t in (x, a, w, dy))
    y = kda.gated_norm_fwd(X, A, W)
    with np.errstate(over="ignore"):
        assert torch.isfinite(y).all()
        assert ref.frob(_np(y[6:]), ref.gated_norm(x[6:], a[6:], w, 1e-6, "silu")) <= ref.F32
        got = kda.gated_norm_bwd(DY, X, A.clamp(-1e3, 1e3), W)
        want = ref.gated_norm_grad(dy, x, np.clip(a, -1e3, 1e3), w, 1e-6, "silu")
    for n in want:
        assert ref.frob(_np(got[n]), want[n]) <= ref.F32, n


@pytest.mark.parametrize("res,dtype", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,D", [(1, 1), (9, 33), (3, 64), (33, 256), (5, 257), (7, 512), (6, 1000), (5, 2048), (3, 2049),
                                    (2, 4096), (2, 8192), (2, 8193), (3, 12000), (1, 16384), (1, 16383)])
@pytest.mark.parametrize("vec", [False, True])
def test_residual_norm(kda, rows, D, res, dtype, vec):
    import torch
    r = np.random.default_rng(D)
    x, dxo = (_t(r.normal(size=(rows, D)), _dt(res)) for _ in range(2))
    y, dn = (_t(r.normal(size=(rows, D)), _dt(dtype)) for _ in range(2))
    w = _t(1 + 0.3 * r.normal(size=D), torch.float32)
    c = _t(0.5 + 0.1 * r.normal(size=D), torch.float32) if vec else 0.37
    cn = _np(c) if vec else float(np.float32(0.37))
    z, n = kda.residual_norm_fwd(x, y, w, scale=c, eps=1e-5)
    rz, rn = ref.residual_norm(_np(x), _np(y), _np(w), cn, 1e-5)
    assert ref.frob(_np(z), rz) <= _tol(res) and ref.frob(_np(n), rn) <= _tol(dtype)
    got = kda.residual_norm_bwd(dn, dxo, z, w, y if vec else None, scale=c, eps=1e-5)
    want = ref.residual_norm_grad(_np(dn), _np(dxo), _np(z), _np(y) if vec else None, _np(w), cn, 1e-5)
    assert set(got) == set(want)
    for k, tol in (("dx", _tol(res)), ("dy", _tol(dtype)), ("dw", ref.F32), ("dscale", ref.F32)):
        if k in want:
            assert ref.frob(_np(got[k]), want[k]) <= tol, k


def test_residual_norm_views_in_place_and_without_residual_gradient(kda):
    import torch
    r = np.random.default_rng(3)
    big = _t(r.normal(size=(2, 50, 3 * 512)), torch.bfloat16)
    x, y = big[..., :512], big[..., 1024:]
    w = _t(r.normal(size=512), torch.float32)
    z0, n0 = kda.residual_norm_fwd(x.contiguous(), y.contiguous(), w, scale=0.5)
    z1, n1 = kda.residual_norm_fwd(x, y, w, scale=0.5)
    assert torch.equal(z0, z1) and torch.equal(n0, n1)
    xc = x.contiguous()
    z2, _ = kda.residual_norm_fwd(xc, y, w, scale=0.5, out=xc)
    assert z2 is xc and torch.equal(xc, z0)
    dn = _t(r.normal(size=(2, 50, 512)), torch.bfloat16)
    a = kda.residual_norm_bwd(dn, None, z0, w)
    b = kda.residual_norm_bwd(dn, torch.zeros_like(z0), z0, w)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_norms_of_no_rows(kda):
    import torch
    x = torch.zeros(0, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert kda.gated_norm_fwd(x, x, w).shape == x.shape
    assert not kda.gated_norm_bwd(x, x, x, w)["dw"].any()
    y = torch.zeros(0, 64, device="cuda")
    assert kda.residual_norm_fwd(y, y, w)[0].shape == y.shape
    assert not kda.residual_norm_bwd(y, y, y, w, y)["dscale"].any()
