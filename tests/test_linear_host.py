"""Linear attention and the block norms without a GPU: the fp64 statements the GPU tests compare with
(pinned by brute force and by differences), and the refusals of the C ABI and the binding, which return
before any CUDA call (the dummy addresses are never read)."""
import ctypes

import numpy as np
import pytest

import _linear_ref as ref


@pytest.fixture(scope="module")
def lib():
    from delta_rule_linear_gb300 import build as b
    b.build()
    from delta_rule_linear_gb300 import _lib
    return _lib.load()


def _inputs(seed=0, B=2, T=7, H=2, m=2, dk=4, dv=3):
    r = np.random.default_rng(seed)
    return (r.normal(size=(B, T, H, dk)), r.normal(size=(B, T, H, dk)), r.normal(size=(B, T, H * m, dv)),
            -0.5 * np.abs(r.normal(size=(B, T, H * m))), r.normal(size=(B, H * m, dk, dv)))


def test_forward_is_the_full_decayed_attention_matrix():
    q, k, v, g, h0 = _inputs()
    o, h = ref.forward(q, k, v, g, h0)
    B, T, HV = g.shape
    qs, ks = ref.spread(q, 2), ref.spread(k, 2)
    G = np.cumsum(g, 1)
    for b in range(B):
        for hv in range(HV):
            W = np.exp(G[b, :, None, hv] - G[b, None, :, hv]) * np.tril(np.ones((T, T)))
            full = 0.5 * (W * (qs[b, :, hv] @ ks[b, :, hv].T)) @ v[b, :, hv]
            full += 0.5 * np.exp(G[b, :, hv])[:, None] * (qs[b, :, hv] @ h0[b, hv])
            assert np.allclose(full, o[b, :, hv], atol=1e-12)
    assert np.allclose(h, sum(np.exp(G[:, -1] - G[:, t])[..., None, None] * ks[:, t, :, :, None] * v[:, t, :, None, :]
                              for t in range(T)) + np.exp(G[:, -1])[..., None, None] * h0, atol=1e-12)


def test_minus_infinity_starts_a_new_document():
    q, k, v, g, h0 = _inputs()
    g = g.copy()
    g[:, 4] = -np.inf
    o, h = ref.forward(q, k, v, g, h0)
    o1, h1 = ref.forward(q[:, 4:], k[:, 4:], v[:, 4:], g[:, 4:], None)
    assert np.allclose(o[:, 4:], o1) and np.allclose(h, h1)


@pytest.mark.parametrize("what", ["q", "k", "v", "decay", "h0"])
def test_gradients_equal_central_differences(what):
    q, k, v, g, h0 = _inputs(3)
    r = np.random.default_rng(9)
    o, h = ref.forward(q, k, v, g, h0)
    do, dh = r.normal(size=o.shape), r.normal(size=h.shape)
    args = dict(q=q, k=k, v=v, decay=g, h0=h0)
    got = ref.backward(q, k, v, g, h0, do, dh)[dict(q="dq", k="dk", v="dv", decay="ddecay", h0="dh0")[what]]
    d = r.normal(size=args[what].shape)

    def loss(e):
        a = dict(args)
        a[what] = a[what] + e * d
        oo, hh = ref.forward(**a)
        return (oo * do).sum() + (hh * dh).sum()
    num = (loss(1e-5) - loss(-1e-5)) / 2e-5
    assert abs(num - (got * d).sum()) <= 1e-7 * max(1.0, abs(num))


@pytest.mark.parametrize("act", ["silu", "sigmoid", None])
def test_gated_norm_gradients_equal_central_differences(act):
    r = np.random.default_rng(1)
    x, a, w, dy = r.normal(size=(5, 3, 6)), r.normal(size=(5, 3, 6)), r.normal(size=6), r.normal(size=(5, 3, 6))
    gate = a if act else None
    got = ref.gated_norm_grad(dy, x, gate, w, 1e-3, act)
    for name, key in (("x", "dx"), ("w", "dw")) + ((("gate", "dgate"),) if act else ()):
        base = dict(x=x, gate=gate, w=w)
        d = r.normal(size=base[name].shape)
        f = lambda e: (ref.gated_norm(**{**base, name: base[name] + e * d}, eps=1e-3, act=act) * dy).sum()  # noqa: E731
        num = (f(1e-5) - f(-1e-5)) / 2e-5
        assert abs(num - (got[key] * d).sum()) <= 1e-7 * max(1.0, abs(num))


def test_residual_norm_gradients_equal_central_differences():
    r = np.random.default_rng(2)
    x, y, w, c = r.normal(size=(4, 6)), r.normal(size=(4, 6)), r.normal(size=6), r.normal(size=6)
    dn, dz = r.normal(size=(4, 6)), r.normal(size=(4, 6))
    got = ref.residual_norm_grad(dn, dz, ref.residual_norm(x, y, w, c, 1e-3)[0], y, w, c, 1e-3)
    for name, key in (("x", "dx"), ("y", "dy"), ("w", "dw"), ("c", "dscale")):
        base = dict(x=x, y=y, w=w, c=c)
        d = r.normal(size=base[name].shape)

        def f(e):
            z, n = ref.residual_norm(**{**base, name: base[name] + e * d}, eps=1e-3)
            return (z * dz).sum() + (n * dn).sum()
        num = (f(1e-5) - f(-1e-5)) / 2e-5
        assert abs(num - (got[key] * d).sum()) <= 1e-7 * max(1.0, abs(num))


# ------------------------------------------------------------------ refusals
P = lambda a=0x1000: ctypes.c_void_p(a)  # noqa: E731


def _fwd(lib, **kw):
    a = dict(q=P(), k=P(), v=P(), g=P(), fixed=0, h0=None, o=P(), hT=None, s=None, B=1, T=64, H=2, HV=4, dk=64, dv=64,
             dt=1, ws=P(), n=1 << 40)
    a.update(kw)
    return lib.kda_linear_chunk_fwd(a["q"], a["k"], a["v"], a["g"], a["fixed"], a["h0"], a["o"], a["hT"], a["s"], a["B"],
                                    a["T"], a["H"], a["HV"], a["dk"], a["dv"], a["dt"], 0.0, a["ws"], a["n"], None)


def test_chunk_fwd_refusals(lib):
    assert _fwd(lib, q=None) == 1 and _fwd(lib, o=None) == 1
    assert _fwd(lib, B=-1) == 2 and _fwd(lib, T=-1) == 2 and _fwd(lib, HV=3) == 2 and _fwd(lib, HV=1) == 2
    assert _fwd(lib, dt=2) == 3
    assert _fwd(lib, dk=48) == 4 and _fwd(lib, dv=256) == 4
    assert _fwd(lib, v=P(0x1008)) == 5 and _fwd(lib, g=P(0x1002)) == 5 and _fwd(lib, ws=P(0x1008)) == 5
    odd = (ctypes.c_longlong * 12)(*[8192, 128, 64] * 2, *[16384, 256, 64], *[16384, 260, 64])
    assert _fwd(lib, s=odd) == 5
    assert _fwd(lib, ws=None) == 6 and _fwd(lib, n=64) == 6
    assert _fwd(lib, B=0) == 0


def test_varlen_refusals(lib):
    def call(host, N=3, total=10, cu=P(), **kw):
        hs = (ctypes.c_int * len(host))(*host)
        return lib.kda_linear_varlen_fwd(P(), P(), P(), P(), 0, cu, ctypes.cast(hs, ctypes.c_void_p), None, P(), None, None,
                                         N, total, 2, 2, kw.get("dk", 64), 64, 1, 0.0, P(), 1 << 40, None)
    assert call([0, 4, 3, 10]) == 9 and call([1, 4, 6, 10]) == 9 and call([0, 4, 6, 9]) == 9
    assert call([0, 4, 6, 10], cu=None) == 1
    assert call([0, 4, 6, 10], dk=40) == 4


def test_decode_refusals(lib):
    def call(**kw):
        a = dict(q=P(), st=P(), B=2, H=2, HV=2, dk=64, dt=1)
        a.update(kw)
        return lib.kda_linear_decode_step(a["q"], P(), P(), None, 0, a["st"], P(), None, a["B"], a["H"], a["HV"], a["dk"],
                                          64, a["dt"], 0.0, None)
    assert call(q=None) == 1 and call(st=None) == 1
    assert call(B=-1) == 2 and call(HV=3) == 2
    assert call(dt=7) == 3 and call(dk=16) == 4
    assert call(st=P(0x1008)) == 5
    assert call(B=0) == 0


def test_bwd_refusals(lib):
    def call(**kw):
        a = dict(do=P(), dq=P(), dk=64, ws=P(), n=1 << 40, g=P(), dg=P())
        a.update(kw)
        return lib.kda_linear_chunk_bwd(P(), P(), P(), a["g"], 0, None, a["do"], None, a["dq"], P(), P(), a["dg"], None,
                                        None, 1, 64, 2, 2, a["dk"], 64, 1, 0.0, a["ws"], a["n"], None)
    assert call(do=None) == 1 and call(dq=None) == 1
    assert call(dk=65) == 4
    assert call(dq=P(0x1004)) == 5 and call(dg=P(0x1001)) == 5
    assert call(ws=None) == 6 and call(n=100) == 6


def test_norm_refusals(lib):
    def g(x=P(), gate=P(), w=P(), y=P(), N=4, H=2, D=64, dt=1, act=1):
        return lib.kda_gated_norm_fwd(x, gate, w, y, None, N, H, D, dt, act, 1e-6, None)
    assert g(x=None) == 1 and g(gate=None) == 1 and g(w=None) == 1
    assert g(N=-1) == 2 and g(H=0) == 2 and g(D=0) == 2
    assert g(dt=3) == 3 and g(D=1025) == 4 and g(act=3) == 4
    assert g(x=P(0x1001)) == 5
    assert g(N=0) == 0

    def r(x=P(), N=4, D=64, res=0, dt=1):
        return lib.kda_residual_norm_fwd(x, P(), P(), None, 1.0, P(), P(), D, D, N, D, res, dt, 1e-6, None)
    assert r(x=None) == 1 and r(N=-1) == 2 and r(D=0) == 2 and r(D=16385) == 4
    assert r(res=1, dt=0) == 3 and r(res=4) == 3
    assert r(x=P(0x1002)) == 5
    assert r(N=0) == 0

    def b(y=P(), ds=P(), n=1 << 30):
        return lib.kda_residual_norm_bwd(P(), None, P(), y, P(), None, 1.0, P(), P(), P(), ds, 4, 64, 0, 0, 1e-6, P(), n, None)
    assert b(y=None) == 1 and b(ds=None) == 1 and b(n=8) == 6


def test_workspace_queries(lib):
    assert lib.kda_linear_chunk_fwd_workspace(1, 4096, 4, 4, 128, 128, 1) >= 256
    assert lib.kda_linear_chunk_fwd_workspace(1, 4096, 4, 6, 128, 128, 1) == 0
    assert lib.kda_linear_varlen_fwd_workspace(16, 34816, 16, 16, 64, 64, 1) >= 256
    assert lib.kda_linear_chunk_bwd_workspace(2, 2048, 16, 16, 128, 96, 1) == 0
    assert lib.kda_gated_norm_bwd_workspace(0) == 0 and lib.kda_residual_norm_bwd_workspace(1 << 20) == 0
    # a packed call needs no more than the query says, whatever the lengths are
    for N, total in ((3, 1000), (40, 1000), (1, 40000)):
        need = lib.kda_linear_varlen_fwd_workspace(N, total, 2, 2, 64, 64, 1)
        assert need >= 256


def test_binding_refuses_host_tensors_and_bad_shapes():
    import torch
    import delta_rule_linear_gb300 as kda
    x, h = torch.zeros(1, 4, 1, 32), torch.zeros(1, 1, 32, 32)
    cu = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: kda.linear_chunk_fwd(x, x, x), lambda: kda.linear_varlen_fwd(x, x, x, cu),
                 lambda: kda.linear_decode_step(x[:, :1], x[:, :1], x[:, :1], None, h),
                 lambda: kda.linear_chunk_bwd(x, x, x, None, None, x),
                 lambda: kda.gated_norm_fwd(x, x, torch.ones(32)), lambda: kda.gated_norm_bwd(x, x, x, torch.ones(32)),
                 lambda: kda.residual_norm_fwd(x, x, torch.ones(32)), lambda: kda.residual_norm_bwd(x, x, x, torch.ones(32)),
                 lambda: kda.linear_chunk_fwd(x.expand(1, 4, 3, 32), x, x.expand(1, 4, 4, 32))):
        with pytest.raises(ValueError):
            call()
