"""The short convolution, the state space scan and beam search without a GPU: the fp64 statements the GPU tests compare
with (pinned by brute force and by differences), and the refusals of the C ABI and the binding, which return before any CUDA
call (the dummy addresses are never read)."""
import ctypes

import numpy as np
import pytest

import _ssm_ref as ref


@pytest.fixture(scope="module")
def lib():
    from delta_rule_linear_gb300 import build as b
    b.build()
    from delta_rule_linear_gb300 import _lib
    return _lib.load()


# ------------------------------------------------------------------ the statements
def _scan_inputs(seed=0, B=2, T=6, D=6, G=2, N=3):
    r = np.random.default_rng(seed)
    n = lambda *s: r.normal(size=s)  # noqa: E731
    return dict(x=n(B, T, D), dt=n(B, T, D), A=-np.exp(n(D, N)), Bm=n(B, T, G, N), Cm=n(B, T, G, N), h0=n(B, D, N), skip=n(D),
                gate=n(B, T, D), dt_bias=n(D))


def test_scan_is_the_sum_over_earlier_tokens():
    """y_t = sum_{s <= t} C_t . exp(A (S_t - S_s)) B_s dt_s x_s, written as one sum for each pair of tokens."""
    a = _scan_inputs()
    y, h = ref.scan(**dict(a, gate=None, skip=None))
    step = ref.softplus(a["dt"] + a["dt_bias"])
    S = np.cumsum(step, 1)
    B, T, D = y.shape
    for b in range(B):
        for d in range(D):
            g = d // 3
            for t in range(T):
                want = (a["Cm"][b, t, g] * np.exp(a["A"][d] * S[b, t, d]) * a["h0"][b, d]).sum()
                for s in range(t + 1):
                    want += (a["Cm"][b, t, g] * np.exp(a["A"][d] * (S[b, t, d] - S[b, s, d])) * a["Bm"][b, s, g]).sum() * step[b, s, d] * a["x"][b, s, d]
                assert abs(want - y[b, t, d]) < 1e-10


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("what", ["x", "dt", "A", "Bm", "Cm", "h0", "skip", "gate", "dt_bias"])
def test_scan_gradients_equal_central_differences(what, softplus):
    a = _scan_inputs(1)
    if not softplus:                # time steps as they are: positive, as a user has them
        a["dt"], a["dt_bias"] = np.abs(a["dt"]), np.abs(a["dt_bias"])
    r = np.random.default_rng(2)
    y, h = ref.scan(**a, use_softplus=softplus)
    dy, dh = r.normal(size=y.shape), r.normal(size=h.shape)
    name = dict(Bm="dB", Cm="dC").get(what, "d" + what)
    got = ref.scan(**a, use_softplus=softplus, grad=(dy, dh))[name]
    d = r.normal(size=a[what].shape)

    def loss(e):
        yy, hh = ref.scan(**dict(a, **{what: a[what] + e * d}), use_softplus=softplus)
        return (yy * dy).sum() + (hh * dh).sum()
    num = (loss(1e-5) - loss(-1e-5)) / 2e-5
    assert abs(num - (got * d).sum()) <= 1e-7 * max(1.0, abs(num))


@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("T", [1, 2, 7])
def test_conv_gradients_equal_central_differences(act, T):
    r = np.random.default_rng(T)
    a = dict(x=r.normal(size=(2, T, 3)), w=r.normal(size=(3, 4)), bias=r.normal(size=3), h0=r.normal(size=(2, 3, 3)))
    y, h = ref.conv(**a, act=act)
    dy, dh = r.normal(size=y.shape), r.normal(size=h.shape)
    got = ref.conv_grad(dy, **a, dhT=dh, act=act)
    for what, key in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("h0", "dstate")):
        d = r.normal(size=a[what].shape)

        def loss(e):
            yy, hh = ref.conv(**dict(a, **{what: a[what] + e * d}), act=act)
            return (yy * dy).sum() + (hh * dh).sum()
        num = (loss(1e-5) - loss(-1e-5)) / 2e-5
        assert abs(num - (got[key] * d).sum()) <= 1e-7 * max(1.0, abs(num))


def test_conv_goes_on_from_its_window():
    r = np.random.default_rng(0)
    x, w = r.normal(size=(2, 9, 3)), r.normal(size=(3, 4))
    y, h = ref.conv(x, w)
    y1, h1 = ref.conv(x[:, :2], w)
    y2, h2 = ref.conv(x[:, 2:], w, h0=h1)
    assert np.allclose(np.concatenate([y1, y2], 1), y) and np.allclose(h2, h)


def test_select_orders_ties_by_index():
    s, p, t = ref.select(np.zeros((1, 2, 3)), np.zeros((1, 2)), 4)
    assert p.tolist() == [[0, 0, 0, 1]] and t.tolist() == [[0, 1, 2, 0]] and np.allclose(s, -np.log(3))


# ------------------------------------------------------------------ refusals of the C ABI
P = lambda a=0x1000: ctypes.c_void_p(a)  # noqa: E731


def test_conv_refusals(lib):
    def f(x=P(), w=P(), b=None, h=None, y=P(0x9000), hT=None, B=2, T=5, C=6, K=4, dt=1, act=1):
        return lib.kda_conv_fwd(x, w, b, h, y, hT, None, B, T, C, K, dt, act, None)
    assert f(x=None) == 1 and f(w=None) == 1 and f(y=None) == 1
    assert f(B=-1) == 2 and f(T=-1) == 2 and f(C=0) == 2 and f(K=0) == 2 and f(B=1 << 16, T=1 << 16) == 2
    assert f(dt=2) == 3
    assert f(K=5) == 4 and f(K=1) == 4 and f(act=2) == 4 and f(act=-1) == 4
    assert f(x=P(0x1001)) == 5 and f(w=P(0x1002)) == 5 and f(h=P(0x1001)) == 5 and f(b=P(0x1001)) == 5
    assert f(y=P()) == 4                # in place
    assert f(B=0) == 0

    def v(host, N=3, total=10, cu=P()):
        hs = ctypes.cast((ctypes.c_int * len(host))(*host), ctypes.c_void_p)
        return lib.kda_conv_varlen_fwd(P(), P(), None, cu, hs, None, P(0x9000), None, None, N, total, 6, 4, 1, 1, None)
    assert v([0, 4, 3, 10]) == 9 and v([1, 4, 6, 10]) == 9 and v([0, 4, 6, 9]) == 9 and v([0], N=0) == 9
    assert v([0, 4, 6, 10], cu=None) == 1 and v([0, 4, 6, 10], cu=P(0x1002)) == 5

    def s(x=P(), st=P(), B=2, K=4, C=6):
        return lib.kda_conv_decode_step(x, P(), None, st, P(), None, B, C, K, 1, 1, None)
    assert s(x=None) == 1 and s(st=None) == 1 and s(B=-1) == 2 and s(K=8) == 4 and s(st=P(0x1001)) == 5 and s(B=0) == 0

    def b(dy=P(), dx=P(), dw=P(), ws=P(), n=1 << 40, N=2, cu=None, T=5):
        return lib.kda_conv_bwd(dy, P(), P(), None, None, None, dx, dw, None, None, cu, None, N, T, 6, 4, 1, 1, ws, n, None)
    assert b(dy=None) == 1 and b(dx=None) == 1 and b(dw=None) == 1 and b(N=-1) == 2
    assert b(dx=P(0x1001)) == 5 and b(ws=P(0x1008)) == 5 and b(ws=None) == 6 and b(n=100) == 6
    assert b(cu=P(), N=0, T=4) == 9
    assert lib.kda_conv_bwd_workspace(0, 4) == 0 and lib.kda_conv_bwd_workspace(64, 5) == 0
    assert lib.kda_conv_bwd_workspace(64, 4) >= 256


def test_ssm_refusals(lib):
    base = dict(x=P(), dt=P(), A=P(), B=P(), C=P(), skip=None, gate=None, bias=None, h0=None, y=P(0x9000), hT=None, nb=2, T=5, D=12,
                G=2, N=16, code=1, ws=P(), n=1 << 50)

    def f(**kw):
        a = dict(base, **kw)
        return lib.kda_ssm_chunk_fwd(a["x"], a["dt"], a["A"], a["B"], a["C"], a["skip"], a["gate"], a["bias"], a["h0"], a["y"],
                                     a["hT"], None, a["nb"], a["T"], a["D"], a["G"], a["N"], a["code"], 1, a["ws"], a["n"], None)
    for name in ("x", "dt", "A", "B", "C", "y"):
        assert f(**{name: None}) == 1, name
    assert f(nb=-1) == 2 and f(T=-1) == 2 and f(D=0) == 2 and f(G=5) == 2 and f(G=0) == 2 and f(nb=70000) == 2
    assert f(code=5) == 3
    assert f(N=12) == 4 and f(N=128) == 4
    assert f(x=P(0x1001)) == 5 and f(A=P(0x1008)) == 5 and f(h0=P(0x1004)) == 5 and f(hT=P(0x1008)) == 5 and f(ws=P(0x1008)) == 5
    assert f(gate=P(0x1001)) == 5 and f(skip=P(0x1002)) == 5
    assert f(ws=None) == 6 and f(n=8) == 6
    assert f(y=P()) == 4 and f(gate=P(0x9000)) == 4         # in place
    assert f(nb=0) == 0

    def v(host, nseq=3, total=10, cu=P(), N=16):
        hs = ctypes.cast((ctypes.c_int * len(host))(*host), ctypes.c_void_p)
        return lib.kda_ssm_varlen_fwd(P(), P(), P(), P(), P(), None, None, None, cu, hs, None, P(0x9000), None, None, nseq, total, 12, 2,
                                      N, 1, 1, P(), 1 << 50, None)
    assert v([0, 4, 3, 10]) == 9 and v([0, 4, 6, 9]) == 9 and v([0], nseq=0) == 9 and v([0, 4, 6, 10], cu=None) == 1
    assert v([0, 4, 6, 10], N=24) == 4

    def s(st=P(), B=2, N=16, x=P(), A=P()):
        return lib.kda_ssm_decode_step(x, P(), A, P(), P(), None, None, None, st, P(), None, B, 12, 2, N, 1, 1, None)
    assert s(x=None) == 1 and s(st=None) == 1 and s(A=None) == 1 and s(B=-1) == 2 and s(N=4) == 4 and s(st=P(0x1004)) == 5
    assert s(B=0) == 0

    def b(**kw):
        a = dict(dy=P(), dx=P(), dA=P(), dB=P(), gate=None, dgate=None, ws=P(), n=1 << 50, N=16, cu=None, nseq=2, T=5)
        a.update(kw)
        return lib.kda_ssm_chunk_bwd(a["dy"], P(), P(), P(), P(), P(), None, a["gate"], None, None, None, a["dx"], P(), a["dA"],
                                     a["dB"], P(), None, a["dgate"], None, None, a["cu"], None, a["nseq"], a["T"], 12, 2, a["N"], 1,
                                     1, a["ws"], a["n"], None)
    assert b(dy=None) == 1 and b(dx=None) == 1 and b(dA=None) == 1 and b(dB=None) == 1 and b(gate=P()) == 1
    assert b(N=20) == 4 and b(dA=P(0x1008)) == 5 and b(dx=P(0x1001)) == 5
    assert b(ws=None) == 6 and b(n=8) == 6 and b(cu=P(), nseq=0) == 9 and b(nseq=-1) == 2
    assert lib.kda_ssm_chunk_fwd_workspace(1, 64, 12, 5, 16, 1) == 0 and lib.kda_ssm_chunk_fwd_workspace(1, 64, 12, 1, 16, 1) >= 256
    assert lib.kda_ssm_chunk_bwd_workspace(1, 64, 0, 12, 1, 16, 1) >= 256 and lib.kda_ssm_chunk_bwd_workspace(1, 64, 0, 12, 1, 9, 1) == 0


def test_beam_refusals(lib):
    def f(x=P(), s=P(), fin=None, eos=0, o=P(), B=2, W=3, V=50, k=3, dt=1, ws=P(), n=1 << 40):
        return lib.kda_beam_select(x, None, s, fin, eos, o, P(), P(), B, W, V, k, dt, ws, n, None)
    assert f(x=None) == 1 and f(s=None) == 1 and f(o=None) == 1
    assert f(B=-1) == 2 and f(W=0) == 2 and f(V=0) == 2 and f(k=0) == 2 and f(k=151) == 2 and f(W=128, V=1 << 25) == 2
    assert f(dt=9) == 3
    assert f(k=33) == 4 and f(W=129) == 4
    assert f(x=P(0x1001)) == 5 and f(ws=P(0x1004)) == 5
    assert f(ws=None) == 6 and f(n=8) == 6
    assert f(fin=P(), eos=50) == 9 and f(fin=P(), eos=-1) == 9
    assert f(B=0) == 0

    def r(ptrs=(0x1000, 0x9000), sizes=(64, 64), par=P(), B=2, W=3):
        a, n = (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_longlong * len(sizes))(*sizes)
        return lib.kda_beam_reorder(a, n, len(ptrs), par, B, W, None)
    assert r(ptrs=(0x1000, None)) == 1 and r(par=None) == 1
    assert r(B=-1) == 2 and r(W=0) == 2 and r(sizes=(64, -1)) == 2 and r(B=70000) == 2
    assert r(W=33) == 4 and r(par=P(0x1002)) == 5
    assert r(ptrs=(0x1000, 0x1000)) == 9 and r(ptrs=(0x1000, 0x1000 + 64 * 6 - 1)) == 9
    assert r(B=0) == 0 and r(W=1) == 0 and r(ptrs=(), sizes=()) == 0


def test_reorder_refuses_parents_among_the_arrays(lib):
    """B W parents of four bytes: moved rows would be read as parents by CTAs that have not begun."""
    def r(par, sizes=(64, 64), B=2, W=3):
        a, n = (ctypes.c_void_p * 2)(0x1000, 0x9000), (ctypes.c_longlong * 2)(*sizes)
        return lib.kda_beam_reorder(a, n, 2, P(par), B, W, None)
    last = 64 * 6
    for at in (0x1000, 0x1000 + last - 4, 0x1000 - 4 * 6 + 4, 0x9000, 0x9000 + 8):
        assert r(at) == 9, hex(at)
    assert r(0x1000, B=0) == 0 and r(0x1000, W=1) == 0


def test_conv_gradients_refuse_outputs_in_place_of_inputs(lib):
    """A run reads rows that its neighbours write, and the first run writes the window that the last one reads."""
    def b(dy=0x1000, x=0x2000, dx=0x3000, h0=0x4000, dhT=0x5000, dh0=0x6000):
        return lib.kda_conv_bwd(P(dy), P(x), P(), None, P(h0), P(dhT), P(dx), P(), None, P(dh0), None, None, 2, 5, 6, 4, 1, 1, P(),
                                1 << 40, None)
    assert b(dx=0x1000) == 4 and b(dx=0x2000) == 4
    assert b(dh0=0x4000) == 4 and b(dh0=0x5000) == 4


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refuses_host_tensors_and_bad_arguments():
    import torch
    import delta_rule_linear_gb300 as kda
    x, w, st = torch.zeros(2, 4, 8), torch.zeros(8, 4), torch.zeros(2, 3, 8)
    A, Bc, h = torch.zeros(8, 16), torch.zeros(2, 4, 1, 16), torch.zeros(2, 8, 16)
    cu, lg, sc = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, 50), torch.zeros(2, 3)
    for call in (lambda: kda.conv_fwd(x, w), lambda: kda.conv_varlen_fwd(x[:1], w, cu), lambda: kda.conv_decode_step(x[:, 0], w, st),
                 lambda: kda.conv_bwd(x, x, w), lambda: kda.conv_fwd(x, w, activation="tanh"), lambda: kda.conv_fwd(x[0], w),
                 lambda: kda.ssm_chunk_fwd(x, x, A, Bc, Bc), lambda: kda.ssm_varlen_fwd(x[:1], x[:1], A, Bc[:1], Bc[:1], cu),
                 lambda: kda.ssm_decode_step(x[:, 0], x[:, 0], A, Bc[:, 0], Bc[:, 0], h),
                 lambda: kda.ssm_chunk_bwd(x, x, x, A, Bc, Bc), lambda: kda.beam_select(lg, sc),
                 lambda: kda.beam_reorder(h, torch.zeros(2, 1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()


def test_scan_refuses_outputs_in_place_of_any_input(lib):
    """CTAs of a group read the same B and C rows, and every CTA reads A, skip, dt_bias and the prefix array, while others
    write y already.  An empty call writes nothing: nothing is refused."""
    at = dict(x=0x1000, dt=0x2000, A=0x3000, B=0x4000, C=0x5000, skip=0x6000, gate=0x7000, bias=0x8000, h0=0x9000, cu=0xa000)

    def chunk(y, T=5, nb=2):
        p = {k: P(v) for k, v in at.items()}
        return lib.kda_ssm_chunk_fwd(p["x"], p["dt"], p["A"], p["B"], p["C"], p["skip"], p["gate"], p["bias"], p["h0"], P(y), P(0xb000),
                                     None, nb, T, 32, 2, 16, 1, 1, P(0xc000), 1 << 50, None)

    def packed(y):
        p = {k: P(v) for k, v in at.items()}
        return lib.kda_ssm_varlen_fwd(p["x"], p["dt"], p["A"], p["B"], p["C"], p["skip"], p["gate"], p["bias"], p["cu"], None, p["h0"],
                                      P(y), P(0xb000), None, 2, 10, 32, 2, 16, 1, 1, P(0xc000), 1 << 50, None)
    for name, y in at.items():
        assert packed(y) == 4, name
        assert name == "cu" or chunk(y) == 4, name
    assert chunk(0x4000, nb=0) == 0


def test_scan_gradients_refuse_outputs_in_place_of_inputs(lib):
    """The chain of the gradients writes dinitial_state beside the chain of the memories, which reads initial_state; the last
    launch writes what CTAs of the same or an earlier one read.  The smallest call of each kind is refused too."""
    ins = ("dy", "x", "dt", "A", "B", "C", "skip", "gate", "bias", "h0", "dhT")
    outs = ("dx", "ddt", "dA", "dB", "dC", "dskip", "dgate", "dbias", "dh0")
    at = {k: 0x1000 * (i + 1) for i, k in enumerate(ins + outs)}

    def b(nseq=2, T=5, cu=None, **kw):
        p = {k: P(v) if v else None for k, v in dict(at, **kw).items()}
        return lib.kda_ssm_chunk_bwd(*(p[k] for k in ins), *(p[k] for k in outs), cu, None, nseq, T, 32, 2, 16, 1, 1, P(0x100000),
                                     1 << 50, None)
    for o in outs:
        for i in ins:
            assert b(**{o: at[i]}) == 4, (o, i)
    assert b(dB=0x200000, cu=P(0x200000)) == 4
    assert b(T=0, dh0=at["h0"]) == 4 and b(nseq=1, T=1, dA=at["A"]) == 4


def test_conv_gradients_refuse_any_output_that_is_an_input(lib):
    """The weights and biases are inputs too: without a sequence their gradients are set to zero before anything is read."""
    ins, outs = ("dy", "x", "w", "b", "h0", "dhT"), ("dx", "dw", "db", "dh0")
    at = {k: 0x1000 * (i + 1) for i, k in enumerate(ins + outs)}

    def f(N=2, T=5, cu=None, **kw):
        p = {k: P(v) for k, v in dict(at, **kw).items()}
        return lib.kda_conv_bwd(*(p[k] for k in ins), *(p[k] for k in outs), cu, None, N, T, 8, 4, 1, 1, P(0x100000), 1 << 40, None)
    for o in outs:
        for i in ins:
            assert f(**{o: at[i]}) == 4, (o, i)
    assert f(dw=0x200000, cu=P(0x200000)) == 4
    assert f(N=0, dw=at["w"]) == 4 and f(T=0, db=at["b"]) == 4


def test_reorder_takes_empty_arrays_wherever_they_lie(lib):
    """Rows of no bytes overlap nothing (one beam: the call ends before a launch, after these checks)."""
    def r(ptrs, sizes):
        a, n = (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_longlong * len(sizes))(*sizes)
        return lib.kda_beam_reorder(a, n, len(ptrs), P(), 2, 1, None)
    assert r((0x1000, 0x1040), (64, 0)) == 0 and r((0x1040, 0x1000), (0, 64)) == 0
    assert r((0x1000, 0x1040), (64, 1)) == 9
