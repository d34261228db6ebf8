"""The state space scan on the GPU against its fp64 statement: prompts, packed prompts, single tokens, gradients."""
import numpy as np
import pytest

import _ssm_ref as ref
from _util import to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import delta_rule_linear_gb300 as m
    from delta_rule_linear_gb300 import build as b
    b.build()
    m.load()
    return m


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _inputs(dtype, B, T, D, G, N, *, gate=True, skip=True, bias=True, h0=True, seqs=None, view=False, seed=0):
    """Time steps of 1e-3 to 0.1 around which the input moves them, decays -1 .. -N."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + D)
    dt = _dt(dtype)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if view:        # slices of one projection
        z = rn(B, T, 3 * D + 2 * G * N + 1).to(dt)
        x, step, z_gate = z[..., 1:D + 1], 0.5 * z[..., D:2 * D], z[..., 2 * D:3 * D]
        step = torch.cat([step, step], -1)[..., :D]
        Bm, Cm = z[..., 3 * D:3 * D + G * N].unflatten(-1, (G, N)), z[..., 3 * D + G * N:3 * D + 2 * G * N].unflatten(-1, (G, N))
    else:
        x, step, z_gate, Bm, Cm = rn(B, T, D).to(dt), (0.5 * rn(B, T, D)).to(dt), rn(B, T, D).to(dt), rn(B, T, G, N).to(dt), rn(B, T, G, N).to(dt)
    base = torch.exp(np.log(1e-3) + np.log(100.0) * torch.rand(D, generator=g, device="cuda"))
    a = dict(x=x, dt=step, A=-torch.arange(1, N + 1, device="cuda") * (0.1 * rn(D, N)).exp(), B=Bm, C=Cm)
    kw = dict(skip=1 + 0.1 * rn(D) if skip else None, gate=z_gate if gate else None,
              dt_bias=base + torch.log(-torch.expm1(-base)) if bias else None)
    n = B if seqs is None else seqs
    return a, kw, 0.3 * rn(n, D, N) if h0 else None, rn(B, T, D).to(dt), 0.3 * rn(n, D, N)


def _n(t):
    return None if t is None else to_np(t)


def _ref(a, kw, h0, softplus=True, grad=None):
    return ref.scan(_n(a["x"]), _n(a["dt"]), _n(a["A"]), _n(a["B"]), _n(a["C"]), _n(h0), _n(kw["skip"]), _n(kw["gate"]),
                    _n(kw["dt_bias"]), softplus, grad)


def _tol(dtype, T):
    return ref.scan_tol(T) + (ref.U8 if dtype == "bf16" else 0.0)


def _check(name, got, want, tol):
    e = ref.frob(to_np(got), want)
    assert e <= tol, f"{name}: {e:.2e} > {tol:.2e}"


def _check_grads(got, want, dtype, T, keys):
    assert set(got) == set(keys)
    for k in keys:
        _check(k, got[k], want[k], 2 * ref.scan_tol(T) + (ref.U8 if dtype == "bf16" and k in ("dx", "ddt", "dB", "dC", "dgate") else 0.0))


ALL = ["dx", "ddt", "dA", "dB", "dC", "dskip", "dgate", "ddt_bias", "dh0"]
SHAPES = [(1, 1, 8, 1, 16), (2, 3, 40, 1, 16), (1, 31, 33, 1, 16), (3, 32, 64, 2, 16), (2, 33, 250, 1, 16), (1, 129, 96, 3, 16),
          (2, 50, 70, 1, 8), (1, 65, 36, 2, 32), (2, 40, 20, 1, 64), (1, 300, 128, 1, 16), (1, 200, 130, 1, 64), (1, 257, 136, 1, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D,G,N", SHAPES)
@pytest.mark.parametrize("full", [True, False])
def test_fwd_and_gradients(kda, dtype, B, T, D, G, N, full):
    a, kw, h0, dy, dh = _inputs(dtype, B, T, D, G, N, gate=full, skip=full, bias=full, h0=full)
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    wy, wh = _ref(a, kw, h0)
    _check("y", y, wy, _tol(dtype, T))
    _check("h", h, wh, ref.scan_tol(T))
    got = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh if full else None, **kw)
    want = _ref(a, kw, h0, grad=(to_np(dy), _n(dh) if full else None))
    _check_grads(got, want, dtype, T, ALL if full else ["dx", "ddt", "dA", "dB", "dC"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D,G,N", [(2, 45, 48, 1, 16), (3, 20, 37, 1, 8), (1, 70, 24, 3, 32)])
def test_views_and_a_time_step_as_it_is(kda, dtype, B, T, D, G, N):
    """Slices of one projection, an odd element off the 16-byte boundary; dt + dt_bias without softplus."""
    a, kw, h0, dy, dh = _inputs(dtype, B, T, D, G, N, view=True)
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    wy, wh = _ref(a, kw, h0)
    _check("y", y, wy, _tol(dtype, T))
    _check("h", h, wh, ref.scan_tol(T))
    _check_grads(kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw), _ref(a, kw, h0, grad=(to_np(dy), to_np(dh))), dtype, T, ALL)
    a["dt"] = (0.05 * a["dt"].abs()).contiguous()
    kw["dt_bias"] = kw["dt_bias"] * 0 + 0.01
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw, softplus=False)
    wy, wh = _ref(a, kw, h0, False)
    _check("y", y, wy, _tol(dtype, T))
    _check("h", h, wh, ref.scan_tol(T))
    got = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw, softplus=False)
    _check_grads(got, _ref(a, kw, h0, False, grad=(to_np(dy), to_np(dh))), dtype, T, ALL)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[5], [0, 3, 1, 0, 50, 2, 0], [200, 7, 129], [33] * 9])
@pytest.mark.parametrize("D,N", [(24, 16), (37, 8)])
def test_packed(kda, dtype, lens, D, N):
    import torch
    cu, extra = [0] + np.cumsum(lens).tolist(), 3
    S = len(lens)
    a, kw, h0, dy, dh = _inputs(dtype, 1, cu[-1] + extra, D, 1, N, seqs=S)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = torch.full_like(a["x"], 7.0)
    y, h = kda.ssm_varlen_fwd(*a.values(), cud, h0, out=out, **kw)
    assert bool((y[:, cu[-1]:] == 7.0).all())
    rows = [to_np(a[k]) for k in ("x", "dt", "B", "C")] + [to_np(kw["gate"])]
    one = lambda x, dt, B, C, z, s: ref.scan(x, dt, to_np(a["A"]), B, C, s, to_np(kw["skip"]), z, to_np(kw["dt_bias"]))  # noqa: E731
    want = ref.packed(cu, one, rows, [to_np(h0)])
    T = max(lens)
    _check("y", y[:, :cu[-1]], np.concatenate([o[0] for o in want], 1), _tol(dtype, T))
    _check("h", h, np.concatenate([o[1] for o in want]), ref.scan_tol(T))
    cut = {k: (v[:, :cu[-1]] if k != "A" else v) for k, v in a.items()}
    kc = dict(kw, gate=kw["gate"][:, :cu[-1]])
    y2, h2 = kda.ssm_varlen_fwd(*cut.values(), cud, h0, cu_seqlens_cpu=torch.tensor(cu), **kc)
    _check("y (host copy)", y2, to_np(y[:, :cu[-1]]), _tol(dtype, T))
    _check("h (host copy)", h2, to_np(h), ref.scan_tol(T))
    got = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, cu_seqlens=cud, **kw)
    grads = ref.packed(cu, lambda x, dt, B, C, z, d, s, e: ref.scan(x, dt, to_np(a["A"]), B, C, s, to_np(kw["skip"]), z,
                                                                   to_np(kw["dt_bias"]), grad=(d, e)),
                       rows + [to_np(dy)], [to_np(h0), to_np(dh)])
    full = {k: (np.concatenate([o[k] for o in grads], 1) if k in ("dx", "ddt", "dB", "dC", "dgate") else
                np.concatenate([o[k] for o in grads]) if k == "dh0" else sum(o[k] for o in grads)) for k in ALL}
    _check_grads({k: (v[:, :cu[-1]] if k in ("dx", "ddt", "dB", "dC", "dgate") else v) for k, v in got.items()}, full, dtype, T, ALL)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,G,N", [(1, 8, 1, 16), (3, 250, 1, 16), (17, 64, 2, 8), (5, 33, 1, 64), (2, 36, 3, 32)])
def test_steps_equal_the_recurrence(kda, dtype, B, D, G, N):
    T = 5
    a, kw, h0, _, _ = _inputs(dtype, B, T, D, G, N, view=True)
    wy, wh = _ref(a, kw, h0)
    st = h0.clone()
    for t in range(T):
        at = lambda v: v[:, t]  # noqa: E731
        y = kda.ssm_decode_step(at(a["x"]), at(a["dt"]), a["A"], at(a["B"]), at(a["C"]), st, skip=kw["skip"], gate=at(kw["gate"]),
                                dt_bias=kw["dt_bias"])
        _check(f"y {t}", y, wy[:, t], _tol(dtype, T))
    _check("state", st, wh, ref.scan_tol(T))
    one = lambda v: v[:, :1]  # noqa: E731
    y = kda.ssm_decode_step(one(a["x"]), one(a["dt"]), a["A"], one(a["B"]), one(a["C"]), h0.clone(), softplus=True)
    assert y.shape == (B, 1, D)


@pytest.mark.parametrize("D,B,T", [(64, 1, 5000), (40, 2, 2100)])
def test_a_long_sequence_is_split_and_joined(kda, D, B, T):
    """Few channels and many tokens: the sequence's parts run side by side.  In place (one memory array for both) it is
    walked in one part; both agree with the statement."""
    a, kw, h0, dy, dh = _inputs("f32", B, T, D, 1, 16)
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    wy, wh = _ref(a, kw, h0)
    tol = ref.scan_tol(1000)        # a memory of time steps of 1e-3 holds some 1000 tokens
    _check("y", y, wy, tol)
    _check("h", h, wh, tol)
    st = h0.clone()
    y2, back = kda.ssm_chunk_fwd(*a.values(), st, final_state=st, **kw)
    assert back is st
    _check("y in place", y2, wy, tol)
    _check("h in place", st, wh, tol)
    got = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw)
    want = _ref(a, kw, h0, grad=(to_np(dy), to_np(dh)))
    for k in ALL:
        _check(k, got[k], want[k], 2 * tol)


def test_batch_larger_than_the_machine(kda):
    """More (sequence, channel block) pairs than run at once, lengths that end inside a tile."""
    a, kw, h0, dy, dh = _inputs("bf16", 37, 45, 512, 1, 16)
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    wy, wh = _ref(a, kw, h0)
    _check("y", y, wy, _tol("bf16", 45))
    _check("h", h, wh, ref.scan_tol(45))
    _check_grads(kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw), _ref(a, kw, h0, grad=(to_np(dy), to_np(dh))), "bf16", 45, ALL)


def test_strong_and_weak_decays(kda):
    """Time steps up to 50 with decays of -16 (the memory is forgotten at once: exp underflows to 0), and of 1e-6 (it is
    kept): no infinities, no NaN, and the statement's values."""
    import torch
    a, kw, h0, dy, dh = _inputs("f32", 2, 60, 48, 1, 16)
    a["dt"][:, ::3] = 50.0
    a["dt"][:, 1::3] = -14.0
    kw["dt_bias"] = torch.zeros_like(kw["dt_bias"])
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    wy, wh = _ref(a, kw, h0)
    _check("y", y, wy, ref.scan_tol(60))
    _check("h", h, wh, ref.scan_tol(60))
    _check_grads(kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw), _ref(a, kw, h0, grad=(to_np(dy), to_np(dh))), "f32", 60, ALL)


def test_an_infinite_token_stays_in_its_channel(kda):
    """x = inf at one token reaches that channel's outputs from there on, and no other channel's or sequence's."""
    import torch
    a, kw, h0, _, _ = _inputs("f32", 2, 40, 40, 1, 16, gate=False)
    a["x"][1, 10, 5] = float("inf")
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 10:, 5] = True
    assert torch.equal(bad, want)
    assert torch.isfinite(h[0]).all() and not torch.isfinite(h[1, 5]).any()


def test_empty_calls(kda):
    import torch
    a, kw, h0, dy, dh = _inputs("f32", 2, 1, 24, 1, 16)
    e = {k: (v[:, :0] if k != "A" else v) for k, v in a.items()}
    ke = dict(kw, gate=kw["gate"][:, :0])
    y, h = kda.ssm_chunk_fwd(*e.values(), h0, **ke)
    assert y.shape == (2, 0, 24) and torch.equal(h, h0)
    assert not kda.ssm_chunk_fwd(*e.values(), None, **ke)[1].any()
    got = kda.ssm_chunk_bwd(dy[:, :0], *e.values(), h0, dh, **ke)
    assert torch.equal(got["dh0"], dh) and not got["dA"].any() and not got["dskip"].any()
    z = {k: (v[:0] if k != "A" else v) for k, v in a.items()}
    kz = dict(kw, gate=kw["gate"][:0])
    assert kda.ssm_chunk_fwd(*z.values(), h0[:0], **kz)[0].shape == (0, 1, 24)
    assert not kda.ssm_chunk_bwd(dy[:0], *z.values(), h0[:0], None, **kz)["dA"].any()


def test_results_do_not_depend_on_the_run(kda):
    """The same call twice, and beside others on a second stream, gives the same bits."""
    import torch
    a, kw, h0, dy, dh = _inputs("bf16", 2, 300, 256, 1, 16)
    first, fwd = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw), kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        other = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw, stream=st)
        again, f2 = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw), kda.ssm_chunk_fwd(*a.values(), h0, **kw)
        st.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(first[k], again[k]) and torch.equal(first[k], other[k]) for k in first)
        assert all(torch.equal(p, q) for p, q in zip(fwd, f2))


def test_captured_in_a_graph(kda):
    import torch
    a, kw, h0, dy, dh = _inputs("bf16", 1, 700, 64, 1, 16)
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    want = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, h2 = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
        got = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y2, y) and torch.equal(h2, h) and all(torch.equal(got[k], want[k]) for k in want)


def test_gradients_equal_differences_of_the_kernel(kda):
    """fp32: a loss of about 1 with rounding of some 1e-6, central differences over steps of 1e-2 of the input's size."""
    import torch
    a, kw, h0, dy, dh = _inputs("f32", 2, 90, 40, 2, 16)
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    dy, dh = dy / dy.numel() ** 0.5, dh / dh.numel() ** 0.5
    got = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw)
    g = torch.Generator(device="cuda").manual_seed(3)
    base = dict(a, **kw, h0=h0)
    for name in base:
        d = torch.randn(base[name].shape, generator=g, device="cuda")
        d *= base[name].norm() / d.norm()

        def loss(e):
            m = dict(base, **{name: base[name] + e * d})
            yy, hh = kda.ssm_chunk_fwd(*(m[k] for k in ("x", "dt", "A", "B", "C", "h0")), skip=m["skip"], gate=m["gate"], dt_bias=m["dt_bias"])
            return float((yy.double() * dy.double()).sum() + (hh.double() * dh.double()).sum())
        num = (loss(1e-2) - loss(-1e-2)) / 2e-2
        ana = float((got["d" + name].double() * d.double()).sum())
        assert abs(num - ana) <= 2e-2 * max(abs(ana), 0.1), (name, num, ana)


def test_two_calls_feed_one_another(kda):
    """A prompt in parts, each from the memory that the one before left, with nothing waited for in between."""
    import torch
    a, kw, h0, _, _ = _inputs("f32", 2, 170, 96, 1, 16)
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    st, parts = h0, []
    for lo, hi in ((0, 1), (1, 64), (64, 65), (65, 170)):
        cut = {k: (v[:, lo:hi] if k != "A" else v) for k, v in a.items()}
        yy, st = kda.ssm_chunk_fwd(*cut.values(), st, **dict(kw, gate=kw["gate"][:, lo:hi]))
        parts.append(yy)
    _check("y", torch.cat(parts, 1), to_np(y), ref.scan_tol(170))
    _check("h", st, to_np(h), ref.scan_tol(170))
