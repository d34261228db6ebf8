"""Linear attention on the GPU at the edges of its arguments."""
import numpy as np
import pytest

import _linear_ref as ref
from test_gpu_linear import _make, _np, _t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import delta_rule_linear_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_batches_raise_no_device_error(kda, dtype):
    """The workspace of an empty batch may hold anything: the allocator's memory is filled first."""
    import torch
    d, _ = _make(2, 40, 2, 1, 64, 64, dtype)
    e = {n: t[:0] for n, t in d.items()}
    for _ in range(3):
        fill = [torch.full((1 << k,), 8, dtype=torch.int32, device="cuda") for k in (6, 8, 12, 18)]
        del fill
        o, h = kda.linear_chunk_fwd(e["q"], e["k"], e["v"], e["decay"], e["h0"], check_device=True)
        assert o.shape == (0, 40, 2, 64) and h.shape == (0, 2, 64, 64)
        g = kda.linear_chunk_bwd(e["q"], e["k"], e["v"], e["decay"], e["h0"], e["d_o"], e["dhT"], check_device=True)
        assert g["dq"].shape == e["q"].shape and g["dh0"].shape == e["h0"].shape
        none = torch.zeros(1, dtype=torch.int32, device="cuda")
        p = {n: d[n][:1, :0] for n in ("q", "k", "v", "decay")}
        o, h = kda.linear_varlen_fwd(p["q"], p["k"], p["v"], none, p["decay"].contiguous(), check_device=True)
        assert o.shape == (1, 0, 2, 64) and h.shape == (0, 2, 64, 64)
        # sequences without tokens are looked at, and hand their memory on
        o, h = kda.linear_chunk_fwd(d["q"][:, :0], d["k"][:, :0], d["v"][:, :0], d["decay"][:, :0].contiguous(), d["h0"],
                                    check_device=True)
        assert torch.equal(h, d["h0"])


def test_a_first_call_in_a_capture_leaves_nothing_of_the_graph_behind(kda):
    """A call that needs no more than a header, captured on a stream that made none before, replayed, and called again on
    that stream after the graph has gone."""
    import torch
    from delta_rule_linear_gb300 import _linear
    d, n = _make(1, 20, 2, 1, 32, 32, "f32")
    ro, _ = ref.forward(n["q"], n["k"], n["v"], n["decay"], n["h0"])
    call = lambda: kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"])[0]  # noqa: E731
    call()
    torch.cuda.synchronize()
    before = set(_linear._headers)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        o = call()
    assert set(_linear._headers) == before
    g.replay()
    torch.cuda.synchronize()
    assert ref.frob(_np(o), ro) <= ref.F32
    del g, o
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        o = call()
    s.synchronize()
    assert ref.frob(_np(o), ro) <= ref.F32


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 150])
def test_broadcast_inputs_equal_copies(kda, T, dtype):
    """q, k, v and d_o expanded over requests, tokens or heads (strides of 0), in both forms and the single step."""
    import torch
    d, _ = _make(2, T, 2, 1, 64, 64, dtype)
    names = ("q", "k", "v", "d_o")
    for name, cut in ((n, c) for n in names for c in (slice(0, 1), (slice(None), slice(0, 1)), (slice(None), slice(None), slice(0, 1)))):
        x = dict(d)
        x[name] = d[name][cut].expand(2, T, 2, 64)
        c = dict(d)
        c[name] = x[name].contiguous()
        run = lambda a: (*kda.linear_chunk_fwd(a["q"], a["k"], a["v"], a["decay"], a["h0"]),  # noqa: E731
                         *kda.linear_chunk_bwd(a["q"], a["k"], a["v"], a["decay"], a["h0"], a["d_o"], a["dhT"]).values())
        assert all(torch.equal(p, q) for p, q in zip(run(x), run(c))), (name, cut)
        if name != "d_o":
            s0, s1 = d["h0"].clone(), d["h0"].clone()
            o0 = kda.linear_decode_step(*(x[n][:, 0] for n in names[:3]), d["decay"][:, 0].contiguous(), s0)
            o1 = kda.linear_decode_step(*(c[n][:, 0] for n in names[:3]), d["decay"][:, 0].contiguous(), s1)
            assert torch.equal(o0, o1) and torch.equal(s0, s1)


def _terms(q, k, v, decay, h0, d_o, dhT):
    """Root sum of squares of the terms of each row of o, dq, dk and dv of one chunk (one head per q/k head): what the
    roundings of the weights and of the memories' elements are relative to, where the terms cancel too."""
    G = np.cumsum(decay, 1).transpose(0, 2, 1)                                     # [B, H, T]
    w = np.exp(G[..., :, None] - G[..., None, :]) * np.tril(np.ones(G.shape[-1:] * 2))
    c = q.shape[-1] ** -0.5
    t = lambda x: x.transpose(0, 2, 1, 3)  # noqa: E731
    q, k, v, d_o = t(q), t(k), t(v), t(d_o)
    P, M = c * w * (q @ np.swapaxes(k, -1, -2)), c * w * (d_o @ np.swapaxes(v, -1, -2))
    into, out = np.exp(G)[..., None], np.exp(G[..., -1:] - G)[..., None]
    norm2 = lambda x: (x * x).sum(-1, keepdims=True)  # noqa: E731
    T = lambda x: np.swapaxes(x, -1, -2)  # noqa: E731
    rows = dict(o=(P ** 2 @ norm2(v), c * into, q, h0), dq=(M ** 2 @ norm2(k), c * into, d_o, T(h0)),
                dk=(T(M) ** 2 @ norm2(q), out, v, T(dhT)), dv=(T(P) ** 2 @ norm2(d_o), out, k, dhT))
    return {n: np.sqrt(a + f ** 2 * (x ** 2 @ m ** 2).sum(-1, keepdims=True))[..., 0].transpose(0, 2, 1)
            for n, (a, f, x, m) in rows.items()}


@pytest.mark.parametrize("heads", [2, 24])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first,size", [("fall", 4), ("grow", 32)])
def test_decays_that_fall_and_grow_in_a_chunk(kda, first, size, D, heads):
    """Log decays that sum to -60 (base 2) and then to +60 within a chunk, or the other way round: weights of 2^120 between
    its tokens or the inverse of them, times scores of some 2^8 (fall) or 2^14 (grow), and finite results in every row (v
    and d_o are small enough).  A row may hang on one weight, rounded to bf16 (2^-8 = 2 U8 of its term), beside its own
    rounding and, before the growth, that of the memory's operand (U8 each): 4 U8 of the row's terms.  (ddecay adds
    products of all four inputs and may pass fp32.)"""
    import torch
    T = 128
    d, _ = _make(1, T, heads, 1, D, D, "bf16", seed=31)
    for x, f in (("q", size), ("k", size), ("v", 2.0 ** -10), ("d_o", 2.0 ** -10), ("h0", 2.0 ** -10), ("dhT", 2.0 ** -10)):
        d[x] = f * d[x]
    g = np.zeros(T)
    g[:40], g[40:120] = -60 / 40 * np.log(2), 120 / 80 * np.log(2)
    d["decay"] = _t(np.repeat((g if first == "fall" else -g)[None, :, None], heads, 2), torch.float32)
    n = {x: None if t is None else _np(t) for x, t in d.items()}
    ro, rh = ref.forward(n["q"], n["k"], n["v"], n["decay"], n["h0"])
    want = dict(ref.backward(n["q"], n["k"], n["v"], n["decay"], n["h0"], n["d_o"], n["dhT"]), o=ro)
    terms = _terms(**n)
    assert max(np.abs(x).max() for x in (rh, *want.values())) < 2.0 ** 124 or first == "grow"
    o, h = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], check_device=True)
    got = dict(kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["d_o"], d["dhT"], check_device=True), o=o)
    for x in ("o", "dq", "dk", "dv"):
        assert torch.isfinite(got[x]).all(), x
        err = np.linalg.norm(_np(got[x]) - want[x], axis=-1) / np.maximum(terms[x], np.linalg.norm(want[x], axis=-1))
        assert err.max() <= 4 * ref.U8, (x, err.max())
    assert ref.frob(_np(h), rh) <= ref.TC_STATE
    assert ref.frob(_np(got["dh0"]), want["dh0"]) <= ref.TC_STATE


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 200, 500])
def test_decays_that_keep_nothing_have_no_gradient(kda, T, D, dtype):
    """ddecay_t = e^{decay_t} <h_{t-1}, D_t> is exactly 0 at a restart and, without an initial memory, at the first token: not
    what rounding leaves of the sums that it is taken from.  With an initial memory the first token's is not."""
    import torch
    d, n = _make(2, T, 3, 1, D, D, dtype, seed=40)
    g = n["decay"].copy()
    if T > 2:
        g[0, 1], g[1, T - 1], g[1, T // 2] = -np.inf, -200.0, -np.inf
    d["decay"] = _t(g, torch.float32)
    for h0 in (None, d["h0"]):
        got = _np(kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["decay"], h0, d["d_o"], d["dhT"], check_device=True)["ddecay"])
        want = ref.backward(n["q"], n["k"], n["v"], _np(d["decay"]), None if h0 is None else n["h0"], n["d_o"], n["dhT"])["ddecay"]
        with np.errstate(under="ignore"):
            nothing = np.exp(_np(d["decay"])) < 1e-45
        if h0 is None:
            nothing[:, 0] = True
        assert (got[nothing] == 0).all() and (got[~nothing] != 0).all()
        assert ref.frob(got, np.where(nothing, 0.0, want)) <= (2e-5 if T > 1 else 1e-5)
