"""The short convolution on the GPU against its fp64 statement: prompts, packed prompts, single tokens, gradients."""
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


def _rn(g, *s, dt=None):
    import torch
    t = torch.randn(s, generator=g, device="cuda")
    return t if dt is None else t.to(dt)


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def _tol(dtype):
    return ref.CONV + (ref.U8 if dtype == "bf16" else 0.0)


def _check(name, got, want, tol):
    e = ref.frob(to_np(got), want)
    assert e <= tol, f"{name}: {e:.2e} > {tol:.2e}"


SHAPES = [(1, 1, 8, 4), (2, 2, 16, 4), (1, 3, 40, 4), (3, 5, 7, 3), (2, 37, 250, 2), (1, 100, 264, 4), (2, 64, 512, 3), (1, 700, 72, 4)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,K", SHAPES)
@pytest.mark.parametrize("act,bias,h0,view", [("silu", True, False, False), (None, False, True, True), ("silu", False, True, True)])
def test_fwd_and_gradients(kda, dtype, B, T, C, K, act, bias, h0, view):
    g, dt = _gen(T * C + K), _dt(dtype)
    wide = _rn(g, B, T, 3 * C, dt=dt)
    x = wide[..., C:2 * C] if view else wide[..., :C].contiguous()
    w, b = _rn(g, C, K), _rn(g, C) if bias else None
    s0 = _rn(g, B, K - 1, C, dt=dt) if h0 else None
    y, s = kda.conv_fwd(x, w, b, s0, activation=act)
    n = lambda t: None if t is None else to_np(t)  # noqa: E731
    wy, ws = ref.conv(n(x), n(w), n(b), n(s0), act)
    _check("y", y, wy, _tol(dtype))
    assert np.array_equal(to_np(s), ws)             # rows are moved, not computed
    dy, ds = (wide[..., 2 * C:] if view else _rn(g, B, T, C, dt=dt)), _rn(g, B, K - 1, C, dt=dt)
    got = kda.conv_bwd(dy, x, w, b, s0, ds, activation=act)
    want = ref.conv_grad(n(dy), n(x), n(w), n(b), n(s0), n(ds), act)
    assert set(got) == {"dx", "dw"} | ({"dbias"} if bias else set()) | ({"dstate"} if h0 else set())
    for k, v in got.items():
        _check(k, v, want[k], _tol(dtype) if k in ("dx", "dstate") else ref.CONV_SUMS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[5], [0, 3, 1, 0, 50, 2, 0], [1, 1, 1], [300, 7, 129]])
@pytest.mark.parametrize("C", [24, 37])
def test_packed(kda, dtype, lens, C):
    """Every sequence by itself; rows behind the last one are left as they were, in the outputs."""
    import torch
    g, dt, K, extra = _gen(sum(lens)), _dt(dtype), 4, 3
    cu = [0] + np.cumsum(lens).tolist()
    x = _rn(g, 1, cu[-1] + extra, C, dt=dt)
    w, b, s0 = _rn(g, C, K), _rn(g, C), _rn(g, len(lens), K - 1, C, dt=dt)
    out = torch.full_like(x, 7.0)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, s = kda.conv_varlen_fwd(x, w, cud, b, s0, out=out)
    assert y is out and bool((y[:, cu[-1]:] == 7.0).all())
    want = ref.packed(cu, lambda xx, ss: ref.conv(xx, to_np(w), to_np(b), ss), [to_np(x)], [to_np(s0)])
    _check("y", y[:, :cu[-1]], np.concatenate([o[0] for o in want], 1), _tol(dtype))
    assert np.array_equal(to_np(s), np.concatenate([o[1] for o in want]))
    xs = x[:, :cu[-1]]
    if cu[-1]:
        y2, s2 = kda.conv_varlen_fwd(xs, w, cud, b, s0, cu_seqlens_cpu=torch.tensor(cu))
        assert torch.equal(y2, y[:, :cu[-1]]) and torch.equal(s2, s)
    dy, ds = _rn(g, 1, cu[-1] + extra, C, dt=dt), _rn(g, len(lens), K - 1, C, dt=dt)
    got = kda.conv_bwd(dy, x, w, b, s0, ds, cu_seqlens=cud)
    want = ref.packed(cu, lambda d, xx, ss, e: ref.conv_grad(d, xx, to_np(w), to_np(b), ss, e), [to_np(dy), to_np(x)], [to_np(s0), to_np(ds)])
    _check("dx", got["dx"][:, :cu[-1]], np.concatenate([o["dx"] for o in want], 1), _tol(dtype))
    _check("dstate", got["dstate"], np.concatenate([o["dstate"] for o in want]), _tol(dtype))
    for k in ("dw", "dbias"):
        _check(k, got[k], sum(o[k] for o in want), ref.CONV_SUMS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,C,K", [(1, 8, 4), (3, 250, 4), (17, 64, 2), (5, 33, 3)])
def test_steps_equal_the_prompt(kda, dtype, B, C, K):
    """Tokens one at a time give the prompt's bits: the same sums in the same order."""
    import torch
    g, dt, T = _gen(C), _dt(dtype), 6
    x, w, b = _rn(g, B, T, 2 * C, dt=dt)[..., C:], _rn(g, C, K), _rn(g, C)
    s0 = _rn(g, B, K - 1, C, dt=dt)
    y, s = kda.conv_fwd(x, w, b, s0)
    st = s0.clone()
    for t in range(T):
        yt = kda.conv_decode_step(x[:, t], w, st, b)
        _check("y", yt, to_np(y[:, t]), _tol(dtype))
    assert torch.equal(st, s)
    yt = kda.conv_decode_step(x[:, :1], w, s0.clone(), b, activation=None)
    assert yt.shape == (B, 1, C)


def test_window_updated_in_place(kda):
    """A prompt in two calls over one window array; the second call reads what the first one wrote."""
    import torch
    g = _gen(5)
    x, w = _rn(g, 2, 40, 48, dt=torch.bfloat16), _rn(g, 48, 4)
    y, s = kda.conv_fwd(x, w)
    st = torch.zeros(2, 3, 48, dtype=torch.bfloat16, device="cuda")
    for a, b in ((0, 17), (17, 18), (18, 40)):
        yy, back = kda.conv_fwd(x[:, a:b], w, None, st, final_state=st)
        assert back is st and torch.equal(yy, y[:, a:b])
    assert torch.equal(st, s)


def test_empty_calls(kda):
    import torch
    w, x = torch.ones(8, 4, device="cuda"), torch.zeros(2, 0, 8, device="cuda")
    s0 = torch.randn(2, 3, 8, device="cuda")
    y, s = kda.conv_fwd(x, w, None, s0)
    assert y.shape == (2, 0, 8) and torch.equal(s, s0)
    got = kda.conv_bwd(x, x, w, None, s0, s0 + 1)
    assert torch.equal(got["dstate"], s0 + 1) and not got["dw"].any()
    y, s = kda.conv_fwd(x[:0], w)
    assert y.shape == (0, 0, 8) and s.shape == (0, 3, 8)
    assert not kda.conv_bwd(x[:0], x[:0], w, w[:, 0].contiguous())["dw"].any()
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert kda.conv_varlen_fwd(x[:1], w, cu)[1].shape == (0, 3, 8)


def test_captured_and_on_another_stream(kda):
    import torch
    g = _gen(9)
    x, w, s0 = _rn(g, 2, 33, 64), _rn(g, 64, 4), _rn(g, 2, 3, 64)
    dy = _rn(g, 2, 33, 64)
    y, s = kda.conv_fwd(x, w, None, s0)
    want = kda.conv_bwd(dy, x, w, None, s0, s0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y2, _ = kda.conv_fwd(x, w, None, s0, stream=st)
    st.synchronize()
    assert torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, s3 = kda.conv_fwd(x, w, None, s0)
        got = kda.conv_bwd(dy, x, w, None, s0, s0)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y3, y) and torch.equal(s3, s) and all(torch.equal(got[k], want[k]) for k in want)


def test_an_infinite_token_stays_where_it_is(kda):
    """It reaches the K outputs that read it and no others, and no other channel."""
    import torch
    g = _gen(11)
    x, w = _rn(g, 1, 30, 16), _rn(g, 16, 4)
    x[0, 10, 5] = float("inf")
    y, _ = kda.conv_fwd(x, w, activation=None)
    bad = ~torch.isfinite(y[0])
    want = torch.zeros_like(bad)
    want[10:14, 5] = True
    assert torch.equal(bad, want)


def _packed64(x, w, b, s0, cu):
    """Packed sequences in fp64 without a loop over them: x [total,C] and windows [N,K-1,C] (both with a gradient), y [total,C]."""
    import torch
    K, total = w.shape[1], x.shape[0]
    lens = (cu[1:] - cu[:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), lens)
    t = torch.arange(total, device="cuda") - cu.long()[seq]             # the token's place in its sequence
    flat = torch.cat([s0.flatten(0, 1), x])
    p = b.expand(total, -1)
    for j in range(K):
        back = t - (K - 1) + j
        at = torch.where(back >= 0, len(s0) * (K - 1) + cu.long()[seq] + back, seq * (K - 1) + back + K - 1)
        p = p + w[:, j] * flat[at]
    return p * torch.sigmoid(p)


@pytest.mark.parametrize("N,most,C", [(31, 60, 40), (512, 30, 36), (513, 30, 37), (1100, 9, 256), (33000, 1, 24), (40000, 3, 32)])
def test_packed_sequences_of_any_number(kda, N, most, C):
    """A warp finds its run's sequence among any number of them: lengths from none on, a run's length and its multiples among
    them.  Tolerances: CONV; sums over up to 60,000 rows err like sqrt(n) 2^-24, 1.5e-5."""
    import torch
    g, K = _gen(N), 4
    lens = torch.randint(0, most + 1, (N,), generator=torch.Generator().manual_seed(N))
    lens[::5] = lens[::5] // 8 * 8
    lens[1::7] = 0
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    cud, total = cu.cuda(), int(cu[-1])
    x, w, b, s0 = _rn(g, 1, total, C), _rn(g, C, K), _rn(g, C), _rn(g, N, K - 1, C)
    y, s = kda.conv_varlen_fwd(x, w, cud, b, s0, cu_seqlens_cpu=cu)
    leaf = [t.double().requires_grad_(True) for t in (x[0], w, b, s0)]
    want = _packed64(*leaf, cud)
    _check("y", y[0], to_np(want.detach()), ref.CONV)
    rows = cud[1:].long()[:, None] - (K - 1) + torch.arange(K - 1, device="cuda")
    back = (cud[1:] - cud[:-1]).long()[:, None] - (K - 1) + torch.arange(K - 1, device="cuda")
    old = s0.gather(1, (back + K - 1).clamp(0, K - 2)[..., None].expand(-1, -1, C))
    assert torch.equal(s, torch.where((back >= 0)[..., None], x[0][rows.clamp(min=0)], old))
    dy = _rn(g, 1, total, C)
    got = kda.conv_bwd(dy, x, w, b, s0, None, cu_seqlens=cud)
    grads = torch.autograd.grad(want, leaf, dy[0].double())
    for k, v, tol in zip(("dx", "dw", "dbias", "dstate"), grads, (ref.CONV, 1.5e-5, 1.5e-5, ref.CONV)):
        _check(k, got[k].reshape(v.shape), to_np(v), tol)


def test_many_short_sequences_cost_what_their_tokens_do(kda):
    """A token for each of 200,000 sequences: packed it is the same work as a batch of that many, 0.19 and 0.14 ms (a search
    whose time grows with the number of sequences, for each of them, took twelve times as long already at 16,384; ten times the batch's
    time are allowed)."""
    import torch
    g, N, C = _gen(1), 200000, 128
    x, w, s0 = _rn(g, N, 1, C, dt=torch.bfloat16), _rn(g, C, 4), _rn(g, N, 3, C, dt=torch.bfloat16)
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    want = kda.conv_fwd(x, w, None, s0)
    got = kda.conv_varlen_fwd(x.view(1, N, C), w, cu, None, s0)
    assert torch.equal(got[0].view_as(want[0]), want[0]) and torch.equal(got[1], want[1])

    def us(call):
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(6)]
        for e in ev:
            e.record()
            call()
        torch.cuda.synchronize()
        return min(a.elapsed_time(b) for a, b in zip(ev, ev[1:]))
    assert us(lambda: kda.conv_varlen_fwd(x.view(1, N, C), w, cu, None, s0)) <= 10 * us(lambda: kda.conv_fwd(x, w, None, s0))
