"""Beam search's selection and the reordering of states on the GPU against plain statements."""
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


def _logits(B, W, V, dtype, seed=0, scale=3.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + V)
    x = (scale * torch.randn((B, W, V), generator=g, device="cuda")).to(_dt(dtype))
    s = -torch.rand((B, W), generator=g, device="cuda").cumsum(1) * 2 - 5
    return x, s.contiguous()


def _compare(kda, x, s, k, finished=None, eos=None):
    got = kda.beam_select(x, s, k, finished=finished, eos=eos)
    want = ref.select(x.double().cpu().numpy(), to_np(s), k, None if finished is None else finished.cpu().numpy(), eos)
    assert np.array_equal(got[1].cpu().numpy(), want[1]) and np.array_equal(got[2].cpu().numpy(), want[2])
    g = to_np(got[0])
    assert np.array_equal(np.isfinite(g), np.isfinite(want[0]))
    ok = np.isfinite(want[0])
    assert np.all(np.abs(g - want[0])[ok] <= 1e-6 + 2.0 ** -23 * np.abs(want[0][ok]))
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,W,V,k", [(1, 1, 1, 1), (2, 3, 5, 15), (1, 4, 1000, 4), (3, 4, 1023, 8), (2, 5, 1024, 5), (2, 2, 1025, 32),
                                     (1, 16, 5003, 16), (5, 8, 20011, 16), (1, 32, 3001, 32), (1, 128, 700, 1), (40, 1, 2048, 4)])
def test_select(kda, dtype, B, W, V, k):
    x, s = _logits(B, W, V, dtype)
    _compare(kda, x, s, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_large_vocabulary(kda, dtype):
    x, s = _logits(2, 4, 131072, dtype)
    _compare(kda, x, s, 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 700, 4099])
def test_equal_totals_go_to_the_lowest_index(kda, dtype, V):
    """All logits equal in all beams; two beams that are the same; logits of few different values."""
    import torch
    x = torch.zeros(2, 3, V, device="cuda", dtype=_dt(dtype))
    s = torch.zeros(2, 3, device="cuda")
    _, p, t = _compare(kda, x, s, 8)
    assert not p.any() and t[0].tolist() == list(range(8))
    x, _ = _logits(2, 3, V, dtype)
    x[:, 2] = x[:, 0]
    _compare(kda, x.round(), s, 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_views_of_a_padded_vocabulary(kda, dtype):
    """Rows that start at any element, padding that must not be looked at."""
    import torch
    x, s = _logits(2, 3, 4111, dtype)
    big = torch.full((2, 3, 4200), 1e4, device="cuda", dtype=x.dtype)
    for at in (0, 1, 3, 8):
        big[..., at:at + 4111] = x
        _compare(kda, big[..., at:at + 4111], s, 6)
        big[..., at:at + 4111] = 1e4
    _compare(kda, x.transpose(0, 1).contiguous().transpose(0, 1), s, 6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eos", [0, 2, 1499])
def test_finished_beams(kda, dtype, eos):
    import torch
    x, s = _logits(4, 4, 1500, dtype)
    f = torch.tensor([[0, 1, 0, 0], [1, 1, 1, 1], [0, 0, 0, 0], [1, 0, 0, 1]], device="cuda", dtype=torch.bool)
    x[0, 1] = float("nan")                  # a finished beam's logits are not looked at
    got = _compare(kda, x, s, 4, f, eos)
    assert got[2][1].tolist() == [eos] * 4 and torch.equal(got[0][1], s[1].sort(descending=True)[0])
    _compare(kda, x, s, 12, f, eos)         # more than the finished beams have: -inf candidates by index


def test_first_step_and_masked_logits(kda):
    """All beams but one at -inf; logits of -inf and of the type's lowest value; rows without a distribution."""
    import torch
    x, s = _logits(3, 4, 900, "f32")
    s[:, 1:] = float("-inf")
    _compare(kda, x, s, 8)
    x, s = _logits(3, 4, 900, "f32")
    x[0, :, 5:] = float("-inf")
    x[1, :, 7:] = torch.finfo(torch.float32).min
    x[2, 1] = float("-inf")
    x[2, 2, 17] = float("nan")
    x[2, 3, 3] = float("inf")
    _compare(kda, x, s, 25)
    x[2, 0] = float("-inf")
    got = _compare(kda, x, s, 4)
    assert got[2][2].tolist() == [0, 1, 2, 3] and not got[1][2].any()


def test_totals_are_compared_in_64_bits(kda):
    """Two beams whose totals differ by less than an fp32 total's rounding keep their order."""
    import torch
    V = 1000
    x = torch.zeros(1, 2, V, device="cuda")
    x[..., 100] = 9.0
    s = torch.tensor([[-60.0, -60.0 + 2.0 ** -18]], device="cuda")        # half a step of fp32 at -61.x is 2^-19
    got = kda.beam_select(x, s, 2)
    assert got[1].tolist() == [[1, 0]]


def test_scores_in_place_captured_and_on_another_stream(kda):
    import torch
    x, s = _logits(3, 4, 5000, "bf16")
    want = kda.beam_select(x, s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = kda.beam_select(x, s, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.beam_select(x, s)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    mine = s.clone()
    out = kda.beam_select(x, mine, out=(mine, torch.empty_like(want[1]), torch.empty_like(want[2])))
    assert out[0] is mine and all(torch.equal(a, b) for a, b in zip(want, out))


def test_empty_batch(kda):
    import torch
    x, s = _logits(1, 2, 50, "f32")
    got = kda.beam_select(x[:0], s[:0])
    assert got[0].shape == (0, 2)
    t = torch.ones(0, 2, 5, device="cuda")
    kda.beam_reorder(t, torch.zeros(0, 2, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------------------ reordering
def _moved(t, parents):
    import torch
    B, W = parents.shape
    at = torch.arange(W, device=t.device)
    p = torch.where((parents < 0) | (parents >= W), at, parents).long()
    rows = (torch.arange(B, device=t.device)[:, None] * W + p).flatten()
    return t.reshape(B * W, -1)[rows].reshape(t.shape)


@pytest.mark.parametrize("B,W", [(1, 1), (1, 2), (3, 4), (2, 5), (2, 8), (3, 13), (1, 16), (2, 32)])
def test_reorder(kda, B, W):
    """Arrays of several types and row sizes in one call; every array exactly as an indexed copy."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(W)
    mk = lambda *s, dt=torch.float32: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    states = [mk(B * W, 3, 64, 32), mk(B, W, 250, 16), mk(B * W, 3, 250, dt=torch.bfloat16), mk(B, W, 7), mk(B * W, 3, dt=torch.bfloat16),
              torch.randint(0, 256, (B, W, 5), generator=g, device="cuda").to(torch.uint8), mk(B, W), mk(B * W, 1000, dt=torch.bfloat16)]
    for kind in range(4):
        if kind == 0:
            p = torch.randint(0, W, (B, W), generator=g, device="cuda")
        elif kind == 1:         # a cycle through all beams
            p = (torch.arange(W, device="cuda") + 1).remainder(W).expand(B, W)
        elif kind == 2:         # all follow one, which is moved itself
            p = torch.full((B, W), W // 2, device="cuda")
        else:                   # some out of range: those stay
            p = torch.randint(-2, W + 3, (B, W), generator=g, device="cuda")
        p = p.to(torch.int32).contiguous()
        want = [_moved(t, p) for t in states]
        assert kda.beam_reorder(states, p) is states
        for t, w in zip(states, want):
            assert torch.equal(t, w)


def test_reorder_many_arrays_and_captured(kda):
    """More arrays than a launch takes; a graph of the reordering moves on by one with every replay."""
    import torch
    states = [torch.arange(12, device="cuda", dtype=torch.float32).reshape(6, 2) + 100 * i for i in range(70)]
    p = torch.tensor([[1, 2, 0], [2, 2, 1]], dtype=torch.int32, device="cuda")
    want = [_moved(t, p) for t in states]
    kda.beam_reorder(states, p)
    assert all(torch.equal(t, w) for t, w in zip(states, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.beam_reorder(states, p)
    for _ in range(3):
        want = [_moved(t, p) for t in states]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip(states, want))


def test_reorder_refusals(kda):
    import torch
    t, p = torch.zeros(6, 4, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for bad in (lambda: kda.beam_reorder(t[:5], p), lambda: kda.beam_reorder(t.t(), p), lambda: kda.beam_reorder(t, p[0]),
                lambda: kda.beam_reorder([t, torch.zeros(6)], p)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        kda.beam_reorder(t, p.long())
    with pytest.raises(kda.KdaError):
        kda.beam_reorder([t, t], p)
    with pytest.raises(kda.KdaError):
        kda.beam_select(torch.zeros(1, 1, 4, device="cuda"), torch.zeros(1, 1, device="cuda"), 5)
    with pytest.raises(ValueError):
        kda.beam_select(torch.zeros(1, 1, 4, device="cuda"), torch.zeros(1, 1, device="cuda"), finished=torch.zeros(1, 1, dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("V", [1, 3, 512, 513, 1025])
def test_many_beams_that_do_not_count(kda, V):
    """Nothing but -inf, or a few beams that count: the lowest indices follow, also where a row's last chunk is empty."""
    import torch
    x, s = _logits(2, 64, V, "f32")
    s[0] = float("-inf")
    s[1, 5:] = float("-inf")
    _compare(kda, x, s, 32)


def test_scores_without_a_value(kda):
    """A beam whose score is NaN, or +inf and not finished, has no candidates; a finished one keeps +inf."""
    import torch
    x, _ = _logits(1, 4, 700, "f32")
    s = torch.tensor([[float("nan"), -1.0, float("inf"), -2.0]], device="cuda")
    got = kda.beam_select(x, s, 8)
    assert set(got[1][0].tolist()) <= {1, 3} and bool(torch.isfinite(got[0]).all())
    want = kda.beam_select(x[:, 1::2].contiguous(), s[:, 1::2].contiguous(), 8)
    assert torch.equal(got[1], 2 * want[1] + 1) and torch.equal(got[2], want[2])
    f = torch.tensor([[True, False, True, False]], device="cuda")
    got = kda.beam_select(x, s, 4, finished=f, eos=9)
    assert float(got[0][0, 0]) == float("inf") and int(got[1][0, 0]) == 2 and int(got[2][0, 0]) == 9 and 0 not in got[1][0].tolist()
