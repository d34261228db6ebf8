"""Memories of linear attention that are kept over thousands of tokens.

Without decays a memory and its gradient are plain sums, h_T = h_0 + sum k_t v_t^T and dh_0 = dh_T + c sum q_t do_t^T.
Tensor-core accumulators cut each addition, always towards 0, so a chunk's contribution (24 steps of 16 tokens and parts)
loses some 24 2^-25 = 7e-7 of itself however long the sequence is, as long as it is not added to the memory in there, which
would lose as much of the whole every chunk: 64 chunks would be 1.5e-5 or more.  Added in fp32, rounded to nearest, 64
chunks err by sqrt(64) 2^-25 = 2.4e-7 beside it: 2^-19 together, with a margin of two.
"""
import pytest

pytestmark = pytest.mark.gpu
MEMORY = 2.0 ** -19


@pytest.fixture(scope="module")
def kda():
    import delta_rule_linear_gb300 as m
    m.load()
    return m


def _inputs(T, H, dk, dv):
    import torch
    g = torch.Generator(device="cuda").manual_seed(17)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, v, d_o = (r(1, T, H, d).bfloat16() for d in (dk, dk, dv, dv))
    return q, k, v, d_o, r(1, H, dk, dv), r(1, H, dk, dv)


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("heads", [2, 40])
@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)], ids=str)
def test_gradient_of_a_memory_kept_throughout(kda, dims, heads):
    import torch
    q, k, v, d_o, h0, dhT = _inputs(8192, heads, *dims)
    got = kda.linear_chunk_bwd(q, k, v, None, h0, d_o, dhT, check_device=True)["dh0"]
    want = dhT.double() + dims[0] ** -0.5 * torch.einsum("bthi,bthj->bhij", q.double(), d_o.double())
    assert _rel(got, want) <= MEMORY


@pytest.mark.parametrize("heads", [2, 40])
@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)], ids=str)
def test_a_memory_kept_throughout_a_whole_walk(kda, dims, heads):
    """In place, a sequence is not cut: one walk over all its chunks."""
    import torch
    q, k, v, _, h0, _ = _inputs(8192, heads, *dims)
    want = h0.double() + torch.einsum("bthi,bthj->bhij", k.double(), v.double())
    st = h0.clone()
    kda.linear_chunk_fwd(q, k, v, None, st, final_state=st, check_device=True)
    assert _rel(st, want) <= MEMORY


def test_a_memory_kept_over_calls(kda):
    """The memory handed on from call to call, decays between: as the fp64 sum of all its tokens."""
    import torch
    q, k, v, _, h0, _ = _inputs(8192, 4, 128, 128)
    g = torch.full((1, 8192, 4), -2.0 ** -13, device="cuda")
    w = ((8191 - torch.arange(8192, device="cuda")).double() * -2.0 ** -13).exp()
    want = h0.double() * float(torch.tensor(-1.0).exp()) + torch.einsum("t,bthi,bthj->bhij", w, k.double(), v.double())
    h = h0
    for t in range(0, 8192, 1024):
        s = slice(t, t + 1024)
        h = kda.linear_chunk_fwd(q[:, s], k[:, s], v[:, s], g[:, s].contiguous(), h, check_device=True)[1]
    assert _rel(h, want) <= MEMORY


@pytest.mark.parametrize("heads", [1, 3, 20, 40])
@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)], ids=str)
def test_a_memory_kept_throughout_segments(kda, dims, heads):
    """A long sequence of few heads is cut, up to 64 chunks to a segment, whose local memories are added."""
    import torch
    q, k, v, _, h0, _ = _inputs(8192, heads, *dims)
    want = h0.double() + torch.einsum("bthi,bthj->bhij", k.double(), v.double())
    assert _rel(kda.linear_chunk_fwd(q, k, v, None, h0, check_device=True)[1], want) <= MEMORY


def test_memories_kept_throughout_a_long_packed_sequence(kda):
    """Packed sequences longer than an SM's share are cut as well."""
    import torch
    lens = [16384, 70, 3000]
    q, k, v, _, _, _ = _inputs(sum(lens), 4, 64, 64)
    cu = torch.tensor([0, 16384, 16454, 19454], dtype=torch.int32)
    h = kda.linear_varlen_fwd(q, k, v, cu.cuda(), cu_seqlens_cpu=cu, check_device=True)[1]
    for i, (a, b) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
        want = torch.einsum("bthi,bthj->bhij", k[:, a:b].double(), v[:, a:b].double())
        assert _rel(h[i:i + 1], want) <= MEMORY
