"""The chunked form of linear attention, from the first length that takes it, in both of its kinds of chunk, held to bounds
that one rounding too many would pass.

Memories (h, dh0).  Values go in as three bf16 parts, all of fp32's 24 bits, k is exact and sums are fp32: left are the
rounding of the products' sums (24 steps of 16 tokens and parts a chunk, five chunks: sqrt(120) 2^-24 = 6.5e-7), of the
weights' exponents (sums of up to 128 log2 decays, at most 8 where the weights count, seven additions deep: sqrt(7) 2^-22
ln 2 = 4.4e-7) and of ex2 (2^-23).  8e-7 together: 2^-19.  Without the third part of the values, cut to 16 bits, it would
be 5e-6.

bf16 outputs and gradients.  One rounding is 1.7e-3 of an array; the weights P (M) and the memory's operand are rounded
once each and share a row between them, so they count as one, and the output rounds: 1.7e-3 sqrt(2) = 2.4e-3.  A third
rounding would make it 2.9e-3: 2.7e-3.

ddecay.  fp32 from exact or two-part operands (2^-17 each, which the dots average): 2^-17.  That holds for restarts too,
however many a chunk has: the running sums that the weights' exponents are differences of (150 a restart) must not cost them
their bits, 2^-24 of a sum of 2000 being 1e-4 of a weight.
"""
import numpy as np
import pytest

import _linear_ref as ref
from test_gpu_linear import _make, _np, _t

pytestmark = pytest.mark.gpu
MEMORY = 2.0 ** -19
OUT = 2.7e-3
DDECAY = 2.0 ** -17


@pytest.fixture(scope="module")
def kda():
    import delta_rule_linear_gb300 as m
    m.load()
    return m


def _check(kda, d, n):
    o, h = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], check_device=True)
    got = kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["d_o"], d["dhT"], check_device=True)
    ro, rh = ref.forward(n["q"], n["k"], n["v"], n["decay"], n["h0"])
    want = ref.backward(n["q"], n["k"], n["v"], n["decay"], n["h0"], n["d_o"], n["dhT"])
    err = {x: ref.frob(_np(a), b) for x, a, b in [("o", o, ro), ("h", h, rh)] + [(x, got[x], want[x]) for x in ("dq", "dk", "dv")]}
    if "dh0" in got:
        err["dh0"] = ref.frob(_np(got["dh0"]), want["dh0"])
    bound = dict(o=OUT, h=MEMORY, dq=OUT, dk=OUT, dv=OUT, dh0=MEMORY)
    if n["decay"] is not None:
        w = want["ddecay"]
        fixed = n["decay"].ndim == 1
        err["ddecay"] = ref.frob(_np(got["ddecay"]), w.sum((0, 1)) if fixed else w)
        bound["ddecay"] = DDECAY
    print({x: f"{e:.1e}" for x, e in err.items()})
    assert all(err[x] <= bound[x] for x in err), (err, bound)


@pytest.mark.parametrize("heads", [(16, 1), (8, 2)], ids=str)
@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)], ids=str)
@pytest.mark.parametrize("T", [16, 17, 31, 32, 33, 127, 128, 129, 600])
def test_lengths(kda, T, dims, heads):
    """16 tokens are walked one by one, 17 are a chunk; q/k heads of their own and shared."""
    H, m = heads
    _check(kda, *_make(2 if T < 200 else 1, T, H, m, *dims, "bf16", seed=T))


@pytest.mark.parametrize("heads", [4, 40])
@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)], ids=str)
@pytest.mark.parametrize("decay", ["none", "fixed", "strong", "reset", "grow"])
def test_decays(kda, decay, dims, heads):
    """Few heads (segments, chains over the chunks) and many (whole walks); decays beyond 2^62 within a chunk, restarts."""
    _check(kda, *_make(1, 389, heads, 1, *dims, "bf16", decay=decay, seed=7))


@pytest.mark.parametrize("dims", [(64, 64), (128, 128)], ids=str)
def test_mild_and_strong_chunks_beside_one_another(kda, dims):
    """One sequence whose chunks alternate between the two kinds, and a restart as the first and the last token of one."""
    d, _ = _make(2, 900, 4, 1, *dims, "bf16", seed=9)
    g = _np(d["decay"])
    g[:, 128:256] *= 60
    g[0, 384], g[1, 511], g[0, 899] = -np.inf, -np.inf, -np.inf
    g[:, 640:700] = -1.0
    import torch
    d["decay"] = _t(g, torch.float32)
    _check(kda, d, {x: None if t is None else _np(t) for x, t in d.items()})


@pytest.mark.parametrize("heads", [2, 40])
@pytest.mark.parametrize("dims", [(64, 64), (128, 128)], ids=str)
def test_many_documents_in_a_row(kda, dims, heads):
    """A restart every few tokens: some twenty documents a chunk."""
    import torch
    d, _ = _make(1, 500, heads, 1, *dims, "bf16", seed=10)
    g = _np(d["decay"])
    g[:, np.cumsum(np.random.default_rng(1).integers(2, 12, size=70))] = -np.inf
    d["decay"] = _t(g, torch.float32)
    _check(kda, d, {x: None if t is None else _np(t) for x, t in d.items()})


@pytest.mark.parametrize("dims", [(64, 64), (128, 128)], ids=str)
def test_packed_lengths(kda, dims):
    """Sequences of 0, 1, 16, 17, 32, 33, 127, 128, 129 and 300 tokens in one packed call, with strong decays in some."""
    import torch
    lens = [0, 17, 1, 128, 33, 16, 300, 129, 32, 127]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    d, n = _make(1, int(cu[-1]), 4, 2, *dims, "bf16", h0=False, seed=3)
    g = n["decay"].copy()
    g[:, 200:420] *= 40
    d["decay"] = _t(g, torch.float32)
    n["decay"] = _np(d["decay"])
    h0 = np.random.default_rng(5).normal(size=(len(lens), 8, *dims))
    h0t = _t(h0, torch.float32)
    o, h = kda.linear_varlen_fwd(d["q"], d["k"], d["v"], _t(cu, torch.int32), d["decay"], h0t,
                                 cu_seqlens_cpu=torch.from_numpy(cu), check_device=True)
    ro, rh = np.zeros(o.shape), np.zeros(h.shape)
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        oo, hh = ref.forward(n["q"][:, a:b], n["k"][:, a:b], n["v"][:, a:b], n["decay"][:, a:b], _np(h0t[i:i + 1]))
        ro[:, a:b], rh[i] = oo, hh[0]
    assert ref.frob(_np(o), ro) <= OUT and ref.frob(_np(h), rh) <= MEMORY


@pytest.mark.parametrize("heads", [4, 40])
@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)], ids=str)
def test_a_chunks_product_is_added_up_from_its_small_parts(kda, dims, heads):
    """The accumulator cuts each step by half a unit of its own size: 8 steps of the large part are 8 2^-25 = 2.4e-7 of a
    chunk's product (24, if that came first, 7e-7), beside 1.2e-7 of ex2 and some 2e-7 of exponents of mild decays: 6e-7.
    (ddecay's terms through S or R err by their two-part operands, 2^-18 / sqrt(3) of an element, beside that.)"""
    d, n = _make(2, 640, heads, 1, *dims, "bf16", seed=12)
    h = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], check_device=True)[1]
    got = kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["d_o"], d["dhT"], check_device=True)
    want = ref.backward(n["q"], n["k"], n["v"], n["decay"], n["h0"], n["d_o"], n["dhT"])
    err = (ref.frob(_np(h), ref.forward(n["q"], n["k"], n["v"], n["decay"], n["h0"])[1]), ref.frob(_np(got["dh0"]), want["dh0"]))
    assert max(err) <= 6e-7, err
