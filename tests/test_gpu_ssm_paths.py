"""The loops and launch forms of the convolution, the state space scan and beam search that training and serving shapes take:
gradients whose CTAs take several chunks, scans of two groups to a CTA whose rings wrap, segments of them, warps that take
several parts of a row of logits or several runs of tokens.  Which of these a shape takes is asserted without a GPU.

Tolerances, derived before the first run.  Memories, sums over tokens and other fp32 results, relative in the Frobenius norm:
a factor exp(dt A) errs by at most 2^-22.5 + 2^-23, 3e-7, of either sign and independently from token to token, so that a memory of
T tokens errs like the square root of their number; time steps err by 5e-7 and sums round: tight(T) = 2e-6 + 3e-7 sqrt(T), and
gradients, which run through two chains, twice that.  bf16 results, element by element: half a step, 2^-8 of the value, beside
that error of the array's scale (its root mean square, with a factor of 8 for the largest of some 10^7 elements).
"""
import numpy as np
import pytest

import _ssm_ref as ref
from _util import to_np
from test_gpu_ssm import ALL, _dt, _inputs, _n, _ref

gpu = pytest.mark.gpu
SMS = 152


@pytest.fixture(scope="module")
def kda():
    import delta_rule_linear_gb300 as m
    from delta_rule_linear_gb300 import build as b
    b.build()
    m.load()
    return m


def tight(T):
    return 2e-6 + 3e-7 * T ** 0.5


def _check32(name, got, want, tol):
    e = ref.frob(to_np(got), want)
    assert e <= tol, f"{name}: {e:.2e} > {tol:.2e}"


def _check_rows(name, got, want, dtype, tol):
    if dtype == "f32":
        return _check32(name, got, want, tol)
    g = to_np(got).astype(np.float64)
    assert g.shape == want.shape
    off = np.abs(g - want) - 2.0 ** -8 * np.abs(want)
    scale = np.sqrt((want ** 2).mean())
    assert off.max() <= 8 * tol * scale, f"{name}: {off.max() / scale:.2e} of the array's scale beyond a rounding, > {8 * tol:.2e}"


ROWS = ("dx", "ddt", "dB", "dC", "dgate")


def _compare_scan(kda, dtype, B, T, D, G, N, view=False, grads=True):
    a, kw, h0, dy, dh = _inputs(dtype, B, T, D, G, N, view=view)
    y, h = kda.ssm_chunk_fwd(*a.values(), h0, **kw)
    wy, wh = _ref(a, kw, h0)
    tol = tight(T)
    _check_rows("y", y, wy, dtype, tol)
    _check32("h", h, wh, tol)
    if not grads:
        return
    got = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, **kw)
    want = _ref(a, kw, h0, grad=(to_np(dy), _n(dh)))
    for k in ALL:
        if k in ROWS:
            _check_rows(k, got[k], want[k], dtype, 2 * tol)
        else:
            _check32(k, got[k], want[k], 2 * tol)


# ------------------------------------------------------------------ gradients: several chunks to a CTA
MANY_CHUNKS = [("bf16", 2, 330, 4096, 1, 16), ("f32", 2, 330, 4096, 1, 16), ("bf16", 2, 330, 4095, 1, 16), ("bf16", 2, 330, 2048, 1, 32),
               ("bf16", 2, 330, 1024, 1, 64), ("f32", 1, 700, 1026, 2, 64), ("bf16", 1, 650, 8200, 1, 8), ("bf16", 3, 230, 3900, 3, 16)]


def _chunks_and_slots(kda, B, T, D, G, N):
    """(chunks, CTAs that share a block's chunks), from the bytes that the gradients ask for."""
    chunks = B * -(-T // 32)
    per = -(-D // G // (4 * 64 // (N // 4)))
    rest = kda.load().kda_ssm_chunk_bwd_workspace(B, T, 0, D, G, N, 1) - 256
    rest = rest // 4 - 2 * chunks * D * N - -(-chunks * D // 4) * 4 - per * B * T * G * 2 * N
    slots, left = divmod(rest, D * N + 2 * D)
    assert left == 0
    return chunks, slots


def test_shapes_of_several_chunks_to_a_cta(kda):
    for _, *s in MANY_CHUNKS:
        chunks, slots = _chunks_and_slots(kda, *s)
        assert 1 < slots < chunks, (s, chunks, slots)


def _two_groups(B, T, D, G, N):
    """How a bf16 scan of equal lengths is launched: (tokens of a segment or 0, whether CTAs hold two groups)."""
    ch = 128 // (N // 4)
    blocks = -(-D // G // ch) * G
    even = B * T * blocks // (2 * SMS)
    seg = 0 if T <= 256 or T <= 3 * even else max(128, -(-even // 32) * 32)
    return seg, N > 8 and B * (-(-T // seg) if seg else 1) * blocks > SMS and D // G > ch


def test_shapes_of_two_groups(kda):
    bf16 = [s for dtype, *s in MANY_CHUNKS if dtype == "bf16"]
    assert sum(_two_groups(*s) == (0, True) and s[1] > 5 * 32 for s in bf16) >= 5 and {s[-1] for s in bf16 if _two_groups(*s)[1]} == {16, 32, 64}


@gpu
@pytest.mark.parametrize("dtype,B,T,D,G,N", MANY_CHUNKS)
def test_gradients_of_several_chunks_to_a_cta(kda, dtype, B, T, D, G, N):
    """And the scans of these shapes: two groups to a CTA in bf16, with more tiles than the ring holds."""
    _compare_scan(kda, dtype, B, T, D, G, N)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_gradients_of_several_chunks_to_a_cta(kda, dtype):
    import torch
    lens, D, N = [200, 0, 1, 33, 400, 64], 4096, 16
    cu = [0] + np.cumsum(lens).tolist()
    a, kw, h0, dy, dh = _inputs(dtype, 1, cu[-1], D, 1, N, seqs=len(lens))
    got = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), **kw)
    y, h = kda.ssm_varlen_fwd(*a.values(), torch.tensor(cu, dtype=torch.int32, device="cuda"), h0, **kw)
    A, skip, bias = to_np(a["A"]), to_np(kw["skip"]), to_np(kw["dt_bias"])
    rows = [to_np(t) for t in (a["x"], a["dt"], a["B"], a["C"], kw["gate"], dy)]
    fwd = ref.packed(cu, lambda x, dt, B, C, z, d, s, e: ref.scan(x, dt, A, B, C, s, skip, z, bias), rows, [to_np(h0), to_np(dh)])
    _check_rows("y", y, np.concatenate([o[0] for o in fwd], 1), dtype, tight(400))
    _check32("h", h, np.concatenate([o[1] for o in fwd]), tight(400))
    want = ref.packed(cu, lambda x, dt, B, C, z, d, s, e: ref.scan(x, dt, A, B, C, s, skip, z, bias, grad=(d, e)), rows,
                      [to_np(h0), to_np(dh)])
    for k in ALL:
        if k in ROWS:
            _check_rows(k, got[k], np.concatenate([o[k] for o in want], 1), dtype, 2 * tight(400))
        else:
            _check32(k, got[k], np.concatenate([o[k] for o in want]) if k == "dh0" else sum(o[k] for o in want), 2 * tight(400))


# ------------------------------------------------------------------ scans: segments of two groups to a CTA
SEGMENTS = [(1, 2500, 512, 1, 16), (1, 2500, 480, 3, 16), (1, 2500, 511, 1, 16), (1, 2500, 510, 1, 16), (1, 2500, 250, 2, 32), (2, 2300, 72, 1, 64)]


def test_shapes_of_segments_of_two_groups(kda):
    """Among them odd numbers of channel blocks (the second group of a head's last CTA has no channels), rows off the
    boundary of what a lane loads, and rows that can be read by neither one load nor two elements."""
    for s in SEGMENTS:
        seg, pair = _two_groups(*s)
        assert seg and pair, s
    assert any(-(-D // G // (512 // N)) % 2 for _, _, D, G, N in SEGMENTS)


@gpu
@pytest.mark.parametrize("B,T,D,G,N", SEGMENTS)
def test_segments_of_two_groups(kda, B, T, D, G, N):
    _compare_scan(kda, "bf16", B, T, D, G, N, grads=False)


@gpu
def test_packed_segments_of_two_groups(kda):
    """With the host copy that tells the longest length, and without one."""
    import torch
    lens, D, N = [1400, 33, 0, 700, 1], 480, 16
    cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32)
    total = int(cu[-1])
    assert 1400 > 3 * (total * 15 // (2 * SMS))
    a, kw, h0, _, _ = _inputs("bf16", 1, total, D, 1, N, seqs=len(lens))
    A, skip, bias = to_np(a["A"]), to_np(kw["skip"]), to_np(kw["dt_bias"])
    want = ref.packed(cu.tolist(), lambda x, dt, B, C, z, s: ref.scan(x, dt, A, B, C, s, skip, z, bias),
                      [to_np(t) for t in (a["x"], a["dt"], a["B"], a["C"], kw["gate"])], [to_np(h0)])
    for host in (cu, None):
        y, h = kda.ssm_varlen_fwd(*a.values(), cu.cuda(), h0, cu_seqlens_cpu=host, **kw)
        _check_rows("y", y, np.concatenate([o[0] for o in want], 1), "bf16", tight(1400))
        _check32("h", h, np.concatenate([o[1] for o in want]), tight(1400))


# ------------------------------------------------------------------ scans: B and C
@gpu
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_fp32_heads_of_very_different_sizes(kda, N):
    """B and C from 1e-15 to 1e15 beside one another.  One token and nothing negative: y and h are sums of positive terms, each good to
    5e-7 of a time step and four roundings, 2^-24 each, and 16 or fewer additions: 2e-6 of every element."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(N)
    B, D, G = 40, 72, 2
    ru = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    x, dt, A = 0.5 + ru(B, 1, D), 2 * ru(B, 1, D) - 1, -0.5 - ru(D, N)
    Bm, Cm = (10.0 ** (30 * ru(B, 1, G, N) - 15) for _ in range(2))
    y, h = kda.ssm_chunk_fwd(x, dt, A, Bm, Cm)
    wy, wh = ref.scan(*(to_np(t) for t in (x, dt, A, Bm, Cm)))
    assert (np.abs(to_np(y) - wy) <= 2e-6 * wy).all() and (np.abs(to_np(h) - wh) <= 2e-6 * wh).all()


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("D", [48, 4096])
def test_heads_without_a_value_stay_in_their_group(kda, dtype, bad, D):
    """B that is infinite or NaN at one token reaches its group's memories from there on, C that token's outputs; neither another
    group, nor another sequence, nor a token before."""
    import torch
    a, kw, h0, _, _ = _inputs(dtype, 2, 100, D, 2, 16, gate=False)
    t0, half = 45, D // 2
    for name in ("B", "C"):
        m = dict(a, **{name: a[name].clone()})
        m[name][1, t0, 1, 5] = bad
        y, h = kda.ssm_chunk_fwd(*m.values(), h0, **kw)
        want = torch.zeros_like(y, dtype=torch.bool)
        want[1, t0:t0 + 1 if name == "C" else None, half:] = True
        assert torch.equal(~torch.isfinite(y), want)
        lost = ~torch.isfinite(h)
        assert not lost[0].any() and not lost[1, :half].any() and bool(lost[1, half:].any()) == (name == "B")
    st = h0.clone()
    m = {k: (v[:, t0] if k != "A" else v) for k, v in dict(a, B=a["B"].clone()).items()}
    m["B"][1, 1, 5] = bad
    y = kda.ssm_decode_step(*m.values(), st, **dict(kw, gate=None))
    want = torch.zeros_like(y, dtype=torch.bool)
    want[1, half:] = True
    assert torch.equal(~torch.isfinite(y), want) and bool(torch.isfinite(st[0]).all()) and bool(torch.isfinite(st[1, :half]).all())


# ------------------------------------------------------------------ convolution: long runs, several to a warp
CONV = [("bf16", 3, 700, 16384, 4), ("f32", 3, 700, 16384, 4), ("bf16", 7, 2000, 1023, 4), ("bf16", 3, 701, 16384, 2), ("f32", 3, 699, 16384, 3)]


def _runs(B, T, C):
    """(tokens of a run, runs, warps over a channel block) of the gradients."""
    blocks = -(-C // (128 if C % 4 == 0 else 32))
    warps = max(1, 2 * SMS // blocks) * 8
    most = warps * -(-B * T // (warps * 64))
    run = max(8, -(-B * T // most))
    while run < 64 and B * -(-T // run) > most:
        run += 1
    items = B * -(-T // run)
    parts = min(-(-items // 8), max(1, min(max(1, 4 * SMS // -(-C // 128)), 4 * SMS // blocks)))
    return run, items, parts * 8


def test_shapes_of_several_runs_to_a_warp():
    for _, B, T, C, _ in CONV:
        run, items, warps = _runs(B, T, C)
        assert run >= 3 + 2 * 6 and items > warps, (C, run, items, warps)


@gpu
@pytest.mark.parametrize("dtype,B,T,C,K", CONV)
def test_convolution_of_several_runs_to_a_warp(kda, dtype, B, T, C, K):
    """CONV = 1e-6 (fp32) beside a rounding; sums over up to 14,000 rows err like sqrt(n) 2^-24 = 7e-6: 1e-5."""
    import torch
    g, dt = torch.Generator(device="cuda").manual_seed(C + K), _dt(dtype)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w, b, s0, dy, ds = rn(B, T, C).to(dt), rn(C, K), rn(C), rn(B, K - 1, C).to(dt), rn(B, T, C).to(dt), rn(B, K - 1, C).to(dt)
    y, s = kda.conv_fwd(x, w, b, s0)
    got = kda.conv_bwd(dy, x, w, b, s0, ds)
    leaf = [t.double().requires_grad_(True) for t in (x, w, b, s0)]
    rows = torch.cat([leaf[3], leaf[0]], 1)
    p = leaf[2] + sum(leaf[1][:, j] * rows[:, j:j + T] for j in range(K))
    want = p * torch.sigmoid(p)
    grads = torch.autograd.grad([want, rows[:, T:]], leaf, [dy.double(), ds.double()])

    def rel(a, b):
        return float((a.double() - b).norm() / b.norm())

    def close(name, a, b):
        scale = float(b.square().mean().sqrt())
        off = (a.double() - b).abs() - (2.0 ** -8 * b.abs() if dtype == "bf16" else 0.0)
        assert float(off.max()) <= 1e-5 * scale, (name, float(off.max()) / scale)     # ten times CONV for the largest element
    close("y", y, want.detach())
    close("dx", got["dx"], grads[0])
    close("dstate", got["dstate"], grads[3])
    assert torch.equal(s, x[:, T - K + 1:])
    assert rel(got["dw"], grads[1]) <= 1e-5 and rel(got["dbias"], grads[2]) <= 1e-5


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,C,K,act", [(1, 8, 4, "silu"), (3, 250, 4, "silu"), (17, 64, 2, None), (5, 33, 3, "silu")])
def test_convolution_steps_have_the_prompts_bits(kda, dtype, B, C, K, act):
    """The same sums in the same order."""
    import torch
    g, dt, T = torch.Generator(device="cuda").manual_seed(C), _dt(dtype), 6
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w, b, st = rn(B, T, C).to(dt), rn(C, K), rn(C), rn(B, K - 1, C).to(dt)
    y, s = kda.conv_fwd(x, w, b, st, activation=act)
    for t in range(T):
        assert torch.equal(kda.conv_decode_step(x[:, t], w, st, b, activation=act), y[:, t])
    assert torch.equal(st, s)


# ------------------------------------------------------------------ selection: several parts of a row to a warp
SELECT = [(160, 8, 40011, 8), (64, 8, 131072, 8), (1300, 1, 20000, 5)]


def test_shapes_of_several_parts_to_a_warp(kda):
    for B, W, V, _ in SELECT:
        takes = -(-V // 1024)
        splits, left = divmod(kda.load().kda_beam_select_workspace(B, W, V, 1) - 256 - B * W * 2 * takes * 4, B * W * 16)
        assert left == 0 and takes > 2 * 8 * splits, (B, W, V, splits)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,W,V,k", SELECT)
@pytest.mark.parametrize("trend", ["rises", "falls", "waves"])
def test_selection_whose_maxima_change_along_the_row(kda, dtype, B, W, V, k, trend):
    """A warp's sum is carried on from maximum to maximum.  A sum of exp errs by at most the rounding of its exponents, 2^-24 of up to 14
    (what is further below the maximum has no weight), and of exp2, 2^-22.5: totals by 1e-6 and their rounding, 2^-24.  Beams
    whose totals are nearer to one another than twice that may come in either order, tokens of a beam may not."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(V)
    at = torch.linspace(0, 1, V, device="cuda")
    slope = {"rises": 40 * at, "falls": -40 * at, "waves": 15 * torch.sin(40 * at)}[trend]
    x = (3 * torch.randn((B, W, V), generator=g, device="cuda") + slope).to(_dt(dtype))
    s = -torch.rand((B, W), generator=g, device="cuda").cumsum(1) * 2 - 5
    got = kda.beam_select(x, s, k)
    d = x.double()
    total = (s.double()[..., None] + d - torch.logsumexp(d, -1, keepdim=True)).flatten(1)
    best = total.topk(k, 1)[0]
    flat = got[1].long() * V + got[2].long()
    mine = total.gather(1, flat)
    assert int(got[2].min()) >= 0 and int(got[2].max()) < V and int(got[1].min()) >= 0 and int(got[1].max()) < W
    assert float((mine - best).abs().max()) <= 2e-6
    assert float((got[0].double() - mine).abs().sub(2.0 ** -24 * mine.abs()).max()) <= 1e-6
    picked = d.flatten(1).gather(1, flat)
    later = torch.ones(k, k, device="cuda", dtype=torch.bool).triu(1)
    same = (got[1][:, :, None] == got[1][:, None, :]) & later
    order = (picked[:, :, None] > picked[:, None, :]) | ((picked[:, :, None] == picked[:, None, :]) & (got[2][:, :, None] < got[2][:, None, :]))
    assert bool(order[same].all())


@gpu
def test_totals_that_fp32_cannot_tell_apart_keep_their_order(kda):
    """Scores 2^-23 apart, candidates 60 below the best: totals of -61, whose fp32 neighbours are 2^-18 away, are returned equal and
    are in order all the same."""
    import torch
    x = torch.full((1, 2, 700), float("-inf"), device="cuda")
    x[..., 0], x[..., 600] = 0.0, -60.0
    s = torch.tensor([[-1.0, -1.0 + 2.0 ** -23]], device="cuda")
    got = kda.beam_select(x, s, 4)
    assert got[1].tolist() == [[1, 0, 1, 0]] and got[2].tolist() == [[0, 0, 600, 600]]
    assert float(got[0][0, 2]) == float(got[0][0, 3])
    got = kda.beam_select(x, s.flip(1).contiguous(), 4)
    assert got[1].tolist() == [[0, 1, 0, 1]]


# ------------------------------------------------------------------ packed batches of many sequences
def _scan64(x, dt, A, B, C, h, skip, gate, bias, cu):
    """Packed sequences in fp64, side by side: rows [total,..] of one group, h [N,D,S]; (y [total,D], the memories after)."""
    import torch
    lens = (cu[1:] - cu[:-1]).long()
    y, places = [], []
    for t in range(int(lens.max())):
        live = torch.nonzero(lens > t)[:, 0]
        r = cu[:-1].long()[live] + t
        step = torch.nn.functional.softplus(dt[r] + bias, threshold=50.0)
        new = torch.exp(step[..., None] * A) * h[live] + (step * x[r])[..., None] * B[r][:, None]
        h = h.index_copy(0, live, new)
        out = ((new * C[r][:, None]).sum(-1) + skip * x[r]) * gate[r] * torch.sigmoid(gate[r])
        y.append(out)
        places.append(r)
    order = torch.cat(places).argsort()
    return torch.cat(y)[order], h


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,most,D,S", [(512, 40, 24, 16), (513, 40, 24, 16), (1100, 9, 24, 16), (600, 300, 33, 8), (33000, 1, 24, 8),
                                        (2000, 3, 700, 16)])
def test_packed_batches_of_many_sequences(kda, dtype, N, most, D, S):
    """A sequence or its part is found among any number of them: lengths from none on, multiples of a chunk and of a segment among
    them, split into segments (no host copy, few channels) and not."""
    import torch
    lens = torch.randint(0, most + 1, (N,), generator=torch.Generator().manual_seed(N))
    lens[::5] = lens[::5] // 32 * 32
    lens[1::7] = 0
    lens[3] = min(128, 32 * most)
    lens[-1] = 0
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    cud, total, T = cu.cuda(), int(cu[-1]), int(lens.max())
    a, kw, h0, dy, dh = _inputs(dtype, 1, total, D, 1, S, seqs=N)
    leaf = dict(dx=a["x"][0], ddt=a["dt"][0], dA=a["A"], dB=a["B"][0, :, 0], dC=a["C"][0, :, 0], dh0=h0, dskip=kw["skip"], dgate=kw["gate"][0],
                ddt_bias=kw["dt_bias"])
    leaf = {k: v.double().requires_grad_(True) for k, v in leaf.items()}
    wy, wh = _scan64(*leaf.values(), cud)
    for host in (None, cu):
        y, h = kda.ssm_varlen_fwd(*a.values(), cud, h0, cu_seqlens_cpu=host, **kw)
        _check_rows("y", y[0], to_np(wy.detach()), dtype, tight(T))
        _check32("h", h, to_np(wh.detach()), tight(T))
    got = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, cu_seqlens=cud, **kw)
    want = torch.autograd.grad([wy, wh], list(leaf.values()), [dy[0].double(), dh.double()])
    assert set(got) == set(leaf)
    for k, v in zip(leaf, want):
        if k in ROWS:
            _check_rows(k, got[k].reshape(v.shape), to_np(v), dtype, 2 * tight(T))
        else:
            _check32(k, got[k], to_np(v), 2 * tight(T))


@gpu
def test_packed_batch_of_a_chunks_rows(kda):
    """32 rows of 600 sequences: the empty ones behind them have their chunks too."""
    import torch
    cu = torch.full((601,), 32, dtype=torch.int32, device="cuda")
    cu[0] = 0
    a, kw, h0, dy, dh = _inputs("f32", 1, 32, 24, 1, 16, seqs=600)
    _, h = kda.ssm_varlen_fwd(*a.values(), cu, h0, **kw)
    assert torch.equal(h[1:], h0[1:])
    one = kda.ssm_chunk_bwd(dy, *a.values(), h0[:1], dh[:1], **kw)
    got = kda.ssm_chunk_bwd(dy, *a.values(), h0, dh, cu_seqlens=cu, **kw)
    assert torch.equal(got["dh0"][1:], dh[1:]) and torch.equal(got["dh0"][:1], one["dh0"])
    assert torch.equal(got["dx"], one["dx"]) and torch.equal(got["dB"], one["dB"])


@gpu
def test_many_short_sequences_cost_what_their_tokens_do(kda):
    """A token for each of 40,000 sequences: packed it is the work of a batch of that many, gradients too: 4.7 ms (two launches, since
    without a host copy of the lengths it is split) and 2.4, 5.8 and 5.2 (counting all the sequences before one's own, for each of them,
    took 19 and 8 times as long as that already at 16,384; four times the batch's are allowed)."""
    import torch
    N = 40000
    a, kw, _, dy, _ = _inputs("bf16", N, 1, 128, 1, 16, h0=False)
    p = {k: (v if k == "A" else v.transpose(0, 1)) for k, v in a.items()}
    pw = dict(kw, gate=kw["gate"].transpose(0, 1))
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    calls = [(lambda: kda.ssm_varlen_fwd(*p.values(), cu, **pw), lambda: kda.ssm_chunk_fwd(*a.values(), **kw)),
             (lambda: kda.ssm_chunk_bwd(dy.transpose(0, 1), *p.values(), cu_seqlens=cu, **pw), lambda: kda.ssm_chunk_bwd(dy, *a.values(), **kw))]

    def ms(call):
        call()
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(5)]
        for e in ev:
            e.record()
            call()
        torch.cuda.synchronize()
        return min(a.elapsed_time(b) for a, b in zip(ev, ev[1:]))
    for packed, batch in calls:
        t = ms(packed), ms(batch)
        assert t[0] <= 4 * t[1], t
    y, h = calls[0][0]()
    wy, wh = calls[0][1]()
    assert torch.equal(y[0], wy[:, 0]) and torch.equal(h, wh)
