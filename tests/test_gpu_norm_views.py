"""The block norms on views whose leading dimensions are of size 1 or cut: the same bits as of contiguous copies, or a
refusal where no one stride leads from row to row."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import delta_rule_linear_gb300 as m
    m.load()
    return m


def _rand(*s, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*s, generator=g, device="cuda")


def _cuts(D):
    """Views [.., D] with one stride from row to row."""
    return {"last token": _rand(6, 4, D)[:, -1:], "one": _rand(1, 9, D)[:, 2:7], "every other": _rand(8, 1, D)[::2],
            "between": _rand(2, 1, 8, D)[:, :, 3], "wide": _rand(2, 1, 5, D + 8)[..., :D]}


@pytest.mark.parametrize("D", [64, 77])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_residual_norm_of_cut_views(kda, D, dtype):
    import torch
    dt = getattr(torch, dtype)
    w = 1 + 0.1 * _rand(D, seed=1)
    for name, x in _cuts(D).items():
        y = _rand(*x.shape, seed=2).to(dt)
        want = kda.residual_norm_fwd(x.contiguous(), y, w, scale=0.5)
        got = kda.residual_norm_fwd(x, y, w, scale=0.5)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        yv = torch.empty(*y.shape[:-1], D + 8, device="cuda", dtype=dt)[..., :D]
        yv.copy_(y)
        got = kda.residual_norm_fwd(x, yv, w, scale=0.5)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


@pytest.mark.parametrize("D", [64, 77])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gated_norm_of_cut_views_and_into_them(kda, D, dtype):
    import torch
    dt = getattr(torch, dtype)
    w = 1 + 0.1 * _rand(D, seed=1)
    for name, x in _cuts(3 * D).items():
        x = x.to(dt).unflatten(-1, (3, D)) if name == "wide" else x.unflatten(-1, (3, D)).to(dt)
        big = torch.full((*x.shape[:-2], 5, D), 7.0, device="cuda", dtype=dt)
        gate, dy = _rand(*x.shape, seed=3).to(dt), _rand(*x.shape, seed=4).to(dt)
        want = kda.gated_norm_fwd(x.contiguous(), gate, w)
        assert torch.equal(kda.gated_norm_fwd(x, gate, w), want), name
        g0, g1 = kda.gated_norm_bwd(dy, x, gate, w), kda.gated_norm_bwd(dy, x.contiguous(), gate, w)
        assert all(torch.equal(g0[n], g1[n]) for n in g0), name
        kda.gated_norm_fwd(x, gate, w, out=big[..., 1:4, :])
        assert torch.equal(big[..., 1:4, :], want) and (big[..., 0, :] == 7).all() and (big[..., 4, :] == 7).all()


def test_views_without_one_stride_are_refused(kda):
    """[2, 1, 8, ...] cut in its third dimension: behind row 4 comes row 8, not row 5."""
    import torch
    w = torch.ones(64, device="cuda")
    x, y = _rand(2, 1, 8, 64)[:, :, :5], _rand(2, 1, 5, 64)
    for call in (lambda: kda.residual_norm_fwd(x, y, w), lambda: kda.residual_norm_fwd(y, x, w)):
        with pytest.raises(ValueError, match="step evenly"):
            call()
    x, y = _rand(2, 1, 8, 3, 64)[:, :, :5], _rand(2, 1, 5, 3, 64)
    for call in (lambda: kda.gated_norm_fwd(x, y, w), lambda: kda.gated_norm_fwd(y, x, w),
                 lambda: kda.gated_norm_fwd(y, y, w, out=x), lambda: kda.gated_norm_bwd(x, y, y, w)):
        with pytest.raises(ValueError, match="step evenly"):
            call()
