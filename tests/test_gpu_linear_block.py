"""The linear-attention block of examples/linear_block.py: its kernels together, as a model runs them."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "linear_block.py")
    spec = importlib.util.spec_from_file_location("linear_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _inputs(B, T, D, dtype, seed=3):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((B, T, D), generator=g, device="cuda"),
            torch.randn((B, T, D), generator=g, device="cuda").to(dtype), g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_served_tokens_equal_the_prefill(block, dtype):
    """Two bf16 paths through the same block: every bf16 intermediate of either may differ by its
    rounding, 2^-8 of a value each over about six roundings in a row: 2.4e-2.  fp32: 1e-4."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    p = block.make_params(256, H=2, m=2, dk=64, dv=64, dtype=dt)
    x, y, _ = _inputs(3, 150, 256, dt)
    _, n, h, _ = block.forward(p, x, y)
    got, hs = block.serve(p, x, y, 140)
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
    assert rel(got, n) <= (1e-4 if dtype == "f32" else 2.4e-2)
    assert rel(hs, h) <= (1e-4 if dtype == "f32" else 2.4e-2)


@pytest.mark.parametrize("name", ["x", "y", "w_in", "w_gate", "w_out", "A_log", "dt_bias", "W", "Wo", "state"])
def test_training_gradients_equal_differences(block, name):
    """fp32: the loss is about 1 with rounding of some 1e-6, so central differences over steps of 1e-2 (of
    directions normalised to the parameter's size) are good to 1e-4 of the loss and their curvature."""
    import torch
    torch.backends.cuda.matmul.allow_tf32 = False
    p = block.make_params(128, H=2, m=2, dk=32, dv=64, dtype=torch.float32)
    x, y, g = _inputs(2, 70, 128, torch.float32)
    state = 0.1 * torch.randn((2, 4, 32, 64), generator=g, device="cuda")
    _, n, h, saved = block.forward(p, x, y, state)
    dn = torch.randn(n.shape, generator=g, device="cuda") / n.numel() ** 0.5
    dh = torch.randn(h.shape, generator=g, device="cuda") / h.numel() ** 0.5
    got = block.backward(p, saved, dn, None, dh)[name]
    base = dict(p, x=x, y=y, state=state)
    d = torch.randn(base[name].shape, generator=g, device="cuda")
    d *= base[name].double().norm().float() / d.norm()

    def loss(e):
        a = dict(base, **{name: base[name] + e * d})
        _, nn, hh, _ = block.forward({k: a[k] for k in p}, a["x"], a["y"], a["state"])
        return float((nn.double() * dn.double()).sum() + (hh.double() * dh.double()).sum())
    e = 1e-2
    num = (loss(e) - loss(-e)) / (2 * e)
    ana = float((got.double() * d.double()).sum())
    assert np.isfinite(ana) and abs(num - ana) <= 2e-2 * max(abs(ana), 0.1), (num, ana)


def test_example_runs(block, capsys):
    block.main()
    assert "training step" in capsys.readouterr().out
