"""The state space block of examples/ssm_block.py: its kernels together, as a model runs them."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ssm_block.py")
    spec = importlib.util.spec_from_file_location("ssm_block", path)
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
    """Two bf16 paths through the same block: every bf16 intermediate of either may differ by its rounding, 2^-8 of a
    value each over about eight roundings in a row: 3.2e-2.  fp32: 1e-4."""
    import torch
    torch.backends.cuda.matmul.allow_tf32 = False
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    p = block.make_params(256, Di=320, rank=24, V=64, dtype=dt)
    x, y, _ = _inputs(3, 150, 256, dt)
    _, n, win, h, _ = block.forward(p, x, y)
    got, ws, hs = block.serve(p, x, y, 140)
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
    tol = 1e-4 if dtype == "f32" else 3.2e-2
    assert rel(got, n) <= tol and rel(ws, win) <= tol and rel(hs, h) <= tol


@pytest.mark.parametrize("name", ["x", "y", "w_in", "w_out", "conv_w", "conv_b", "A_log", "skip", "dt_bias", "W", "Wx", "Wdt", "Wo",
                                  "window", "state"])
def test_training_gradients_equal_differences(block, name):
    """fp32: the loss is about 1 with rounding of some 1e-6, so central differences over steps of 1e-2 (of directions
    normalised to the parameter's size) are good to 1e-4 of the loss and their curvature."""
    import torch
    torch.backends.cuda.matmul.allow_tf32 = False
    p = block.make_params(128, Di=160, rank=16, V=64, dtype=torch.float32)
    x, y, g = _inputs(2, 70, 128, torch.float32)
    window = torch.randn((2, block.K - 1, 160), generator=g, device="cuda")
    state = 0.3 * torch.randn((2, 160, 16), generator=g, device="cuda")
    _, n, win, h, saved = block.forward(p, x, y, window, state)
    rn = lambda t: torch.randn(t.shape, generator=g, device="cuda") / t.numel() ** 0.5  # noqa: E731
    dn, dw, dh = rn(n), rn(win), rn(h)
    got = block.backward(p, saved, dn, None, dw, dh)[name]
    base = dict(p, x=x, y=y, window=window, state=state)
    d = torch.randn(base[name].shape, generator=g, device="cuda")
    d *= base[name].double().norm().float() / d.norm()

    def loss(e):
        a = dict(base, **{name: base[name] + e * d})
        _, nn, ww, hh, _ = block.forward({k: a[k] for k in p}, a["x"], a["y"], a["window"], a["state"])
        return sum(float((s.double() * t.double()).sum()) for s, t in ((nn, dn), (ww, dw), (hh, dh)))
    e = 1e-2
    num = (loss(e) - loss(-e)) / (2 * e)
    ana = float((got.double() * d.double()).sum())
    assert np.isfinite(ana) and abs(num - ana) <= 2e-2 * max(abs(ana), 0.1), (num, ana)


def test_beam_scores_are_the_sequences_log_probabilities(block):
    """Each beam's score is what a prefill of its whole sequence gives its tokens: the windows and memories followed the
    beams.  fp32: some 1e-4 of a log probability a token."""
    import torch
    torch.backends.cuda.matmul.allow_tf32 = False
    B, W, new, V, eos = 3, 4, 9, 50, 7
    p = block.make_params(64, Di=96, rank=8, V=V, dtype=torch.float32, seed=2)
    prompt = torch.randint(0, V, (B, 11), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    seqs, scores = block.search(p, prompt, W, new, eos)
    assert bool((scores[:, :-1] >= scores[:, 1:]).all())
    full = torch.cat([prompt[:, None].expand(B, W, -1), seqs.long()], -1).flatten(0, 1)
    n = block.forward(p, *block.tokens_in(p, full[:, :-1]))[1]
    lp = torch.log_softmax((n @ p["embed"].T).double(), -1)[:, prompt.shape[1] - 1:]
    each = lp.gather(-1, seqs.flatten(0, 1).long()[..., None])[..., 0]
    done = (seqs.flatten(0, 1) == eos).cumsum(-1) - (seqs.flatten(0, 1) == eos).int()
    want = torch.where(done > 0, 0.0, each).sum(-1).unflatten(0, (B, W))
    assert float((scores.double() - want).abs().max()) <= 1e-4 * new
    rows = {tuple(s) for s in seqs[0].tolist()}
    assert len(rows) == W                   # beams are different sequences


def test_example_runs(block, capsys):
    block.main()
    assert "training step" in capsys.readouterr().out
