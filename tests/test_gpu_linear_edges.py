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
