"""The binding of the short convolution, the state space scan and beam search on the host: what is refused before a launch
and what is asked after it (the library and the tensors' device are stood in for: nothing is launched), and an order in the
scan kernel's source on which its launches' progress rests."""
import os
import re

import pytest
import torch

import delta_rule_linear_gb300 as kda
from delta_rule_linear_gb300 import _linear
from test_linear_binding import _Lib, _on_device, _zeros

I32 = torch.int32


@pytest.fixture
def lib(monkeypatch):
    lib, sizes = _Lib(), _linear._bytes
    sizes.cache_clear()
    monkeypatch.setattr(_linear, "load", lambda: lib)
    monkeypatch.setattr(_linear, "_raw", lambda t: 0)
    monkeypatch.setattr(_linear, "_here", lambda: 0)
    monkeypatch.setattr(_linear, "query_device_error", lambda ws: 8)
    yield lib
    sizes.cache_clear()


def _scan(i=0, T=4, D=8, N=16):
    z = lambda *s: _zeros(*s, index=i)  # noqa: E731
    return z(1, T, D), z(1, T, D), z(D, N), z(1, T, 1, N), z(1, T, 1, N)


def _step(i=0):
    x, dt, A, B, C = _scan(i)
    return x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0]


# each call of tensors of which the last is on device j, the others on device i
_CALLS = {
    "conv_fwd": lambda i, j: kda.conv_fwd(_zeros(1, 4, 8, index=i), _zeros(8, 4, index=i), _zeros(8, index=j)),
    "conv_varlen_fwd": lambda i, j: kda.conv_varlen_fwd(_zeros(1, 4, 8, index=i), _zeros(8, 4, index=i), _zeros(2, dtype=I32, index=j)),
    "conv_decode_step": lambda i, j: kda.conv_decode_step(_zeros(2, 8, index=i), _zeros(8, 4, index=i), _zeros(2, 3, 8, index=j)),
    "conv_bwd": lambda i, j: kda.conv_bwd(_zeros(1, 4, 8, index=j), _zeros(1, 4, 8, index=i), _zeros(8, 4, index=i)),
    "ssm_chunk_fwd": lambda i, j: kda.ssm_chunk_fwd(*_scan(i), _zeros(1, 8, 16, index=j)),
    "ssm_chunk_fwd gate": lambda i, j: kda.ssm_chunk_fwd(*_scan(i), gate=_zeros(1, 4, 8, index=j)),
    "ssm_varlen_fwd": lambda i, j: kda.ssm_varlen_fwd(*_scan(i), _zeros(2, dtype=I32, index=j)),
    "ssm_decode_step": lambda i, j: kda.ssm_decode_step(*_step(i), _zeros(1, 8, 16, index=j)),
    "ssm_chunk_bwd": lambda i, j: kda.ssm_chunk_bwd(_zeros(1, 4, 8, index=j), *_scan(i)),
    "beam_select": lambda i, j: kda.beam_select(_zeros(2, 3, 50, index=i), _zeros(2, 3, index=j)),
    "beam_reorder": lambda i, j: kda.beam_reorder([_zeros(6, 5, index=j)], _zeros(2, 3, dtype=I32, index=i)),
}


@pytest.mark.parametrize("name", list(_CALLS))
def test_tensors_of_another_device_are_refused(lib, name):
    _CALLS[name](0, 0)
    assert len(lib.launched) == 1
    for devices in ((0, 1), (1, 0), (1, 1)):
        with pytest.raises(ValueError, match="device"):
            _CALLS[name](*devices)
    assert len(lib.launched) == 1


@pytest.mark.parametrize("name", ["conv_bwd", "ssm_chunk_fwd", "ssm_varlen_fwd", "ssm_chunk_bwd", "beam_select"])
def test_a_workspace_is_whole_and_on_the_device(lib, name):
    x, w = _zeros(1, 4, 8), _zeros(8, 4)
    call = {"conv_bwd": lambda ws: kda.conv_bwd(x, x, w, workspace=ws),
            "ssm_chunk_fwd": lambda ws: kda.ssm_chunk_fwd(*_scan(), workspace=ws),
            "ssm_varlen_fwd": lambda ws: kda.ssm_varlen_fwd(*_scan(), _zeros(2, dtype=I32), workspace=ws),
            "ssm_chunk_bwd": lambda ws: kda.ssm_chunk_bwd(x, *_scan(), workspace=ws),
            "beam_select": lambda ws: kda.beam_select(_zeros(2, 3, 50), _zeros(2, 3), workspace=ws)}[name]
    call(_zeros(4096))
    assert len(lib.launched) == 1
    for ws in (torch.zeros(4096), _zeros(4096, index=1), _on_device(torch.zeros(4096)[::2]), _on_device(torch.zeros(1).expand(4096))):
        with pytest.raises(ValueError, match="workspace"):
            call(ws)
    assert len(lib.launched) == 1


def test_outputs_are_no_broadcast_views(lib):
    into = lambda *s: _on_device(torch.zeros(s[-1]).expand(*s))  # noqa: E731
    x, w = _zeros(1, 4, 8), _zeros(8, 4)
    for call in (lambda: kda.conv_fwd(x, w, out=into(1, 4, 8)), lambda: kda.conv_decode_step(_zeros(2, 8), w, _zeros(2, 3, 8), out=into(2, 8)),
                 lambda: kda.ssm_chunk_fwd(*_scan(), out=into(1, 4, 8)), lambda: kda.ssm_decode_step(_zeros(2, 8), _zeros(2, 8), _zeros(8, 16), _zeros(2, 16), _zeros(2, 16), _zeros(2, 8, 16), out=into(2, 8))):
        with pytest.raises(ValueError, match="broadcast"):
            call()
    assert not lib.launched


def test_shapes_and_types_are_refused(lib):
    x, dt, A, B, C = _scan()
    w, cu = _zeros(8, 4), _zeros(2, dtype=I32)
    bf = lambda t: _on_device(t.as_subclass(torch.Tensor).bfloat16())  # noqa: E731
    for call in (lambda: kda.conv_fwd(x, bf(w)), lambda: kda.ssm_chunk_fwd(x, bf(dt), A, B, C), lambda: kda.ssm_chunk_fwd(x, dt, bf(A), B, C),
                 lambda: kda.ssm_chunk_fwd(x, dt, A, bf(B), C), lambda: kda.conv_varlen_fwd(x, w, _zeros(2)),
                 lambda: kda.beam_select(_zeros(2, 3, 50), _zeros(2, 3), finished=_zeros(2, 3), eos=1),
                 lambda: kda.conv_decode_step(x[:, 0], w, bf(_zeros(1, 3, 8))), lambda: kda.conv_fwd(_on_device(torch.zeros(1, 4, 8).half()), w)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: kda.conv_fwd(x, _zeros(7, 4)), lambda: kda.conv_fwd(x, w, _zeros(7)), lambda: kda.conv_fwd(x, w, None, _zeros(1, 4, 8)),
                 lambda: kda.conv_varlen_fwd(_zeros(2, 4, 8), w, cu), lambda: kda.conv_decode_step(x, w, _zeros(1, 3, 8)),
                 lambda: kda.ssm_chunk_fwd(x, dt, A, _zeros(1, 4, 3, 16), _zeros(1, 4, 3, 16)), lambda: kda.ssm_chunk_fwd(x, dt, A, B, C[:, :, 0]),
                 lambda: kda.ssm_chunk_fwd(x, dt, A, B, _zeros(1, 4, 2, 16)), lambda: kda.ssm_chunk_fwd(x, dt, A[0], B, C),
                 lambda: kda.ssm_chunk_fwd(x, dt, A, _zeros(1, 4, 1, 8), C), lambda: kda.ssm_varlen_fwd(x, dt, A, B, C, cu, cu_seqlens_cpu=torch.zeros(3)),
                 lambda: kda.ssm_chunk_fwd(x, dt, A, B, C, _zeros(1, 8, 8)), lambda: kda.ssm_chunk_bwd(_zeros(1, 3, 8), x, dt, A, B, C),
                 lambda: kda.beam_select(_zeros(2, 3, 50), _zeros(2, 4)), lambda: kda.beam_select(_zeros(3, 50), _zeros(3)),
                 lambda: kda.beam_select(_zeros(2, 3, 50), _zeros(2, 3), finished=_zeros(2, 3, dtype=torch.bool))):
        with pytest.raises(ValueError):
            call()
    assert not lib.launched
    kda.ssm_chunk_fwd(x, dt, A, B[:, :, 0], C[:, :, 0])           # one group without its dimension
    assert len(lib.launched) == 1


def test_check_device_asks_for_the_error_word(lib):
    x, dt, A, B, C = _scan()
    for call in (lambda **k: kda.ssm_chunk_fwd(x, dt, A, B, C, **k), lambda **k: kda.ssm_varlen_fwd(x, dt, A, B, C, _zeros(2, dtype=I32), **k)):
        call()
        with pytest.raises(kda.KdaError):
            call(check_device=True)
    e = [t[:0] for t in (x, dt)] + [A] + [t[:0] for t in (B, C)]
    kda.ssm_chunk_fwd(*e, check_device=True)        # an empty batch has none


def test_the_next_launch_may_start_only_after_the_tmem_allocation():
    """A CTA of the second launch of a split scan takes TMEM and then waits for the first launch: that one has to have its
    own by then, which a barrier after the allocation makes sure of (read from the text: a wrong order would hang)."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "delta_rule_linear_gb300", "csrc", "ssm_scan.cu")
    with open(path) as f:
        body = re.split(r"ssm_scan_kernel\(", re.sub(r"//[^\n]*", "", f.read()))[1]
    alloc = body.index("tmem_alloc(")
    barrier = body.index("__syncthreads()", alloc)
    calls = [m.start() for m in re.finditer(r"next_may_start\(", body)]
    # before it only on the way out of a CTA that has nothing to do
    assert any(c > barrier for c in calls) and all(c > barrier or "return;" in body[c:c + 120] for c in calls)
