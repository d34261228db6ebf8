"""The binding of linear attention and the block norms on the host: which rows a view's strides name, what is refused
before a launch and what is asked after it (the library and the tensors' device are stood in for: nothing is launched)."""
import itertools

import pytest
import torch

import delta_rule_linear_gb300 as kda
from delta_rule_linear_gb300 import _linear


# ------------------------------------------------------------------------------ strides
def _views():
    """Views whose leading dimensions may be of size 1 and may be slices, named by how they are made."""
    for sizes in itertools.product((1, 2, 3), repeat=3):
        for cut in range(4):
            for axis in range(3):
                big = [s + (2 if cut & 1 and i == axis else 0) for i, s in enumerate(sizes)]
                x = torch.empty(*big, 2, 8 if cut & 2 else 5)
                yield f"{sizes} {axis} {cut}", x.narrow(axis, 1 if cut & 1 else 0, sizes[axis])[..., :5]
    x = torch.empty(4, 6, 2, 5)
    yield "last token", x[:, -1:]
    yield "one request", x[:1, 1:4]
    yield "heads first", x.transpose(1, 2)
    yield "every other", x[::2, ::2]
    yield "broadcast", torch.empty(1, 1, 2, 5).expand(3, 4, 2, 5)
    yield "two rows", torch.empty(2, 1, 8, 2, 8)[:, :, :5, :, :5]


def _offsets(t, lead):
    """Offsets of the places of the first `lead` dimensions, in order."""
    return [sum(i * s for i, s in zip(at, t.stride())) for at in itertools.product(*(range(n) for n in t.shape[:lead]))]


def _even(offs):
    return all(o == i * (offs[1] if len(offs) > 1 else 0) for i, o in enumerate(offs))


@pytest.mark.parametrize("name,t", list(_views()), ids=lambda x: x if isinstance(x, str) else "")
def test_one_stride_reaches_every_row_or_the_view_is_refused(name, t):
    """Rows [..., D] and tokens [..., H, D]: row i lies at i times the stride, or no stride says where."""
    rows = t.flatten(-2) if t.is_contiguous() else t[..., 0, :]
    for x, lead, get in ((rows, rows.dim() - 1, lambda x: _linear._rows(x, x.shape[-1])),
                         (t, t.dim() - 2, lambda x: _linear._token_strides(x)[0])):
        offs = _offsets(x, lead)
        if _even(offs):
            step = get(x)
            assert offs == [i * step for i in range(len(offs))]
        else:
            with pytest.raises(ValueError, match="step evenly"):
                get(x)


def test_the_head_stride_of_one_head_is_its_width():
    """One head: no other head is looked for, and an odd stride must not cost the wide loads."""
    t = torch.empty(7, 3, 64)[:, :1].transpose(0, 1)[:, :1]
    assert t.shape == (1, 1, 64) and _linear._token_strides(torch.empty(5, 9, 64)[:, 3:4])[1] == 64
    assert _linear._token_strides(t)[1] == 64


# ------------------------------------------------------------------------------ refusals
@pytest.mark.parametrize("activation", [None, "tanh", "SiLU", 1])
def test_a_gate_needs_one_of_the_two_activations(activation):
    """Without one the kernels would take no gate: the forward would drop it, and its gradient would never be written."""
    x, w = torch.zeros(2, 3, 8), torch.ones(8)
    for call in (lambda: kda.gated_norm_fwd(x, x, w, activation=activation),
                 lambda: kda.gated_norm_bwd(x, x, x, w, activation=activation)):
        with pytest.raises(ValueError, match="activation"):
            call()


# ------------------------------------------------------------------------------ calls of a library that is stood in for
class _Cuda(torch.Tensor):
    """Host memory that calls itself a CUDA tensor of device ``index``."""
    index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


def _on_device(t, index=0):
    t = t.as_subclass(_Cuda)
    t.index = index
    return t


class _Lib:
    """Every call succeeds and is counted; the error word of every workspace says that a wait ran out."""

    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return lambda *a: 512
        if name == "kda_status_string":
            return lambda code: b"status"

        def call(*a):
            self.launched.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib, sizes = _Lib(), _linear._bytes
    sizes.cache_clear()
    monkeypatch.setattr(_linear, "load", lambda: lib)
    monkeypatch.setattr(_linear, "_raw", lambda t: 0)
    monkeypatch.setattr(_linear, "_here", lambda: 0, raising=False)
    monkeypatch.setattr(_linear, "query_device_error", lambda ws: 8)
    yield lib
    sizes.cache_clear()


def _zeros(*s, dtype=torch.float32, index=0):
    return _on_device(torch.zeros(*s, dtype=dtype), index)


def test_an_empty_batch_has_no_error_word(lib):
    """No kernel runs and none clears the header, so what a fresh workspace holds must not be read as an error."""
    x, cu = _zeros(0, 4, 1, 32), _zeros(1, dtype=torch.int32)
    p = _zeros(1, 0, 1, 32)
    for call in (lambda x: kda.linear_chunk_fwd(x, x, x, check_device=True),
                 lambda x: kda.linear_chunk_bwd(x, x, x, None, None, x, check_device=True)):
        call(x)
        with pytest.raises(kda.KdaError):          # with sequences, the word is asked for
            call(_zeros(2, 4, 1, 32))
    kda.linear_varlen_fwd(p, p, p, cu, check_device=True)
    with pytest.raises(kda.KdaError):
        kda.linear_varlen_fwd(p, p, p, _zeros(3, dtype=torch.int32), check_device=True)


_CU = lambda i: _zeros(2, dtype=torch.int32, index=i)  # noqa: E731
# each call of tensors of which the last is on device j, the others on device i
_CALLS = {
    "chunk_fwd": lambda i, j: kda.linear_chunk_fwd(*(_zeros(1, 4, 1, 32, index=i) for _ in range(3)),
                                                   _zeros(1, 4, 1, index=i), _zeros(1, 1, 32, 32, index=j)),
    "chunk_fwd out": lambda i, j: kda.linear_chunk_fwd(*(_zeros(1, 4, 1, 32, index=i) for _ in range(3)),
                                                       out=_zeros(1, 4, 1, 32, index=j)),
    "varlen_fwd": lambda i, j: kda.linear_varlen_fwd(*(_zeros(1, 4, 1, 32, index=i) for _ in range(3)), _CU(j)),
    "decode_step": lambda i, j: kda.linear_decode_step(*(_zeros(1, 1, 1, 32, index=i) for _ in range(3)), None,
                                                       _zeros(1, 1, 32, 32, index=j)),
    "chunk_bwd": lambda i, j: kda.linear_chunk_bwd(*(_zeros(1, 4, 1, 32, index=i) for _ in range(3)), None, None,
                                                   _zeros(1, 4, 1, 32, index=j)),
    "gated_norm_fwd": lambda i, j: kda.gated_norm_fwd(_zeros(2, 3, 8, index=i), _zeros(2, 3, 8, index=i), _zeros(8, index=j)),
    "gated_norm_bwd": lambda i, j: kda.gated_norm_bwd(_zeros(2, 3, 8, index=j), _zeros(2, 3, 8, index=i),
                                                      _zeros(2, 3, 8, index=i), _zeros(8, index=i)),
    "residual_norm_fwd": lambda i, j: kda.residual_norm_fwd(_zeros(2, 8, index=i), _zeros(2, 8, index=i), _zeros(8, index=i),
                                                            scale=_zeros(8, index=j)),
    "residual_norm_bwd": lambda i, j: kda.residual_norm_bwd(_zeros(2, 8, index=i), None, _zeros(2, 8, index=i),
                                                            _zeros(8, index=i), _zeros(2, 8, index=j)),
}


@pytest.mark.parametrize("name", list(_CALLS))
def test_tensors_of_another_device_are_refused(lib, name):
    """The kernels run on the current device, on the stream of that number there: tensors of another device would be
    reached through the wrong stream, or not at all."""
    _CALLS[name](0, 0)
    assert len(lib.launched) == 1
    for devices in ((0, 1), (1, 0), (1, 1)):
        with pytest.raises(ValueError, match="device"):
            _CALLS[name](*devices)
    assert len(lib.launched) == 1


@pytest.mark.parametrize("name", ["chunk_fwd", "varlen_fwd", "chunk_bwd", "gated_norm_bwd", "residual_norm_bwd"])
def test_a_workspace_is_whole_and_on_the_device(lib, name):
    """Kernels write to all the bytes a workspace is said to have, so those have to be its own and the device's."""
    x, n, w = _zeros(1, 4, 1, 32), _zeros(2, 8), _zeros(8)
    call = {"chunk_fwd": lambda ws: kda.linear_chunk_fwd(x, x, x, workspace=ws),
            "varlen_fwd": lambda ws: kda.linear_varlen_fwd(x, x, x, _CU(0), workspace=ws),
            "chunk_bwd": lambda ws: kda.linear_chunk_bwd(x, x, x, None, None, x, workspace=ws),
            "gated_norm_bwd": lambda ws: kda.gated_norm_bwd(x, x, x, _zeros(32), workspace=ws),
            "residual_norm_bwd": lambda ws: kda.residual_norm_bwd(n, None, n, w, workspace=ws)}[name]
    call(_zeros(4096))
    assert len(lib.launched) == 1
    for ws in (torch.zeros(4096), _zeros(4096, index=1), _on_device(torch.zeros(4096)[::2]),
               _on_device(torch.zeros(1).expand(4096)), _on_device(torch.zeros(64, 64).t())):
        with pytest.raises(ValueError, match="workspace"):
            call(ws)
    assert len(lib.launched) == 1


def test_a_header_taken_in_a_capture_is_not_kept(lib, monkeypatch):
    """Memory that is first asked for while a graph is captured belongs to that graph."""
    x = _zeros(1, 4, 1, 32)
    monkeypatch.setattr(_linear, "_headers", {})
    monkeypatch.setattr(_linear, "_bytes", lambda *a: _linear._HEADER)
    capturing = [True]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(_linear, "_capturing", lambda: capturing[0], raising=False)
    kda.linear_chunk_fwd(x, x, x)
    assert not _linear._headers
    capturing[0] = False
    kda.linear_chunk_fwd(x, x, x)
    kept = dict(_linear._headers)
    assert len(kept) == 1
    capturing[0] = True                     # what is kept already is nobody's but this process's
    kda.linear_chunk_fwd(x, x, x)
    assert _linear._headers == kept and len(lib.launched) == 3


def test_outputs_are_no_broadcast_views(lib):
    """Rows that share memory would be written by several CTAs at once."""
    x, cu, st = _zeros(2, 4, 2, 32), _zeros(2, dtype=torch.int32), _zeros(2, 2, 32, 32)
    into = lambda *s: _on_device(torch.zeros(s[-1]).expand(*s))  # noqa: E731
    for call in (lambda: kda.linear_chunk_fwd(x, x, x, out=into(2, 4, 2, 32)),
                 lambda: kda.linear_varlen_fwd(x[:1], x[:1], x[:1], cu, out=into(1, 4, 2, 32)),
                 lambda: kda.linear_decode_step(x[:, 0], x[:, 0], x[:, 0], None, st, out=into(2, 2, 32)),
                 lambda: kda.gated_norm_fwd(x, x, _zeros(32), out=into(2, 4, 2, 32))):
        with pytest.raises(ValueError, match="broadcast"):
            call()
    assert not lib.launched
    kda.linear_chunk_fwd(x, x, x, out=_on_device(torch.zeros(2, 4, 3, 32)[:, :, :2]))
    assert len(lib.launched) == 1


def test_tokens_of_no_sequence_are_refused():
    """Packed tokens with an empty list of sequences: no kernel would write their outputs (dummy addresses, never read)."""
    import ctypes
    from delta_rule_linear_gb300 import build, _lib
    build.build()
    lib, p = _lib.load(), ctypes.c_void_p(0x1000)
    call = lambda total: lib.kda_linear_varlen_fwd(p, p, p, p, 0, p, None, None, p, None, None, 0, total, 2, 2, 64, 64, 1,  # noqa: E731
                                                   0.0, p, 1 << 40, None)
    assert call(10) == 9 and call(0) == 0
