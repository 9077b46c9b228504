"""What the binding of the packed operators refuses before it touches a device."""

import numpy as np
import pytest

import exact_softmax_attention_fa_gb300 as fa

torch = pytest.importorskip("torch")


def plan_of(rows):
    """A PackedPlan as its constructor leaves it, without the device work."""
    plan = object.__new__(fa.PackedPlan)
    plan.rows, plan.causal, plan.B = rows, True, 1
    plan.buffer = torch.zeros(max(1, fa.fa_packed_plan_size(1, rows)), dtype=torch.uint8)
    return plan


@pytest.mark.parametrize("rows", [9, 11, 0])
def test_a_plan_of_other_rows_is_refused(rows):
    x, lse = torch.zeros(10, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 10)
    with pytest.raises(ValueError, match="rows"):
        fa.forward_packed(x, x, x, plan_of(rows))
    with pytest.raises(ValueError, match="rows"):
        fa.backward_packed(x, x, x, x, lse, x, plan_of(rows))
    with pytest.raises(ValueError, match="rows"):
        fa.backward_packed(x, x, x, x, lse, x, plan_of(rows), out=(x, x, x), workspace=torch.zeros(1, dtype=torch.uint8))


AXES = [0, 1, 2, 1, 0, 2, 2, 2]


@pytest.mark.parametrize("kind", [list, tuple, bytes, bytearray, iter, np.int64, np.int32, np.uint8, np.int8, torch.tensor],
                         ids=lambda k: k.__name__)
def test_axes_are_taken_number_by_number(kind):
    positions = torch.zeros(3, 1, 4, dtype=torch.int32)
    axes = np.array(AXES, dtype=kind) if isinstance(kind, type) and issubclass(kind, np.generic) else kind(AXES)
    assert fa._axes(axes, positions, 16) == (bytes(AXES), 3)


@pytest.mark.parametrize("axes", [8, np.int64(8), True, 8.0, [0.0] * 8, "00000000", [None] * 8, [-1] * 8, [256] * 8, [0] * 7,
                                  np.zeros(1, np.int64), np.zeros(2, np.int32), torch.zeros(8), object()], ids=repr)
def test_what_is_no_axes(axes):
    """An integer is no sequence, and an array's bytes are not its numbers (2 int32 are 8 bytes)."""
    with pytest.raises(ValueError):
        fa._axes(axes, torch.zeros(1, 1, 4, dtype=torch.int32), 16)


def test_the_calls_by_axes_need_axes():
    """Without them they would be the calls by one position."""
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    cos, pos = torch.zeros(8, 32), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="axes"):
        fa.fa_norm_rope_axes_fwd(x, x, x, None, None, cos, cos, pos, None, x, x, x)
    with pytest.raises(ValueError, match="axes"):
        fa.fa_norm_rope_axes_bwd(x, x, x, None, None, None, None, cos, cos, pos, None, x, x, x, None, None, None)


def test_without_a_rotation_axes_and_positions_are_not_used():
    for axes in ([], b"", [0] * 32, 7):
        for positions in (None, torch.zeros(3, 1, 4, dtype=torch.int32)):
            assert fa._axes(axes, positions, 0) == (None, 0)
    with pytest.raises(ValueError, match="positions"):
        fa._axes([0] * 8, None, 16)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Buffer:
    """The plan's memory as the binding looks at it."""
    dtype, shape = torch.uint8, (1 << 20,)

    def __init__(self):
        self.recorded = []

    def is_contiguous(self):
        return True

    def get_device(self):
        return -1

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return 1 << 20

    def element_size(self):
        return 1

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


class Library:
    """Calls that do nothing but say which stream they were given."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 256
        return lambda *a: self.streams.append(a[-1]) or 0


def test_a_plans_memory_waits_for_every_stream_that_uses_it(monkeypatch):
    """A plan is dropped as soon as the last call is queued, and its memory came from the stream it was made on: without
    a word to the allocator that stream's next tensor could take it while another stream's kernels still read it."""
    lib = Library()
    monkeypatch.setattr(fa, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 11, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(11))
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    plan = plan_of(10)
    plan.buffer, plan._streams = Buffer(), {11}
    x, lse, ws = torch.zeros(10, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 10), torch.zeros(8, dtype=torch.uint8)
    forward = lambda stream: fa.fa_fwd_packed(x, x, x, x, lse, plan, True, 0.1, stream=stream)
    backward = lambda stream: fa.fa_bwd_packed(x, x, x, x, lse, x, x, x, x, plan, True, 0.1, ws, stream=stream)
    forward(None), backward(None)
    assert plan.buffer.recorded == []  # the stream it was made on
    forward(Stream(12)), forward(12), backward(Stream(12))
    assert plan.buffer.recorded == [12]
    backward(13)
    plan.update(torch.zeros(2, dtype=torch.int32), Stream(14))
    assert plan.buffer.recorded == [12, 13, 14] and lib.streams == [11, 11, 12, 12, 12, 13, 14]
    with pytest.raises(ValueError):  # a refused call uses nothing
        fa.fa_fwd_packed(x, x[:3], x, x, lse, plan, True, 0.1, stream=15)
    assert plan.buffer.recorded == [12, 13, 14]
