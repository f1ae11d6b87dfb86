"""The binding of the 8-bit products and the row movements without a GPU: what it
asks of torch's streams, devices and allocator, and what it hands to the library,
both replaced by recorders."""

import contextlib

import pytest
import torch

import prefill_q8_mxfp4_amd as q
from prefill_q8_mxfp4_amd import _rows


class FakeStream:
    def __init__(self, number, device=0):
        self.cuda_stream, self.device_index = number, device

    def __repr__(self):
        return "s%d" % self.cuda_stream


class Machine:
    """Streams and capture state of a machine that is not there."""

    def __init__(self):
        self.current = FakeStream(1)
        self.capture = None          # id of the capture that is on
        self.recorded = []           # (address, stream) of record_stream


@pytest.fixture
def machine(monkeypatch):
    m = Machine()

    @contextlib.contextmanager
    def on(stream):
        before, m.current = m.current, stream
        yield
        m.current = before

    cpu = torch.device("cpu")
    monkeypatch.setattr(torch, "device", lambda *a: cpu)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: m.current)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: m.capture is not None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: m.recorded.append((t.data_ptr(), s)), raising=False)
    monkeypatch.setattr(_rows, "_raw_stream", lambda dev: m.current.cuda_stream)
    return m


def test_workspace_is_recorded_after_a_capture(machine):
    """A workspace that a capture took, on a stream other than the one it was made
    on, is recorded on that stream by the first eager call there: the block must
    not go back to the allocator while that stream's work on it is pending."""
    plan = q.Plan("int8", 5120, 5120, act="bf16")
    s0, st = machine.current, FakeStream(2)
    at, n = _rows._workspace(plan, "auto", 64, 0, None)
    assert n >= plan.workspace_bytes(64) and (at, s0) in machine.recorded
    machine.current, machine.capture = st, 7
    assert _rows._workspace(plan, "auto", 64, 0, None) == (at, n)
    machine.capture = None
    assert _rows._workspace(plan, "auto", 64, 0, None) == (at, n)
    assert (at, st) in machine.recorded


def on_gpu(monkeypatch, device=0):
    """Host tensors pass for tensors of a GPU, which is the current one."""
    monkeypatch.setattr(_rows, "_gpu", lambda t: device)
    monkeypatch.setattr(_rows, "_addr", lambda t, name, dev: t.data_ptr())
    monkeypatch.setattr(_rows, "_codes_addr", lambda t, dev: t.data_ptr())
    monkeypatch.setattr(_rows, "_current_device", lambda: device)


def test_refusals_come_from_the_library(machine, monkeypatch):
    """Calls for which there is no workspace to ask for reach the library's checks."""
    on_gpu(monkeypatch)
    plan = q.Plan("int8", 32, 48, act="bf16", out="bf16")
    w = torch.zeros(plan.weight_bytes, dtype=torch.uint8)
    x, y = torch.zeros(4, 48, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(q.QgemmError) as e:
        plan.run(x, w, y, B=-1)
    assert e.value.status == q.EINVAL
    plan.close()
    for call in (lambda: plan.run(x, w, y),
                 lambda: plan.run_codes(torch.zeros(4, 48, dtype=torch.int8), torch.zeros(4), w, y)):
        with pytest.raises(q.QgemmError) as e:
            call()
        assert e.value.status == q.EINVAL


def test_outputs_belong_to_the_launch_stream(machine, monkeypatch):
    """Outputs that the binding allocates for a call on a stream are that stream's
    blocks: those of the current stream could still be in use there, or be handed
    out again there while the kernel writes them."""
    on_gpu(monkeypatch)
    made, calls = [], []
    empty, empty_like = torch.empty, torch.empty_like

    def note(f):
        def made_by(*a, **k):
            t = f(*a, **k)
            made.append((t.data_ptr(), machine.current))
            return t
        return made_by

    monkeypatch.setattr(torch, "empty", note(empty))
    monkeypatch.setattr(torch, "empty_like", note(empty_like))
    monkeypatch.setattr(_rows, "_call", lambda f, dev, stream, *args: calls.append(stream))
    side = FakeStream(5)
    x, ids = torch.zeros(4, 48), torch.zeros(4, 2, dtype=torch.int32)
    weights = torch.zeros(16, 48, dtype=torch.int8), torch.zeros(16)
    for stream in (None, side):
        for call in (lambda: q.quantize_rows(x, stream=stream), lambda: q.route(ids, 8, stream=stream),
                     lambda: (q.pack_int8(*weights, stream=stream),)):
            outs = call()
            assert len(made) == len(outs)
            assert {at for at, _ in made} == {t.data_ptr() for t in outs}
            assert all(s is (stream or machine.current) for _, s in made), made
            assert calls == [stream] and machine.current.cuda_stream == 1
            made.clear(), calls.clear()
    q.quantize_rows(x, torch.zeros(4, 48, dtype=torch.int8), torch.zeros(4), stream=side)
    assert not made                                 # given outputs: nothing allocated


def test_one_row_of_codes_keeps_to_itself(machine, monkeypatch):
    """Codes are written with zeros up to their pitch.  One row whose own stride has
    no room for them, a row of a matrix without padding, is refused as an output,
    like two rows are: the next row begins there.  As an input it is fine."""
    on_gpu(monkeypatch)
    pitches = []
    monkeypatch.setattr(_rows, "_call", lambda f, dev, stream, *args: pitches.append(args))
    K = 20
    dense, padded = torch.zeros(4, K, dtype=torch.int8), torch.zeros(4, 48, dtype=torch.int8)
    x, pos, s = torch.zeros(1, K), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(4)
    for rows in (1, 2):
        with pytest.raises(ValueError, match="pitch"):
            q.quantize_rows(torch.zeros(rows, K), dense[:rows], s)
    with pytest.raises(ValueError, match="pitch"):
        q.dispatch_codes(x, pos, dense[:1], s)
    with pytest.raises(ValueError, match="pitch"):
        q.quantize_rows(x, torch.zeros(64, dtype=torch.int8)[:K].unsqueeze(0), s)
    assert not pitches
    # room of its own: a pitch, or a row that ends on a multiple of 16
    q.quantize_rows(x, padded[1:2, :K], s)
    q.quantize_rows(x)
    q.quantize_rows(torch.zeros(1, 32), dense.view(-1)[:32].unsqueeze(0), s)
    assert [a[5] for a in pitches] == [48, 32, 32]
    plan = q.Plan("int8", 32, K, act="bf16", out="f32")
    plan.run_codes(dense[:1], s, torch.zeros(plan.weight_bytes, dtype=torch.uint8), torch.zeros(1, 32))
    assert pitches[-1][4] == 32


def test_workspace_made_under_capture(machine, monkeypatch):
    """A workspace made inside a capture is zeroed by that graph's replays alone.
    An eager call, which may come before any replay, takes another one; a second
    capture zeroes it for its own replays, which may come first."""
    zeroed = []
    monkeypatch.setattr(q, "_capture_id", lambda stream: machine.capture, raising=False)
    zero_ = torch.Tensor.zero_
    monkeypatch.setattr(torch.Tensor, "zero_", lambda t: zeroed.append(t.data_ptr()) or zero_(t))
    plan = q.Plan("q8_0", 2048, 1024, act="f32", out="f32")
    assert plan.workspace_bytes(5) > 0

    def at(B=5, capture=None):
        machine.capture = capture
        return plan._workspace(B, torch.device("cuda", 0), machine.current).data_ptr()

    first = at(capture=7)
    assert at(capture=7) == first and not zeroed     # once for all calls of a capture
    assert at(capture=8) == first and zeroed == [first]
    assert at(capture=8) == first and zeroed == [first]
    eager = at()
    assert eager != first and at() == eager
    assert at(capture=9) == eager and zeroed == [first]   # zero since its own first call
    assert at() == eager
    kept = {t.data_ptr() for t in plan._ws_captured}
    assert kept == {first, eager}
    assert [a for a, _ in machine.recorded] == [eager] * 3


def test_stream_of_another_device(machine, monkeypatch):
    """A stream of another GPU than the tensors' is refused before the call: its
    kernels would run on that GPU."""
    on_gpu(monkeypatch, 1)
    ran = []

    def f(*args):
        ran.append(args[-1])
        return q.OK

    _rows._call(f, 1, FakeStream(6, 1), 3)
    assert ran == [6]
    with pytest.raises(ValueError, match="stream"):
        _rows._call(f, 1, FakeStream(6, 0), 3)
    assert ran == [6]


def test_call_on_another_device(monkeypatch):
    """A call runs with the tensors' GPU as the current one and puts the caller's
    back, after an error too."""
    now, seen = [0], []
    monkeypatch.setattr(_rows, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "set_device", lambda d: now.__setitem__(0, d))
    monkeypatch.setattr(_rows, "_raw_stream", lambda dev: 100 + dev)

    def f(*args):
        seen.append((now[0], args))
        return args[0]

    _rows._call(f, 2, None, q.OK, "x")
    assert seen == [(2, (q.OK, "x", 102))] and now == [0]
    with pytest.raises(q.QgemmError):
        _rows._call(f, 2, None, q.EINVAL)
    assert now == [0] and seen[-1][0] == 2
    _rows._call(f, 0, None, q.OK)
    assert seen[-1] == (0, (q.OK, 100))
