"""Which streams a call's own buffers are ordered and kept on (CPU: the streams
and tensors are stand-ins that note what is asked of them)."""

import pytest
import torch

import paged_kv_cache_449_b200 as pa
from paged_kv_cache_449_b200 import ops


class Stream:
    def __init__(self, raw):
        self.cuda_stream, self.waits = raw, []
        self.device = torch.device("cuda", 0)

    def wait_stream(self, other):
        self.waits.append(other)


class Buffer:
    """A tensor made for a call."""

    def __init__(self):
        self.device, self.recorded = torch.device("cuda", 0), []

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def streams(monkeypatch):
    """The legacy default stream, and a stream of the caller's that is current;
    raw handles are opened as torch does: handle 0 means "none given", and gives
    a stream of the pool."""
    default, current, pool = Stream(0), Stream(0x1000), Stream(0x9000)
    made = {}

    def external(raw, device=None):
        return made.setdefault(raw, Stream(raw)) if raw else pool

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: default)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(pa, "_stream", lambda stream: current.cuda_stream if stream is None else
                        getattr(stream, "cuda_stream", stream))
    monkeypatch.setattr(ops, "_stream", pa._stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    return default, current, made


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_streams_handle_is_that_stream(streams, handle):
    """Handles 0 and 1 both name the legacy default stream."""
    default, current, made = streams
    buffer = Buffer()
    assert ops._side_stream(handle, (buffer,)) == handle
    assert buffer.recorded == [default] and default.waits == [current] and not made


def test_a_raw_handle_and_a_stream_object(streams):
    default, current, made = streams
    buffer = Buffer()
    assert ops._side_stream(0x2000, (buffer,)) == 0x2000
    assert buffer.recorded == [made[0x2000]] and made[0x2000].waits == [current]
    mine = Stream(0x3000)
    assert ops._side_stream(mine, (buffer,)) == 0x3000
    assert buffer.recorded[1:] == [mine] and mine.waits == [current]


def test_the_current_stream_needs_neither(streams):
    default, current, made = streams
    buffer = Buffer()
    for stream in (None, current, current.cuda_stream):
        assert ops._side_stream(stream, (buffer,)) == current.cuda_stream
    assert not buffer.recorded and not current.waits


class Held(torch.Tensor):
    """A CPU tensor that passes for one of the caller's CUDA buffers."""

    @staticmethod
    def of(t):
        return torch.Tensor._make_subclass(Held, t)

    @property
    def is_cuda(self):
        return True


def test_only_buffers_made_for_a_handle_are_waited_for(monkeypatch):
    """A prepared call waits, on the host, for the counters made for it, and for
    nothing where the workspace and counters are the caller's."""
    waited = []

    class Busy:
        def synchronize(self):
            waited.append(self)

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Busy())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    workspace, counts = Held.of(torch.zeros(256, dtype=torch.uint8)), Held.of(torch.zeros(8, dtype=torch.int32))
    kept = pa.Counters()
    kept.buf, kept.get = counts, lambda n, device: counts
    for counters in (counts, kept):
        got = ops._partials(256, workspace, counters, 8, torch.device("cpu"), True)
        assert got[0] == [workspace.data_ptr(), 256, counts.data_ptr(), 8]
        args, held, made = ops._settled(*got)
        assert made == ()
        assert held[0] is workspace and held[1] is counts and not waited
    assert ops._settled(*ops._partials(0, None, None, 8, torch.device("cpu"), True)) == ([None, 0, None, 0], (), ())
    made = torch.zeros(8, dtype=torch.int32)
    ops._settled([], (workspace, made), (made,))
    assert len(waited) == 1


def test_counters_that_outlive_a_captured_call_are_not_made_in_the_capture(monkeypatch):
    """They would be zeroed by the graph's replays only: a handle refuses, and a
    Counters that is too small stays as it is (the call has its own)."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(ops, "_dev_ptr", lambda t, name: t.data_ptr())
    cpu, workspace = torch.device("cpu"), Held.of(torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="capturing"):
        ops._partials(256, workspace, None, 8, cpu, True)
    small = pa.Counters()
    for buf in (None, Held.of(torch.zeros(7, dtype=torch.int32))):
        small.buf = buf
        with pytest.raises(ValueError, match="capturing"):
            ops._partials(256, workspace, small, 8, cpu, True)
        args, held, made = ops._partials(256, workspace, small, 8, cpu, False)
        assert small.buf is buf and held[1] is made[0] and held[1].numel() == 8 and args[2] == held[1].data_ptr()
    # given, large enough, or not needed
    given = Held.of(torch.zeros(8, dtype=torch.int32))
    small.buf, small.get = given, lambda n, device: given
    for counters in (given, small):
        assert ops._partials(256, workspace, counters, 8, cpu, True)[1][1] is given
    assert ops._partials(0, None, None, 8, cpu, True)[1] == ()


def test_a_handles_own_buffers_are_kept_on_every_stream_it_runs_on(streams, monkeypatch):
    """A handle may be dropped while its kernel still runs on another stream than
    the one that its workspace and counters were made on."""
    import ctypes
    default, current, made = streams
    launches = []

    def entry(*args):
        launches.append(args[-1])
        return 0

    entry.argtypes = [ctypes.c_int, ctypes.c_void_p]
    monkeypatch.setattr(pa, "load", lambda: type("Library", (), {"pa_entry": staticmethod(entry)}))
    mine, buffers = Stream(0x4000), (Buffer(), Buffer())
    call = pa.Prepared("pa_entry", [3], torch.device("cuda", 0), (), buffers)
    for stream in (None, mine, 0x5000, 0, mine, None, 0x5000):
        call(stream)
    assert launches == [current.cuda_stream, 0x4000, 0x5000, 0, 0x4000, current.cuda_stream, 0x5000]
    for b in buffers:
        assert [s.cuda_stream for s in b.recorded] == [current.cuda_stream, 0x4000, 0x5000, 0]
        assert b.recorded[1] is mine and b.recorded[3] is default
    plain = pa.Prepared("pa_entry", [3], torch.device("cuda", 0), ())
    plain(mine)
    assert launches[-1] == 0x4000 and not mine.waits


def test_the_shared_prefix_handles_workspace_is_its_own_where_none_is_given(monkeypatch):
    own = object()
    monkeypatch.setattr(pa, "_tensor_device", lambda *a: torch.device("cuda", 0))
    monkeypatch.setattr(pa, "_shared_prefix_args", lambda *a: ([], a[11] if a[11] is not None else own, object()))
    assert pa.prepare_decode_shared_prefix(*[None] * 8, 0.1, 4)._made == (own,)
    assert pa.prepare_decode_shared_prefix(*[None] * 8, 0.1, 4, workspace=object())._made == ()
