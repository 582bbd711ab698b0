"""Calls on other streams than the current one, by object and by raw handle: the
buffers that a call makes for itself are ordered before its kernel and kept
until it has run.  The current stream is kept busy meanwhile, so that what is
not ordered would show."""

import pytest
import torch

import opsutil as ou
import paged_kv_cache_449_b200 as pa
from paged_kv_cache_449_b200 import ops

pytestmark = pytest.mark.gpu

LENS, D, B, BUSY = [3000, 3000], 64, 16, 20_000_000      # (cycles: about 10 ms)


@pytest.fixture(scope="module")
def setting():
    """fn(stream, out, **kw) -> a partitioned decode of each kind, and its result."""
    g = ou.gen(3)
    table, N = ou.tables_of(LENS, B, 3)
    lens = torch.tensor(LENS, dtype=torch.int32).cuda()
    table, q = table.cuda(), ou.normal((2, 8, D), torch.bfloat16, g).cuda()
    k, v = (ou.normal(pa.pool_shape(N, 1, D, B, torch.bfloat16), torch.bfloat16, g).cuda() for _ in range(2))
    k4, v4 = (torch.zeros(pa.int4_pool_shape(N, 1, D, B), dtype=torch.uint8, device="cuda") for _ in range(2))
    rows = [ou.normal((N * B, 1, D), torch.bfloat16, g).cuda() for _ in range(2)]
    ops.pa_reshape_and_cache_int4(*rows, k4, v4, torch.arange(N * B).cuda())
    calls = {
        "int4": (ops.pa_decode_int4, pa.prepare_decode_int4, lambda o: (o, q, k4, v4, table, lens, 0.125), {}),
        "window": (ops.pa_decode_window, pa.prepare_decode_window,
                   lambda o: (o, q, None, None, k, v, table, lens, 0.125), dict(window=2500)),
    }
    base = {}
    for name, (fn, _, args, kw) in calls.items():
        out = torch.zeros_like(q)
        fn(*args(out), partition_size=64, **kw)
        base[name] = out
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    return calls, base


def handles():
    side = torch.cuda.Stream()
    return {"default": 0, "legacy": 1, "raw": side.cuda_stream, "object": side}, side


@pytest.mark.parametrize("kind", ["int4", "window"])
@pytest.mark.parametrize("which", ["default", "legacy", "raw", "object"])
def test_a_call_on_another_stream(setting, kind, which):
    calls, base = setting
    fn, _, args, kw = calls[kind]
    named, side = handles()
    mine = torch.cuda.Stream()
    outs = [torch.zeros_like(base[kind]) for _ in range(4)]
    torch.cuda.synchronize()
    with torch.cuda.stream(mine):
        for out in outs:
            torch.cuda._sleep(BUSY // 4)
            fn(*args(out), partition_size=64, stream=named[which], **kw)
            # memory that the call gave back is written over at once
            junk = [torch.full((n,), 0x7f7f7f7f, dtype=torch.int32, device="cuda") for n in (2, 4, 8, 1 << 16, 1 << 17)]
        del junk
    torch.cuda.synchronize()
    assert all(torch.equal(o, base[kind]) for o in outs)
    assert pa.pa_get_device_error() == 0
    del side


@pytest.mark.parametrize("kind", ["int4", "window"])
def test_a_handle_over_the_callers_buffers_is_made_at_once(setting, kind):
    calls, base = setting
    _, prepare, args, kw = calls[kind]
    done = torch.cuda.Event()
    out = torch.zeros_like(base[kind])
    workspace, counters = torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(20 * BUSY)
    done.record()
    call = prepare(*args(out), partition_size=64, workspace=workspace, counters=counters, **kw)
    at_once = not done.query()
    call()
    torch.cuda.synchronize()
    assert at_once and torch.equal(out, base[kind])


@pytest.mark.parametrize("kind", ["int4", "window"])
def test_a_handle_is_not_made_in_a_capture(setting, kind):
    """... where it would have counters that only the graph zeroes; with the
    caller's, or made before, its captured calls are the eager ones."""
    calls, base = setting
    fn, prepare, args, kw = calls[kind]
    outs = [torch.zeros_like(base[kind]) for _ in range(4)]
    kept = pa.Counters()
    counters = torch.zeros(2, dtype=torch.int32, device="cuda")
    before = prepare(*args(outs[0]), partition_size=64, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="capturing"):
            prepare(*args(outs[0]), partition_size=64, **kw)
        with pytest.raises(ValueError, match="capturing"):
            prepare(*args(outs[0]), partition_size=64, counters=kept, **kw)
        before()
        given = prepare(*args(outs[1]), partition_size=64, counters=counters, **kw)
        given()
        fn(*args(outs[2]), partition_size=64, **kw)     # buffers of its own, in the graph
        fn(*args(outs[3]), partition_size=64, counters=kept, **kw)     # as well: a Counters does not grow there
    given()
    fn(*args(outs[3]), partition_size=64, counters=kept, **kw)         # eagerly, before any replay
    torch.cuda.synchronize()
    assert torch.equal(outs[1], base[kind]) and torch.equal(outs[3], base[kind])
    for _ in range(2):
        for out in outs:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, base[kind]) for o in outs)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("kind", ["int4", "window"])
@pytest.mark.parametrize("which", ["default", "raw", "object"])
def test_a_handle_may_be_dropped_while_its_call_waits(setting, kind, which):
    """... on another stream: its workspace and counters are not given to new
    work on the stream that they were made on."""
    calls, base = setting
    _, prepare, args, kw = calls[kind]
    named, side = handles()
    busy = torch.cuda.default_stream() if which == "default" else side
    mine = torch.cuda.Stream()
    for _ in range(3):
        out = torch.zeros_like(base[kind])
        torch.cuda.synchronize()
        with torch.cuda.stream(mine):
            call = prepare(*args(out), partition_size=64, **kw)
            with torch.cuda.stream(busy):
                torch.cuda._sleep(BUSY)
            call(named[which])
            del call
            junk = [torch.full((n,), 0x7f7f7f7f, dtype=torch.int32, device="cuda") for n in (2, 2, 4, 8, 1 << 16, 1 << 17, 1 << 17)]
        torch.cuda.synchronize()
        assert torch.equal(out, base[kind])
        del junk
    assert pa.pa_get_device_error() == 0
