"""Sliding windows with first tokens that stay visible: decode (one pass,
partitions, append, 8-bit pools) and chunked prefill, against a plain 64-bit
attention; tolerances as for the attention without a window (pagedutil)."""

import numpy as np
import pytest
import torch

import opsutil as ou
import oracle
import paged_kv_cache_449_b200 as pa
import pagedutil as pu
from paged_kv_cache_449_b200 import ops

pytestmark = pytest.mark.gpu

LENS = [1, 0, 8, 9, 16, 33, 64, 100, 129, 300]
WINDOWS = [(1, 0), (1, 3), (7, 0), (16, 16), (33, 1), (40, 70), (64, 4), (1000, 4), (2 ** 31 - 1, 2 ** 31 - 1)]


def batch(lens, Hq, H, D, B, dtype, seed, queries=None):
    g = ou.gen(seed)
    table, N = ou.tables_of(lens, B, seed)
    k, v = (ou.normal(pa.pool_shape(N, H, D, B, dtype), dtype, g) for _ in range(2))
    q = ou.normal((len(lens) if queries is None else queries, Hq, D), dtype, g)
    return q, k, v, table


def poison(k, v, table, lens, B, hidden):
    """Not-a-number wherever no query looks: in the pools' hidden tokens (a
    bool per token of each sequence), free blocks and unused rows; blocks
    without a visible token leave the table."""
    k, v, table = k.clone(), v.clone(), table.clone()
    live = torch.zeros(k.shape[0], B, dtype=torch.bool)
    for s, L in enumerate(lens):
        for t in range(L):
            if not hidden(s, t):
                live[int(table[s, t // B]), t % B] = True
    dead = ~live[:, None, None, :, None].expand_as(k)
    k[dead], v[dead] = float("nan"), float("inf")
    for s, L in enumerate(lens):
        for j in range(table.shape[1]):
            if all(hidden(s, t) for t in range(j * B, min(j * B + B, L))):
                table[s, j] = 1 << 30
    return k, v, table


def dev(*tensors):
    return [t.cuda() for t in tensors]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("dtype,D,B", [(torch.float32, 64, 16), (torch.float32, 128, 8), (torch.float16, 64, 8),
                                       (torch.float16, 128, 32), (torch.bfloat16, 128, 16),
                                       (torch.bfloat16, 64, 32), (torch.bfloat16, 128, 8), (torch.float32, 64, 32)])
def test_decode(dtype, D, B, window, sinks):
    q, k, v, table = batch(LENS, 8, 2, D, B, dtype, D + B)
    scale = D ** -0.5
    want = ou.decode(q, lambda s: tuple(ou.pool_rows(x, table[s, :-(-LENS[s] // B)].long(), LENS[s]) for x in (k, v)),
                     LENS, scale, window, sinks)
    hidden = lambda s, t: not (t >= LENS[s] - window or t < sinks)  # noqa: E731
    kp, vp, tp = poison(k, v, table, LENS, B, hidden)
    qd, kd, vd, td, ld = dev(q, kp, vp, tp, torch.tensor(LENS, dtype=torch.int32))
    for part in (0, 32, 128, None):
        out = torch.full_like(qd, float("nan"))
        ops.pa_decode_window(out, qd, None, None, kd, vd, td, ld, scale, window, sinks, partition_size=part)
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == 0
        pu.check_tolerance(pu.as_f64(out), want.numpy(), dtype)


@pytest.mark.parametrize("group", [1, 2, 8])
def test_decode_groups(group):
    lens = [500, 77]
    q, k, v, table = batch(lens, 3 * group, 3, 128, 16, torch.bfloat16, group)
    want = ou.decode(q, lambda s: tuple(ou.pool_rows(x, table[s].long(), lens[s]) for x in (k, v)), lens, 0.1, 100, 5)
    qd, kd, vd, td, ld = dev(q, k, v, table, torch.tensor(lens, dtype=torch.int32))
    out = torch.empty_like(qd)
    ops.pa_decode_window(out, qd, None, None, kd, vd, td, ld, 0.1, 100, 5)
    pu.check_tolerance(pu.as_f64(out), want.numpy(), torch.bfloat16)


@pytest.mark.parametrize("many", [False, True])
def test_a_window_past_the_context_is_the_plain_decode(many):
    """Bit-identical to pa_decode, in the deep and the wide shape."""
    lens = ([700, 20, 333] if not many else [40, 300, 90, 11] * 40)
    q, k, v, table = batch(lens, 32, 8, 64, 16, torch.float16, 3)
    qd, kd, vd, td, ld = dev(q, k, v, table, torch.tensor(lens, dtype=torch.int32))
    a, b = torch.empty_like(qd), torch.empty_like(qd)
    pa.pa_decode(a, qd, kd, vd, td, ld, 0.125)
    ops.pa_decode_window(b, qd, None, None, kd, vd, td, ld, 0.125, 10000, 4, partition_size=0)
    assert torch.equal(a, b)
    # a window of whole blocks without sinks: the plain decode of the table's end
    part = [n for n in lens if n > 64]
    q, k, v, table = batch([n - n % 16 for n in part], 32, 8, 64, 16, torch.float16, 4)
    cut = torch.stack([table[s, (n - n % 16) // 16 - 4:(n - n % 16) // 16] for s, n in enumerate(part)])
    qd, kd, vd, td, cd = dev(q, k, v, table, cut.contiguous())
    a, b = torch.empty_like(qd), torch.empty_like(qd)
    pa.pa_decode(a, qd, kd, vd, cd, torch.full((len(part),), 64, dtype=torch.int32).cuda(), 0.125)
    ops.pa_decode_window(b, qd, None, None, kd, vd, td,
                         torch.tensor([n - n % 16 for n in part], dtype=torch.int32).cuda(), 0.125, 64, 0,
                         partition_size=0)
    assert torch.equal(a, b)


@pytest.mark.parametrize("part", [0, 32])
@pytest.mark.parametrize("fp8", [False, True])
def test_append_equals_write_then_decode(fp8, part):
    lens, B, D, H = [1, 17, 100, 129, 64], 16, 128, 2
    q, k, v, table = batch(lens, 8, H, D, B, torch.bfloat16, 9)
    g = ou.gen(10)
    key, value = ou.normal((5, H, D), torch.bfloat16, g), ou.normal((5, H, D), torch.bfloat16, g)
    slots = torch.tensor([int(table[s, (n - 1) // B]) * B + (n - 1) % B for s, n in enumerate(lens)])
    qd, td, ld, kn, vn, sd = dev(q, table, torch.tensor(lens, dtype=torch.int32), key, value, slots)
    scales = dev(torch.tensor([0.01, 0.02]), torch.tensor([0.015, 0.01])) if fp8 else []
    if fp8:
        N = k.shape[0]
        k, v = (torch.randint(0, 120, pa.fp8_pool_shape(N, H, D, B), generator=g, dtype=torch.uint8) for _ in range(2))
    pools = [dev(k, v), dev(k, v)]
    outs = [torch.empty_like(qd), torch.empty_like(qd)]
    kw = dict(window=50, num_sinks=3, partition_size=part)
    if fp8:
        ops.pa_decode_window_fp8(outs[0], qd, kn, vn, *pools[0], *scales, td, ld, 0.1, **kw)
        pa.pa_reshape_and_cache_fp8(kn, vn, *pools[1], sd, *scales)
        ops.pa_decode_window_fp8(outs[1], qd, None, None, *pools[1], *scales, td, ld, 0.1, **kw)
    else:
        ops.pa_decode_window(outs[0], qd, kn, vn, *pools[0], td, ld, 0.1, **kw)
        pa.pa_reshape_and_cache(kn, vn, *pools[1], sd)
        ops.pa_decode_window(outs[1], qd, None, None, *pools[1], td, ld, 0.1, **kw)
    assert torch.equal(outs[0], outs[1])
    for a, b in zip(*pools):
        assert torch.equal(a, b)
    assert pa.pa_get_device_error() == 0


def test_append_leaves_shared_blocks():
    lens, B = [20, 30], 16
    q, k, v, table = batch(lens, 4, 1, 64, B, torch.float16, 2)
    counts = torch.ones(k.shape[0], dtype=torch.int32)
    counts[int(table[1, 1])] = 2
    key = ou.normal((2, 1, 64), torch.float16, ou.gen(1))
    qd, kd, vd, td, ld, cd, kn = dev(q, k, v, table, torch.tensor(lens, dtype=torch.int32), counts, key)
    out = torch.empty_like(qd)
    ops.pa_decode_window(out, qd, kn, kn, kd, vd, td, ld, 0.125, 10, 0, ref_counts=cd)
    assert pa.pa_get_device_error() == pa.DEVERR_SHARED_BLOCK
    changed = (kd.cpu() != k).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert changed == [int(table[0, 1])]


@pytest.mark.parametrize("window,sinks", [(5, 0), (40, 20), (500, 4)])
@pytest.mark.parametrize("D,B", [(64, 8), (128, 16), (64, 32)])
def test_decode_8_bit(D, B, window, sinks):
    lens = [1, 9, 100, 300, 0, 31]
    g = ou.gen(B)
    table, N = ou.tables_of(lens, B, B)
    H, T = 2, sum(lens)
    k, v = ou.normal((T, H, D), torch.float16, g), ou.normal((T, H, D), torch.float16, g)
    slots = torch.tensor([int(table[s, t // B]) * B + t % B for s, n in enumerate(lens) for t in range(n)])
    ks, vs = torch.tensor([0.01, 0.02]), torch.tensor([0.015, 0.01])
    kc, vc = (torch.zeros(pa.fp8_pool_shape(N, H, D, B), dtype=torch.uint8, device="cuda") for _ in range(2))
    ksd, vsd, kd, vd, sd = dev(ks, vs, k, v, slots)
    pa.pa_reshape_and_cache_fp8(kd, vd, kc, vc, sd, ksd, vsd)
    held = lambda x, sc: ((x.float() / sc[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double()  # noqa: E731
                          * sc.double()[None, :, None])
    kv, vv = held(k, ks), held(v, vs)
    first = np.cumsum([0] + lens)
    q = ou.normal((len(lens), 8, D), torch.float16, g)
    want = ou.decode(q, lambda s: (kv[first[s]:first[s + 1]], vv[first[s]:first[s + 1]]), lens, 0.1, window, sinks)
    qd, td, ld = dev(q, table, torch.tensor(lens, dtype=torch.int32))
    for part in (0, 32):
        out = torch.full_like(qd, float("nan"))
        ops.pa_decode_window_fp8(out, qd, None, None, kc, vc, ksd, vsd, td, ld, 0.1, window, sinks,
                                 partition_size=part)
        assert pa.pa_get_device_error() == 0
        pu.check_tolerance(pu.as_f64(out), want.numpy(), torch.float16)


def test_order_graph_and_prepared_calls():
    lens = [900, 31, 450]
    q, k, v, table = batch(lens, 8, 2, 128, 16, torch.bfloat16, 6)
    qd, kd, vd, td, ld = dev(q, k, v, table, torch.tensor(lens, dtype=torch.int32))
    outs = [torch.zeros_like(qd) for _ in range(3)]
    kw = dict(window=300, num_sinks=4, partition_size=64)
    ops.pa_decode_window(outs[0], qd, None, None, kd, vd, td, ld, 0.1, **kw)
    ops.pa_decode_window(outs[1], qd, None, None, kd, vd, td, ld, 0.1, seq_order=pa.longest_first(lens).cuda(), **kw)
    call = pa.prepare_decode_window(outs[2], qd, None, None, kd, vd, td, ld, 0.1, **kw)
    call()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        outs[2].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[2])


def test_refused_ids_and_lengths():
    lens = [100]
    q, k, v, table = batch(lens, 4, 1, 64, 16, torch.float16, 12)
    table = table.clone()
    table[0, 4] = -7      # inside the window
    qd, kd, vd, td = dev(q, k, v, table)
    out = torch.empty_like(qd)
    ops.pa_decode_window(out, qd, None, None, kd, vd, td, torch.tensor([100], dtype=torch.int32).cuda(), 0.1, 50, 4)
    assert pa.pa_get_device_error() == pa.DEVERR_BLOCK_ID
    ops.pa_decode_window(out, qd, None, None, kd, vd, td, torch.tensor([-3], dtype=torch.int32).cuda(), 0.1, 50, 4)
    assert pa.pa_get_device_error() == pa.DEVERR_CONTEXT_LEN
    assert torch.equal(out.cpu(), torch.zeros_like(q))


# ------------------------------------------------------------------ prefill

CHUNKS = [(1, 1), (40, 17), (0, 0), (130, 130), (300, 64), (257, 1), (500, 200), (64, 3)]


def prefill_case(chunks, Hq, H, D, B, dtype, seed):
    lens = [n for n, _ in chunks]
    start = np.cumsum([0] + [c for _, c in chunks]).tolist()
    q, k, v, table = batch(lens, Hq, H, D, B, dtype, seed, queries=start[-1])
    return lens, start, q, k, v, table


def run_prefill(lens, start, q, k, v, table, scale, window, sinks, **kw):
    qd, kd, vd, td, ld, sd = dev(q, k, v, table, torch.tensor(lens, dtype=torch.int32),
                                 torch.tensor(start, dtype=torch.int32))
    out = torch.full_like(qd, float("nan"))
    ops.pa_prefill_window(out, qd, kd, vd, td, ld, sd, scale, window, sinks, **kw)
    torch.cuda.synchronize()
    return out


def prefill_want(lens, start, q, k, v, table, B, scale, window, sinks):
    out = torch.zeros(q.shape, dtype=torch.float64)
    for s, L in enumerate(lens):
        a, z = start[s], start[s + 1]
        if z > a:
            kk, vv = (ou.pool_rows(x, table[s, :-(-L // B)].long(), L) for x in (k, v))
            out[a:z] = ou.attend(q[a:z], kk, vv, L - (z - a), scale, window, sinks)
    return out


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 5), (7, 1), (64, 0), (65, 64), (100, 70), (128, 4), (500, 130),
                                          (2 ** 31 - 1, 0)])
@pytest.mark.parametrize("dtype,D,B,group", [(torch.float16, 64, 8, 4), (torch.bfloat16, 128, 16, 4),
                                             (torch.float16, 128, 32, 8), (torch.bfloat16, 128, 8, 1),
                                             (torch.float16, 64, 16, 2), (torch.bfloat16, 64, 32, 1)])
def test_prefill(dtype, D, B, group, window, sinks):
    lens, start, q, k, v, table = prefill_case(CHUNKS, 2 * group, 2, D, B, dtype, D + B + group)
    scale = D ** -0.5
    want = prefill_want(lens, start, q, k, v, table, B, scale, window, sinks)
    first = [L - (start[s + 1] - start[s]) for s, L in enumerate(lens)]
    hidden = lambda s, t: lens[s] == first[s] or not (t > first[s] - window or t < sinks)  # noqa: E731
    kp, vp, tp = poison(k, v, table, lens, B, hidden)
    got = run_prefill(lens, start, q, kp, vp, tp, scale, window, sinks)
    assert pa.pa_get_device_error() == 0
    pu.check_tolerance(pu.as_f64(got), want.numpy(), dtype)


def test_prefill_of_one_long_chunk():
    lens, start, q, k, v, table = prefill_case([(1501, 1501)], 4, 1, 64, 16, torch.float16, 5)
    for window, sinks in ((129, 3), (64, 0)):
        want = prefill_want(lens, start, q, k, v, table, 16, 0.125, window, sinks)
        pu.check_tolerance(pu.as_f64(run_prefill(lens, start, q, k, v, table, 0.125, window, sinks)), want.numpy(),
                           torch.float16)


def test_a_prefill_window_past_the_context_is_the_plain_prefill():
    lens, start, q, k, v, table = prefill_case(CHUNKS, 8, 2, 128, 16, torch.bfloat16, 8)
    got = run_prefill(lens, start, q, k, v, table, 0.1, 100000, 0)
    qd, kd, vd, td, ld, sd = dev(q, k, v, table, torch.tensor(lens, dtype=torch.int32),
                                 torch.tensor(start, dtype=torch.int32))
    out = torch.empty_like(qd)
    pa.pa_prefill(out, qd, kd, vd, td, ld, sd, 0.1)
    assert torch.equal(out, got)


def test_prefill_flags_a_refused_id_in_the_window():
    lens, start, q, k, v, table = prefill_case([(300, 20)], 4, 1, 64, 16, torch.float16, 4)
    table[0, 17] = -1
    run_prefill(lens, start, q, k, v, table, 0.125, 64, 4)
    assert pa.pa_get_device_error() == pa.DEVERR_BLOCK_ID
    table[0, 17], table[0, 5] = 0, -1        # outside every window: not looked at
    run_prefill(lens, start, q, k, v, table, 0.125, 64, 4)
    assert pa.pa_get_device_error() == 0


def test_prefill_graph():
    lens, start, q, k, v, table = prefill_case([(300, 64), (77, 77)], 4, 1, 64, 16, torch.float16, 4)
    base = run_prefill(lens, start, q, k, v, table, 0.125, 50, 4)
    qd, kd, vd, td, ld, sd = dev(q, k, v, table, torch.tensor(lens, dtype=torch.int32),
                                 torch.tensor(start, dtype=torch.int32))
    out = torch.zeros_like(qd)
    call = pa.prepare_prefill_window(out, qd, kd, vd, td, ld, sd, 0.125, 50, 4, max_query_len=77)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, base)


@pytest.mark.parametrize("L", [5, 20, 70])
def test_plain_prefill_of_8_token_blocks_ignores_what_lies_behind_the_context(L):
    """The pool's tokens past the context may hold anything."""
    q, k, v, table = batch([L], 4, 1, 64, 8, torch.float16, 7, queries=L)
    want = prefill_want([L], [0, L], q, k, v, table, 8, 0.125, 2 ** 31 - 1, 0)
    kp, vp, tp = poison(k, v, table, [L], 8, lambda s, t: False)
    qd, kd, vd, td, ld, sd = dev(q, kp, vp, tp, torch.tensor([L], dtype=torch.int32),
                                 torch.tensor([0, L], dtype=torch.int32))
    out = torch.empty_like(qd)
    pa.pa_prefill(out, qd, kd, vd, td, ld, sd, 0.125)
    assert pa.pa_get_device_error() == 0
    pu.check_tolerance(pu.as_f64(out), want.numpy(), torch.float16)


def test_reference_agrees_with_the_oracle():
    """The plain form used here, without a window, is the oracle's decode."""
    lens = [40, 7]
    q, k, v, table = batch(lens, 4, 2, 64, 16, torch.float16, 1)
    mine = ou.decode(q, lambda s: tuple(ou.pool_rows(x, table[s, :-(-lens[s] // 16)].long(), lens[s]) for x in (k, v)),
                     lens, 0.125)
    ref = oracle.default().decode(q, k, v, table, torch.tensor(lens, dtype=torch.int32), 0.125, 16, 2)
    assert np.allclose(mine.numpy(), ref, rtol=1e-12, atol=1e-12)
