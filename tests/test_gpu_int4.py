"""4-bit pools on the GPU: the write and read-back bit for bit, the decode
against a plain 64-bit attention over the stored values.

Decode tolerance, per (sequence, head) row in the 2-norm: the output is rounded
once (u of its type), and p * scale of V is rounded to fp16 (2^-11 relative) for
the product with the codes, whose terms scale * code are 2.55 times a normal
group's values in rms (64 normal values span 4.7 sigma: sqrt(2.35^2 + 1)), so u
+ 3 * 2^-11 bounds the error; everything else is fp32.
"""

import pytest
import torch

import opsutil as ou
import paged_kv_cache_449_b200 as pa
from paged_kv_cache_449_b200 import ops

pytestmark = pytest.mark.gpu

BOUND = {dt: ou.U[dt] + 3 * 2.0 ** -11 for dt in (torch.float16, torch.bfloat16)}


def empty_pools(N, H, D, B, fill=0):
    shape = ops.int4_pool_shape(N, H, D, B)
    return (torch.full(shape, fill, dtype=torch.uint8), torch.full(shape, fill, dtype=torch.uint8))


def build(lens, Hq, H, D, B, dtype, seed, fill=0, spread=1.0, offset=0.0):
    """A batch whose tokens were written by the library into pools that held `fill`."""
    g = ou.gen(seed)
    table, N = ou.tables_of(lens, B, seed)
    T = sum(lens)
    k = ou.normal((T, H, D), torch.float32, g) * spread + offset
    v = ou.normal((T, H, D), torch.float32, g) * spread + offset
    k, v = k.to(dtype), v.to(dtype)
    slots, first = [], []
    for s, L in enumerate(lens):
        first.append(len(slots))
        slots += [int(table[s, t // B]) * B + t % B for t in range(L)]
    kc, vc = (x.cuda() for x in empty_pools(N, H, D, B, fill))
    ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), kc, vc, torch.tensor(slots, dtype=torch.int64).cuda())
    kv, vv = ou.values4(k), ou.values4(v)
    rows = lambda s: (kv[first[s]:first[s] + lens[s]], vv[first[s]:first[s] + lens[s]])  # noqa: E731
    q = ou.normal((len(lens), Hq, D), dtype, g)
    return q, kc, vc, table, rows


def run(q, kc, vc, table, lens, **kw):
    out = torch.full_like(q, float("nan"), device="cuda")
    ops.pa_decode_int4(out, q.cuda(), kc, vc, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                       q.shape[-1] ** -0.5, **kw)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_write_and_read_back_bit_for_bit(B, D, dtype):
    g = ou.gen(B * D)
    T, H, N = 75, 3, 12
    k, v = ou.normal((T, H, D), dtype, g), ou.normal((T, H, D), dtype, g)
    k[3] = 0.5                     # a group of one value: scale 0
    k[4] = 0
    v[5, :, :64] = torch.arange(64) / 8.0      # quotients that are ties
    k[6] *= 1e-30 if dtype != torch.float16 else 1e-7
    v[7] *= 1e30 if dtype != torch.float16 else 1e4
    v[8] += 1000
    slots = torch.randperm(N * B, generator=g)[:T]
    slots[10] = -1
    kc, vc = empty_pools(N, H, D, B, 0xee)
    got = [x.cuda() for x in (kc, vc)]
    ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), *got, slots.cuda())
    for pool, rows, side in ((kc, k, False), (vc, v, True)):
        ou.write4(pool, rows, slots, B, side)
    for a, b in zip(got, (kc, vc)):
        assert torch.equal(a.cpu(), b)        # untouched bytes as they were, codes and group words equal
    back = [torch.full_like(k, 7).cuda(), torch.full_like(v, 7).cuda()]
    ops.pa_gather_cache_int4(*back, *got, slots.cuda())
    for x, rows in zip(back, (k, v)):
        want = ou.values4(rows).to(torch.float32).to(dtype)
        want[10] = 7
        assert torch.equal(x.cpu(), want)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,B", [(64, 8), (64, 16), (128, 32), (128, 8), (128, 16)])
def test_many_tokens_bit_for_bit(D, B, dtype):
    """Chunks that start and end anywhere in their blocks, padding, single
    tokens, a run of slots that crosses into another block's."""
    g = ou.gen(D + B)
    H, N = 11, 64
    order = torch.randperm(N, generator=g)
    slots, used = [], 0
    for start, count in ((5, 150), (0, 97), (B - 1, 2 * B + 3), (3, 1), (0, B), (7, 100)):
        blocks = order[used:used + (start + count + B - 1) // B]
        used += len(blocks)
        slots += [int(blocks[(start + i) // B]) * B + (start + i) % B for i in range(count)]
        slots.append(-1)
    free = [int(b) * B + t for b in order[used:used + 3] for t in torch.randperm(B, generator=g).tolist()]
    slots = torch.tensor(slots + free)
    T = len(slots)
    assert T * H > 4096 and used + 3 <= N
    k, v = ou.normal((T, H, D), dtype, g), ou.normal((T, H, D), dtype, g)
    k[:, :, 0] = torch.arange(T)[:, None] / 4.0            # quotients that are ties, or near them
    k[3], v[4] = 0.25, 0
    v[:, 0] = torch.arange(D) % 64 / 8.0
    v[6] *= 1e-30 if dtype != torch.float16 else 1e-7
    kc, vc = empty_pools(N, H, D, B, 0xee)
    got = [x.cuda() for x in (kc, vc)]
    ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), *got, slots.cuda())
    for pool, rows, side in ((kc, k, False), (vc, v, True)):
        ou.write4(pool, rows, slots, B, side)
    for a, b in zip(got, (kc, vc)):
        assert torch.equal(a.cpu(), b)
    back = [torch.full_like(k, 7).cuda(), torch.full_like(v, 7).cuda()]
    ops.pa_gather_cache_int4(*back, *got, slots.cuda())
    for x, rows in zip(back, (k, v)):
        want = ou.values4(rows).to(torch.float32).to(dtype)
        want[slots < 0] = 7
        assert torch.equal(x.cpu(), want)
    assert pa.pa_get_device_error() == 0


def test_a_row_that_is_not_finite_keeps_to_itself():
    D, B, T, H = 128, 16, 1024, 5
    g = ou.gen(4)
    k, v = ou.normal((T, H, D), torch.bfloat16, g), ou.normal((T, H, D), torch.bfloat16, g)
    slots = torch.arange(T)
    pools = []
    for bad in (False, True):
        if bad:
            k[5, 1, 3], k[17, 0, 70], v[5, 1, 3], v[30, 2, 9] = float("nan"), float("inf"), float("-inf"), float("nan")
        kc, vc = (x.cuda() for x in empty_pools(T // B, H, D, B))
        ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), kc, vc, slots.cuda())
        back = [torch.zeros_like(k).cuda(), torch.zeros_like(k).cuda()]
        ops.pa_gather_cache_int4(*back, kc, vc, slots.cuda())
        pools.append([x.cpu() for x in back])
    for x, y in zip(*pools):
        x, y = x.unflatten(2, (2, 64)), y.unflatten(2, (2, 64))
        same = (x == y).all(-1)
        assert (~same).sum() <= 2      # the groups that hold such a value


@pytest.mark.parametrize("write", [True, False])
def test_a_slot_past_the_pool_is_flagged(write):
    k = torch.ones(2, 1, 64, dtype=torch.float16).cuda()
    kc, vc = (x.cuda() for x in empty_pools(2, 1, 64, 8))
    fn = ops.pa_reshape_and_cache_int4 if write else ops.pa_gather_cache_int4
    fn(k, k.clone(), kc, vc, torch.tensor([16, 3]).cuda())
    assert pa.pa_get_device_error() == pa.DEVERR_SLOT
    many = torch.ones(5000, 1, 64, dtype=torch.float16).cuda()
    slots = torch.full((5000,), -1, dtype=torch.int64)
    slots[100:108] = torch.arange(12, 20)      # a run that leaves the pool
    fn(many, many.clone(), kc, vc, slots.cuda())
    assert pa.pa_get_device_error() == pa.DEVERR_SLOT


LENS = [1, 0, 7, 8, 9, 15, 16, 17, 31, 33, 130, 257]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_decode_whole(group, B, D, dtype):
    # 0xff bytes in the free tokens: NaN scales and zeros
    q, kc, vc, table, rows = build(LENS, 2 * group, 2, D, B, dtype, group + B + D, fill=0xff)
    want = ou.decode(q, rows, LENS, D ** -0.5)
    for part in (0, 32, None):
        got = run(q, kc, vc, table, LENS, partition_size=part)
        assert ou.worst_row(got, want) <= BOUND[dtype]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (16, 4), (40, 17), (100, 40), (300, 4), (64, 300)])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_decode_window(B, window, sinks):
    q, kc, vc, table, rows = build(LENS, 8, 2, 64, B, torch.bfloat16, B + window, fill=0xff)
    want = ou.decode(q, rows, LENS, 64 ** -0.5, window, sinks)
    table = table.clone()
    for s, L in enumerate(LENS):   # blocks without a visible token have left the table
        for j in range(table.shape[1]):
            if j * B + B <= L - window and j * B >= sinks:
                table[s, j] = 1 << 30
    for part in (0, 32, None):
        got = run(q, kc, vc, table, LENS, window=window, num_sinks=sinks, partition_size=part)
        assert ou.worst_row(got, want) <= BOUND[torch.bfloat16]


@pytest.mark.parametrize("spread,offset", [(1e-3, 0.0), (300.0, 0.0), (1.0, 6.0), (1e-3, 0.25)])
def test_decode_scales_of_other_sizes(spread, offset):
    lens = [200, 64, 5]
    q, kc, vc, table, rows = build(lens, 4, 1, 128, 16, torch.bfloat16, 5, spread=spread, offset=offset)
    q = (q.float() / (spread + 8 * abs(offset))).bfloat16()   # scores of a few units
    want = ou.decode(q, rows, lens, 128 ** -0.5)
    assert ou.worst_row(run(q, kc, vc, table, lens), want) <= BOUND[torch.bfloat16]


def test_decode_rising_scores_and_scales():
    """The softmax reference and the unit of V's scales move many times: keys
    ever closer to the query, values ever larger."""
    L, D = 512, 64
    g = ou.gen(11)
    q = ou.normal((1, 1, D), torch.float16, g)
    k = (q[0] * torch.linspace(0.0, 4.0, L)[:, None] + 0.1 * ou.normal((L, D), torch.float32, g))[:, None].half()
    v = (ou.normal((L, 1, D), torch.float32, g) * torch.exp2(torch.linspace(-10, 8, L))[:, None, None]).half()
    table, N = ou.tables_of([L], 16, 3)
    slots = torch.tensor([int(table[0, t // 16]) * 16 + t % 16 for t in range(L)])
    kc, vc = (x.cuda() for x in empty_pools(N, 1, D, 16))
    ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), kc, vc, slots.cuda())
    want = ou.decode(q, lambda s: (ou.values4(k), ou.values4(v)), [L], D ** -0.5)
    for part in (0, 64):
        assert ou.worst_row(run(q, kc, vc, table, [L], partition_size=part), want) <= BOUND[torch.float16]


def test_decode_of_equal_values_and_zero_queries():
    lens, D = [70], 64
    k = torch.zeros(70, 1, D, dtype=torch.float16)
    v = torch.full((70, 1, D), 0.75, dtype=torch.float16)
    table, N = ou.tables_of(lens, 8, 1)
    slots = torch.tensor([int(table[0, t // 8]) * 8 + t % 8 for t in range(70)])
    kc, vc = (x.cuda() for x in empty_pools(N, 1, D, 8))
    ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), kc, vc, slots.cuda())
    out = run(torch.zeros(1, 2, D, dtype=torch.float16), kc, vc, table, lens)
    assert torch.equal(out.cpu(), torch.full((1, 2, D), 0.75, dtype=torch.float16))


def test_long_context_partitions():
    lens = [9001, 300, 4096]
    q, kc, vc, table, rows = build(lens, 4, 1, 64, 16, torch.float16, 21)
    want = ou.decode(q, rows, lens, 64 ** -0.5)
    for part in (None, 32, 1024, 0):
        assert ou.worst_row(run(q, kc, vc, table, lens, partition_size=part), want) <= BOUND[torch.float16]


def test_refused_ids_and_lengths():
    lens = [40, 33]
    q, kc, vc, table, rows = build(lens, 2, 1, 64, 16, torch.float16, 8)
    table = table.clone()
    table[0, 1] = 1 << 20     # tokens 16..31 of sequence 0 drop out
    out = torch.zeros_like(q, device="cuda")
    ops.pa_decode_int4(out, q.cuda(), kc, vc, table.cuda(), torch.tensor([40, 33], dtype=torch.int32).cuda(), 0.125)
    assert pa.pa_get_device_error() == pa.DEVERR_BLOCK_ID
    k, v = rows(0)
    keep = torch.cat([torch.arange(16), torch.arange(32, 40)])
    want = torch.cat([ou.attend(q[:1], k[keep], v[keep], 23, 0.125, 0, 0),
                      ou.attend(q[1:], *rows(1), 32, 0.125, 0, 0)])
    assert ou.worst_row(out, want) <= BOUND[torch.float16]
    ops.pa_decode_int4(out, q.cuda(), kc, vc, table.cuda(), torch.tensor([-1, 33], dtype=torch.int32).cuda(), 0.125)
    assert pa.pa_get_device_error() == pa.DEVERR_CONTEXT_LEN
    assert torch.equal(out[0].cpu(), torch.zeros_like(q[0]))


def test_order_graph_and_prepared_calls():
    lens = [300, 17, 1000, 64]
    q, kc, vc, table, rows = build(lens, 8, 2, 128, 16, torch.bfloat16, 13)
    base = run(q, kc, vc, table, lens, partition_size=128)
    order = pa.longest_first(lens).cuda()
    assert torch.equal(base, run(q, kc, vc, table, lens, partition_size=128, seq_order=order))
    out, qd = torch.zeros_like(base), q.cuda()
    call = pa.prepare_decode_int4(out, qd, kc, vc, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                  128 ** -0.5, partition_size=128)
    call()
    assert torch.equal(out, base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, base)
    assert pa.pa_get_device_error() == 0


def test_two_streams_at_once():
    """Calls without a workspace of the caller's share nothing."""
    lens = [3000] * 2
    q, kc, vc, table, rows = build(lens, 8, 1, 64, 16, torch.bfloat16, 14)
    base = run(q, kc, vc, table, lens, partition_size=64)
    lens_d, table_d, qd = torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), q.cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(base) for _ in range(8)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(8):
        for st, o in zip(streams, outs):
            ops.pa_decode_int4(o[i], qd, kc, vc, table_d, lens_d, 0.125, partition_size=64, stream=st)
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert torch.equal(o, base)
    assert pa.pa_get_device_error() == 0


def test_blocks_of_byte_pools_are_copied():
    lens = [50]
    q, kc, vc, table, rows = build(lens, 4, 2, 64, 16, torch.float16, 15)
    base = run(q, kc, vc, table, lens)
    free = [b for b in range(kc.shape[0]) if b not in table[0].tolist()]
    pairs = torch.tensor([[int(table[0, 1]), free[0]], [-1, -1]], dtype=torch.int64).cuda()
    pa.pa_copy_blocks(kc, vc, kc, vc, pairs)
    table = table.clone()
    old = int(table[0, 1])
    table[0, 1] = free[0]
    kc[old], vc[old] = 0xff, 0xff
    assert torch.equal(run(q, kc, vc, table, lens), base)


def row_errors(got, want):
    return ((got.double().cpu() - want).norm(dim=-1) / want.norm(dim=-1))


@pytest.mark.parametrize("big", [float("inf"), float("nan"), 2.0 ** 40])
@pytest.mark.parametrize("group", [2, 4, 8])
def test_a_head_of_another_size_keeps_to_itself(group, big):
    lens = [200, 33]
    q, kc, vc, table, rows = build(lens, 2 * group, 2, 128, 16, torch.bfloat16, group)
    want = ou.decode(q, rows, lens, 128 ** -0.5)
    q[:, 1] *= big
    q[:, group + 1, 5] = big
    others = [h for h in range(2 * group) if h % group != 1]
    for part in (0, 64):
        got = run(q, kc, vc, table, lens, partition_size=part)
        assert float(row_errors(got, want)[:, others].max()) <= BOUND[torch.bfloat16]
        if big != 2.0 ** 40:
            assert not torch.isfinite(got[:, 1]).any()


@pytest.mark.parametrize("group", [2, 8])
@pytest.mark.parametrize("bad", ["inf", "nan", "span"])
def test_a_group_of_v_that_is_not_finite_keeps_to_its_dims(bad, group):
    """One token's first 64 dims of V: the other dims' output stays what it is."""
    L, D, B = 150, 128, 16
    g = ou.gen(31)
    k, v = (ou.normal((L, 1, D), torch.float32, g) for _ in range(2))
    q = ou.normal((1, group, D), torch.bfloat16, g)
    want = ou.attend(q, ou.values4(k), ou.values4(v), L - 1, D ** -0.5, 0, 0)[..., 64:]
    v[77, 0, 3] = 3e38 if bad == "span" else float(bad)
    v[77, 0, 9] = -3e38 if bad == "span" else 1.0
    N = -(-L // B)
    kc, vc = (x.cuda() for x in empty_pools(N, 1, D, B))
    ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), kc, vc, torch.arange(L).cuda())
    for part in (0, 32):
        got = run(q, kc, vc, torch.arange(N, dtype=torch.int32).reshape(1, -1), [L], partition_size=part)
        assert not torch.isfinite(got[..., :64]).any()
        assert float(row_errors(got[..., 64:], want).max()) <= BOUND[torch.bfloat16]


@pytest.mark.parametrize("size", [2.0 ** 116, 2.0 ** -116])
def test_values_of_far_sizes(size):
    L, D, B = 150, 64, 16
    g = ou.gen(32)
    k, v = (ou.normal((L, 1, D), torch.float32, g) for _ in range(2))
    v = v.bfloat16().float() * size
    q = ou.normal((1, 4, D), torch.bfloat16, g)
    N = -(-L // B)
    kc, vc = (x.cuda() for x in empty_pools(N, 1, D, B))
    ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), kc, vc, torch.arange(L).cuda())
    want = ou.attend(q, ou.values4(k), ou.values4(v), L - 1, D ** -0.5, 0, 0)
    got = run(q, kc, vc, torch.arange(N, dtype=torch.int32).reshape(1, -1), [L])
    assert float(row_errors(got, want).max()) <= BOUND[torch.bfloat16]


def test_prepared_calls_on_a_stream_of_their_own():
    """The handle's counters are zero before any stream uses them."""
    lens = [3000] * 2
    q, kc, vc, table, rows = build(lens, 8, 1, 64, 16, torch.bfloat16, 14)
    base = run(q, kc, vc, table, lens, partition_size=64)
    lens_d, table_d, qd = torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), q.cuda()
    side = torch.cuda.Stream()
    out = torch.zeros_like(base)
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(8):
        busy = busy @ busy * 1e-3
        call = pa.prepare_decode_int4(out, qd, kc, vc, table_d, lens_d, 0.125, partition_size=64)
        call(side)
        side.synchronize()
        assert torch.equal(out, base)
        out.zero_()
        torch.cuda.synchronize()
