"""Rotary positions, head norms and the cache write in one pass, against the
formulas in 64 bits.

Tolerance: an element a cos - b sin is a sum of two products of fp32 values,
each factor within a few fp32 roundings (norm: the fp32 sum of D squares, a
square root, a division, two products; sine and cosine within 2 ulp of an angle
within 2^-25 of a turn), so its error is at most 40 * 2^-24 of |a| + |b|; the
result is then rounded once, u relative.
"""

import pytest
import torch

import opsutil as ou
import paged_kv_cache_449_b200 as pa
from paged_kv_cache_449_b200 import ops

pytestmark = pytest.mark.gpu


def inputs(T, Hq, H, D, B, dtype, seed, fused=False, far=2048):
    g = ou.gen(seed)
    q, k, v = (ou.normal((T, h, D), dtype, g) for h in (Hq, H, H))
    N = -(-T // B) + 2
    slots = torch.randperm(N * B, generator=g)[:T]
    pos = torch.randint(0, far, (T,), generator=g)
    if fused:
        wide = torch.cat([x.flatten(1) for x in (q, k, v)], 1).cuda()
        qd, kd, vd = (x.unflatten(1, (-1, D)) for x in wide.split([Hq * D, H * D, H * D], 1))
    else:
        qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    return (q, k, v), (qd, kd, vd), N, slots, pos


def close(got, want, source, weight, dtype):
    """|got - want| within the bound above; rows [.., D]."""
    size = source.double().abs().amax(-1, keepdim=True)
    if weight is not None:
        rms = source.double().square().mean(-1, keepdim=True).sqrt()
        size = size / rms.clamp(min=1e-30) * weight.double().abs().max()
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    bound = ou.U[dtype] * want.abs() + 80 * 2.0 ** -24 * size
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25      # subnormal results
    assert (err <= bound * 2.0).all() if dtype == torch.float32 else (err <= bound * (1 + 1e-3)).all()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,R,B", [(64, 64, 8), (64, 16, 16), (128, 128, 16), (128, 64, 32), (128, 96, 8), (128, 0, 16)])
def test_rows_and_pools(D, R, B, dtype, interleaved, norm):
    T, Hq, H = 13, 6, 3
    (q, k, v), (qd, kd, vd), N, slots, pos = inputs(T, Hq, H, D, B, dtype, D + R + B, fused=True, far=1000000)
    slots[4] = -1
    freq = pa.rope_frequencies(R, 500000.0)[0] if R else None
    g = ou.gen(1)
    qw, kw = (1 + 0.2 * ou.normal((D,), torch.float32, g)).to(dtype), (1 + 0.2 * ou.normal((D,), torch.float32, g)).to(dtype)
    if not norm:
        qw = kw = None
    shape = pa.pool_shape(N, H, D, B, dtype)
    kc, vc = (torch.full(shape, 3.0, dtype=dtype, device="cuda") for _ in range(2))
    q_out = torch.empty(T, Hq, D, dtype=dtype, device="cuda")
    ops.pa_rope_and_cache(q_out, qd, kd, vd, kc, vc, pos.cuda(), slots.cuda(), None if freq is None else freq.cuda(),
                          interleaved=interleaved, rope_scale=1.25, eps=1e-5,
                          q_weight=None if qw is None else qw.cuda(), k_weight=None if kw is None else kw.cuda())
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    close(q_out.cpu(), ou.rope(q, pos, freq, interleaved, 1.25, qw, 1e-5), q, qw, dtype)
    want = ou.rope(k, pos, freq, interleaved, 1.25, kw, 1e-5)
    kc, vc = kc.cpu(), vc.cpu()
    touched = torch.zeros(N, B, dtype=torch.bool)
    for i in range(T):
        if i != 4:
            s = int(slots[i])
            close(ou.pool_row(kc, s, B), want[i], k[i], kw, dtype)
            assert torch.equal(ou.pool_row(vc, s, B), v[i])
            touched[s // B, s % B] = True
    for pool in (kc, vc):
        assert (pool[~touched[:, None, None, :, None].expand_as(pool)] == 3.0).all()


def test_far_positions():
    """Angles of a million turns and more keep their place."""
    D, T = 64, 8
    q = torch.zeros(T, 1, D)
    q[..., :32] = 1.0
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 10 ** 7 + 3, 2 ** 30 + 5, 2 ** 31 - 1, -5, 123456789])
    freq = pa.rope_frequencies(D, 10000.0)[0]
    kc = torch.zeros(pa.pool_shape(1, 1, D, 8, torch.float32), device="cuda")
    out = torch.empty_like(q, device="cuda")
    ops.pa_rope_and_cache(out, q.cuda(), q.cuda(), q.cuda(), kc, kc.clone(), pos.cuda(), torch.arange(8).cuda(), freq.cuda())
    assert (out.cpu().double() - ou.rope(q, pos, freq, False, 1.0, None, 0)).abs().max() <= 80 * 2.0 ** -24


def test_one_token_in_place_and_no_tokens():
    D, B = 128, 16
    (q, k, v), (qd, kd, vd), N, slots, pos = inputs(1, 4, 1, D, B, torch.bfloat16, 2)
    freq = pa.rope_frequencies(D)[0].cuda()
    pools = [torch.zeros(pa.pool_shape(N, 1, D, B, torch.bfloat16), device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    out = torch.empty_like(qd)
    ops.pa_rope_and_cache(out, qd, kd, vd, *pools[:2], pos.cuda(), slots.cuda(), freq)
    ops.pa_rope_and_cache(qd, qd, kd, vd, *pools[2:], pos.cuda(), slots.cuda(), freq)
    assert torch.equal(out, qd) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    ops.pa_rope_and_cache(out[:0], qd[:0], kd[:0], vd[:0], *pools[:2], pos[:0].cuda(), slots[:0].cuda(), freq)
    assert pa.pa_get_device_error() == 0


def test_a_slot_past_the_pool_is_flagged():
    D, B = 64, 8
    (q, k, v), (qd, kd, vd), N, slots, pos = inputs(3, 2, 1, D, B, torch.float16, 2)
    slots[1] = N * B
    kc = torch.zeros(pa.pool_shape(N, 1, D, B, torch.float16), device="cuda", dtype=torch.float16)
    out = torch.zeros_like(qd)
    ops.pa_rope_and_cache(out, qd, kd, vd, kc, kc.clone(), pos.cuda(), slots.cuda(), pa.rope_frequencies(D)[0].cuda())
    assert pa.pa_get_device_error() == pa.DEVERR_SLOT
    assert (out != 0).any(-1).all()       # every query row is there


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,B", [(64, 8), (64, 32), (128, 16)])
@pytest.mark.parametrize("pool", ["fp8", "int4"])
def test_quantised_pools_hold_the_written_rows(pool, D, B, dtype):
    """Every byte equals the plain write of the rows that the native pool gets."""
    T, Hq, H = 11, 4, 2
    (q, k, v), (qd, kd, vd), N, slots, pos = inputs(T, Hq, H, D, B, dtype, D + B, fused=True)
    slots[2] = -1
    w = (1 + 0.1 * ou.normal((D,), torch.float32, ou.gen(3))).to(dtype).cuda()
    freq = pa.rope_frequencies(D)[0].cuda()
    native = [torch.zeros(pa.pool_shape(N, H, D, B, dtype), device="cuda", dtype=dtype) for _ in range(2)]
    outs = [torch.empty(T, Hq, D, dtype=dtype, device="cuda") for _ in range(2)]
    args = (pos.cuda(), slots.cuda(), freq)
    kw = dict(q_weight=w, k_weight=w, interleaved=True)
    ops.pa_rope_and_cache(outs[0], qd, kd, vd, *native, *args, **kw)
    at = [int(s) if s >= 0 else 0 for s in slots]
    rows = torch.stack([ou.pool_row(native[0].cpu(), s, B) for s in at]).cuda()
    if pool == "fp8":
        scales = torch.tensor([0.02, 0.03]).cuda(), torch.tensor([0.01, 0.05]).cuda()
        a, b = ([torch.full(pa.fp8_pool_shape(N, H, D, B), 9, device="cuda", dtype=torch.uint8) for _ in range(2)]
                for _ in range(2))
        ops.pa_rope_and_cache_fp8(outs[1], qd, kd, vd, *a, *scales, *args, **kw)
        pa.pa_reshape_and_cache_fp8(rows, vd.contiguous(), *b, slots.cuda(), *scales)
    else:
        a, b = ([torch.full(pa.int4_pool_shape(N, H, D, B), 9, device="cuda", dtype=torch.uint8) for _ in range(2)]
                for _ in range(2))
        ops.pa_rope_and_cache_int4(outs[1], qd, kd, vd, *a, *args, **kw)
        ops.pa_reshape_and_cache_int4(rows, vd.contiguous(), *b, slots.cuda())
    assert torch.equal(outs[0], outs[1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("pool", ["native", "int4"])
def test_a_serving_step(pool):
    """The operators together, captured once and replayed: every sequence's
    newest token normed, rotated and written, then attended with a window."""
    S, Hq, H, D, B, W, K = 5, 8, 2, 64, 16, 40, 3
    lens = [1, 18, 64, 100, 47]
    g = ou.gen(4)
    table, N = ou.tables_of(lens, B, 4)
    freq = pa.rope_frequencies(D, 10000.0)[0]
    w = (1 + 0.1 * ou.normal((D,), torch.float32, g)).bfloat16()
    past = ou.normal((sum(lens), H, D), torch.bfloat16, g), ou.normal((sum(lens), H, D), torch.bfloat16, g)
    pos = torch.tensor([t for n in lens for t in range(n)])
    slots = torch.tensor([int(table[s, t // B]) * B + t % B for s, n in enumerate(lens) for t in range(n)])
    last = torch.tensor([sum(lens[:s + 1]) - 1 for s in range(S)])
    q = ou.normal((sum(lens), Hq, D), torch.bfloat16, g)
    if pool == "native":
        pools = [torch.zeros(pa.pool_shape(N, H, D, B, torch.bfloat16), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    else:
        pools = [torch.zeros(pa.int4_pool_shape(N, H, D, B), device="cuda", dtype=torch.uint8) for _ in range(2)]
    old = [i for i in range(sum(lens)) if i not in last.tolist()]
    rope = ops.pa_rope_and_cache if pool == "native" else ops.pa_rope_and_cache_int4
    qo = torch.empty(len(old), Hq, D, dtype=torch.bfloat16, device="cuda")
    kw = dict(q_weight=w.cuda(), k_weight=w.cuda())
    rope(qo, q[old].cuda(), past[0][old].cuda(), past[1][old].cuda(), *pools, pos[old].cuda(), slots[old].cuda(), freq.cuda(), **kw)
    qn, kn, vn = q[last].cuda(), past[0][last].cuda(), past[1][last].cuda()
    qr, out = torch.empty_like(qn), torch.empty_like(qn)
    lens_d, table_d = torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda()
    write = pa.prepare_rope_and_cache(qr, qn, kn, vn, *pools, pos[last].cuda(), slots[last].cuda(), freq.cuda(), **kw)
    if pool == "native":
        attend = pa.prepare_decode_window(out, qr, None, None, *pools, table_d, lens_d, 0.125, W, K)
    else:
        attend = pa.prepare_decode_int4(out, qr, *pools, table_d, lens_d, 0.125, window=W, num_sinks=K)
    write()
    attend()
    torch.cuda.synchronize()
    base, qs = out.clone(), qr.cpu()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        write()
        attend()
    out.zero_()
    qr.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, base) and pa.pa_get_device_error() == 0
    # the stored rows are the rounded ones; the attention over them in 64 bits
    if pool == "native":
        rows = lambda s: tuple(ou.pool_rows(x.cpu(), table[s, :-(-lens[s] // B)].long(), lens[s]) for x in pools)  # noqa: E731
    else:
        back = [torch.zeros(sum(lens), H, D, device="cuda") for _ in range(2)]
        ops.pa_gather_cache_int4(*back, *pools, slots.cuda())
        rows = lambda s: tuple(x.cpu().double()[sum(lens[:s]):sum(lens[:s + 1])] for x in back)  # noqa: E731
    want = ou.decode(qs, rows, lens, 0.125, W, K)
    assert ou.worst_row(base, want) <= ou.U[torch.bfloat16] + (2.0 ** -8 if pool == "native" else 3 * 2.0 ** -11)
