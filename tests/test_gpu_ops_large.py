"""Pools whose tiles lie past 2^32 bytes and 2^32 elements, and contexts of tens of
thousands of tokens.  The pools' last blocks hold what a small pool holds, so
the results have to be the small pool's bit for bit."""

import pytest
import torch

import opsutil as ou
import paged_kv_cache_449_b200 as pa
from paged_kv_cache_449_b200 import ops

pytestmark = pytest.mark.gpu

S, HQ, H, D = 3, 8, 8, 128
LENS = [70, 33, 129]


def setting(B, N, seed):
    """Table and slots of the sequences in a pool of N blocks, in its last ones."""
    table, used = ou.tables_of(LENS, B, seed)
    table = table + (N - used)
    slots = [int(table[s, t // B]) * B + t % B for s, n in enumerate(LENS) for t in range(n)]
    return table.cuda(), torch.tensor(slots, dtype=torch.int64).cuda(), used


def inputs(T, dtype, seed):
    g = ou.gen(seed)
    q, k, v = (ou.normal((T, h, D), dtype, g).cuda() for h in (HQ, H, H))
    return q, k, v, torch.arange(T, dtype=torch.int64).cuda(), pa.rope_frequencies(D, 10000.0)[0].cuda()


@pytest.mark.parametrize("B", [8, 16, 32])
def test_4_bit_pools_past_32_bits(B):
    T = sum(LENS)
    q, k, v, positions, freq = inputs(T, torch.bfloat16, 3)
    lens = torch.tensor(LENS, dtype=torch.int32).cuda()
    results = []
    used = setting(B, 10 ** 6, 1)[2]
    tile = H * (B * D * 9 // 16)
    for N in (used, (1 << 33) // (tile * 16 // 9) + used):       # 2^33 elements, 4.5 GiB a pool
        table, slots, _ = setting(B, N, 1)
        pools = [torch.empty(pa.int4_pool_shape(N, H, D, B), dtype=torch.uint8, device="cuda") for _ in range(2)]
        assert N == used or pools[0].numel() > 1 << 32
        back, out = [torch.empty_like(k) for _ in range(4)], [torch.empty(S, HQ, D, dtype=k.dtype, device="cuda") for _ in range(2)]
        ops.pa_reshape_and_cache_int4(k, v, *pools, slots)
        ops.pa_gather_cache_int4(*back[:2], *pools, slots)
        ops.pa_decode_int4(out[0], q[:S].contiguous(), *pools, table, lens, D ** -0.5)
        turned = torch.empty_like(q)
        ops.pa_rope_and_cache_int4(turned, q, k, v, *pools, positions, slots, freq)
        ops.pa_gather_cache_int4(*back[2:], *pools, slots)
        ops.pa_decode_int4(out[1], turned[:S].contiguous(), *pools, table, lens, D ** -0.5, window=40, num_sinks=3,
                           partition_size=32)
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == 0
        results.append([x.cpu() for x in back + out])
        del pools
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("B", [8, 16, 32])
def test_rotary_write_and_windows_past_32_bits(B):
    T = sum(LENS)
    q, k, v, positions, freq = inputs(T, torch.bfloat16, 4)
    lens = torch.tensor(LENS, dtype=torch.int32).cuda()
    start = torch.tensor([0, 5, 38, 100], dtype=torch.int32).cuda()
    results = []
    used = setting(B, 10 ** 6, 2)[2]
    for N in (used, (1 << 32) // (H * B * D) + used):            # 2^32 elements, 8 GiB a pool
        table, slots, _ = setting(B, N, 2)
        pools = [torch.empty(pa.pool_shape(N, H, D, B, k.dtype), dtype=k.dtype, device="cuda") for _ in range(2)]
        turned = torch.empty_like(q)
        out = [torch.empty(S, HQ, D, dtype=k.dtype, device="cuda") for _ in range(2)]
        ops.pa_rope_and_cache(turned, q, k, v, *pools, positions, slots, freq)
        ops.pa_decode_window(out[0], turned[:S].contiguous(), None, None, *pools, table, lens, D ** -0.5, 40, 3)
        ops.pa_decode_window(out[1], turned[:S].contiguous(), k[:S].contiguous(), v[:S].contiguous(), *pools, table, lens,
                             D ** -0.5, 64, 0, partition_size=32)
        chunk = torch.empty_like(q[:100])
        ops.pa_prefill_window(chunk, turned[:100].contiguous(), *pools, table, lens, start, D ** -0.5, 40, 3)
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == 0
        results.append([x.cpu() for x in out + [chunk]])
        del pools
    assert all(torch.isfinite(x).all() for x in results[0])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("group", [4, 8])
@pytest.mark.parametrize("spread", [0.05, 1.0])
def test_a_context_of_30000_tokens_in_one_pass(group, spread):
    """Near-uniform weights: the error may not grow with the tokens that one
    warp adds up.  The bound is the output's rounding (2^-11) and that of P
    times V's scale (2^-11 times 2.55, taken as 3; test_gpu_int4)."""
    L, dtype = 30001, torch.float16
    g = ou.gen(group)
    k, v = ((ou.normal((L, 1, D), torch.float32, g) * f).to(dtype) for f in (spread, 1.0))
    B = 16
    N = -(-L // B)
    table = torch.arange(N, dtype=torch.int32).reshape(1, -1).cuda()
    pools = [torch.zeros(pa.int4_pool_shape(N, 1, D, B), dtype=torch.uint8, device="cuda") for _ in range(2)]
    ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), *pools, torch.arange(L).cuda())
    q = ou.normal((1, group, D), dtype, g)
    want = ou.attend(q, ou.values4(k), ou.values4(v), L - 1, D ** -0.5, 0, 0)
    for part in (0, 8192, None):
        out = torch.empty_like(q, device="cuda")
        ops.pa_decode_int4(out, q.cuda(), *pools, table, torch.tensor([L], dtype=torch.int32).cuda(), D ** -0.5,
                           partition_size=part)
        assert ou.worst_row(out, want) <= ou.U[dtype] + 3 * 2.0 ** -11
