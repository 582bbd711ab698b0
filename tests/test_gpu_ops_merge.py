"""The partitions' merge where a thread block's shared memory cannot hold every
partition's weight (group x partitions of them): one partition after the other
then.  The bounds are those of the other decode tests."""

import pytest
import torch

import opsutil as ou
import paged_kv_cache_449_b200 as pa
import pagedutil as pu
from paged_kv_cache_449_b200 import ops
from test_gpu_int4 import BOUND

pytestmark = pytest.mark.gpu


# wide thread blocks of 16-token blocks hold 12288 (fp32: 8192) weights; 8 heads x 1563 (1126) partitions of 16
@pytest.mark.parametrize("dtype,L", [(torch.bfloat16, 25000), (torch.float32, 18003)])
def test_window_decode(dtype, L):
    B, D, group = 16, 64, 8
    g = ou.gen(L)
    table, N = ou.tables_of([L, 100], B, 1)
    k, v = (ou.normal(pa.pool_shape(N, 1, D, B, dtype), dtype, g) for _ in range(2))
    q = ou.normal((2, group, D), dtype, g)
    want = ou.decode(q, lambda s: tuple(ou.pool_rows(x, table[s, :-(-n // B)].long(), n) for x, n in
                                        zip((k, v), ((L, 100)[s],) * 2)), [L, 100], 0.5, L - 40, 3).numpy()
    qd, kd, vd, td, ld = (x.cuda() for x in (q, k, v, table, torch.tensor([L, 100], dtype=torch.int32)))
    counters = torch.zeros(2, dtype=torch.int32, device="cuda")
    for part in (16, 512):
        for _ in range(2):
            out = torch.full_like(qd, float("nan"))
            ops.pa_decode_window(out, qd, None, None, kd, vd, td, ld, 0.5, L - 40, 3, partition_size=part, counters=counters)
            torch.cuda.synchronize()
            assert pa.pa_get_device_error() == 0 and not counters.any()
            pu.check_tolerance(pu.as_f64(out), want, dtype)


# 13824 weights; 8 heads x 1735 partitions of 32
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_4_bit_decode(dtype):
    L, B, D, group = 55500, 16, 64, 8
    g = ou.gen(5)
    k, v = (ou.normal((L, 1, D), torch.float32, g).to(dtype) for _ in range(2))
    N = -(-L // B)
    pools = [torch.zeros(ops.int4_pool_shape(N, 1, D, B), dtype=torch.uint8, device="cuda") for _ in range(2)]
    ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), *pools, torch.arange(L).cuda())
    q = ou.normal((1, group, D), dtype, g)
    want = ou.attend(q, ou.values4(k), ou.values4(v), L - 1, 0.5, 0, 0)
    table, lens = torch.arange(N, dtype=torch.int32).reshape(1, -1).cuda(), torch.tensor([L], dtype=torch.int32).cuda()
    counters = torch.zeros(1, dtype=torch.int32, device="cuda")
    for part in (32, 1024):
        out = torch.full_like(q, float("nan"), device="cuda")
        ops.pa_decode_int4(out, q.cuda(), *pools, table, lens, 0.5, partition_size=part, counters=counters)
        assert pa.pa_get_device_error() == 0 and not counters.any()
        assert ou.worst_row(out, want) <= BOUND[dtype]
