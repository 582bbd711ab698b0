"""The windowed decode's bounded waits run out without a fault or a hang, through
the test hooks of include/pa_test.h (see test_gpu_timeout): one warp of one
thread block leaves its first stage unfilled; the block waits (bounded) for its
other copies, reports PA_DEVERR_TIMEOUT and ends; a partition counts as empty,
its merge still runs and brings the counters back to zero."""

import pytest
import torch

import opsutil as ou
import paged_kv_cache_449_b200 as pa
import pagedutil as pu
from paged_kv_cache_449_b200 import ops
from test_gpu_timeout import LIMIT_NS, hooked, test_lib  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

LENS, HQ, H, B, WINDOW, SINKS = [300, 130, 77, 1], 16, 4, 16, 150, 4


@pytest.mark.parametrize("part", [0, 32])
@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float16, 64), (torch.float32, 64)])
def test_window_decode_timeout_path(hooked, dtype, D, part):  # noqa: F811
    g = ou.gen(D)
    table, N = ou.tables_of(LENS, B, D)
    k, v = (ou.normal(pa.pool_shape(N, H, D, B, dtype), dtype, g) for _ in range(2))
    q = ou.normal((len(LENS), HQ, D), dtype, g)
    want = ou.decode(q, lambda s: tuple(ou.pool_rows(x, table[s, :-(-LENS[s] // B)].long(), LENS[s]) for x in (k, v)),
                     LENS, 0.1, WINDOW, SINKS).numpy()
    qd, kd, vd, td, ld = (x.cuda() for x in (q, k, v, table, torch.tensor(LENS, dtype=torch.int32)))
    counters = torch.zeros(len(LENS) * H, dtype=torch.int32, device="cuda")
    args = (qd, None, None, kd, vd, td, ld, 0.1, WINDOW, SINKS)
    assert hooked.pa_test_set_hooks(LIMIT_NS, 1) == 0
    out = torch.zeros_like(qd)
    ops.pa_decode_window(out, *args, partition_size=part, counters=counters)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == pa.DEVERR_TIMEOUT
    # every other sequence, and the first one's other kv heads, are as ever
    got, group = pu.as_f64(out), HQ // H
    pu.check_tolerance(got[1:], want[1:], dtype)
    pu.check_tolerance(got[0, group:], want[0, group:], dtype)
    assert torch.isfinite(out).all() and not counters.any()
    # hooks off: the next call on the same context and counters is the whole attention
    assert hooked.pa_test_set_hooks(1_000_000_000, 0) == 0
    out.fill_(float("nan"))
    ops.pa_decode_window(out, *args, partition_size=part, counters=counters)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0 and not counters.any()
    pu.check_tolerance(pu.as_f64(out), want, dtype)
