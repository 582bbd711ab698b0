"""Rows that 4 bits cannot hold (pa/ops.h: a group that is not finite, or whose
span is not, reads back as values that are not finite): exactly those groups,
all 64 values of them, through the row-by-row kernels, the grouped ones and the
rotary step's write."""

import pytest
import torch

import opsutil as ou
import paged_kv_cache_449_b200 as pa
from paged_kv_cache_449_b200 import ops

pytestmark = pytest.mark.gpu

H, D = 5, 128


def spoil(k, v):
    """Bad values into k and v; the (token, head, group) entries that hold one, for each."""
    inf, nan = float("inf"), float("nan")
    bad = [[(5, 1, 3, inf), (5, 4, 127, nan), (17, 0, 70, inf), (18, 2, 64, -inf)],
           [(0, 0, 0, nan), (5, 1, 3, -inf), (30, 2, 9, nan), (31, 3, 63, inf)]]
    groups = []
    for x, entries in zip((k, v), bad):
        for t, h, d, value in entries:
            x[t, h, d] = value
        x[21, 2, 64:] = inf                  # whole groups
        x[22, 2, :64] = -inf
        places = {(t, h, d // 64) for t, h, d, _ in entries} | {(21, 2, 1), (22, 2, 0)}
        if x.dtype != torch.float16:         # finite, but its span is not
            x[23, 1, 70], x[23, 1, 71] = 3e38, -3e38
            places.add((23, 1, 1))
        groups.append(places)
    return groups


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("form", ["rows", "groups", "groups at scattered slots", "rotary"])
def test_bad_groups_read_back_as_such(form, B, dtype):
    T = 1024 if form.startswith("groups") else 96          # (more than 4096 rows go by groups)
    g = ou.gen(B)
    k, v = (ou.normal((T, H, D), dtype, g) for _ in range(2))
    slots = torch.randperm(T, generator=g) if form == "groups at scattered slots" else torch.arange(T)
    q = ou.normal((T, H, D), dtype, g).cuda()
    results = []
    for spoilt in (False, True):
        groups = spoil(k, v) if spoilt else None
        pools = [torch.zeros(ops.int4_pool_shape(-(-T // B), H, D, B), dtype=torch.uint8, device="cuda") for _ in range(2)]
        if form == "rotary":       # no rotation, no norm: the write alone
            ops.pa_rope_and_cache_int4(torch.empty_like(q), q, k.cuda(), v.cuda(), *pools, slots.cuda(), slots.cuda(), None)
        else:
            ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), *pools, slots.cuda())
        back = [torch.zeros(T, H, D, dtype=dtype, device="cuda") for _ in range(2)]
        ops.pa_gather_cache_int4(*back, *pools, slots.cuda())
        results.append([x.cpu() for x in back])
    assert pa.pa_get_device_error() == 0
    for clean, got, places in zip(*results, groups):
        assert torch.isfinite(clean).all()
        clean, got = clean.unflatten(2, (2, 64)), got.unflatten(2, (2, 64))
        differs = {tuple(i) for i in (clean != got).any(-1).nonzero().tolist()}
        assert differs == places
        for t, h, n in places:
            assert not torch.isfinite(got[t, h, n]).any()
