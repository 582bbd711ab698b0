"""4-bit decode: how exact the scores are for queries of any size.

The queries' elements lie within a factor of two of one another, so that the
products with the codes (8 or 11 bits times 4) and the sums of q add up without
loss, and what is left can be bounded row by row.  With o = sum p_t v_t the exact output:
  u |o|                                the output's one rounding
  2^-11 sum p_t |s_t (n_t - 7.5)|      p times V's scale, rounded to fp16 for the product
  2 e sum p_t |v_t - o|                an error e of every score: the weights change by 2 e at most
  L 2^-23 sum p_t (|v_t| + |s_t n_t|)  sums of L terms in fp32, each within 2^-23
A score is ks acc + kz sum(q) over two groups of dims, times the scale, less the
reference, in base 2: eight fp32 roundings (2^-24) of at most the sum M of the two
groups' |ks acc| + |kz sum(q)|, and the exponential's 2^-22."""

import math

import pytest
import torch

import opsutil as ou
import paged_kv_cache_449_b200 as pa
from paged_kv_cache_449_b200 import ops

L, D, HQ, SEQS, B = 320, 128, 8, 6, 16


def inputs(dtype, size, seed):
    g = ou.gen(seed)
    k, v = (ou.normal((SEQS * L, 1, D), torch.float32, g).to(dtype) for _ in range(2))
    q = size * (1 + torch.rand(SEQS, HQ, D, generator=g)) * torch.where(torch.rand(SEQS, HQ, D, generator=g) < 0.5, -1.0, 1.0)
    return q.to(dtype), k, v


def parts(x):
    """Codes [T, D], scales and zeros [T, D / 64], float64, of rows [T, 1, D]."""
    codes, scale, zero = ou.quantise4(x.float().numpy())
    return tuple(torch.from_numpy(a).double()[:, 0] for a in (codes, scale, zero))


def reference(q, k, v, dtype):
    """(the outputs in 64 bits, the bound of each row's error in the 2-norm)."""
    want, bound = torch.zeros(SEQS, HQ, D, dtype=torch.float64), torch.zeros(SEQS, HQ, dtype=torch.float64)
    (kn, ks, kz), (vn, vs, _) = parts(k), parts(v)
    kv, vv = ou.values4(k)[:, 0], ou.values4(v)[:, 0]
    wide = lambda x: x.repeat_interleave(64, -1)  # noqa: E731
    scale = D ** -0.5
    for s in range(SEQS):
        rows = slice(s * L, (s + 1) * L)
        vt, centred = vv[rows], (wide(vs[rows]) * (vn[rows] - 7.5)).norm(dim=-1)
        span = vt.norm(dim=-1) + (wide(vs[rows]) * vn[rows]).norm(dim=-1)
        for h in range(HQ):
            x = q[s, h].double()
            p = torch.softmax(kv[rows] @ x * scale, 0)
            o = p @ vt
            acc = (kn[rows] * x).unflatten(-1, (-1, 64)).sum(-1)
            zsum = kz[rows] * x.unflatten(-1, (-1, 64)).sum(-1)
            m = ((ks[rows] * acc).abs() + zsum.abs()).sum(-1)
            e = 8 * 2.0 ** -24 * float(m.max()) * scale + 2.0 ** -22
            want[s, h] = o
            bound[s, h] = (ou.U[dtype] * o.norm() + 2.0 ** -11 * (p @ centred) +
                           2 * e * (p @ (vt - o).norm(dim=-1)) + L * 2.0 ** -23 * (p @ span))
    return want, bound


def share(got, want, bound):
    """The largest part of its bound that a row's error takes."""
    assert torch.isfinite(got).all()
    return float(((got.double().cpu() - want).norm(dim=-1) / bound).max())


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** -20, 1.0, 8.0, 16.0, 32.0, 64.0])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [4, 8])
def test_queries_of_any_size(group, dtype, size):
    q, k, v = inputs(dtype, size, int(math.log2(size)) + 40)
    want, bound = reference(q, k, v, dtype)
    pool = torch.empty(pa.int4_pool_shape(SEQS * L // B, 1, D, B), dtype=torch.uint8, device="cuda")
    pools = pool, pool.clone()
    ops.pa_reshape_and_cache_int4(k.cuda(), v.cuda(), *pools, torch.arange(SEQS * L).cuda())
    table = torch.arange(SEQS * L // B, dtype=torch.int32).reshape(SEQS, -1).cuda()
    lens = torch.full((SEQS,), L, dtype=torch.int32).cuda()
    for first in range(0, HQ, group):      # one kv head: a call takes `group` of the query heads
        part = q[:, first:first + group].contiguous().cuda()
        for split in (0, 64):
            out = torch.full_like(part, math.nan)
            ops.pa_decode_int4(out, part, *pools, table, lens, D ** -0.5, partition_size=split)
            assert share(out, want[:, first:first + group], bound[:, first:first + group]) <= 1.0
    assert pa.pa_get_device_error() == 0


def test_the_bound_tells_a_rounded_query():
    """The same sums with q_d - q_{d+8} / 16 rounded to fp16 and multiplied by
    the codes of d (0..15) leave the bound: it would show scores that depend
    on the query's size."""
    worst = {}
    for dtype in (torch.float16, torch.bfloat16):
        q, k, v = inputs(dtype, 32.0, 45)
        want, bound = reference(q, k, v, dtype)
        kn, ks, kz = parts(k)
        vv = ou.values4(v)[:, 0]
        for rounded in (True, False):
            got = torch.zeros(SEQS, HQ, D, dtype=torch.float64)
            for s in range(SEQS):
                rows = slice(s * L, (s + 1) * L)
                code = kn[rows].unflatten(-1, (-1, 2, 8))
                for h in range(HQ):
                    x = q[s, h].double().unflatten(-1, (-1, 2, 8)) * 2.0 ** 8      # (to [2^13, 2^14])
                    low, high = x[:, 0] - x[:, 1] / 16, x[:, 1] / 16
                    if rounded:
                        low, high = low.half().double(), high.half().double()
                    acc = (code[:, :, 0] * low + (code[:, :, 0] + 16 * code[:, :, 1]) * high).sum(-1)
                    z = (ks[rows] * acc.unflatten(-1, (-1, 4)).sum(-1) * 2.0 ** -8 +
                         kz[rows] * q[s, h].double().unflatten(-1, (-1, 64)).sum(-1)).sum(-1)
                    got[s, h] = torch.softmax(z * D ** -0.5, 0) @ vv[rows]
            worst[dtype, rounded] = share(got.to(dtype), want, bound)
    assert worst[torch.float16, True] > 1.0 and worst[torch.bfloat16, True] > 1.0
    assert worst[torch.float16, False] <= 1.0 and worst[torch.bfloat16, False] <= 1.0
