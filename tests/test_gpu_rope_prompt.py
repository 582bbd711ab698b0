"""The rotary step over a prompt's tokens: small thread blocks and several batches
of rows a token (from 8 tokens an SM on), many heads in a few tokens' large
blocks, and a norm of the queries or of the keys alone.  A token's rows do not
depend on the tokens beside it, so a large call has to equal the same tokens in
small calls bit for bit; sampled tokens are held against the formulas in 64 bits
(test_gpu_rope's tolerance)."""

import pytest
import torch

import opsutil as ou
import paged_kv_cache_449_b200 as pa
from paged_kv_cache_449_b200 import ops
from test_gpu_rope import close, inputs

pytestmark = pytest.mark.gpu

T, SMALL = 1231, 200      # (148 SMs: 1184 tokens and more are many)


def pools_of(kind, N, H, D, B, dtype):
    shape = {"native": pa.pool_shape(N, H, D, B, dtype), "fp8": pa.fp8_pool_shape(N, H, D, B),
             "int4": pa.int4_pool_shape(N, H, D, B)}[kind]
    return [torch.full(shape, 9, dtype=dtype if kind == "native" else torch.uint8, device="cuda") for _ in range(2)]


ENTRY = {"native": ops.pa_rope_and_cache, "fp8": ops.pa_rope_and_cache_fp8, "int4": ops.pa_rope_and_cache_int4}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", ["none", "both", "q", "k"])
@pytest.mark.parametrize("dtype,D,B,Hq,H", [(torch.bfloat16, 128, 16, 32, 13), (torch.float16, 64, 8, 40, 25),
                                            (torch.float32, 128, 32, 17, 8), (torch.float32, 64, 16, 32, 16)])
@pytest.mark.parametrize("kind", ["native", "fp8", "int4"])
def test_a_prompts_tokens(kind, dtype, D, B, Hq, H, norm, interleaved):
    assert T >= 8 * torch.cuda.get_device_properties(0).multi_processor_count
    (q, k, v), (qd, kd, vd), N, slots, pos = inputs(T, Hq, H, D, B, dtype, D + Hq, fused=True, far=1000000)
    slots[::97] = -1
    g = ou.gen(7)
    qw, kw = ((1 + 0.2 * ou.normal((D,), torch.float32, g)).to(dtype) for _ in range(2))
    qw, kw = qw if norm in ("both", "q") else None, kw if norm in ("both", "k") else None
    freq = pa.rope_frequencies(D // 2, 500000.0)[0]
    scales = [(0.01 + 0.002 * torch.arange(H)).cuda()] * 2 if kind == "fp8" else []
    opt = dict(interleaved=interleaved, q_weight=None if qw is None else qw.cuda(),
               k_weight=None if kw is None else kw.cuda(), eps=1e-5)
    pd, sd, fd = pos.cuda(), slots.cuda(), freq.cuda()
    large, small = pools_of(kind, N, H, D, B, dtype), pools_of(kind, N, H, D, B, dtype)
    outs = [torch.zeros(T, Hq, D, dtype=dtype, device="cuda") for _ in range(2)]
    ENTRY[kind](outs[0], qd, kd, vd, *large, *scales, pd, sd, fd, **opt)
    for a in range(0, T, SMALL):
        part = slice(a, min(a + SMALL, T))
        ENTRY[kind](outs[1][part], qd[part], kd[part], vd[part], *small, *scales, pd[part], sd[part], fd, **opt)
    again = pools_of(kind, N, H, D, B, dtype)
    mine = qd.contiguous()
    ENTRY[kind](mine, mine, kd, vd, *again, *scales, pd, sd, fd, **opt)      # q in its own place
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], mine)
    for x, y, z in zip(large, small, again):
        assert torch.equal(x, y) and torch.equal(x, z)
    at = torch.tensor([0, 1, 97, 500, 1183, 1184, T - 1])      # (0 and 97 have no slot)
    close(outs[0].cpu()[at], ou.rope(q[at], pos[at], freq, interleaved, 1.0, qw, 1e-5), q[at], qw, dtype)
    if kind == "native":
        want = ou.rope(k[at], pos[at], freq, interleaved, 1.0, kw, 1e-5)
        kc, vc = (x.cpu() for x in large)
        for i, t in enumerate(at.tolist()):
            if int(slots[t]) >= 0:
                close(ou.pool_row(kc, int(slots[t]), B), want[i], k[t], kw, dtype)
                assert torch.equal(ou.pool_row(vc, int(slots[t]), B), v[t])
    elif kind == "int4":      # the plain write of the rows that the native pool gets
        native, plain = pools_of("native", N, H, D, B, dtype), pools_of(kind, N, H, D, B, dtype)
        ops.pa_rope_and_cache(outs[1], qd, kd, vd, *native, pd, sd, fd, **opt)
        s = sd.clamp(min=0)
        rows = native[0][s // B, :, :, s % B, :].flatten(2).contiguous()
        ops.pa_reshape_and_cache_int4(rows, vd.contiguous(), *plain, sd)
        assert torch.equal(plain[0], large[0]) and torch.equal(plain[1], large[1])


@pytest.mark.parametrize("dtype,D,Hq,H", [(torch.bfloat16, 128, 96, 56), (torch.float32, 128, 56, 28), (torch.float16, 64, 112, 100)])
@pytest.mark.parametrize("kind", ["native", "int4"])
def test_many_heads_of_a_few_tokens(kind, dtype, D, Hq, H):
    """More rows than a large block takes at once: equal to the heads in two halves."""
    n, B = 5, 16
    (q, k, v), (qd, kd, vd), N, slots, pos = inputs(n, Hq, H, D, B, dtype, Hq, far=5000)
    freq = pa.rope_frequencies(D, 10000.0)[0].cuda()
    w = (1 + 0.1 * ou.normal((D,), torch.float32, ou.gen(3))).to(dtype).cuda()
    opt = dict(q_weight=w, k_weight=w)
    whole = pools_of(kind, N, H, D, B, dtype)
    out = torch.zeros_like(qd)
    ENTRY[kind](out, qd, kd, vd, *whole, pos.cuda(), slots.cuda(), freq, **opt)
    for a in range(2):
        hq, h = slice(a * Hq // 2, (a + 1) * Hq // 2), slice(a * H // 2, (a + 1) * H // 2)
        half, got = pools_of(kind, N, H // 2, D, B, dtype), torch.zeros_like(qd[:, hq]).contiguous()
        ENTRY[kind](got, qd[:, hq], kd[:, h], vd[:, h], *half, pos.cuda(), slots.cuda(), freq, **opt)
        assert torch.equal(got, out[:, hq])
        for x, y in zip(whole, half):
            assert torch.equal(x[:, h], y)
    assert pa.pa_get_device_error() == 0
