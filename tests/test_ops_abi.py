"""include/pa/ops.h on the CPU: the binding's argument types, the exports, the
refusals before any launch, the plans and the frequencies."""

import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import paged_kv_cache_449_b200 as pa
from paged_kv_cache_449_b200 import build as pabuild
from paged_kv_cache_449_b200 import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.load()


def signatures():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pa", "ops.h")).read(), flags=re.S)
    return [(m.group(2), [" ".join(x.split()) for x in m.group(3).split(",")])
            for m in re.finditer(r"^\s*(pa_status)\s+(pa_\w+)\s*\(([^)]*)\)\s*;", text, flags=re.M)]


def test_binding_argument_types_match_the_header(lib):
    scalar = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "float": ctypes.c_float, "size_t": ctypes.c_size_t,
              "pa_dtype": ctypes.c_int}
    sigs = signatures()
    assert {n for n, _ in sigs} == {n for n in ops.__all__ if n.startswith("pa_")}
    out = subprocess.run(["nm", "-D", "--defined-only", pa.library_path()], capture_output=True, text=True).stdout
    for name, params in sigs:
        assert re.search(rf"\bT\s+{name}$", out, flags=re.M), name
        fn = getattr(lib, name)
        assert len(fn.argtypes) == len(params) and fn.restype is ctypes.c_int, name
        for decl, ct in zip(params, fn.argtypes):
            if "*" in decl:
                assert ct is ctypes.c_void_p or issubclass(ct, ctypes._Pointer), (name, decl)
            else:
                assert ct is scalar[decl.rsplit(" ", 1)[0].replace("const ", "")], (name, decl)


def call(lib, name, **kw):
    """The entry point with good arguments, some of them replaced (no launch is
    reached: a call that would pass its checks has no tokens or sequences)."""
    params = dict(signatures())[name]
    good = dict(eps=1e-6, rope_scale=1.0, interleaved=0, rotary_dim=64, q_stride=256, k_stride=128, v_stride=128,
                num_tokens=4, num_q_heads=4, num_kv_heads=2, head_dim=64, block_size=16, num_blocks=64, dtype=2,
                stream=None, scale=0.125, num_seqs=4, max_blocks_per_seq=7, max_context_len=100, window=10,
                num_sinks=2, partition_size=0, workspace_bytes=1 << 20, num_counters=64, max_query_len=10,
                ref_counts=None, seq_order=None)
    good.update(kw)
    args = []
    for p in params:
        n = re.split(r"[\s*]+", p)[-1]
        args.append(good.pop(n) if n in good else 16)
    assert not (set(kw) & set(good)), kw
    return getattr(lib, name)(*args)


DECODES = ["pa_decode_window", "pa_decode_window_fp8", "pa_decode_int4"]
ROPES = ["pa_rope_and_cache", "pa_rope_and_cache_fp8", "pa_rope_and_cache_int4"]
ROWS = ["pa_reshape_and_cache_int4", "pa_gather_cache_int4"]


@pytest.mark.parametrize("name", DECODES + ["pa_prefill_window"])
def test_attention_refusals(lib, name):
    assert call(lib, name, num_seqs=0) == 0
    for bad in (dict(head_dim=96), dict(block_size=12), dict(num_q_heads=6, num_kv_heads=2), dict(dtype=9),
                dict(num_seqs=70000)):
        assert call(lib, name, **bad) == 2, bad
    low = 0 if name == "pa_decode_int4" else 1
    for bad in (dict(num_seqs=-1), dict(num_q_heads=5), dict(scale=math.nan), dict(scale=math.inf), dict(q=0),
                dict(k_cache=24), dict(v_cache=None), dict(block_tables=18), dict(context_lens=None),
                dict(window=low - 1), dict(num_sinks=-1), dict(out=8), dict(num_blocks=0)):
        assert call(lib, name, **bad) == 1, bad
    if name != "pa_decode_window":
        assert call(lib, name, dtype=0) == 2          # fp32


@pytest.mark.parametrize("name", DECODES)
def test_partition_refusals(lib, name):
    for bad in (dict(partition_size=-16), dict(partition_size=24), dict(seq_order=18)):
        assert call(lib, name, **bad) == 1, bad
    if name != "pa_decode_int4":
        assert call(lib, name, partition_size=16, block_size=32, window=64) == 1
        for bad in (dict(ref_counts=18), dict(key=None), dict(value=None), dict(key=24, value=24)):
            assert call(lib, name, **bad) == 1, bad
    # 4 sequences x 4 heads, 100 visible tokens in partitions of 32
    split = dict(partition_size=32, window=100, num_sinks=0)
    need = 4 * 4 * 4 * 66 * 4
    for bad in (dict(workspace=None), dict(workspace=24), dict(workspace_bytes=need - 1), dict(counters=None),
                dict(counters=18), dict(num_counters=7)):
        assert call(lib, name, **split, **bad) == 3, bad


def test_scales_are_needed(lib):
    for bad in (dict(k_scale=None), dict(v_scale=18)):
        assert call(lib, "pa_decode_window_fp8", **bad) == 1
        assert call(lib, "pa_rope_and_cache_fp8", **bad) == 1


def test_prefill_refusals(lib):
    assert call(lib, "pa_prefill_window", max_query_len=0) == 0
    for bad in (dict(max_query_len=-1), dict(query_start=None), dict(query_start=18), dict(scale=0.0), dict(scale=-1.0)):
        assert call(lib, "pa_prefill_window", **bad) == 1, bad


@pytest.mark.parametrize("name", ROPES + ROWS)
def test_row_refusals(lib, name):
    assert call(lib, name, num_tokens=0) == 0
    for bad in (dict(head_dim=96), dict(block_size=12), dict(dtype=9)):
        assert call(lib, name, **bad) == 2, bad
    for bad in (dict(num_tokens=-1), dict(num_kv_heads=0), dict(num_blocks=0), dict(key=0), dict(value=24),
                dict(k_cache=24), dict(v_cache=None), dict(slot_mapping=12)):
        assert call(lib, name, **bad) == 1, bad


@pytest.mark.parametrize("name", ROPES)
def test_rope_refusals(lib, name):
    assert call(lib, name, rotary_dim=24) == 2
    for bad in (dict(rotary_dim=-16), dict(rotary_dim=80), dict(eps=-1.0), dict(eps=math.nan), dict(rope_scale=math.inf),
                dict(q_stride=248), dict(q_stride=260), dict(k_stride=127), dict(v_stride=64), dict(positions=12),
                dict(inv_freq=None), dict(inv_freq=18), dict(q_weight=24), dict(k_weight=8), dict(num_q_heads=0),
                dict(q_out=None)):
        assert call(lib, name, **bad) == 1, bad


def test_plans(lib):
    # 3 sequences x 8 heads; 1000 tokens in partitions of 128
    assert ops.pa_decode_int4_plan(3, 8, 2, 64, 1000, partition_size=128) == (128, 3 * 8 * 8 * 66 * 4)
    assert ops.pa_decode_int4_plan(3, 8, 2, 64, 1000, partition_size=0) == (0, 0)
    assert ops.pa_decode_int4_plan(3, 8, 2, 64, 0, partition_size=128) == (128, 0)
    # a window of 100 touches 5 steps of 32 tokens at most, 20 first tokens one more; 8 and 2 blocks of 16
    assert ops.pa_decode_int4_plan(3, 8, 2, 64, 1000, 100, 20, 32) == (32, 3 * 8 * 6 * 66 * 4)
    assert ops.pa_decode_window_plan(3, 8, 2, 64, 16, 1000, 100, 20, 32) == (32, 3 * 8 * 5 * 66 * 4)
    assert ops.pa_decode_window_plan(3, 8, 2, 64, 16, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1 << 20)[1] > 0
    for bad in ((-1, 8, 2, 64, 16, 100, 10), (3, 8, 2, 64, 16, 100, 0), (3, 8, 2, 64, 16, 100, 10, -1),
                (3, 8, 2, 64, 16, 100, 10, 0, 24), (3, 8, 2, 64, 32, 100, 10, 0, 16)):
        with pytest.raises(pa.PagedAttentionError):
            ops.pa_decode_window_plan(*bad)
    part, size = ops.pa_decode_int4_plan(1, 8, 2, 64, 100000)
    assert part % 16 == 0 and (size == 0) == (part == 0)


def test_every_tensor_entry_checks_the_device():
    from test_abi import _FakeCudaTensor
    a, b = _FakeCudaTensor.make(0), _FakeCudaTensor.make(1)
    tensors = {"pa_rope_and_cache": 9, "pa_rope_and_cache_fp8": 11, "pa_rope_and_cache_int4": 9,
               "pa_reshape_and_cache_int4": 5, "pa_gather_cache_int4": 5, "pa_decode_int4": 6, "pa_decode_window": 8,
               "pa_decode_window_fp8": 10, "pa_prefill_window": 7}
    assert set(tensors) == {n for n in ops.__all__ if n.startswith("pa_") and not n.endswith("_plan")}
    for name, n in tensors.items():
        with pytest.raises(ValueError, match="one CUDA device"):
            getattr(ops, name)(*([a] * (n - 1) + [b]), *([0] * 3))


def test_binding_refusals():
    pool = torch.zeros(2, 1, 8 * 64 * 9 // 16, dtype=torch.uint8)
    assert ops._int4_block_size(pool, pool, 64) == 8
    for k, v in ((pool.float(), pool), (pool, pool[:1]), (pool[0], pool[0]), (pool[..., :-1], pool[..., :-1])):
        with pytest.raises(ValueError):
            ops._int4_block_size(k, v, 64)
    q = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops._token_rows(q, "q")
    with pytest.raises(ValueError):
        ops._batch(q, q.half(), torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        ops._batch(q, q, torch.zeros(3, 4, dtype=torch.int64), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        ops._batch(q, q, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        pa._bytes_as_pool(torch.zeros(4, 4, dtype=torch.uint8))


def test_frequencies():
    R, base = 64, 10000.0
    plain, m = pa.rope_frequencies(R, base)
    want = torch.tensor([base ** (-2 * j / R) for j in range(R // 2)], dtype=torch.float64).float()
    assert torch.equal(plain, want) and m == 1.0
    half, _ = pa.rope_frequencies(R, base, "linear", 2.0)
    assert torch.equal(half, plain / 2)
    ntk, _ = pa.rope_frequencies(R, base, "ntk", 4.0)
    assert ntk[0] == 1.0 and abs(float(ntk[-1] * 4 / plain[-1]) - 1) < 1e-6
    # a context of 8192: frequencies that turn more than four times are kept, those under once are divided by 8
    l3, m = pa.rope_frequencies(R, 500000.0, "llama3", 8.0, 8192)
    p3, _ = pa.rope_frequencies(R, 500000.0)
    turns = 8192 * p3.double() / (2 * math.pi)
    assert torch.equal(l3[turns > 4], p3[turns > 4]) and torch.equal(l3[turns < 1], p3[turns < 1] / 8) and m == 1.0
    between = (turns > 1) & (turns < 4)
    smooth = (turns[between] - 1) / 3
    assert torch.allclose(l3[between].double(), p3[between].double() * (smooth + (1 - smooth) / 8), rtol=1e-6)
    y, m = pa.rope_frequencies(R, base, "yarn", 4.0, 4096)
    assert y[0] == plain[0] and abs(float(y[-1] * 4 / plain[-1]) - 1) < 1e-6 and m == 0.1 * math.log(4.0) + 1
    assert ((y <= plain) & (y >= plain / 4 * (1 - 1e-6))).all()
    for bad in (dict(scaling="other"), dict(scaling="yarn"), dict(factor=0.0), dict(scaling="llama3")):
        with pytest.raises(ValueError):
            pa.rope_frequencies(R, base, **bad)
    with pytest.raises(ValueError):
        pa.rope_frequencies(15)


class _Cuda(torch.Tensor):
    """A CPU tensor that passes the binding's check for CUDA tensors."""

    @staticmethod
    def of(*shape, dtype=torch.bfloat16):
        return torch.Tensor._make_subclass(_Cuda, torch.zeros(shape, dtype=dtype))

    @property
    def is_cuda(self):
        return True


def window_args(key, value, fp8=False):
    """ops._decode_window_args of a batch of 3 sequences, 4 query and 2 kv heads of 64 dims."""
    q, i32 = _Cuda.of(3, 4, 64), dict(dtype=torch.int32)
    pool = _Cuda.of(*pa.fp8_pool_shape(5, 2, 64, 16), dtype=torch.uint8) if fp8 else \
        _Cuda.of(*pa.pool_shape(5, 2, 64, 16, torch.bfloat16))
    scales = [_Cuda.of(2, dtype=torch.float32)] * 2 if fp8 else [None, None]
    return ops._decode_window_args(q, q, key, value, pool, pool, *scales, _Cuda.of(3, 7, **i32), _Cuda.of(3, **i32),
                                   0.125, 10, 0, None, 0, None, None, None, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_windowed_append_takes_a_row_per_sequence(lib, fp8):
    """Fewer rows than sequences would be read out of range."""
    good = _Cuda.of(3, 2, 64)
    assert window_args(good, good, fp8)[0][2:4] == [good.data_ptr()] * 2
    assert window_args(None, None, fp8)[0][2:4] == [None, None]
    for bad in (_Cuda.of(2, 2, 64), _Cuda.of(4, 2, 64), _Cuda.of(3, 1, 64), _Cuda.of(3, 2, 32), _Cuda.of(2, 3, 64),
                _Cuda.of(3, 2, 64, dtype=torch.float32), _Cuda.of(3, 2, 128)[..., ::2]):
        for key, value in ((bad, good), (good, bad), (bad, bad)):
            with pytest.raises(ValueError):
                window_args(key, value, fp8)
    for key, value in ((good, None), (None, good)):
        with pytest.raises(ValueError):
            window_args(key, value, fp8)


def test_append_rows_of_the_plain_decodes(lib):
    """pa_decode_append, its 8-bit form and the shared-prefix form: at least a row
    per sequence, of q's type (contiguous rows of any shape, as ever)."""
    q, i32 = _Cuda.of(3, 4, 64), dict(dtype=torch.int32)
    tables, lens, scales = _Cuda.of(3, 7, **i32), _Cuda.of(3, **i32), [_Cuda.of(2, dtype=torch.float32)] * 2
    pool = _Cuda.of(*pa.pool_shape(5, 2, 64, 16, torch.bfloat16))
    pool8 = _Cuda.of(*pa.fp8_pool_shape(5, 2, 64, 16), dtype=torch.uint8)
    work, counts = _Cuda.of(1 << 20, dtype=torch.uint8), _Cuda.of(6, **i32)
    forms = [lambda k, v: pa._append_args(q, q, k, v, pool, pool, tables, lens, 0.125, None, None, None),
             lambda k, v: pa._append_fp8_args(q, q, k, v, pool8, pool8, *scales, tables, lens, 0.125, None, None, None),
             lambda k, v: pa._shared_prefix_args(q, q, k, v, pool, pool, tables, lens, 0.125, 1, None, work, None, counts)[0]]
    good = _Cuda.of(3, 2, 64)
    for form in forms:
        for ok in (good, _Cuda.of(3, 128), _Cuda.of(5, 2, 64)):
            assert form(ok, good)[2:4] == [ok.data_ptr(), good.data_ptr()]
        for bad in (_Cuda.of(2, 2, 64), _Cuda.of(3, 1, 64), _Cuda.of(3, 2, 64, dtype=torch.float32)):
            for key, value in ((bad, good), (good, bad)):
                with pytest.raises(ValueError):
                    form(key, value)
    assert forms[2](None, None)[2:4] == [None, None]


def test_8_bit_scales_are_one_per_kv_head(lib):
    """A scale is read for every kv head of the pools."""
    q, i32, f32 = _Cuda.of(3, 4, 64), dict(dtype=torch.int32), dict(dtype=torch.float32)
    rows, slots, freq = _Cuda.of(3, 2, 64), _Cuda.of(3, dtype=torch.int64), _Cuda.of(32, **f32)
    pool = _Cuda.of(*pa.fp8_pool_shape(5, 2, 64, 16), dtype=torch.uint8)
    tables, lens = _Cuda.of(3, 7, **i32), _Cuda.of(3, **i32)
    forms = [lambda k, v: ops._decode_window_args(q, q, None, None, pool, pool, k, v, tables, lens, 0.125, 10, 0, None, 0,
                                                  None, None, None, None),
             lambda k, v: ops._rope_args("fp8", q, q, rows, rows, pool, pool, k, v, slots, slots, freq, False, 1.0, None,
                                         None, 1e-6),
             lambda k, v: pa._fp8_args(q, q, pool, pool, k, v, tables, lens, 0.125, None),
             lambda k, v: pa.pa_reshape_and_cache_fp8.__wrapped__(rows[:0], rows[:0], pool, pool, slots[:0], k, v, stream=0)]
    good = _Cuda.of(2, **f32)
    for form in forms:
        form(good, good)
        for bad in (_Cuda.of(1, **f32), _Cuda.of(2, dtype=torch.float64)):
            for k, v in ((bad, good), (good, bad)):
                with pytest.raises(ValueError, match="scale"):
                    form(k, v)
    # ... and the windowed form's pools are both of bytes
    with pytest.raises(ValueError):
        ops._decode_window_args(q, q, None, None, pool, pool.half(), good, good, tables, lens, 0.125, 10, 0, None, 0, None,
                                None, None, None)


def test_byte_pools_are_copied_between_pools_of_one_shape(lib):
    """The sizes of a copy are read off one pool of a pair: the others have them too."""
    def copy(*pools):
        pairs = _Cuda.of(0, 2, dtype=torch.int64)
        return pa.pa_copy_blocks.__wrapped__(*pools, pairs, stream=0)

    u8 = dict(dtype=torch.uint8)
    four, fewer = _Cuda.of(*ops.int4_pool_shape(6, 2, 64, 16), **u8), _Cuda.of(*ops.int4_pool_shape(4, 2, 64, 16), **u8)
    eight, turned = _Cuda.of(*pa.fp8_pool_shape(6, 2, 64, 16), **u8), _Cuda.of(*pa.fp8_pool_shape(6, 2, 128, 8), **u8)
    copy(four, four, fewer, fewer)      # swap-out: pools of other lengths
    copy(eight, eight, eight, eight)
    for pools in ((four, fewer, four, four), (four, four, four, fewer), (fewer, fewer, four, fewer),
                  (eight, eight, turned, turned), (eight, turned, eight, eight),
                  (four, four, _Cuda.of(*ops.int4_pool_shape(6, 1, 64, 32), **u8), _Cuda.of(*ops.int4_pool_shape(6, 1, 64, 32), **u8))):
        with pytest.raises(ValueError, match="shape"):
            copy(*pools)
