"""Binding of the operators of include/pa/ops.h: rotary positions and head norms
with the cache write, 4-bit pools, and attention with a sliding window.

Argument marshalling only, as in the package itself: calls run on the current
torch CUDA stream of their tensors' device unless `stream` is given.  The
prepare_* functions check and marshal a call's arguments once for a loop over
fixed buffers (see Prepared).
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import (_DTYPE, Counters, Prepared, _check, _counts_ptr, _decode_args, _dev_ptr, _fp8_args, _on_tensor_device,
               _order_ptr, _pool_dims, _scale_ptr, _stream, _stream_object, _tensor_device, load)

__all__ = ["pa_rope_and_cache", "pa_rope_and_cache_fp8", "pa_rope_and_cache_int4", "prepare_rope_and_cache",
           "rope_frequencies", "int4_pool_shape", "pa_reshape_and_cache_int4", "prepare_reshape_and_cache_int4",
           "pa_gather_cache_int4", "prepare_gather_cache_int4", "pa_decode_int4", "pa_decode_int4_plan",
           "prepare_decode_int4", "pa_decode_window", "pa_decode_window_fp8", "pa_decode_window_plan",
           "prepare_decode_window", "pa_prefill_window", "prepare_prefill_window"]


# ---- rotary positions, head norms and the cache write in one pass

def rope_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_max_position=None, device=None,
                     low_freq_factor=1.0, high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0):
    """(inv_freq, rope_scale) of pa_rope_and_cache: base^(-2j / rotary_dim),
    formed in fp64 and rounded once to fp32, with a scaling for contexts
    `factor` times longer than original_max_position:
      None       as they are
      "linear"   every frequency / factor (position interpolation)
      "ntk"      base * factor^(R / (R - 2)): the lowest frequency / factor, the highest kept
      "llama3"   frequencies of wavelengths above original_max_position / low_freq_factor / factor, those
                 below original_max_position / high_freq_factor kept, between them blended
      "yarn"     frequencies that turn fewer than beta_slow times in original_max_position / factor, those
                 that turn more than beta_fast times kept, a ramp over j between; rope_scale = 0.1 ln(factor) + 1"""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be positive and even")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling in ("llama3", "yarn") and not original_max_position:
        raise ValueError(f"scaling {scaling!r} needs original_max_position")
    if scaling == "ntk":
        if rotary_dim <= 2:
            raise ValueError("scaling 'ntk' needs rotary_dim > 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    j = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    freq = float(base) ** (-j / rotary_dim)
    rope_scale = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "llama3":
        turns = original_max_position * freq / (2 * math.pi)
        keep = ((turns - low_freq_factor) / (high_freq_factor - low_freq_factor)).clamp(0.0, 1.0)
        freq = freq * (keep + (1 - keep) / factor)
    elif scaling == "yarn":
        def index(turns):   # the j at which a frequency turns that often within the original context
            return rotary_dim * math.log(original_max_position / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(index(beta_fast)), 0), min(math.ceil(index(beta_slow)), rotary_dim - 1)
        ramp = ((j / 2 - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        freq = freq * ((1 - ramp) + ramp / factor)
        rope_scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(torch.float32).to(device), rope_scale


def _token_rows(t, name, heads=None, dim=None):
    """Pointer and token stride (elements) of [T, heads, head_dim] rows, a
    token's row contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or (dim is not None and t.shape[2] != dim):
        raise ValueError(f"{name} must be [T, heads, head_dim] of the pools' and q's head dims")
    T, h, d = t.shape
    if t.numel() and (t.stride(2) != 1 or (h > 1 and t.stride(1) != d)):
        raise ValueError(f"{name}: a token's row must be contiguous")
    return t.data_ptr(), (t.stride(0) if T > 1 else h * d)


def _per_token(t, T, name):
    if t.dtype != torch.int64 or t.numel() != T:
        raise ValueError(f"{name} must be int64 [T]")
    return _dev_ptr(t, name)


def _int4_block_size(k_cache, v_cache, head_dim):
    """Block size of 4-bit pools [num_blocks, Hkv, block_size * head_dim * 9 / 16]."""
    if k_cache.dtype != torch.uint8 or k_cache.dim() != 3 or k_cache.shape != v_cache.shape or \
            v_cache.dtype != torch.uint8:
        raise ValueError("4-bit pools are uint8 tensors [num_blocks, Hkv, block_size * head_dim * 9 // 16]")
    b, rest = divmod(int(k_cache.shape[2]) * 16, int(head_dim) * 9)
    if rest:
        raise ValueError("a 4-bit pool's tile holds block_size * head_dim * 9 // 16 bytes")
    return b


def _rope_args(pool, q_out, q, key, value, k_cache, v_cache, k_scale, v_scale, positions, slot_mapping, inv_freq,
               interleaved, rope_scale, q_weight, k_weight, eps):
    T, Hq, D = q.shape
    if pool == "int4":
        n, hkv, b = k_cache.shape[0], k_cache.shape[1], _int4_block_size(k_cache, v_cache, D)
    else:
        n, hkv, d, b = _pool_dims(k_cache)
        if d != D or k_cache.shape != v_cache.shape:
            raise ValueError("the pools' shapes differ, or their head dim from q's")
        want = torch.uint8 if pool == "fp8" else q.dtype
        if k_cache.dtype != want or v_cache.dtype != want:
            raise ValueError(f"the pools must be {want}")
    if key.dtype != q.dtype or value.dtype != q.dtype or q_out.dtype != q.dtype or q_out.shape != q.shape:
        raise ValueError("q, key, value and q_out share one dtype, and q_out q's shape")
    if key.shape[0] != T or value.shape[0] != T:
        raise ValueError("q, key and value hold the same tokens")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and (w.dtype != q.dtype or w.numel() != D):
            raise ValueError(f"{name} must be [head_dim] of q's dtype")
    if inv_freq is not None and inv_freq.dtype != torch.float32:
        raise ValueError("inv_freq must be float32 [rotary_dim // 2]")
    qp, qs = _token_rows(q, "q")
    kp, ks = _token_rows(key, "key", hkv, D)
    vp, vs = _token_rows(value, "value", hkv, D)
    scales = [_scale_ptr(k_scale, "k_scale", hkv), _scale_ptr(v_scale, "v_scale", hkv)] if pool == "fp8" else []
    return [_dev_ptr(q_out, "q_out"), qp, kp, vp, _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"),
            *scales, _per_token(positions, T, "positions"), _per_token(slot_mapping, T, "slot_mapping"),
            None if inv_freq is None else _dev_ptr(inv_freq, "inv_freq"),
            None if q_weight is None else _dev_ptr(q_weight, "q_weight"),
            None if k_weight is None else _dev_ptr(k_weight, "k_weight"), float(eps), float(rope_scale),
            int(bool(interleaved)), 0 if inv_freq is None else 2 * inv_freq.numel(), qs, ks, vs, T, Hq, hkv, D, b, n,
            _DTYPE[q.dtype]]


@_on_tensor_device
def pa_rope_and_cache(q_out, q, key, value, k_cache, v_cache, positions, slot_mapping, inv_freq, interleaved=False,
                      rope_scale=1.0, q_weight=None, k_weight=None, eps=1e-6, stream=None):
    """Rotary positions of q [T, Hq, D] and key [T, Hkv, D] (positions int64
    [T], inv_freq fp32 [rotary_dim // 2] or None; see rope_frequencies), after
    an RMS norm of each head where a weight [D] is given; q goes to q_out, key
    and value into the pools at slot_mapping.  q, key and value may be slices
    of one fused projection; q_out may be q."""
    args = _rope_args("native", q_out, q, key, value, k_cache, v_cache, None, None, positions, slot_mapping, inv_freq,
                      interleaved, rope_scale, q_weight, k_weight, eps)
    _check(load().pa_rope_and_cache(*args, _stream(stream)), "pa_rope_and_cache")


@_on_tensor_device
def pa_rope_and_cache_fp8(q_out, q, key, value, k_cache, v_cache, k_scale, v_scale, positions, slot_mapping, inv_freq,
                          interleaved=False, rope_scale=1.0, q_weight=None, k_weight=None, eps=1e-6, stream=None):
    """pa_rope_and_cache into 8-bit pools."""
    args = _rope_args("fp8", q_out, q, key, value, k_cache, v_cache, k_scale, v_scale, positions, slot_mapping,
                      inv_freq, interleaved, rope_scale, q_weight, k_weight, eps)
    _check(load().pa_rope_and_cache_fp8(*args, _stream(stream)), "pa_rope_and_cache_fp8")


@_on_tensor_device
def pa_rope_and_cache_int4(q_out, q, key, value, k_cache, v_cache, positions, slot_mapping, inv_freq,
                           interleaved=False, rope_scale=1.0, q_weight=None, k_weight=None, eps=1e-6, stream=None):
    """pa_rope_and_cache into 4-bit pools."""
    args = _rope_args("int4", q_out, q, key, value, k_cache, v_cache, None, None, positions, slot_mapping, inv_freq,
                      interleaved, rope_scale, q_weight, k_weight, eps)
    _check(load().pa_rope_and_cache_int4(*args, _stream(stream)), "pa_rope_and_cache_int4")


def _settled(args, held, made):
    """A prepared call may run on any stream: counters that were made (zeroed)
    for it on the current one are complete before it exists.  (Buffers of the
    caller's are the caller's to order, and are not waited for; a capturing
    stream has made no counters, see _partials.)"""
    if made and not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(made[0].device).synchronize()
    return args, held, made


def _prepared(name, args, tensors, made=()) -> Prepared:
    dev = _tensor_device(tensors, {})
    if dev is None:
        raise ValueError(f"{name} takes CUDA tensors")
    return Prepared(name, args, dev, tensors, made)


def prepare_rope_and_cache(q_out, q, key, value, k_cache, v_cache, positions, slot_mapping, inv_freq,
                           interleaved=False, rope_scale=1.0, q_weight=None, k_weight=None, eps=1e-6, k_scale=None,
                           v_scale=None) -> Prepared:
    """The arguments of pa_rope_and_cache (of pa_rope_and_cache_fp8 where
    scales are given, of pa_rope_and_cache_int4 for 4-bit pools) checked and
    marshalled once (see Prepared)."""
    pool = "fp8" if k_scale is not None else ("int4" if k_cache.dtype == torch.uint8 else "native")
    args = _rope_args(pool, q_out, q, key, value, k_cache, v_cache, k_scale, v_scale, positions, slot_mapping,
                      inv_freq, interleaved, rope_scale, q_weight, k_weight, eps)
    return _prepared("pa_rope_and_cache" + ("" if pool == "native" else "_" + pool), args,
                     (q_out, q, key, value, k_cache, v_cache, positions, slot_mapping, inv_freq, q_weight, k_weight,
                      k_scale, v_scale))


# ---- 4-bit pools: uint8 tensors [num_blocks, Hkv, block_size * head_dim * 9 // 16] (one tile of codes and group
#      words per (block, head); its byte order is that of pa/ops.h)

def int4_pool_shape(num_blocks, num_kv_heads, head_dim, block_size):
    return (num_blocks, num_kv_heads, block_size * head_dim * 9 // 16)


def _rows_int4_args(key, value, k_cache, v_cache, slot_mapping):
    T, hkv, d = key.shape
    if value.shape != key.shape or value.dtype != key.dtype or hkv != k_cache.shape[1]:
        raise ValueError("key and value are [T, Hkv, D] of one dtype, with the pools' heads")
    b = _int4_block_size(k_cache, v_cache, d)
    return [_dev_ptr(key, "key"), _dev_ptr(value, "value"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"),
            _per_token(slot_mapping, T, "slot_mapping"), T, hkv, d, b, k_cache.shape[0], _DTYPE[key.dtype]]


@_on_tensor_device
def pa_reshape_and_cache_int4(key, value, k_cache, v_cache, slot_mapping, stream=None):
    """Quantise key/value [T, Hkv, D] to four bits (a scale and a zero for each
    64 dims of a token and head) and write them at slot_mapping (int64 [T])."""
    args = _rows_int4_args(key, value, k_cache, v_cache, slot_mapping)
    _check(load().pa_reshape_and_cache_int4(*args, _stream(stream)), "pa_reshape_and_cache_int4")


@_on_tensor_device
def pa_gather_cache_int4(key, value, k_cache, v_cache, slot_mapping, stream=None):
    """The values at slot_mapping into key/value [T, Hkv, D] (rows of negative
    slots are left as they were)."""
    args = _rows_int4_args(key, value, k_cache, v_cache, slot_mapping)
    _check(load().pa_gather_cache_int4(*args, _stream(stream)), "pa_gather_cache_int4")


def prepare_reshape_and_cache_int4(key, value, k_cache, v_cache, slot_mapping) -> Prepared:
    """pa_reshape_and_cache_int4's arguments checked and marshalled once (see Prepared)."""
    return _prepared("pa_reshape_and_cache_int4", _rows_int4_args(key, value, k_cache, v_cache, slot_mapping),
                     (key, value, k_cache, v_cache, slot_mapping))


def prepare_gather_cache_int4(key, value, k_cache, v_cache, slot_mapping) -> Prepared:
    """pa_gather_cache_int4's arguments checked and marshalled once (see Prepared)."""
    return _prepared("pa_gather_cache_int4", _rows_int4_args(key, value, k_cache, v_cache, slot_mapping),
                     (key, value, k_cache, v_cache, slot_mapping))


# ---- decode with a sliding window, and over 4-bit pools

def pa_decode_window_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, window,
                          num_sinks=0, partition_size=None):
    """(partition_size, workspace bytes) of pa_decode_window: the library's
    choice for the current device where partition_size is None."""
    part, size = ctypes.c_int(-1 if partition_size is None else int(partition_size)), ctypes.c_size_t(0)
    _check(load().pa_decode_window_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                        int(max_context_len), int(window), int(num_sinks), ctypes.byref(part),
                                        ctypes.byref(size)), "pa_decode_window_plan")
    return int(part.value), int(size.value)


def pa_decode_int4_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len, window=0, num_sinks=0,
                        partition_size=None):
    """(partition_size, workspace bytes) of pa_decode_int4: the library's
    choice for the current device where partition_size is None."""
    part, size = ctypes.c_int(-1 if partition_size is None else int(partition_size)), ctypes.c_size_t(0)
    _check(load().pa_decode_int4_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, int(max_context_len),
                                      int(window), int(num_sinks), ctypes.byref(part), ctypes.byref(size)),
           "pa_decode_int4_plan")
    return int(part.value), int(size.value)


def _partials(need, workspace, counters, num_counters, device, lasting):
    """[pointer, bytes, pointer, count] of a call's workspace and counters, the
    two tensors, and those of them that were made here because they were not
    given, for this call alone (calls that overlap may not share them).
    `lasting`: they outlive this call.  What a capture makes is zeroed by the
    graph's replays, not now, so a handle's counters are not made while the
    stream is capturing, and a Counters does not grow then (the captured call
    has counters of its own)."""
    if need == 0:
        return [None, 0, None, 0], (), ()
    made = ()
    if isinstance(counters, Counters):
        had = counters.buf
        if (had is None or had.numel() < num_counters or had.device != device) and \
                torch.cuda.is_current_stream_capturing():
            counters = None
    if counters is None and lasting and torch.cuda.is_current_stream_capturing():
        raise ValueError("a handle's counters cannot be made while the stream is capturing: prepare the call before "
                         "the capture, or give zeroed counters")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        made += (workspace,)
    if counters is None:
        counters = torch.zeros(num_counters, dtype=torch.int32, device=device)
        made += (counters,)
    buf = counters
    if isinstance(counters, Counters):
        buf = counters.get(num_counters, device)
        if buf is not had:
            made += (buf,)
    if buf.dtype != torch.int32:
        raise ValueError("counters must be int32")
    return [_dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
            _dev_ptr(buf, "counters"), buf.numel()], (workspace, buf), made


def _batch(out, q, block_tables, context_lens):
    """The checks of a batch's tensors that the C side cannot make."""
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have q's shape and dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or context_lens.numel() != block_tables.shape[0]:
        raise ValueError("block_tables is [num_seqs, max_blocks], context_lens [num_seqs]")


def _decode_int4_args(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, window, num_sinks,
                      partition_size, workspace, counters, seq_order, lasting=False):
    _batch(out, q, block_tables, context_lens)
    S, Hq, D = q.shape
    if block_tables.shape[0] != S:
        raise ValueError("q holds one row per sequence")
    b, hkv = _int4_block_size(k_cache, v_cache, D), int(k_cache.shape[1])
    if max_context_len is None:
        max_context_len = int(block_tables.shape[1]) * b
    cap = min(int(max_context_len), int(block_tables.shape[1]) * b)
    part, need = pa_decode_int4_plan(S, Hq, hkv, D, cap, window, num_sinks, partition_size)
    extra, held, made = _partials(need, workspace, counters, S * hkv, q.device, lasting)
    return [_dev_ptr(out, "out"), _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"),
            _dev_ptr(block_tables, "block_tables"), _dev_ptr(context_lens, "context_lens"), float(scale), b, S, Hq,
            hkv, D, int(block_tables.shape[1]), int(max_context_len), k_cache.shape[0], _DTYPE[q.dtype], int(window),
            int(num_sinks), part, *extra, _order_ptr(seq_order, S)], held, made


@_on_tensor_device
def pa_decode_int4(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len=None, window=0,
                   num_sinks=0, partition_size=None, workspace=None, counters=None, stream=None, seq_order=None):
    """pa_decode over 4-bit pools (q/out fp16 or bf16); window > 0: the newest
    `window` tokens and the first num_sinks only.  partition_size: tokens per
    partition of the context (0: one; None: the library's choice); workspace
    and counters (zeroed int32 [S * Hkv], left at zero) as pa_decode_int4_plan
    says, made here for this call where None."""
    args, held, _ = _decode_int4_args(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len,
                                      window, num_sinks, partition_size, workspace, counters, seq_order)
    _check(load().pa_decode_int4(*args, _side_stream(stream, held)), "pa_decode_int4")


def _side_stream(stream, held):
    """The call's raw stream; a workspace and counters that lie on the current
    stream (made there for this call, as a rule) and are used on another are
    ordered before the call and kept from reuse until that one has passed here."""
    raw = _stream(stream)
    current = torch.cuda.current_stream()
    if raw != current.cuda_stream and held:
        side = stream if isinstance(stream, torch.cuda.Stream) else _stream_object(raw, held[0].device)
        side.wait_stream(current)   # (their allocation, and the counters' zeroing, lie on the current stream)
        for t in held:
            t.record_stream(side)
    return raw


def prepare_decode_int4(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len=None, window=0,
                        num_sinks=0, partition_size=None, workspace=None, counters=None, seq_order=None) -> Prepared:
    """pa_decode_int4's arguments checked and marshalled once (see Prepared);
    the object has its own workspace and counters where none are given, so two
    of its calls must not overlap, and it is not made while the stream is
    capturing (captured calls of it are fine, while it lives)."""
    args, held, made = _settled(*_decode_int4_args(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                                                   max_context_len, window, num_sinks, partition_size, workspace,
                                                   counters, seq_order, lasting=True))
    return _prepared("pa_decode_int4", args, (out, q, k_cache, v_cache, block_tables, context_lens, seq_order, *held),
                     made)


def _decode_window_args(out, q, key, value, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                        window, num_sinks, max_context_len, partition_size, workspace, counters, seq_order,
                        ref_counts, lasting=False):
    _batch(out, q, block_tables, context_lens)
    if (key is None) != (value is None):
        raise ValueError("key and value go together (both None: no append)")
    S, Hq, D = q.shape
    n, hkv, d, b = _pool_dims(k_cache)
    for t, name in ((key, "key"), (value, "value")):
        if t is not None and (t.dtype != q.dtype or t.shape != (S, hkv, D)):
            raise ValueError(f"{name} must be [S, Hkv, D] of q's dtype")
    if d != D or v_cache.shape != k_cache.shape or block_tables.shape[0] != S:
        raise ValueError("the pools' head dim is q's, and q holds one row per sequence")
    if k_scale is None:
        if k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
            raise ValueError("the pools share q's dtype")
        args = _decode_args(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len)
    else:
        if v_cache.dtype != k_cache.dtype:
            raise ValueError("8-bit pools are uint8 tensors")
        args = _fp8_args(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                         max_context_len)
    cap = min(args[-3], int(block_tables.shape[1]) * b)
    part, need = pa_decode_window_plan(S, Hq, hkv, D, b, cap, window, num_sinks, partition_size)
    extra, held, made = _partials(need, workspace, counters, S * hkv, q.device, lasting)
    return [args[0], args[1], None if key is None else _dev_ptr(key, "key"),
            None if value is None else _dev_ptr(value, "value"), *args[2:], int(window), int(num_sinks), part, *extra,
            _counts_ptr(ref_counts, n), _order_ptr(seq_order, S)], held, made


@_on_tensor_device
def pa_decode_window(out, q, key, value, k_cache, v_cache, block_tables, context_lens, scale, window, num_sinks=0,
                     max_context_len=None, partition_size=None, workspace=None, counters=None, stream=None,
                     seq_order=None, ref_counts=None):
    """Decode (key = value = None) or decode with append (key/value [S, Hkv,
    D]) with a sliding window: each newest token attends to the newest `window`
    tokens and the first num_sinks.  Blocks outside may have left the block
    table.  partition_size, workspace, counters as in pa_decode_int4 (see
    pa_decode_window_plan)."""
    args, held, _ = _decode_window_args(out, q, key, value, k_cache, v_cache, None, None, block_tables, context_lens,
                                        scale, window, num_sinks, max_context_len, partition_size, workspace, counters,
                                        seq_order, ref_counts)
    _check(load().pa_decode_window(*args, _side_stream(stream, held)), "pa_decode_window")


@_on_tensor_device
def pa_decode_window_fp8(out, q, key, value, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                         window, num_sinks=0, max_context_len=None, partition_size=None, workspace=None,
                         counters=None, stream=None, seq_order=None, ref_counts=None):
    """pa_decode_window over 8-bit pools."""
    args, held, _ = _decode_window_args(out, q, key, value, k_cache, v_cache, k_scale, v_scale, block_tables,
                                        context_lens, scale, window, num_sinks, max_context_len, partition_size,
                                        workspace, counters, seq_order, ref_counts)
    _check(load().pa_decode_window_fp8(*args, _side_stream(stream, held)), "pa_decode_window_fp8")


def prepare_decode_window(out, q, key, value, k_cache, v_cache, block_tables, context_lens, scale, window,
                          num_sinks=0, max_context_len=None, partition_size=None, workspace=None, counters=None,
                          seq_order=None, ref_counts=None, k_scale=None, v_scale=None) -> Prepared:
    """pa_decode_window's arguments (pa_decode_window_fp8's where scales are
    given) checked and marshalled once (see Prepared); its own workspace and
    counters as in prepare_decode_int4."""
    args, held, made = _settled(*_decode_window_args(out, q, key, value, k_cache, v_cache, k_scale, v_scale,
                                                     block_tables, context_lens, scale, window, num_sinks,
                                                     max_context_len, partition_size, workspace, counters, seq_order,
                                                     ref_counts, lasting=True))
    return _prepared("pa_decode_window" + ("" if k_scale is None else "_fp8"), args,
                     (out, q, key, value, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, seq_order,
                      ref_counts, *held), made)


def _prefill_window_args(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, window, num_sinks,
                         max_context_len, max_query_len):
    _batch(out, q, block_tables, context_lens)
    n, hkv, d, b = _pool_dims(k_cache)
    T, Hq, D = q.shape
    S = int(context_lens.numel())
    if d != D or v_cache.shape != k_cache.shape or k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise ValueError("the pools share q's dtype and head dim")
    if query_start.dtype != torch.int32 or query_start.numel() != S + 1:
        raise ValueError("query_start must be int32 [num_seqs + 1]")
    if max_context_len is None:
        max_context_len = int(block_tables.shape[1]) * b
    if max_query_len is None:
        max_query_len = T
    return [_dev_ptr(out, "out"), _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"),
            _dev_ptr(block_tables, "block_tables"), _dev_ptr(context_lens, "context_lens"),
            _dev_ptr(query_start, "query_start"), float(scale), b, S, Hq, hkv, D, int(block_tables.shape[1]),
            int(max_context_len), int(max_query_len), n, _DTYPE[q.dtype], int(window), int(num_sinks)]


@_on_tensor_device
def pa_prefill_window(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, window, num_sinks=0,
                      max_context_len=None, max_query_len=None, stream=None):
    """pa_prefill with a sliding window: the query at position p attends to the
    keys t <= p with t > p - window or t < num_sinks."""
    args = _prefill_window_args(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, window,
                                num_sinks, max_context_len, max_query_len)
    _check(load().pa_prefill_window(*args, _stream(stream)), "pa_prefill_window")


def prepare_prefill_window(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, window,
                           num_sinks=0, max_context_len=None, max_query_len=None) -> Prepared:
    """pa_prefill_window's arguments checked and marshalled once (see Prepared)."""
    args = _prefill_window_args(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, window,
                                num_sinks, max_context_len, max_query_len)
    return _prepared("pa_prefill_window", args,
                     (out, q, k_cache, v_cache, block_tables, context_lens, query_start))
