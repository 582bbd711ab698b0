"""Plain restatements in 64 bits of the operators of include/pa/ops.h, on the
CPU: nothing here shares code with the library."""

from __future__ import annotations

import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(shape, dtype, g):
    return torch.randn(shape, generator=g, dtype=torch.float32).to(dtype)


# ------------------------------------------------------------------ native pools

def pool_row(pool, slot, B):
    """[Hkv, D] of one slot of a [N, Hkv, D / X, B, X] pool."""
    return pool[slot // B, :, :, slot % B, :].flatten(1)


def pool_rows(pool, ids, L):
    """float64 [L, Hkv, D] of the blocks `ids` of a native pool."""
    rows = pool[ids].permute(0, 3, 1, 2, 4)          # [n, B, Hkv, D / X, X]
    return rows.flatten(3).flatten(0, 1)[:L].double()


# ------------------------------------------------------------------ 4-bit pools

def bf16_towards(x, up):
    """fp32 -> the nearest bf16 not below (up) or not above, as fp32."""
    bits = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    away = (x > 0) if up else (x < 0)
    low = (bits & np.uint32(0xffff)) != 0
    bits = (bits & np.uint32(0xffff0000)) + np.where(away & low, np.uint32(0x10000), np.uint32(0))
    return bits.view(np.float32)


def quantise4(x):
    """fp32 [..., D] -> codes uint8 [..., D], scale and zero fp32 [..., D / 64]."""
    y = x.reshape(*x.shape[:-1], -1, 64).astype(np.float32)
    zero = bf16_towards(y.min(-1) + np.float32(0), False)
    scale = bf16_towards((y.max(-1) - zero) / np.float32(15), True)
    scale = np.where((scale > 0) & (scale < 2.0 ** -126), np.float32(2.0 ** -126), scale)
    with np.errstate(all="ignore"):
        part = (y - zero[..., None]) / scale[..., None]
    part = np.where(scale[..., None] > 0, part, np.float32(0))
    return np.clip(np.rint(part), 0, 15).astype(np.uint8).reshape(x.shape), scale, zero


def values4(x):
    """The values the 4-bit pool holds for rows x (a torch tensor), float64."""
    codes, scale, zero = quantise4(x.float().numpy())
    y = zero.astype(np.float64)[..., None] + scale.astype(np.float64)[..., None] * codes.reshape(*scale.shape, 64)
    return torch.from_numpy(y.reshape(codes.shape))


def code_byte(value, B, D, t, d):
    """Offset in a tile of the byte of dims d, d + 8 of token t (pa/ops.h)."""
    u, chunk, m, e = t % 8, d // 64, d % 64 // 16, d % 8
    lane, odd = (4 * e + u // 2, u % 2) if value else (4 * u + e // 2, e % 2)
    if B == 8:
        return (chunk * 32 + lane) * 8 + m // 2 * 4 + m % 2 + 2 * odd
    return ((t // 16 * (D // 64) + chunk) * 32 + lane) * 16 + 4 * m + t % 16 // 8 + 2 * odd


def write4(pool, rows, slots, B, value):
    """Writes rows [T, Hkv, D] at slots into a byte pool [N, Hkv, tile], token by token."""
    T, H, D = rows.shape
    codes, scale, zero = quantise4(rows.float().numpy())
    word = (scale.view(np.uint32) >> 16) | (zero.view(np.uint32) & np.uint32(0xffff0000))
    flat = pool.numpy()
    for i in range(T):
        slot = int(slots[i])
        if slot < 0:
            continue
        n, t = divmod(slot, B)
        for d in range(D):
            if d % 16 < 8:
                flat[n, :, code_byte(value, B, D, t, d)] = codes[i, :, d] | (codes[i, :, d + 8] << 4)
        at = B * D // 2 + t * (D // 64) * 4
        flat[n, :, at:at + D // 64 * 4] = np.ascontiguousarray(word[i]).view(np.uint8)
    return pool


# ------------------------------------------------------------------ rotary positions

def rope(x, positions, inv_freq, interleaved, m, weight, eps):
    """float64 rows [T, H, D] of the normed and rotated x."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    if inv_freq is None or not inv_freq.numel():
        return x
    half = inv_freq.numel()
    out = x.clone()
    for i in range(x.shape[0]):
        for j in range(half):
            t = math.fmod(int(positions[i]) * float(inv_freq[j]), 2 * math.pi)
            c, s = m * math.cos(t), m * math.sin(t)
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            out[i, :, a] = x[i, :, a] * c - x[i, :, b] * s
            out[i, :, b] = x[i, :, b] * c + x[i, :, a] * s
    return out


# ------------------------------------------------------------------ attention

def attend(q, k, v, first, scale, window, sinks):
    """q [Q, Hq, D] at positions first .. of k, v [L, Hkv, D] (float64): [Q, Hq, D]."""
    Q, Hq, D = q.shape
    L, H = k.shape[:2]
    p = torch.arange(first, first + Q)[:, None]
    t = torch.arange(L)[None, :]
    seen = t <= p
    if window:
        seen = seen & ((t > p - window) | (t < sinks))
    out = torch.zeros(Q, Hq, D, dtype=torch.float64)
    for h in range(Hq):
        kvh = h // (Hq // H)
        z = (q[:, h].double() @ k[:, kvh].T) * float(np.float32(scale))
        z = torch.where(seen, z, torch.tensor(-math.inf, dtype=torch.float64))
        w = torch.softmax(z, -1)
        # what is not seen does not count, whatever it is
        vv = torch.where(seen.any(0)[:, None], v[:, kvh], torch.zeros((), dtype=torch.float64))
        out[:, h] = w @ vv
    return out


def decode(q, rows_of, lens, scale, window=0, sinks=0):
    """One query per sequence; rows_of(s) -> (k, v) float64 [L, Hkv, D]."""
    out = torch.zeros(q.shape, dtype=torch.float64)
    for s, L in enumerate(lens):
        if L > 0:
            k, v = rows_of(s)
            out[s] = attend(q[s:s + 1], k, v, L - 1, scale, window, sinks)[0]
    return out


def tables_of(lens, B, seed, spare=3, extra_columns=0):
    """Shuffled tables [S, width] (unused entries -1) and the pool's block count."""
    g = gen(seed)
    need = [-(-n // B) for n in lens]
    N = sum(need) + spare
    ids = torch.randperm(N, generator=g, dtype=torch.int64)
    table = torch.full((len(lens), max(1, max(need)) + extra_columns), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n].int()
        at += n
    return table, N


def worst_row(got, want):
    """Largest 2-norm error of a row relative to that row (rows = last axis)."""
    got, want = got.double().cpu().flatten(0, -2), want.double().flatten(0, -2)
    assert torch.isfinite(got).all()
    norm = want.norm(dim=-1)
    assert (got[norm == 0] == 0).all()
    live = norm > 0
    return float(((got - want).norm(dim=-1)[live] / norm[live]).max()) if live.any() else 0.0
