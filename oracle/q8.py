"""The 8-bit cache in plain fp64: e4m3 bytes with one power-of-two scale for
each page, kv head and K or V.

Written from the format's definition (a byte is a sign, 4 exponent bits with
bias 7 and 3 mantissa bits; exponent 0 is subnormal; 0x7f is NaN; the largest
number is 448) and from the two rules of the cache: the scale of a page is
2^e with the smallest e >= -117 for which max |k| <= 316 * 2^e (before the
rotation) or max |v| <= 448 * 2^e, and a page that holds tokens keeps the
larger of its exponent and the new tokens'.
"""
from __future__ import annotations

import numpy as np

from . import (BLOCK, ERR_BAD_BLOCK, ERR_CTX_RANGE, ERR_FREE_UNDERFLOW, HEAD_DIM, N_KV, N_Q,
               bf16_to_f64, llama3_inv_freq)

ERR_BAD_SCALE = 32
LIMIT_K, LIMIT_V = 316.0, 448.0
E_MIN, E_MAX = -117, 120


def _values() -> np.ndarray:
    v = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[b] = -x if b & 128 else x
    v[0x7F] = v[0xFF] = np.nan
    return v


VALUES = _values()
_POS = VALUES[:127]                          # 0 .. 448, ascending
_MID = (_POS[1:] + _POS[:-1]) / 2.0          # exact in fp64


def encode(x) -> np.ndarray:
    """The byte nearest to x: ties to the even byte, beyond 448 the largest,
    NaN and infinities NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    lo = np.searchsorted(_MID, a, side="left")         # a <= _MID[lo]: byte lo, a tie goes up or stays
    tie = (lo < 126) & (a == _MID[np.minimum(lo, 125)])
    b = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.uint8)
    b = np.where(np.signbit(x), b | 128, b).astype(np.uint8)
    return np.where(np.isfinite(x), b, np.uint8(0x7F))


def decode(bytes_, scales) -> np.ndarray:
    """Values fp64 of a pool [..][2][page][8][64] under scales [..][2][8]."""
    return VALUES[bytes_] * np.asarray(scales, dtype=np.float64)[..., :, None, :, None]


def to_bf16(x) -> np.ndarray:
    """fp64 to bf16 bits, nearest even; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    e = np.maximum(np.frexp(a)[1] - 1, -126)
    step = np.ldexp(1.0, e - 7)
    r = np.rint(a / step) * step
    with np.errstate(over="ignore"):
        u = (r.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    u = np.where(np.isinf(x), np.uint16(0x7F80), u)
    u = np.where(np.isnan(x), np.uint16(0x7FC0), u)
    return np.where(np.signbit(x), u | 0x8000, u).astype(np.uint16)


def pool_bf16(bytes_, scales) -> np.ndarray:
    """The pool as bf16 bits: exact, a byte has 4 significant bits."""
    return to_bf16(decode(bytes_, scales))


def exponent(values, limit) -> int:
    """Smallest e >= E_MIN with max |finite values| <= limit * 2^e."""
    a = np.abs(values[np.isfinite(values)])
    top = float(a.max()) if a.size else 0.0
    e = E_MIN
    while top > np.ldexp(limit, e):
        e += 1
    return e


def rotate(x, positions) -> np.ndarray:
    """Rotate-half RoPE of rows x [T][H][64] at positions [T], fp64."""
    ang = np.asarray(positions, dtype=np.float64)[:, None] * llama3_inv_freq()[None, :]
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
    a, b = x[..., :HEAD_DIM // 2], x[..., HEAD_DIM // 2:]
    with np.errstate(invalid="ignore"):
        return np.concatenate([a * c - b * s, b * c + a * s], axis=-1)


def append(k_new, v_new, q, cu_tokens, pool, scales, block_table, context_lens, layer, free_list,
           free_count):
    """The prefill append (a decode append is one row a sequence).  bf16 bits
    k_new, v_new [T][8][64], q [T][32][64] or None; pool uint8
    [blocks][2][page][8][64], scales fp32 [blocks][2][8].  Returns copies
    (q_rot bits or None, pool, scales, block_table, free_count, err)."""
    pool, scales = pool.copy(), np.array(scales, dtype=np.float32)
    table = np.array(block_table, dtype=np.int32)
    page, num_blocks = pool.shape[2], pool.shape[0]
    cap = table.shape[2] * page
    k, v = bf16_to_f64(k_new), bf16_to_f64(v_new)
    qr = None if q is None else np.array(q, dtype=np.uint16)
    err, count = 0, int(free_count)
    for s in range(table.shape[0]):
        c0, c1, ctx = int(cu_tokens[s]), int(cu_tokens[s + 1]), int(context_lens[s])
        if ctx < 0 or c1 < c0 or c0 < 0 or c1 > len(k) or ctx + c1 - c0 > cap:
            err |= ERR_CTX_RANGE
            continue
        pos = np.arange(ctx, ctx + c1 - c0)
        if q is not None and len(pos):
            qr[c0:c1] = to_bf16(rotate(bf16_to_f64(q[c0:c1]), pos))
        kr = bf16_to_f64(to_bf16(rotate(k[c0:c1], pos)))
        at = 0
        while at < len(pos):
            slot = int(pos[at]) % page
            n = min(page - slot, len(pos) - at)
            rows = slice(c0 + at, c0 + at + n)
            j = int(pos[at]) // page
            if slot == 0:
                if count > 0:
                    count -= 1
                    table[s, layer, j] = free_list[count]
                else:
                    table[s, layer, j] = -1
                    err |= ERR_FREE_UNDERFLOW
            blk = int(table[s, layer, j])
            if not 0 <= blk < num_blocks:
                if slot != 0 or blk != -1:
                    err |= ERR_BAD_BLOCK
                at += n
                continue
            for h in range(N_KV):
                for i, (raw, x, limit) in enumerate(((k[rows, h], kr[at:at + n, h], LIMIT_K),
                                                     (v[rows, h], v[rows, h], LIMIT_V))):
                    e = exponent(raw, limit)
                    if slot:
                        old = float(scales[blk, i, h])
                        if not (old > 0 and np.frexp(old)[0] == 0.5 and
                                E_MIN <= np.frexp(old)[1] - 1 <= E_MAX):
                            err |= ERR_BAD_SCALE
                            continue
                        e = max(e, int(np.frexp(old)[1]) - 1)
                        if np.ldexp(1.0, e) != old:
                            held = VALUES[pool[blk, i, :slot, h]] * (old / np.ldexp(1.0, e))
                            pool[blk, i, :slot, h] = encode(held)
                    scales[blk, i, h] = np.ldexp(1.0, e)
                    pool[blk, i, slot:slot + n, h] = encode(x / np.ldexp(1.0, e))
            at += n
    return qr, pool, scales, table, count, err


def random_pool(rng, num_blocks, page=BLOCK):
    """Bytes of N(0, 1)-like values and scales 2^-8 .. 2^-4."""
    scales = np.ldexp(1.0, rng.integers(-8, -3, size=(num_blocks, 2, N_KV))).astype(np.float32)
    x = np.clip(rng.standard_normal((num_blocks, 2, page, N_KV, HEAD_DIM)) * 90.0, -448.0, 448.0)
    return encode(x), scales


__all__ = ["N_Q", "encode", "decode", "to_bf16", "pool_bf16", "exponent", "rotate", "append",
           "random_pool", "VALUES"]
