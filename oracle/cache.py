"""The 8-bit cache and its eviction (oracle; test infrastructure only).

Plain restatements, one row or block at a time:

* ``quantize_block``  a block's scale and codes: a = max(max |x|, 2^-100),
  scale = a / M, code = x * (M / a) rounded to the nearest value of the format,
  ties to the even code, with the quotients and the product in binary32
  (M = 448 for e4m3, 127 for int8); a block with a value that is not finite has
  the scale NaN and codes 0.
* ``decode``          the value of a code: e4m3 from its fields, int8 as it is.
* ``attention_q8``    softmax attention over the selected rows of such a cache
  and a window, with KV heads; float64.
* ``attention_mass``  the weight every selected row received, summed over the
  heads, added to the rows' accounts; float64.
* ``evict``           the blocks that stay: first, last, then by the sum of the
  rows' accounts (rounded once to binary32), ties to the lower block.
* ``compact``         an array with those blocks moved to the front of another.
"""

import math

import numpy as np

from .attention import _f64

TOP = {"e4m3": 448.0, "int8": 127.0}


def _e4m3_values():
    """The values of the 256 e4m3 codes (4 exponent bits with bias 7, 3 mantissa
    bits, subnormals, no infinities; the all-ones pattern is NaN)."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v = math.nan
        elif e == 0:
            v = m * 2.0 ** -9
        else:
            v = (8 + m) * 2.0 ** (e - 10)
        out[c] = sign * v
    return out


E4M3 = _e4m3_values()


def decode(codes, fmt):
    """float64 values of uint8 codes."""
    codes = np.asarray(codes, dtype=np.uint8)
    return E4M3[codes] if fmt == "e4m3" else codes.view(np.int8).astype(np.float64)


def nearest_e4m3(v):
    """The code (0..255) of the e4m3 value nearest to the float v, ties to the even code."""
    mag = abs(float(v))
    best = min(range(127), key=lambda c: (abs(E4M3[c] - mag), c & 1))
    return best | (128 if math.copysign(1.0, float(v)) < 0 else 0)


def round_e4m3(v):
    """``nearest_e4m3`` of every element of a finite array within [-448, 448]."""
    v = np.asarray(v, dtype=np.float64)
    mag = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3[:127], mag), 1, 126)
    lo = hi - 1
    below, above = mag - E4M3[lo], E4M3[hi] - mag
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantize_block(x, fmt):
    """(codes uint8 like x, scale float32) of one block of one KV head."""
    x = np.asarray(x, dtype=np.float32)
    if not np.all(np.isfinite(x)):
        return np.zeros(x.shape, dtype=np.uint8), np.float32(np.nan)
    top = np.float32(TOP[fmt])
    a = np.float32(max(float(np.abs(x).max()), 2.0 ** -100))
    inv = np.float32(top / a)
    v = (x * inv).astype(np.float32)
    codes = np.rint(v).astype(np.int8).view(np.uint8) if fmt == "int8" else round_e4m3(v)
    return codes, np.float32(a / top)


def cached_row(codes, scales, r, g, block, fmt):
    """float64 values of row r of KV head g: codes [T, heads, d], scales [blocks, heads]."""
    return decode(codes[r, g], fmt) * float(scales[r // block, g])


def _attended(b, g, codes, scales, idx, block, fmt, win, wl):
    """The attended rows of batch row b and KV head g, float64, and their cache rows (-1: window)."""
    T = codes.shape[1]
    at = [int(r) for r in idx[b] if 0 <= int(r) < T]
    if fmt == "bf16":
        rows = [_f64(codes[b, r, g]) for r in at]
    else:
        rows = [cached_row(codes[b], scales[b], r, g, block, fmt) for r in at]
    if win is not None:
        rows += [_f64(win[b, i, g]) for i in range(wl)]
        at = at + [-1] * wl
    d = codes.shape[3]
    return (np.stack(rows) if rows else np.zeros((0, d))), at


def attention_q8(q, codes, scales, idx, block, fmt, scale, win=None, win_len=None, sink=None):
    """float64 (out [B, H, d], lse [B, H], spread [B, H, d], reach [B, H]).

    ``codes`` uint8 [B, T, kv_heads, d] (``fmt`` "bf16": uint16 patterns),
    ``scales`` float32 [B, blocks, kv_heads], ``win`` uint16 [B, W, kv_heads, d].
    For error bounds, ``spread`` is sum_r p_r |row_r| and ``reach`` the largest
    scale * sum_c |q_c row_c| of an attended row.
    """
    qf = _f64(q)
    B, H, d = qf.shape
    G = H // codes.shape[2]
    out, lse = np.zeros((B, H, d)), np.full((B, H), -np.inf)
    spread, reach = np.zeros((B, H, d)), np.zeros((B, H))
    for b in range(B):
        W = 0 if win is None else win.shape[1]
        wl = W if win_len is None else max(0, min(int(win_len[b]), W))
        for h in range(H):
            rows, _ = _attended(b, h // G, codes, scales, idx, block, fmt, win, wl)
            z = float(scale) * (rows @ qf[b, h])
            top = max(list(z) + ([float(sink[h])] if sink is not None else []), default=-math.inf)
            if top == -math.inf:
                continue
            e = np.exp(z - top)
            total = e.sum() + (math.exp(float(sink[h]) - top) if sink is not None else 0.0)
            out[b, h] = (e @ rows) / total
            lse[b, h] = top + math.log(total)
            spread[b, h] = (e @ np.abs(rows)) / total
            reach[b, h] = abs(float(scale)) * float((np.abs(rows) @ np.abs(qf[b, h])).max()) if len(rows) else 0.0
    return out, lse, spread, reach


def attention_mass(q, codes, scales, idx, block, fmt, scale, lse, mass):
    """float64 (mass with the weights added, the weights' sum added to each row, reach [B, H])."""
    qf = _f64(q)
    B, H, _ = qf.shape
    G = H // codes.shape[2]
    added, reach = np.zeros(mass.shape), np.zeros((B, H))
    for b in range(B):
        for h in range(H):
            rows, at = _attended(b, h // G, codes, scales, idx, block, fmt, None, 0)
            if len(rows):
                reach[b, h] = abs(float(scale)) * float((np.abs(rows) @ np.abs(qf[b, h])).max())
            if lse[b, h] == -np.inf:
                continue
            for w, r in zip(np.exp(float(scale) * (rows @ qf[b, h]) - float(lse[b, h])), at):
                added[b, r] += w
    return mass.astype(np.float64) + added, added, reach


def evict(mass, length, block, budget, first, last):
    """(kept int32 [B, budget], new_len int32 [B])."""
    B, T = mass.shape
    kept, new_len = np.full((B, budget), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    for b in range(B):
        L = T if length is None else max(0, min(int(length[b]), T))
        nb = -(-L // block)

        def rank(n):
            # larger keys first, NaN above +inf, then the lower block
            if n < first or n >= nb - last:
                return (0, 0.0, n)
            with np.errstate(over="ignore", invalid="ignore"):
                key = np.float32(np.sum(mass[b, n * block: min(L, (n + 1) * block)].astype(np.float64)))
            return (1, 0.0, n) if np.isnan(key) else (2, -float(key), n)

        stay = sorted(sorted(range(nb), key=rank)[:budget])
        kept[b, :len(stay)] = stay
        new_len[b] = sum(min(block, L - n * block) for n in stay)
    return kept, new_len


def compact(src, dst, kept, length, block, per_block):
    """A copy of dst with the listed blocks of src at its front; arrays [B, items, ...]."""
    out = dst.copy()
    B = kept.shape[0]
    for b in range(B):
        for j, n in enumerate(kept[b]):
            if n < 0:
                continue
            if per_block:
                out[b, j] = src[b, n]
                continue
            for i in range(block):
                if n * block + i < int(length[b]):
                    out[b, j * block + i] = src[b, n * block + i]
    return out
