"""The 4-bit cache in plain numpy: its format, its writer and decode attention
over it, from the definitions.

Format: value = code * scale * g; codes are e2m1 (1 sign, 2 exponent bits with
bias 1, 1 mantissa bit), two to a byte with the even value in the low nibble;
scales are e4m3 bytes (1 sign, 4 exponent bits with bias 7, 3 mantissa bits,
0x7f / 0xff NaN), one per 16 consecutive values.

``quantise`` works in the dtype it is given: float64 for the definition,
float32 to follow a writer that rounds every step to fp32.
"""
from __future__ import annotations

import numpy as np

GROUP = 16


def _minifloat(bits, exp_bits, man_bits, bias):
    e = (bits >> man_bits) & ((1 << exp_bits) - 1)
    m = bits & ((1 << man_bits) - 1)
    if e == 0:
        return m * 2.0 ** (1 - bias - man_bits)
    return (1 + m / 2.0 ** man_bits) * 2.0 ** (e - bias)


E2M1 = np.array([_minifloat(c, 2, 1, 1) for c in range(8)])
E4M3 = np.array([_minifloat(c, 4, 3, 7) for c in range(127)])   # 127 finite magnitudes


def _nearest(table, x):
    """Index of the entry of an ascending table nearest to x (>= 0), a tie
    going to the even index; beyond the last entry, the last."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.minimum(np.searchsorted(table, x), len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - x, x - table[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0)) | (x >= table[hi])
    return np.where(take_hi, hi, lo)


def quantise(x, g=1.0, dtype=np.float64):
    """x [..., d] -> (packed codes uint8 [..., d/2], scale bytes uint8
    [..., d/16])."""
    x = np.asarray(x, dtype=dtype)
    groups = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    with np.errstate(all="ignore"):
        amax = np.abs(groups).max(-1)
        finite = np.isfinite(groups).all(-1)
        want = amax / (dtype(6) * dtype(g))
        s = np.where(finite, _nearest(E4M3, np.where(finite, want, 0)), 0x7F).astype(np.uint8)
        sg = np.where(finite, E4M3[np.minimum(s, 126)], 0.0).astype(dtype) * dtype(g)
        y = np.abs(groups) / sg[..., None]
        y = np.where((sg > 0)[..., None], y, 0.0)
    code = _nearest(E2M1, y).astype(np.uint8)
    code |= np.where(np.signbit(groups) & finite[..., None], 8, 0).astype(np.uint8)
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def values(codes, scales, g=1.0):
    """Packed codes and scale bytes -> float64 values."""
    codes = np.asarray(codes)
    out = np.empty((*codes.shape[:-1], codes.shape[-1] * 2))
    for at, nibble in ((0, codes & 15), (1, codes >> 4)):
        out[..., at::2] = np.where(nibble & 8, -1.0, 1.0) * E2M1[nibble & 7]
    s = np.asarray(scales)
    mag = np.where((s & 0x7F) == 0x7F, np.nan, E4M3[np.minimum(s & 0x7F, 126)])
    mag = np.where(s & 0x80, -mag, mag) * g
    return out * np.repeat(mag, GROUP, axis=-1)


def rows_of(cache, b, hk, L, block_table=None):
    """The first L rows of (sequence b, kv head hk): [L, .], and which of them
    lie on pages that exist."""
    cache = np.asarray(cache)
    if block_table is None:
        return cache[b, hk, :L], np.ones(L, dtype=bool)
    pages, ps = cache.shape[0], cache.shape[2]
    pos = np.arange(L)
    e = np.asarray(block_table)[b, pos // ps] if L else np.zeros(0, dtype=np.int64)
    ok = (e >= 0) & (e < pages)
    return cache[np.where(ok, e, 0), hk, pos % ps], ok


def decode(q, k, v, ks, vs, lengths, causal, scale, k_global=1.0, v_global=1.0, block_table=None):
    """Attention of q [B, n_q, Hq, d] (float64) over a 4-bit cache (uint8
    arrays).  Returns (out, weight, size): the result, the weighted mean of
    |v| for each entry, and the largest scale * sum |q k| of each row."""
    B, n_q, Hq, d = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    cap = k.shape[2] if block_table is None else block_table.shape[1] * k.shape[2]
    out, weight = np.zeros(q.shape), np.zeros(q.shape)
    size = np.zeros(q.shape[:3])
    for b in range(B):
        L = int(min(max(int(lengths[b]), 0), cap))
        for hk in range(Hkv):
            kc, ok = rows_of(k, b, hk, L, block_table)
            kv = values(kc, rows_of(ks, b, hk, L, block_table)[0], k_global)
            vv = values(rows_of(v, b, hk, L, block_table)[0], rows_of(vs, b, hk, L, block_table)[0], v_global)
            for i in range(n_q):
                seen = ok & (np.arange(L) <= (L - n_q + i if causal else L - 1))
                if not seen.any():
                    continue
                for h in range(hk * g, (hk + 1) * g):
                    s = scale * (kv[seen] @ q[b, i, h])
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[b, i, h] = w @ vv[seen]
                    weight[b, i, h] = w @ np.abs(vv[seen])
                    size[b, i, h] = abs(scale) * (np.abs(kv[seen]) @ np.abs(q[b, i, h])).max()
    return out, weight, size


def append(new, codes, scales, lengths, new_lengths, g=1.0, block_table=None, dtype=np.float64):
    """Writes rows new [B, n, Hkv, d] into copies of a cache; returns (codes,
    scales, lengths after)."""
    codes, scales = np.array(codes), np.array(scales)
    B, n, Hkv, _ = new.shape
    ps = codes.shape[2]
    cap = ps if block_table is None else block_table.shape[1] * ps
    after = np.zeros(B, dtype=np.int32)
    for b in range(B):
        base = int(min(max(int(lengths[b]), 0), cap))
        real = n if new_lengths is None else int(min(max(int(new_lengths[b]), 0), n))
        after[b] = min(base + real, cap)
        for i in range(real):
            pos = base + i
            if pos >= cap:
                break
            lead, row = b, pos
            if block_table is not None:
                lead, row = int(block_table[b, pos // ps]), pos % ps
                if not 0 <= lead < codes.shape[0]:
                    continue
            codes[lead, :, row], scales[lead, :, row] = quantise(new[b, i], g, dtype)
    return codes, scales, after
