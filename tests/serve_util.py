"""Helpers of the append, prefill and beam tests: seeded caches, the operators in
64 bits, and the error bound of a prefill call."""
from __future__ import annotations

import math

import numpy as np
import torch

F64 = torch.float64


def ints(x, device="cuda"):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)


def randn(rng, shape, spread=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * spread).float()


def quantise(x):
    """Codes and scales of x [..., d] (fp32) as fd_append has them."""
    s = x.abs().amax(-1) / np.float32(127)
    y = torch.where((s > 0).unsqueeze(-1), x / s.unsqueeze(-1), torch.zeros(()))
    return torch.round(y).clamp(-127, 127).to(torch.int8), s


class Cache:
    """A bf16 or int8 cache, flat or paged, of B sequences of `cap` positions:
    `k`, `v`, `ks`, `vs`, `table` as the calls take them.  filled: with rows
    N(0, 1); else with what must never be read (NaN, or a NaN scale)."""

    def __init__(self, rng, B, cap, Hkv, d, page=0, int8=False, token_major=False, filled=True, spare=2, device="cuda"):
        self.B, self.Hkv, self.d, self.page, self.int8 = B, Hkv, d, page, int8
        self.table, lead, rows = None, B, cap
        if page:
            mp = -(-cap // page)
            lead, rows = B * mp + spare, page
            self.table = ints(rng.permutation(lead)[:B * mp].reshape(B, mp), device)
            cap = mp * page
        self.cap = cap
        shape = (lead, Hkv, rows, d)
        self.ks = self.vs = None
        caches = []
        for _ in range(2):
            x = randn(rng, shape) if filled else torch.full(shape, math.nan)
            if int8:
                c, s = quantise(x) if filled else (torch.full(shape, 99, dtype=torch.int8), torch.full(shape[:3], math.nan))
            else:
                c, s = x.to(torch.bfloat16), None
            c, s = (t if t is None else t.to(device) for t in (c, s))
            if token_major:
                c, s = (t if t is None else t.transpose(1, 2).contiguous().transpose(1, 2) for t in (c, s))
            caches.append((c, s))
        (self.k, self.ks), (self.v, self.vs) = caches

    def kw(self):
        return dict(k_scale=self.ks, v_scale=self.vs, block_table=self.table)

    def at(self, b, n):
        """Where positions 0 .. n-1 of sequence b lie: (leading index, row)."""
        pos = torch.arange(n, device=self.k.device)
        if self.table is None:
            return torch.full_like(pos, b), pos
        return self.table[b].long()[pos // self.page], pos % self.page

    def rows(self, which, b, n):
        """Positions 0 .. n-1 of sequence b as numbers, [n, Hkv, d] in 64 bits."""
        lead, row = self.at(b, n)
        c = (self.k, self.v)[which][lead, :, row].to(F64)
        return c if not self.int8 else c * (self.ks, self.vs)[which][lead, :, row].to(F64).unsqueeze(-1)

    def spoil(self, lens):
        """What must never be read, from each length on (and in pages that
        nobody holds)."""
        for t in (self.k, self.v) if not self.int8 else (self.ks, self.vs):
            keep = torch.zeros(t.shape[0], t.shape[2], dtype=torch.bool, device=t.device)
            for b, n in enumerate(lens):
                keep[self.at(b, int(n))] = True
            t.transpose(1, 2)[~keep] = math.nan
        if self.table is not None:
            for b, n in enumerate(lens):
                self.table[b, -(-int(n) // self.page):] = 1 << 29


def attend(q, cache, lens, new, causal, scale):
    """fd_prefill in 64 bits: out [B, n, Hq, d] and its bound (see below)."""
    B, n, Hq, d = q.shape
    out = torch.zeros(q.shape, dtype=F64, device=q.device)
    bound = torch.zeros_like(out)
    g = Hq // cache.Hkv
    for b in range(B):
        L, t = int(lens[b]), int(new[b])
        if not (L and t):
            continue
        x = q[b, :t].to(F64).view(t, cache.Hkv, g, d)
        k, v = cache.rows(0, b, L), cache.rows(1, b, L)
        s = torch.einsum("ihgd,jhd->hgij", x, k) * scale
        size = torch.einsum("ihgd,jhd->hgij", x.abs(), k.abs()) * abs(scale)
        seen = torch.ones(t, L, dtype=torch.bool, device=q.device)
        if causal:
            i, j = torch.arange(t, device=q.device).view(t, 1), torch.arange(L, device=q.device)
            seen = j <= L - t + i
        s = s.masked_fill(~seen, -math.inf)
        size = torch.where(seen, size, 0.0).amax(-1)
        p = torch.softmax(s, -1).nan_to_num(0.0)
        o = torch.einsum("hgij,jhd->ihgd", p, v)
        w = torch.einsum("hgij,jhd->ihgd", p, v.abs())
        # - the output's rounding to bf16, half a step: 2^-8 of it;
        # - each weight: its rounding to bf16 (2^-8), of 2^x by the special
        #   function unit (2^-22), and the error of its exponent: a sum of d <= 256
        #   products, each step off by at most 2^-23 of the terms' absolute sum
        #   (truncation included), and three roundings of the scaled score;
        # - sums over L weights in fp32, joined over splits: (L / 8 + 64) * 2^-23.
        e = 2.0 ** -8 + 2.0 ** -22 + (264 + 4 + 64) * 2.0 ** -23 * size.permute(2, 0, 1).unsqueeze(-1) + (L / 8 + 64) * 2.0 ** -23
        out[b, :t] = o.reshape(t, Hq, d)
        bound[b, :t] = (2.0 ** -8 * o.abs() * (1 + 1e-3) + e * (w + o.abs()) + 1e-30).reshape(t, Hq, d)
    return out, bound


def check(got, ref, bound, what=""):
    assert got.shape == ref.shape
    assert torch.isfinite(got).all(), what + ": not finite"
    over = (got.to(F64) - ref).abs() - bound
    at = int(over.argmax())
    assert float(over.flatten()[at]) <= 0, "%s: %r against %r at %d, bound %.3g" % (
        what, float(got.flatten()[at]), float(ref.flatten()[at]), at, float(bound.flatten()[at]))


def rope_table(positions, r, base=10000.0):
    a = np.arange(positions)[:, None] * base ** (-np.arange(0, r, 2) / r)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float()


def turned(x, rope, pos, interleaved, dtype=torch.float32):
    """x [n, H, d] (numbers) with its first r values turned to positions pos [n]."""
    x = x.to(dtype).clone()
    r = rope.shape[1]
    c, s = rope[pos, :r // 2].to(dtype).unsqueeze(1), rope[pos, r // 2:].to(dtype).unsqueeze(1)
    at = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    a, b = x[..., at[0]].clone(), x[..., at[1]].clone()
    x[..., at[0]] = a * c - b * s
    x[..., at[1]] = b * c + a * s
    return x
