"""Helpers of the 4-bit cache tests: seeded caches, device copies and the
error bound of a decode call."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import fp4

#: half a step of the output's rounding
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def cache(rng, lead, Hkv, rows, d, g=1.0, spread=1.0):
    """Quantised N(0, spread) rows: packed codes and scale bytes."""
    return fp4.quantise(rng.standard_normal((lead, Hkv, rows, d)) * spread, g)


def to_dev(codes, scales, token_major=False):
    c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    if token_major:
        c, s = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (c, s))
    return c, s.view(torch.float8_e4m3fn)


def bf16(rng, shape, spread=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * spread).to(torch.bfloat16)


def decode_bound(ref, weight, size, L, vmax, out_dtype):
    """How far a decode result may be from the 64-bit one.
    - the output's rounding: half a step of |ref|;
    - each weight: rounded to fp16 (2^-11 of it), 2^x by the special function
      unit (2^-22), and the error of its exponent: a score is a sum of d <= 256
      exact products in fp32 (each of up to 264 steps off by at most 2^-23 of
      the terms' absolute sum, truncation included), scaled twice (2^-23), an
      fp16 q off by 2^-25 of its largest entry where it is small.  A relative
      error e of the weights moves the result by at most e * (weight + |ref|);
    - weights below 2^-24 of fp16's own range: 2^-29 of the largest each;
    - fp32 sums over L weights, merged over splits: (L / 8 + 64) * 2^-24 of
      weight and of the normaliser."""
    e = 2.0 ** -11 + 2.0 ** -22 + (264 + 4 + 64) * 2.0 ** -23 * size[..., None]
    e = e + (L / 8 + 64) * 2.0 ** -23
    return HALF[out_dtype] * np.abs(ref) * (1 + 1e-3) + e * (weight + np.abs(ref)) + L * 2.0 ** -29 * vmax


def check(got, ref, bound, what=""):
    g = got.detach().double().cpu().numpy()
    assert g.shape == ref.shape
    assert np.isfinite(g).all(), what + ": not finite"
    over = np.abs(g - ref) - bound
    at = np.unravel_index(over.argmax(), over.shape)
    assert over[at] <= 0, "%s: %r against %r at %s, bound %.3g" % (what, g[at], ref[at], at, bound[at])


def scale_of(d):
    return 1.0 / math.sqrt(d)
