"""Decode over a 4-bit cache at scores far from 0: queries and factors so large
that a row's softmax picks one position, up to scores near the end of fp32."""
import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from fp4_util import HALF, bf16, cache, scale_of, to_dev
from oracle import fp4

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def picked(q, k, ks, v, vs, lengths, scale, kg):
    """The value row that each causal query row picks, and whether the choice
    is clear of what fp32 scores may be off by: 336 steps of 2^-23 of the
    largest scale * sum |q k|, as in decode_bound, for each of two scores."""
    B, n_q, Hq, d = q.shape
    g = Hq // k.shape[1]
    want, clear = np.zeros(q.shape), np.zeros(q.shape[:3], dtype=bool)
    for b, L in enumerate(lengths):
        for h in range(Hq):
            kv, vv = fp4.values(k[b, h // g, :L], ks[b, h // g, :L], kg), fp4.values(v[b, h // g, :L], vs[b, h // g, :L])
            for i in range(n_q):
                n = L - n_q + i + 1
                s = scale * (kv[:n] @ q[b, i, h])
                size = (scale * (np.abs(kv[:n]) @ np.abs(q[b, i, h]))).max()
                order = np.argsort(s)
                want[b, i, h] = vv[order[-1]]
                # (beyond 40 the second weighs less than 2^-57)
                clear[b, i, h] = s[order[-1]] - s[order[-2]] > 40 + 2 * 336 * 2.0 ** -23 * size
    return want, clear


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("n_q,g", [(1, 4), (3, 4), (6, 4), (5, 8)])
@pytest.mark.parametrize("q_spread,kg", [(1e5, 1.0), (1e7, 1.0), (3e8, 1.0), (1e9, 1.0), (1e13, 1.0), (1e20, 1.0),
                                         (3e36, 1.0), (1.0, 2.0 ** 30), (1.0, 2.0 ** 63), (1e-9, 2.0 ** 63)])
def test_large_scores_pick_one_position(d, out_dtype, n_q, g, q_spread, kg):
    rng = np.random.default_rng(91)
    lengths = [1500, 333]
    # keys of both signs: every row's best score is positive
    k, ks = cache(rng, 2, 2, 1500, d, kg, kg)
    v, vs = cache(rng, 2, 2, 1500, d)
    q = bf16(rng, (2, n_q, 2 * g, d), q_spread)
    (kd, ksd), (vd, vsd) = to_dev(k, ks), to_dev(v, vs)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = fd.decode_fp4(q.cuda(), kd, vd, ksd, vsd, lens, causal=True, k_global=kg, out_dtype=out_dtype).double().cpu().numpy()
    want, clear = picked(q.double().numpy(), k, ks, v, vs, lengths, scale_of(d), kg)
    assert clear.mean() > 0.8
    assert np.isfinite(got).all()
    # one weight and its own sum: the quotient of two numbers that are equal but
    # for the weight's rounding to the MMA's type (2^-11 of it)
    err = np.abs(got - want)[clear]
    assert (err <= (HALF[out_dtype] + 2.0 ** -11 + 2.0 ** -20) * np.abs(want[clear])).all(), err.max()
    # a row that is not clear still lies among the values
    assert np.abs(got).max() <= np.abs(fp4.values(v, vs)).max() * 1.01


def test_scores_that_all_lie_far_below_zero():
    # the largest score of every row is about -2^40
    rng = np.random.default_rng(92)
    d, L = 128, 700
    rows = rng.uniform(1, 2, (1, 1, L, d))
    k, ks = fp4.quantise(rows)
    v, vs = cache(rng, 1, 1, L, d)
    q = -(torch.from_numpy(rng.uniform(1, 2, (1, 2, 4, d))) * 2.0 ** 36).to(BF)
    (kd, ksd), (vd, vsd) = to_dev(k, ks), to_dev(v, vs)
    got = fd.decode_fp4(q.cuda(), kd, vd, ksd, vsd, torch.tensor([L], dtype=torch.int32, device="cuda"), causal=True,
                        out_dtype=F32).double().cpu().numpy()
    want, clear = picked(q.double().numpy(), k, ks, v, vs, [L], scale_of(d), 1.0)
    assert clear.any() and np.isfinite(got).all()
    assert (np.abs(got - want)[clear] <= (2.0 ** -11 + 2.0 ** -20) * np.abs(want[clear])).all()
