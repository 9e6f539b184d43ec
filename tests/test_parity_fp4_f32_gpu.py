"""fp32 outputs of decode over a 4-bit cache: weights in two fp16 numbers, so
that no error of the size of fp16's rounding is left in them."""
import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from fp4_util import bf16, cache, check, scale_of, to_dev
from oracle import fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def bound(ref, weight, size, L, vmax):
    """decode_bound of an fp32 output without its terms of one fp16 weight:
    - the output's rounding: half a step of |ref|;
    - each weight: what fp16 leaves of it, at most 2^-11, is rounded to fp16
      again (2^-11 of that, 2^-22 in all; 2^-37 of the row's largest where that
      is more), 2^x by the special function unit (2^-22), and the error of its
      exponent, 332 steps of 2^-23 of the terms' absolute sum;
    - fp32 sums over L weights, merged over splits: (L / 8 + 64) * 2^-24 of
      weight and of the normaliser."""
    e = 2.0 ** -22 + 2.0 ** -22 + 332 * 2.0 ** -23 * size[..., None] + (L / 8 + 64) * 2.0 ** -23
    return 2.0 ** -24 * np.abs(ref) * (1 + 1e-3) + e * (weight + np.abs(ref)) + L * 2.0 ** -37 * vmax


def case(seed, lengths, n_q, g, d, page=0, num_ctas=0, q_spread=0.05, Hkv=2):
    """Queries so small that the bound lies far below 2^-11."""
    rng = np.random.default_rng(seed)
    B, cap = len(lengths), max(lengths)
    table, lead, rows = None, B, cap
    if page:
        mp = -(-cap // page)
        table = rng.permutation(B * mp + 2)[:B * mp].reshape(B, mp).astype(np.int32)
        lead, rows = B * mp + 2, page
    (k, ks), (v, vs) = (cache(rng, lead, Hkv, rows, d) for _ in range(2))
    q = bf16(rng, (B, n_q, Hkv * g, d), q_spread)
    want, weight, size = fp4.decode(q.double().numpy(), k, v, ks, vs, lengths, True, scale_of(d), block_table=table)
    (kd, ksd), (vd, vsd) = to_dev(k, ks), to_dev(v, vs)
    got = fd.decode_fp4(q.cuda(), kd, vd, ksd, vsd, torch.tensor(lengths, dtype=torch.int32, device="cuda"), causal=True,
                        block_table=None if table is None else torch.from_numpy(table).cuda(), out_dtype=torch.float32,
                        num_ctas=num_ctas)
    check(got, want, bound(want, weight, size, max(lengths), np.abs(fp4.values(v, vs)).max()), "fp32")


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page", [0, 16, 7])
@pytest.mark.parametrize("n_q,g", [(1, 1), (1, 8), (2, 6), (6, 4), (4, 8), (6, 10)])
def test_short_rows(d, page, n_q, g):
    case(101, [6, 9, 17, 33, 64, 100, 1], n_q, g, d, page)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n_q,g", [(1, 4), (3, 4), (6, 4), (5, 6)])
@pytest.mark.parametrize("ctas", [1, 5, 60])
def test_splits(d, n_q, g, ctas):
    case(102, [1400, 300], n_q, g, d, num_ctas=ctas)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("q_spread", [1.0, 30.0])
def test_rising_references(d, q_spread):
    case(103, [900, 64], 6, 4, d, q_spread=q_spread)
