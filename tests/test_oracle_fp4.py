"""Pins of the 4-bit cache oracle and of the page-book oracle: values worked
out by hand, library conversions, closed forms and the fp64 dense oracle."""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp4
from oracle.pages import Books


def test_code_and_scale_tables():
    assert fp4.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert (fp4.E4M3 == want).all() and fp4.E4M3[-1] == 448


@pytest.mark.parametrize("x,code", [(0.25, 0), (0.2500001, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6),
                                    (5.0, 6), (5.0000001, 7), (6.0, 7), (7.9, 7), (-0.75, 10), (-0.1, 8), (0.0, 0)])
def test_nearest_code_ties_to_even(x, code):
    row = np.zeros(16)
    row[0], row[1] = 6.0, x          # 6 fixes the scale at 1
    if abs(x) > 6:
        row[0] = 6.0 * 448 * 2       # a saturated scale of 448
        row[1] = x * 448
    codes, s = fp4.quantise(row)
    assert codes[0] >> 4 == code
    assert fp4.E4M3[s[0]] == (1.0 if abs(x) <= 6 else 448.0)


def test_scale_rounds_to_nearest_even_as_the_library_does():
    rng = np.random.default_rng(0)
    x = np.exp(rng.uniform(-9, 7, 4000))
    x[:126] = (fp4.E4M3[:-1] + fp4.E4M3[1:]) / 2      # ties
    want = torch.from_numpy(np.minimum(x, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    x = np.minimum(x, 448).astype(np.float32)
    assert (fp4._nearest(fp4.E4M3, x) == want).all()


def test_zero_and_non_finite_groups():
    row = np.zeros(48)
    row[16], row[20] = np.nan, 3.0
    row[32], row[33] = -np.inf, 1.0
    codes, s = fp4.quantise(row)
    assert s.tolist() == [0, 0x7F, 0x7F] and not codes.any()
    v = fp4.values(codes, s)
    assert (v[:16] == 0).all() and np.isnan(v[16:]).all()


def test_round_trip_of_representable_values():
    rng = np.random.default_rng(1)
    code = rng.integers(0, 16, (5, 128)).astype(np.uint8)
    code[:, ::16] = 7                                # every group's largest is 6
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    s = rng.integers(1, 127, (5, 8)).astype(np.uint8)
    x = fp4.values(packed, s, 0.5)
    c2, s2 = fp4.quantise(x, 0.5)
    assert (s2 == s).all() and (fp4.values(c2, s2, 0.5) == x).all()


def test_decode_equals_the_dense_oracle_on_representable_values():
    # code * scale has 6 significant bits: bf16 holds it, so the bf16 dense
    # oracle is an independent check of the attention part
    rng = np.random.default_rng(2)
    B, Hkv, g, n_q, cap, d = 2, 2, 3, 3, 40, 128
    kc, vc = (rng.integers(0, 256, (B, Hkv, cap, d // 2)).astype(np.uint8) for _ in range(2))
    ks, vs = (rng.integers(40, 60, (B, Hkv, cap, d // 16)).astype(np.uint8) for _ in range(2))
    q = torch.randn(B, n_q, Hkv * g, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    lens = torch.tensor([37, 2], dtype=torch.int32)
    k, v = (torch.from_numpy(fp4.values(c, s)).to(torch.bfloat16) for c, s in ((kc, ks), (vc, vs)))
    want = oracle.dense(q, k, v, lens, n_q, True, 0.1)
    got, weight, size = fp4.decode(q.double().numpy(), kc, vc, ks, vs, lens.numpy(), True, 0.1)
    assert np.abs(got - want).max() < 1e-12
    assert (got[1, 0] == 0).all()                    # length 2, 3 rows: the first sees nothing
    assert (np.abs(got) <= weight + 1e-12).all() and (size[0] > 0).all()


def test_decode_pages_and_missing_pages():
    rng = np.random.default_rng(4)
    kc, vc = (rng.integers(0, 256, (5, 1, 4, 64)).astype(np.uint8) for _ in range(2))
    ks, vs = (rng.integers(40, 60, (5, 1, 4, 8)).astype(np.uint8) for _ in range(2))
    table = np.array([[3, -1, 1, 0]])
    q = rng.standard_normal((1, 1, 2, 128))
    got = fp4.decode(q, kc, vc, ks, vs, [11], False, 0.1, block_table=table)[0]
    flat = [np.concatenate([c[3], c[1][:, :3]], 1)[None] for c in (kc, vc, ks, vs)]   # 4 rows, none, 3 rows
    want = fp4.decode(q, *flat, [7], False, 0.1)[0]
    assert np.abs(got - want).max() < 1e-12


def books():
    # 3 sequences of 4-position pages in a pool of 8; rows 0 and 1 share page 2
    return Books([[5, 2, -1, -1], [5, 2, -1, -1], [0, -1, -1, -1]], [6, 6, 3], [1, 0, 2, 0, 0, 2, 0, 0], 4)


def test_books_reserve_by_hand():
    k = books()
    assert k.consistent()
    # all three write: row 0 keeps page 2, row 1 moves to page 1 (copied), row
    # 2's next position is the last of page 0
    assert k.reserve(1) == [(2, 1)]
    assert k.table.tolist() == [[5, 2, -1, -1], [5, 1, -1, -1], [0, -1, -1, -1]] and k.consistent()
    # row 1 alone, two pages more; row 0's page is its own now
    assert k.reserve([0, 7, 0]) == []
    assert k.table[1].tolist() == [5, 1, 3, 4] and k.consistent()
    # pages 6 and 7 are left: row 0 wants two and row 2 two, so nothing changes
    before = k.table.copy()
    assert k.reserve([8, 0, 9]) == -2 and (k.table == before).all() and k.consistent()


def test_books_reserve_copies_when_a_holder_does_not_write():
    k = books()
    assert k.reserve([1, 0, 0]) == [(2, 1)]
    assert k.table[0].tolist() == [5, 1, -1, -1] and k.table[1].tolist() == [5, 2, -1, -1] and k.consistent()


def test_books_fork_free_compact_by_hand():
    k = books()
    k.fork([0], [2], [4])
    assert k.table[2].tolist() == [5, -1, -1, -1] and k.lengths[2] == 4
    assert k.refs.tolist() == [0, 0, 2, 0, 0, 3, 0, 0] and k.consistent()
    k.free([1], [5])
    assert k.lengths[1] == 5 and k.table[1].tolist() == [5, 2, -1, -1]
    k.free([1])
    assert k.refs.tolist() == [0, 0, 1, 0, 0, 2, 0, 0] and k.consistent()
    assert k.compact() == [(2, 0), (5, 1)]
    assert k.table.tolist() == [[1, 0, -1, -1], [-1] * 4, [1, -1, -1, -1]] and k.refs[:3].tolist() == [1, 2, 0]


def test_books_fork_skips_ambiguous_entries():
    k = books()
    k.fork([0, 2, 1, 2], [1, 1, 0, 2])   # 1 is a source, 1 again, 0 is a source, 2 onto itself
    assert k.table.tolist() == books().table.tolist() and k.consistent()
