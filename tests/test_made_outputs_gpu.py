"""GPU tests of the outputs that append and prefill make: what no row writes is zero,
not what the memory held."""
import math

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from serve_util import Cache, attend, check, ints, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def dirty(like, stream):
    """Memory of that size, full of NaN, is what the next output gets."""
    with torch.cuda.stream(stream):
        held = [torch.full_like(like, math.nan) for _ in range(4)]
        del held


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("new", [[40, 0, 17], [1, 40, 39]])
def test_padding(new, side):
    rng = np.random.default_rng(81)
    B, n, Hq, Hkv, d = 3, 40, 8, 2, 128
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    given = stream if side else None
    cache = Cache(rng, B, 200, Hkv, d, 16)
    q, kn, vn = (randn(rng, (B, n, h, d)).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    lens, fresh = ints([100, 50, 3]), ints(new)
    after = torch.zeros_like(lens)
    torch.cuda.synchronize()
    for _ in range(3):
        dirty(q, stream)
        q2 = fd.append(kn, vn, cache.k, cache.v, lens, new_lengths=fresh, lengths_out=after, q=q, block_table=cache.table, stream=given)
        dirty(q, stream)
        out = fd.prefill(q2, cache.k, cache.v, after, new_lengths=fresh, block_table=cache.table, stream=given)
        torch.cuda.synchronize()
        for b in range(B):
            assert torch.equal(q2[b, :new[b]], q[b, :new[b]])
            assert (q2[b, new[b]:] == 0).all() and (out[b, new[b]:] == 0).all()
        ref, bound = attend(q, cache, after.tolist(), new, True, d ** -0.5)
        check(out, ref, bound)
