"""GPU tests of fd_prefill where a segment is cut between thread blocks: a row that
scores NaN everywhere in one of its pieces is NaN, wherever the cuts fall."""
import math

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from serve_util import Cache, attend, check, ints, randn

pytestmark = pytest.mark.gpu

CTAS = [0, 1, 2, 3, 7, 152]
# d, page, int8, heads: each kernel of the tensor cores (flat and paged TMA of one tile
# and two, cp.async of one and two, widened codes)
FORMS = [(128, 0, False, 2), (128, 0, False, 8), (128, 64, False, 8), (128, 16, False, 2), (128, 16, False, 8),
         (256, 0, False, 4), (256, 16, False, 4), (128, 0, True, 2), (128, 64, True, 8), (256, 16, True, 4)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


@pytest.mark.parametrize("num_ctas", CTAS)
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_a_query_row_that_is_not_a_number(form, num_ctas):
    d, page, int8, Hq = form
    rng = np.random.default_rng(61)
    n, L = 50, 700
    cache = Cache(rng, 1, L, 1, d, page, int8)
    q = randn(rng, (1, n, Hq, d)).to(torch.bfloat16).cuda()
    ref, bound = attend(q, cache, [L], [n], True, d ** -0.5)
    bad = [(0, 0), (17, Hq - 1), (n - 1, 1)]
    for i, h in bad:
        q[0, i, h, 5] = math.nan
    out = fd.prefill(q, cache.k, cache.v, ints([L]), num_ctas=num_ctas, **cache.kw())
    for i, h in bad:
        assert out[0, i, h].isnan().all(), (i, h)
        out[0, i, h] = ref[0, i, h].to(out.dtype)
    check(out, ref, bound)


@pytest.mark.parametrize("num_ctas", CTAS)
@pytest.mark.parametrize("kernel", [fd.FD_KERNEL_SIMT, fd.FD_KERNEL_AUTO])
@pytest.mark.parametrize("d,page", [(128, 0), (128, 16), (128, 64), (256, 0), (256, 24)])
def test_the_only_position_of_a_piece(kernel, d, page, num_ctas):
    # the last row alone sees position 128, which starts a block of its own
    rng = np.random.default_rng(62)
    n, L = 40, 129
    cache = Cache(rng, 1, L, 1, d, page, True)
    q = randn(rng, (1, n, 3, d)).to(torch.bfloat16).cuda()
    ref, bound = attend(q, cache, [L], [n], True, d ** -0.5)
    for scale in (cache.ks, cache.vs):
        lead, row = cache.at(0, L)
        was = scale[lead[128], 0, row[128]].clone()
        scale[lead[128], 0, row[128]] = math.nan
        out = fd.prefill(q, cache.k, cache.v, ints([L]), num_ctas=num_ctas, kernel=kernel, **cache.kw())
        scale[lead[128], 0, row[128]] = was
        assert out[0, -1].isnan().all()
        out[0, -1] = ref[0, -1].to(out.dtype)
        check(out, ref, bound)


@pytest.mark.parametrize("num_ctas", CTAS)
@pytest.mark.parametrize("d,page,int8", [(128, 0, False), (128, 64, False), (128, 16, False), (256, 0, False), (256, 16, False),
                                         (128, 64, True), (256, 16, True)])
def test_a_whole_block_of_positions(d, page, int8, num_ctas):
    # 128 positions behind which every row lies, and 128 that later rows see more and
    # more of
    rng = np.random.default_rng(63)
    B, n, L, g = 2, 300, 1000, 4
    cache = Cache(rng, B, L, 1, d, page, int8)
    q = randn(rng, (B, n, g, d)).to(torch.bfloat16).cuda()
    ref, bound = attend(q, cache, [L, L], [n, n], True, d ** -0.5)
    for b, first in ((0, 256), (1, 768)):
        lead, row = cache.at(b, L)
        at = slice(first, first + 128)
        if int8:
            cache.ks[lead[at], 0, row[at]] = math.nan
        else:
            cache.k[lead[at], :, row[at]] = math.nan
    out = fd.prefill(q, cache.k, cache.v, ints([L, L]), num_ctas=num_ctas, **cache.kw())
    assert out[0].isnan().all() and out[1, 768 - (L - n):].isnan().all()
    out[0], out[1, 768 - (L - n):] = ref[0].to(out.dtype), ref[1, 768 - (L - n):].to(out.dtype)
    check(out, ref, bound)
