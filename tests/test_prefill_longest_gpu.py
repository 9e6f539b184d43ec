"""GPU tests of fd_prefill at the largest lengths: one page again and again, up to the
last of 2^31 positions, is attended as the page alone."""
import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from serve_util import Cache, attend, ints, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


# TMA boxes of two tiles, cp.async of one and two, codes; pages of 128 rows
@pytest.mark.parametrize("d,n,g,page,int8", [(128, 200, 1, 128, False), (128, 1, 4, 128, False), (128, 140, 1, 32, False),
                                             (256, 2, 4, 128, False), (128, 60, 4, 128, True), (256, 3, 2, 64, True)])
@pytest.mark.parametrize("less", [0, 77])
def test_two_billion_positions(d, n, g, page, int8, less):
    rng = np.random.default_rng(111)
    cache = Cache(rng, 1, page, 1, d, page, int8, spare=0)
    q = randn(rng, (1, n, g, d)).to(torch.bfloat16).cuda()
    ref, _ = attend(q, cache, [page], [n], False, d ** -0.5)
    most = cache.rows(1, 0, page).abs().amax()
    pages = ((1 << 31) - 1) // page
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    ws = fd.Workspace(4096, 16, 256, 1024)
    out = torch.full_like(q, 9.0)
    for causal in (True, False):
        fd.prefill(q, cache.k, cache.v, ints([pages * page - less]), causal=causal, k_scale=cache.ks, v_scale=cache.vs, block_table=table,
                   out=out, workspace=ws)
        assert ws.device_status() == 0
        # a thread block adds some 2^24 / 152 blocks' parts, in 8 steps each, in fp32: by
        # half a step of 2^-23 a time at most in one direction, 2^-4.3 of what it adds up
        assert float((out.double() - ref).abs().max()) <= 2.0 ** -4 * float(most)
