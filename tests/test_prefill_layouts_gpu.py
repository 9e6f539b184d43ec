"""GPU tests of fd_prefill and fd_append over layouts that their documentation allows
besides the usual ones: int8 caches and scales of any strides, groups that do not fill a
tile, inputs that are broadcast."""
import math

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from serve_util import Cache, attend, check, ints, randn, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def spread(t, pad, extra):
    """The same rows `pad` elements further apart, heads and pages `extra` more."""
    lead, H, rows, d = t.shape
    x = torch.full((lead, H * (rows * (d + pad) + extra) + extra), 77, dtype=t.dtype, device=t.device)
    return x.as_strided(t.shape, (x.stride(0), rows * (d + pad) + extra, d + pad, 1)).copy_(t)


def scattered(s):
    """The same scales, no dimension dense, NaN between them."""
    lead, H, rows = s.shape
    x = torch.full((rows, lead, H, 3), math.nan, device=s.device)
    y = x[..., 1].permute(1, 2, 0)
    y.copy_(s)
    return y


@pytest.mark.parametrize("kernel", [fd.FD_KERNEL_SIMT, fd.FD_KERNEL_AUTO])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("d,page", [(128, 0), (128, 16), (128, 24), (128, 64), (256, 0), (256, 16)])
def test_int8_caches_of_any_strides(d, page, apart, kernel):
    rng = np.random.default_rng(101)
    B, n, Hq, Hkv = 2, 70, 8, 2
    cache = Cache(rng, B, 400, Hkv, d, page, True)
    q = randn(rng, (B, n, Hq, d)).to(torch.bfloat16).cuda()
    lens = [400, 171]
    ref, bound = attend(q, cache, lens, [n, n], True, d ** -0.5)
    cache.k = spread(cache.k, 16, 0)
    cache.v = spread(cache.v, 32 if apart else 16, 48 if apart else 0)
    cache.ks, cache.vs = scattered(cache.ks), scattered(cache.vs)
    ws = fd.Workspace(4096, 16, 256, 1024)
    check(fd.prefill(q, cache.k, cache.v, ints(lens), kernel=kernel, workspace=ws, **cache.kw()), ref, bound)
    assert ws.device_status() == 0


@pytest.mark.parametrize("kernel", [fd.FD_KERNEL_SIMT, fd.FD_KERNEL_AUTO])
@pytest.mark.parametrize("g", [3, 11, 43, 65, 85, 127, 128])
@pytest.mark.parametrize("d,page,int8", [(128, 0, False), (128, 64, False), (128, 16, False), (256, 0, False), (256, 48, False),
                                         (128, 32, True), (256, 16, True)])
def test_groups_that_do_not_fill_a_tile(d, page, int8, g, kernel):
    rng = np.random.default_rng(102 + g)
    B, n, L = 2, 150, 420
    cache = Cache(rng, B, L, 1, d, page, int8)
    q = randn(rng, (B, n, g, d)).to(torch.bfloat16).cuda()
    lens, new = [L, 150], [n, 149]
    ref, bound = attend(q, cache, lens, new, True, d ** -0.5)
    cache.spoil(lens)
    for num_ctas in (0, 3):
        out = torch.zeros_like(q)
        fd.prefill(q, cache.k, cache.v, ints(lens), new_lengths=ints(new), out=out, kernel=kernel, num_ctas=num_ctas, **cache.kw())
        check(out, ref, bound)


@pytest.mark.parametrize("d,page,int8", [(128, 0, False), (128, 16, False), (256, 16, True)])
def test_broadcast_inputs(d, page, int8):
    # one query for every head and sequence, one cache for every sequence, one new row for
    # every kv head
    rng = np.random.default_rng(103)
    B, n, Hq, Hkv, L = 3, 33, 8, 2, 300
    one = randn(rng, (1, n, 1, d)).to(torch.bfloat16).cuda()
    q = one.expand(B, n, Hq, d)
    cache = Cache(rng, B if page else 1, L, Hkv, d, page, int8)
    if not page:
        cache.k, cache.v = (t.expand(B, -1, -1, -1) for t in (cache.k, cache.v))
    lens = [L, 33, 190]
    ref, bound = attend(q, cache, lens, [n] * B, True, d ** -0.5)
    for kernel in (fd.FD_KERNEL_AUTO, fd.FD_KERNEL_SIMT):
        check(fd.prefill(q, cache.k, cache.v, ints(lens), kernel=kernel, **cache.kw()), ref, bound)
    if page:
        rope = rope_table(L + n, d).cuda()
        to = Cache(rng, B, L, Hkv, d, page, int8, filled=False)
        plain = Cache(rng, B, L, Hkv, d, page, int8, filled=False)
        plain.table = to.table
        kn = one.expand(B, n, Hkv, d)
        base = ints([0, 100, 267])
        got = fd.append(kn, kn, to.k, to.v, base, q=q, rope=rope, **to.kw())
        want = fd.append(kn.contiguous(), kn.contiguous(), plain.k, plain.v, base, q=q.contiguous(), rope=rope, **plain.kw())
        assert torch.equal(got, want)
        for a, b in zip((to.k, to.v, to.ks, to.vs), (plain.k, plain.v, plain.ks, plain.vs)):
            if a is not None:
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
