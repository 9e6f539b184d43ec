"""GPU tests of fd_prefill over tables with entries that name no page, by every way
that K and V come: nobody sees their positions."""
import math

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from serve_util import Cache, check, ints, randn

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def attend_but(q, cache, lens, new, causal, scale, gone):
    """serve_util.attend with positions gone[b] (a list) that nobody sees, and its bound
    (the derivation stands there)."""
    B, n, Hq, d = q.shape
    out = torch.zeros(q.shape, dtype=F64, device=q.device)
    bound = torch.zeros_like(out)
    g = Hq // cache.Hkv
    for b in range(B):
        L, t = lens[b], new[b]
        x = q[b, :t].to(F64).view(t, cache.Hkv, g, d)
        k, v = cache.rows(0, b, L), cache.rows(1, b, L)
        s = torch.einsum("ihgd,jhd->hgij", x, k) * scale
        size = torch.einsum("ihgd,jhd->hgij", x.abs(), k.abs()) * abs(scale)
        i, j = torch.arange(t, device=q.device).view(t, 1), torch.arange(L, device=q.device)
        seen = j <= L - t + i if causal else (j >= 0).expand(t, L).clone()
        seen[:, gone[b]] = False
        s = s.masked_fill(~seen, -math.inf)
        size = torch.where(seen, size, 0.0).amax(-1)
        p = torch.softmax(s, -1).nan_to_num(0.0)
        o = torch.einsum("hgij,jhd->ihgd", p, v)
        w = torch.einsum("hgij,jhd->ihgd", p, v.abs())
        e = 2.0 ** -8 + 2.0 ** -22 + (264 + 4 + 64) * 2.0 ** -23 * size.permute(2, 0, 1).unsqueeze(-1) + (L / 8 + 64) * 2.0 ** -23
        out[b, :t] = o.reshape(t, Hq, d)
        bound[b, :t] = (2.0 ** -8 * o.abs() * (1 + 1e-3) + e * (w + o.abs()) + 1e-30).reshape(t, Hq, d)
    return out, bound


# boxes of a page and of half of one, gathers, cp.async; codes widened; one tile and two
FORMS = [(128, 64, False, 8), (128, 128, False, 8), (128, 256, False, 8), (128, 64, False, 2), (128, 16, False, 8), (128, 20, False, 2),
         (256, 64, False, 4), (256, 16, False, 4), (128, 16, True, 8), (128, 24, True, 8), (128, 64, True, 8), (128, 64, True, 2),
         (128, 4, True, 8), (256, 16, True, 4), (256, 24, True, 4), (256, 64, True, 4), (256, 128, True, 4)]
# positions whose pages go: a whole block of 128 and more, some of one, the last and partial
# block, everything, and pages that the chunk's own rows lie on
HOLES = ["block", "pages", "tail", "all", "chunk"]


@pytest.mark.parametrize("kernel", [fd.FD_KERNEL_SIMT, fd.FD_KERNEL_AUTO])
@pytest.mark.parametrize("holes", HOLES)
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_pages_that_are_not_there(form, holes, kernel):
    d, page, int8, Hq = form
    rng = np.random.default_rng(page + d)
    B, n, Hkv = 2, 90, 2
    lens, new = [1000, 517], [90, 77]
    cache = Cache(rng, B, 1000, Hkv, d, page, int8)
    q = randn(rng, (B, n, Hkv * Hq // 2, d)).to(torch.bfloat16).cuda()
    spans = {"block": [(256, 400), (0, 140)], "pages": [(130, 131), (300, 301), (511, 515)], "tail": [(990, 1000), (512, 517)],
             "all": [(0, 1000)], "chunk": [(930, 960), (460, 470)]}[holes]
    # every position on the pages of those
    gone = [sorted({p for lo, hi in spans for j in range(lo // page, (hi - 1) // page + 1) for p in range(j * page, (j + 1) * page)
                    if p < lens[b]}) for b in range(B)]
    for causal in (True, False):
        ref, bound = attend_but(q, cache, lens, new, causal, d ** -0.5, gone)
        kept = cache.table.clone()
        for b in range(B):
            for j in {p // page for p in gone[b]}:
                cache.table[b, j] = (-1, cache.k.shape[0], -(1 << 31), (1 << 31) - 1)[j % 4]
        ws = fd.Workspace(4096, 16, 256, 1024)
        for num_ctas in (0, 1, 5):
            ws.reset()
            out = torch.zeros_like(q)
            fd.prefill(q, cache.k, cache.v, ints(lens), new_lengths=ints(new), causal=causal, out=out, kernel=kernel,
                       num_ctas=num_ctas, workspace=ws, **cache.kw())
            assert ws.device_status() == fd.FD_DEV_BAD_INDEX
            check(out, ref, bound, "%s, %s blocks" % (causal, num_ctas))
            if holes == "all":
                assert (out == 0).all()
        ws.close()
        cache.table = kept
