"""GPU tests of fd_prefill against attention in 64 bits."""
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


KERNELS = [fd.FD_KERNEL_SIMT, fd.FD_KERNEL_AUTO]
CASES = [
    # B, n, Hq, Hkv, d, page, int8, causal, token_major, lens, new
    (1, 1, 8, 2, 128, 0, False, True, False, [1], [1]),
    (1, 7, 8, 2, 128, 0, False, True, False, [7], [7]),
    (2, 37, 8, 2, 128, 0, False, True, False, [1000, 37], [37, 20]),
    (3, 64, 4, 4, 128, 0, False, False, True, [129, 64, 1], [64, 1, 64]),
    (3, 200, 16, 2, 128, 16, False, True, True, [200, 517, 300], [200, 17, 199]),
    (2, 130, 10, 2, 128, 64, False, True, False, [640, 131], [130, 130]),
    (2, 130, 7, 1, 128, 20, False, False, False, [333, 500], [130, 77]),
    (1, 300, 64, 1, 128, 128, False, True, False, [512], [300]),
    (1, 5, 128, 1, 128, 256, False, True, False, [700], [5]),
    (2, 90, 9, 3, 128, 1, False, True, False, [91, 260], [90, 90]),
    (2, 50, 16, 4, 256, 0, False, True, False, [50, 400], [50, 44]),
    (2, 260, 8, 2, 256, 48, False, True, True, [260, 700], [259, 128]),
    (1, 129, 5, 1, 256, 16, False, False, False, [1025], [129]),
    (2, 64, 12, 2, 256, 128, False, True, False, [1024, 65], [64, 65]),
    (2, 40, 8, 2, 128, 0, True, True, False, [40, 300], [40, 33]),
    (2, 140, 16, 4, 128, 64, True, True, True, [640, 141], [140, 139]),
    (2, 70, 6, 2, 128, 24, True, False, False, [333, 70], [70, 1]),
    (2, 70, 8, 2, 256, 16, True, True, False, [333, 500], [70, 64]),
    (1, 200, 20, 4, 256, 0, True, True, True, [900], [200]),
    # rows that see nothing: fewer positions than new rows, none at all, no new rows
    (4, 40, 8, 2, 128, 16, False, True, False, [10, 0, 33, 1], [40, 40, 0, 2]),
    (4, 40, 8, 2, 256, 0, True, True, False, [10, 0, 33, 1], [40, 40, 0, 2]),
    # many sequences
    (40, 3, 4, 2, 128, 16, False, True, False, [17 + 13 * b for b in range(40)], [1 + b % 3 for b in range(40)]),
]


def run(case, kernel, num_ctas=0, seed=41, scale=None):
    B, n, Hq, Hkv, d, page, int8, causal, tm, lens, new = case
    rng = np.random.default_rng(seed)
    cache = Cache(rng, B, max(max(lens), 1), Hkv, d, page, int8, tm)
    q = randn(rng, (B, n, Hq, d)).to(torch.bfloat16).cuda()
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    new = [min(x, n) for x in new]
    ref, bound = attend(q, cache, lens, new, causal, scale)
    cache.spoil(lens)
    out = torch.full((B, n, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        q[b, new[b]:] = float("nan")
    ws = fd.Workspace(4096, 16, 256, 1024)
    got = fd.prefill(q, cache.k, cache.v, ints(lens), new_lengths=ints(new), causal=causal, scale=scale, out=out, kernel=kernel,
                     num_ctas=num_ctas, workspace=ws, **cache.kw())
    torch.cuda.synchronize()
    assert got is out and ws.device_status() == 0, ws.diagnostics()
    for b in range(B):
        assert (out[b, new[b]:] == 7).all()              # padding is left as it was
        out[b, new[b]:] = 0
    check(out, ref, bound, str(case))
    for b in range(B):
        if causal and lens[b] < new[b]:
            assert (out[b, :new[b] - lens[b]] == 0).all()
    ws.close()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_prefill(case, kernel):
    run(case, kernel)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_other_factors(kernel, scale):
    run((2, 150, 8, 2, 128, 16, False, True, False, [150, 400], [150, 140]), kernel, scale=scale)
    run((1, 70, 8, 2, 256, 16, True, True, False, [300], [70]), kernel, scale=scale)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d,int8", [(128, False), (256, False), (128, True), (256, True)])
def test_without_lists_and_defaults(kernel, d, int8):
    # every row new, default scale, an output that the call makes
    rng = np.random.default_rng(43)
    cache = Cache(rng, 2, 200, 2, d, 32, int8)
    q = randn(rng, (2, 65, 8, d)).to(torch.bfloat16).cuda()
    ref, bound = attend(q, cache, [150, 65], [65, 65], True, d ** -0.5)
    check(fd.prefill(q, cache.k, cache.v, ints([150, 65]), kernel=kernel, **cache.kw()), ref, bound)


@pytest.mark.parametrize("kernel", KERNELS)
def test_strided_queries_and_outputs(kernel):
    rng = np.random.default_rng(44)
    B, n, Hq, Hkv, d = 2, 100, 8, 2, 128
    cache = Cache(rng, B, 300, Hkv, d, 0)
    wide = randn(rng, (B, n + 3, Hq + 4, d + 8)).to(torch.bfloat16).cuda()
    q = wide[:, 1:n + 1, 2:Hq + 2, 8:]
    room = torch.full((n, B, Hq, d + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    out = room[..., 8:d + 8].transpose(0, 1)
    ref, bound = attend(q, cache, [300, 180], [n, n], True, 0.1)
    fd.prefill(q, cache.k, cache.v, ints([300, 180]), scale=0.1, out=out, kernel=kernel)
    check(out, ref, bound)
    assert (room[..., :8] == 5).all() and (room[..., d + 8:] == 5).all()


@pytest.mark.parametrize("layout", ["odd strides", "K and V apart"])
@pytest.mark.parametrize("page", [0, 16])
def test_caches_of_uncommon_strides(layout, page):
    rng = np.random.default_rng(45)
    B, n, Hq, Hkv, d = 2, 70, 8, 2, 128
    cache = Cache(rng, B, 160, Hkv, d, page)
    lead, _, rows, _ = cache.k.shape

    def spread(t, pad):
        x = torch.full((lead, Hkv * rows * (d + pad) + 24), math.nan, dtype=t.dtype, device="cuda")
        y = x.as_strided(t.shape, (x.stride(0), rows * (d + pad) + 8, d + pad, 1))
        y.copy_(t)
        return y
    cache.k = spread(cache.k, 8)
    cache.v = spread(cache.v, 8) if layout == "odd strides" else cache.v.clone()
    q = randn(rng, (B, n, Hq, d)).to(torch.bfloat16).cuda()
    ref, bound = attend(q, cache, [160, 91], [n, n], True, d ** -0.5)
    check(fd.prefill(q, cache.k, cache.v, ints([160, 91]), **cache.kw()), ref, bound)


@pytest.mark.parametrize("kernel", KERNELS)
def test_bad_lengths_and_tables(kernel):
    rng = np.random.default_rng(46)
    B, n, Hq, Hkv, d, page = 4, 30, 4, 2, 128, 16
    cache = Cache(rng, B, 160, Hkv, d, page)
    q = randn(rng, (B, n, Hq, d)).to(torch.bfloat16).cuda()
    good = Cache.__new__(Cache)
    good.__dict__.update(cache.__dict__, table=cache.table.clone())
    lens, new = [-3, 1000, 100, 160], [30, 99, -2, 30]
    ws = fd.Workspace(4096, 16, 256, 1024)
    out = torch.full((B, n, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    fd.prefill(q, cache.k, cache.v, ints(lens), new_lengths=ints(new), out=out, kernel=kernel, workspace=ws, **cache.kw())
    assert ws.device_status() == fd.FD_DEV_BAD_LENGTH
    lens, new = [0, 160, 100, 160], [30, 30, 0, 30]
    ref, bound = attend(q, cache, lens, new, True, d ** -0.5)
    assert (out[2] == 7).all()
    out[2] = 0
    check(out, ref, bound)
    # an entry that names no page: nobody sees its positions
    ws.reset()
    cache.table[1, 3] = -1
    cache.table[3, 0] = cache.k.shape[0]
    got = fd.prefill(q, cache.k, cache.v, ints(lens), new_lengths=ints([30, 30, 30, 30]), kernel=kernel, workspace=ws, **cache.kw())
    assert ws.device_status() == fd.FD_DEV_BAD_INDEX
    for b, gone in ((1, range(48, 64)), (3, range(16))):
        x = q[b].double().view(n, Hkv, Hq // Hkv, d)
        safe = cache.table.clone()
        safe[b] = safe[b].clamp(0, cache.k.shape[0] - 1)
        pos = torch.arange(160, device="cuda")
        k, v = (t[safe[b].long()[pos // page], :, pos % page].double() for t in (cache.k, cache.v))
        s = torch.einsum("ihgd,jhd->hgij", x, k) * d ** -0.5
        hidden = pos > 130 + torch.arange(n, device="cuda").view(n, 1)
        hidden[:, list(gone)] = True
        p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
        want = torch.einsum("hgij,jhd->ihgd", p, v).reshape(n, Hq, d)
        assert ((got[b].double() - want).abs() <= 0.02 * v.abs().amax()).all()
    check(got[2], *(x[2] for x in attend(q, good, [0, 160, 100, 160], [30] * 4, True, d ** -0.5)))


def test_int8_nan_scales_reach_the_rows_that_see_them():
    rng = np.random.default_rng(47)
    for kernel in KERNELS:
        for which in ("ks", "vs"):
            cache = Cache(rng, 1, 200, 2, 128, 16, True)
            lead, row = cache.at(0, 200)
            getattr(cache, which)[lead[190], 1, row[190]] = math.nan
            q = randn(rng, (1, 40, 4, 128)).to(torch.bfloat16).cuda()
            out = fd.prefill(q, cache.k, cache.v, ints([200]), kernel=kernel, **cache.kw())[0]
            assert torch.isfinite(out[:30]).all() and torch.isfinite(out[:, :2]).all()
            assert out[30:, 2:].isnan().all()


def test_same_result_every_time_and_on_other_streams():
    rng = np.random.default_rng(48)
    cache = Cache(rng, 3, 5000, 2, 128, 16)
    q = randn(rng, (3, 50, 8, 128)).to(torch.bfloat16).cuda()
    lens, new = ints([5000, 1200, 77]), ints([50, 13, 50])
    out = torch.zeros_like(q)
    first = fd.prefill(q, cache.k, cache.v, lens, new_lengths=new, out=out, **cache.kw()).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.zeros_like(q) for _ in range(12)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        with torch.cuda.stream(streams[i % 3]):
            fd.prefill(q, cache.k, cache.v, lens, new_lengths=new, out=o, **cache.kw())
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


def test_captured_and_replayed_with_other_lengths():
    rng = np.random.default_rng(49)
    cache = Cache(rng, 2, 3000, 2, 128, 64)
    q = randn(rng, (2, 90, 8, 128)).to(torch.bfloat16).cuda()
    lens, new, out = ints([90, 90]), ints([90, 90]), torch.zeros_like(q)
    stream = torch.cuda.Stream()
    ws = fd.Workspace(4096, 16, 256, 1024, stream=stream)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        fd.prefill(q, cache.k, cache.v, lens, new_lengths=new, out=out, workspace=ws, **cache.kw())
    for L, t in (([90, 90], [90, 90]), ([3000, 400], [90, 1]), ([2111, 3000], [17, 90]), ([5, 0], [90, 90])):
        lens.copy_(ints(L))
        new.copy_(ints(t))
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(out, *attend(q, cache, L, t, True, 128 ** -0.5), what=str(L))
    assert ws.device_status() == 0
