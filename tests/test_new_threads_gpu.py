"""GPU tests of the first call of a new host thread: the kernel that it takes is the one
that every other call takes."""
import threading

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from serve_util import Cache, ints, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def in_a_thread(f):
    got = []

    def run():
        try:
            got.append(f())
            torch.cuda.synchronize()
        except Exception as e:   # noqa: BLE001 (given to the test)
            got.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    return got[0]


@pytest.mark.parametrize("d,page,int8", [(128, 0, False), (128, 64, False), (128, 16, False), (256, 0, False), (128, 24, True),
                                         (256, 16, True)])
def test_prefill(d, page, int8):
    rng = np.random.default_rng(131)
    cache = Cache(rng, 1, 900, 2, d, page, int8)
    q, lens = randn(rng, (1, 50, 8, d)).to(torch.bfloat16).cuda(), ints([900])
    torch.cuda.synchronize()
    for kernel in (fd.FD_KERNEL_TC, fd.FD_KERNEL_AUTO):
        ws = fd.Workspace(4096, 16, 256, 1024)
        torch.cuda.synchronize()
        got = in_a_thread(lambda: fd.prefill(q, cache.k, cache.v, lens, kernel=kernel, workspace=ws, **cache.kw()))
        assert isinstance(got, torch.Tensor), got
        want = fd.prefill(q, cache.k, cache.v, lens, kernel=fd.FD_KERNEL_TC, workspace=ws, **cache.kw())
        assert torch.equal(got, want)
        # other tensors, other maps
        cache.k, cache.v = cache.k.clone(), cache.v.clone()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("kind", ["dense", "paged", "int8", "append"])
def test_decode(kind, d):
    rng = np.random.default_rng(132)
    for kernel in (fd.FD_KERNEL_TC, fd.FD_KERNEL_AUTO):
        cache = Cache(rng, 2, 900, 2, d, 64 if kind == "paged" else 0, kind == "int8")
        q, lens = randn(rng, (2, 1, 8, d)).to(torch.bfloat16).cuda(), ints([900, 500])
        new = randn(rng, (2, 1, 2, d)).to(torch.bfloat16).cuda()
        ws = fd.Workspace(4096, 64, 256, 1024)

        def call(which):
            kw = dict(kernel=which, workspace=ws)
            if kind == "paged":
                return fd.decode_paged(q, cache.k, cache.v, cache.table, lens, **kw)
            if kind == "int8":
                return fd.decode_int8(q, cache.k, cache.v, cache.ks, cache.vs, lens, **kw)
            if kind == "append":
                return fd.decode_append(q, cache.k, cache.v, new, new, ints([700, 300]), update_lengths=False, **kw)
            return fd.decode(q, cache.k, cache.v, lens, **kw)
        torch.cuda.synchronize()
        got = in_a_thread(lambda: call(kernel))
        assert isinstance(got, torch.Tensor), got
        assert torch.equal(got, call(fd.FD_KERNEL_TC))
