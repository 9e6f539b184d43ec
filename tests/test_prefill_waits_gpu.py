"""fd_prefill with a wait limit too short for its own loads: the launch ends in time
with FD_DEV_INTERNAL, and the next call over the same workspace is right."""
import ctypes
import time

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


def call(q, cache, lens, out, ws, wait_limit_us):
    o = fd.FdOpts()
    o.ws, o.stream = ws.handle, torch.cuda.current_stream().cuda_stream
    o.wait_limit_us = wait_limit_us
    ten = [fd.as_fd_tensor(t) if t is not None else None for t in (q, cache.k, cache.v, cache.ks, cache.vs, out)]
    ref = [None if t is None else ctypes.byref(t) for t in ten]
    table = cache.table
    code = fd.lib().fd_prefill(*ref[:5], None if table is None else table.data_ptr(), 0 if table is None else table.shape[1],
                               lens.data_ptr(), None, 1, q.shape[-1] ** -0.5, ref[5], ctypes.byref(o))
    assert code == 0


# each way that K and V come, one tile and two
@pytest.mark.parametrize("d,page,int8,Hq", [(128, 0, False, 2), (128, 0, False, 8), (128, 64, False, 8), (256, 0, False, 4),
                                            (128, 16, False, 2), (128, 16, False, 8), (256, 16, False, 4),
                                            (128, 64, True, 8), (128, 0, True, 2), (256, 16, True, 4)])
def test_a_wait_that_runs_out(d, page, int8, Hq):
    rng = np.random.default_rng(71)
    B, n, L = 2, 60, 40000
    cache = Cache(rng, B, L, 1, d, page, int8)
    q = randn(rng, (B, n, Hq, d)).to(torch.bfloat16).cuda()
    lens = ints([L, L - 777])
    ref, bound = attend(q, cache, [L, L - 777], [n, n], True, d ** -0.5)
    ws = fd.Workspace(4096, 16, 256, 1024)
    out = torch.zeros_like(q)
    cold = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    call(q, cache, lens, out, ws, 0)                 # (the kernel's code is loaded)
    check(out, ref, bound)
    seen = []
    for _ in range(4):
        cold.add_(1)                                 # K and V leave the caches
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        call(q, cache, lens, out, ws, 1)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 0.5
        seen.append(ws.device_status())
        assert seen[-1] in (0, fd.FD_DEV_INTERNAL)
        if seen[-1] == 0:
            check(out, ref, bound)
        else:
            assert 1 <= ws.diagnostics()[1] <= 12    # the wait that ran out
        ws.reset()
        for _ in range(2):
            out.fill_(7)
            call(q, cache, lens, out, ws, 0)
            torch.cuda.synchronize()
            assert ws.device_status() == 0
            check(out, ref, bound)
    assert fd.FD_DEV_INTERNAL in seen
    ws.close()
