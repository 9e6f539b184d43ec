"""GPU tests of host threads that share a stream and a workspace: what one call's first
launch leaves in the workspace for its second is not overwritten between them."""
import threading

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from serve_util import Cache, attend, check, ints, randn
from test_beam_gpu import expect

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def test_prefill_beside_beam_selection():
    rng = np.random.default_rng(121)
    cache = Cache(rng, 1, 2000, 2, 128)
    q = randn(rng, (1, 16, 8, 128)).to(torch.bfloat16).cuda()
    ref, bound = attend(q, cache, [2000], [16], True, 128 ** -0.5)
    # (its scratch covers what the first blocks of prefill leave)
    B, n = 512, 64
    logits, scores = randn(rng, (B, 4, 500)).cuda(), randn(rng, (B, 4)).cuda()
    want = expect(logits, scores, n)
    lens, ws = ints([2000]), fd.Workspace(4096, 16, 256, 1024)
    rounds, errors, others = 2500, [], 4
    outs = [torch.zeros_like(q) for _ in range(rounds)]
    best = [[(torch.zeros(B, n, device="cuda"), ints(np.zeros((B, n))), ints(np.zeros((B, n)))) for _ in range(20)] for _ in range(others)]
    torch.cuda.synchronize()
    start = threading.Barrier(1 + others)
    done = threading.Event()

    def run(f):
        try:
            start.wait()
            f()
        except Exception as e:   # noqa: BLE001 (a thread's failure is the test's)
            errors.append(e)
        finally:
            done.set()

    def chunks():
        for o in outs:
            fd.prefill(q, cache.k, cache.v, lens, out=o, workspace=ws)

    def beams(mine):
        while not done.is_set():
            for o in mine:
                fd.beam_select(logits, scores, n, out=o, workspace=ws)
    threads = [threading.Thread(target=run, args=(f,)) for f in [chunks] + [lambda m=m: beams(m) for m in best]]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    check(outs[0], ref, bound)
    assert [i for i, o in enumerate(outs) if not torch.equal(o, outs[0])] == []
    tokens = [[x[2] for x in r] for r in want]
    assert all(b[2].tolist() == tokens for mine in best for b in mine)
    assert ws.device_status() == 0
