"""The workspaces that the binding keeps per (device, stream): growing one leaves
what others hold of it usable.  On the CPU with a stand-in for the device
memory; on a GPU with two threads on one stream."""
import gc
import threading
import weakref

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd


class StandIn(fd.Workspace):
    """A workspace without device memory that records what becomes of it."""

    def __init__(self, max_segments, max_rows, head_dim, max_ctas, stream=None, device=None):
        self.max_segments, self.max_rows, self.head_dim, self.max_ctas = max_segments, max_rows, head_dim, max_ctas
        self.stream, self.device = stream, device
        self.closed = False
        if type(self).made:
            type(self).made(self)

    made = None

    def close(self):
        self.closed = True


@pytest.fixture
def cache(monkeypatch):
    kept = {}
    monkeypatch.setattr(fd, "Workspace", StandIn)
    monkeypatch.setattr(fd, "_ws_cache", kept)
    monkeypatch.setattr(StandIn, "made", None)
    return kept


def test_a_growth_closes_nothing(cache, monkeypatch):
    first = fd.workspace_for("cuda:0", 7, 10, 4, 128, 100)
    assert fd.workspace_for("cuda:0", 7, 64, 16, 256, 1024) is first
    seen = []
    # while the larger one is being made, another thread finds the smaller one
    monkeypatch.setattr(StandIn, "made", lambda ws: seen.append((cache[(0, 7)], first.closed)))
    second = fd.workspace_for("cuda:0", 7, 5000, 4, 128, 100)
    assert seen == [(first, False)]
    assert cache[(0, 7)] is second and second is not first and not first.closed
    # a captured graph holds no reference, and still replays
    alive = weakref.ref(first)
    seen.clear()
    del first
    gc.collect()
    assert alive() is not None and not alive().closed


def test_a_workspace_that_cannot_be_made_leaves_the_smaller_one(cache, monkeypatch):
    first = fd.workspace_for("cuda:0", 7, 10, 4, 128, 100)

    def fail(ws):
        raise fd.FdError(fd.FD_ERR_CUDA, "fd_workspace_create")

    fdbuild.build()
    monkeypatch.setattr(StandIn, "made", fail)
    with pytest.raises(fd.FdError):
        fd.workspace_for("cuda:0", 7, 5000, 4, 128, 100)
    assert cache[(0, 7)] is first and not first.closed


def test_few_workspaces_pile_up(cache, monkeypatch):
    made = []
    monkeypatch.setattr(StandIn, "made", made.append)
    for n in range(1, 5000):
        ws = fd.workspace_for("cuda:0", 7, n, 1 + n % 64, 256, n)
        assert ws.fits(n, 1 + n % 64, 256, n)
        assert ws.max_segments <= max(64, 2 * n) and ws.max_rows <= fd.FD_MAX_ROWS and ws.max_ctas <= max(1024, 2 * n)
    assert len(made) <= 1 + 7 + 2 + 3          # 64 -> 8192, 16 -> 64, 1024 -> 8192
    assert fd.workspace_for("cuda:0", 8, 1, 1, 256, 1).max_segments == 64   # another stream's own


def test_a_workspace_is_zeroed_on_the_stream_of_its_calls(cache):
    # a call given a stream that is not the current one
    assert fd._stream_handle(fd.workspace_for("cuda:0", 7, 10, 4, 128, 100).stream, torch.device("cuda", 0)) == 7
    assert fd._stream_handle(fd.workspace_for("cuda:0", 7, 5000, 4, 128, 100).stream, torch.device("cuda", 0)) == 7
    assert fd._stream_handle(fd.workspace_for("cuda:0", 0, 10, 4, 128, 100).stream, torch.device("cuda", 0)) == 0


@pytest.mark.gpu
def test_two_threads_on_one_stream_while_the_workspace_grows():
    from fp4_util import bf16, cache as quantised, to_dev
    fdbuild.build()
    rng = np.random.default_rng(84)
    (kd, ksd), (vd, vsd) = (to_dev(*quantised(rng, 2, 2, 3000, 128)) for _ in range(2))
    q = bf16(rng, (2, 3, 8, 128)).cuda()
    lens = torch.tensor([3000, 1234], dtype=torch.int32, device="cuda")
    want = fd.decode_fp4(q, kd, vd, ksd, vsd, lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    errors, counts, steps = [], {"decode": 0, "grow": 0}, 60

    def decode():
        with torch.cuda.stream(side):
            got = [fd.decode_fp4(q, kd, vd, ksd, vsd, lens) for _ in range(steps * 5)]
            side.synchronize()
            counts["decode"] = sum(bool((g == want).all()) for g in got)

    def grow():
        with torch.cuda.stream(side):
            for i in range(steps):
                # one used page at the end of ever larger pools
                P = 100_000 * (i + 1)
                refs = torch.zeros(P, dtype=torch.int32, device="cuda")
                table = torch.tensor([[P - 1, -1]], dtype=torch.int32, device="cuda")
                refs[P - 1] = 1
                _, count = fd.pages_reserve(table, torch.full((1,), 4, dtype=torch.int32, device="cuda"), refs, 4, 1)
                counts["grow"] += table.tolist() == [[P - 1, 0]] and count.item() == 0

    def run(job):
        try:
            job()
        except Exception as e:   # (a thread's own exception ends nothing)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(job,)) for job in (decode, grow)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads) and not errors
    assert counts == {"decode": steps * 5, "grow": steps}


@pytest.mark.gpu
def test_two_threads_share_a_workspace_and_its_scratch():
    # compaction's second launch reads what its first left in the room of the
    # split partials, which the other thread's calls write
    from fp4_util import bf16, cache as quantised, to_dev
    from oracle.pages import Books
    fdbuild.build()
    rng = np.random.default_rng(85)
    (kd, ksd), (vd, vsd) = (to_dev(*quantised(rng, 2, 2, 3000, 128)) for _ in range(2))
    q = bf16(rng, (2, 3, 8, 128)).cuda()
    lens = torch.tensor([3000, 1234], dtype=torch.int32, device="cuda")
    dense = [torch.from_numpy(rng.standard_normal((2, 2, 3000, 128))).to(torch.bfloat16).cuda() for _ in range(2)]
    ws = fd.Workspace(1024, 32, 256, 1024)
    calls = (lambda: fd.decode_fp4(q, kd, vd, ksd, vsd, lens, workspace=ws),
             lambda: fd.decode(q, *dense, lens, n_q=3, workspace=ws))
    want = [call() for call in calls]
    P = 4000
    table = np.full((8, 300), -1)
    used = rng.permutation(P)[:8 * 200]
    table[:, :200] = used.reshape(8, 200)
    refs = np.zeros(P, dtype=np.int64)
    refs[used] = 1
    model = Books(table, np.full(8, 200), refs, 1)
    model.compact()
    after = torch.from_numpy(model.table).cuda()
    books = [torch.from_numpy(x.astype(np.int32)).cuda() for x in (table, refs)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    errors, counts, steps = [], [0, 0], 300

    def decode():
        with torch.cuda.stream(stream):
            got = [(i % 2, calls[i % 2]()) for i in range(2 * steps)]
            stream.synchronize()
            counts[0] = sum(bool((x == want[i]).all()) for i, x in got)

    def compact():
        with torch.cuda.stream(stream):
            tables = []
            for _ in range(steps):
                t, r = (x.clone() for x in books)
                fd.pages_compact(t, r, workspace=ws)
                tables.append(t)
            stream.synchronize()
            counts[1] = sum(bool((t == after).all()) for t in tables)

    def run(job):
        try:
            job()
        except Exception as e:   # (a thread's own exception ends nothing)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(job,)) for job in (decode, compact)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads) and not errors
    assert counts == [2 * steps, steps]


@pytest.mark.gpu
def test_a_workspace_that_does_not_fit_the_device_fails_no_later_call():
    from fp4_util import bf16, cache as quantised, to_dev
    fdbuild.build()
    rng = np.random.default_rng(86)
    (kd, ksd), (vd, vsd) = (to_dev(*quantised(rng, 1, 2, 300, 128)) for _ in range(2))
    q, lens = bf16(rng, (1, 1, 8, 128)).cuda(), torch.tensor([300], dtype=torch.int32, device="cuda")
    want = fd.decode_fp4(q, kd, vd, ksd, vsd, lens)
    with pytest.raises(fd.FdError) as e:
        fd.Workspace(1 << 31, 64, 256, 1 << 30)          # some 200 TB
    assert e.value.code == fd.FD_ERR_CUDA
    assert torch.equal(fd.decode_fp4(q, kd, vd, ksd, vsd, lens), want)
