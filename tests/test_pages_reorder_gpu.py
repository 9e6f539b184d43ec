"""GPU tests of fd_pages_reorder against the sequential model, entry for entry."""
import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from oracle.pages import Books
from test_pages_gpu import Dev, ints, random_books

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def both(k, src, status=0):
    dev = Dev(k)
    k.reorder(src)
    fd.pages_reorder(*dev.books, ints(src), workspace=dev.ws)
    dev.same(k)
    assert dev.ws.device_status() == status
    return dev


@pytest.mark.parametrize("B,max_pages,ps", [(1, 1, 1), (2, 3, 16), (4, 128, 16), (8, 33, 1), (50, 31, 20), (300, 65, 8), (2000, 5, 4)])
def test_random_books(B, max_pages, ps):
    rng = np.random.default_rng(B)
    for trial in range(3):
        k = random_books(rng, B, max_pages, B * max_pages + 5, ps)
        assert k.consistent()
        src = rng.integers(0, B, B) if trial else rng.permutation(B)
        if trial == 2:
            src = np.where(rng.random(B) < 0.3, -1, src)     # rows that end
        both(k, src)
        assert k.consistent()


def test_swaps_and_copies_of_one_row():
    for src in ([1, 0, 3, 2], [0, 0, 0, 0], [3, 3, 3, 3], [1, 2, 3, 0], [0, 1, 2, 3], [-1, -1, 2, -7]):
        k = random_books(np.random.default_rng(3), 4, 6, 30, 16)
        both(k, src)


def test_pages_reserved_ahead_stay_with_rows_that_stay():
    k = Books([[2, 5, 7], [1, -1, -1], [0, 3, -1]], [17, 9, 32], [1, 1, 1, 1, 0, 1, 0, 1], 16)
    k.table[0, 2] = 7                                         # past the length of row 0
    dev = both(k, [0, 0, 1])
    assert dev.table.tolist() == [[2, 5, 7], [2, 5, -1], [1, -1, -1]] and dev.lengths.tolist() == [17, 17, 9]
    assert k.consistent()


def test_bad_sources_lengths_and_entries():
    k = Books([[2, 5], [1, -1], [0, 3]], [17, 9, 32], [1, 1, 1, 1, 0, 1], 16)
    both(k, [3, 0, 1], fd.FD_DEV_BAD_INDEX)                   # a row that does not exist
    k = Books([[2, 5], [1, -1], [0, 3]], [99, 9, -2], [1, 1, 1, 1, 0, 1], 16)
    dev = Dev(k)
    fd.pages_reorder(*dev.books, ints([2, 0, 0]), workspace=dev.ws)
    assert dev.ws.device_status() == fd.FD_DEV_BAD_LENGTH
    assert dev.table.tolist() == [[-1, -1], [2, 5], [2, 5]] and dev.lengths.tolist() == [0, 32, 32]
    assert dev.refs.tolist() == [0, 0, 2, 0, 0, 2]
    k = Books([[2, -1], [9, 1]], [20, 30], [0, 1, 1], 16)     # entries that name no page
    dev = Dev(k)
    fd.pages_reorder(*dev.books, ints([1, 0]), workspace=dev.ws)
    assert dev.ws.device_status() == fd.FD_DEV_BAD_INDEX
    assert dev.table.tolist() == [[-1, 1], [2, -1]] and dev.refs.tolist() == [0, 1, 1]


def test_many_rows():
    B = 40000
    k = Books(np.full((B, 2), -1), np.zeros(B), np.zeros(2 * B), 4)
    k.table[:, 0] = np.arange(B)
    k.lengths[:] = 1 + np.arange(B) % 4
    k.refs[:B] = 1
    dev = Dev(k)
    src = np.random.default_rng(4).integers(0, B, B)
    fd.pages_reorder(*dev.books, ints(src), workspace=dev.ws)
    assert (dev.table[:, 0].cpu().numpy() == src).all() and (dev.lengths.cpu().numpy() == 1 + src % 4).all()
    assert (dev.refs.cpu().numpy()[:B] == np.bincount(src, minlength=B)).all()
    assert dev.ws.device_status() == 0


def test_replayed():
    k = random_books(np.random.default_rng(6), 12, 40, 500, 16)
    dev, src = Dev(k), ints(np.zeros(12))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        fd.pages_reorder(*dev.books, src, workspace=dev.ws)
    rng = np.random.default_rng(7)
    for _ in range(5):
        s = rng.integers(0, 12, 12) if rng.random() < 0.5 else rng.permutation(12)
        src.copy_(ints(s))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        k.reorder(s)
        dev.same(k)
