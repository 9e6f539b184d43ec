"""GPU tests of the page bookkeeping (fd_pages_*) against the sequential
model, entry for entry, and a paged 4-bit serving loop end to end."""
import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from fp4_util import bf16, check, decode_bound, scale_of, to_dev
from oracle import fp4
from oracle.pages import Books

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Dev:
    """The same books on the device."""

    def __init__(self, k: Books):
        self.table, self.lengths, self.refs, self.ps = ints(k.table), ints(k.lengths), ints(k.refs), k.ps
        self.ws = fd.Workspace(64, 32, 256, 1024)

    @property
    def books(self):
        return self.table, self.lengths, self.refs, self.ps

    def same(self, k: Books):
        assert self.table.cpu().numpy().tolist() == k.table.tolist()
        assert self.refs.tolist() == k.refs.tolist()
        assert self.lengths.tolist() == k.lengths.tolist()

    def reserve(self, n_new, want):
        B = len(self.lengths)
        pairs = torch.full((B, 2), -7, dtype=torch.int32, device="cuda")
        _, count = fd.pages_reserve(*self.books, n_new if isinstance(n_new, int) else ints(n_new), pairs=pairs, workspace=self.ws)
        if isinstance(want, int):
            assert count.item() == want and (pairs == -7).all()
            assert self.ws.device_status() & fd.FD_DEV_NO_PAGES
        else:
            assert count.item() == len(want)
            assert pairs[:len(want)].tolist() == [list(p) for p in want] and (pairs[len(want):] == -7).all()


def random_books(rng, B, max_pages, pages, ps, share=0.3):
    """Rows of random lengths; some rows are forks of earlier ones."""
    k = Books(np.full((B, max_pages), -1), np.zeros(B), np.zeros(pages), ps)
    order = list(rng.permutation(pages))
    for b in range(B):
        L = int(rng.integers(0, max_pages * ps + 1))
        if b and rng.random() < share:
            k.fork([int(rng.integers(0, b))], [b], [L])
            continue
        need = -(-L // ps)
        if need > len(order):
            L, need = 0, 0
        for j in range(need):
            k.table[b, j] = order.pop()
            k.refs[k.table[b, j]] = 1
        k.lengths[b] = L
    assert k.consistent()
    return k


SIZES = [(1, 1, 2, 1), (3, 4, 20, 4), (9, 7, 60, 5), (40, 33, 1200, 16), (100, 20, 2500, 16), (70, 64, 6000, 8)]


@pytest.mark.parametrize("B,max_pages,pages,ps", SIZES)
@pytest.mark.parametrize("seed", range(3))
def test_random_books(B, max_pages, pages, ps, seed):
    rng = np.random.default_rng(seed * 100 + B)
    k = random_books(rng, B, max_pages, pages, ps)
    d = Dev(k)
    for step in range(6):
        n = int(rng.integers(1, 2 * ps + 1)) if step % 2 else [int(x) for x in rng.integers(-1, 2 * ps + 1, B)]
        d.reserve(n, k.reserve(n))
        d.same(k)
        assert k.consistent()
        n = int(rng.integers(1, B + 1))
        seqs = [int(x) for x in rng.choice(B, n, replace=False)]
        given = [int(x) for x in rng.integers(-1, max_pages * ps + 5, n)]
        k.free(seqs, given)
        fd.pages_free(*d.books, seqs=ints(seqs), lengths=ints(given), workspace=d.ws)
        d.same(k)
        if B > 2:
            perm = [int(x) for x in rng.permutation(B)]
            m = int(rng.integers(1, B // 2 + 1))
            dst, src = perm[:m], [int(x) for x in rng.choice(perm[m:], m)]
            lens = [int(x) for x in rng.integers(0, max_pages * ps + 1, m)] if step % 2 else None
            k.fork(src, dst, lens)
            fd.pages_fork(*d.books, ints(src), ints(dst), None if lens is None else ints(lens), workspace=d.ws)
            d.same(k)
        assert k.consistent()
        pairs, count = fd.pages_compact(d.table, d.refs, workspace=d.ws)
        want = k.compact()
        assert count.item() == len(want) and pairs[:len(want)].tolist() == [list(p) for p in want]
        d.same(k)
        assert k.consistent()


@pytest.mark.parametrize("seed", range(4))
def test_reserve_by_lists(seed):
    rng = np.random.default_rng(seed)
    k = random_books(rng, 50, 12, 900, 8, share=0.6)
    d = Dev(k)
    for _ in range(4):
        n = [int(x) for x in rng.integers(-1, 20, 50)]
        d.reserve(n, k.reserve(n))
        d.same(k)
        assert k.consistent()


def test_all_holders_write_and_the_first_keeps():
    k = Books([[-1] * 3, [4, 1, -1], [4, 1, -1], [4, 1, -1]], [0, 6, 6, 6], [0, 3, 0, 0, 3, 0, 0], 4)
    d = Dev(k)
    d.reserve(1, [(1, 2), (1, 3)])
    assert d.table.tolist() == [[0, -1, -1], [4, 1, -1], [4, 2, -1], [4, 3, -1]]


def test_too_few_pages_change_nothing():
    k = Books([[3, 0, -1, -1], [3, 0, -1, -1], [1, -1, -5, -1]], [7, 7, 2], [2, 1, 0, 2], 4)
    d = Dev(k)
    before = d.table.clone()
    d.reserve([9, 9, 9], k.reserve([9, 9, 9]))
    assert torch.equal(d.table[:2], before[:2]) and d.refs.tolist() == [2, 1, 0, 2]
    d.reserve([1, 0, 0], [(0, 2)])                      # the last page


def test_free_the_same_sequence_twice_and_unknown_ones():
    k = Books([[0, 1, 2, -1], [3, -1, -1, -1]], [11, 2], [1, 1, 1, 1, 0], 4)
    d = Dev(k)
    fd.pages_free(*d.books, seqs=ints([0, 0, 5, -1]), lengths=ints([9, 3, 0, 0]), workspace=d.ws)
    assert d.lengths.tolist() == [3, 2] and d.table.tolist() == [[0, -1, -1, -1], [3, -1, -1, -1]]
    assert d.refs.tolist() == [1, 0, 0, 1, 0] and d.ws.device_status() == fd.FD_DEV_BAD_INDEX
    fd.pages_free(*d.books, workspace=d.ws)
    assert d.lengths.tolist() == [0, 0] and (d.table == -1).all() and not d.refs.any()


def test_fork_ambiguous_entries_are_skipped_and_flagged():
    k = Books([[0, 1], [2, -1], [-1, -1], [-1, -1]], [6, 3, 0, 0], [1, 1, 1, 0], 4)
    d = Dev(k)
    src, dst = [0, 1, 0, 1, 9], [1, 2, 2, 1, 3]     # 1 is a source; 2 twice; 1 onto itself; no sequence 9
    k.fork(src, dst)
    fd.pages_fork(*d.books, ints(src), ints(dst), workspace=d.ws)
    d.same(k)
    assert k.table[2].tolist() == [2, -1] and d.ws.device_status() == fd.FD_DEV_BAD_INDEX


def test_entries_that_name_no_page():
    k = Books([[9, 0], [-3, -1]], [5, 0], [1, 0, 0], 4)
    d = Dev(k)
    d.reserve(4, [])                                # row 0 writes page 1 alone; row 1's bad entry gets page 1
    assert d.table.tolist() == [[9, 0], [1, -1]]
    fd.pages_compact(d.table, d.refs, workspace=d.ws)
    # (5 + 4 positions are one more than row 0 holds)
    assert d.table.tolist() == [[-1, 0], [1, -1]]
    assert d.ws.device_status() == fd.FD_DEV_BAD_INDEX | fd.FD_DEV_BAD_LENGTH


@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16, torch.float32])
def test_copy(dtype):
    gen = torch.Generator().manual_seed(1)
    shapes = [(12, 2, 5, 64), (12, 3), (12,), (12, 1, 700, 8), (12, 3, 7, 1)]
    host = [torch.randint(0, 200, s, generator=gen).to(dtype) for s in shapes]
    dev = [t.cuda() for t in host]
    wide = torch.zeros(12, 40, dtype=dtype, device="cuda")
    major = torch.randint(0, 200, (12, 5, 2, 64), generator=gen).to(dtype)
    dev += [wide[:, 3:20], major.cuda().transpose(1, 2)]
    host += [wide.cpu()[:, 3:20], major.transpose(1, 2)]
    dev[5].copy_(torch.arange(12 * 17).view(12, 17) % 200)
    host[5] = dev[5].cpu().clone()
    pairs = ints([[3, 0], [4, 11], [3, 7], [2, 30], [5, 6]])
    ws = fd.Workspace(1, 1, 128, 1)
    fd.pages_copy(dev, pairs, ints([4]), workspace=ws)     # the fourth names no page, the fifth is past the count
    for h, t in zip(host, dev):
        h = h.clone()
        h[0], h[11], h[7] = h[3], h[4], h[3]
        assert torch.equal(h, t.cpu())
    assert not wide[:, :3].any() and not wide[:, 20:].any() and ws.device_status() == fd.FD_DEV_BAD_INDEX
    before = [t.cpu().clone() for t in dev]
    for c in (0, -3):
        fd.pages_copy(dev, pairs, ints([c]), workspace=ws)
    assert all(torch.equal(a, t.cpu()) for a, t in zip(before, dev))
    fd.pages_copy(dev, pairs[:1], ints([99]), workspace=ws)   # never past the list


def test_workspace_too_small_is_refused():
    k = Books([[0, -1]], [3], [1] + [0] * 4999, 4)
    d = Dev(k)
    small = fd.Workspace(1, 1, 1, 1)
    for call in (lambda: fd.pages_reserve(*d.books, 1, workspace=small), lambda: fd.pages_compact(d.table, d.refs, workspace=small)):
        with pytest.raises(fd.FdError) as e:
            call()
        assert e.value.code == fd.FD_ERR_WORKSPACE


def test_default_workspace_grows_with_the_pool():
    P = 3_000_000
    table, lengths, refs = ints([[P - 1, -1]]), ints([4]), torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[P - 1] = 1
    _, count = fd.pages_reserve(table, lengths, refs, 4, 1)
    assert table.tolist() == [[P - 1, 0]] and count.item() == 0
    pairs, count = fd.pages_compact(table, refs)
    assert table.tolist() == [[1, 0]] and count.item() == 1 and pairs[0].tolist() == [P - 1, 1]


# ------------------------------------------------ a paged 4-bit serving loop
@pytest.mark.parametrize("d", [128, 256])
def test_serving_loop(d):
    """Prompts are reserved and appended, forked, decoded token by token with
    copy on write, rolled back, freed and compacted; every step's attention is
    compared with an oracle that keeps each sequence's rows apart."""
    rng = np.random.default_rng(d)
    B, Hkv, Hq, ps, mp, P, steps = 5, 2, 8, 8, 12, 48, 5
    zero = np.zeros((P, Hkv, ps, d // 2), np.uint8), np.zeros((P, Hkv, ps, d // 16), np.uint8)
    (kd, ksd), (vd, vsd) = to_dev(*zero), to_dev(*zero)
    pools = fd.PagePools([kd, vd, ksd, vsd])
    books = Books(np.full((B, mp), -1), np.zeros(B), np.zeros(P), ps)
    dev = Dev(books)
    rows = [[np.zeros((0, Hkv, d)), np.zeros((0, Hkv, d))] for _ in range(B)]

    def step(n, new):
        pairs, count = fd.pages_reserve(*dev.books, ints(new), workspace=dev.ws)
        fd.pages_copy(pools, pairs, count, workspace=dev.ws)
        got = books.reserve(new)
        assert count.item() == len(got)
        kn, vn = bf16(rng, (B, n, Hkv, d)), bf16(rng, (B, n, Hkv, d))
        fd.append_fp4(kn.cuda(), vn.cuda(), kd, vd, ksd, vsd, dev.lengths, new_lengths=ints(new), lengths_out=dev.lengths,
                      block_table=dev.table, workspace=dev.ws)
        for b in range(B):
            for t, x in enumerate((kn, vn)):
                rows[b][t] = np.concatenate([rows[b][t], fp4.values(*fp4.quantise(x[b, :new[b]].double().numpy()))])
        books.lengths += np.array(new, dtype=np.int32)
        dev.same(books)

    def attend(n_q):
        q = bf16(rng, (B, n_q, Hq, d))
        got = fd.decode_fp4(q.cuda(), kd, vd, ksd, vsd, dev.lengths, causal=True, block_table=dev.table, workspace=dev.ws)
        top = max(len(r[0]) for r in rows)
        flat = [np.zeros((B, Hkv, top, d)) for _ in range(2)]
        for b in range(B):
            for t in range(2):
                flat[t][b, :, :len(rows[b][t])] = rows[b][t].transpose(1, 0, 2)
        (k, ks), (v, vs) = (fp4.quantise(x) for x in flat)      # representable: exact
        want, weight, size = fp4.decode(q.double().numpy(), k, v, ks, vs, [len(r[0]) for r in rows], True, scale_of(d))
        check(got, want, decode_bound(want, weight, size, top, np.abs(flat[1]).max(), torch.bfloat16), "serving")

    step(30, [30, 13, 0, 0, 0])
    attend(2)
    books.fork([0, 0, 1], [2, 3, 4], [30, 21, 13])
    fd.pages_fork(*dev.books, ints([0, 0, 1]), ints([2, 3, 4]), ints([30, 21, 13]), workspace=dev.ws)
    for s, t, L in ((0, 2, 30), (0, 3, 21), (1, 4, 13)):
        rows[t] = [x[:L] for x in rows[s]]
    dev.same(books)
    attend(1)
    for i in range(steps):
        step(3, [3, 1, 3, 2, 0 if i % 2 else 1])
        attend(3)
        drop = [int(x) - 1 for x in books.lengths]           # one draft refused
        books.free(None, drop)
        fd.pages_free(*dev.books, lengths=ints(drop), workspace=dev.ws)
        for b in range(B):
            rows[b] = [x[:drop[b]] for x in rows[b]]
        dev.same(books)
        attend(1)
    books.free([1, 3])
    fd.pages_free(*dev.books, seqs=ints([1, 3]), workspace=dev.ws)
    for b in (1, 3):
        rows[b] = [x[:0] for x in rows[b]]
    pairs, count = fd.pages_compact(dev.table, dev.refs, workspace=dev.ws)
    fd.pages_copy(pools, pairs, count, workspace=dev.ws)
    assert count.item() == len(books.compact())
    dev.same(books)
    attend(2)
    step(9, [0, 9, 2, 9, 1])
    attend(6)
    assert books.consistent() and dev.ws.device_status() == 0


@pytest.mark.parametrize("B,max_pages,pages,ps", [(300, 40, 50000, 8), (5000, 3, 9000, 4), (9000, 2, 40000, 3)])
def test_large_books(B, max_pages, pages, ps):
    """Pools large enough for the cluster, and more sequences than are looked
    at together; shared rows, rows that are full, and a request too large."""
    rng = np.random.default_rng(B)
    k = random_books(rng, B, max_pages, pages, ps, share=0.2)
    d = Dev(k)
    for n in ([int(x) for x in rng.integers(-1, ps + 2, B)], 1):
        d.reserve(n, k.reserve(n))
        d.same(k)
    assert k.consistent()
    gone = [int(x) for x in rng.choice(B, B // 2, replace=False)]
    k.free(gone)
    fd.pages_free(*d.books, seqs=ints(gone), workspace=d.ws)
    d.same(k)
    pairs, count = fd.pages_compact(d.table, d.refs, workspace=d.ws)
    want = k.compact()
    assert count.item() == len(want) and pairs[:len(want)].tolist() == [list(p) for p in want]
    d.same(k)
    assert k.consistent()
