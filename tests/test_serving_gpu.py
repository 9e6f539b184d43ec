"""GPU tests of a beam search over a paged cache as a server runs it: prompts are
appended and attended to in chunks, their pages shared by the beams, and each step
selects, reorders, reserves, copies, appends and attends; eager, and as one graph
that is replayed.  Also prefill calls of every split, from two threads at once, and
on workspaces that are too small."""
import math
import threading

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from oracle.pages import Books
from serve_util import Cache, attend, check, ints, randn, rope_table
from test_beam_gpu import expect
from test_pages_gpu import Dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


class Server:
    """R requests of K beams (rows r*K + k of the books) over one layer's pools, and
    what every row's positions hold, bit for bit, kept on the host."""

    def __init__(self, R, K, Hq, Hkv, d, ps, mp, int8, seed):
        self.rng = np.random.default_rng(seed)
        self.R, self.K, self.Hq, self.Hkv, self.d, self.V, self.end = R, K, Hq, Hkv, d, 5000, 3
        B, P = R * K, R * K * mp
        self.B = B
        # (a Cache to read the pools through the table)
        self.cache = Cache(self.rng, B, mp * ps, Hkv, d, ps, int8, filled=False, spare=0)
        self.books = Books(np.full((B, mp), -1), np.zeros(B), np.zeros(P), ps)
        self.dev = Dev(self.books)
        self.dev.ws = fd.Workspace(4096, 16, 256, 1024)
        self.cache.table = self.dev.table
        c = self.cache
        self.pools = fd.PagePools([c.k, c.v] + ([c.ks, c.vs] if int8 else []))
        self.rows = [[] for _ in range(B)]            # a row's positions: what its pools hold there
        self.rope = rope_table(mp * ps, d).cuda()
        self.scores = torch.full((R, K), -math.inf, device="cuda")
        self.scores[:, 0] = 0
        self.finished = torch.zeros(R, K, dtype=torch.int32, device="cuda")
        # what a step reads and writes
        self.n_new = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.pairs = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
        self.count = torch.zeros(1, dtype=torch.int32, device="cuda")

    def bf16(self, *shape):
        return randn(self.rng, shape).to(torch.bfloat16).cuda()

    def held(self, b, pos):
        lead, row = self.dev.table[b, pos // self.cache.page], pos % self.cache.page
        ts = [self.cache.k, self.cache.v] + ([self.cache.ks, self.cache.vs] if self.cache.int8 else [])
        return [t[int(lead), :, row].clone() for t in ts]

    def launch(self, k, v, q, turned, out):
        """New rows of every sequence (n_new of them), and attention to them."""
        d, c = self.dev, self.cache
        fd.pages_reserve(*d.books, self.n_new, pairs=self.pairs, count=self.count, workspace=d.ws)
        fd.pages_copy(self.pools, self.pairs, self.count, workspace=d.ws)
        fd.append(k, v, c.k, c.v, d.lengths, new_lengths=self.n_new, lengths_out=d.lengths, q=q, q_out=turned, rope=self.rope,
                  workspace=d.ws, **c.kw())
        fd.prefill(turned, c.k, c.v, d.lengths, new_lengths=self.n_new, out=out, workspace=d.ws, **c.kw())

    def checked(self, new, turned, out):
        """The books, the pools under every row and the outputs after `launch`."""
        self.dev.same(self.books)
        assert self.books.consistent() and self.dev.ws.device_status() == 0
        for b in range(self.B):
            L = int(self.books.lengths[b])
            self.rows[b] = self.rows[b][:L - int(new[b])] + [self.held(b, i) for i in range(L - int(new[b]), L)]
            for i, want in enumerate(self.rows[b]):          # (rows before these moved and copied whole)
                if i % 7 == 0 or i + 20 > L:
                    assert all(torch.equal(x, y) for x, y in zip(self.held(b, i), want)), (b, i)
        ref, bound = attend(turned, self.cache, self.books.lengths, new, True, self.d ** -0.5)
        for b in np.flatnonzero(new):
            check(out[b, :new[b]], ref[b, :new[b]], bound[b, :new[b]], "row %d" % b)

    def prompts(self, lens, chunk):
        done = np.zeros(self.R, int)
        while (done < lens).any():
            new = np.zeros(self.B, int)
            new[::self.K] = np.minimum(chunk, lens - done)
            done += new[::self.K]
            self.n_new.copy_(ints(new))
            q = self.bf16(self.B, chunk, self.Hq, self.d)
            k, v = self.bf16(self.B, chunk, self.Hkv, self.d), self.bf16(self.B, chunk, self.Hkv, self.d)
            turned, out = torch.zeros_like(q), torch.zeros_like(q)
            self.launch(k, v, q, turned, out)
            assert self.books.reserve(new) == []
            self.books.lengths += new
            self.checked(new, turned, out)

    def moved(self, src):
        self.books.reorder(src)
        self.rows = [list(self.rows[s]) if s >= 0 else [] for s in src]


def start(int8, d=128):
    s = Server(3, 4, 8, 2, d, 16, 12, int8, 90 + d)
    s.prompts(np.array([61, 16, 150]), 64)
    return s


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [128, 256])
def test_a_beam_search(int8, d):
    s = start(int8, d)
    for step in range(6):
        logits = s.bf16(s.R, s.K, s.V) * 3
        logits[..., s.end] += 8
        scores, beams, tokens = fd.beam_select(logits, s.scores, s.K, finished=s.finished, end_token=s.end, workspace=s.dev.ws)
        want = expect(logits, s.scores, s.K, s.finished, s.end)
        assert beams.tolist() == [[x[1] for x in r] for r in want] and tokens.tolist() == [[x[2] for x in r] for r in want]
        src = beams.flatten().cpu().numpy()
        fd.pages_reorder(*s.dev.books, beams.flatten(), workspace=s.dev.ws)
        s.moved(src)
        s.finished = torch.maximum(s.finished.flatten()[beams.flatten().long()].view(s.R, s.K), (tokens == s.end).int())
        s.scores = scores
        new = 1 - s.finished.flatten().cpu().numpy()          # ended beams append nothing
        s.n_new.copy_(ints(new))
        q, k, v = s.bf16(s.B, 1, s.Hq, d), s.bf16(s.B, 1, s.Hkv, d), s.bf16(s.B, 1, s.Hkv, d)
        turned, out = torch.zeros_like(q), torch.zeros_like(q)
        s.launch(k, v, q, turned, out)
        got = s.books.reserve(new)
        assert s.count.item() == len(got)
        s.books.lengths += new
        s.checked(new, turned, out)
        # the decode call over the same pages answers the same
        c = s.cache
        one = fd.decode_paged(turned, c.k, c.v, c.table, s.dev.lengths, k_scale=c.ks, v_scale=c.vs, workspace=s.dev.ws)
        ref, bound = attend(turned, c, s.books.lengths, new, True, d ** -0.5)
        for b in np.flatnonzero(new):
            # (the decode kernels round a weight, or one times its scale, at most twice)
            check(one[b], ref[b], 2 * bound[b], "decode")
    assert s.finished.any() and len(set(s.books.table[:, 0].tolist())) < s.B      # some ended, pages are shared


@pytest.mark.parametrize("int8", [False, True])
def test_a_step_captured_and_replayed(int8):
    s = start(int8)
    d, B = s.d, s.B
    stream = torch.cuda.Stream()
    logits = torch.zeros(s.R, s.K, s.V, dtype=torch.bfloat16, device="cuda")
    scores, beams = torch.zeros(s.R, s.K, device="cuda"), torch.zeros(s.R, s.K, dtype=torch.int32, device="cuda")
    tokens = torch.zeros_like(beams)
    q, k, v = s.bf16(B, 1, s.Hq, d), s.bf16(B, 1, s.Hkv, d), s.bf16(B, 1, s.Hkv, d)
    turned, out = torch.zeros_like(q), torch.zeros_like(q)
    s.n_new.fill_(1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        fd.beam_select(logits, s.scores, s.K, out=(scores, beams, tokens), workspace=s.dev.ws)
        fd.pages_reorder(*s.dev.books, beams.view(-1), workspace=s.dev.ws)
        s.launch(k, v, q, turned, out)
        s.scores.copy_(scores)
    for step in range(5):
        for t, x in ((q, s.bf16(*q.shape)), (k, s.bf16(*k.shape)), (v, s.bf16(*v.shape)), (logits, s.bf16(*logits.shape) * 3)):
            t.copy_(x)
        want = expect(logits, s.scores, s.K)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert beams.tolist() == [[x[1] for x in r] for r in want] and tokens.tolist() == [[x[2] for x in r] for r in want]
        s.moved(beams.flatten().cpu().numpy())
        assert s.count.item() == len(s.books.reserve([1] * B))
        s.books.lengths += 1
        s.checked(np.ones(B, int), turned, out)


# ------------------------------------------------------------- prefill alone
@pytest.mark.parametrize("d,n,int8,page", [(128, 200, False, 0), (128, 200, False, 64), (128, 16, False, 16), (128, 200, True, 16),
                                            (256, 100, False, 0), (256, 100, False, 48), (256, 40, True, 0)])
def test_every_split(d, n, int8, page):
    rng = np.random.default_rng(95)
    lens, new = [700, 1, 255, 0, 1500], [n, 1, min(n, 128), 0, n // 2]
    cache = Cache(rng, 5, 1500, 2, d, page, int8)
    q = randn(rng, (5, n, 6, d)).to(torch.bfloat16).cuda()
    ref, bound = attend(q, cache, lens, new, True, d ** -0.5)
    cache.spoil(lens)
    ws = fd.Workspace(4096, 16, 256, 4096)
    for ctas in (1, 2, 3, 7, 31, 152, 153, 400):
        out = torch.zeros_like(q)
        fd.prefill(q, cache.k, cache.v, ints(lens), new_lengths=ints(new), out=out, num_ctas=ctas, workspace=ws, **cache.kw())
        check(out, ref, bound, "%d shares" % ctas)
    assert ws.device_status() == 0


@pytest.mark.parametrize("page", [0, 64, 16])
def test_long_caches_past_32_bits(page):
    # rows far apart: byte offsets past 2^32 (bf16 elements past 2^31)
    rng = np.random.default_rng(96)
    B, n, Hkv, d, L = 2, 40, 2, 128, 300
    cache = Cache(rng, B, L, Hkv, d, page)
    lead = cache.k.shape[0]
    step = ((1 << 31) // (lead - 1) // 1024 + 1) * 1024
    q = randn(rng, (B, n, 8, d)).to(torch.bfloat16).cuda()
    ref, bound = attend(q, cache, [L, 77], [n, n], True, d ** -0.5)

    def far(t):
        room = torch.empty((lead - 1) * step + t[0].numel(), dtype=torch.bfloat16, device="cuda")
        return room.as_strided(t.shape, (step,) + t.stride()[1:]).copy_(t)
    k, v = far(cache.k), far(cache.v)
    for kernel in (fd.FD_KERNEL_AUTO, fd.FD_KERNEL_SIMT):
        check(fd.prefill(q, k, v, ints([L, 77]), kernel=kernel, **cache.kw()), ref, bound)


def test_workspaces_too_small_are_refused():
    rng = np.random.default_rng(97)
    cache = Cache(rng, 1, 300, 2, 128)
    q = randn(rng, (1, 40, 8, 128)).to(torch.bfloat16).cuda()
    small = fd.Workspace(1, 1, 1, 1)
    logits, scores = torch.zeros(4, 4, 32000, device="cuda"), torch.zeros(4, 4, device="cuda")
    for call in (lambda: fd.prefill(q, cache.k, cache.v, ints([300]), workspace=small),
                 lambda: fd.beam_select(logits, scores, 4, workspace=small)):
        with pytest.raises(fd.FdError) as e:
            call()
        assert e.value.code == fd.FD_ERR_WORKSPACE
    # (the plain kernel needs none)
    check(fd.prefill(q, cache.k, cache.v, ints([300]), kernel=fd.FD_KERNEL_SIMT, workspace=small),
          *attend(q, cache, [300], [40], True, 128 ** -0.5))
    assert small.device_status() == 0


def test_two_threads():
    rng = np.random.default_rng(98)
    jobs = []
    for i in range(2):
        cache = Cache(rng, 2, 2000, 2, 128, 16 if i else 0)
        q = randn(rng, (2, 64, 8, 128)).to(torch.bfloat16).cuda()
        logits, scores = randn(rng, (2, 4, 30000)).cuda(), randn(rng, (2, 4)).cuda()
        jobs.append((cache, q, logits, scores, attend(q, cache, [2000, 900 + i], [64, 64], True, 128 ** -0.5), expect(logits, scores, 8)))
    errors = []

    def work(job):
        cache, q, logits, scores, (ref, bound), want = job
        try:
            stream = torch.cuda.Stream()
            lens = ints([2000, 900 + (cache.page > 0)])
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    out = fd.prefill(q, cache.k, cache.v, lens, **cache.kw())
                    best = fd.beam_select(logits, scores, 8)
                stream.synchronize()
            check(out, ref, bound)
            assert best[2].tolist() == [[x[2] for x in r] for r in want]
        except Exception as e:   # noqa: BLE001 (a thread's failure is the test's)
            errors.append(e)
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_one_workspace_on_two_streams_by_turns():
    # calls that share a workspace are ordered by their streams' waits
    rng = np.random.default_rng(99)
    cache = Cache(rng, 1, 3000, 2, 128)
    q = randn(rng, (1, 64, 8, 128)).to(torch.bfloat16).cuda()
    ref, bound = attend(q, cache, [3000], [64], True, 128 ** -0.5)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ws = fd.Workspace(4096, 16, 256, 1024)
    lens, outs = ints([3000]), [torch.zeros_like(q) for _ in range(8)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        s, other = (a, b) if i % 2 else (b, a)
        s.wait_stream(other)
        with torch.cuda.stream(s):
            fd.prefill(q, cache.k, cache.v, lens, out=o, workspace=ws)
    torch.cuda.synchronize()
    for o in outs:
        check(o, ref, bound)
