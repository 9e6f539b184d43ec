"""GPU tests of fd_append against its formula: bit for bit in fp32, and within
its roundings in 64 bits."""
import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from serve_util import F64, Cache, ints, quantise, randn, rope_table, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def new_rows(rng, B, n, Hq, Hkv, d):
    """q, k_new, v_new as parts of one projection."""
    qkv = randn(rng, (B, n, Hq + 2 * Hkv, d)).to(torch.bfloat16).cuda()
    return qkv.split([Hq, Hkv, Hkv], 2)


def same(a, b):
    return torch.equal(*(x.reshape(-1).contiguous().view(torch.uint8) for x in (a, b)))


def expect(cache, q, k_new, v_new, q_out, lens, new, rope, interleaved):
    """Writes what the call should leave into copies on the CPU."""
    want = {x: None if getattr(cache, x) is None else getattr(cache, x).cpu().clone() for x in ("k", "v", "ks", "vs")}
    qo = None if q is None else q_out.cpu().clone()
    for b in range(k_new.shape[0]):
        base = int(lens[b])
        pos = torch.arange(base, base + int(new[b]))
        if rope is not None:
            pos = pos[pos < rope.shape[0]]
        t = len(pos)

        def turn(x, dtype=torch.float32):
            x = x[b, :t].cpu().to(dtype)
            return x if rope is None else turned(x, rope, pos, interleaved, dtype)
        if q is not None:
            qo[b, :t] = turn(q).to(torch.bfloat16)
            exact = turn(q, F64)
            size = q[b, :t].cpu().to(F64).abs().amax(-1, keepdim=True) * 2
            assert ((qo[b, :t].to(F64) - exact).abs() <= 2.0 ** -8 * exact.abs() + 2.0 ** -22 * size).all()
        keep = pos < cache.cap
        lead, row = (x.cpu() for x in cache.at(b, cache.cap))
        lead, row = lead[pos[keep]], row[pos[keep]]
        there = (lead >= 0) & (lead < cache.k.shape[0])
        for x, new_x in (("k", turn(k_new)), ("v", v_new[b, :t].cpu().float())):
            rows = new_x[keep][there]
            if cache.int8:
                c, s = quantise(rows)
                want[x][lead[there], :, row[there]] = c
                want[x + "s"][lead[there], :, row[there]] = s
            else:
                want[x][lead[there], :, row[there]] = rows.to(torch.bfloat16)
    return want, qo


CASES = [
    # B, n, Hq, Hkv, d, cap, page, int8, token_major, r, interleaved, lens, new
    (1, 1, 8, 2, 128, 64, 0, False, False, 128, False, [0], [1]),
    (3, 5, 8, 2, 128, 40, 0, False, True, 128, True, [0, 7, 35], [5, 0, 3]),
    (2, 9, 5, 1, 256, 64, 16, False, False, 64, False, [3, 20], [9, 1]),
    (2, 33, 12, 4, 128, 90, 20, False, True, 64, True, [17, 0], [20, 33]),
    (2, 3, 4, 4, 256, 33, 1, False, False, 256, False, [30, 0], [3, 2]),
    (1, 1, 8, 2, 128, 64, 0, True, False, 128, False, [63], [1]),
    (3, 17, 16, 2, 128, 64, 16, True, True, 16, True, [0, 47, 5], [17, 17, 2]),
    (2, 40, 24, 3, 256, 100, 48, True, False, 256, False, [60, 0], [40, 39]),
    (2, 4, 64, 1, 256, 30, 0, True, True, 96, True, [1, 2], [4, 4]),
    (70, 2, 2, 1, 128, 20, 4, False, False, 128, False, list(range(70)), [2] * 70),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("form", ["rope", "rope in place", "no rope", "no q"])
def test_append(case, form):
    B, n, Hq, Hkv, d, cap, page, int8, tm, r, inter, lens, new = case
    lens = [x % (cap - n + 1) if B > 10 else x for x in lens]
    rng = np.random.default_rng(31)
    cache = Cache(rng, B, cap, Hkv, d, page, int8, tm, filled=False)
    q, k_new, v_new = new_rows(rng, B, n, Hq, Hkv, d)
    for b in range(B):                                  # padding is not read
        for x in (q, k_new, v_new):
            x[b, new[b]:] = float("nan")
    rope = None if form == "no rope" else rope_table(cap, r)
    q_out = q if form == "rope in place" else torch.full((B, n, Hq, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")[..., :d]
    if form == "no q":
        q, q_out = None, None
    want, qo = expect(cache, q, k_new, v_new, q_out, lens, new, rope, inter)
    after = ints(lens) if form == "rope in place" else ints([-5] * B)
    at = after if form == "rope in place" else ints(lens)
    ws = fd.Workspace(64, 16, 256, 1024)
    got = fd.append(k_new, v_new, cache.k, cache.v, at, new_lengths=ints(new), lengths_out=after, q=q, q_out=q_out,
                    rope=None if rope is None else rope.cuda(), interleaved=inter, workspace=ws, **cache.kw())
    torch.cuda.synchronize()
    assert after.tolist() == [a + b for a, b in zip(lens, new)]
    assert ws.device_status() == 0
    for x in ("k", "v", "ks", "vs"):
        if want[x] is not None:
            assert same(getattr(cache, x).cpu(), want[x]), x
    if q is None:
        assert got is None
    else:
        assert got is q_out and same(q_out.cpu(), qo)


@pytest.mark.parametrize("int8", [False, True])
def test_bad_lengths_tables_and_positions(int8):
    rng = np.random.default_rng(32)
    B, n, cap, page = 5, 6, 32, 8
    cache = Cache(rng, B, cap, 2, 128, page, int8, filled=False)
    q, k_new, v_new = new_rows(rng, B, n, 4, 2, 128)
    cache.table[3, 1] = 1 << 28                          # names no page
    cache.table[4, 0] = -1
    lens, new = [-4, 30, 2, 6, 0], [6, 6, 99, 4, 3]
    rope = rope_table(31, 128)                           # position 31 and on are past it
    q_out = torch.zeros_like(q)
    clamped, real = [0, 30, 2, 6, 0], [6, 6, 6, 4, 3]
    want, qo = expect(cache, q, k_new, v_new, q_out, clamped, real, rope, False)
    ws = fd.Workspace(64, 16, 256, 1024)
    after = torch.zeros(B, dtype=torch.int32, device="cuda")
    fd.append(k_new, v_new, cache.k, cache.v, ints(lens), new_lengths=ints(new), lengths_out=after, q=q, q_out=q_out,
              rope=rope.cuda(), workspace=ws, **cache.kw())
    assert after.tolist() == [6, 32, 8, 10, 3]
    assert ws.device_status() == fd.FD_DEV_BAD_LENGTH | fd.FD_DEV_BAD_INDEX
    for x in ("k", "v", "ks", "vs"):
        if want[x] is not None:
            assert same(getattr(cache, x).cpu(), want[x]), x
    assert same(q_out.cpu(), qo)


def test_int8_extremes():
    # rows of zeros, tiny, huge and not finite numbers
    rng = np.random.default_rng(33)
    x = randn(rng, (1, 8, 1, 128))
    x[0, 0] = 0
    x[0, 1] *= 1e-38
    x[0, 2] *= 1e37
    x[0, 3, 0, 5] = float("inf")
    x[0, 4, 0, 9] = float("nan")
    x[0, 5] = -0.0
    x[0, 6] = torch.tensor(9.2e-41)                      # the least number of bf16
    x = x.to(torch.bfloat16).cuda()
    cache = Cache(rng, 1, 8, 1, 128, int8=True, filled=False)
    fd.append(x, x, cache.k, cache.v, ints([0]), **cache.kw())
    k, s = cache.k[0, 0].cpu(), cache.ks[0, 0].cpu()
    for i in (3, 4):
        assert s[i].isnan() and (k[i] == 0).all()
    for i in (0, 1, 2, 5, 7):
        c, t = quantise(x[0, i, 0].cpu().float())
        assert same(k[i], c) and same(s[i], t), i
    assert s[0] == 0 and s[5] == 0
    assert (k[6].abs() <= 127).all() and s[6] > 0
    assert same(cache.v[0, 0].cpu(), k) and torch.equal(cache.vs.isnan().cpu(), cache.ks.isnan().cpu())


def test_strides_past_32_bits():
    rng = np.random.default_rng(34)
    for int8 in (False, True):
        got = []
        for stretch in (lambda t: t, lambda t: t.as_strided(t.shape, (1 << 33, *t.stride()[1:]), t.storage_offset())):
            rng = np.random.default_rng(34)
            cache = Cache(rng, 1, 50, 2, 128, int8=int8, filled=False)
            q, k_new, v_new = new_rows(rng, 1, 9, 4, 2, 128)
            kw = {a: None if b is None else stretch(b) for a, b in cache.kw().items()}
            out = torch.zeros(1, 9, 4, 128, dtype=torch.bfloat16, device="cuda")
            fd.append(stretch(k_new), stretch(v_new), stretch(cache.k), stretch(cache.v), ints([5]), q=stretch(q), q_out=stretch(out),
                      rope=rope_table(50, 128).cuda(), **kw)
            got.append((cache.k, cache.v, out))
        assert all(same(a, b) for a, b in zip(*got))


def test_captured_with_lengths_in_place():
    rng = np.random.default_rng(35)
    B, cap, steps = 3, 40, 7
    one, two = (Cache(np.random.default_rng(36), B, cap, 2, 128, 8, filled=False) for _ in range(2))
    rope = rope_table(cap, 128).cuda()
    rows = [new_rows(rng, B, 1, 4, 2, 128) for _ in range(steps)]
    lens = ints([0, 9, 30])
    wants = []
    for q, k, v in rows:
        wants.append(fd.append(k, v, one.k, one.v, lens, lengths_out=lens, q=q, rope=rope, **one.kw()))
    q, k, v = (x.clone() for x in rows[0])
    lens2, out = ints([0, 9, 30]), torch.empty(B, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    ws = fd.Workspace(64, 16, 256, 1024, stream=stream)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        fd.append(k, v, two.k, two.v, lens2, lengths_out=lens2, q=q, q_out=out, rope=rope, workspace=ws, **two.kw())
    for (a, b, c), want in zip(rows, wants):
        for to, x in ((q, a), (k, b), (v, c)):
            to.copy_(x)
        g.replay()
        assert same(out, want)
    assert lens2.tolist() == lens.tolist() == [7, 16, 37]
    assert same(one.k, two.k) and same(one.v, two.v)
