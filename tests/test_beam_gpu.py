"""GPU tests of fd_beam_select against its definition: the same beams and words,
scores within their roundings."""
import math

import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from serve_util import ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def expect(logits, scores, n_out, finished=None, end=None):
    """In 64 bits; lse rounded to fp32, as the definition has it."""
    x = logits.double().cpu().numpy()
    B, K, V = x.shape
    s = scores.double().cpu().numpy()
    with np.errstate(all="ignore"):
        m = x.max(-1, keepdims=True)
        m = np.where(np.isinf(m) & (m < 0), 0.0, m)
        lse = (m + np.log(np.exp(x - m).sum(-1, keepdims=True))).astype(np.float32).astype(np.float64)
        total = s[..., None] + (x - lse)
    if finished is not None:
        f = finished.cpu().numpy() != 0
        total[f] = -np.inf
        total[..., end] = np.where(f, s, total[..., end])
    out = []
    for b in range(B):
        flat = np.where(np.isnan(total[b].reshape(-1)), -np.inf, total[b].reshape(-1))
        order = np.argsort(-flat, kind="stable")[:n_out]
        order = [o for o in order if flat[o] > -np.inf]
        row = [(flat[o], b * K + o // V, o % V) for o in order] + [(-np.inf, -1, -1)] * (n_out - len(order))
        out.append(row)
    return out


def check(logits, scores, n_out, finished=None, end=None, got=None):
    got = fd.beam_select(logits, scores, n_out, finished=finished, end_token=end) if got is None else got
    want = expect(logits, scores, n_out, finished, end)
    assert got[1].tolist() == [[x[1] for x in r] for r in want]
    assert got[2].tolist() == [[x[2] for x in r] for r in want]
    a, b = got[0].double().cpu().numpy(), np.array([[x[0] for x in r] for r in want])
    there = np.isfinite(b)
    assert (a[~there] == -np.inf).all()
    # lse is off by the step of its rounding at most (two of 2^-24), and by the
    # errors of the exponentials and their sum (2^-20); the score is rounded once
    a, b = a[there], b[there]
    assert (np.abs(a - b) <= 2.0 ** -24 * np.abs(b) + 2.0 ** -19 + 2.0 ** -22 * 40).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,K,V,n", [(1, 1, 1, 1), (1, 1, 2, 5), (2, 3, 7, 4), (1, 4, 32000, 8), (3, 5, 2049, 10), (2, 8, 8192, 16),
                                     (2, 2, 8193, 64), (1, 128, 300, 64), (20, 8, 1001, 16), (1, 1, 131072, 1), (40, 4, 40000, 7)])
def test_select(B, K, V, n, dtype):
    g = torch.Generator("cuda").manual_seed(B * 7 + K * 11 + V)
    # (bf16 logits have many equal numbers)
    logits = (3 * torch.randn(B, K, V, generator=g, device="cuda")).to(dtype)
    scores = -9 * torch.rand(B, K, generator=g, device="cuda")
    check(logits, scores, n)
    if K > 1:
        fin = ints(np.arange(B * K).reshape(B, K) % 3 == 1)
        check(logits, scores, n, fin, V // 2)


def test_ties_go_to_the_lower_beam_and_word():
    logits = torch.zeros(2, 3, 5000, device="cuda")
    scores = torch.zeros(2, 3, device="cuda")
    check(logits, scores, 20)                            # every word alike: too many for the list
    logits[:, 1, 4000] = 1.0
    logits[:, 2, 17] = 1.0
    check(logits, scores, 64)
    logits = torch.full((1, 2, 20000), -1.0, device="cuda").to(torch.bfloat16)
    logits[0, :, ::3] = 2.0
    check(logits, torch.tensor([[-1.0, -1.0]], device="cuda"), 33)
    logits = torch.zeros(1, 2, 100, device="cuda")       # both zeros are one
    logits[0, 0, :50] = -0.0
    check(logits, torch.zeros(1, 2, device="cuda"), 60)


def test_masked_words_dead_beams_and_bad_numbers():
    g = torch.Generator("cuda").manual_seed(5)
    V = 9000
    logits = torch.randn(4, 4, V, generator=g, device="cuda")
    keep = torch.rand(4, 4, V, generator=g, device="cuda") < 0.0005
    scores = -torch.rand(4, 4, generator=g, device="cuda")
    masked = logits.masked_fill(~keep, -math.inf)
    check(masked, scores, 24)                            # fewer words than wanted
    masked[1] = -math.inf                                # nothing at all
    masked[2, :3] = -math.inf
    check(masked, scores, 24)
    first = scores.clone()
    first[:, 1:] = -math.inf                             # a search's first step
    check(logits, first, 8)
    first[3] = -math.inf
    check(logits, first, 8)
    bad = logits.clone()
    bad[0, 1, 77] = math.nan                             # such a beam has no words
    bad[1, 2, 5] = math.inf
    bad[2, 0, V - 1] = math.nan
    scores[3, 2] = math.nan
    check(bad, scores, 16)
    lowest = torch.finfo(torch.float32).min
    check(logits.masked_fill(~keep, lowest), -torch.rand(4, 4, generator=g, device="cuda"), 30)
    check(logits * 1e30, torch.zeros(4, 4, device="cuda"), 12)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_given_outputs(dtype):
    g = torch.Generator("cuda").manual_seed(6)
    wide = torch.randn(3, 4, 3, 1003, generator=g, device="cuda").to(dtype)
    scores = -torch.rand(3, 4, generator=g, device="cuda")
    for logits in (wide[:, :, 1, 1:], wide[:, :, 0], wide[..., 2, :1000], wide.transpose(0, 1)[:3, :, 2].transpose(0, 1)[:3, :3]):
        K = logits.shape[1]
        out = (torch.zeros(3, 9, device="cuda"), ints(np.zeros((3, 9))), ints(np.zeros((3, 9))))
        s = scores[:, :K].contiguous()
        got = fd.beam_select(logits, s, 9, out=out)
        assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, out))
        check(logits, s, 9, got=got)


def test_captured_replayed_and_repeated():
    g = torch.Generator("cuda").manual_seed(8)
    logits = torch.randn(6, 4, 50001, generator=g, device="cuda")
    scores = -torch.rand(6, 4, generator=g, device="cuda")
    stream = torch.cuda.Stream()
    ws = fd.Workspace(64, 16, 256, 2048, stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = fd.beam_select(logits, scores, 8, workspace=ws)
    for _ in range(3):
        logits.copy_(torch.randn(6, 4, 50001, generator=g, device="cuda"))
        scores.uniform_(-3, 0, generator=g)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(logits, scores, 8, got=got)
        first = [x.clone() for x in got]
        for _ in range(5):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_beams_far_apart_and_many_alike(dtype):
    # more candidates near the best than the join's list holds, in some beams only
    rng = np.random.default_rng(11)
    logits = torch.from_numpy(rng.standard_normal((3, 16, 10623))).float().cuda().to(dtype) * 2
    scores = torch.from_numpy(rng.standard_normal((3, 16)) * 3).float().cuda()
    check(logits, scores, 32)
    check(torch.zeros(2, 8, 50000, device="cuda", dtype=dtype), torch.zeros(2, 8, device="cuda"), 32)
    logits[1] = 0.5
    check(logits, torch.where(scores > 0, 1.0, scores), 64)
