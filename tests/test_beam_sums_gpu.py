"""GPU tests of the log sum exp that fd_beam_select takes its scores from."""
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spread", [0.0, 0.01, 1.0, 3.0, 30.0])
@pytest.mark.parametrize("B,V", [(40, 1), (40, 7), (40, 1003), (30, 32000), (30, 50257), (4, 1000001)])
def test_error(B, V, spread, dtype):
    g = torch.Generator("cuda").manual_seed(V)
    x = spread * torch.randn(B, 1, V, generator=g, device="cuda")
    # the best word's logit is 0, so its score is -lse without another rounding
    x = (x - x.amax(-1, keepdim=True)).to(dtype)
    got = fd.beam_select(x, torch.zeros(B, 1, device="cuda"), 1)[0].view(-1).double()
    want = -torch.logsumexp(x.double().view(B, V), -1)
    # Its rounding, half a step, and before that (relative, in units of 2^-24):
    # - a term exp(x - m): the difference, its product with log2 e and that constant, 2.25
    #   |x - m|, whose mean over the weights is at most ln V <= 17: 38; 2^y of the special
    #   function unit 4;
    # - sums: 128 in a thread (16 steps of 16 words, two at a time), 5 over a warp, 8 over a
    #   block, 16 slices a lane and 5 over a warp: 162;
    # - references that move: each of 16 steps and some 8 joins at most one more 2^y, 4: 96.
    # 300 in all, below 2^-15.7.
    assert ((got - want).abs() <= 2.0 ** -24 * want.abs() * (1 + 1e-6) + 2.0 ** -15).all()


def test_near_ties_fall_by_the_scores_that_come_back():
    # two beams whose best words differ by some fp32 steps: the one that is returned first
    # scores no less, and by the definition no less than what lse may be off by
    g = torch.Generator("cuda").manual_seed(9)
    x = torch.randn(200, 2, 5001, generator=g, device="cuda") * 2
    x -= x.amax(-1, keepdim=True)
    lse = torch.logsumexp(x.double(), -1)
    s = (lse - 11 + torch.randint(-9, 10, (200, 2), generator=g, device="cuda") * 2.0 ** -21).float()
    got, beams, _ = fd.beam_select(x, s, 2)
    assert (got[:, 0] >= got[:, 1]).all()
    true = s.double() - lse
    first = true.gather(1, (beams[:, :1] % 2).long())[:, 0]
    assert (true.amax(-1) - first <= 2 * (2.0 ** -24 * lse.abs().amax(-1) + 2.0 ** -15)).all()
