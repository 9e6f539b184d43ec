"""GPU tests of fd_beam_select on beams of the same logits, which tie word by word
wherever their rows start."""
import numpy as np
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
@pytest.mark.parametrize("B,K,V,n", [(3, 8, 1001, 16), (2, 8, 8193, 32), (4, 5, 50003, 20), (2, 9, 32000, 27), (1, 16, 128001, 48),
                                     (30, 8, 10623, 16), (3, 8, 23, 64)])
def test_copies_of_one_beam(dtype, B, K, V, n):
    g = torch.Generator("cuda").manual_seed(V + K)
    for _ in range(4):
        row = (3 * torch.randn(B, 1, V, generator=g, device="cuda")).to(dtype)
        logits = row.expand(B, K, V).contiguous()
        scores = (-9 * torch.rand(B, 1, generator=g, device="cuda")).expand(B, K).contiguous()
        got = fd.beam_select(logits, scores, n)
        # words by falling logit, equal ones by rising number; each beam's in turn
        order = np.argsort(-row[:, 0].double().cpu().numpy(), axis=-1, kind="stable")
        for b in range(B):
            x = row[b, 0].double().cpu().numpy()
            want, i = [], 0
            while len(want) < n and i < V:
                j = i
                while j < V and x[order[b, j]] == x[order[b, i]]:
                    j += 1
                want += [(b * K + k, int(w)) for k in range(K) for w in order[b, i:j]]
                i = j
            want = want[:n] + [(-1, -1)] * (n - len(want))
            assert list(zip(got[1][b].tolist(), got[2][b].tolist())) == want
        # a word's scores are the same in every beam
        for b in range(B):
            of = {}
            for s, w in zip(got[0][b].tolist(), got[2][b].tolist()):
                assert of.setdefault(w, s) == s
