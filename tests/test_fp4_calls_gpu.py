"""Calls of the 4-bit cache that the binding alone can tell apart."""
import numpy as np
import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from fp4_util import bf16, cache, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fdbuild.build()
    fd.lib()


def test_a_block_table_without_columns_is_refused():
    # two sequences and two pages: without its table the pool would pass for a
    # flat cache
    rng = np.random.default_rng(111)
    (kd, ksd), (vd, vsd) = (to_dev(*cache(rng, 2, 2, 16, 128)) for _ in range(2))
    lens = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    new = bf16(rng, (2, 1, 2, 128)).cuda()
    before = kd.clone()
    for call in (lambda: fd.decode_fp4(bf16(rng, (2, 1, 4, 128)).cuda(), kd, vd, ksd, vsd, lens, block_table=table),
                 lambda: fd.append_fp4(new, new, kd, vd, ksd, vsd, lens, block_table=table),
                 lambda: fd.read_fp4(kd, vd, ksd, vsd, lens, 3, block_table=table)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(before, kd)
