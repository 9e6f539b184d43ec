"""GPU tests of fd_pages_reorder at row counts around those where a block's shared
memory passes the size that needs no opt-in, each as the first call of a process."""
import os
import subprocess
import sys

import pytest

from decode_attention_preallocated_gb300 import build as fdbuild

pytestmark = pytest.mark.gpu

SCRIPT = """
import sys
import numpy as np
import torch
from decode_attention_preallocated_gb300 import fd
B, pages = int(sys.argv[1]), int(sys.argv[2])
table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages).clone()
lens = torch.full((B,), 4 * pages, dtype=torch.int32, device="cuda")
refs = torch.ones(B * pages, dtype=torch.int32, device="cuda")
src = np.random.default_rng(B).integers(0, B, B)
ws = fd.Workspace(64, 16, 256, 1024)
fd.pages_reorder(table, lens, refs, 4, torch.tensor(src, dtype=torch.int32, device="cuda"), workspace=ws)
rows = np.arange(B * pages).reshape(B, pages)[src]
assert ws.device_status() == 0
assert (table.cpu().numpy() == rows).all() and (lens == 4 * pages).all()
assert (refs.cpu().numpy() == np.bincount(rows.ravel(), minlength=B * pages)).all()
print("ok")
"""


# eight columns a block around 48 KB; four, two and one
@pytest.mark.parametrize("B", [1535, 1536, 1537, 6145, 12288, 24577, 49152])
def test_first_call_of_a_process(B):
    fdbuild.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SCRIPT, str(B), "3" if B > 3000 else "20"], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
