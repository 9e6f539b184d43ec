"""Refusals of beam selection's outputs, on the host before the workspace is looked
into (no GPU needed)."""
import pytest

from decode_attention_preallocated_gb300 import build as fdbuild
from decode_attention_preallocated_gb300 import fd
from test_abi_serve import ARG, PTR, fake, opts, select


@pytest.fixture(scope="module", autouse=True)
def L():
    fdbuild.build()
    return fd.lib()


def apart(**kw):
    # 2 x 4 scores, 2 x 8 winners; each array far from the others
    a = dict(logits=fake((2, 4, 1000), fd.FD_F32), scores=PTR, fin=PTR + 0x1000, end=1, so=PTR + 0x2000, bo=PTR + 0x3000, to=PTR + 0x4000)
    a.update(kw)
    return a


@pytest.mark.parametrize("name", ["so", "bo", "to"])
def test_outputs_on_inputs(name):
    # (a workspace that nobody looks into: the call is refused before)
    for at in (PTR, PTR + 28, PTR - 60, PTR + 0x1000, PTR + 0x1000 + 28, PTR + 0x1000 - 60):
        assert select(**apart(**{name: at}), o=opts(ws=8)) == ARG


@pytest.mark.parametrize("a,b", [("so", "bo"), ("bo", "to"), ("to", "so")])
def test_outputs_on_one_another(a, b):
    for off in (0, 60, -60):
        assert select(**apart(**{a: PTR + 0x8000, b: PTR + 0x8000 + off}), o=opts(ws=8)) == ARG
