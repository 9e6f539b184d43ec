"""When the extension is built again."""
import os
import types

import pytest
import torch

from decode_attention_preallocated_gb300 import build as fdbuild


@pytest.fixture
def runs(tmp_path, monkeypatch):
    """Builds that write an empty file in place of the extension."""
    made = []

    def run(cmd, **kw):
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(fdbuild, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(fdbuild, "NATIVE", str(tmp_path / "_fd_torch.so"))
    monkeypatch.setattr(fdbuild, "NATIVE_FOR", str(tmp_path / "_build" / "_fd_torch.for"))
    monkeypatch.setattr(fdbuild, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(fdbuild, "subprocess", types.SimpleNamespace(run=run))
    return made


def test_another_pytorch_or_python_builds_the_extension_again(runs, monkeypatch):
    fdbuild.build_native()
    fdbuild.build_native()
    assert len(runs) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    fdbuild.build_native()
    fdbuild.build_native()
    assert len(runs) == 2
    monkeypatch.setattr(fdbuild.sysconfig, "get_config_var", lambda name: "cpython-999")
    fdbuild.build_native()
    assert len(runs) == 3
    fdbuild.build_native(force=True)
    assert len(runs) == 4


def test_an_extension_of_unknown_origin_is_built_again(runs):
    fdbuild.build_native()
    os.remove(fdbuild.NATIVE_FOR)
    fdbuild.build_native()
    assert len(runs) == 2
