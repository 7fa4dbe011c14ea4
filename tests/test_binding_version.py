"""The paged cache's module is compiled against one PyTorch: it is built anew for another one, and is
not used with it."""
import importlib.metadata
import os

import pytest
import torch

from block_causal_attention_b200 import _abi, build


def test_used_with_the_pytorch_that_it_was_built_for(monkeypatch):
    assert _abi.paged_binding().torch_version == torch.__version__.split("+")[0]
    monkeypatch.setattr(torch, "__version__", "2.10.1+cu128")
    with pytest.raises(ImportError, match="2.10.1"):
        _abi.paged_binding()


def test_built_anew_for_another_pytorch(monkeypatch, tmp_path):
    """With sources older than the module, only the version it was built for tells."""
    made = []
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_paged_binding.so"))
    monkeypatch.setattr(build, "BINDING_FOR", str(tmp_path / "for"))

    def command(target):
        made.append(target)
        return ["touch", target]
    monkeypatch.setattr(build, "_binding_command", command)
    build.build()
    assert len(made) == 1 and os.path.exists(build.BINDING)
    build.build()
    assert len(made) == 1
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "2.10.1" if name == "torch" else version(name))
    build.build()
    assert len(made) == 2
    build.build()
    assert len(made) == 2


def test_a_pytorch_that_was_not_installed_says_its_version_itself(monkeypatch):
    def none(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", none)
    assert build._torch_version() == torch.__version__
