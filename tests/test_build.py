"""The build's order: libmxfp4.so needs hipcc alone, and is there whatever
becomes of the torch binding. (One small source stands for all; no GPU.)"""
import os
import shutil

import pytest

from mxfp4_quantized_gemm_amd import build as b


@pytest.fixture
def apart(tmp_path, monkeypatch):
    try:
        b.hipcc()
    except RuntimeError:
        pytest.skip("hipcc is missing")
    for name, file in (("BUILD", "_build"), ("LIB", "libmxfp4.so"), ("OPS", "_ops.so")):
        monkeypatch.setattr(b, name, str(tmp_path / file))
    monkeypatch.setattr(b, "SOURCES", ["api_int8.cpp"])
    return tmp_path


def test_a_failing_binding_leaves_the_library(apart, monkeypatch):
    def fails():
        raise RuntimeError("g++ on torch_ops.cpp failed")
    monkeypatch.setattr(b, "_compile_ops", fails)
    with pytest.raises(RuntimeError, match="torch_ops"):
        b.build()
    assert os.path.exists(b.LIB)


@pytest.mark.parametrize("missing", ["g++", "torch", "torch's headers"])
def test_without_what_the_binding_needs(apart, monkeypatch, capsys, missing):
    """The library alone, a word about it, and no older binding beside it."""
    if missing == "g++":
        which = shutil.which
        monkeypatch.setattr(shutil, "which", lambda n, *a, **k: None if n == "g++" else which(n, *a, **k))
    elif missing == "torch":
        monkeypatch.setitem(__import__("sys").modules, "torch", None)
    else:
        from torch.utils import cpp_extension
        monkeypatch.setattr(cpp_extension, "include_paths", lambda *a, **k: [str(apart)])
    (apart / "_ops.so").write_bytes(b"older")
    assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not os.path.exists(b.OPS)
    assert missing in capsys.readouterr().err
