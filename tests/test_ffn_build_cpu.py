"""The library builds, and is in place, whatever becomes of its torch binding
(compilers replaced by stand-ins that write empty files)."""
import os
import subprocess
import sys

import pytest

from tiled_dense_gemm_06_amd import build as B


@pytest.fixture
def places(tmp_path, monkeypatch):
    """Outputs in a folder of the test, and a compiler that only makes its output file."""
    lib, binding = tmp_path / "libtlg.so", tmp_path / "_ffn_torch.so"
    monkeypatch.setattr(B, "LIB", str(lib))
    monkeypatch.setattr(B, "BINDING", str(binding))
    monkeypatch.setattr(B, "OBJ_DIR", str(tmp_path / "obj"))
    fails = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        bad = any(f in os.path.basename(out) for f in fails)
        if not bad:
            open(out, "w").close()
        return subprocess.CompletedProcess(cmd, int(bad), "", "stand-in failure" if bad else "")

    monkeypatch.setattr(B.subprocess, "run", run)
    return lib, binding, fails


def test_without_torch(places, monkeypatch):
    lib, binding, _ = places
    for name in [n for n in sys.modules if n == "torch" or n.startswith("torch.utils.cpp_extension")]:
        monkeypatch.setitem(sys.modules, name, None)
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setitem(sys.modules, "torch.utils", None)
    assert B.build() == str(lib)
    assert lib.exists() and not binding.exists()


@pytest.mark.parametrize("fails", ["ffn_torch.cpp.o", "_ffn_torch.so.tmp"])
def test_binding_fails_after_the_library(places, fails):
    pytest.importorskip("torch")
    lib, binding, bad = places
    bad.append(fails)
    with pytest.raises(RuntimeError, match="_ffn_torch.so"):
        B.build()
    assert lib.exists() and not binding.exists()


def test_both(places):
    pytest.importorskip("torch")
    lib, binding, _ = places
    assert B.build() == str(lib)
    assert lib.exists() and binding.exists()
