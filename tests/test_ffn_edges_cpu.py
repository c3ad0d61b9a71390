"""Edges of the feed-forward operators that need no GPU: infinities at the end
of a sum (tests/emu/ffn_mixed_emu.cpp)."""
import os
import subprocess

from tiled_dense_gemm_06_amd import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def test_infinities_in_the_last_channels(tmp_path):
    """No element that the loads bring meets the zeros of a masked one."""
    exe = str(tmp_path / "ffn_mixed_emu")
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-I", B.CSRC,
                        os.path.join(HERE, "emu", "ffn_mixed_emu.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
