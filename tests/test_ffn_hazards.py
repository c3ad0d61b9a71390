"""The pipelined feed-forward kernels' assembly with the branches of their
inline assembly followed (the wait at a step's end is skipped by all steps but
the last, so the loop's way back carries the matrix instructions' debts), and
the distance from vector-ALU results to the matrix instructions that read them."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import asm_labels as al  # noqa: E402
import mfma_hazards as mh  # noqa: E402

from tiled_dense_gemm_06_amd import build as B  # noqa: E402

WAIT = {"v_mfma_f32_16x16x32_f16": 18, "v_mfma_f32_16x16x32_bf16": 18, "v_mfma_i32_16x16x64_i8": 18}
MFMA = "v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]"


def test_numeric_labels_are_followed():
    loop = [".LBB0:", "s_nop 0", "v_accvgpr_read_b32 v9, a0", "s_nop 7", "s_nop 7", MFMA, "s_cmp_lt_i32 s0, s1",
            "s_cbranch_scc1 1f", "s_nop 7", "s_nop 7", "s_nop 7", "1:", "s_cbranch_vccnz .LBB0", "s_endpgm"]
    named = al.named_labels(loop)
    assert named[7] == "s_cbranch_scc1 " + named[11][:-1] and named[11] != "1:"
    assert not mh.scan(loop, WAIT) and mh.scan(named, WAIT)  # the way round the wait owes the result
    waits = loop[:1] + ["s_nop 7", "s_nop 7"] + loop[1:]
    assert not mh.scan(al.named_labels(waits), WAIT)
    two = al.named_labels(["1:", "s_branch 1b", "s_branch 1f", "1:"])
    assert two == [".Lnumeric0:", "s_branch .Lnumeric0", "s_branch .Lnumeric3", ".Lnumeric3:"]


@pytest.mark.parametrize("between,found", [([], True), (["s_nop 0"], True), (["s_nop 1"], False),
                                           (["v_mov_b32_e32 v20, v21", "v_mov_b32_e32 v22, v21"], False)])
def test_source_distance_is_counted(between, found):
    for write in ("v_mov_b32_e32 v2, v30", "v_accvgpr_write_b32 a1, 0"):
        assert bool(al.scan_sources([write, *between, MFMA])) == found


SOURCES = [f"ffn_panel_{t}_gfx950.hip" for t in ("f16", "bf16", "i8")]


def test_pipelined_kernels(tmp_path):
    flags = [f for f in B.HIP_FLAGS if f != "-shared"]

    def listing(name):
        out = str(tmp_path / (name + ".s"))
        r = subprocess.run([B.hipcc(), *flags, *B.SOURCE_FLAGS[name], "-I", B.INCLUDE, "-I", B.CSRC, "-S",
                            "--offload-device-only", os.path.join(B.CSRC, name), "-o", out], capture_output=True,
                           text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return mh.functions(open(out).read())

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        functions = [f for fns in ex.map(listing, SOURCES) for f in fns.items()]
    kernels = branches = 0
    for name, lines in functions:
        if not any(ln.startswith("v_mfma") for ln in lines):
            continue
        named = al.named_labels(lines)
        kernels += 1
        branches += named != lines
        assert mh.scan(named, WAIT) == [], name
        assert mh.scan_sgpr_vmem(named) == [], name
        assert al.scan_sources(named) == [], name
    assert kernels >= 46 and branches >= 10
