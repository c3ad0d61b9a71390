"""Builds libtlg.so (the C-ABI library and its gfx950 kernels) in place with
hipcc, and, where torch is installed, _ffn_torch.so (the torch binding of the
feed-forward operators) with the host compiler.

Each source is compiled to its own object (in parallel), then the objects are
linked into the shared libraries.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libtlg.so")
OBJ_DIR = os.path.join(ROOT, "_build")
SOURCES = [os.path.join(CSRC, f) for f in ("api.cpp", "gemm_relu_gfx950.hip", "gemm_relu_pipe_gfx950.hip",
                                                 "gemm_relu_pipe16_gfx950.hip",
                                                 "gemm_relu_streamk_gfx950.hip", "gemm_relu_skinny_gfx950.hip",
                                                 "gemm_relu_mx_gfx950.hip", "gemm_relu_pingpong_gfx950.hip",
                                                 "noalloc.hip", "ffn_api.cpp", "ffn_general_gfx950.hip",
                                                 "ffn_panel_f16_gfx950.hip", "ffn_panel_bf16_gfx950.hip",
                                                 "ffn_panel_i8_gfx950.hip", "ffn_skinny_gfx950.hip")]

# gfx950 only. Packed fp32 instructions are disabled for every GPU code path
# (the host pass reports the feature as unknown, which is harmless).
HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-inline-asm", "-Wno-unused-command-line-argument",
]
# Per-source flags. The 16 x 16 x 32 kernels' K step is one fully unrolled
# loop of up to 128 MFMA slots, larger than the unroller's default budget for a
# loop it is asked to unroll completely.
SOURCE_FLAGS = {
    "gemm_relu_pipe16_gfx950.hip": ["-mllvm", "-pragma-unroll-threshold=1000000"],
    "ffn_panel_f16_gfx950.hip": ["-mllvm", "-pragma-unroll-threshold=1000000"],
    "ffn_panel_bf16_gfx950.hip": ["-mllvm", "-pragma-unroll-threshold=1000000"],
    "ffn_panel_i8_gfx950.hip": ["-mllvm", "-pragma-unroll-threshold=1000000"],
}


# The torch binding: host code only.
BINDING_SOURCE = os.path.join(CSRC, "ffn_torch.cpp")
BINDING = os.path.join(HERE, "_ffn_torch.so")


def _binding_cmds(obj: str, out: str) -> tuple[list[str], list[str]] | None:
    """The compile and the link command of the torch binding; None without torch."""
    try:
        from torch.utils import cpp_extension as ext
    except ImportError:
        return None

    inc = [f"-I{p}" for p in (*ext.include_paths("cuda"), sysconfig.get_paths()["include"], INCLUDE, CSRC)
           if os.path.isdir(p)]
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
                "-DTORCH_EXTENSION_NAME=_ffn_torch", *inc, "-c", BINDING_SOURCE, "-o", obj]
    link = [cxx, "-shared", obj, "-o", out, *(f"-L{p}" for p in ext.library_paths()), f"-L{HERE}",
            *(f"-Wl,-rpath,{p}" for p in ext.library_paths()), "-Wl,-rpath,$ORIGIN", "-l:libtlg.so", "-lc10",
            "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python"]
    return compile_, link


def hipcc() -> str:
    cand = os.environ.get("HIPCC") or shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    return cand


def compile_cmd(output: str, extra=()) -> list[str]:
    """One hipcc command that builds the whole library from the sources
    (per-source flags are applied to every source)."""
    per = [f for flags in SOURCE_FLAGS.values() for f in flags]
    return [hipcc(), *HIP_FLAGS, *per, *extra, "-I", INCLUDE, "-I", CSRC, *SOURCES, "-o", output]


def _compile_one(src: str, obj: str) -> subprocess.CompletedProcess:
    flags = [f for f in HIP_FLAGS if f != "-shared"]
    cmd = [hipcc(), *flags, *SOURCE_FLAGS.get(os.path.basename(src), []), "-I", INCLUDE, "-I", CSRC,
           "-c", src, "-o", obj]
    return subprocess.run(cmd, capture_output=True, text=True)


def build(verbose: bool = False) -> str:
    """Compile the library, and where torch is installed its binding; always
    recompiles. Returns the path of libtlg.so, which is in place before anything
    of the binding can fail."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    objs = [os.path.join(OBJ_DIR, os.path.basename(s) + ".o") for s in SOURCES]
    binding_obj = os.path.join(OBJ_DIR, os.path.basename(BINDING_SOURCE) + ".o")
    binding_cmds = _binding_cmds(binding_obj, BINDING + ".tmp")
    jobs = max(1, min(len(SOURCES) + 1, int(os.environ.get("MAX_JOBS", os.cpu_count() or 4))))
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        binding = binding_cmds and ex.submit(subprocess.run, binding_cmds[0], capture_output=True, text=True)
        results = list(ex.map(_compile_one, SOURCES, objs))
    for src, r in zip(SOURCES, results):
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed on {os.path.basename(src)} ({r.returncode}):\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
    tmp = LIB + ".tmp"
    r = subprocess.run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc link failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if binding is None:
        if verbose:
            print(f"no torch: {os.path.basename(BINDING)} is not built")
        return LIB
    r = binding.result()
    if r.returncode == 0:
        r = subprocess.run(binding_cmds[1], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building {os.path.basename(BINDING)} failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
