"""Edges of the feed-forward operators that need no GPU: infinities at the end
of a sum (tests/emu/ffn_mixed_emu.cpp), launches of very large problems."""
import os
import re
import subprocess

import pytest

import tiled_dense_gemm_06_amd as tlg
from tiled_dense_gemm_06_amd import _native as nat
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


SHAPES = {"256x256": (256, 256), "256x128": (256, 128), "128x128": (128, 128), "64x128": (64, 128)}


def launch_threads(product, name, splits, M, N, K):
    """Threads of the launch that a planned kernel makes of a product."""
    ceil = lambda a, b: -(-a // b)  # noqa: E731
    gated = product in (nat.TLG_FFN_GATED, nat.TLG_FFN_GATED_I8)
    rows, cols, twice = {nat.TLG_FFN_DX: (M, K, 1), nat.TLG_FFN_DW: (N, K, 2)}.get(product, (M, N, 1))
    if name == "strip_16":
        return ceil(cols, 16) * 512
    if name == "general_64x64":
        return 0  # what no kernel serves is refused by the call
    bm, bn = SHAPES[name.split("_")[1]]
    return (ceil(rows, bm) * ceil(cols, bn // 2 if gated else bn) * twice + (512 if splits > 1 else 0)) * 256


@pytest.mark.parametrize("product", [nat.TLG_FFN_GATED, nat.TLG_FFN_DX, nat.TLG_FFN_DW, nat.TLG_FFN_I8,
                                     nat.TLG_FFN_GATED_I8])
def test_planned_launches_stay_below_2_to_the_32_threads(product):
    sizes = [1, 8, 63, 300, 1 << 20, (1 << 24) + 1, (1 << 27) - 15, 1 << 27, (1 << 27) + 1, 1 << 30, (1 << 31) - 1024]
    served = 0
    for M in sizes:
        for N in sizes:
            for K in (1, 8, 65, 1 << 20, (1 << 27) + 1):
                cfg, splits = nat.tlg_ffn_plan(product, M, N, K, 2, 0)
                name = nat.tlg_ffn_config_name(cfg)
                assert launch_threads(product, name, splits, M, N, K) < 1 << 32, (M, N, K, name)
                served += name != "general_64x64"
    assert served > 300
    # few tokens against more outputs than strips, or 64-token tiles, can take
    if product in (nat.TLG_FFN_GATED, nat.TLG_FFN_I8):
        for N in ((1 << 27) + 1, 1 << 30):
            assert nat.tlg_ffn_config_name(nat.tlg_ffn_plan(product, 1, N, 8, 0, 0)[0]).startswith("panel_")


def test_forward_mode_derivatives_are_refused():
    """... before anything else, where a result without a tangent would pass for a zero derivative."""
    torch = pytest.importorskip("torch")
    import torch.autograd.forward_ad as fwad

    x, w = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(6, 8, dtype=torch.float16)
    with fwad.dual_level():
        dual = fwad.make_dual(x, torch.ones_like(x))
        for fn in (lambda: tlg.gated_ffn(dual, w, w), lambda: tlg.gated_ffn(dual, w, w, save=True),
                   lambda: tlg.gated_ffn_backward(x, dual, w, w, x, x), lambda: tlg.quantize_i8(dual)):
            with pytest.raises(NotImplementedError):
                fn()
    with pytest.raises(NotImplementedError):
        torch.func.jvp(lambda v: tlg.gated_ffn(v, w, w), (x,), (x,))
    with pytest.raises(NotImplementedError):
        torch.func.vmap(lambda v: tlg.quantize_i8(v)[1])(x.expand(3, 4, 8))


def test_polynomial_of_the_normal_distribution():
    """The coefficients of ffn_phi, rounded to fp32 and evaluated in 64 bits, against erfc scaled by e^(z^2):
    within the relative error that stands beside them."""
    np = pytest.importorskip("numpy")
    erfcx = pytest.importorskip("scipy.special").erfcx
    text = open(os.path.join(B.CSRC, "ffn_ops.h")).read()
    bound = float(re.search(r"fp32 ([0-9.e-]+) at most up to z = 31", text).group(1))
    body = text[text.index("float ffn_phi("):]
    body = body[:body.index("*gauss =")]
    c = [float(np.float32(v)) for v in re.findall(r"(?:float r = |fmaf\(r, t, )(-?[0-9.]+)f", body)]
    assert len(c) == 10 and bound < 2e-7
    z = np.linspace(0, 31, 400001)
    t = 1 / (1 + z / 2)
    assert float(np.abs(t * np.polyval(c, t) / erfcx(z) - 1).max()) < bound


def test_stream_of_another_device_is_refused():
    """A call runs on its operands' device, where such a stream is not the current one."""
    torch = pytest.importorskip("torch")

    class Stream:
        device = torch.device("cuda", 1)

    x, w, s = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(6, 8, dtype=torch.float16), torch.ones(4)
    q, p = x.to(torch.int8), w.to(torch.int8)
    for fn in (lambda **k: tlg.gated_ffn(x, w, w, **k), lambda **k: tlg.gated_ffn_backward(x, x, w, w, x, x, **k),
               lambda **k: tlg.quantize_i8(x, **k), lambda **k: tlg.gemm_i8(q, s, p, s, **k),
               lambda **k: tlg.gated_ffn_i8(q, s, p, s, p, s, **k)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            fn(stream=Stream())
