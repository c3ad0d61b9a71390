"""GPU parity of the feed-forward operators at their edges: values that are no
numbers and values at the ends of the types' ranges, against 64 bits
(tests/ffn_ref.py derives the bounds)."""
import zlib

import pytest

import tiled_dense_gemm_06_amd as tlg
from tiled_dense_gemm_06_amd import _native as nat

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import ffn_ref as R  # noqa: E402

T16 = [torch.float16, torch.bfloat16]
CONFIGS = [-1] + [c for c in range(32) if nat.tlg_ffn_config_name(c)]


def config_name(c):
    return "auto" if c < 0 else nat.tlg_ffn_config_name(c)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def gen_for(dev, *key):
    return torch.Generator(device=dev).manual_seed(zlib.crc32(repr(key).encode()))


def served(fn):
    """fn(), or None where a forced kernel does not serve the problem."""
    try:
        return fn()
    except tlg.TlgError as e:
        if e.status == nat.TLG_ERROR_NOT_SUPPORTED:
            return None
        raise


@pytest.mark.parametrize("config", CONFIGS, ids=config_name)
@pytest.mark.parametrize("t", T16, ids=["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(300, 513, 259), (70, 77, 8), (130, 512, 130), (9, 13, 1)],
                         ids=lambda s: "x".join(map(str, s)))
def test_backward_infinity_in_the_last_channel(dev, shape, t, config):
    """An infinite gradient of one token's last output makes that token's dX,
    and the last channels' weight gradients, infinite (not NaN), and leaves the
    other tokens and channels as they are. Inputs of the token and weights of
    the channel are positive, so every term that meets the infinity agrees."""
    M, K, N = shape
    print(f"infinity {shape} {t} {config_name(config)}", flush=True)
    g = gen_for(dev, *shape)
    X = R.exact_ints(M, K, g, dev, t)
    Wg, Wu = (R.exact_ints(N, K, g, dev, t) for _ in range(2))
    G, U = (torch.randint(1, 4, (M, N), generator=g, device=dev).to(t) for _ in range(2))
    dH = R.exact_ints(M, N, g, dev, t)
    m = M // 2
    X[m], Wg[N - 1], Wu[N - 1] = 1, 2, 1
    clean = served(lambda: tlg.gated_ffn_backward(dH, X, Wg, Wu, G, U, act="relu", config=config))
    if clean is None:
        pytest.skip("not served by this kernel")
    dH[m, N - 1] = float("inf")
    dX, dWg, dWu = tlg.gated_ffn_backward(dH, X, Wg, Wu, G, U, act="relu", config=config)
    torch.cuda.synchronize()
    assert bool((dX[m] == float("inf")).all()), dX[m]
    assert bool((dWg[N - 1] == float("inf")).all()) and bool((dWu[N - 1] == float("inf")).all())
    others = torch.arange(M, device=dev) != m
    assert torch.equal(dX[others], clean[0][others])
    assert torch.equal(dWg[:N - 1], clean[1][:N - 1]) and torch.equal(dWu[:N - 1], clean[2][:N - 1])


@pytest.mark.parametrize("t", T16, ids=["fp16", "bf16"])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gates_far_from_zero(dev, name, t):
    """Past |g| = 256 every activation is g or 0 and its slope 1 or 0, up to the
    largest finite value of the type: both gradients are exact."""
    far = [256.0, 1000.0, 2.0 ** 14, float(torch.finfo(t).max)]
    if t == torch.bfloat16:
        far += [2.0 ** 62, 2.0 ** 64, 2.0 ** 80, 2.0 ** 120]
    row = torch.tensor(far + [-v for v in far], device=dev).to(t)
    n = 64
    G = row.repeat(n // len(row))[None].repeat(5, 1)
    G[2:] = G[2:].flip(1)
    print(f"far gates {name} {t}", flush=True)
    on = (G > 0).double()
    eye, zero = torch.eye(n, dtype=t, device=dev), torch.zeros(n, n, dtype=t, device=dev)
    U, dH = torch.full_like(G, 2), torch.full_like(G, 0.5)
    one = torch.ones(5, n, dtype=t, device=dev)
    _, Gk, _ = tlg.gated_ffn(G, eye, zero, act=name, save=True)
    dg = tlg.gated_ffn_backward(dH, one, eye, zero, G, U, act=name)[0]
    du = tlg.gated_ffn_backward(dH, one, zero, eye, G, U, act=name)[0]
    torch.cuda.synchronize()
    assert torch.equal(Gk, G)
    assert torch.equal(dg, on.to(t))
    assert torch.equal(du, (G.double() * on * 0.5).to(t))


def ranged_case(kind, M, K, N, dev):
    """fp16 inputs whose dG and dU lie outside fp16's range while the gradients lie inside."""
    t = torch.float16
    g = gen_for(dev, kind, M, K, N)
    dh, u, x, w = {"large": (256, 300, 0.005, 0.005), "small": (1e-6, 2e-2, 30, 300), "mixed": (1e-3, 1e-3, 30, 1)}[kind]
    normal = lambda r, c, s: (torch.randn(r, c, generator=g, device=dev) * s).to(t)  # noqa: E731
    X, Wg, Wu = normal(M, K, x), normal(N, K, w), normal(N, K, w)
    G, U, dH = normal(M, N, 1), normal(M, N, u), normal(M, N, dh)
    if kind == "mixed":  # one channel ten million times the others
        U[:, 0] = 1e4
    return X, Wg, Wu, G, U, dH


@pytest.mark.parametrize("config", CONFIGS, ids=config_name)
@pytest.mark.parametrize("kind", ["large", "small", "mixed"])
@pytest.mark.parametrize("shape", [(300, 264, 200), (130, 77, 90), (40, 5, 33)], ids=lambda s: "x".join(map(str, s)))
def test_backward_past_the_range_of_fp16(dev, shape, kind, config):
    """dG and dU carry one rounding (u) and the activation's error, and 2^-38 of
    the largest |dH U| or |dH G| at most; the sums K 2^-24 of their magnitudes, the results
    one rounding more (half a subnormal step near zero)."""
    M, K, N = shape
    t = torch.float16
    name = ["silu", "gelu", "gelu_tanh", "relu"][(M + config) % 4]
    print(f"range {shape} {kind} {name} {config_name(config)}", flush=True)
    X, Wg, Wu, G, U, dH = ranged_case(kind, M, K, N, dev)
    got = served(lambda: tlg.gated_ffn_backward(dH, X, Wg, Wu, G, U, act=name, config=config))
    if got is None:
        pytest.skip("not served by this kernel")
    torch.cuda.synchronize()
    x, wg, wu, dh, u = (v.double() for v in (X, Wg, Wu, dH, U))
    value, slope = R.act(name, G)
    dG, dU = dh * u * slope, dh * value
    low = 2.0 ** -38 * float(torch.maximum((dh * u).abs(), (dh * G.double()).abs()).max())
    eG = dG.abs() * (R.unit(t) + 2.0 ** -21) + (dh * u).abs() * R.slope_bound(name, G) + low
    eU = dU.abs() * (R.unit(t) + 2.0 ** -21 + R.act_rel(name, G)) + low
    for what, y, ref, err, mag, k in (
            ("dX", got[0], dG @ wg + dU @ wu, eG @ wg.abs() + eU @ wu.abs(), dG.abs() @ wg.abs() + dU.abs() @ wu.abs(), 2 * N),
            ("dWg", got[1], dG.T @ x, eG.T @ x.abs(), dG.abs().T @ x.abs(), M),
            ("dWu", got[2], dU.T @ x, eU.T @ x.abs(), dU.abs().T @ x.abs(), M)):
        assert float(ref.abs().max()) < 65504, what  # the case itself: a gradient that fp16 holds
        bound = err * (1 + R.unit(t)) + mag * (k + 2) * 2.0 ** -24 + ref.abs() * R.unit(t) + R.tiny(t)
        d = (y.double() - ref).abs()
        assert bool((d <= bound).all()), (what, float((d / bound).max()))


def test_backward_scale_with_infinities_and_zeros(dev):
    """The scale goes by finite values: an infinite or NaN gradient leaves the
    other tokens' dX as it is, and gradients of zeros are zeros."""
    M, K, N = 70, 96, 130
    X, Wg, Wu, G, U, dH = ranged_case("large", M, K, N, dev)
    dH[3] = 0  # so the token that loses its gradient below does not hold the largest
    clean = tlg.gated_ffn_backward(dH, X, Wg, Wu, G, U)
    for bad in (float("inf"), float("nan")):
        broken = dH.clone()
        broken[3, 5] = bad
        dX, _, _ = tlg.gated_ffn_backward(broken, X, Wg, Wu, G, U)
        torch.cuda.synchronize()
        others = torch.arange(M, device=dev) != 3
        assert torch.equal(dX[others], clean[0][others])
        assert not bool(torch.isfinite(dX[3]).any())
    zero = tlg.gated_ffn_backward(torch.zeros_like(dH), X, Wg, Wu, G, U)
    torch.cuda.synchronize()
    assert all(bool((v == 0).all()) for v in zero)


@pytest.mark.parametrize("M,K", [((1 << 26) + 5, 3), ((1 << 26) + 5, 16), ((1 << 24) + 5, 1040)])
def test_quantize_more_tokens_than_one_launch_holds(dev, M, K):
    """Every token's codes and scale, where one launch's threads would pass 2^32."""
    print(f"quantize {M} x {K}", flush=True)
    base = torch.randn(997, K, generator=gen_for(dev, K), device=dev).to(torch.bfloat16)
    rq, rs = R.quantize(base)
    which = torch.arange(M, device=dev) % 997
    X = base[which]
    q, s = tlg.quantize_i8(X)
    torch.cuda.synchronize()
    assert torch.equal(s, rs[which])
    step = 1 << 22
    for m in range(0, M, step):
        assert torch.equal(q[m:m + step], rq[which[m:m + step]]), m


@pytest.mark.parametrize("config", CONFIGS, ids=config_name)
def test_empty_sums_of_every_kernel(dev, config):
    """K = 0: every product is +0, whichever kernel takes it; none fails."""
    print(f"empty sums {config_name(config)}", flush=True)
    for M, N in ((3, 5), (70, 130)):
        h = [torch.zeros(r, 0, dtype=torch.float16, device=dev) for r in (M, N)]
        q = [torch.zeros(r, 0, dtype=torch.int8, device=dev) for r in (M, N)]
        s = [torch.ones(r, device=dev) for r in (M, N)]
        outs = [served(lambda: tlg.gated_ffn(h[0], h[1], h[1], save=True, config=config)),
                served(lambda: (tlg.gemm_i8(q[0], s[0], q[1], s[1], config=config),)),
                served(lambda: (tlg.gated_ffn_i8(q[0], s[0], q[1], s[1], q[1], s[1], config=config),))]
        torch.cuda.synchronize()
        assert all(bool((v == 0).all()) and v.shape == (M, N) for o in outs if o is not None for v in o)


def test_derivatives_that_are_not_computed_raise(dev):
    """Forward mode, torch.func transforms and scales that require a gradient;
    under no_grad, and detached, the same calls are served."""
    import torch.autograd.forward_ad as fwad

    X, W = torch.ones(4, 8, dtype=torch.float16, device=dev), torch.ones(6, 8, dtype=torch.float16, device=dev)
    G = torch.ones(4, 6, dtype=torch.float16, device=dev)
    Q, S = tlg.quantize_i8(X)
    QW, SW = tlg.quantize_i8(W)
    with fwad.dual_level():
        dual = lambda v: fwad.make_dual(v, torch.ones_like(v))  # noqa: E731
        grad = X.clone().requires_grad_()
        for fn in (lambda: tlg.gated_ffn(dual(X), W, W), lambda: tlg.gated_ffn(X, dual(W), W),
                   lambda: tlg.gated_ffn(X, W, dual(W), save=True), lambda: tlg.gated_ffn(grad, W, dual(W)),
                   lambda: tlg.gated_ffn_backward(dual(G), X, W, W, G, G),
                   lambda: tlg.gated_ffn_backward(G, X, W, W, G, dual(G)), lambda: tlg.quantize_i8(dual(X)),
                   lambda: tlg.gemm_i8(Q, dual(S), QW, SW),
                   lambda: tlg.gated_ffn_i8(Q, S, QW, SW, QW, dual(SW))):
            with pytest.raises(RuntimeError):  # NotImplementedError is one, and so is autograd's own
                fn()
    for fn in (lambda: torch.func.jvp(lambda v: tlg.gated_ffn(v, W, W), (X,), (X,)),
               lambda: torch.func.jvp(lambda v: tlg.gated_ffn(X, v, W), (W,), (W,)),
               lambda: torch.func.vmap(lambda v: tlg.gated_ffn(v, W, W))(X.expand(3, 4, 8)),
               lambda: torch.func.grad(lambda v: tlg.gated_ffn(v, W, W).float().sum())(X)):
        with pytest.raises(RuntimeError):
            fn()
    for i in range(2):
        scales = [S, SW]
        scales[i] = scales[i].clone().requires_grad_()
        calls = (lambda: tlg.gemm_i8(Q, scales[0], QW, scales[1]),
                 lambda: tlg.gated_ffn_i8(Q, scales[0], QW, SW, QW, scales[1]))
        for fn in calls:
            with pytest.raises(NotImplementedError):
                fn()
            with torch.no_grad():
                fn()
    torch.cuda.synchronize()


def test_forward_calls_without_room_for_a_workspace(dev):
    """Aligned copies of odd rows as large as the operands: where the allocator
    cannot give them, the call goes on without."""
    M, K, N = 1 << 16, 8193, 2049
    for product in (nat.TLG_FFN_GATED, nat.TLG_FFN_I8, nat.TLG_FFN_GATED_I8):
        assert config_name(nat.tlg_ffn_plan(product, M, N, K, 2)[0]).endswith("_packed")
    print("no room", flush=True)
    t = torch.bfloat16
    g = gen_for(dev, "room")
    # made on the GPU, kept on the host, so that no input lies in a block with room to spare
    X, Wg, Wu = [R.exact_ints(r, K, g, dev, t, scale=0.125).cpu() for r in (M, N, N)]
    q = [torch.randint(-127, 128, (r, K), generator=g, device=dev, dtype=torch.int8).cpu() for r in (M, N, N)]
    torch.cuda.empty_cache()
    X, Wg, Wu = [v.to(dev) for v in (X, Wg, Wu)]
    q = [v.to(dev) for v in q]
    s = [torch.rand(r, generator=g, device=dev) * 0.01 for r in (M, N, N)]
    calls = {"gated_ffn": lambda: tlg.gated_ffn(X, Wg, Wu, act="relu"),
             "gemm_i8": lambda: tlg.gemm_i8(q[0], s[0], q[1], s[1], out_dtype=t),
             "gated_ffn_i8": lambda: tlg.gated_ffn_i8(q[0], s[0], q[1], s[1], q[2], s[2], act="relu", out_dtype=t)}
    want = {k: fn().cpu() for k, fn in calls.items()}
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(dev).total_memory
    need = [f(M, N, K) for f in (nat.lib().tlg_gated_ffn_workspace, nat.lib().tlg_gemm_i8_workspace,
                                 nat.lib().tlg_gated_ffn_i8_workspace)]
    assert min(need) > 3 * M * N  # (a result takes 2 M N)
    try:
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved(dev) + 3 * M * N) / total, dev)
        with pytest.raises(torch.OutOfMemoryError):
            torch.empty(min(need), dtype=torch.uint8, device=dev)
        for name, fn in calls.items():
            got = fn()
            torch.cuda.synchronize()
            # int8 sums are exact, and so are those of small integers
            assert torch.equal(got.cpu(), want[name]), name
            del got
            torch.cuda.empty_cache()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0, dev)


@pytest.mark.parametrize("config", CONFIGS, ids=config_name)
@pytest.mark.parametrize("t", T16, ids=["fp16", "bf16"])
def test_backward_nan_stays_in_its_token_and_channel(dev, t, config):
    """A NaN in one token's dH spoils that token's dX and that channel's weight gradients, nothing else."""
    M, K, N = 150, 77, 131
    print(f"nan {t} {config_name(config)}", flush=True)
    g = gen_for(dev, "nan", M)
    X = R.exact_ints(M, K, g, dev, t)
    Wg, Wu = (R.exact_ints(N, K, g, dev, t) for _ in range(2))
    G, U, dH = (R.exact_ints(M, N, g, dev, t) for _ in range(3))
    clean = served(lambda: tlg.gated_ffn_backward(dH, X, Wg, Wu, G, U, act="relu", config=config))
    if clean is None:
        pytest.skip("not served by this kernel")
    for m, n in ((0, 0), (M - 1, N - 1), (64, 128)):
        bad = dH.clone()
        bad[m, n] = float("nan")
        dX, dWg, dWu = tlg.gated_ffn_backward(bad, X, Wg, Wu, G, U, act="relu", config=config)
        torch.cuda.synchronize()
        rows, cols = torch.arange(M, device=dev) != m, torch.arange(N, device=dev) != n
        assert bool(torch.isnan(dX[m]).all()) and bool(torch.isnan(dWg[n]).all()) and bool(torch.isnan(dWu[n]).all())
        assert torch.equal(dX[rows], clean[0][rows])
        assert torch.equal(dWg[cols], clean[1][cols]) and torch.equal(dWu[cols], clean[2][cols])


def test_graph_replays_of_the_fp16_backward_pass(dev):
    """The scale of dG and dU is found anew by every replay: gradients of other
    magnitudes from one to the next, eager calls between them."""
    M, K, N = 96, 136, 200
    X, Wg, Wu, G, U, dH = ranged_case("large", M, K, N, dev)
    step = lambda: tlg.gated_ffn_backward(dH, X, Wg, Wu, G, U)  # noqa: E731
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream(dev).wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    g = gen_for(dev, "replays")
    for scale in (256, 1e-6, 1, 0, 256):
        dH.copy_(torch.randn(M, N, generator=g, device=dev) * scale)
        for o in outs:
            o.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b) and bool(torch.isfinite(a).all())
        torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
def test_closed_gates_do_not_set_the_scale(dev, name):
    """A far negative gate passes nothing on, so it takes nothing from the
    precision of the others: bounds as above, with |dH G| at most 0.28 |dH|
    where G < 0."""
    M, K, N = 130, 77, 90
    t = torch.float16
    g = gen_for(dev, "closed", name)
    X, Wg, Wu = (torch.randn(r, K, generator=g, device=dev).to(t) for r in (M, N, N))
    G = torch.randn(M, N, generator=g, device=dev).to(t)
    U, dH = ((torch.randn(M, N, generator=g, device=dev) * s).to(t) for s in (1, 1e-6))
    G[7, 5], dH[7, 5], U[7, 5] = -60000, 1, 1e-7
    dX, dWg, dWu = tlg.gated_ffn_backward(dH, X, Wg, Wu, G, U, act=name)
    torch.cuda.synchronize()
    x, wg, wu, dh, u, g64 = (v.double() for v in (X, Wg, Wu, dH, U, G))
    value, slope = R.act(name, G)
    dG, dU = dh * u * slope, dh * value
    gate = torch.where(g64 > 0, g64, (-g64).clamp(max=0.28))
    low = 2.0 ** -38 * float(torch.maximum((dh * u).abs(), dh.abs() * gate).max())
    eG = dG.abs() * (R.unit(t) + 2.0 ** -21) + (dh * u).abs() * R.slope_bound(name, G) + low
    eU = dU.abs() * (R.unit(t) + 2.0 ** -21 + R.act_rel(name, G)) + low
    for what, y, ref, err, mag, k in (
            ("dX", dX, dG @ wg + dU @ wu, eG @ wg.abs() + eU @ wu.abs(), dG.abs() @ wg.abs() + dU.abs() @ wu.abs(), 2 * N),
            ("dWg", dWg, dG.T @ x, eG.T @ x.abs(), dG.abs().T @ x.abs(), M),
            ("dWu", dWu, dU.T @ x, eU.T @ x.abs(), dU.abs().T @ x.abs(), M)):
        bound = err * (1 + R.unit(t)) + mag * (k + 2) * 2.0 ** -24 + ref.abs() * R.unit(t) + R.tiny(t)
        d = (y.double() - ref).abs()
        assert bool((d <= bound).all()), (what, float((d / bound).max()))
