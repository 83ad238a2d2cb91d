"""The dense projections with bias, activation and residual on the GPU against
float64, in every regime of the dispatch.

Tolerance: products of exact codes (int4 at large batches: code times scale
rounded to fp16, 2^-11 of each weight) summed in float32 in any order, (K + 16) 2^-23 of
sum |x w|; the activations have slopes below 1.2 and are evaluated to (|z| + 4) |z| 2^-21
(the exponential's argument is rounded); additions 2^-22; one rounding."""
import math

import numpy as np
import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.serving_ref import HALF, TINY

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]
_weights = {}


def weights(bits, group, act, N, K, act_order=False):
    """(float64 W [N, K], packed tensors) made once for a shape."""
    key = (bits, group, act, N, K, act_order)
    if key not in _weights:
        rng = np.random.default_rng(N * 7 + K + bits)
        dt = TYPES[act]
        q = rng.integers(-8 if bits == 4 else -127, 8 if bits == 4 else 128, (1, N, K)).astype(np.int8)
        G = K // 128 if group == 128 else 1
        s = torch.from_numpy(rng.uniform(0.005, 0.02, (1, G, N)) / (1 if bits == 4 else 16)).to(dt)
        sb = s.view(torch.int16).numpy().view(np.uint16)
        gi = (rng.permutation(K) // 128).astype(np.int32)[None] if act_order else None
        kp = None
        if bits == 4:
            packed, sp, kp = wq.pack_w4(q, sb, group, g_idx=gi)
        else:
            packed, sp = wq.pack_w8(q, sb)
        of = gi[0] if act_order else np.arange(K) // (128 if group == 128 else K)
        W = torch.from_numpy(q[0].astype(np.float64)) * s[0].double()[torch.from_numpy(np.asarray(of)).long()].t()
        _weights[key] = (W, torch.from_numpy(packed).cuda(), torch.from_numpy(sp.view(np.int16)).cuda(),
                         None if kp is None else torch.from_numpy(kp).cuda())
    return _weights[key]


def f64(z, act):
    if act == "relu":
        return torch.where(z < 0, 0.0, z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def check(bits, group, act, M, N, K, bias, activation, residual, act_order=False, seed=0):
    need_gpu()
    say("dense epilogue", bits, group, act, M, N, K, bias, activation, residual)
    W, wp, sp, kp = weights(bits, group, act, N, K, act_order)
    g = torch.Generator().manual_seed(seed + M)
    dt = TYPES[act]
    x = torch.randn((M, K), generator=g).to(dt)
    b = torch.randn(N, generator=g).to(dt) if bias else None
    r = torch.randn((M, N), generator=g).to(dt)
    how = {"bias": None if b is None else b.cuda(), "activation": activation}
    out = None
    if residual == "strided":
        wide = torch.full((M, N + 24), 9.0, dtype=dt, device="cuda")
        wide[:, 8:8 + N] = r.cuda()
        how["residual"] = wide[:, 8:8 + N]
    elif residual == "in place":
        out = how["residual"] = r.cuda()
    elif residual:
        how["residual"] = r.cuda()
    call = (lambda **k: wq.dense_w4a16_gemm(x.cuda(), N, wp, sp, group, kp, **k)) if bits == 4 else (
        lambda **k: wq.dense_w8a16_gemm(x.cuda(), N, wp, sp, **k))
    y = call(out=out, **how)
    torch.cuda.synchronize()
    assert out is None or y is out
    z = x.double() @ W.t()
    size = x.double().abs() @ W.abs().t()
    tol = size * ((K + 16) * 2.0 ** -23 + (2.0 ** -11 if bits == 4 and M > 128 else 0))
    if b is not None:
        z = z + b.double()
    tol = tol + z.abs() * 2.0 ** -22
    if activation:
        tol = 1.2 * tol + (z.abs() + 4) * z.abs() * 2.0 ** -21
    want = f64(z, activation)
    if residual:
        want = want + r.double()
        tol = tol + (want.abs() + r.double().abs()) * 2.0 ** -22
    off = (y.cpu().double() - want).abs()
    assert bool((off <= tol + HALF[act] * (want.abs() + tol) + TINY[act]).all()), float((off - tol).max())


KINDS = {"w4": (4, 128, "f16", False), "w4pc": (4, -1, "f16", False), "w4ao": (4, 128, "f16", True),
         "w8b": (8, -1, "bf16", False), "w8h": (8, -1, "f16", False)}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("M", [1, 2, 3, 16, 17, 33, 64, 65, 128, 129, 150, 192, 193, 300])
def test_rows(kind, M):
    bits, group, act, ao = KINDS[kind]
    check(bits, group, act, M, 400, 512, True, ACTS[M % 5], True, act_order=ao)


@pytest.mark.parametrize("kind", ["w4", "w8b"])
@pytest.mark.parametrize("N", [16, 48, 128, 512, 1040])
@pytest.mark.parametrize("M", [1, 29, 100, 161, 257])
def test_widths(kind, N, M):
    bits, group, act, ao = KINDS[kind]
    check(bits, group, act, M, N, 256, False, "silu", True)


@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("M", [2, 40, 200])
@pytest.mark.parametrize("bias,residual", [(True, None), (False, True), (True, "strided"), (True, "in place")])
def test_forms(activation, M, bias, residual):
    check(8, -1, "bf16", M, 208, 320, bias, activation, residual)
    check(4, 128, "f16", M, 208, 384, bias, activation, residual)


@pytest.mark.parametrize("kind", ["w4", "w8b", "w8h"])
@pytest.mark.parametrize("M,N,K", [(200, 128, 4096), (513, 528, 4096), (140, 1024, 8192), (29, 4096, 4096), (1, 6144, 4096),
                                   (5, 16, 8192), (64, 256, 4096), (2, 48, 28672), (100, 272, 7168)])
def test_long_sums(kind, M, N, K):
    bits, group, act, ao = KINDS[kind]
    check(bits, group, act, M, N, K, True, None, "in place")


@pytest.mark.parametrize("kind", ["w4", "w8b"])
@pytest.mark.parametrize("M,N,K", [(129, 1040, 128), (200, 32992, 128), (300, 32992, 128), (520, 32992, 256), (1000, 16400, 1024),
                                   (129, 1040, 8192), (129, 8208, 4096), (200, 8208, 2048), (1000, 1040, 4096), (129, 2064, 1024),
                                   (1000, 528, 1024), (4096, 144, 1024), (16, 20480, 256), (32, 20480, 256), (100, 20480, 256),
                                   (7, 20480, 256)])
def test_plans(kind, M, N, K):
    """Every tile shape, split of K and cut by columns of the dispatch, ends of rows and columns within them."""
    bits, group, act, ao = KINDS[kind]
    check(bits, group, act, M, N, K, True, "relu", "in place" if M % 2 else "strided")
    _weights.clear()


def test_values_that_overflow():
    """A sum beyond the type's range, an infinite bias, a NaN in one row of x: each in its own outputs."""
    need_gpu()
    N, K = 64, 256
    W, wp, sp, _ = weights(8, -1, "f16", N, K)
    for M in (2, 30, 200):
        x = torch.zeros((M, K), dtype=torch.float16)
        x[0] = 60000.0
        x[M - 1, 3] = float("nan")
        b = torch.zeros(N, dtype=torch.float16)
        b[5] = float("inf")
        for activation in (None, "relu"):
            y = wq.dense_w8a16_gemm(x.cuda(), N, wp, sp, bias=b.cuda(), activation=activation).cpu()
            big = x[0].double() @ W.t()
            want = big.clamp(min=0) if activation else big
            want[5] = math.inf
            over = want.abs() > 66000
            assert torch.equal(torch.isinf(y[0]), over)
            assert bool(torch.isnan(y[M - 1]).all())
            if M > 2:
                assert float(y[1, 5]) == math.inf and bool((y[1, :5] == 0).all())


@pytest.mark.parametrize("M", [1, 20, 100, 300])
def test_streams_and_graphs(M):
    need_gpu()
    N, K = 400, 512
    _, wp, sp, _ = weights(4, 128, "f16", N, K)
    g = torch.Generator().manual_seed(M)
    x, r = torch.randn((M, K), generator=g).half().cuda(), torch.randn((M, N), generator=g).half().cuda()
    b = torch.randn(N, generator=g).half().cuda()
    how = {"bias": b, "activation": "gelu", "residual": r}
    want = wq.dense_w4a16_gemm(x, N, wp, sp, **how)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        one = wq.dense_w4a16_gemm(x, N, wp, sp, **how)
        two = wq.dense_w4a16_gemm(x, N, wp, sp, stream=side.cuda_stream, **how)
        torch.cuda.synchronize()
        assert torch.equal(one, want) and torch.equal(two, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = wq.dense_w4a16_gemm(x, N, wp, sp, **how)
    for k in range(3):
        x.copy_(torch.roll(x, 1, 1))
        graph.replay()
        torch.cuda.synchronize()
        got = held.clone()
        assert torch.equal(got, wq.dense_w4a16_gemm(x, N, wp, sp, **how))


def test_with_adapters():
    """The adapters come after the epilogue: y = x W^T + bias + residual, then the rows' adapters."""
    need_gpu()
    M, N, K = 20, 400, 512
    _, wp, sp, _ = weights(8, -1, "bf16", N, K)
    g = torch.Generator().manual_seed(4)
    x, r = torch.randn((M, K), generator=g).bfloat16().cuda(), torch.randn((M, N), generator=g).bfloat16().cuda()
    b = torch.randn(N, generator=g).bfloat16().cuda()
    lora = wq.Lora(torch.randint(-1, 3, (M,), generator=g).int().cuda(), torch.randn((3, 16, K), generator=g).bfloat16().cuda(),
                   torch.randn((3, N, 16), generator=g).bfloat16().cuda(), None)
    y = wq.dense_w8a16_gemm(x, N, wp, sp, bias=b, residual=r, lora=lora)
    z = wq.dense_lora_gemm(x, *lora, wq.dense_w8a16_gemm(x, N, wp, sp, bias=b, residual=r))
    assert torch.equal(y, z)
