"""Calls with stream=, on inputs that are ready: a call on the current stream and
one on another, neither waiting for the other, have memory of their own."""
import numpy as np
import pytest

import gen
import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, torch

pytestmark = pytest.mark.gpu


def stream_of(t):
    """The stream whose memory a tensor's block was taken from."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


def inputs(seed, M, K=1024, N=2048, R=64, L=4):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=g).bfloat16().cuda()

    return {"x": rnd(M, K), "r": rnd(M, K), "logits": torch.randn(M, 64, generator=g).cuda(), "y": rnd(M, N),
            "lora": (torch.randint(-1, L, (M,), generator=g).int().cuda(), rnd(L, R, K) * 0.05, rnd(L, N, R), None)}


def run(d, stream=None):
    n = wq.rms_norm(d["x"], residual=d["r"], quant="row", stream=stream)
    z = wq.dense_lora_gemm(d["x"], *d["lora"], d["y"], stream=stream)
    return (*n, z, *wq.moe_route_grouped_align(d["logits"], 4, 16, scoring="sigmoid", stream=stream),
            *wq.moe_route_grouped(d["logits"], 4, stream=stream), *wq.moe_route(d["logits"], 4, stream=stream))


def test_outputs_are_the_streams_memory():
    need_gpu()
    side = torch.cuda.Stream()
    d = inputs(1, 33)
    torch.cuda.synchronize()
    got = run(d, side.cuda_stream)
    q, s = wq.quantize_w8(d["x"][:32].t(), stream=side.cuda_stream)
    side.synchronize()
    for t in (*got, q, s):
        if t is not d["y"]:
            assert stream_of(t) == side.cuda_stream
    want = wq.quantize_w8(d["x"][:32].t().contiguous())
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])


@pytest.mark.parametrize("M", [64, 2000])
def test_two_streams_that_do_not_wait(M):
    need_gpu()
    want = []
    for seed in (1, 2):
        want.append([t.clone() for t in run(inputs(seed, M))])
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        one, two = inputs(1, M), inputs(2, M)
        torch.cuda.synchronize()
        got1 = run(one)
        got2 = run(two, side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got1, want[0]))
        assert all(torch.equal(a, b) for a, b in zip(got2, want[1]))
        del got1, got2


def test_dense_with_adapters_and_a_layer():
    """The dense projection's workspace and output, and a layer call's buffers."""
    need_gpu()
    rng = np.random.default_rng(5)
    M, K, N, R, L = 96, 512, 512, 16, 3
    q = rng.integers(-127, 128, (1, N, K)).astype(np.int8)
    s = (rng.random((1, 1, N)) * 0.01 + 0.001).astype(np.float16).view(np.uint16)
    wp, sp = wq.pack_w8(q, s)
    wp, sp = torch.from_numpy(wp).cuda(), torch.from_numpy(sp.view(np.int16)).cuda()
    spec = gen.CFG1
    wts, toks = gen.make_moe_weights(spec), gen.make_tokens(spec, 24)
    p = wq.pack_moe(4, wts.w1q, wts.s1, wts.w2q, wts.s2, torch.float16, 128)
    mx, lg = torch.from_numpy(toks.x.view(np.int16)).cuda().view(torch.float16), torch.from_numpy(toks.logits).cuda()
    xs = [torch.from_numpy(rng.standard_normal((M, K)).astype(np.float16)).cuda() for _ in range(2)]
    lora = wq.Lora(torch.from_numpy(rng.integers(-1, L, M).astype(np.int32)).cuda(),
                   torch.from_numpy((rng.standard_normal((L, R, K)) * 0.05).astype(np.float16)).cuda(),
                   torch.from_numpy(rng.standard_normal((L, N, R)).astype(np.float16)).cuda(), None)

    def both(x, stream=None):
        return wq.dense_w8a16_gemm(x, N, wp, sp, lora=lora, stream=stream), wq.fused_moe(mx, lg, p, spec.topk, stream=stream)

    want = []
    for x in xs:
        want.append([t.clone() for t in both(x)])
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        got = [both(xs[0]), both(xs[1], side.cuda_stream)]
        torch.cuda.synchronize()
        assert stream_of(got[1][0]) == stream_of(got[1][1]) == side.cuda_stream
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_default_stream_by_its_handle():
    """stream=0 with another stream current."""
    need_gpu()
    d = inputs(3, 65)
    torch.cuda.synchronize()
    want = [t.clone() for t in run(d)]
    torch.cuda.synchronize()
    d = inputs(3, 65)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = run(d, 0)
        torch.cuda.synchronize()
        assert all(stream_of(t) == 0 for t in got)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_stream_forked_in_a_capture():
    """Calls on a second stream of a captured graph, replayed with new inputs, eager work between."""
    need_gpu()
    d = inputs(4, 200)
    y0, x0 = d["y"].clone(), d["x"].clone()
    side = torch.cuda.Stream()
    run(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        two = wq.rms_norm(d["r"], quant="row")
        held = run(d, side.cuda_stream)
        here.wait_stream(side)
    for k in range(4):
        d["x"].copy_(torch.roll(x0, k, 0))
        d["y"].copy_(y0)
        graph.replay()
        torch.cuda.synchronize()
        got, got2 = [t.clone() for t in held], [t.clone() for t in two if t is not None]
        d["y"].copy_(y0)
        assert all(torch.equal(a, b) for a, b in zip(got, run(d)))
        assert all(torch.equal(a, b) for a, b in zip(got2, [t for t in wq.rms_norm(d["r"], quant="row") if t is not None]))
