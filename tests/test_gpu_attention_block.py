"""The attention half of a decoder block as it is served, over several decode
steps: norm -> qkv projection with its bias -> cache write -> attention -> output
projection onto the residual stream -> norm -> router -> experts; eager, against
float64, and captured with slots and lengths advanced in place.  And the new
entry points' refusal of host memory, and their streams' memory."""
import ctypes as C
import math

import numpy as np
import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.kv_ref import attention
from tests.test_gpu_serving_device_check import pinned
from tests.test_gpu_stream_memory import stream_of
from weight_only_quantized_topk_amd._lib import WqEpilogue, WqKvCache

pytestmark = pytest.mark.gpu

B, HIDDEN, HEADS, KV, D, P, WIDTH = 5, 512, 8, 2, 64, 16, 8
QKV = (HEADS + 2 * KV) * D


def int8_weight(rng, N, K):
    q = rng.integers(-127, 128, (1, N, K)).astype(np.int8)
    s = torch.from_numpy(rng.uniform(0.5, 1.5, (1, 1, N)) / (74 * math.sqrt(K))).bfloat16()
    packed, sp = wq.pack_w8(q, s.view(torch.int16).numpy().view(np.uint16))
    W = torch.from_numpy(q[0].astype(np.float64)) * s[0, 0].double()[:, None]
    return W, torch.from_numpy(packed).cuda(), torch.from_numpy(sp.view(np.int16)).cuda()


class Block:
    def __init__(self, quant, seed=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.W1, self.w1, self.s1 = int8_weight(rng, QKV, HIDDEN)
        self.W2, self.w2, self.s2 = int8_weight(rng, HIDDEN, HEADS * D)
        self.b = torch.randn(QKV, generator=g).bfloat16().cuda()
        self.n1, self.n2 = (1 + 0.1 * torch.randn((2, HIDDEN), generator=g)).bfloat16().cuda()
        codes = [torch.randint(0x20, 0x48, shape, generator=g).to(torch.uint8).numpy() for shape in
                 ((4, 2 * 256, HIDDEN), (4, HIDDEN, 256))]
        scales = [np.full(c.shape[:2], 0.02, np.float32) for c in codes]
        self.moe = wq.pack_moe_fp8(codes[0], scales[0], codes[1], scales[1], torch.bfloat16, 0.02, 0.05)
        self.gate = torch.randn((HIDDEN, 4), generator=g).cuda()
        self.cache = wq.kv_cache(B * WIDTH, KV, P, D, torch.bfloat16, quant, *((0.03, 0.03) if quant == "static" else ()))
        for t in self.cache:
            if isinstance(t, torch.Tensor):
                t.view(torch.uint8).fill_(0xFF)  # NaN in every row that is not written
        self.table = torch.randperm(B * WIDTH, generator=g).int().view(B, WIDTH).cuda()
        self.length = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.x = torch.zeros((B, HIDDEN), dtype=torch.bfloat16, device="cuda")

    def step(self):
        """One decode step on self.x, the tokens' positions in self.length."""
        at = self.length.long()
        slots = self.table.gather(1, (at // P)[:, None])[:, 0].long() * P + at % P
        n = self.length + 1
        h = wq.rms_norm(self.x, self.n1).out
        qkv = wq.dense_w8a16_gemm(h, QKV, self.w1, self.s1, bias=self.b).view(B, HEADS + 2 * KV, D)
        wq.kv_cache_write(qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:], self.cache, slots)
        a = wq.paged_attention(qkv[:, :HEADS], self.cache, self.table, n)
        y = wq.dense_w8a16_gemm(a.view(B, HEADS * D), HIDDEN, self.w2, self.s2, residual=self.x)
        z = wq.rms_norm(y, self.n2, quant="row")
        out = wq.fused_moe_fp8((z.codes, z.scales), z.out.float() @ self.gate, self.moe, topk=2)
        self.length.copy_(n)
        return qkv, a, y, out


def inputs(step, seed=3):
    return torch.randn((B, HIDDEN), generator=torch.Generator().manual_seed(100 * seed + step)).bfloat16()


@pytest.mark.parametrize("quant", [None, "row", "static"])
def test_decode_steps(quant):
    need_gpu()
    blk = Block(quant)
    blk.length.copy_(torch.tensor([0, 0, 0, 0, 0]))
    for step in range(40):
        blk.x.copy_(inputs(step))
        qkv, a, y, out = blk.step()
    torch.cuda.synchronize()
    say("decode steps", quant)
    host = [t.cpu() if isinstance(t, torch.Tensor) else t for t in blk.cache]
    want, _, tol, _ = attention(qkv[:, :HEADS].cpu(), host, blk.table.cpu(), blk.length.cpu(), D ** -0.5, 0)
    got = a.cpu().double()
    assert bool(((got - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())
    # the projections around it: sums of K products in float32 of exact codes, one rounding
    x = inputs(39).double()
    h = wq.rms_norm(inputs(39).cuda(), blk.n1).out.cpu().double()
    for src, W, add, res in ((h, blk.W1, blk.b.cpu().double(), qkv.reshape(B, QKV)), (got.reshape(B, -1), blk.W2, x, y)):
        z = src @ W.t() + add
        size = src.abs() @ W.abs().t() * (src.shape[1] + 16) * 2.0 ** -23 + z.abs() * 2.0 ** -21
        assert bool(((res.cpu().double() - z).abs() <= size + 2.0 ** -8 * (z.abs() + size)).all())
    assert bool(torch.isfinite(out.float()).all())
    # the cache's rows back
    slots = blk.table[2].long()[torch.arange(40).cuda() // P] * P + torch.arange(40).cuda() % P
    k, v = wq.kv_cache_read(blk.cache, slots, torch.bfloat16)
    assert bool(torch.isfinite(k.float()).all()) and torch.equal(k[39].float().abs() > 0, k[39] != 0)


def test_captured_steps():
    need_gpu()
    one, two = Block("row"), Block("row")
    two.x.copy_(inputs(0))
    two.step()  # (what a first call sets up stays out of the graph)
    two.length.zero_()
    for t in two.cache:
        t.view(torch.uint8).fill_(0xFF)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = two.step()
    two.length.zero_()
    for step in range(35):
        x = inputs(step)
        one.x.copy_(x)
        two.x.copy_(x)
        want = one.step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g.contiguous().view(torch.int16), w.contiguous().view(torch.int16)) for g, w in zip(held, want)), step


def c_status(fn, *args):
    st = getattr(wq.load(), fn)(*[a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args],
                                torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return st


def each_on_the_host(call, tensors, outputs):
    """call(tensors) with each of them in host memory, one at a time: refused, every output as it was."""
    assert call(tensors) == wq.WQ_OK
    for name, t in tensors.items():
        say("on the host:", name)
        for o in outputs:
            tensors[o].view(torch.uint8).fill_(7)
        assert call({**tensors, name: pinned(t)}) == wq.WQ_ERR_DEVICE, name
        assert all(bool((tensors[o].view(torch.uint8) == 7).all()) for o in outputs), name


def cache_of(t):
    return C.byref(WqKvCache(C.sizeof(WqKvCache), t["k"].data_ptr(), t["v"].data_ptr(), t["ks"].data_ptr(),
                             t["vs"].data_ptr(), 0.0, 0.0, 3, 4, 2, 16, 64))


def test_host_memory_is_refused():
    need_gpu()
    dev = "cuda"
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    cache = {"k": u8(4, 2, 16, 64), "v": u8(4, 2, 16, 64), "ks": torch.zeros((4, 2, 16), device=dev),
             "vs": torch.zeros((4, 2, 16), device=dev)}
    rows = {"nk": bf(3, 2, 64), "nv": bf(3, 2, 64), "slots": torch.tensor([1, 2, 40], device=dev)}
    each_on_the_host(lambda t: c_status("wq_kv_cache_write", cache_of(t), t["nk"], 128, t["nv"], 128, t["slots"], 3, wq.WQ_BF16),
                     {**cache, **rows}, ("k", "v", "ks", "vs"))
    each_on_the_host(lambda t: c_status("wq_kv_cache_read", cache_of(t), t["slots"], 3, t["nk"], 128, t["nv"], 128, wq.WQ_BF16),
                     {**cache, **rows}, ("nk", "nv"))
    width = 40
    att = {"q": bf(2, 4, 64), "table": torch.zeros((2, width), dtype=torch.int32, device=dev),
           "n": torch.tensor([5, 600], dtype=torch.int32, device=dev), "out": bf(2, 4, 64), "lse": torch.zeros((2, 4), device=dev),
           "ws": u8(wq.paged_attention_workspace_bytes(2, 4, 2, 64, 16, width))}
    assert att["ws"].numel() > 0
    each_on_the_host(lambda t: c_status("wq_paged_attention", cache_of(t), t["q"], 256, 2, 4, t["table"], width, t["n"], 0.1, 0,
                                        t["out"], 256, t["lse"], wq.WQ_BF16, t["ws"], t["ws"].numel()),
                     {**cache, **att}, ("out", "lse", "ws"))
    M, K, N = 200, 4096, 128
    lin = {"x": bf(M, K), "w": u8(N * K), "s": bf(N), "b": bf(N), "r": bf(M, N), "y": bf(M, N),
           "ws": u8(wq.dense_epilogue_workspace_bytes(8, M, K, N) or 256)}

    def dense(t):
        e = WqEpilogue(C.sizeof(WqEpilogue), t["b"].data_ptr(), t["r"].data_ptr(), N, 2)
        return c_status("dense_w8a16_epilogue_gemm", t["x"], M, K, N, t["w"], t["s"], C.byref(e), t["y"], wq.WQ_BF16, t["ws"],
                        t["ws"].numel())

    if wq.dense_epilogue_workspace_bytes(8, M, K, N) == 0:
        lin["ws"] = lin["y"].clone()  # (not looked at)
        lin.pop("ws")
        dense_call = lambda t: dense({**t, "ws": t["y"]})  # noqa: E731
    else:
        dense_call = dense
    each_on_the_host(dense_call, lin, ("y",))


def test_outputs_are_the_streams_memory():
    need_gpu()
    side = torch.cuda.Stream()
    cache = wq.kv_cache(40, 2, 16, 64, torch.bfloat16, "row")
    for t in cache:
        t.view(torch.uint8).zero_()
    q = torch.randn((2, 4, 64), device="cuda").bfloat16()
    table = torch.arange(80, device="cuda").int().view(2, 40) % 40
    n = torch.tensor([600, 9], dtype=torch.int32, device="cuda")
    slots = torch.arange(9, device="cuda")
    rng = np.random.default_rng(1)
    _, w, s = int8_weight(rng, 64, 512)
    x, r = torch.randn((3, 512), device="cuda").bfloat16(), torch.randn((3, 64), device="cuda").bfloat16()
    torch.cuda.synchronize()

    def run(stream=None):
        return (*wq.paged_attention(q, cache, table, n, want_lse=True, stream=stream),
                *wq.kv_cache_read(cache, slots, torch.bfloat16, stream=stream),
                wq.dense_w8a16_gemm(x, 64, w, s, residual=r, stream=stream))

    want = run()
    got = run(side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert stream_of(a) == side.cuda_stream and torch.equal(a, b)
