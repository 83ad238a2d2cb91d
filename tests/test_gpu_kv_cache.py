"""kv_cache_write and kv_cache_read on the GPU: every step is one float32
operation, so codes, scales and values are compared bit for bit."""
import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.kv_ref import F8, TYPES, quantise

pytestmark = pytest.mark.gpu


def make(act, quant, pages, H, P, D, seed=0):
    """A cache on the device full of known bytes, and its copy on the host."""
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[act]
    if quant is None:
        c = [torch.randn((pages, H, P, D), generator=g).to(dt) for _ in range(2)] + [None, None]
    else:
        c = [torch.randint(0, 0x7F, (pages, H, P, D), generator=g).to(torch.uint8) for _ in range(2)]
        c += [torch.rand((pages, H, P), generator=g) + 0.5 for _ in range(2)] if quant == "row" else [0.02, 0.013]
    return wq.KVCache(*[t.cuda() if isinstance(t, torch.Tensor) else t for t in c]), c


def bits(t):
    return t.cpu().contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2
                                     else torch.int32)


def put(host, k, v, slots, quant):
    P = host[0].shape[2]
    ok = (slots >= 0) & (slots < host[0].shape[0] * P)
    page, slot = slots[ok] // P, slots[ok] % P
    for i, rows in enumerate((k, v)):
        if quant is None:
            host[i][page, :, slot] = rows[ok]
        else:
            codes, c = quantise(rows[ok], quant, host[2 + i])
            host[i][page, :, slot] = codes
            if quant == "row":
                host[2 + i][page, :, slot] = c


def same(dev, host):
    for d, h in zip(dev, host):
        if isinstance(h, torch.Tensor):
            a, b = bits(d), bits(h)
            if h.dtype == torch.uint8:  # a NaN's code of either sign
                a, b = torch.where((a & 0x7F) == 0x7F, 0x7F, a), torch.where((b & 0x7F) == 0x7F, 0x7F, b)
            assert torch.equal(a, b)


@pytest.mark.parametrize("quant", [None, "row", "static"])
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,P,D", [(1, 8, 16, 128), (2, 1, 16, 16), (61, 3, 48, 96), (257, 2, 64, 256), (1000, 4, 32, 64),
                                     (33, 5, 16, 80), (40, 2, 4096, 240), (0, 2, 16, 64)])
def test_write_and_read(act, quant, T, H, P, D):
    need_gpu()
    say("kv cache", act, quant, T, H, P, D)
    g = torch.Generator().manual_seed(T + D)
    pages = max(3, -(-T // P) + 2)
    cache, host = make(act, quant, pages, H, P, D)
    qkv = (torch.randn((T, 3 * H, D), generator=g) * torch.exp(2 * torch.randn((T, 3 * H, 1), generator=g))).to(TYPES[act])
    slots = torch.randperm(pages * P, generator=g)[:T]
    if T > 4:
        slots[::5] = torch.tensor([-1, pages * P, -(2 ** 40), 2 ** 40, pages * P + 7])[torch.arange(len(slots[::5])) % 5]
    d = qkv.cuda()
    got = wq.kv_cache_write(d[:, H:2 * H], d[:, 2 * H:], cache, slots.cuda())
    assert got is cache
    put(host, qkv[:, H:2 * H], qkv[:, 2 * H:], slots, quant)
    torch.cuda.synchronize()
    same(cache, host)

    k, v = wq.kv_cache_read(cache, slots.cuda(), TYPES[act])
    wide = torch.full((T, 3 * H, D), 7.0, dtype=TYPES[act], device="cuda")
    wq.kv_cache_read(cache, slots.cuda(), TYPES[act], k=wide[:, :H], v=wide[:, H:2 * H])
    torch.cuda.synchronize()
    ok = (slots >= 0) & (slots < pages * P)
    for i, r in enumerate((k, v)):
        want = torch.zeros((T, H, D), dtype=TYPES[act])
        page, slot = slots[ok] // P, slots[ok] % P
        rows = host[i][page, :, slot]
        if quant is not None:
            c = host[2 + i][page, :, slot][..., None] if quant == "row" else torch.tensor(host[2 + i])
            rows = (rows.view(F8).float() * c).to(TYPES[act])
        want[ok] = rows
        assert torch.equal(bits(r), bits(want))
        assert torch.equal(bits(wide[:, i * H:(i + 1) * H]), bits(want))
    assert bool((wide[:, 2 * H:] == 7).all())


@pytest.mark.parametrize("quant", ["row", "static"])
def test_values_beyond_the_codes(quant):
    """Zeros, subnormals, the largest values, infinities and NaN: their own rows only."""
    need_gpu()
    cache, host = make("bf16", quant, 2, 1, 16, 32)
    x = torch.zeros((8, 1, 32))
    x[1] = 1e-38
    x[2] = 3e38
    x[3, 0, 5] = float("inf")
    x[4, 0, 7] = float("nan")
    x[4, 0, 9] = 3.0
    x[5] = -448.0
    x[6, 0, ::2] = -float("inf")
    x[7] = torch.linspace(-2, 2, 32)
    x = x.bfloat16()
    slots = torch.arange(8) + 3
    wq.kv_cache_write(x.cuda(), x.flip(0).contiguous().cuda(), cache, slots.cuda())
    put(host, x, x.flip(0), slots, quant)
    torch.cuda.synchronize()
    same(cache, host)


def test_far_offsets():
    """Rows beyond 2^32 bytes and 2^31 elements from the cache's beginning."""
    need_gpu()
    H, P, D = 8, 64, 128
    pages = (5 << 30) // (H * P * D * 2)
    cache = wq.kv_cache(pages, H, P, D, torch.bfloat16)
    x = torch.randn((20, H, D)).bfloat16().cuda()
    slots = (torch.arange(20) * 3 + (pages - 1) * P).cuda()
    wq.kv_cache_write(x, -x, cache, slots)
    k, v = wq.kv_cache_read(cache, slots, torch.bfloat16)
    assert torch.equal(k, x) and torch.equal(v, -x)
    flat = cache.k.view(-1)
    at = ((pages - 1) * H * P + 0) * D
    assert torch.equal(flat[at:at + D], x[0, 0])


def test_the_same_slot_read_twice_and_graph_and_stream():
    need_gpu()
    cache, _ = make("f16", "row", 4, 2, 16, 64)
    slots = torch.tensor([5, 5, 63, -1, 0, 5]).cuda()
    want = wq.kv_cache_read(cache, slots, torch.float16)
    torch.cuda.synchronize()
    assert torch.equal(want[0][0], want[0][1]) and torch.equal(want[0][0], want[0][5])
    side = torch.cuda.Stream()
    got = wq.kv_cache_read(cache, slots, torch.float16, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = torch.randn((6, 2, 64), device="cuda").half()
    y = torch.randn((6, 2, 64), device="cuda").half()
    to = torch.tensor([1, 2, 40, -1, 7, 9]).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.kv_cache_write(x, y, cache, to)
        held = wq.kv_cache_read(cache, to, torch.float16)
    for k in range(3):
        x.copy_(torch.randn((6, 2, 64), device="cuda").half())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        host = [t.cpu() if isinstance(t, torch.Tensor) else t for t in cache]
        wq.kv_cache_write(x, y, cache, to)
        torch.cuda.synchronize()
        same(cache, host)
        assert all(torch.equal(a, b) for a, b in zip(got, wq.kv_cache_read(cache, to, torch.float16)))


@pytest.mark.parametrize("quant", [None, "row", "static"])
def test_two_tokens_with_one_slot(quant):
    """Of the two either's values are kept, and the other rows are their own."""
    need_gpu()
    x = torch.randn((40, 3, 80), generator=torch.Generator().manual_seed(5)).half()
    slots = torch.arange(40)
    slots[31] = 2
    cache, host = make("f16", quant, 4, 3, 16, 80)
    wq.kv_cache_write(x.cuda(), -x.cuda(), cache, slots.cuda())
    one, _ = make("f16", quant, 4, 3, 16, 80)
    rest = slots.clone()
    rest[31] = -1
    wq.kv_cache_write(x.cuda(), -x.cuda(), one, rest.cuda())
    other, _ = make("f16", quant, 4, 3, 16, 80)
    rest[2], rest[31] = -1, 2
    wq.kv_cache_write(x.cuda(), -x.cuda(), other, rest.cuda())
    for a, b, c in zip(cache, one, other):
        if isinstance(a, torch.Tensor):
            eq_b, eq_c = bits(a) == bits(b), bits(a) == bits(c)
            assert bool((eq_b | eq_c).all())
            eq_b[0, :, 2] = True
            assert bool(eq_b.all())
