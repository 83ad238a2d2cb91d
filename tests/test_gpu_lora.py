"""GPU parity of dense_lora_gemm against a plain float64 form.

Integer cases (small integers, power-of-two scales: every product and sum is
exact in float32, the intermediate in two 16-bit parts) are compared bit for
bit with the exact sum rounded once.  Random cases: y is off by its rounding's
half step plus scale * sum_r |B| dt, where dt bounds the intermediate's error:
(K + 16) 2^-24 sum_k |A x| for a float32 sum of K products in any order, its
two-part split (2^-16 |t| in bf16, 2^-22 |t| in fp16, and 2^-24 of the row's
largest), and (R + 8) 2^-24 sum_r |B t| for the second sum."""
import numpy as np
import pytest

import gen
import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.serving_ref import HALF, TINY

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
SPLIT = {"bf16": 2.0 ** -16, "f16": 2.0 ** -22}


def f64(t):
    return t.double().cpu().numpy()


def ids_of(M, L, kind, rng):
    if kind == "prompts":  # runs of one adapter
        cuts = np.sort(rng.integers(0, M, 5))
        ids = rng.integers(-1, L, 6)[np.searchsorted(cuts, np.arange(M), side="right")]
    elif kind == "one":
        ids = np.full(M, L - 1)
    elif kind == "none":
        ids = np.full(M, -1)
    else:  # one request a row; ids out of range count as none
        ids = rng.integers(-2, L + 2, M)
    return torch.from_numpy(ids.astype(np.int32))


def case(M, K, N, R, L, kind, dt, seed, integers=False, pad=0):
    rng = np.random.default_rng(seed)

    def rnd(shape, size):
        v = rng.integers(-size, size + 1, shape).astype(np.float32) if integers else rng.standard_normal(shape)
        return torch.from_numpy(np.asarray(v, np.float32))

    x = rnd((M, K + pad), 2).to(dt).cuda()[:, :K]
    a = (rnd((L, R, K), 1) if integers else rnd((L, R, K), 1) / K ** 0.5).to(dt).cuda()
    b = (rnd((L, N, R), 2) if integers else rnd((L, N, R), 1) * 0.3).to(dt).cuda()
    y = rnd((M, N + pad), 30).to(dt).cuda()[:, :N]
    s = 2.0 ** rng.integers(-3, 3, L) if integers else rng.uniform(0.2, 2.0, L)
    return x, ids_of(M, L, kind, rng).cuda(), a, b, torch.from_numpy(s.astype(np.float32)).cuda(), y


def plain(x, ids, a, b, s, y, kind):
    """(y, its tolerance), float64."""
    x, a, b, y = f64(x), f64(a), f64(b), f64(y)
    s = np.ones(a.shape[0]) if s is None else f64(s)
    ref, lim = y.copy(), np.zeros_like(y)
    K, R = a.shape[2], a.shape[1]
    for l in range(a.shape[0]):
        m = np.flatnonzero(ids.cpu().numpy() == l)
        if not m.size:
            continue
        t = x[m] @ a[l].T
        dt = (K + 16) * 2.0 ** -24 * (np.abs(x[m]) @ np.abs(a[l]).T) + SPLIT[kind] * np.abs(t) \
            + 2.0 ** -24 * np.abs(t).max(1, keepdims=True)
        ref[m] += s[l] * (t @ b[l].T)
        lim[m] = s[l] * (dt + (R + 8) * 2.0 ** -24 * np.abs(t)) @ np.abs(b[l]).T
    return ref, lim + HALF[kind] * (np.abs(ref) + lim) + TINY[kind]


def check(M, K, N, R, L, ids, kind, seed=1, integers=False, pad=0, scaled=True):
    say("lora", M, K, N, R, L, ids, kind, integers, pad)
    x, i, a, b, s, y = case(M, K, N, R, L, ids, DT[kind], seed, integers, pad)
    s = s if scaled else None
    ref, lim = plain(x, i, a, b, s, y, kind)
    before = y.clone()
    got = wq.dense_lora_gemm(x, i, a, b, s, y)
    torch.cuda.synchronize()
    assert got is y
    what = "%d x %d x %d rank %d of %d, %s %s" % (M, K, N, R, L, ids, kind)
    none = ((i < 0) | (i >= L))
    assert torch.equal(y[none], before[none]), what
    if integers:
        assert np.array_equal(f64(y), f64(torch.from_numpy(ref).to(DT[kind]))), what
    else:
        bad = np.abs(f64(y) - ref) > lim
        assert not bad.any(), "%s: %d off, worst %.3g" % (what, bad.sum(), (np.abs(f64(y) - ref) / lim).max())


# small batches (lora.hip), then large ones (lora_wide.hip, by rows x (K + 2 N) and rank)
SHAPES = [(1, 8, 8, 8, 1), (1, 4096, 4096, 16, 1), (3, 40, 72, 8, 2), (16, 512, 256, 16, 16), (17, 136, 264, 24, 5),
          (33, 1024, 520, 64, 40), (64, 256, 1032, 72, 3), (100, 64, 64, 128, 7), (203, 520, 328, 200, 4),
          (511, 264, 200, 32, 9), (513, 264, 200, 32, 9), (700, 136, 1288, 64, 70), (1025, 72, 72, 136, 3),
          (1100, 520, 1608, 40, 6), (2500, 1000, 6664, 16, 9), (3000, 4096, 4104, 24, 5), (700, 264, 3000, 128, 3),
          (400, 264, 4000, 72, 3), (300, 520, 5000, 64, 40), (2600, 136, 6504, 32, 70)]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("ids", ["rows", "prompts", "one", "none"])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, ids, kind):
    need_gpu()
    check(*shape, ids, kind)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("ids", ["rows", "prompts"])
@pytest.mark.parametrize("shape", SHAPES)
def test_integers_exact(shape, ids, kind):
    need_gpu()
    M, K, N, R, L = shape
    if K <= 1024:
        check(M, K, N, R, L, ids, kind, integers=True, pad=8)


def test_no_scales_and_column_ranges():
    """scales None; y a column range of a wider output, whose other columns stay."""
    need_gpu()
    check(37, 512, 256, 16, 4, "rows", "bf16", scaled=False)
    x, i, a, b, s, _ = case(37, 512, 256, 16, 4, "rows", torch.bfloat16, 3)
    wide = torch.randn((37, 800), device="cuda").bfloat16()
    keep = wide.clone()
    ref, lim = plain(x, i, a, b, s, wide[:, 264:520], "bf16")
    wq.dense_lora_gemm(x, i, a, b, s, wide[:, 264:520])
    torch.cuda.synchronize()
    assert torch.equal(wide[:, :264], keep[:, :264]) and torch.equal(wide[:, 520:], keep[:, 520:])
    assert (np.abs(f64(wide[:, 264:520]) - ref) <= lim).all()


@pytest.mark.parametrize("M", [40, 600, 3001])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_adapters_and_rows_are_apart(M, kind):
    """NaN and infinities in one adapter's weights, or one row's input, reach that adapter's rows, that row, only."""
    need_gpu()
    x, i, a, b, s, y = case(M, 256, 264 if M < 3000 else 6000, 16 if M < 3000 else 56, 6, "rows", DT[kind], 5)
    ref = wq.dense_lora_gemm(x, i, a, b, s, y.clone())
    bad_a, bad_b, bad_x = a.clone(), b.clone(), x.clone()
    bad_a[2] = float("nan")
    bad_a[3, :, 7] = float("inf")
    bad_b[4] = float("inf")
    bad_x[M // 2] = float("nan")
    got = wq.dense_lora_gemm(bad_x, i, bad_a, bad_b, s, y.clone())
    torch.cuda.synchronize()
    touched = (i == 2) | (i == 3) | (i == 4)
    touched[M // 2] = True
    assert torch.equal(got[~touched], ref[~touched])
    assert bool(torch.isnan(got[i == 2]).all()) and not bool(torch.isfinite(got[i == 4]).any())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_range_of_the_intermediate(kind):
    """An intermediate beyond fp16's range, and one far below it, keep their precision."""
    need_gpu()
    x, i, a, b, s, y = case(20, 512, 128, 16, 3, "one", DT[kind], 6)
    for up, down in ((256.0, 2.0 ** -14), (2.0 ** -8, 64.0)):
        big, small = (x * up).contiguous(), (b * down).contiguous()
        wide = (a * (up if up > 1 else 1.0)).contiguous()
        y0 = torch.zeros_like(y)
        ref, lim = plain(big, i, wide, small, s, y0, kind)
        got = wq.dense_lora_gemm(big, i, wide, small, s, y0)
        torch.cuda.synchronize()
        assert (np.abs(f64(got) - ref) <= lim).all()


def test_offsets_beyond_32_bits():
    """x, y and t of more than 2^31 bytes, y of more than 2^31 values: the last rows against the plain form."""
    need_gpu()
    M, K, N, R = 70030, 16384, 32768, 8
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    tail = case(77, K, N, R, 2, "one", torch.bfloat16, 9)
    x[-77:], y[-77:] = tail[0], tail[5]
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[-77:] = tail[1]
    ids[::1000] = 0
    ref, lim = plain(tail[0], ids[-77:], *tail[2:5], tail[5], "bf16")
    wq.dense_lora_gemm(x, ids, tail[2], tail[3], tail[4], y)
    torch.cuda.synchronize()
    assert (np.abs(f64(y[-77:]) - ref) <= lim).all()
    assert not bool(y[:-77].any())


def test_dense_with_adapters_is_the_two_calls():
    need_gpu()
    K, N = 512, 384
    rng = np.random.default_rng(2)
    q8 = rng.integers(-127, 128, (1, N, K)).astype(np.int8)
    q4 = rng.integers(-8, 8, (1, N, K)).astype(np.int8)
    sc = gen.f32_to_f16_bits(rng.uniform(0.001, 0.002, (1, 1, N)).astype(np.float32))
    w8, s8 = (torch.from_numpy(t).cuda() for t in wq.pack_w8(q8, sc))
    w4, s4, _ = wq.pack_w4(q4, sc, -1)
    w4, s4 = torch.from_numpy(w4).cuda(), torch.from_numpy(s4).cuda()
    low = [(torch.randn(r, K) / K ** 0.5, torch.randn(N, r) * 0.3, 2.0 / r) for r in (4, 16, 9)]
    a, b, s = wq.pack_lora(low, torch.float16)
    assert a.shape == (3, 16, K) and b.shape == (3, N, 16)
    for M in (1, 20, 300):
        x = torch.randn((M, K)).half().cuda()
        ids = torch.from_numpy((np.arange(M) % 4 - 1).astype(np.int32)).cuda()
        lora = wq.Lora(ids, a, b, s)
        for base, both in ((wq.dense_w8a16_gemm(x, N, w8, s8), wq.dense_w8a16_gemm(x, N, w8, s8, lora=lora)),
                           (wq.dense_w4a16_gemm(x, N, w4, s4, -1), wq.dense_w4a16_gemm(x, N, w4, s4, -1, lora=lora))):
            ref, lim = plain(x, ids, a, b, s, base, "f16")
            two = wq.dense_lora_gemm(x, *lora, base.clone())
            torch.cuda.synchronize()
            assert torch.equal(both, two)
            assert (np.abs(f64(both) - ref) <= lim).all()


def test_graph_stream_and_repeats():
    """Replays with new inputs, another stream, and the same bits every time; M = 0."""
    need_gpu()
    for M, N, R in ((24, 520, 24), (900, 520, 24), (900, 2056, 64), (2000, 8200, 24), (900, 520, 200)):
        x, i, a, b, s, y = case(M, 1024, N, R, 5, "rows", torch.bfloat16, 8)
        ref = wq.dense_lora_gemm(x, i, a, b, s, y.clone())
        for _ in range(3):
            assert torch.equal(wq.dense_lora_gemm(x, i, a, b, s, y.clone()), ref)
        side = torch.cuda.Stream()
        mine = y.clone()
        side.wait_stream(torch.cuda.current_stream())
        wq.dense_lora_gemm(x, i, a, b, s, mine, stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(mine, ref)
        live, out = x.clone(), y.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            wq.dense_lora_gemm(live, i, a, b, s, out)
        for k in range(4):
            live.copy_(torch.roll(x, k, 0))
            out.copy_(y)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, wq.dense_lora_gemm(live, i, a, b, s, y.clone()))
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    wq.dense_lora_gemm(e, torch.empty(0, dtype=torch.int32, device="cuda"),
                       torch.zeros((1, 8, 64), dtype=torch.bfloat16, device="cuda"),
                       torch.zeros((1, 64, 8), dtype=torch.bfloat16, device="cuda"), None, e.clone())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("ids", ["rows", "prompts", "one"])
@pytest.mark.parametrize("shape", [(300, 1000, 5008, 24, 9), (517, 520, 3208, 32, 7), (263, 4096, 4104, 24, 33),
                                   (1001, 1032, 1056, 32, 40), (290, 136, 6504, 24, 1)])
def test_ranks_17_to_32_in_large_batches(shape, ids, kind):
    """From 3 Mi elements of x and y on they take the large-batch kernels."""
    need_gpu()
    check(*shape, ids, kind)
    if shape[1] <= 1024:
        check(*shape, ids, kind, integers=True, pad=8)


@pytest.mark.parametrize("shape", [(40, 512, 264, 24, 5), (700, 136, 1288, 64, 9)])
def test_what_the_workspace_held_does_not_matter(shape):
    """NaN in it beforehand: rows without an adapter have no intermediate, the others' is written first."""
    need_gpu()
    M, K, N, R, L = shape
    x, i, a, b, s, y = case(M, K, N, R, L, "rows", torch.bfloat16, 4)
    i[::3] = -1
    ref = wq.dense_lora_gemm(x, i, a, b, s, y.clone())
    ws = torch.full((wq.dense_lora_workspace_bytes(M, K, N, R, L),), 0xFF, dtype=torch.uint8, device="cuda")
    got = wq.dense_lora_gemm(x, i, a, b, s, y.clone(), workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(got, ref) and bool(torch.isfinite(got).all()) and torch.equal(got[::3], y[::3])
