"""moe_fp8_codes_gemm and the layer on E4M3 rows: against moe_fp8_w8a8_gemm on
the same codes bit for bit (the kernels and their sums are the same), and the
chain rms_norm -> router -> FP8 layer against a plain float64 form within the
layer's float tolerance."""
import numpy as np
import pytest

import gen
import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.helpers import assert_close_fp
from tests.serving_ref import e4m3_values, rms_norm, route

pytestmark = pytest.mark.gpu

SPEC = gen.CFG_FP8.with_(name="fp8-codes", E=8, topk=2, K=512, N=384)
_made = {}


def setup():
    if not _made:
        wts = gen.make_fp8_weights(SPEC, seed_config=1501)
        _made["it"] = wts, wq.pack_moe_fp8(wts.w1, wts.s1, wts.w2, wts.s2, torch.bfloat16, SPEC.a1, SPEC.a2)
    return _made["it"]


def batch(M, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (M, SPEC.K)).astype(np.uint8)
    codes[(codes & 0x7F) >= 0x70] &= 0x8F  # no NaN, and nothing above 28
    ids = np.stack([rng.permutation(SPEC.E)[:SPEC.topk] for _ in range(M)]).astype(np.int32)
    return codes, torch.from_numpy(ids).cuda()


def call(stage, p, x, row_scales, ids, bs, in_scale):
    """The stage on codes (uint8) or on 16-bit values."""
    M = x.shape[0]
    cap = wq.moe_align_capacity(M, SPEC.topk, SPEC.E, bs)
    st, ex, nt = wq.moe_align(ids, SPEC.E, bs, cap)
    out = (torch.zeros((cap, SPEC.N), dtype=torch.uint8, device="cuda") if stage == wq.WQ_STAGE_GATE_UP
           else torch.zeros((M * SPEC.topk, 2 * SPEC.N), device="cuda"))
    common = (M, SPEC.topk, SPEC.E, 2 * SPEC.N, SPEC.K, p.w1, p.s1, st, ex, nt, cap, bs)
    if x.dtype == torch.uint8:
        wq.moe_fp8_codes_gemm(stage, x, row_scales, *common, out, in_scale=in_scale, out_scale=SPEC.a2)
    else:
        ws = wq.moe_fp8_gemm_workspace_bytes(stage, M, SPEC.topk, SPEC.E, 2 * SPEC.N, SPEC.K)
        work = torch.empty(ws, dtype=torch.uint8, device="cuda")
        wq.moe_fp8_w8a8_gemm(stage, x, *common, None, out, work, in_scale, SPEC.a2)
    torch.cuda.synchronize()
    return out, st


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 16, 77, 300])
def test_equals_the_quantising_call(M, bs):
    """Rows with scales 2^-4 .. 2^-2: each row has the bits of the quantising call with that scale on codes * scale
    (exact in bf16); one scale for all likewise."""
    need_gpu()
    wts, p = setup()
    codes, ids = batch(M, M + bs)
    dev = torch.from_numpy(codes).cuda()
    value = torch.from_numpy(e4m3_values(codes)).cuda()
    which = np.arange(M) % 3
    scales = np.float32([2.0 ** -4, 2.0 ** -3, 2.0 ** -2])
    rows = torch.from_numpy(scales[which]).cuda()
    for stage in (wq.WQ_STAGE_GATE_UP, wq.WQ_STAGE_RAW):
        say("codes", M, bs, stage)
        got, st = call(stage, p, dev, rows, ids, bs, 1.0)
        token = np.minimum(st.cpu().numpy() // SPEC.topk, M) if stage == wq.WQ_STAGE_GATE_UP else np.arange(M * SPEC.topk) // SPEC.topk
        for k, s in enumerate(scales):
            ref, _ = call(stage, p, (value * float(s)).bfloat16(), None, ids, bs, float(s))
            one, _ = call(stage, p, dev, None, ids, bs, float(s))
            of = torch.from_numpy(np.append(which, -1)[token] == k).cuda()
            if M > 1 or stage == wq.WQ_STAGE_RAW:
                assert torch.equal(one, ref) and torch.equal(got[of], ref[of])
            else:  # one token: the quantising call has a launch shape of its own, whose sums may round apart
                d = np.abs(e4m3_values(one.cpu().numpy()) - e4m3_values(ref.cpu().numpy()))
                assert (d <= np.abs(e4m3_values(ref.cpu().numpy())) / 8 + 2.0 ** -9).all()
                assert torch.equal(one[of], got[of])
        if stage == wq.WQ_STAGE_GATE_UP:
            pad = torch.from_numpy(token == M).cuda()
            assert not bool(got[pad].any())


@pytest.mark.parametrize("M,N", [(300, 256), (4300, 256), (2200, 512), (9001, 256), (2200, 1280), (50001, 256)])
def test_large_batch_shapes_equal_the_quantising_call(M, N):
    """Each tile shape of the 128-row blocks (by the number of tiles), with one power-of-two scale a row."""
    need_gpu()
    E, K, topk, bs = 8, 128, 2, 128
    g = torch.Generator().manual_seed(M)
    w = torch.randint(0, 256, (E, 2 * N, K), generator=g, dtype=torch.uint8).numpy()
    w[(w & 0x7F) >= 0x60] &= 0x8F
    wp, sp = wq.pack_fp8(w, np.full((E, 2 * N), 2.0 ** -6, np.float32), interleave_gate_up=True)
    wp, sp = torch.from_numpy(wp).cuda(), torch.from_numpy(sp).cuda()
    codes = torch.randint(0, 256, (M, K), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) >= 0x70] &= 0x8F
    value = torch.from_numpy(e4m3_values(codes.numpy())).cuda()
    codes = codes.cuda()
    ids = torch.argsort(torch.rand((M, E), generator=g), dim=1)[:, :topk].int().cuda()
    cap = wq.moe_align_capacity(M, topk, E, bs)
    st, ex, nt = wq.moe_align(ids, E, bs, cap)
    say("shapes", M, N, cap)
    got, ref = torch.zeros((2, cap, N), dtype=torch.uint8, device="cuda")
    common = (M, topk, E, 2 * N, K, wp, sp, st, ex, nt, cap, bs)
    wq.moe_fp8_codes_gemm(wq.WQ_STAGE_GATE_UP, codes, torch.full((M,), 0.125, device="cuda"), *common, got, out_scale=0.5)
    work = torch.empty(M * K + 256, dtype=torch.uint8, device="cuda")
    wq.moe_fp8_w8a8_gemm(wq.WQ_STAGE_GATE_UP, (value * 0.125).bfloat16(), *common, None, ref, work, 0.125, 0.5)
    torch.cuda.synchronize()
    assert bool(got.any()) and torch.equal(got, ref)


@pytest.mark.parametrize("bs", [128, 256])
@pytest.mark.parametrize("stage", [wq.WQ_STAGE_GATE_UP, wq.WQ_STAGE_RAW])
def test_tiles_by_xcd_under_uneven_routing(stage, bs):
    """The ordered 64-row tiles: an expert with nearly all rows, one with one, one with none, blocks of several tiles,
    a buffer larger than needed, an odd number of K steps."""
    need_gpu()
    M, N, E, K, topk = 1500, 1280, 4, 384, 2
    g = torch.Generator().manual_seed(bs)
    w = torch.randint(0, 256, (E, 2 * N, K), generator=g, dtype=torch.uint8).numpy()
    w[(w & 0x7F) >= 0x60] &= 0x8F
    wp, sp = wq.pack_fp8(w, np.full((E, 2 * N), 2.0 ** -6, np.float32), interleave_gate_up=stage == wq.WQ_STAGE_GATE_UP)
    wp, sp = torch.from_numpy(wp).cuda(), torch.from_numpy(sp).cuda()
    codes = torch.randint(0, 256, (M, K), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) >= 0x70] &= 0x8F
    value = torch.from_numpy(e4m3_values(codes.numpy())).cuda()
    codes = codes.cuda()
    ids = torch.tensor([2, 0], dtype=torch.int32).repeat(M, 1)
    ids[700, 1] = 3
    ids = ids.cuda()
    cap = wq.moe_align_capacity(M, topk, E, bs) + 5 * bs
    st, ex, nt = wq.moe_align(ids, E, bs, cap)
    say("by xcd", stage, bs, cap)
    if stage == wq.WQ_STAGE_GATE_UP:
        got, ref = torch.full((2, cap, N), 0x55, dtype=torch.uint8, device="cuda")
    else:
        got, ref = torch.full((2, M * topk, 2 * N), 7.0, device="cuda")
    common = (M, topk, E, 2 * N, K, wp, sp, st, ex, nt, cap, bs)
    wq.moe_fp8_codes_gemm(stage, codes, None, *common, got, in_scale=0.125, out_scale=0.5)
    work = torch.empty(wq.moe_fp8_gemm_workspace_bytes(stage, M, topk, E, 2 * N, K), dtype=torch.uint8, device="cuda")
    wq.moe_fp8_w8a8_gemm(stage, (value * 0.125).bfloat16(), *common, None, ref, work, 0.125, 0.5)
    torch.cuda.synchronize()
    used = int(nt)
    if stage == wq.WQ_STAGE_GATE_UP:
        assert torch.equal(got[:used], ref[:used]) and bool((got[used:] == 0x55).all())
    else:
        assert torch.equal(got, ref)


@pytest.mark.parametrize("bs", [16, 128])
def test_nan_rows_stay_their_own(bs):
    need_gpu()
    wts, p = setup()
    codes, ids = batch(40, 3)
    rows = torch.full((40,), 0.125, device="cuda")
    ref, st = call(wq.WQ_STAGE_GATE_UP, p, torch.from_numpy(codes).cuda(), rows, ids, bs, 1.0)
    codes[7, 5] = 0x7F
    rows[9] = float("nan")
    got, _ = call(wq.WQ_STAGE_GATE_UP, p, torch.from_numpy(codes).cuda(), rows, ids, bs, 1.0)
    token = np.minimum(st.cpu().numpy() // SPEC.topk, 40)
    hit = torch.from_numpy((token == 7) | (token == 9)).cuda()
    assert torch.equal(got[~hit], ref[~hit])
    assert np.isnan(e4m3_values(got[hit].cpu().numpy())).all()


def layer_plain(wts, x, w, ids):
    """float64 FP8 layer on dequantised rows x (H quantised to E4M3 with a2)."""
    W1 = e4m3_values(wts.w1) * wts.s1.reshape(SPEC.E, 2 * SPEC.N, 1)
    W2 = e4m3_values(wts.w2) * wts.s2.reshape(SPEC.E, SPEC.K, 1)
    out = np.zeros((x.shape[0], SPEC.K))
    for m in range(x.shape[0]):
        for j in range(ids.shape[1]):
            z = W1[ids[m, j]] @ x[m]
            h = z[:SPEC.N] / (1 + np.exp(-z[:SPEC.N])) * z[SPEC.N:]
            q = torch.from_numpy((h / SPEC.a2).clip(-448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
            out[m] += w[m, j] * (W2[ids[m, j]] @ (q * SPEC.a2))
    return out


@pytest.mark.parametrize("quant", ["row", "static"])
@pytest.mark.parametrize("M", [1, 5, 33, 200])
def test_norm_router_layer(M, quant):
    """rms_norm (residual, codes) -> logits of its 16-bit output -> grouped router -> FP8 layer, eager and captured."""
    need_gpu()
    wts, p = setup()
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, SPEC.K), generator=g).bfloat16().cuda()
    r = torch.randn((M, SPEC.K), generator=g).bfloat16().cuda()
    nw = (1 + 0.1 * torch.randn(SPEC.K, generator=g)).bfloat16().cuda()
    gate = (torch.randn((SPEC.E, SPEC.K), generator=g) / SPEC.K ** 0.5).cuda()
    router = wq.Router("sigmoid", 0.05 * torch.randn(SPEC.E, generator=g).cuda(), 4, 2, "top2", True, 2.5)
    run = wq.Fp8MoERunner(p, M, SPEC.topk, router=router)

    def step():
        n = wq.rms_norm(x, nw, 1e-6, residual=r, quant=quant, scale=SPEC.a1 if quant == "static" else None)
        logits = n.out.float() @ gate.t()
        return n, logits, run((n.codes, n.scales), logits)

    n, logits, out = step()
    torch.cuda.synchronize()
    w_ref, ids_ref = route(logits.double().cpu().numpy(), SPEC.topk, "sigmoid", router.bias.double().cpu().numpy(), 4, 2,
                           "top2", True, 2.5)
    assert np.array_equal(run.ids.cpu().numpy(), ids_ref)
    rows = e4m3_values(n.codes.cpu().numpy()) * (n.scales.double().cpu().numpy()[:, None] if quant == "row" else SPEC.a1)
    # the codes stand for the norm's output: half a step (2^-4) and the row's smallest step
    _, y = rms_norm(x.double().cpu().numpy(), r.double().cpu().numpy(), nw.double().cpu().numpy(), 1e-6)
    step_ = rows.max() if quant == "static" else n.scales.double().cpu().numpy()[:, None]
    assert (np.abs(rows - y) <= np.abs(y) * 0.0626 + (SPEC.a1 if quant == "static" else step_) * 2.0 ** -10).all()
    assert_close_fp(out.float().cpu().numpy(), layer_plain(wts, rows, w_ref, ids_ref), "chain M=%d" % M)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()[2]
    for k in range(4):
        x.copy_(torch.roll(x, 1, 1))
        graph.replay()
        torch.cuda.synchronize()
        got = held.clone()
        assert torch.equal(got, step()[2])


def test_layers_with_a_router():
    """fused_moe and fused_moe_fp8 with a router: its ids and weights in the 16-bit layers too."""
    need_gpu()
    spec = gen.CFG2.with_(name="w8-router", E=16, topk=4, K=256, N=128)
    wts = gen.make_moe_weights(spec, seed_config=1502)
    p = wq.pack_moe(8, wts.w1q, wts.s1, wts.w2q, wts.s2, torch.bfloat16, -1)
    bias = torch.linspace(-0.1, 0.1, 16)
    for M in (1, 3, 64, 300):
        x = torch.randn((M, 256)).bfloat16().cuda()
        logits = torch.randn((M, 16)).bfloat16()
        how = dict(scoring="sigmoid", n_group=4, topk_group=2, group_score="top2", routed_scale=2.5)
        out, aux = wq.fused_moe(x, logits.cuda(), p, 4, keep=True, router=wq.Router(bias=bias.cuda(), **how))
        torch.cuda.synchronize()
        w, ids = route(logits.double().numpy(), 4, bias=bias.double().numpy(), **how)
        assert np.array_equal(aux["topk_ids"].cpu().numpy(), ids)
        import oracle
        ref = oracle.moe_layer_from_weights(wts, x.float().cpu().numpy(), w.astype(np.float32), ids)["out"]
        assert_close_fp(out.float().cpu().numpy(), ref, "router layer M=%d" % M)


def of_size(M, N, E, topk, K, bs, stage, seed):
    """Codes, row scales 2^-2 .. 2^-4 by token, random routing -> (run on codes, quantising run at one scale, token of each row)."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(0, 256, (E, 2 * N, K), generator=g, dtype=torch.uint8).numpy()
    w[(w & 0x7F) >= 0x60] &= 0x8F
    ws = (2.0 ** torch.randint(-7, -4, (E, 2 * N), generator=g).float()).numpy()
    wp, sp = wq.pack_fp8(w, ws, interleave_gate_up=stage == wq.WQ_STAGE_GATE_UP)
    wp, sp = torch.from_numpy(wp).cuda(), torch.from_numpy(sp).cuda()
    codes = torch.randint(0, 256, (M, K), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) >= 0x70] &= 0x8F
    value = torch.from_numpy(e4m3_values(codes.numpy())).cuda()
    codes = codes.cuda()
    ids = torch.argsort(torch.rand((M, E), generator=g), dim=1)[:, :topk].int().cuda()
    cap = wq.moe_align_capacity(M, topk, E, bs)
    st, ex, nt = wq.moe_align(ids, E, bs, cap)
    gate_up = stage == wq.WQ_STAGE_GATE_UP
    token = st[:int(nt)].long() // topk if gate_up else torch.arange(M * topk, device="cuda") // topk
    rows = 2.0 ** -(2 + torch.arange(M, device="cuda") % 3).float()

    def out():
        return (torch.zeros((cap, N), dtype=torch.uint8, device="cuda") if gate_up
                else torch.zeros((M * topk, 2 * N), device="cuda"))

    common = (M, topk, E, 2 * N, K, wp, sp, st, ex, nt, cap, bs)

    def on_codes():
        got = wq.moe_fp8_codes_gemm(stage, codes, rows, *common, out(), out_scale=0.5)
        return got[:len(token)]

    def quantising(scale):
        work = torch.empty(wq.moe_fp8_gemm_workspace_bytes(stage, M, topk, E, 2 * N, K), dtype=torch.uint8, device="cuda")
        got = out()
        wq.moe_fp8_w8a8_gemm(stage, (value * scale).bfloat16(), *common, None, got, work, scale, 0.5)
        return got[:len(token)]

    plain = dict(w=w, ws=ws, x=value, ids=ids.cpu().numpy())
    return on_codes, quantising, token, plain


def compare_row_scales(on_codes, quantising, token, M):
    got = on_codes()
    torch.cuda.synchronize()
    assert bool(got.any())
    for k in range(3):
        ref = quantising(2.0 ** -(2 + k))
        torch.cuda.synchronize()
        of = (token < M) & (token % 3 == k)
        assert bool(of.any()) and torch.equal(got[of], ref[of]), k
    pad = token >= M
    assert not bool(got[pad].any())
    return got


@pytest.mark.parametrize("stage", [wq.WQ_STAGE_GATE_UP, wq.WQ_STAGE_RAW])
@pytest.mark.parametrize("M,N", [(300, 256), (4300, 256), (9001, 256), (9001, 384), (50001, 256), (40001, 384), (700, 192)])
def test_row_scales_in_each_tile_shape(M, N, stage):
    """128-row blocks: 128 x 128, 256 x 128, 256 x 64 by XCD and 512 x 128 tiles (and widths that only one of them
    takes), every token with a scale that its neighbours do not have."""
    need_gpu()
    say("row scales", M, N, stage)
    made = of_size(M, N, 8, 2, 384, 128, stage, M + N)
    compare_row_scales(*made[:3], M)


@pytest.mark.parametrize("stage", [wq.WQ_STAGE_GATE_UP, wq.WQ_STAGE_RAW])
@pytest.mark.parametrize("bs", [16, 64, 128])
@pytest.mark.parametrize("M,E,topk,N", [(3, 64, 6, 128), (100, 64, 6, 128), (200, 160, 6, 128), (333, 256, 8, 64), (1500, 64, 6, 512)])
def test_many_experts(M, E, topk, N, bs, stage):
    """64 experts and more: the small-batch kernel's shape for them, 64- and 128-row blocks with most of them part empty;
    RAW also against float64 on some rows.  There each of the 3 products of 128 channels is off by at most 2^-9 of the
    largest value it adds (the matrix instruction drops bits 2^-11 below it in 4 groups, as test_gpu_fp8.py bounds it):
    a term, or the sum so far, which the 3 products' own sums bound in any order; the sums and the two scalings add 5
    roundings of float32."""
    need_gpu()
    say("many experts", M, E, topk, N, bs, stage)
    K = 384
    on_codes, quantising, token, plain = of_size(M, N, E, topk, K, bs, stage, M + E + bs)
    got = compare_row_scales(on_codes, quantising, token, M)
    if stage == wq.WQ_STAGE_RAW:
        x = plain["x"].double().cpu().numpy()
        for pair in range(0, M * topk, max(1, M * topk // 50)):
            m, e = pair // topk, plain["ids"][pair // topk, pair % topk]
            terms = e4m3_values(plain["w"][e]) * x[m]  # [2N, K]
            scale = plain["ws"][e] * 2.0 ** -(2 + m % 3)
            ref = terms.sum(1) * scale
            largest = np.maximum(np.abs(terms).max(1), np.abs(terms.reshape(2 * N, 3, 128).sum(2)).sum(1))
            off = (3 * 2.0 ** -9 * largest + 5 * 2.0 ** -24 * np.abs(terms).sum(1)) * scale
            assert (np.abs(got[pair].double().cpu().numpy() - ref) <= off).all(), pair


def test_more_64_row_tiles_than_a_grid_dimension_takes():
    """Beyond 65535 tiles of 64 rows the 128-row tiles go on."""
    need_gpu()
    M, N, E, K, topk, bs = 2_100_001, 128, 8, 128, 2, 128
    w = torch.randint(0, 256, (E, 2 * N, K), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).numpy()
    w[(w & 0x7F) >= 0x60] &= 0x8F
    wp, sp = wq.pack_fp8(w, np.full((E, 2 * N), 2.0 ** -6, np.float32), interleave_gate_up=True)
    wp, sp = torch.from_numpy(wp).cuda(), torch.from_numpy(sp).cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    codes = torch.randint(0, 0x70, (M, K), generator=g, dtype=torch.uint8, device="cuda")
    ids = torch.argsort(torch.rand((M, E), generator=g, device="cuda"), dim=1)[:, :topk].int().contiguous()
    cap = wq.moe_align_capacity(M, topk, E, bs)
    assert cap // 64 > 65535 >= cap // 128
    st, ex, nt = wq.moe_align(ids, E, bs, cap)
    say("many tiles", M, cap)
    got, ref = torch.zeros((2, cap, N), dtype=torch.uint8, device="cuda")
    common = (M, topk, E, 2 * N, K, wp, sp, st, ex, nt, cap, bs)
    wq.moe_fp8_codes_gemm(wq.WQ_STAGE_GATE_UP, codes, torch.full((M,), 0.125, device="cuda"), *common, got, out_scale=0.5)
    x = codes.view(torch.float8_e4m3fn).bfloat16() * 0.125
    work = torch.empty(M * K + 256, dtype=torch.uint8, device="cuda")
    wq.moe_fp8_w8a8_gemm(wq.WQ_STAGE_GATE_UP, x, *common, None, ref, work, 0.125, 0.5)
    torch.cuda.synchronize()
    assert bool(got[-cap // 4:].any()) and torch.equal(got, ref)
