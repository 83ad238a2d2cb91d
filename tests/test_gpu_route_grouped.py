"""GPU parity of moe_route_grouped(_align) against a plain float64 form: ids are
compared exactly.  Weights: the device's and the host's double exponentials may
differ in their last bits, which is far below float32's half step, so a weight
is off by that half step, and by one more where the double value lies on the
border between two floats: one step in all."""
import numpy as np
import pytest

import oracle
import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.serving_ref import route

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def logits_of(M, E, dt, seed, spread=1.5):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal((M, E)) * spread).astype(np.float32)).to(DT[dt])


def bias_of(E, seed):
    return torch.from_numpy((np.random.default_rng(seed).standard_normal(E) * 0.05).astype(np.float32))


def check(logits, topk, bias=None, block=None, what="", **how):
    """Both calls (the sort for a block size), against the plain form."""
    say("route_grouped", what, list(logits.shape), logits.dtype, topk, bias is not None, block, how)
    w_ref, ids_ref = route(logits.double().numpy(), topk, bias=None if bias is None else bias.double().numpy(), **how)
    dev = None if bias is None else bias.cuda()
    runs = [wq.moe_route_grouped(logits.cuda(), topk, bias=dev, **how)]
    if block:
        full = wq.moe_route_grouped_align(logits.cuda(), topk, block, bias=dev, **how)
        runs.append(full[:2])
    torch.cuda.synchronize()
    for w, ids in runs:
        assert np.array_equal(ids.cpu().numpy(), ids_ref), "%s: ids differ" % what
        err = np.abs(w.double().cpu().numpy() - w_ref)
        assert (err <= 2.0 ** -23 * np.abs(w_ref) + 2.0 ** -149).all(), what
    if block:
        st, ex, nt = oracle.align(ids_ref, logits.shape[1], block)
        assert np.array_equal(full[2].cpu().numpy()[:st.size], st), what
        assert np.array_equal(full[3].cpu().numpy()[:ex.size], ex), what
        assert int(full[4].cpu()[0]) == nt, what
    return runs[0]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_scores_and_groups(dt, scoring, biased):
    need_gpu()
    for E, G, TG, k in ((1, 1, 1, 1), (2, 1, 1, 2), (8, 1, 1, 2), (8, 4, 2, 3), (60, 3, 2, 5), (64, 64, 7, 6), (64, 8, 8, 8),
                        (96, 1, 1, 4), (100, 5, 1, 7), (160, 8, 3, 6), (256, 8, 4, 8), (257, 1, 1, 9), (384, 1, 1, 8),
                        (512, 16, 3, 16), (1023, 33, 5, 16), (1024, 1, 1, 16), (1024, 64, 9, 10)):
        for score in ("max", "top2"):
            if score == "top2" and G > 1 and E // G < 2:
                continue
            for renorm in (True, False):
                check(logits_of(19, E, dt, E + G), k, bias_of(E, E) if biased else None, scoring=scoring, n_group=G,
                      topk_group=TG, group_score=score, renormalize=renorm, routed_scale=2.5 if renorm else 16.0)


@pytest.mark.parametrize("M", [1, 2, 7, 15, 16, 17, 31, 63, 64, 65, 300])
@pytest.mark.parametrize("block", [16, 64, 256])
def test_align(M, block):
    """The fused sort (one wave up to 64 pairs, a workgroup above) and the separate one."""
    need_gpu()
    check(logits_of(M, 160, "f32", M), 6, None, block, n_group=8, topk_group=3, renormalize=False)
    check(logits_of(M, 256, "bf16", M), 8, bias_of(256, 1), block, scoring="sigmoid", n_group=8, topk_group=4,
          group_score="top2", routed_scale=2.5)
    check(logits_of(M, 8, "f16", M), 2, None, block)
    check(logits_of(M, 64, "f32", M), 16, bias_of(64, 1), block, n_group=4, topk_group=3, group_score="top2")
    check(logits_of(M, 96, "bf16", M), 4, bias_of(96, 1), block, scoring="sigmoid")
    check(logits_of(M, 1024, "f32", M), 16, bias_of(1024, 1), block, scoring="sigmoid")


def test_ties_and_signs():
    need_gpu()
    rng = np.random.default_rng(1)
    few = torch.from_numpy(rng.integers(-2, 3, size=(64, 96)).astype(np.float32))
    zero = torch.zeros((5, 128))
    zero[:, ::3] = -0.0
    for how in (dict(), dict(scoring="sigmoid"), dict(n_group=8, topk_group=3), dict(n_group=8, topk_group=3, group_score="top2"),
                dict(scoring="sigmoid", n_group=4, topk_group=4, group_score="top2")):
        check(few, 8, None, None, "few values", **how)
        check(few, 8, torch.zeros(96), None, "few values, bias of zeros", **how)
        check(zero, 8, None, None, "zeros", **how)
        check(zero, 8, torch.full((128,), -0.5), None, "equal negative scores", **how)
    # scores that saturate: float(s + b) is 1 + b for all of them
    check(torch.full((3, 64), 40.0) + torch.arange(64), 5, torch.zeros(64), None, "saturated", scoring="sigmoid")


def test_masked_experts_and_empty_rows():
    """-inf logits (a masked expert), rows of them, a bias of -inf."""
    need_gpu()
    lg = logits_of(9, 96, "f32", 3)
    lg[0] = -np.inf
    lg[1, 1:] = -np.inf
    lg[2, :90] = -np.inf
    lg[3] = -3.0e38
    lg[4] = 3.0e38
    lg[5] = lg[5] * 1e4
    shut = bias_of(96, 2)
    shut[10:20] = -np.inf
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for how in (dict(), dict(n_group=8, topk_group=2), dict(n_group=8, topk_group=2, group_score="top2")):
                for b in (None, bias_of(96, 1), shut):
                    check(lg, 6, b, None, "masked", scoring=scoring, renormalize=renorm, **how)


def test_nan_rows_name_distinct_experts():
    need_gpu()
    lg = logits_of(6, 160, "f32", 5)
    lg[0] = np.nan
    lg[1, ::2] = np.nan
    lg[2, 7] = np.inf
    lg[3, :] = np.inf
    for how in (dict(), dict(scoring="sigmoid"), dict(n_group=8, topk_group=3, group_score="top2")):
        for b in (None, bias_of(160, 1)):
            w, ids = wq.moe_route_grouped(lg.cuda(), 8, bias=None if b is None else b.cuda(), **how)
            ids = ids.cpu().numpy()
            assert ((ids >= 0) & (ids < 160)).all() and all(len(set(r)) == 8 for r in ids)
            w_ref, ids_ref = route(lg[4:].numpy(), 8, bias=None if b is None else b.numpy(), **how)
            assert np.array_equal(ids[4:], ids_ref)
            assert np.allclose(w.cpu().numpy()[4:], w_ref, rtol=2.0 ** -23, atol=0)


def test_plain_softmax_is_moe_route():
    need_gpu()
    for E, k in ((8, 2), (64, 6), (160, 6), (256, 16)):
        lg = logits_of(201, E, "f32", E).cuda()
        for renorm in (True, False):
            a, b = wq.moe_route(lg, k, renorm), wq.moe_route_grouped(lg, k, renormalize=renorm)
            torch.cuda.synchronize()
            assert torch.equal(a[1], b[1])
            assert float(((a[0] - b[0]).abs() / a[0]).max()) <= 2.0 ** -23


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_large_batches(dt):
    """Four tokens a wave, over group and expert counts (16-byte loads or not, lanes left over)."""
    need_gpu()
    for E, G, TG, k in ((1, 1, 1, 1), (8, 1, 1, 2), (9, 3, 2, 4), (60, 3, 2, 5), (64, 16, 5, 7), (96, 1, 1, 16), (160, 8, 3, 6),
                        (256, 8, 4, 8), (256, 1, 1, 8), (250, 5, 2, 10), (272, 1, 1, 8), (512, 32, 7, 8), (1024, 4, 2, 16)):
        lg = logits_of(2051, E, dt, E + G)
        for scoring, biased, score, renorm in (("softmax", False, "max", True), ("softmax", True, "top2", False),
                                               ("sigmoid", True, "max", True), ("sigmoid", False, "top2", True)):
            if score == "top2" and G > 1 and E // G < 2:
                continue
            check(lg, k, bias_of(E, E) if biased else None, None, "large", scoring=scoring, n_group=G, topk_group=TG,
                  group_score=score, renormalize=renorm)


def test_large_batches_of_special_rows():
    """Ties, masked experts, empty rows and NaN rows among the four tokens of a wave."""
    need_gpu()
    rng = np.random.default_rng(4)
    lg = torch.from_numpy(rng.integers(-2, 3, size=(2050, 160)).astype(np.float32))
    lg[5] = -np.inf
    lg[6, 3:] = -np.inf
    lg[9] = 3.0e38
    for how in (dict(n_group=8, topk_group=3), dict(scoring="sigmoid", n_group=8, topk_group=3, group_score="top2")):
        for b in (None, bias_of(160, 1)):
            check(lg, 6, b, None, "special rows", **how)
            bad = lg.clone()
            bad[4] = np.nan
            bad[7, ::3] = np.nan
            ids = wq.moe_route_grouped(bad.cuda(), 6, bias=None if b is None else b.cuda(), **how)[1].cpu().numpy()
            keep = np.delete(np.arange(2050), [4, 7])
            ref = route(lg.double().numpy(), 6, bias=None if b is None else b.double().numpy(), **how)[1]
            assert np.array_equal(ids[keep], ref[keep])
            assert all(len(set(ids[m])) == 6 and 0 <= ids[m].min() and ids[m].max() < 160 for m in (4, 7))


def test_large_batch_and_empty():
    need_gpu()
    check(logits_of(5001, 256, "bf16", 1), 8, bias_of(256, 1), None, "large", scoring="sigmoid", n_group=8, topk_group=4,
          group_score="top2")
    check(logits_of(20011, 8, "f32", 1), 2, None, 64, "large", scoring="sigmoid")
    w, ids, st, ex, nt = wq.moe_route_grouped_align(torch.empty((0, 8), device="cuda"), 2, 16)
    torch.cuda.synchronize()
    assert w.shape == (0, 2) and int(nt.cpu()[0]) == 0
    # a capacity above the least: the tail holds the sentinel
    lg = logits_of(3, 160, "f32", 2)
    full = wq.moe_route_grouped_align(lg.cuda(), 6, 16, capacity=1024)
    st, ex, nt = oracle.align(route(lg.numpy(), 6)[1], 160, 16)
    got = full[2].cpu().numpy()
    assert np.array_equal(got[:st.size], st) and (got[st.size:] == 18).all() and got.size == 1024
    assert (full[3].cpu().numpy()[ex.size:] == -1).all()


def test_graph_and_stream():
    need_gpu()
    lg, b = logits_of(13, 160, "f32", 9).cuda(), bias_of(160, 2).cuda()
    how = dict(scoring="sigmoid", bias=b, n_group=8, topk_group=3, group_score="top2")
    ref = wq.moe_route_grouped_align(lg, 6, 16, **how)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = wq.moe_route_grouped_align(lg, 6, 16, stream=side.cuda_stream, **how)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(got, ref):
        assert torch.equal(x, y)
    live = lg.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = wq.moe_route_grouped_align(live, 6, 16, **how)
    for k in range(4):
        live.copy_(torch.roll(lg, k, 1))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(held, wq.moe_route_grouped_align(live, 6, 16, **how)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("M", [7, 5003])  # 64 and 16 lanes a token
@pytest.mark.parametrize("biased", [False, True])
def test_nan_under_sigmoid_scores(M, biased):
    """A NaN logit ranks below every number, also where its bias is the largest, and is not hidden in the weights."""
    need_gpu()
    E, k = 16, 5
    lg, b = logits_of(M, E, "f32", 21), bias_of(E, 3)
    lg[0] = np.nan
    lg[1, 2:14] = np.nan  # four numbers are left
    lg[2, ::2] = np.nan
    lg[3, 6] = np.nan
    b[6] = 3.0
    order = torch.sigmoid(lg.double()) + b.double() if biased else lg.double()
    for renorm in (True, False):
        say("nan, sigmoid", M, biased, renorm)
        w, ids = wq.moe_route_grouped(lg.cuda(), k, scoring="sigmoid", bias=b.cuda() if biased else None, renormalize=renorm)
        w, ids = w.cpu().double(), ids.cpu()
        for m in range(7):
            nan = torch.isnan(lg[m])
            rank = sorted(range(E), key=lambda e: (bool(nan[e]), 0.0 if nan[e] else -float(order[m, e].float() if biased else order[m, e]), e))
            assert ids[m].tolist() == rank[:k], m
            s = torch.sigmoid(lg[m].double())[ids[m].long()]
            ref = s / s.sum() if renorm else s
            assert torch.equal(torch.isnan(w[m]), torch.isnan(ref)), m
            num = ~torch.isnan(ref)
            assert bool(((w[m] - ref).abs()[num] <= 2.0 ** -23 * ref[num]).all()), m
    # groups by their two best numbers: group 1 holds the largest number and NaN otherwise, so it has no second
    lg[4] = torch.arange(16.0) / 16
    lg[4, 4:8] = torch.tensor([9.0, np.nan, np.nan, np.nan])
    ids = wq.moe_route_grouped(lg.cuda(), 4, scoring="sigmoid", n_group=4, topk_group=2, group_score="top2")[1].cpu()
    assert ids[4].tolist() == [15, 14, 13, 12]
