"""paged_attention on the GPU against float64 over the same cache."""
import math

import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.kv_ref import TYPES, assert_near, attention, quantise

pytestmark = pytest.mark.gpu


def make(act, quant, H, P, D, lengths, width=None, seed=0, spare=2, garbage=True, loud=1.5):
    """(q maker, cache on device, cache on host, table): pages in random order, NaN in every row that no sequence owns."""
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[act]
    need = [-(-max(n, 0) // P) for n in lengths]
    pages = sum(need) + spare
    width = max(max(need), 1) if width is None else width
    k, v = (torch.randn((pages, H, P, D), generator=g).to(dt) for _ in range(2))
    order = torch.randperm(pages, generator=g).int()
    table = torch.full((len(lengths), width), -7, dtype=torch.int32)  # (past the end: not read)
    owned = torch.zeros((pages, P), dtype=torch.bool)
    at = 0
    for b, n in enumerate(lengths):
        table[b, :need[b]] = order[at:at + need[b]]
        t = torch.arange(max(n, 0))
        owned[table[b, t // P].long(), t % P] = True
        at += need[b]
    if quant is None:
        host = [k, v, None, None]
    else:
        static = (0.02, 0.017)
        (ck, sk), (cv, sv) = quantise(k, quant, static[0]), quantise(v, quant, static[1])
        host = [ck, cv, sk, sv] if quant == "row" else [ck, cv, *static]
    if garbage:
        for i in range(2):
            view = host[i].transpose(1, 2)
            view[~owned] = 0x7F if quant else float("nan")
            if quant == "row":
                host[2 + i].transpose(1, 2)[~owned] = float("nan")
    cache = wq.KVCache(*[t.cuda() if isinstance(t, torch.Tensor) else t for t in host])

    def query(heads, wide=0):
        q = (loud * torch.randn((len(lengths), heads + wide, D), generator=g)).to(dt)
        return q[:, :heads], q.cuda()[:, :heads]

    return query, cache, host, table


def check(act, quant, H, G, P, D, lengths, window=0, scale=None, **k):
    need_gpu()
    say("attention", act, quant, H, G, P, D, lengths, window)
    query, cache, host, table = make(act, quant, H, P, D, lengths, **k)
    q, qd = query(H * G, wide=2 * H)
    n = torch.tensor(lengths, dtype=torch.int32)
    out, lse = wq.paged_attention(qd, cache, table.cuda(), n.cuda(), scale=scale, window=window, want_lse=True)
    torch.cuda.synchronize()
    want, wl, tol, ltol = attention(q, host, table, n, D ** -0.5 if scale is None else scale, window)
    assert_near(out, want, tol, act)
    got = lse.cpu().double()
    assert bool((((got - wl).abs() <= ltol) | (got == wl)).all())
    return qd, cache, table.cuda(), n.cuda(), out, lse


@pytest.mark.parametrize("quant", [None, "row", "static"])
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("D", [16, 64, 80, 96, 128, 144, 192, 256])
def test_head_dims(act, quant, D):
    check(act, quant, 2, 3, 16, D, [37, 200, 1])


@pytest.mark.parametrize("quant", [None, "row"])
@pytest.mark.parametrize("lengths", [[0], [1], [15, 16, 17], [31, 32, 33, 0], [63, 64, 65, 127, 128, 129], [-3, 255, 256, 257]])
def test_short_lengths(quant, lengths):
    check("bf16", quant, 1, 4, 16, 128, lengths)


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (1, 7), (2, 16), (1, 17), (2, 20), (1, 71), (16, 2)])
def test_head_groups(H, G):
    check("f16", "row", H, G, 32, 64, [130, 5])


@pytest.mark.parametrize("P", [16, 32, 48, 64, 112, 1024])
@pytest.mark.parametrize("quant", [None, "static"])
def test_page_sizes(P, quant):
    check("bf16", quant, 2, 2, P, 64, [P - 1, P, P + 1, 3 * P + 17])


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 300, 5000])
@pytest.mark.parametrize("quant", [None, "row"])
def test_windows(window, quant):
    check("f16", quant, 2, 4, 16, 128, [0, 1, 16, 99, 333, 2049], window=window)


@pytest.mark.parametrize("quant", [None, "row"])
@pytest.mark.parametrize("H,G,D,lengths", [(1, 8, 128, [3001]), (8, 4, 64, [1, 0, 5000, 17, 900]), (2, 20, 256, [1500, 700]),
                                           (4, 1, 96, [2500] + [40] * 70)])
def test_split_over_the_length(quant, H, G, D, lengths):
    assert wq.paged_attention_workspace_bytes(len(lengths), H * G, H, D, 16, -(-max(lengths) // 16)) > 0
    qd, cache, table, n, out, lse = check("bf16", quant, H, G, 16, D, lengths)
    # the same bits again, from a workspace of other values
    ws = torch.full((wq.paged_attention_workspace_bytes(len(lengths), H * G, H, D, 16, table.shape[1]),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    for _ in range(3):
        again, l2 = wq.paged_attention(qd, cache, table, n, want_lse=True, workspace=ws)
        assert torch.equal(again, out) and torch.equal(l2, lse)


def test_many_sequences():
    """More sequences than a wave's lanes share out one each."""
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 60, (300,), generator=g).tolist()
    lengths[7], lengths[299] = 3000, 1300
    check("f16", None, 1, 2, 16, 32, lengths)


def test_a_long_table_for_short_sequences():
    """The table has room for far more than the batch holds: its other entries are not read."""
    check("bf16", "row", 2, 4, 16, 128, [40, 0, 700], width=4096)


def test_length_past_the_table_ends_there():
    need_gpu()
    query, cache, host, table = make("bf16", None, 1, 16, 64, [48])
    q, qd = query(2)
    a = wq.paged_attention(qd, cache, table.cuda(), torch.tensor([48], dtype=torch.int32).cuda())
    b = wq.paged_attention(qd, cache, table.cuda(), torch.tensor([2 ** 31 - 1], dtype=torch.int32).cuda())
    assert torch.equal(a, b)


def test_bad_pages_hold_no_tokens():
    need_gpu()
    for quant in (None, "row"):
        query, cache, host, table = make("bf16", quant, 2, 16, 64, [100, 800, 40])
        table[0, 2], table[1, 0], table[1, 20], table[2, :] = -1, 10 ** 6, -(2 ** 31), 2 ** 31 - 1
        q, qd = query(8)
        n = torch.tensor([100, 800, 40], dtype=torch.int32)
        out, lse = wq.paged_attention(qd, cache, table.cuda(), n.cuda(), want_lse=True)
        torch.cuda.synchronize()
        want, wl, tol, _ = attention(q, host, table, n, 64 ** -0.5, 0)
        assert_near(out, want, tol, "bf16")
        assert bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())


def test_shared_pages():
    """A prefix that two sequences share."""
    need_gpu()
    query, cache, host, table = make("f16", None, 2, 16, 128, [70, 64])
    table[1, :3] = table[0, :3]
    q, qd = query(4)
    n = torch.tensor([70, 64], dtype=torch.int32)
    out = wq.paged_attention(qd, cache, table.cuda(), n.cuda())
    want, _, tol, _ = attention(q, host, table, n, 128 ** -0.5, 0)
    assert_near(out, want, tol, "f16")


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_peaked_and_flat(act):
    """Scores far apart (one weight takes all; the maximum last, so it is raised again and again) and all the same."""
    need_gpu()
    for scale in (0.0, 3.0):
        check(act, None, 1, 4, 16, 64, [1000, 33], scale=scale)
    query, cache, host, table = make(act, None, 1, 16, 64, [600], garbage=False)
    host[0][:] = 0
    for t in range(600):  # scores 0, 0.5, 1, ... 299.5
        host[0][table[0, t // 16], 0, t % 16, 0] = 0.5 * t
    q = torch.zeros((1, 1, 64), dtype=TYPES[act])
    q[..., 0] = 1
    n = torch.tensor([600], dtype=torch.int32)
    out, lse = wq.paged_attention(q.cuda(), wq.KVCache(host[0].cuda(), host[1].cuda()), table.cuda(), n.cuda(), scale=1.0, want_lse=True)
    want, wl, tol, ltol = attention(q, host, table, n, 1.0, 0)
    assert_near(out, want, tol, act)
    assert float((lse.cpu().double() - wl).abs().max()) <= float(ltol.max())


def test_infinities_and_nan_stay_in_their_own():
    need_gpu()
    query, cache, host, table = make("bf16", None, 2, 16, 64, [50, 60, 70, 80])
    host[0][table[0, 1], 0, 3, 5] = float("nan")    # a key: sequence 0, head 0
    host[1][table[1, 2], 1, 4, 9] = float("inf")    # a value: sequence 1, head 1, channel 9
    host[0][table[2, 0], 1, 0, :] = float("inf")    # infinite keys: scores of inf, -inf or NaN
    cache = wq.KVCache(host[0].cuda(), host[1].cuda())
    q, qd = query(4)
    n = torch.tensor([50, 60, 70, 80], dtype=torch.int32)
    out, lse = wq.paged_attention(qd, cache, table.cuda(), n.cuda(), want_lse=True)
    out = out.float().cpu()
    assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isfinite(out[0, 2:]).all())
    # (an infinite value times the two parts of its weight: infinite or NaN)
    assert not bool(torch.isfinite(out[1, 2:, 9]).any()) and bool(torch.isfinite(out[1, :2]).all())
    assert bool(torch.isfinite(out[1, 2:, :9]).all()) and bool(torch.isfinite(out[1, 2:, 10:]).all())
    assert bool(torch.isnan(out[2, 2:]).all()) and bool(torch.isfinite(out[2, :2]).all())
    assert bool(torch.isfinite(out[3]).all()) and bool(torch.isfinite(lse[3].cpu()).all())


def test_rows_that_are_strided():
    """q and out as column ranges of one projection's output; what lies beside out stays."""
    need_gpu()
    query, cache, host, table = make("bf16", "row", 2, 16, 64, [50, 1300])
    g = torch.Generator().manual_seed(9)
    wide = torch.randn((2, 20, 64), generator=g).bfloat16()
    d = wide.cuda()
    n = torch.tensor([50, 1300], dtype=torch.int32)
    got = wq.paged_attention(d[:, :8], cache, table.cuda(), n.cuda(), out=d[:, 10:18])
    assert got.data_ptr() == d[:, 10:18].data_ptr()
    want, _, tol, _ = attention(wide[:, :8], host, table, n, 64 ** -0.5, 0)
    assert_near(d[:, 10:18], want, tol, "bf16")
    assert torch.equal(d[:, :10].cpu(), wide[:, :10]) and torch.equal(d[:, 18:].cpu(), wide[:, 18:])


def test_far_offsets():
    """Pages beyond 2^32 bytes from the cache's beginning."""
    need_gpu()
    H, P, D = 8, 64, 128
    pages = (5 << 30) // (H * P * D * 2)
    cache = wq.kv_cache(pages, H, P, D, torch.bfloat16)
    for t in cache[:2]:
        t[-4:] = torch.randn((4, H, P, D), device="cuda").bfloat16()
    table = torch.tensor([[pages - 1, pages - 3, pages - 2, pages - 4]], dtype=torch.int32)
    q = torch.randn((1, 16, D)).bfloat16()
    n = torch.tensor([250], dtype=torch.int32)
    out = wq.paged_attention(q.cuda(), cache, table.cuda(), n.cuda())
    host = [cache.k[-4:].cpu(), cache.v[-4:].cpu(), None, None]
    want, _, tol, _ = attention(q, host, table - (pages - 4), n, D ** -0.5, 0)
    assert_near(out, want, tol, "bf16")


@pytest.mark.parametrize("lengths", [[90, 3], [2600, 40, 0]])
def test_streams_and_graphs(lengths):
    need_gpu()
    jobs = []
    for seed in (1, 2):
        query, cache, host, table = make("bf16", "row", 2, 16, 128, lengths, seed=seed)
        _, qd = query(8)
        jobs.append((qd.contiguous(), cache, table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda()))
    want = [wq.paged_attention(*j, want_lse=True) for j in jobs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        one = wq.paged_attention(*jobs[0], want_lse=True)
        two = wq.paged_attention(*jobs[1], want_lse=True, stream=side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in ((one, want[0]), (two, want[1])) for a, b in zip(g, w))
    graphs, held = [], []
    for j in jobs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(wq.paged_attention(*j, want_lse=True))
    for k in range(4):  # lengths and queries change in place between replays
        for j in jobs:
            j[0].copy_(torch.roll(j[0], k, 2))
            j[3].copy_(torch.tensor([max(0, n - 7 * k) for n in lengths], dtype=torch.int32))
        graphs[k % 2].replay()
        graphs[1 - k % 2].replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in h] for h in held]
        for j, g in zip(jobs, got):
            assert all(torch.equal(a, b) for a, b in zip(g, wq.paged_attention(*j, want_lse=True)))


def test_no_sequences():
    need_gpu()
    query, cache, host, table = make("bf16", None, 2, 16, 64, [50])
    out, lse = wq.paged_attention(torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"), cache,
                                  torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                                  torch.empty(0, dtype=torch.int32, device="cuda"), want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("quant", [None, "row"])
def test_shares_of_more_steps_than_a_block_of_pages(quant):
    """Many heads and long sequences: a workgroup's share goes on past the 32 steps whose pages it has fetched at once,
    within a sequence and from one to the next."""
    check("f16", quant, 256, 1, 32, 16, [9001, 260, 8400, 0, 70])


def test_pages_before_the_window_may_be_gone():
    need_gpu()
    for P, window, n in ((16, 100, 1000), (48, 17, 650), (64, 640, 700)):
        query, cache, host, table = make("bf16", "row", 2, P, 128, [n, n - 3])
        q, qd = query(4)
        lengths = torch.tensor([n, n - 3], dtype=torch.int32).cuda()
        want = wq.paged_attention(qd, cache, table.cuda(), lengths, window=window, want_lse=True)
        for b, length in enumerate((n, n - 3)):
            table[b, :(length - window) // P] = torch.tensor([-1, 1 << 30])[b]
        got = wq.paged_attention(qd, cache, table.cuda(), lengths, window=window, want_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("quant", [None, "static"])
def test_the_largest_workgroup_in_a_graph(quant):
    """16 heads of 256 a workgroup: more than 64 KB of LDS, asked for by a captured call as by any other."""
    need_gpu()
    query, cache, host, table = make("bf16", quant, 2, 32, 256, [700, 1, 90])
    q, qd = query(32)
    qd, table = qd.contiguous(), table.cuda()
    lengths = torch.tensor([700, 1, 90], dtype=torch.int32).cuda()
    wq.paged_attention(qd, cache, table, lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = wq.paged_attention(qd, cache, table, lengths)
    for k in range(3):
        qd.copy_(torch.roll(qd, 1, 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, wq.paged_attention(qd, cache, table, lengths))
