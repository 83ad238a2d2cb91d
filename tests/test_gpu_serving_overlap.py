"""Serving operators on two streams at once, and two captured graphs replayed in
turn: each with its own buffers (the binding's own allocations) gives the
results of the calls one after the other."""
import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, torch

pytestmark = pytest.mark.gpu


def work(seed, M):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=g).bfloat16().cuda()

    K, N, R, L = 512, 384 if M < 100 else 2048, 64, 4
    x, r, w = rnd(M, K), rnd(M, K), rnd(K)
    a, b, y = rnd(L, R, K) * 0.05, rnd(L, N, R), rnd(M, N)
    ids = torch.randint(-1, L, (M,), generator=g).int().cuda()
    logits = torch.randn(M, 64, generator=g).cuda()

    def run():
        n = wq.rms_norm(x, w, residual=r, quant="row")
        z = wq.dense_lora_gemm(n.out, ids, a, b, None, y.clone())
        return (*n, z, *wq.moe_route_grouped_align(logits, 4, 16, scoring="sigmoid", n_group=8, topk_group=4))

    return x, run


def same(got, want):
    # (expert_ids and the sorted rows are written whole; every output is compared)
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M", [9, 700])
def test_two_streams(M):
    need_gpu()
    jobs = [work(s, M)[1] for s in (1, 2)]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(j())
        torch.cuda.synchronize()
        assert all(same(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("M", [9, 700])
def test_two_graphs(M):
    need_gpu()
    made = [work(s, M) for s in (3, 4)]
    graphs, held = [], []
    for _, run in made:
        run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(run())
    for k in range(4):
        for x, _ in made:
            x.copy_(torch.roll(x, k, 1))
        graphs[k % 2].replay()
        graphs[1 - k % 2].replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in h] for h in held]
        for (_, run), g in zip(made, got):
            assert same(g, run())
