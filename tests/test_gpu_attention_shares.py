"""paged_attention where a share holds several steps and runs from one sequence to the next, for every form of the kernel, and
over caches of more than the last-level cache (non-temporal loads)."""
import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.kv_ref import assert_near, attention
from tests.test_gpu_paged_attention import make

pytestmark = pytest.mark.gpu


def shares_of(lengths, D, H, G, P, width, window):
    """[(sequence, first step, last step)] of every share, from the sizes alone, as the kernel's description gives them."""
    resident = 256 * (4 if D <= 64 else 3 if D <= 128 else 2)
    units = H * -(-G // 16)
    steps = []
    for n in lengths:
        n = min(max(n, 0), width * P)
        lo = max(0, n - window) // 16 * 16 if window else 0
        steps.append(max(1, -(-(n - lo) // 128)))
    cut = -(-sum(steps) // max(1, resident // units))
    owner = [b for b, k in enumerate(steps) for _ in range(k)]
    return cut, [owner[i:i + cut] for i in range(0, len(owner), cut)]


RAGGED = [1900, 1, 700, 0, 2049, 128, 1300, 33, 2500, 640]
FORMS = [("bf16", None), ("f16", None), ("bf16", "row"), ("f16", "row"), ("bf16", "static"), ("f16", "static")]


@pytest.mark.parametrize("act,quant", FORMS)
@pytest.mark.parametrize("D,H,G", [(64, 64, 1), (96, 48, 1), (128, 48, 1), (128, 24, 2), (192, 32, 1), (256, 32, 1), (256, 2, 250)])
def test_shares_across_sequences(act, quant, D, H, G):
    need_gpu()
    say("shares", act, quant, D, H, G)
    P = 16
    lengths = RAGGED if G < 100 else [1900, 1, 700, 0, 1500, 200]
    query, cache, host, table = make(act, quant, H, P, D, lengths, seed=D + H)
    width = table.shape[1]
    cut, shares = shares_of(lengths, D, H, G, P, width, 0)
    assert wq.paged_attention_workspace_bytes(len(lengths), H * G, H, D, P, width) > 0
    # several steps a share; some share ends a sequence and begins another, which the next goes on with
    assert cut >= 3 and any(x[0] != x[-1] and x[-1] == y[0] for x, y in zip(shares, shares[1:]))
    q, qd = query(H * G)
    n = torch.tensor(lengths, dtype=torch.int32)
    out, lse = wq.paged_attention(qd, cache, table.cuda(), n.cuda(), want_lse=True)
    want, wl, tol, ltol = attention(q, host, table, n, D ** -0.5, 0)
    assert_near(out, want, tol, act)
    got = lse.cpu().double()
    assert bool((((got - wl).abs() <= ltol) | (got == wl)).all())


@pytest.mark.parametrize("act,quant", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_caches_beyond_the_last_level(act, quant, D):
    """The same sequences in a small cache and at the end of one of 4 GiB of keys and more: the same bits, and float64's."""
    need_gpu()
    say("large cache", act, quant, D)
    H, G, P, lengths = 2, 3, 64, [5000, 0, 70, 2100]
    query, cache, host, table = make(act, quant, H, P, D, lengths, seed=D)
    assert wq.paged_attention_workspace_bytes(len(lengths), H * G, H, D, P, table.shape[1]) > 0
    q, qd = query(H * G)
    n = torch.tensor(lengths, dtype=torch.int32)
    small = wq.paged_attention(qd, cache, table.cuda(), n.cuda(), want_lse=True)
    pages = (9 << 29) // (H * P * D * cache.k.element_size())
    first = pages - cache.k.shape[0]
    big = []
    for t in cache:
        if isinstance(t, torch.Tensor):
            u = torch.empty((pages, *t.shape[1:]), dtype=t.dtype, device="cuda")
            u[first:] = t
            t = u
        big.append(t)
    got = wq.paged_attention(qd, wq.KVCache(*big), (table + first).cuda(), n.cuda(), want_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, small))
    want, wl, tol, ltol = attention(q, host, table, n, D ** -0.5, 0)
    assert_near(got[0], want, tol, act)
    lse = got[1].cpu().double()
    assert bool((((lse - wl).abs() <= ltol) | (lse == wl)).all())
