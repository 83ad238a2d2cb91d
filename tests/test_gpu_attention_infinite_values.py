"""Infinite values in a 16-bit cache: a weight above 0 times an infinity is one."""
import math

import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.kv_ref import TYPES, assert_near, attention
from tests.test_gpu_attention_far_scores import paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("B,H,G,n", [(1, 1, 1, 1), (2, 2, 3, 17), (3, 2, 4, 300), (1, 4, 2, 3001)])
def test_infinite_values(act, D, B, H, G, n):
    """Channel 1: one infinity; 3: one of the other sign; 5: both (NaN); the other channels as without."""
    need_gpu()
    say("infinite values", act, D, B, H, G, n)
    g = torch.Generator().manual_seed(n + D)
    k, v = (torch.randn((B, n, H, D), generator=g).to(TYPES[act]) for _ in range(2))
    q = torch.randn((B, H * G, D), generator=g).to(TYPES[act])  # weights within 2^-37 of the largest
    plain, table, lengths = paged(k.cuda(), v.cuda())
    want, wl, tol, _ = attention(q, [t.cpu() for t in plain[:2]] + [None, None], table.cpu(), lengths.cpu(), D ** -0.5, 0)
    for i, t in enumerate({0, n // 2, n - 1}):
        w = v.clone()
        w[:, t, :, 1], w[:, t, :, 3], w[:, t, :, 5] = math.inf, -math.inf, math.inf
        w[:, (t + 1) % n, :, 5] = -math.inf
        cache, _, _ = paged(k.cuda(), w.cuda())
        out, lse = wq.paged_attention(q.cuda(), cache, table, lengths, want_lse=True)
        got = out.cpu()
        assert bool((got[..., 1] == math.inf).all()) and bool((got[..., 3] == -math.inf).all()), (t, got[..., :6])
        assert bool(torch.isnan(got[..., 5]).all()) if n > 1 else bool((got[..., 5] == -math.inf).all())
        rest = [c for c in range(D) if c not in (1, 3, 5)]
        assert_near(got[..., rest], want[..., rest], tol[..., rest], act)
        assert bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("act,gaps", [("f16", [0.0, 5.0, 11.0, 16.5, 20.0, 23.0, 25.5]), ("bf16", [0.0, 16.5, 25.5, 45.0, 60.0, 69.0])])
@pytest.mark.parametrize("n,first,at", [(300, 0, 3), (300, 200, 3), (300, 3, 290), (3001, 5, 2900), (3001, 2900, 5)])
def test_infinite_values_of_small_weight(act, gaps, n, first, at):
    """The infinity's weight is exp(-gap) of the largest, seen before or after it: down to 2^-37 (fp16) and 2^-100 (bf16)."""
    need_gpu()
    D, H = 64, len(gaps)
    say("small weights", act, n, first, at)
    dt = TYPES[act]
    k = torch.zeros((1, n, H, D), dtype=dt, device="cuda")
    v = torch.ones((1, n, H, D), dtype=dt, device="cuda")
    k[..., 0] = -60000.0  # of no weight
    k[0, first, :, 0] = 0
    for h, gap in enumerate(gaps):
        k[0, at, h, 0] = -gap
    v[0, at, :, 2], v[0, at, :, 7] = math.inf, -math.inf
    q = torch.zeros((1, H, D), dtype=dt, device="cuda")
    q[..., 0] = 1
    cache, table, lengths = paged(k, v)
    out = wq.paged_attention(q, cache, table, lengths, scale=1.0)[0]
    assert bool((out[:, 2] == math.inf).all()) and bool((out[:, 7] == -math.inf).all()), out[:, [2, 7]]
    rest = [c for c in range(D) if c not in (2, 7)]
    assert float((out[:, rest].float() - 1).abs().max()) <= 2.0 ** -7  # (the weights' mean of ones: bf16's step)
