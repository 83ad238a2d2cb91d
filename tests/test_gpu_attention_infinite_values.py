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
