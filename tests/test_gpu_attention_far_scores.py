"""paged_attention at scores so large that a step of float32 is more than the maximum's slack."""
import math

import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.kv_ref import TYPES
from tests.serving_ref import HALF

pytestmark = pytest.mark.gpu


def paged(k, v, P=16):
    """Rows [B, n, H, D] on the device -> (cache, table, lengths), pages one sequence's after another's."""
    B, n, H, D = k.shape
    width = -(-n // P)
    pad = width * P - n

    def pages(t):
        t = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, pad))
        return t.view(B * width, P, H, D).transpose(1, 2).contiguous()

    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    return wq.KVCache(pages(k), pages(v)), table, torch.full((B,), n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("n,second", [(200, 130), (1000, 129), (40, 20), (40, 1)])
@pytest.mark.parametrize("steps", [(1, 2), (2, 3), (3, 5), (-1, 0)])
def test_scores_a_step_of_float32_apart(act, n, second, steps):
    """Scores in exponents of 2 (scale = ln 2) of 2^27 + 16 j, whose neighbours in float32 are 16 apart: token 0 at the
    first j, `second` at the larger one, all others at 0.  Products, sums and differences are exact in float32, so the
    weights are 2^(16 (j0 - j1)) and 1, and out = (v1 + w v0) / (1 + w) but for parts (2^-16), exp2 (2^-22) and one rounding."""
    need_gpu()
    say("far scores", act, n, second, steps)
    dt, D = TYPES[act], 64
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.zeros((1, n, 1, D), dtype=dt, device="cuda")
    for t, j in zip((0, second), steps):
        k[0, t, 0, 0], k[0, t, 0, 1] = 16384.0, 4.0 * j
    v = torch.randn((1, n, 1, D), generator=g, device="cuda").to(dt)
    q = torch.zeros((1, 1, D), dtype=dt, device="cuda")
    q[..., 0], q[..., 1] = 8192.0, 4.0
    cache, table, lengths = paged(k, v)
    out, lse = wq.paged_attention(q, cache, table, lengths, scale=math.log(2.0), want_lse=True)
    w = 2.0 ** (16 * (steps[0] - steps[1]))
    a, b = v[0, second, 0].double(), w * v[0, 0, 0].double()
    want, size = (a + b) / (1 + w), (a.abs() + b.abs()) / (1 + w)
    tol = size * 2.0 ** -15
    off = (out[0, 0].double() - want).abs()
    assert bool((off <= tol + HALF[act] * (want.abs() + tol)).all()), out
    top = (2.0 ** 27 + 16 * steps[1] + math.log2(1 + w)) * math.log(2.0)
    assert abs(float(lse) - top) <= top * 2.0 ** -22  # (the logarithm's sum, its product with ln 2 and ln 2 itself)
