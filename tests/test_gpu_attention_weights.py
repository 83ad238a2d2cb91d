"""The softmax weights of paged_attention where their 16-bit parts are at the ends of the types' ranges."""
import math

import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.kv_ref import TYPES
from tests.serving_ref import HALF, TINY
from tests.test_gpu_attention_far_scores import paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("gap", [9.0, 13.875, 15.53, 17.05, 18.0, 20.0])
@pytest.mark.parametrize("B,H,n,D,at", [(1, 1, 500, 64, 3), (3, 32, 1000, 64, 3), (1, 64, 20000, 64, 3), (1, 64, 20000, 64, 9000),
                                        (1, 2, 240, 256, 3), (1, 16, 20000, 256, 700), (2, 3, 500, 80, 490)])
def test_one_key_far_above_the_others(act, gap, B, H, n, D, at):
    """Every other weight is exp(-gap) of one token's, whose value is 0: out = w sum v / (1 + (n - 1) w), all terms of one sign,
    so what each term is off by, relative to itself, is what the sum is.

    A weight w of the largest 1: its two parts are right to 2^-16 (bf16) of itself or 2^-22 (fp16) and, there, 2^-37 of the
    largest; the exponent's rounding is gap 2^-22 and exp2's 2^-22, in w and in the sum; a lane adds 8 values a step of 128
    tokens, the matrix unit 32 (off by 2^-23 each), and the pieces of a sequence are at most n / 128."""
    need_gpu()
    say("one key above", act, gap, B, H, n, D, at)
    dt = TYPES[act]
    g = torch.Generator(device="cuda").manual_seed(n + D)
    k = torch.zeros((B, n, H, D), dtype=dt, device="cuda")
    k[:, at, :, 0] = gap
    v = (1024.0 * (0.5 + torch.rand((B, n, H, D), generator=g, device="cuda"))).to(dt)
    v[:, at] = 0
    cache, table, lengths = paged(k, v)
    q = torch.zeros((B, H, D), dtype=dt, device="cuda")
    q[..., 0] = 1
    out, lse = wq.paged_attention(q, cache, table, lengths, scale=1.0, want_lse=True)
    s = float(torch.tensor(gap, dtype=dt))
    w = math.exp(-s)
    total = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
    for t in range(0, n, 4096):
        total += v[:, t:t + 4096].double().sum(1)
    want = w * total / (1 + (n - 1) * w)
    rel = (2.0 ** -16 if act == "bf16" else 2.0 ** -22 + 2.0 ** -37 / w) + 2 * (s + 1) * 2.0 ** -22 \
        + 2 * (32 * n / 128 + 64) * 2.0 ** -23
    off = (out.double() - want).abs()
    assert bool((off <= rel * want + HALF[act] * (1 + rel) * want + TINY[act]).all()), float((off / want).max())
    top = s + math.log1p((n - 1) * w)
    assert float((lse.double() - top).abs().max()) <= (s + 1) * 2.0 ** -22 + (32 * n / 128 + 64) * 2.0 ** -23 + top * 2.0 ** -22
