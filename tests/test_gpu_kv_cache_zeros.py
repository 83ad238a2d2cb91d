"""A zero keeps its sign through kv_cache_write and kv_cache_read: v / c of -0 is -0, a code of its own."""
import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.kv_ref import F8, TYPES, quantise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quant", [None, "row", "static"])
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("D", [16, 128, 176])
def test_zeros_keep_their_sign(act, quant, D):
    need_gpu()
    say("signed zeros", act, quant, D)
    g = torch.Generator().manual_seed(D)
    x = torch.randn((6, 2, D), generator=g)
    x[:, :, 1::4], x[:, :, 2::4] = -0.0, 0.0
    x[1] = torch.where(torch.arange(D) % 2 == 0, -0.0, 0.0)  # a row of zeros
    x[2] *= 60000.0 / x[2].abs().max()
    x[3] *= 2.0 ** -12
    if act == "bf16":
        x[4] *= 2.0 ** 125  # scales beyond 2^100
        x[5] *= 2.0 ** -120
    x = x.to(TYPES[act])
    static = (0.02, 3.0)
    cache = wq.kv_cache(2, 2, 16, D, TYPES[act], quant, *(static if quant == "static" else ()), device="cuda")
    slots = torch.tensor([3, 31, 0, 17, 8, 9])
    wq.kv_cache_write(x.cuda(), (-x).cuda(), cache, slots.cuda())
    back = wq.kv_cache_read(cache, slots.cuda(), TYPES[act])
    for i, rows in enumerate((x, -x)):
        want = rows
        if quant is not None:
            codes, c = quantise(rows, quant, static[i])
            assert torch.equal(cache[i].cpu()[slots // 16, :, slots % 16], codes)
            assert bool((codes[0, :, 1] == (0x80 if i == 0 else 0)).all())
            want = (codes.view(F8).float() * (c[..., None] if quant == "row" else torch.tensor(static[i]))).to(TYPES[act])
        assert torch.equal(back[i].cpu().view(torch.int16), want.view(torch.int16))
