"""What a decode step writes into the cache is what is read back, bit for bit."""
import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.kv_ref import F8, quantise
from tests.test_gpu_attention_block import B, D, HEADS, KV, P, Block, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quant", [None, "row", "static"])
def test_the_steps_rows_come_back(quant):
    need_gpu()
    say("rows back", quant)
    blk = Block(quant)
    new = []
    for step in range(2 * P + 3):  # into a third page
        blk.x.copy_(inputs(step))
        new.append(blk.step()[0].clone())
    torch.cuda.synchronize()
    new = torch.stack(new, 1).cpu()  # [B, steps, heads, D]
    at = torch.arange(new.shape[1], device="cuda")
    for b in range(B):
        slots = blk.table[b].long()[at // P] * P + at % P
        for got, rows in zip(wq.kv_cache_read(blk.cache, slots, torch.bfloat16),
                             (new[b, :, HEADS:HEADS + KV], new[b, :, HEADS + KV:])):
            if quant is not None:
                codes, c = quantise(rows, quant, 0.03)
                c = c[..., None] if quant == "row" else torch.tensor(0.03)
                rows = (codes.view(F8).float() * c).bfloat16()
            assert tuple(got.shape) == (len(at), KV, D)
            assert torch.equal(got.cpu().view(torch.int16), rows.contiguous().view(torch.int16))
