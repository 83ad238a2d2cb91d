"""The serving operators refuse host memory and leave every output as it was:
the buffers handed over are pinned host tensors, which the GPU could read, so a
missing check shows as a wrong status or a written output, never as a fault."""
import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch

pytestmark = pytest.mark.gpu


def pinned(t):
    h = torch.empty(t.shape, dtype=t.dtype, pin_memory=True)
    h.copy_(t.cpu())
    return h


def c_call(fn, *args):
    """Through the C ABI (the binding refuses tensors of two devices itself)."""
    st = getattr(wq.load(), fn)(*[a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args],
                                torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return st, wq.load().wq_last_error().decode()


def each_on_the_host(fn, args, outputs):
    """The call with each tensor argument in host memory, one at a time."""
    for k, a in enumerate(args):
        if not isinstance(a, torch.Tensor):
            continue
        say(fn, "argument", k)
        for t in outputs:
            t.fill_(7)
        st, msg = c_call(fn, *[pinned(v) if i == k else v for i, v in enumerate(args)])
        assert st == wq.WQ_ERR_DEVICE, (fn, k, st, msg)
        assert all(bool((t == 7).all()) for t in outputs)


def test_rms_norm():
    need_gpu()
    x, r, w = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((4, 64), (4, 64), (64,)))
    ro, out = torch.empty_like(x), torch.empty_like(x)
    codes, scales = torch.empty((4, 64), dtype=torch.uint8, device="cuda"), torch.empty(4, device="cuda")
    each_on_the_host("wq_rms_norm", (x, 64, r, 64, w, 4, 64, 1e-6, wq.WQ_BF16, ro, 64, out, 64, codes, scales, 0.0),
                     (ro, out, codes, scales))


def test_route_grouped():
    need_gpu()
    lg, bias = torch.zeros((4, 16), device="cuda"), torch.zeros(16, device="cuda")
    w, ids = torch.empty((4, 2), device="cuda"), torch.empty((4, 2), dtype=torch.int32, device="cuda")
    st, ex, nt = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (128, 8, 4))
    head = (lg, wq._lib.WQ_F32, 4, 16, 2, 1, bias, 4, 2, 0, 1, 1.0)
    each_on_the_host("moe_route_grouped", head + (w, ids), (w, ids))
    each_on_the_host("moe_route_grouped_align", head + (16, w, ids, st, ex, nt, 128), (w, ids, st, ex, nt))


def test_lora():
    need_gpu()
    bf = torch.bfloat16
    x, y = torch.zeros((4, 64), dtype=bf, device="cuda"), torch.zeros((4, 32), dtype=bf, device="cuda")
    ids, s = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(2, device="cuda")
    a, b = torch.zeros((2, 8, 64), dtype=bf, device="cuda"), torch.zeros((2, 32, 8), dtype=bf, device="cuda")
    ws = torch.zeros(wq.dense_lora_workspace_bytes(4, 64, 32, 8, 2), dtype=torch.uint8, device="cuda")
    each_on_the_host("dense_lora_gemm", (x, 64, 4, 64, 32, 8, 2, ids, a, b, s, y, 32, wq.WQ_BF16, ws, ws.numel()), (y, ws))
