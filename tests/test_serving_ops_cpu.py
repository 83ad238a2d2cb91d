"""Refusals of the serving operators around the quantised layers, before any
device work: through the C ABI (sizes, codes, pointers, overlaps) and in the
Python binding (shapes, types, strides, which arguments go together)."""
import ctypes as C

import pytest
import torch

import weight_only_quantized_topk_amd as wq

FAKE = 0x100000  # aligned, non-null: only ever seen by host-side validation


def at(off=0):
    return C.c_void_p(FAKE + off)


def status(fn, *args):
    L = wq.load()
    st = getattr(L, fn)(*args)
    return st, L.wq_last_error().decode()


INV, UNS = wq.WQ_ERR_INVALID, wq.WQ_ERR_UNSUPPORTED
BF = wq.WQ_BF16


# ---------------------------------------------------------------------------
# moe_route_grouped, moe_route_grouped_align
# ---------------------------------------------------------------------------
def route_args(align=False, **k):
    d = dict(logits=at(), dt=2, M=4, E=64, topk=4, scoring=0, bias=None, n_group=8, topk_group=2, score=0, renorm=1,
             scale=1.0, bs=16, w=at(), ids=at(), st=at(), ex=at(), nt=at(), cap=1024)
    d.update(k)
    a = [d[n] for n in ("logits", "dt", "M", "E", "topk", "scoring", "bias", "n_group", "topk_group", "score", "renorm",
                        "scale")]
    return a + ([d["bs"], d["w"], d["ids"], d["st"], d["ex"], d["nt"], d["cap"], None] if align
                else [d["w"], d["ids"], None])


@pytest.mark.parametrize("fn", ["moe_route_grouped", "moe_route_grouped_align"])
@pytest.mark.parametrize("change,want", [
    (dict(dt=3), INV), (dict(dt=-1), INV), (dict(M=-1), INV), (dict(topk=0), INV), (dict(topk=65), INV),
    (dict(E=0), INV), (dict(E=2048, n_group=1, topk_group=1), UNS), (dict(topk=17, topk_group=8), UNS),
    (dict(M=1 << 24), UNS), (dict(scoring=2), INV), (dict(score=2), INV), (dict(n_group=0), INV),
    (dict(n_group=7), INV), (dict(n_group=-8), INV), (dict(E=256, n_group=128), UNS), (dict(topk_group=0), INV),
    (dict(topk_group=9), INV), (dict(topk=9, topk_group=1), INV), (dict(n_group=64, topk_group=8, score=1), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(logits=None), INV), (dict(w=None), INV),
    (dict(ids=None), INV), (dict(bias=at(4)), INV), (dict(logits=at(2)), INV)])
def test_route_grouped_refusals(fn, change, want):
    assert status(fn, *route_args(fn.endswith("align"), **change))[0] == want


def test_route_grouped_align_refusals():
    for change, want in ((dict(bs=24), UNS), (dict(bs=0), UNS), (dict(cap=16), INV), (dict(cap=1032), INV),
                         (dict(cap=1 << 31), UNS), (dict(st=None), INV), (dict(ex=at(8)), INV), (dict(nt=None), INV)):
        assert status("moe_route_grouped_align", *route_args(True, **change))[0] == want, change
    assert status("moe_route_grouped", *route_args(M=0, logits=None, w=None, ids=None))[0] == wq.WQ_OK


def test_route_grouped_binding_refusals():
    lg = torch.zeros((4, 64))
    for call in (lambda **k: wq.moe_route_grouped(k.pop("logits", lg), k.pop("topk", 4), **k),
                 lambda **k: wq.moe_route_grouped_align(k.pop("logits", lg), k.pop("topk", 4), 16, **k)):
        with pytest.raises(TypeError):
            call(logits=lg.double())
        with pytest.raises(ValueError):
            call(logits=torch.zeros(64))
        with pytest.raises(ValueError):
            call(logits=torch.zeros((4, 128))[:, ::2])
        with pytest.raises(ValueError):
            call(scoring="relu")
        with pytest.raises(ValueError):
            call(group_score="mean")
        with pytest.raises(ValueError):
            call(topk=0)
        with pytest.raises(ValueError):
            call(topk=1 << 32)
        with pytest.raises(ValueError):
            call(n_group=(1 << 32) + 1)
        with pytest.raises(ValueError):
            call(bias=torch.zeros(63))
        with pytest.raises(TypeError):
            call(bias=torch.zeros(64, dtype=torch.bfloat16))
        with pytest.raises(ValueError):
            call(topk_weights=torch.zeros((4, 5)))
        with pytest.raises(TypeError):
            call(topk_ids=torch.zeros((4, 4), dtype=torch.int64))
    with pytest.raises(ValueError):
        wq.moe_route_grouped_align(lg, 4, 0)
    with pytest.raises(ValueError):
        wq.moe_route_grouped_align(lg, 4, 16, sorted_token_ids=torch.zeros(16, dtype=torch.int32))
    with pytest.raises(TypeError):
        wq.moe_route_grouped_align(lg, 4, 16, num_tokens_post_padded=torch.zeros(1))


# ---------------------------------------------------------------------------
# wq_rms_norm
# ---------------------------------------------------------------------------
MB = 1 << 20


def norm_args(**k):
    d = dict(x=at(), xs=512, r=at(MB), rs=512, w=at(2 * MB), rows=4, n=512, eps=1e-6, dt=BF, ro=at(3 * MB), ros=512,
             out=at(4 * MB), os=512, codes=at(5 * MB), scales=at(6 * MB), static=0.0)
    d.update(k)
    return [d[n] for n in ("x", "xs", "r", "rs", "w", "rows", "n", "eps", "dt", "ro", "ros", "out", "os", "codes",
                           "scales", "static")] + [None]


@pytest.mark.parametrize("change", [
    dict(dt=2), dict(dt=7), dict(rows=-1), dict(n=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(ro=None, out=None, codes=None, scales=None), dict(codes=None), dict(scales=None),
    dict(scales=None, static=float("inf")), dict(scales=None, static=-1.0), dict(xs=511), dict(rs=0), dict(ros=-512),
    dict(os=8), dict(xs=1 << 62), dict(x=None), dict(x=at(2)), dict(out=at(4 * MB + 8)), dict(w=at(2 * MB + 4)),
    dict(codes=at(5 * MB + 1)),
    # overlaps: shifted rows, another stride, outputs on one another, on the weight, codes on x
    dict(out=at(16)), dict(ro=at(MB + 512)), dict(out=at(), os=520), dict(ro=at(4 * MB)), dict(codes=at()),
    dict(scales=at(4 * MB)), dict(out=at(2 * MB)), dict(scales=at(5 * MB)), dict(out=at(2 * MB - 1024)),
    dict(x=at(4 * MB + 512), xs=1024, os=1024)])
def test_rms_norm_refusals(change):
    assert status("wq_rms_norm", *norm_args(**change))[0] == INV


def test_rms_norm_no_rows_and_sizes():
    assert status("wq_rms_norm", *norm_args(rows=0, x=None))[0] == wq.WQ_OK
    assert status("wq_rms_norm", *norm_args(rows=0, ro=None, out=None, codes=None, scales=None))[0] == wq.WQ_OK
    n = (1 << 30) + 8
    assert status("wq_rms_norm", *norm_args(n=n, xs=n, rs=n, ros=n, os=n))[0] == UNS


def test_rms_norm_allowed_overlaps_pass_the_checks():
    """Exact in-place forms and rows in each other's gaps reach the device check (there is no device memory at these
    addresses): the status is another one."""
    for change in (dict(ro=at(MB)), dict(out=at()), dict(ro=at(), out=at(MB)), dict(w=None, r=None, rs=0),
                   dict(x=at(4 * MB + 1024), xs=1024, os=1024), dict(out=at(4 * MB + 1024), os=1024, ro=at(4 * MB), ros=1024)):
        st, msg = status("wq_rms_norm", *norm_args(**change))
        assert st in (wq.WQ_ERR_DEVICE, wq.WQ_ERR_HIP), (change, msg)


def test_rms_norm_binding_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    bad_value = [dict(x=torch.zeros(64, dtype=torch.bfloat16)), dict(x=torch.zeros((4, 128), dtype=torch.bfloat16)[:, ::2]),
                 dict(x=torch.zeros((1, 64), dtype=torch.bfloat16).expand(4, 64)), dict(x=x.float()),
                 dict(weight=torch.ones(63, dtype=torch.bfloat16)), dict(quant="token"), dict(quant="static"),
                 dict(quant="row", scale=1.0), dict(codes=torch.zeros((4, 64), dtype=torch.uint8)),
                 dict(quant="static", scale=1.0, scales=torch.zeros(4)), dict(want_out=False, out=x.clone()),
                 dict(residual_out=x.clone()), dict(residual=torch.zeros((4, 65), dtype=torch.bfloat16)),
                 dict(quant="row", codes=torch.zeros((4, 128), dtype=torch.uint8)[:, :64])]
    bad_type = [dict(weight=w.float()), dict(residual=x.half()), dict(out=x.float()),
                dict(quant="row", codes=torch.zeros((4, 64), dtype=torch.int8)),
                dict(quant="row", scales=torch.zeros(4, dtype=torch.bfloat16))]
    for change in bad_value:
        with pytest.raises(ValueError):
            wq.rms_norm(change.pop("x", x), change.pop("weight", w), **change)
    for change in bad_type:
        with pytest.raises(TypeError):
            wq.rms_norm(x, change.pop("weight", w), **change)


# ---------------------------------------------------------------------------
# moe_fp8_codes_gemm
# ---------------------------------------------------------------------------
def codes_desc(**k):
    d = wq.ops.WqMoeGemmDesc()
    d.struct_size = C.sizeof(d)
    v = dict(stage=0, act_dtype=BF, M=4, topk=2, E=8, n_out=256, k_in=256, group_size=-1, capacity=128, block_size=16,
             d_a=FAKE, d_w_packed=FAKE, d_scales=FAKE, d_sorted_token_ids=FAKE, d_expert_ids=FAKE,
             d_num_tokens_post_padded=FAKE, d_out=FAKE)
    v.update(k)
    for n, x in v.items():
        setattr(d, n, x)
    return C.byref(d)


@pytest.mark.parametrize("change,want", [
    (dict(stage=1), INV), (dict(stage=5), INV), (dict(k_in=200), UNS), (dict(n_out=250), UNS), (dict(d_a=None), INV),
    (dict(d_a=FAKE + 1), INV), (dict(block_size=24), UNS), (dict(capacity=16), INV), (dict(topk=9), INV),
    (dict(d_k_perm=FAKE), INV)])
def test_codes_gemm_refusals(change, want):
    assert status("moe_fp8_codes_gemm", codes_desc(**change), at(), 1.0, 1.0, None)[0] == want


def test_codes_gemm_scales():
    for rows, one, out in ((None, 0.0, 1.0), (None, float("nan"), 1.0), (None, -1.0, 1.0), (at(), 1.0, 0.0),
                           (at(), 1.0, float("inf")), (at(4), 1.0, 1.0)):
        assert status("moe_fp8_codes_gemm", codes_desc(), rows, one, out, None)[0] == INV
    assert status("moe_fp8_codes_gemm", None, None, 1.0, 1.0, None)[0] == INV
    assert status("moe_fp8_codes_gemm", codes_desc(M=0), at(), 1.0, 1.0, None)[0] == wq.WQ_OK


def test_codes_gemm_binding_refusals():
    i32 = torch.zeros(128, dtype=torch.int32)

    def call(codes=torch.zeros((4, 256), dtype=torch.uint8), rows=torch.ones(4),
             out=torch.zeros((128, 128), dtype=torch.uint8), stage=wq.WQ_STAGE_GATE_UP):
        wq.moe_fp8_codes_gemm(stage, codes, rows, 4, 2, 8, 256, 256, i32, i32, i32, i32, i32, 128, 16, out)

    for change in (dict(codes=torch.zeros((4, 255), dtype=torch.uint8)), dict(rows=torch.ones(5)),
                   dict(out=torch.zeros((64, 128), dtype=torch.uint8)),
                   dict(stage=wq.WQ_STAGE_RAW, out=torch.zeros((8, 128))),
                   dict(codes=torch.zeros((4, 512), dtype=torch.uint8)[:, :256])):
        with pytest.raises(ValueError):
            call(**change)
    for change in (dict(codes=torch.zeros((4, 256), dtype=torch.bfloat16)), dict(rows=torch.ones(4).double()),
                   dict(out=torch.zeros((128, 128)))):
        with pytest.raises(TypeError):
            call(**change)


# ---------------------------------------------------------------------------
# dense_lora_gemm
# ---------------------------------------------------------------------------
def lora_args(**k):
    d = dict(x=at(), xs=512, M=4, K=512, N=256, R=16, L=3, ids=at(MB), a=at(2 * MB), b=at(3 * MB), s=at(4 * MB),
             y=at(5 * MB), ys=256, dt=BF, ws=at(6 * MB), wsb=1 << 24)
    d.update(k)
    return [d[n] for n in ("x", "xs", "M", "K", "N", "R", "L", "ids", "a", "b", "s", "y", "ys", "dt", "ws", "wsb")] + [None]


@pytest.mark.parametrize("change,want", [
    (dict(dt=2), INV), (dict(M=-1), INV), (dict(K=0), INV), (dict(N=-8), INV), (dict(R=0), INV), (dict(L=0), INV),
    (dict(K=508), UNS), (dict(N=252), UNS), (dict(R=12), UNS), (dict(R=264), UNS), (dict(M=(1 << 24) + 1), UNS),
    (dict(K=(1 << 24) + 8, xs=(1 << 24) + 8), UNS), (dict(ys=(1 << 25) + 8), UNS),
    (dict(xs=504), INV), (dict(ys=0), INV), (dict(xs=516), UNS), (dict(ys=260), UNS), (dict(wsb=64), INV),
    (dict(x=None), INV), (dict(ids=None), INV), (dict(a=None), INV), (dict(b=at(2)), INV), (dict(s=at(4)), INV),
    (dict(y=None), INV), (dict(ws=None), INV),
    # overlaps
    (dict(y=at()), INV), (dict(y=at(MB)), INV), (dict(y=at(2 * MB)), INV), (dict(y=at(6 * MB)), INV),
    (dict(ws=at(3 * MB)), INV), (dict(ws=at()), INV), (dict(y=at(16)), INV)])
def test_lora_refusals(change, want):
    assert status("dense_lora_gemm", *lora_args(**change))[0] == want


def test_lora_workspace_and_empty():
    L = wq.load()
    assert L.dense_lora_workspace_bytes(0, 512, 256, 16, 3) == 0
    assert L.dense_lora_workspace_bytes(4, 500, 256, 16, 3) == 0
    assert L.dense_lora_workspace_bytes(4, 512, 256, 16, 3) >= 4 * 16 * 4
    need = L.dense_lora_workspace_bytes(4, 512, 256, 16, 3)
    assert status("dense_lora_gemm", *lora_args(wsb=need - 1))[0] == INV
    assert status("dense_lora_gemm", *lora_args(M=0, x=None, y=None, ids=None, ws=None, wsb=0))[0] == wq.WQ_OK
    # y in the gaps of x's rows (one buffer) passes the host's checks
    st, msg = status("dense_lora_gemm", *lora_args(xs=1024, y=at(1024), ys=1024))
    assert st in (wq.WQ_ERR_DEVICE, wq.WQ_ERR_HIP), msg


def test_lora_binding_refusals():
    bf = torch.bfloat16
    x, y = torch.zeros((4, 512), dtype=bf), torch.zeros((4, 256), dtype=bf)
    ids, s = torch.zeros(4, dtype=torch.int32), torch.ones(3)
    a, b = torch.zeros((3, 16, 512), dtype=bf), torch.zeros((3, 256, 16), dtype=bf)
    good = dict(x=x, adapter_ids=ids, a=a, b=b, scales=s, y=y)
    for change in (dict(x=x[0]), dict(a=a[0]), dict(b=b[:2]), dict(a=torch.zeros((3, 16, 504), dtype=bf)), dict(y=y[:3]),
                   dict(adapter_ids=ids[:3]), dict(scales=s[:2]), dict(y=torch.zeros((4, 512), dtype=bf)[:, ::2]),
                   dict(b=torch.zeros((3, 16, 256), dtype=bf).transpose(1, 2)), dict(x=x.float()),
                   dict(workspace=torch.zeros((64, 2), dtype=torch.uint8)[:, 0])):
        with pytest.raises(ValueError):
            wq.dense_lora_gemm(**{**good, **change})
    for change in (dict(y=y.half()), dict(a=a.half()), dict(adapter_ids=ids.long()), dict(scales=s.to(bf))):
        with pytest.raises(TypeError):
            wq.dense_lora_gemm(**{**good, **change})


def test_dense_refuses_bad_adapters_before_it_launches():
    """The binding's checks of the adapters come before the projection: the error is theirs, not the device's."""
    bf = torch.bfloat16
    x, w, s = torch.zeros((4, 512), dtype=bf), torch.zeros(512 * 256, dtype=torch.uint8), torch.zeros(256, dtype=bf)
    ids = torch.zeros(4, dtype=torch.int32)
    a, b = torch.zeros((3, 16, 512), dtype=bf), torch.zeros((3, 256, 16), dtype=bf)
    for bad, err in ((wq.Lora(ids[:3], a, b, None), ValueError), (wq.Lora(ids, a, b[:, :128], None), ValueError),
                     (wq.Lora(ids.long(), a, b, None), TypeError), (wq.Lora(ids, a.half(), b.half(), None), TypeError),
                     (wq.Lora(ids, a[:, :12], b[:, :, :12], None), ValueError),
                     (wq.Lora(ids, a[:, :4].contiguous(), b[:, :, :4].contiguous(), None), ValueError)):
        with pytest.raises(err):
            wq.dense_w8a16_gemm(x, 256, w, s, lora=bad)
    good = wq.Lora(ids, a, b, None)
    with pytest.raises(ValueError):
        wq.dense_w8a16_gemm(x, 256, w, s, out=torch.zeros((4, 512), dtype=bf)[:, :256], lora=good)
    with pytest.raises(ValueError):
        wq.dense_w8a16_gemm(x, 256, w, s, out=torch.zeros((4, 128), dtype=bf), lora=good)


def test_pack_lora():
    low = [(torch.randn(r, 64), torch.randn(32, r), 0.5 * r) for r in (3, 8, 20)]
    a, b, s = wq.pack_lora(low, torch.bfloat16, device="cpu")
    assert a.shape == (3, 24, 64) and b.shape == (3, 32, 24) and s.tolist() == [1.5, 4.0, 10.0]
    for i, (A, B, _) in enumerate(low):
        r = A.shape[0]
        assert torch.equal(a[i, :r], A.bfloat16()) and torch.equal(b[i, :, :r], B.bfloat16())
        assert not a[i, r:].any() and not b[i, :, r:].any()
    for bad in ([], [(torch.randn(3, 64), torch.randn(32, 4), 1.0)],
                [(torch.randn(3, 64), torch.randn(32, 3), 1.0), (torch.randn(3, 65), torch.randn(32, 3), 1.0)]):
        with pytest.raises(ValueError):
            wq.pack_lora(bad, torch.bfloat16, device="cpu")


def test_codes_gemm_binding_refuses_short_or_foreign_arrays():
    """What the kernels read beside the rows: too few values, another type, no contiguous layout."""
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    E, n_out, k_in, cap, bs = 8, 256, 256, 128, 16
    good = dict(w_packed=torch.zeros(E * n_out * k_in, dtype=u8), scales=torch.zeros((E, n_out)),
                sorted_token_ids=torch.zeros(cap, dtype=i32), expert_ids=torch.zeros(cap // bs, dtype=i32),
                num_tokens_post_padded=torch.zeros(1, dtype=i32))

    def call(**change):
        wq.moe_fp8_codes_gemm(wq.WQ_STAGE_GATE_UP, torch.zeros((4, k_in), dtype=u8), torch.ones(4), 4, 2, E, n_out, k_in,
                              capacity=cap, block_size=bs, out=torch.zeros((cap, n_out // 2), dtype=u8),
                              stream=0, **{**good, **change})

    for name, t in good.items():
        flat = t.reshape(-1)
        with pytest.raises(ValueError, match=name):
            call(**{name: flat[:-1]})
        with pytest.raises(ValueError, match=name):
            call(**{name: torch.cat([flat, flat])[::2] if len(flat) > 1 else flat[:0]})
        with pytest.raises(TypeError, match=name):
            call(**{name: t.to(torch.int64)})
    with pytest.raises(wq.WqError):  # as it should be, it goes on to the library, which refuses host memory
        call()


def test_a_router_and_renormalize():
    """renormalize=False is not overruled without a word by a router that renormalises."""
    import types
    p = types.SimpleNamespace(act=torch.bfloat16, act_code=BF, k_perm1=None, bits=8, E=8, K=256, N=128)
    for runner in (wq.MoERunner, wq.Fp8MoERunner):
        with pytest.raises(ValueError, match="renormalize"):
            runner(p, 4, 2, renormalize=False, device="cpu", router=wq.Router())
        for mine, its in ((True, True), (True, False), (False, False)):
            r = runner(p, 4, 2, renormalize=mine, device="cpu", router=wq.Router(renormalize=its))
            assert r.router.renormalize == its
        assert runner(p, 4, 2, renormalize=False, device="cpu").renormalize is False


def test_adapters_the_library_would_refuse_stop_the_projection():
    """Unaligned arrays and too large ones, which dense_lora_gemm refuses, are found before the projection is launched."""
    bf = torch.bfloat16
    x, w, s = torch.zeros((4, 512), dtype=bf), torch.zeros(512 * 256, dtype=torch.uint8), torch.zeros(256, dtype=bf)
    ids, one, work = torch.zeros(5, dtype=torch.int32), torch.ones(4), torch.zeros(1 << 20, dtype=torch.uint8)
    a, b = torch.zeros((3, 16, 512), dtype=bf), torch.zeros((3, 256, 16), dtype=bf)
    for bad, name in ((wq.Lora(ids[1:], a, b, None), "adapter_ids"), (wq.Lora(ids[:4], a, b, one[1:]), "scales"),
                      (wq.Lora(ids[:4], torch.zeros(3 * 16 * 512 + 1, dtype=bf)[1:].view(3, 16, 512), b, None), "a is")):
        with pytest.raises(ValueError, match=name):
            wq.dense_w8a16_gemm(x, 256, w, s, lora=bad, out=torch.zeros((4, 256), dtype=bf), workspace=work, stream=0)
        with pytest.raises(ValueError, match=name):
            wq.dense_lora_gemm(x, *bad, torch.zeros((4, 256), dtype=bf), stream=0)
    with pytest.raises(wq.WqError):  # as they should be, the call goes on to the library, which refuses host memory
        wq.dense_w8a16_gemm(x, 256, w, s, lora=wq.Lora(ids[:4], a, b, one[:3]), out=torch.zeros((4, 256), dtype=bf),
                            workspace=work, stream=0)
    assert wq.dense_lora_workspace_bytes(4, 512, 1 << 24, 128, 1) == 0
    assert status("dense_lora_gemm", *lora_args(N=1 << 24, R=128, ys=1 << 24))[0] == UNS


def test_codes_gemm_row_limit():
    """More token tiles than a grid dimension takes are refused before any device work."""
    for bs, tile in ((64, 64), (128, 128), (256, 128)):
        M = 65535 * tile // 2 + 1
        cap = wq.moe_align_capacity(M, 2, 8, bs)
        how = dict(M=M, capacity=cap, block_size=bs, k_in=128)
        assert status("moe_fp8_codes_gemm", codes_desc(**how), at(), 1.0, 1.0, None)[0] == UNS
    how = dict(M=65535 * 32 - 1000, k_in=128, block_size=64)
    how["capacity"] = wq.moe_align_capacity(how["M"], 2, 8, 64)
    assert status("moe_fp8_codes_gemm", codes_desc(**how), at(), 1.0, 1.0, None)[0] in (wq.WQ_ERR_DEVICE, wq.WQ_ERR_HIP)
