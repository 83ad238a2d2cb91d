"""Refusals of the paged cache's operators before any device work: through the C
ABI and in the Python binding."""
import ctypes as C

import pytest
import torch

import weight_only_quantized_topk_amd as wq
from weight_only_quantized_topk_amd._lib import WqKvCache

GB = 1 << 30
FAKE = 1 << 40  # aligned, non-null: only ever seen by host-side validation
INV, UNS = wq.WQ_ERR_INVALID, wq.WQ_ERR_UNSUPPORTED
NO_DEVICE = (wq.WQ_ERR_DEVICE, wq.WQ_ERR_HIP)  # past the checks: there is no device memory at these addresses


def at(off=0):
    return C.c_void_p(FAKE + off)


def desc(**k):
    d = dict(struct_size=C.sizeof(WqKvCache), d_k=FAKE, d_v=FAKE + GB, d_k_scales=FAKE + 2 * GB, d_v_scales=FAKE + 3 * GB,
             k_scale=0.0, v_scale=0.0, dtype=3, pages=100, kv_heads=8, page_size=16, head_dim=128)
    d.update(k)
    return C.byref(WqKvCache(**d))


def status(fn, *args):
    L = wq.load()
    return getattr(L, fn)(*args), L.wq_last_error().decode()


def rows(write, cache=None, **k):
    d = dict(k=at(4 * GB), ks=2048, v=at(4 * GB + 2048), vs=2048, slots=at(5 * GB), T=4, dt=wq.WQ_BF16)
    d.update(k)
    c = desc() if cache is None else cache
    if write:
        return status("wq_kv_cache_write", c, d["k"], d["ks"], d["v"], d["vs"], d["slots"], d["T"], d["dt"], None)
    return status("wq_kv_cache_read", c, d["slots"], d["T"], d["k"], d["ks"], d["v"], d["vs"], d["dt"], None)


def attend(cache=None, **k):
    d = dict(q=at(4 * GB), qs=4096, B=4, heads=32, table=at(5 * GB), width=64, n=at(5 * GB + 4096), scale=0.1, window=0,
             out=at(6 * GB), os=4096, lse=at(7 * GB), dt=wq.WQ_BF16, ws=at(8 * GB), nb=GB)
    d.update(k)
    return status("wq_paged_attention", desc() if cache is None else cache, d["q"], d["qs"], d["B"], d["heads"], d["table"],
                  d["width"], d["n"], d["scale"], d["window"], d["out"], d["os"], d["lse"], d["dt"], d["ws"], d["nb"], None)


CALLS = [lambda c: rows(True, c), lambda c: rows(False, c), attend]


@pytest.mark.parametrize("change,want", [
    (dict(struct_size=8), INV), (dict(dtype=0), INV), (dict(dtype=2), INV), (dict(dtype=4), INV), (dict(pages=0), INV),
    (dict(kv_heads=0), INV), (dict(page_size=0), INV), (dict(head_dim=0), INV), (dict(pages=-1), INV),
    (dict(page_size=8), UNS), (dict(page_size=24), UNS), (dict(page_size=8192), UNS), (dict(head_dim=72), UNS),
    (dict(head_dim=272), UNS), (dict(pages=1 << 27), UNS), (dict(kv_heads=65536), UNS), (dict(d_k=None), INV),
    (dict(d_v=None), INV), (dict(d_k=FAKE + 8), INV), (dict(d_v=FAKE + GB + 1), INV), (dict(d_k_scales=None), INV),
    (dict(d_v_scales=None), INV), (dict(d_v_scales=FAKE + 3 * GB + 4), INV), (dict(dtype=wq.WQ_BF16), INV),
    (dict(d_k_scales=None, d_v_scales=None), INV),
    (dict(d_k_scales=None, d_v_scales=None, k_scale=1.0, v_scale=float("nan")), INV),
    (dict(d_k_scales=None, d_v_scales=None, k_scale=-1.0, v_scale=1.0), INV),
    (dict(d_k_scales=None, d_v_scales=None, k_scale=1e-31, v_scale=1.0), INV),
    (dict(d_k_scales=None, d_v_scales=None, k_scale=1.0, v_scale=float("inf")), INV)])
def test_cache_refusals(change, want):
    for call in CALLS:
        st, msg = call(desc(**change))
        assert st == want, (change, msg)


def test_null_cache():
    for call in CALLS:
        assert call(C.cast(None, C.POINTER(WqKvCache)))[0] == INV


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INV), (dict(T=(1 << 24) + 1), UNS), (dict(dt=2), INV), (dict(ks=1023), INV), (dict(vs=0), INV),
    (dict(vs=-2048), INV), (dict(ks=1 << 62), INV), (dict(ks=1028), UNS), (dict(k=None), INV), (dict(v=None), INV),
    (dict(slots=None), INV), (dict(k=at(4 * GB + 8)), INV), (dict(slots=at(5 * GB + 8)), INV),
    (dict(k=at(16)), INV), (dict(v=at(2 * GB + 64)), INV), (dict(slots=at(GB)), INV)])
def test_rows_refusals(write, change, want):
    st, msg = rows(write, **change)
    assert st == want, msg


def test_rows_overlaps():
    # two arrays of the cache on one another: written together, not read
    for change in (dict(d_v=FAKE), dict(d_k_scales=FAKE + 64), dict(d_v_scales=FAKE + 2 * GB)):
        assert rows(True, desc(**change))[0] == INV
        assert rows(False, desc(**change))[0] in NO_DEVICE
    # outputs on one another; in each other's gaps they are fine, and inputs may be the same
    assert rows(False, v=at(4 * GB + 1024))[0] == INV
    assert rows(False, slots=at(4 * GB + 4096))[0] == INV
    assert rows(True, v=at(4 * GB))[0] in NO_DEVICE
    assert rows(True)[0] in NO_DEVICE and rows(False)[0] in NO_DEVICE


def test_no_rows():
    for write in (True, False):
        assert rows(write, T=0, k=None, v=None, slots=None)[0] == wq.WQ_OK
    assert attend(B=0, q=None, table=None, n=None, out=None, lse=None, ws=None, nb=0)[0] == wq.WQ_OK


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), INV), (dict(heads=0), INV), (dict(heads=12), INV), (dict(width=0), INV), (dict(window=-1), INV),
    (dict(dt=3), INV), (dict(B=65536), UNS), (dict(heads=65536), UNS), (dict(width=(1 << 26) + 1), UNS),
    (dict(B=65535, width=1 << 21), UNS), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(qs=4095), INV),
    (dict(os=4088), INV), (dict(qs=4100), UNS), (dict(os=1 << 62), INV), (dict(q=None), INV), (dict(table=None), INV),
    (dict(n=None), INV), (dict(out=None), INV), (dict(ws=None), INV), (dict(nb=1024), INV), (dict(q=at(4 * GB + 8)), INV),
    (dict(lse=at(7 * GB + 4)), INV), (dict(ws=at(8 * GB + 8)), INV), (dict(out=at(4 * GB + 16)), INV),
    (dict(out=at(5 * GB)), INV), (dict(out=at(GB)), INV), (dict(lse=at(6 * GB)), INV), (dict(lse=at(4 * GB)), INV),
    (dict(ws=at(6 * GB)), INV), (dict(ws=at(2 * GB)), INV), (dict(lse=at(3 * GB)), INV)])
def test_attention_refusals(change, want):
    st, msg = attend(**change)
    assert st == want, (change, msg)


def test_scales_whose_product_is_not_finite():
    fixed = desc(k_scale=2.0 ** 100, v_scale=1.0, d_k_scales=None, d_v_scales=None)
    assert attend(fixed, scale=3e38)[0] == INV and attend(fixed, scale=1.0)[0] in NO_DEVICE


def test_attention_allowed():
    for change in (dict(lse=None), dict(out=at(4 * GB + 8192), os=8192, qs=8192), dict(width=1, ws=None, nb=0)):
        st, msg = attend(**change)
        assert st in NO_DEVICE, (change, msg)
    st, msg = attend(desc(page_size=4096), width=1 << 16)  # page index by a multiplication: not exact there
    assert st == UNS, msg


def test_workspace_bytes():
    f = wq.paged_attention_workspace_bytes
    assert f(1, 32, 8, 128, 16, 4) == 0          # short tables: no split
    assert f(0, 32, 8, 128, 16, 4096) == 0
    assert f(1, 32, 8, 128, 16, 4096, 64) == 0   # nor under a short window
    one, many = f(1, 32, 8, 128, 16, 4096), f(64, 32, 8, 128, 16, 4096)
    assert 0 < one <= many
    with pytest.raises(ValueError):
        f(1 << 32, 32, 8, 128, 16, 4)


BFT = torch.bfloat16


def cache(quant=None, **k):
    d = dict(pages=4, kv_heads=2, page_size=16, head_dim=32, act=BFT, device="cpu")
    if quant == "static":
        d.update(k_scale=0.1, v_scale=0.1)
    d.update(k)
    return wq.kv_cache(quant=quant, **d)


def refused(call, *kinds):
    with pytest.raises(kinds or ValueError):
        call()


def test_kv_cache_binding():
    assert cache().k.shape == (4, 2, 16, 32) and cache().k.dtype == BFT and cache().k_scale is None
    c = cache("row")
    assert c.k.dtype == torch.uint8 and c.v_scale.shape == (4, 2, 16) and c.v_scale.dtype == torch.float32
    refused(lambda: cache("int8"))
    refused(lambda: cache(k_scale=1.0))
    refused(lambda: cache("static", v_scale=None))
    refused(lambda: cache(act=torch.float32))


def test_write_and_read_binding_refusals():
    x = torch.zeros((3, 2, 32), dtype=BFT)
    s = torch.zeros(3, dtype=torch.int64)
    w = lambda k=x, v=x, c=cache("row"), slots=s: wq.kv_cache_write(k, v, c, slots)  # noqa: E731
    r = lambda c=cache("row"), slots=s, act=BFT, **kw: wq.kv_cache_read(c, slots, act, **kw)  # noqa: E731
    refused(lambda: w(k=x.float()), TypeError, ValueError)
    refused(lambda: w(v=x.half()), TypeError)
    refused(lambda: w(k=torch.zeros((3, 2, 16), dtype=BFT)))
    refused(lambda: w(k=torch.zeros((), dtype=BFT)))
    refused(lambda: w(k=torch.zeros((3, 3, 32), dtype=BFT)))
    refused(lambda: w(v=torch.zeros((4, 2, 32), dtype=BFT)))
    refused(lambda: w(k=torch.zeros((3, 2, 64), dtype=BFT)[:, :, ::2]))
    refused(lambda: w(k=torch.zeros((3, 32, 2), dtype=BFT).transpose(1, 2)))
    refused(lambda: w(k=torch.zeros((1, 2, 32), dtype=BFT).expand(3, 2, 32)))
    refused(lambda: w(slots=s.int()), TypeError)
    refused(lambda: w(slots=s[:2]))
    refused(lambda: w(slots=torch.zeros(6, dtype=torch.int64)[::2]))
    refused(lambda: r(slots=s[:, None]))
    refused(lambda: r(act=torch.float32))
    refused(lambda: r(k=torch.zeros((3, 2, 33), dtype=BFT)))
    refused(lambda: r(v=x.half()), TypeError)
    good = cache("row")
    for c in (good._replace(k=good.k[:, :, ::2]), good._replace(v=good.v[:3]), good._replace(v=cache().v),
              good._replace(k_scale=None), good._replace(k_scale=1.0), good._replace(k_scale=None, v_scale=None),
              good._replace(v_scale=good.v_scale.double()), good._replace(k_scale=good.k_scale[:, :1]),
              good._replace(k=good.k[0]), cache()._replace(k_scale=1.0, v_scale=1.0)):
        refused(lambda: w(c=c), ValueError, TypeError)
        refused(lambda: r(c=c), ValueError, TypeError)
    refused(lambda: w(c=cache(act=torch.float16)), TypeError)
    refused(lambda: r(c=cache(), act=torch.float16), TypeError)


def test_attention_binding_refusals():
    q = torch.zeros((3, 4, 32), dtype=BFT)
    tab, n = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)

    def call(**k):
        d = dict(q=q, cache=cache("row"), block_table=tab, lengths=n)
        d.update(k)
        return wq.paged_attention(**d)

    for k in (dict(q=q[0]), dict(q=torch.zeros((3, 3, 32), dtype=BFT)), dict(q=torch.zeros((3, 4, 16), dtype=BFT)),
              dict(q=torch.zeros((3, 8, 32), dtype=BFT)[:, ::2]), dict(block_table=tab[:2]), dict(block_table=tab[0]),
              dict(block_table=torch.zeros((3, 4), dtype=torch.int32)[:, ::2]), dict(lengths=n[:2]), dict(window=1 << 40),
              dict(lse=torch.zeros((3, 4))), dict(want_lse=True, lse=torch.zeros((3, 5))), dict(out=q[:2]),
              dict(workspace=torch.zeros(100, dtype=torch.uint8)[::2])):
        refused(lambda: call(**k))
    for k in (dict(q=q.half(), cache=cache()), dict(block_table=tab.long()), dict(lengths=n.long()), dict(out=q.half()),
              dict(want_lse=True, lse=torch.zeros((3, 4), dtype=BFT))):
        refused(lambda: call(**k), TypeError)


# ---------------------------------------------------------------------------
# dense projections with an epilogue
# ---------------------------------------------------------------------------
def dense(bits=8, epi=None, **k):
    from weight_only_quantized_topk_amd._lib import WqEpilogue
    d = dict(x=at(), M=4, K=256, N=64, w=at(GB), s=at(2 * GB), group=128, perm=None, y=at(3 * GB), dt=wq.WQ_F16, ws=at(8 * GB),
             nb=GB, struct_size=C.sizeof(WqEpilogue), bias=FAKE + 4 * GB, act=2, r=FAKE + 5 * GB, rs=64)
    d.update(k)
    e = C.byref(WqEpilogue(d["struct_size"], d["bias"], d["r"], d["rs"], d["act"])) if epi is None else epi
    head = [d["x"], d["M"], d["K"], d["N"], d["w"], d["s"]]
    tail = [e, d["y"], d["dt"], d["ws"], d["nb"], None]
    if bits == 4:
        return status("dense_w4a16_epilogue_gemm", *head, d["group"], d["perm"], *tail)
    return status("dense_w8a16_epilogue_gemm", *head, *tail)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("change,want", [
    (dict(M=-1), INV), (dict(K=0), INV), (dict(N=0), INV), (dict(dt=2), INV), (dict(K=96), UNS), (dict(N=72, rs=72), UNS),
    (dict(M=(1 << 24) + 1), UNS), (dict(M=65535 * 64 + 1), UNS), (dict(M=1 << 20, K=8192), UNS), (dict(struct_size=0), INV),
    (dict(act=5), INV), (dict(act=-1), INV), (dict(rs=63), INV), (dict(rs=0), INV), (dict(rs=1 << 62), INV), (dict(rs=68), UNS),
    (dict(x=None), INV), (dict(w=None), INV), (dict(s=None), INV), (dict(y=None), INV), (dict(x=at(8)), INV),
    (dict(bias=FAKE + 4), INV), (dict(r=FAKE + 8), INV), (dict(y=at(GB)), INV), (dict(y=at(4 * GB)), INV),
    (dict(y=at(1024)), INV), (dict(y=at(5 * GB + 16)), INV), (dict(y=at(5 * GB), rs=128), INV)])
def test_dense_refusals(bits, change, want):
    st, msg = dense(bits, **change)
    assert st == want, (change, msg)


def test_dense_workspace_and_forms():
    f = wq.dense_epilogue_workspace_bytes
    assert f(8, 64, 4096, 4096) == 0 and f(8, 0, 4096, 4096) == 0 and f(8, 64, 100, 64) == 0
    assert f(4, 5, 256, 64, True) > 0
    many = f(8, 129, 8192, 1040)
    assert many > 0  # K is split there
    big = dict(M=129, K=8192, N=1040, rs=1040)
    assert dense(8, nb=many - 1, **big)[0] == INV
    for change in (dict(ws=None), dict(ws=at(8 * GB + 16)), dict(ws=at(3 * GB)), dict(ws=at(5 * GB)), dict(ws=at(GB))):
        assert dense(8, **{**big, **change})[0] == INV, change
    assert dense(8, **big)[0] in NO_DEVICE
    from weight_only_quantized_topk_amd._lib import WqEpilogue
    assert dense(8, epi=C.cast(None, C.POINTER(WqEpilogue)))[0] == INV
    for change in (dict(y=at(5 * GB)), dict(bias=None), dict(r=None, rs=0), dict(bias=None, r=None, rs=0, act=0)):
        assert dense(8, **change)[0] in NO_DEVICE, change
    assert dense(4, dt=wq.WQ_BF16)[0] == UNS and dense(4, group=64)[0] == UNS
    assert dense(8, M=0, x=None, y=None, r=None)[0] == wq.WQ_OK


def test_dense_binding_refusals():
    x, b, r = torch.zeros((4, 256), dtype=BFT), torch.zeros(64, dtype=BFT), torch.zeros((4, 64), dtype=BFT)
    w, s = torch.zeros(64 * 256, dtype=torch.int8), torch.zeros(64, dtype=torch.int16)

    def call(x=x, N=64, w=w, s=s, **k):
        return wq.dense_w8a16_gemm(x, N, w, s, **k)

    lora = wq.Lora(torch.zeros(4, dtype=torch.int32), torch.zeros((1, 8, 256), dtype=BFT), torch.zeros((1, 64, 8), dtype=BFT), None)
    for k in (dict(activation="swish"), dict(bias=b[:63]), dict(bias=torch.zeros(128, dtype=BFT)[::2]), dict(residual=r[:3]),
              dict(residual=torch.zeros((4, 128), dtype=BFT)[:, ::2]), dict(bias=b, out=torch.zeros((4, 128), dtype=BFT)[:, :64]),
              dict(bias=b, out=r[:3]), dict(bias=b, x=x[:, ::2]), dict(bias=b, x=x[0]), dict(bias=b, w=w[:-1]), dict(bias=b, s=s[:-1]),
              dict(activation="gelu", lora=lora), dict(bias=b, workspace=torch.zeros(64, dtype=torch.uint8)[::2]),
              dict(bias=b, N=1 << 40)):
        refused(lambda: call(**k))
    for k in (dict(bias=b.half()), dict(residual=r.float()), dict(bias=b, out=r.half()), dict(bias=b, s=s.float())):
        refused(lambda: call(**k), TypeError)
    with pytest.raises(TypeError):
        wq.dense_w4a16_gemm(x.half(), 64, w, s.repeat(2), bias=b.half(), k_perm=torch.zeros(256))
