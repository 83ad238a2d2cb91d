"""GPU parity of rms_norm against a plain float64 form.

Tolerances: a 16-bit output is off by the rounding's half step plus the float32
arithmetic before it.  That is, relative to y: 2^-24 for s, 2^-24 each for the
mean's division, the two products and the reciprocal scale, 2^-23 for the
reciprocal square root, and half the relative error of the sum of squares,
which a sum of at most 64 values per thread and 10 levels of a tree holds under
74 * 2^-24.  Together under 2^-18.  Where a cancellation leaves s small, s is
still the float32 rounding of the exact sum, so the bound is relative."""
import numpy as np
import pytest

import weight_only_quantized_topk_amd as wq
from tests.gpu_common import need_gpu, say, torch
from tests.serving_ref import HALF, MIN_SCALE, TINY, e4m3_values, rms_norm

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -18
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def f64(t):
    return t.double().cpu().numpy()


def close(got, ref, kind, what, extra=F32):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    lim = (HALF[kind] * (1 + extra) + extra) * np.abs(ref) + TINY[kind]
    bad = ~np.isnan(ref) & (np.abs(got - ref) > lim)
    assert not bad.any(), "%s: %d of %d off, worst %.3g at %s" % (
        what, bad.sum(), bad.size, np.abs(got - ref)[bad].max(), np.argwhere(bad)[0])


def inputs(rows, n, dt, seed, residual=True, weight=True, pad=0):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=g).to(dt).cuda()

    x = rnd(rows, n + pad)[:, :n]
    r = (2 * rnd(rows, n + pad))[:, :n] if residual else None
    w = (1 + 0.2 * rnd(n)) if weight else None
    return x, r, w


def check(x, r, w, kind, quant, want_out=True, what="", eps=EPS, scale=0.03, **kw):
    s, y = rms_norm(f64(x), None if r is None else f64(r), None if w is None else f64(w), eps)
    got = wq.rms_norm(x, w, eps, residual=r, quant=quant, scale=scale if quant == "static" else None,
                      want_out=want_out, **kw)
    torch.cuda.synchronize()
    if r is not None:
        close(f64(got.residual), s, kind, what + " residual", 2.0 ** -24)
    else:
        assert got.residual is None
    if want_out:
        close(f64(got.out), y, kind, what + " out")
    else:
        assert got.out is None
    if quant is None:
        assert got.codes is None and got.scales is None
        return got
    if quant == "row":
        ref = np.maximum(np.abs(y).max(-1) / 448, MIN_SCALE)
        close(f64(got.scales), ref, "f32", what + " scales")
        ref = ref[:, None]
    else:
        assert got.scales is None
        ref = scale
    close(e4m3_values(got.codes.cpu().numpy()), np.clip(y / ref, -448, 448), "e4m3", what + " codes")
    return got


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("quant", [None, "row", "static"])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 64, 250, 512, 520, 1001, 1024, 1032, 2048, 2049, 4096, 4104, 5120, 7168, 8192,
                               8200, 9001, 16384, 16392, 40000])
def test_widths(n, quant, kind):
    """Every width class (a wave, a workgroup, several vectors a thread, the long rows), aligned and not."""
    need_gpu()
    for rows in (1, 5, 67) + ((300,) if n in (520, 1024, 4104, 5120, 8192) else ()):
        say("rms_norm", rows, n, quant, kind)
        check(*inputs(rows, n, DT[kind], n + rows), kind, quant, what="%d x %d" % (rows, n))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_options(kind):
    """No residual, no weight, single outputs, strided rows."""
    need_gpu()
    for n in (96, 1001, 4096):
        for residual in (False, True):
            for weight in (False, True):
                for pad in (0, 8, 3):
                    say("options", n, residual, weight, pad)
                    a = inputs(9, n, DT[kind], n, residual, weight, pad)
                    check(*a, kind, None, what="options")
                    check(*a, kind, "row", False, what="codes only")
        x, r, w = inputs(9, n, DT[kind], 5)
        h = n // 8 * 8 + 16  # a column that starts at 16 bytes, as every pointer
        wide = torch.full((9, h + n + 8), 7.0, dtype=DT[kind], device="cuda")
        check(x, r, w, kind, None, what="strided outputs", out=wide[:, :n], residual_out=wide[:, h:h + n])
        assert bool((wide[:, n:h] == 7).all()) and bool((wide[:, h + n:] == 7).all())


def test_residual_only_through_the_c_call():
    """The residual's sum may be the only output."""
    need_gpu()
    x, r, w = inputs(5, 640, torch.bfloat16, 3)
    ro = torch.empty_like(x)
    s = torch.cuda.current_stream().cuda_stream
    st = wq.load().wq_rms_norm(x.data_ptr(), 640, r.data_ptr(), 640, w.data_ptr(), 5, 640, EPS, wq.WQ_BF16,
                               ro.data_ptr(), 640, None, 0, None, None, 0.0, s)
    assert st == wq.WQ_OK
    torch.cuda.synchronize()
    assert torch.equal(ro, (x.float() + r.float()).bfloat16())


def test_many_rows():
    need_gpu()
    for rows, n in ((70001, 64), (4099, 1024), (2050, 5120)):
        say("many rows", rows, n)
        check(*inputs(rows, n, torch.bfloat16, 1), "bf16", "row", what="%d x %d" % (rows, n))
    # more workgroups than one dimension of a launch is given: 256 and 1024 threads a row
    for rows, n in (((1 << 20) + 3, 520), (4 * (1 << 20) + 9, 8), ((1 << 20) + 5, 2049)):
        say("many rows", rows, n)
        x = torch.full((rows, n), 3.0, dtype=torch.bfloat16, device="cuda")
        x[-1] = torch.arange(n, device="cuda") % 7
        out = wq.rms_norm(x, quant=None).out
        one = wq.rms_norm(x[-1:].clone()).out
        torch.cuda.synchronize()
        assert torch.equal(out[-1:], one) and bool((out[:-1] == 1).all())
        del x, out


@pytest.mark.parametrize("n", [512, 1001, 4096, 40000])
def test_in_place(n):
    """out over x and residual_out over residual, and each other way round."""
    need_gpu()
    x, r, w = inputs(6, n, torch.bfloat16, 2)
    ref = wq.rms_norm(x, w, EPS, residual=r)
    for swap in (False, True):
        a, b = x.clone(), r.clone()
        got = wq.rms_norm(a, w, EPS, residual=b, out=b if swap else a, residual_out=a if swap else b)
        torch.cuda.synchronize()
        assert torch.equal(got.out, ref.out) and torch.equal(got.residual, ref.residual)
        assert got.out.data_ptr() == (b if swap else a).data_ptr()


@pytest.mark.parametrize("n", [256, 1001, 4096, 40000])
def test_extreme_rows(n):
    """Rows of zeros, of bf16's largest values, of tiny values, with infinities and NaN: each touches itself only."""
    need_gpu()
    x, _, w = inputs(8, n, torch.bfloat16, 4)
    x[1] = 0
    x[2] = 3.0e38
    x[3] = x[3] * 1e25
    x[4] = x[4] * 1e-30
    x[5, n // 2] = float("inf")
    x[6, n // 3] = float("nan")
    say("extreme rows", n)
    got = wq.rms_norm(x, w, EPS, quant="row")
    torch.cuda.synchronize()
    keep = [0, 1, 2, 3, 4, 7]
    _, y = rms_norm(f64(x)[keep], None, f64(w), EPS)
    close(f64(got.out)[keep], y, "bf16", "out")
    sc = np.maximum(np.abs(y).max(-1) / 448, MIN_SCALE)
    close(f64(got.scales)[keep], sc, "f32", "scales")
    close(e4m3_values(got.codes.cpu().numpy())[keep], y / sc[:, None], "e4m3", "codes")
    out, codes = f64(got.out), e4m3_values(got.codes.cpu().numpy())
    assert np.isnan(out[5, n // 2]) and np.isnan(codes[5, n // 2])
    others = np.arange(n) != n // 2
    assert (out[5, others] == 0).all() and (codes[5, others] == 0).all()
    assert np.isnan(out[6]).all() and np.isnan(codes[6]).all()


def test_rows_do_not_depend_on_the_batch():
    need_gpu()
    x, r, w = inputs(37, 4096, torch.bfloat16, 6)
    all_ = wq.rms_norm(x, w, EPS, residual=r, quant="row")
    one = wq.rms_norm(x[11:12], w, EPS, residual=r[11:12], quant="row")
    torch.cuda.synchronize()
    assert torch.equal(all_.codes[11:12], one.codes) and torch.equal(all_.out[11:12], one.out)
    assert torch.equal(all_.scales[11:12], one.scales)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n", [520, 1001, 1024, 2048, 4104, 5120, 8192, 16384])
def test_rows_do_not_depend_on_the_number_of_rows(n, kind):
    """The launch shape goes by the rows (up to 256, more) at some widths; a row's bits do not, also where its squares
    pass float32's range."""
    need_gpu()
    x, r, w = inputs(300, n, DT[kind], 6)
    if kind == "bf16":
        x[17] = x[17] * 1e25
    all_ = wq.rms_norm(x, w, EPS, residual=r, quant="row")
    for at, rows in ((0, 1), (17, 1), (0, 256), (40, 257)):
        say("rows", n, kind, at, rows)
        part = wq.rms_norm(x[at:at + rows].clone(), w, EPS, residual=r[at:at + rows].clone(), quant="row")
        torch.cuda.synchronize()
        for a, b in zip(all_, part):
            assert torch.equal(a[at:at + rows], b)


def test_empty_graph_and_stream():
    need_gpu()
    e = wq.rms_norm(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), quant="row")
    assert e.out.shape == (0, 64) and e.scales.shape == (0,)
    x, r, w = inputs(33, 4096, torch.bfloat16, 8)
    ref = wq.rms_norm(x, w, EPS, residual=r, quant="row")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = wq.rms_norm(x, w, EPS, residual=r, quant="row", stream=side.cuda_stream)
    side.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    x2, r2 = x.clone(), r.clone()
    with torch.cuda.stream(side):
        wq.rms_norm(x2, w, EPS, residual=r2, quant="row")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = wq.rms_norm(x2, w, EPS, residual=r2, quant="row")
    for k in range(4):
        x2.copy_(x * (k + 1))
        r2.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        now = wq.rms_norm(x2, w, EPS, residual=r2, quant="row")
        for a, b in zip(held, now):
            assert torch.equal(a, b)
