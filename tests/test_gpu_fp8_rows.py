"""quantize_fp8, rmsnorm_fp8 and rmsnorm_backward against plain NumPy: codes
and scales of the quantiser for equality (its definition is float32
arithmetic), the norm and its gradient in float64 within bounds derived from
the arithmetic, and the gradient against differences."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
import software_pipelined_tiled_pipeline_gb300 as gp

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 128), (3, 16), (8, 130), (127, 129), (128, 256), (130, 127), (1, 4096), (333, 1000), (200, 2056),
          (16, 5000), (257, 640)]


def matrix(rows, cols, type, rng, ld=None, scale=1.0):
    x = scale * rng.standard_normal((rows, cols)) * np.exp2(2 * rng.standard_normal((rows, 1)))
    wide = torch.full((rows, ld or cols), float("nan"), dtype=ref.REAL[type], device="cuda")
    wide[:, :cols] = torch.from_numpy(x).cuda().to(ref.REAL[type])
    return wide[:, :cols]


def check_codes(data, scales, x, kind, fmt):
    want, s = ref.quantize(x, kind, fmt)
    assert data.dtype == ref.TORCH[fmt] and data.stride(0) % 16 == 0
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    got = ref.codes(data)
    assert ref.same_codes(got, want, fmt), np.argwhere(got != want)[:3]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", ["rows", "blocks"])
@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
def test_quantize(rows, cols, kind, type):
    rng = np.random.default_rng(rows + cols)
    fmt = "e4m3" if (rows + cols) % 2 else "e5m2"
    x = matrix(rows, cols, type, rng)
    host = x.float().cpu().numpy()
    q, s, qt, st = gp.quantize_fp8(x, kind, format=fmt, transpose=True)
    assert gp.gemm_stats(sync=True)["status"] == 0
    check_codes(q, s, host, kind, fmt)
    check_codes(qt, st, host.T, kind, fmt)
    alone = gp.quantize_fp8(x, kind, format=fmt)
    only = gp.quantize_fp8(x, kind, format=fmt, transpose="only")
    assert torch.equal(alone[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(alone[1], s)
    assert torch.equal(only[0].view(torch.uint8), qt.view(torch.uint8)) and torch.equal(only[1], st)
    np.testing.assert_array_equal(gp.dequantize_fp8(q, s, torch.float64).cpu().numpy(),
                                  ref.values(ref.codes(q), s.cpu().numpy(), fmt))


@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 8, 24])
def test_quantize_strides_and_rows_off_16_bytes(type, pad):
    rng = np.random.default_rng(pad)
    x = matrix(150, 200, type, rng, ld=200 + pad)
    q, s, qt, st = gp.quantize_fp8(x, "rows", transpose=True)
    check_codes(q, s, x.float().cpu().numpy(), "rows", "e4m3")
    check_codes(qt, st, x.float().cpu().numpy().T, "rows", "e4m3")
    y = x[3:, 1:]                                       # begins one element further
    q, s = gp.quantize_fp8(y, "blocks")
    check_codes(q, s, y.float().cpu().numpy(), "blocks", "e4m3")


@pytest.mark.parametrize("kind", ["rows", "blocks"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_zeros_extremes_and_not_finite(kind, fmt):
    x = np.random.default_rng(1).standard_normal((300, 300)).astype(np.float32)
    x[5, :] = 0.0
    x[130:260, 128:256] = 0.0                           # a block of zeros
    x[7, :128] *= 1e-30                                 # a scale below the least one
    x[8, :128] *= 1e38
    x[9, 3] = np.inf
    x[10, 200] = np.nan
    x[11, 130], x[11, 131] = -np.inf, np.nan
    x[12, :128] = np.float32(3.4e38)
    t = torch.from_numpy(x).cuda()
    q, s, qt, st = gp.quantize_fp8(t, kind, format=fmt, transpose=True)
    for got, scales, src in ((q, s, x), (qt, st, x.T)):
        want, ws = ref.quantize(src, kind, fmt)
        np.testing.assert_array_equal(scales.cpu().numpy(), ws)
        assert ref.same_codes(ref.codes(got), want, fmt)


def test_quantize_writes_nothing_between_rows():
    x = torch.randn(130, 200, device="cuda")
    from software_pipelined_tiled_pipeline_gb300 import _binding as b
    bufs, mats = [], []
    for rows, cols, groups in ((130, 200, 130), (200, 130, 200)):
        ld = 256
        data = torch.full((rows + 2, ld), 0xAB, dtype=torch.uint8, device="cuda")
        s = torch.full((groups + 2, 4), -1.0, device="cuda")
        bufs.append((data, s, rows, cols, groups))
        mats.append(b.GpFp8Matrix(data[1:].data_ptr(), s[1:].data_ptr(), ld, 4, 1, 0, 1))
    assert gp.lib().fp8_quantize(x.data_ptr(), 200, 130, 200, 2, mats[0], mats[1], None) == 0
    torch.cuda.synchronize()
    for data, s, rows, cols, groups in bufs:
        assert bool((data[0] == 0xAB).all() and (data[-1] == 0xAB).all() and (data[:, cols:] == 0xAB).all())
        blocks = -(-cols // 128)
        assert bool((s[0] == -1).all() and (s[-1] == -1).all() and (s[:, blocks:] == -1).all())
        assert bool((s[1:-1, :blocks] > 0).all())


def test_quantize_offsets_past_32_bits():
    rows, ld = 140, 1 << 25                             # 4.7e9 elements
    x = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")[:, :200]
    x.copy_(torch.randn(rows, 200, device="cuda"))
    q, s = gp.quantize_fp8(x)
    check_codes(q, s, x.float().cpu().numpy(), "rows", "e4m3")


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
NORM_SHAPES = [(1, 1), (2, 7), (5, 128), (70, 200), (3, 256), (9, 1000), (1, 4096), (4, 2049), (300, 2056), (3, 8192),
               (2, 16384), (2, 16385), (3, 20001), (1, 40000)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(rows, cols, type, residual):
    rng = np.random.default_rng(rows * 3 + cols)
    fmt = "e5m2" if rows == 3 else "e4m3"
    wtype = "f32" if cols % 2 else type
    x = matrix(rows, cols, type, rng)
    r = matrix(rows, cols, type, rng) if residual else None
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(cols)).cuda().to(ref.REAL[wtype])
    q, s, h, rstd, y = gp.rmsnorm_fp8(x, w, r, eps=1e-5, format=fmt, normed=True)
    assert gp.gemm_stats(sync=True)["status"] == 0
    if residual:
        want_h = (x.float() + r.float()).to(x.dtype)
        assert torch.equal(h, want_h)
    else:
        assert h is x
    check_norm(q, s, rstd, y, h, w, 1e-5, type, fmt)


def check_norm(q, s, rstd, y, h, w, eps, type, fmt):
    hd, wd = ref.f64(h), ref.f64(w)
    cols = hd.shape[1]
    want = 1.0 / np.sqrt((hd * hd).sum(1) / cols + eps)
    # a sum of `cols` squares with at most cols / 256 + 20 additions in a row in FP32, halved by the root
    rel = (cols / 256 + 24) * 2.0 ** -24
    np.testing.assert_allclose(rstd.cpu().numpy(), want, rtol=rel)
    yd = hd * want[:, None] * wd
    least = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}[type]
    near = (rel + 4 * 2.0 ** -24) * np.abs(yd)
    assert np.all(np.abs(ref.f64(y) - yd) <= near + ref.UNIT[type] * (np.abs(yd) + near) + least)
    # scales follow the largest value; the codes' values are off by the rounding of y to the format
    ws = np.maximum(ref.group_max(yd, 1) / ref.FMAX[fmt], float(ref.FLOOR))
    np.testing.assert_allclose(s.cpu().numpy(), ws, rtol=rel + 8 * 2.0 ** -24)
    got = ref.values(ref.codes(q), s.cpu().numpy(), fmt)
    wide = ref.spread(ws, *yd.shape, 1)
    unit, small = (2.0 ** -4, 2.0 ** -10) if fmt == "e4m3" else (2.0 ** -3, 2.0 ** -17)
    assert np.all(np.abs(got - yd) <= (1 + 1e-4) * np.maximum(unit * np.abs(yd), small * wide))


def test_norm_in_place_strides_and_no_quantisation():
    rng = np.random.default_rng(2)
    for type, cols in (("bf16", 1000), ("f32", 333), ("f16", 17000)):
        x, r = matrix(20, cols, type, rng, ld=cols + 7), matrix(20, cols, type, rng, ld=cols + 8)
        w = torch.ones(cols + 1, device="cuda")[1:]     # 4 bytes off a 16-byte boundary
        q, s, h, rstd, y = gp.rmsnorm_fp8(x, w, r, normed=True)
        check_norm(q, s, rstd, y, h, w, 1e-6, type, "e4m3")
        real = {"f16": 0, "bf16": 1, "f32": 2}[type]
        # (the order of a row's FP32 sum follows its alignment: the same bits for the same strides)
        q, s, h, rstd = gp.rmsnorm_fp8(x.contiguous(), w, r.contiguous())
        check_norm(q, s, rstd, y, h, w, 1e-6, type, "e4m3")
        for place in (x, r):                            # h over x, then over the residual
            xx, rr = x.clone(), r.clone()
            at = xx if place is x else rr
            got = torch.empty_like(rstd)
            assert gp.lib().fp8_rmsnorm(xx.data_ptr(), cols, rr.data_ptr(), cols, w.data_ptr(), 2, 1e-6, 20, cols, real,
                                        at.data_ptr(), cols, got.data_ptr(), None, 0, None, None) == 0
            torch.cuda.synchronize()
            assert torch.equal(at, h) and torch.equal(got, rstd)


def test_norm_of_zeros_and_not_finite():
    x = torch.randn(6, 300, device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    w = torch.ones(300, device="cuda")
    q, s, h, rstd, y = gp.rmsnorm_fp8(x, w, eps=1e-6, normed=True)
    v = gp.dequantize_fp8(q, s)
    assert bool((v[1] == 0).all()) and abs(float(rstd[1]) - 1000.0) < 1e-3
    assert bool(torch.isnan(v[2]).all()) and bool(torch.isnan(v[3, 7]))
    for r in (0, 4, 5):
        check_norm(q[r:r + 1], s[r:r + 1], rstd[r:r + 1], y[r:r + 1], h[r:r + 1], w, 1e-6, "f32", "e4m3")
    z = gp.rmsnorm_fp8(torch.zeros(2, 64, device="cuda"), w[:64], eps=0.0)   # 1 / sqrt(0): infinite
    assert bool(torch.isinf(z[3]).all())


def grad_f64(dy, h, w, rstd, dres):
    unit = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - unit * (g * unit).mean(1, keepdims=True))
    return dx + (0 if dres is None else dres), (dy * unit).sum(0)


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(1000, 64), (700, 3000)])
@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_gradient(rows, cols, type, residual):
    rng = np.random.default_rng(rows + 5 * cols)
    pad = 8 if cols % 2 else 0
    dy, h = matrix(rows, cols, type, rng, ld=cols + pad), matrix(rows, cols, type, rng)
    dres = matrix(rows, cols, type, rng, ld=cols + 1) if residual else None
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(cols)).cuda().to(ref.REAL["f32" if rows % 2 else type])
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dx, dw = gp.rmsnorm_backward(dy, h, w, rstd, dres)
    assert gp.gemm_stats(sync=True)["status"] == 0
    D, H, W, R = ref.f64(dy), ref.f64(h), ref.f64(w), ref.f64(rstd)
    E = None if dres is None else ref.f64(dres)
    want, want_w = grad_f64(D, H, W, R, E)
    # the mean: cols products, at most cols / 256 + 20 additions in a row; four more roundings around it
    unit = H * R[:, None]
    mean_mag = (np.abs(D * W * unit)).mean(1, keepdims=True)
    e = 2.0 ** -24
    err = R[:, None] * (4 * e * np.abs(D * W) + ((cols / 256 + 28) * e) * np.abs(unit) * mean_mag) + 2 * e * (
        np.abs(want) + (0 if E is None else np.abs(E)) + R[:, None] * (np.abs(D * W) + np.abs(unit) * mean_mag))
    least = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -149}[type]
    assert np.all(np.abs(ref.f64(dx) - want) <= err + ref.UNIT[type] * (np.abs(want) + err) + least)
    mag = np.abs(D * unit).sum(0)
    assert np.all(np.abs(dw.cpu().numpy() - want_w) <= (rows / 8 + 48) * e * mag + 1e-40)
    again = gp.rmsnorm_backward(dy, h, w, rstd, dres, weight_grad=False)
    assert again[1] is None and torch.equal(again[0], dx)


@pytest.mark.parametrize("cols", [5, 300, 2100])
def test_norm_gradient_against_differences(cols):
    # central differences of L = sum(c * y) in float64; the kernel runs in float32
    rng = np.random.default_rng(cols)
    rows, eps, step = 3, 1e-5, 1e-5
    h, c, w = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols)), 1 + 0.2 * rng.standard_normal(cols)

    def loss(h, w):
        return (c * h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w).sum()

    t = [torch.from_numpy(v.astype(np.float32)).cuda() for v in (c, h, w)]
    rstd = gp.rmsnorm_fp8(t[1], t[2], eps=eps)[3]
    dx, dw = gp.rmsnorm_backward(t[0], t[1], t[2], rstd)
    h, c, w = (ref.f64(v) for v in (t[1], t[0], t[2]))
    for r, k in [(0, 0), (1, cols // 2), (2, cols - 1)]:
        d = np.zeros_like(h)
        d[r, k] = step
        diff = (loss(h + d, w) - loss(h - d, w)) / (2 * step)
        assert abs(float(dx[r, k]) - diff) <= 1e-5 * (1 + abs(diff))   # differences: step^2 and 1e-16 * |L| / step
        d = np.zeros_like(w)
        d[k] = step
        diff = (loss(h, w + d) - loss(h, w - d)) / (2 * step)
        assert abs(float(dw[k]) - diff) <= 1e-5 * (1 + abs(diff))


@pytest.mark.parametrize("over", ["dy", "h", "dres"])
@pytest.mark.parametrize("cols", [600, 17000])
def test_norm_gradient_in_place(over, cols):
    rng = np.random.default_rng(3)
    dy, h, dres = (matrix(40, cols, "bf16", rng) for _ in range(3))
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    want, want_w = gp.rmsnorm_backward(dy, h, w, rstd, dres)
    place = {"dy": dy, "h": h, "dres": dres}[over]
    dw, work = torch.empty(cols, device="cuda"), torch.empty(4 << 20, device="cuda")
    assert gp.lib().fp8_rmsnorm_backward(dy.data_ptr(), cols, h.data_ptr(), cols, dres.data_ptr(), cols, w.data_ptr(), 1,
                                         rstd.data_ptr(), 40, cols, 1, place.data_ptr(), cols, dw.data_ptr(), work.data_ptr(),
                                         work.numel() * 4, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(place, want) and torch.equal(dw, want_w)


def test_norm_gradient_replays_in_graphs():
    # Two graphs captured on one stream, a larger call between, then both replayed side by side on two streams: each
    # has sums of its own, so their results are those of the calls.
    rng = np.random.default_rng(8)
    sets = [[matrix(rows, 1000, "bf16", rng) for _ in range(2)] for rows in (1700, 1900)]
    w = torch.ones(1000, device="cuda")
    side, graphs, outs, wants = torch.cuda.Stream(), [], [], []
    for dy, h in sets:
        rstd = torch.rsqrt(h.float().square().mean(1))
        wants.append(gp.rmsnorm_backward(dy, h, w, rstd))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(gp.rmsnorm_backward(dy, h, w, rstd))
        graphs.append((g, rstd))
    big = torch.ones((3000, 8000), device="cuda")
    gp.rmsnorm_backward(big, big, big[0], big[:, 0].contiguous(), stream=side)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_norm_gradient_with_too_small_a_workspace():
    x = torch.ones((4000, 600), device="cuda")
    dw, dx = torch.full((600,), 7.0, device="cuda"), torch.full((4000, 600), 7.0, device="cuda")
    p = x.data_ptr()
    assert gp.lib().fp8_rmsnorm_backward(p, 600, p, 600, None, 0, p, 2, p, 4000, 600, 2, dx.data_ptr(), 600, dw.data_ptr(),
                                         p, 600 * 4, None) == gp.GP_ERR_ARG
    torch.cuda.synchronize()
    assert bool((dx == 7).all()) and bool((dw == 7).all())


def test_norm_gradient_of_no_rows_and_same_bits():
    w = torch.ones(300, device="cuda")
    none = torch.empty((0, 300), device="cuda")
    dx, dw = gp.rmsnorm_backward(none, none, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 300) and bool((dw == 0).all())
    dy, h = torch.randn(2000, 300, device="cuda"), torch.randn(2000, 300, device="cuda")
    rstd = torch.rand(2000, device="cuda")
    first = gp.rmsnorm_backward(dy, h, w, rstd)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [gp.rmsnorm_backward(dy, h, w, rstd, stream=side if i % 2 else None) for i in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(o[0], first[0]) and torch.equal(o[1], first[1]) for o in outs)


def test_refusals():
    x = torch.randn(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (lambda: gp.quantize_fp8(x.double()), lambda: gp.quantize_fp8(x, "columns"),
                lambda: gp.quantize_fp8(x, format="e3m4"), lambda: gp.quantize_fp8(x.cpu()),
                lambda: gp.quantize_fp8(x.t()), lambda: gp.quantize_fp8(x[0]), lambda: gp.quantize_fp8(x, transpose="no"),
                lambda: gp.rmsnorm_fp8(x, w[:63]), lambda: gp.rmsnorm_fp8(x, w.cpu()),
                lambda: gp.rmsnorm_fp8(x, w, x[:3]), lambda: gp.rmsnorm_fp8(x, w, x.half()),
                lambda: gp.rmsnorm_backward(x, x.half(), w, w[:4]), lambda: gp.rmsnorm_backward(x, x, w, w),
                lambda: gp.rmsnorm_backward(x, x, w, w[:4], x[:, :32])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gp.GemmError):
        gp.rmsnorm_fp8(x, w, eps=-1.0)


@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
def test_rows_without_columns(type, residual):
    # the mean of nothing is NaN, and so is rstd; the buffer it is written to held other values before
    rows = 700
    x = torch.empty((rows, 0), dtype=ref.REAL[type], device="cuda")
    w = torch.empty(0, device="cuda")
    for _ in range(3):
        before = torch.full((rows,), 5.0, device="cuda")
        del before                                      # (the allocator hands the same memory out again)
        q, s, h, rstd, y = gp.rmsnorm_fp8(x, w, x.clone() if residual else None, normed=True)
        assert q.shape == h.shape == y.shape == (rows, 0) and s.shape == (rows, 0) and rstd.shape == (rows,)
        assert bool(torch.isnan(rstd).all())
    dx, dw = gp.rmsnorm_backward(x, x, w, rstd)
    assert dx.shape == (rows, 0) and dw.shape == (0,)
    guard = torch.full((rows + 2,), 7.0, device="cuda")
    assert gp.lib().fp8_rmsnorm(None, 0, None, 0, None, 0, 1e-6, rows, 0, 1, None, 0, guard[1:].data_ptr(), None, 0, None,
                                None) == 0
    torch.cuda.synchronize()
    assert float(guard[0]) == float(guard[-1]) == 7.0 and bool(torch.isnan(guard[1:-1]).all())
    for kind in ("rows", "blocks"):
        q, s, qt, st = gp.quantize_fp8(x, kind, transpose=True)
        groups = rows if kind == "rows" else -(-rows // 128)
        assert q.shape == (rows, 0) and s.shape == (groups, 0) and qt.shape == (0, rows) and st.shape == (0, -(-rows // 128))


@pytest.mark.parametrize("cols", [200, 1000, 5000, 17000])
@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("wtype", ["f16", "bf16", "f32"])
def test_weights_of_every_type_on_and_off_alignment(cols, type, wtype):
    rng = np.random.default_rng(cols)
    rows = 6
    x, dy = matrix(rows, cols, type, rng), matrix(rows, cols, type, rng)
    wide = torch.from_numpy(1 + 0.2 * rng.standard_normal(cols + 1)).cuda().to(ref.REAL[wtype])
    for w in (wide[:-1], wide[1:]):                     # the second begins one element past a 16-byte boundary
        q, s, h, rstd, y = gp.rmsnorm_fp8(x, w, eps=1e-5, normed=True)
        check_norm(q, s, rstd, y, h, w, 1e-5, type, "e4m3")
        same = w.to(torch.float32)                      # the same values in 32 bits: the same bits come out
        again = gp.rmsnorm_fp8(x, same, eps=1e-5, normed=True)
        assert torch.equal(q.view(torch.uint8), again[0].view(torch.uint8))
        assert torch.equal(s, again[1]) and torch.equal(rstd, again[3]) and torch.equal(y, again[4])
        dx, dw = gp.rmsnorm_backward(dy, x, w, rstd)
        dx2, dw2 = gp.rmsnorm_backward(dy, x, same, rstd)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("rows,cols,pad", [(5, 200, 0), (77, 1000, 0), (133, 65, 0), (200, 2056, 0), (90, 1004, 4), (512, 130, 1)])
def test_weight_gradient_of_few_rows_with_values_that_are_not_finite(rows, cols, pad):
    # each stays in its own column, where the rows' number is no multiple of what a block takes at a time too
    rng = np.random.default_rng(rows + cols)
    for type in ("bf16", "f32"):
        dy, h = matrix(rows, cols, type, rng, ld=cols + pad), matrix(rows, cols, type, rng, ld=cols + pad)
        w = torch.ones(cols, device="cuda")
        rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
        want = gp.rmsnorm_backward(dy, h, w, rstd)[1]
        assert bool(torch.isfinite(want).all())
        dy[rows - 1, 3] = float("inf")
        h[0, cols - 1] = float("nan")
        h[rows // 2, cols // 2] = -float("inf")
        dw = gp.rmsnorm_backward(dy, h, w, rstd)[1]
        bad = {3: torch.isinf(dw[3]), cols - 1: torch.isnan(dw[cols - 1]), cols // 2: torch.isinf(dw[cols // 2])}
        assert all(bool(v) for v in bad.values())
        keep = [c for c in range(cols) if c not in bad]
        assert torch.equal(dw[keep], want[keep])
