"""The feed-forward operators against their formulas in float64, element by
element within bounds derived from the arithmetic (ffn_ref): sizes around the
tiles, both types, every activation, what is kept, strides, addends, values that
are not finite, every tile, refusals, streams and graphs."""
import numpy as np
import pytest
import torch

import ffn_ref as ref
import fp8_ref
import software_pipelined_tiled_pipeline_gb300 as gp

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def status_ok():
    st = gp.gemm_stats(sync=True)
    assert st["status"] == 0, (gp.strerror(st["status"]), st["device_status"], st["cuda_error"], st["cuda_error_site"])
    return st["plan"]


def check_linear(M, N, K, dtype=BF16, act=None, bias=None, residual=False, keep=None, out_dtype=None, seed=0, pads=(0, 0, 0),
                 whole=None, ld=None, **kw):
    rng = np.random.default_rng(seed + 7 * M + 3 * N + K)
    x, w = ref.matrix(rng, M, K, dtype, pad=pads[0], whole=whole), ref.matrix(rng, N, K, dtype, 1.2 * max(K, 1) ** -0.5,
                                                                             pad=pads[1], whole=whole)
    out_dtype = out_dtype or dtype
    b = ref.matrix(rng, 1, N, bias, whole=whole)[0] if bias else None
    r = ref.matrix(rng, M, N, out_dtype, 2.0, pad=pads[2], whole=whole) if residual else None
    out, buf = ref.guarded(M, N, out_dtype, ld)
    got = gp.linear(x, w, b, activation=act, residual=r, keep=keep, out=out, **kw)
    kept = None
    if keep:
        got, kept = got
    assert got is out
    plan = status_ok()
    a, c = ref.f64(x), ref.f64(w)
    z = a @ c.T + (ref.f64(b) if b is not None else 0)
    wide = out_dtype is F32 or keep == "fp8"
    err = ref.sum_error(ref.magnitudes(a, c), K, wide) + 2.0 ** -24 * (np.abs(z) + np.abs(a @ c.T))
    y = ref.value(z, act)
    yerr = 1.2 * err + ref.steps(z) * 2.0 ** -24 * np.abs(y) if act else err      # (no activation's slope is above 1.13)
    if r is not None:
        y = y + ref.f64(r)
        yerr = yerr + (K // ref.RESTART + 2) * 2.0 ** -24 * (np.abs(y) + np.abs(ref.f64(r)))
    worst = ref.worst(ref.f64(out), y, ref.rounded(y, yerr, out_dtype), out_dtype)
    assert worst <= 1.0, "%g of the bound (plan %s)" % (worst, plan)
    assert ref.outside_untouched(buf, M, N, ld or N), "write outside of the output"
    if keep == "real":
        assert ref.kept_real(z, err, kept[0]) <= 1.0, plan
    elif keep == "fp8":
        assert ref.kept_codes(z, err, *kept) <= 1.0, plan
    if whole:       # every sum is exact in FP32 in any order: so is what the epilogue starts from
        if act is None:
            assert torch.equal(out.cpu(), torch.from_numpy(y).to(out_dtype))
        if keep == "fp8":
            code, s = fp8_ref.quantize(z, "rows", "e4m3")
            assert np.array_equal(ref.f64(kept[1]).astype(np.float32), s)
            assert fp8_ref.same_codes(fp8_ref.codes(kept[0]), code, "e4m3")
    return plan


def check_gated(M, N, K, dtype=BF16, act="silu", keep=None, seed=0, pads=(0, 0, 0), ld=None, whole=None, **kw):
    rng = np.random.default_rng(seed + 5 * M + 3 * N + K)
    x = ref.matrix(rng, M, K, dtype, pad=pads[0], whole=whole)
    wg, wu = (ref.matrix(rng, N, K, dtype, 1.2 * max(K, 1) ** -0.5, pad=p, whole=whole) for p in pads[1:])
    out, buf = ref.guarded(M, N, dtype, ld)
    got = gp.gated(x, wg, wu, activation=act, keep=keep, out=out, **kw)
    kept = None
    if keep:
        got, kept = got
    assert got is out
    plan = status_ok()
    a, b, c = ref.f64(x), ref.f64(wg), ref.f64(wu)
    g, u = a @ b.T, a @ c.T
    eg, eu = (ref.sum_error(ref.magnitudes(a, w), K, keep == "fp8") for w in (b, c))
    v = ref.value(g, act)
    ev = 1.2 * eg + ref.steps(g) * 2.0 ** -24 * np.abs(v)
    h = v * u
    err = ev * (np.abs(u) + eu) + np.abs(v) * eu + 2.0 ** -24 * np.abs(h)
    worst = ref.worst(ref.f64(out), h, ref.rounded(h, err, dtype), dtype)
    assert worst <= 1.0, "%g of the bound (plan %s)" % (worst, plan)
    assert ref.outside_untouched(buf, M, N, ld or N), "write outside of the output"
    if keep == "real":
        assert ref.kept_real(g, eg, kept[0]) <= 1.0 and ref.kept_real(u, eu, kept[1]) <= 1.0, plan
    elif keep == "fp8":
        assert ref.kept_codes(g, eg, *kept[:2]) <= 1.0 and ref.kept_codes(u, eu, *kept[2:]) <= 1.0, plan
        if whole:
            for z, (data, s) in ((g, kept[:2]), (u, kept[2:])):
                code, want = fp8_ref.quantize(z, "rows", "e4m3")
                assert np.array_equal(ref.f64(s).astype(np.float32), want)
                assert fp8_ref.same_codes(fp8_ref.codes(data), code, "e4m3")
    return plan


SHAPES = [(1, 1, 1), (1, 16, 16), (1, 300, 4096), (2, 129, 128), (16, 128, 130), (17, 127, 257), (31, 1000, 520), (33, 257, 129),
          (64, 640, 1024), (65, 200, 384), (128, 128, 128), (129, 130, 1000), (300, 70, 257), (70, 300, 2057), (511, 385, 640),
          (260, 1030, 300), (1000, 776, 2056), (5, 4096, 8192), (500, 600, 4100), (2100, 2300, 256), (3, 700, 513),
          (1, 41, 20001), (200, 8, 64)]


# ---------------------------------------------------------------------------
# forward
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_linear_shapes(M, N, K, dtype):
    check_linear(M, N, K, dtype, act="gelu" if M % 2 else None, bias=dtype, residual=N % 2 == 0)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_whole_numbers_are_exact(M, N, K):
    check_linear(M, N, K, F16, whole=2 if K < 3000 else 1, bias=F16, residual=True, out_dtype=F32)
    check_linear(M, N, K, BF16, whole=2 if K < 3000 else 1, bias=F32, keep="fp8", out_dtype=F32)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M", [3, 200, 700])
@pytest.mark.parametrize("dtype,out", [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)])
def test_linear_activations_and_types(act, M, dtype, out):
    check_linear(M, 264, 200, dtype, act, bias=F32, residual=True, out_dtype=out)
    check_linear(M, 260, 200, dtype, act, out_dtype=out, keep="real")


@pytest.mark.parametrize("tile", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("M,N,K", [(1, 200, 700), (100, 1000, 333), (513, 700, 1300)])
def test_linear_every_tile(tile, M, N, K):
    for splits in (0, 1, 2, 4, 8) if 16 < tile < 128 else (0, 1, 4) if tile == 16 else (0,):
        check_linear(M, N, K, BF16, "silu", bias=BF16, residual=True, tile=tile, k_splits=splits)
        check_linear(M, N, K, F16, None, keep="real", out_dtype=F32, tile=tile, k_splits=splits)
    if tile >= 128:
        check_linear(M, N, K, BF16, "gelu", bias=BF16, keep="fp8", tile=tile)


@pytest.mark.parametrize("M,N", [(2560, 2304), (2300, 2500), (5000, 1100)])
def test_tiles_cut_in_halves(M, N):
    """More tiles of two CTAs than pairs, and few enough in the last round: those are cut in halves of their columns."""
    for K in (64, 200):
        plan = check_linear(M, N, K, BF16, "relu", bias=BF16, residual=True, whole=2, tile=256)
        assert plan["half_tiles"] > 0 and plan["dp_tiles"] + plan["half_tiles"] == plan["tiles"]
        check_linear(M, N, K, F16, whole=2, out_dtype=F32, residual=True, tile=256)
        check_linear(M, N, K, F16, whole=2, keep="fp8", tile=256)
        assert check_gated(M, N // 2, K, BF16, keep="real", tile=256)["half_tiles"] > 0
        assert check_gated(M, N // 2, K, BF16, keep="fp8", tile=256)["half_tiles"] == 0
    rng = np.random.default_rng(1)
    for K in (64, 200):
        dy, x, w = (ref.matrix(rng, r, c, BF16, whole=1) for r, c in ((K, M), (K, N), (M, N)))
        _, dw, _ = gp.linear_backward(dy, x, w, input_grad=False, out_dtype=F32, tile=256)       # M x N of K tokens
        assert gp.gemm_stats()["plan"]["half_tiles"] > 0
        assert torch.equal(dw.cpu().double(), dy.cpu().double().t() @ x.cpu().double())
        dy, w = ref.matrix(rng, M, K, BF16, whole=1), ref.matrix(rng, K, N, BF16, whole=1)
        dx, _, _ = gp.linear_backward(dy, ref.matrix(rng, M, N, BF16), w, weight_grad=False, tile=256)
        assert gp.gemm_stats()["plan"]["half_tiles"] > 0
        assert torch.equal(dx.cpu(), (dy.cpu().double() @ w.cpu().double()).to(BF16))


@pytest.mark.parametrize("M", [1, 40, 130, 600])
@pytest.mark.parametrize("pads,ld", [((0, 8, 0), None), ((1, 3, 5), 301), ((8, 8, 4), 308), ((7, 0, 1), 304)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_linear_strides(M, pads, ld, out):
    check_linear(M, 300, 264, BF16, "relu", bias=BF16, residual=True, pads=pads, ld=ld, out_dtype=out)
    check_linear(M, 300, 263, BF16, "relu", bias=BF16, residual=True, pads=pads, ld=ld, out_dtype=out)


@pytest.mark.parametrize("M,N", [(3, 200), (300, 301), (300, 304)])
@pytest.mark.parametrize("out", [F16, F32])
def test_linear_residual_in_place(M, N, out):
    rng = np.random.default_rng(4)
    x, w = ref.matrix(rng, M, 260, F16), ref.matrix(rng, N, 260, F16)
    r = ref.matrix(rng, M, N, out, pad=8)
    apart = gp.linear(x, w, residual=r, out_dtype=out)
    here = r.clone(memory_format=torch.preserve_format)
    wide = torch.zeros((M, N + 8), dtype=out, device="cuda")
    wide[:, :N] = r
    here = wide[:, :N]
    assert gp.linear(x, w, residual=here, out=here) is here
    assert torch.equal(here, apart) and bool((wide[:, N:] == 0).all())


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gated_shapes(M, N, K, dtype):
    check_gated(M, N, K, dtype, keep=[None, "real", "fp8"][(M + N) % 3])


@pytest.mark.parametrize("M,N,K", SHAPES[:20])
def test_gated_whole_numbers_kept_in_8_bits(M, N, K):
    check_gated(M, N, K, BF16, keep="fp8", whole=2 if K < 3000 else 1)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M", [3, 200, 700])
@pytest.mark.parametrize("keep", [None, "real", "fp8"])
def test_gated_activations(act, M, keep):
    check_gated(M, 264, 200, F16, act, keep)
    check_gated(M, 333, 200, BF16, act, keep)


@pytest.mark.parametrize("tile", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("M,N,K", [(1, 200, 700), (100, 1000, 333), (513, 700, 1300)])
def test_gated_every_tile(tile, M, N, K):
    check_gated(M, N, K, BF16, tile=tile)
    for splits in (1, 2, 4) if tile < 128 else ():
        check_gated(M, N, K, F16, keep="real", tile=tile, k_splits=splits)


@pytest.mark.parametrize("M", [1, 40, 130, 600])
@pytest.mark.parametrize("pads,ld", [((0, 8, 0), None), ((1, 3, 5), 301), ((8, 8, 8), 304)])
def test_gated_strides(M, pads, ld):
    check_gated(M, 300, 264, BF16, keep="real", pads=pads, ld=ld)
    check_gated(M, 300, 263, F16, keep="fp8", pads=pads, ld=ld)


def test_few_tokens_alone_and_together():
    """A token's outputs do not depend on what else is in the batch (the same tile, so the same order of sums)."""
    rng = np.random.default_rng(2)
    x, w, u = ref.matrix(rng, 16, 1030, BF16), ref.matrix(rng, 500, 1030, BF16, 0.03), ref.matrix(rng, 500, 1030, BF16, 0.03)
    whole = gp.linear(x, w, activation="gelu")
    both = gp.gated(x, w, u)
    for i in (0, 7, 15):
        assert torch.equal(gp.linear(x[i:i + 1], w, activation="gelu"), whole[i:i + 1])
        assert torch.equal(gp.gated(x[i:i + 1], w, u), both[i:i + 1])


@pytest.mark.parametrize("M", [2, 300, 600])
def test_values_that_are_not_finite(M):
    """A NaN or an infinity reaches the outputs of its own row or column alone, and the scale of its own groups."""
    rng = np.random.default_rng(3)
    N, K = 300, 200
    x, w, u = ref.matrix(rng, M, K, BF16), ref.matrix(rng, N, K, BF16, 0.1), ref.matrix(rng, N, K, BF16, 0.1)
    x[1, 5] = float("nan")
    x[0, 7] = float("inf")
    w[4, 9] = float("nan")
    y = gp.linear(x, w)
    want = x.double().cpu() @ w.double().cpu().t()
    assert torch.equal(torch.isnan(y).cpu(), torch.isnan(want)) and torch.equal(torch.isinf(y).cpu(), torch.isinf(want))
    h = gp.gated(x, w, u, activation="sigmoid")
    assert bool(torch.isnan(h[1]).all()) and bool(torch.isnan(h[:, 4]).all())
    assert M < 3 or bool(torch.isfinite(h[2:, torch.arange(N) != 4]).all())
    y, (data, s) = gp.linear(x, w, keep="fp8")
    z = want.float()
    assert torch.equal(torch.isnan(s).cpu(), torch.stack([torch.isnan(z[:, j:j + 128]).any(1) for j in (0, 128, 256)], 1))
    inf = torch.stack([torch.isinf(z[:, j:j + 128]).any(1) & ~torch.isnan(z[:, j:j + 128]).any(1) for j in (0, 128, 256)], 1)
    assert torch.equal(torch.isinf(s).cpu(), inf)


@pytest.mark.parametrize("M,N,K", [(4, 8, 0), (300, 129, 0), (0, 64, 64), (64, 0, 64)])
def test_empty(M, N, K):
    x, w = torch.ones(M, K, dtype=BF16, device="cuda"), torch.ones(N, K, dtype=BF16, device="cuda")
    b, r = torch.full((N,), 0.5, dtype=BF16, device="cuda"), torch.full((M, N), 2.0, dtype=BF16, device="cuda")
    y, kept = gp.linear(x, w, b, activation="relu", residual=r, keep="real")
    assert y.shape == (M, N) and bool((y == 2.5).all()) and bool((kept[0] == 0.5).all())
    h = gp.gated(x, w, w)
    assert h.shape == (M, N) and bool((h == 0).all())
    dx, dw, db = gp.linear_backward(r, x, w, bias_grad=True)
    assert dx.shape == (M, K) and dw.shape == (N, K) and bool((db == 2.0 * M).all())
    assert bool((dx == (2.0 * N if K else 0)).all()) and bool((dw == 2.0 * M).all())
    add = torch.full((N, K), 3.0, dtype=F32, device="cuda")
    _, dw, _ = gp.linear_backward(r, x, w, addend=add, out_dtype=F32)
    assert bool((dw == 2.0 * M + 3).all())
    dx, dg, du, h = gp.gated_backward(r, x, w, w, (r, r), product=True)
    assert dx.shape == (M, K) and dg.shape == du.shape == (N, K) and h.shape == (M, N)


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------
def make_kept(rng, M, N, dtype, keep, pad=0, fmt="e4m3"):
    z = ref.matrix(rng, M, N, dtype, 1.5, pad=pad)
    if keep == "real":
        return (z,)
    return gp.quantize_fp8(z, format=fmt)


def check_products(dz, edz, x, w, dx, dw, addend=None):
    """dx = sum dz w and dw = dz^T x, from gradients dz that the kernel rounded to x's type, off by edz before that."""
    dtype = x.dtype
    a = ref.f64(x)
    want, err = 0.0, 0.0
    summed = 0
    for z, e, weight, got in zip(dz, edz, w, dw):
        e = ref.rounded(z, e, dtype)
        b = ref.f64(weight)
        want = want + z @ b
        err = err + e @ np.abs(b) + 0 * want
        summed += z.shape[1]
        if got is not None:
            g, ge = z.T @ a, e.T @ np.abs(a)
            ge = ge + ref.sum_error((np.abs(z) + e).T @ np.abs(a), len(a), got.dtype is F32)
            if addend is not None:
                i = [j for j, t in enumerate(dw) if t is got][0]
                ge = ge + (len(a) // ref.RESTART + 2) * 2.0 ** -24 * (np.abs(g) + np.abs(ref.f64(addend[i])))
                g = g + ref.f64(addend[i])
            far = ref.worst(ref.f64(got), g, ref.rounded(g, ge, got.dtype), got.dtype)
            assert far <= 1.0, "weight gradient: %g of the bound" % far
    if dx is not None:
        mag = sum((np.abs(z) + ref.rounded(z, e, dtype)) @ np.abs(ref.f64(weight)) for z, e, weight in zip(dz, edz, w))
        err = err + ref.sum_error(mag, summed, False)
        far = ref.worst(ref.f64(dx), want, ref.rounded(want, err, dtype), dtype)
        assert far <= 1.0, "input gradient: %g of the bound" % far


def check_linear_backward(M, N, K, dtype=BF16, act=None, keep="real", out_dtype=None, add=False, pads=(0, 0, 0, 0), seed=0, **kw):
    rng = np.random.default_rng(seed + M + 3 * N + 5 * K)
    dy, x = ref.matrix(rng, M, N, dtype, 0.1, pad=pads[0]), ref.matrix(rng, M, K, dtype, pad=pads[1])
    w = ref.matrix(rng, N, K, dtype, 0.05, pad=pads[2])
    kept = make_kept(rng, M, N, dtype, keep, pads[3]) if act else None
    addend = ref.matrix(rng, N, K, out_dtype or dtype) if add else None
    dx, dw, db = gp.linear_backward(dy, x, w, activation=act, kept=kept, bias_grad=True, out_dtype=out_dtype, addend=addend, **kw)
    status_ok()
    assert dx.dtype is dtype and db.dtype is F32 and (dw is None or dw.dtype is (out_dtype or dtype))
    d = ref.f64(dy)
    if act:
        z = ref.held(kept, dtype)
        s = ref.slope(z, act)
        es = ref.steps(z) * 2.0 ** -23 * (1 + np.abs(z)) * (z != 0 if act == "relu" else 1)
        dz, e = d * s, np.abs(d) * (es + 2.0 ** -24 * np.abs(s))
    else:
        dz, e = d, np.zeros_like(d)
    # without an activation dy itself is the operand: it is in its type already
    check_products([dz], [e], x, [w], dx, [dw], None if addend is None else [addend])
    want = dz.sum(0)
    bound = e.sum(0) + M * 2.0 ** -24 * (np.abs(dz) + e).sum(0) + 2.0 ** -150
    assert ref.worst(ref.f64(db), want, bound) <= 1.0


BACK = [(1, 1, 1), (1, 300, 130), (16, 128, 64), (17, 127, 257), (130, 129, 131), (200, 2056, 776), (333, 1000, 776),
        (260, 70, 1030), (1000, 264, 520), (2100, 300, 256), (5, 4096, 1000), (4100, 65, 72)]


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_linear_backward_shapes(M, N, K, dtype):
    check_linear_backward(M, N, K, dtype)
    check_linear_backward(M, N, K, dtype, out_dtype=F32, add=True)
    check_linear_backward(M, N, K, dtype, act="gelu", keep="fp8" if M % 2 else "real")


@pytest.mark.parametrize("act", ref.ACTS[1:])
@pytest.mark.parametrize("keep", ["real", "fp8"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_linear_backward_activations(act, keep, dtype):
    check_linear_backward(150, 264, 200, dtype, act, keep, add=True)
    check_linear_backward(150, 261, 200, dtype, act, keep)


@pytest.mark.parametrize("tile", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("M,N,K", [(100, 333, 700), (700, 513, 300), (300, 1300, 520), (20, 2000, 128), (1000, 64, 192)])
def test_backward_every_tile(tile, M, N, K):
    weight = tile >= 64            # (a weight's gradient has no narrower one)
    check_linear_backward(M, N, K, BF16, tile=tile, out_dtype=F32, add=weight, weight_grad=weight)
    check_linear_backward(M, N, K, F16, "silu", "fp8", tile=tile, weight_grad=weight)
    check_gated_backward(M, N, K, BF16, tile=tile, weight_grad=weight)


@pytest.mark.parametrize("pads", [(1, 3, 5, 7), (8, 8, 8, 8), (0, 1, 0, 0), (4, 0, 0, 1)])
@pytest.mark.parametrize("M,N,K", [(40, 300, 264), (300, 129, 333)])
def test_backward_strides(pads, M, N, K):
    check_linear_backward(M, N, K, F16, "gelu_tanh", pads=pads)
    check_linear_backward(M, N, K, F16, pads=pads)
    check_gated_backward(M, N, K, BF16, pads=pads)


@pytest.mark.parametrize("M,N,K", [(8, 200, 64), (300, 264, 520), (700, 300, 1024)])
def test_backward_whole_numbers_are_exact(M, N, K):
    rng = np.random.default_rng(6)
    dy, x, w = (ref.matrix(rng, r, c, BF16, whole=2) for r, c in ((M, N), (M, K), (N, K)))
    a, b, c = (t.cpu().double() for t in (dy, x, w))
    for tile in (0, 64, 128, 256):
        dx, dw, db = gp.linear_backward(dy, x, w, bias_grad=True, out_dtype=F32, tile=tile)
        assert torch.equal(dw.cpu().double(), a.t() @ b) and torch.equal(db.cpu().double(), a.sum(0))
        assert torch.equal(dx.cpu(), (a @ c).to(BF16))
        # both weights' gradients in one launch, with addends in place
        relu = torch.ones(M, N, dtype=BF16, device="cuda")
        acc = [torch.full((N, K), float(i + 1), dtype=F32, device="cuda") for i in range(2)]
        dx, dg, du = gp.gated_backward(dy, x, w, w, (relu, relu + 1), activation="relu", addend=acc, out=acc, tile=tile)
        assert dg is acc[0] and du is acc[1]
        assert torch.equal(dg.cpu().double(), 2 * (a.t() @ b) + 1) and torch.equal(du.cpu().double(), a.t() @ b + 2)
        assert torch.equal(dx.cpu(), (3 * (a @ c)).to(BF16))


def check_gated_backward(M, N, K, dtype=BF16, act="silu", keep="real", product=True, pads=(0, 0, 0, 0), seed=0, fmt="e4m3", **kw):
    rng = np.random.default_rng(seed + M + 3 * N + 5 * K)
    dh, x = ref.matrix(rng, M, N, dtype, 0.1, pad=pads[0]), ref.matrix(rng, M, K, dtype, pad=pads[1])
    wg, wu = ref.matrix(rng, N, K, dtype, 0.05, pad=pads[2]), ref.matrix(rng, N, K, dtype, 0.05)
    kg, ku = (make_kept(rng, M, N, dtype, keep, pads[3], fmt) for _ in range(2))
    got = gp.gated_backward(dh, x, wg, wu, kg + ku, activation=act, product=product, **kw)
    status_ok()
    d, g, u = ref.f64(dh), ref.held(kg, dtype), ref.held(ku, dtype)
    s, v = ref.slope(g, act), ref.value(g, act)
    es = ref.steps(g) * 2.0 ** -23 * (1 + np.abs(g)) * (g != 0 if act == "relu" else 1)
    ev = ref.steps(g) * 2.0 ** -24 * np.abs(v)
    dg, du = d * u * s, d * v
    eg = np.abs(d * u) * (es + 2.0 ** -22 * np.abs(s))
    eu = np.abs(d) * (ev + 2.0 ** -23 * np.abs(v))
    check_products([dg, du], [eg, eu], x, [wg, wu], got[0], list(got[1:3]))
    if product:
        h = v * u
        err = np.abs(u) * ev + 2.0 ** -22 * np.abs(h)
        assert ref.worst(ref.f64(got[3]), h, ref.rounded(h, err, dtype), dtype) <= 1.0


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gated_backward_shapes(M, N, K, dtype):
    check_gated_backward(M, N, K, dtype, keep="fp8" if M % 2 else "real", product=bool(N % 2))


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("keep,fmt", [("real", ""), ("fp8", "e4m3"), ("fp8", "e5m2")])
def test_gated_backward_activations(act, keep, fmt):
    check_gated_backward(150, 264, 200, F16, act, keep, fmt=fmt)
    check_gated_backward(150, 261, 200, BF16, act, keep, fmt=fmt)


# ---------------------------------------------------------------------------
# calls together: streams, graphs, threads, refusals, waits that run out
# ---------------------------------------------------------------------------
def block_pass(x, w, wd, b, r):
    """A gated block forward and backward, as a program calls it."""
    h, kept = gp.gated(x, w[0], w[1], keep="fp8")
    y, z = gp.linear(h, wd, b, activation="gelu", residual=r, keep="real")
    dh, dwd, db = gp.linear_backward(y, h, wd, activation="gelu", kept=z, bias_grad=True)
    dx, dg, du, again = gp.gated_backward(dh, x, w[0], w[1], kept, product=True)
    return h, y, dh, dwd, db, dx, dg, du, again, kept[0].view(torch.uint8), kept[1]


def block_operands(M, N, K, seed):
    rng = np.random.default_rng(seed)
    x, r = ref.matrix(rng, M, K, BF16), ref.matrix(rng, M, K, BF16)
    w = [ref.matrix(rng, N, K, BF16, 0.05) for _ in range(2)]
    return x, w, ref.matrix(rng, K, N, BF16, 0.05), ref.matrix(rng, 1, K, BF16)[0], r


SIZES = [(1, 200, 136), (48, 520, 264), (300, 640, 333), (2000, 1100, 520)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_repeated_calls_give_the_same_bits(M, N, K):
    ops = block_operands(M, N, K, 3)
    first = [t.clone() for t in block_pass(*ops)]
    for _ in range(3):
        for a, b in zip(first, block_pass(*ops)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_chained_calls_in_a_graph(M, N, K):
    """A captured pass replayed on new inputs, and two graphs that share what can be shared, give what the calls give."""
    ops, other = block_operands(M, N, K, 1), block_operands(M, N, K, 2)
    want, want_other = [[t.clone() for t in block_pass(*o)] for o in (ops, other)]
    stream = torch.cuda.Stream()
    graphs, outs = [], []
    for o in (ops, other):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            block_pass(*o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append(block_pass(*o))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    block_pass(*ops)                      # an eager call between replays
    graphs[0].replay()
    torch.cuda.synchronize()
    for got, w in ((outs[0], want), (outs[1], want_other)):
        for a, b in zip(got, w):
            assert torch.equal(a, b)
    ops[0].copy_(other[0])                # new inputs in the same memory
    graphs[0].replay()
    torch.cuda.synchronize()
    for a, b in zip(outs[0], block_pass(*ops)):
        assert torch.equal(a, b)


def test_streams():
    """Calls on a stream of their own, given as an argument or made current, after work on another one."""
    x, w, wd, b, r = block_operands(300, 640, 264, 5)
    want = gp.gated(x, *w)
    side = torch.cuda.Stream()
    late = torch.empty_like(x)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
        got = gp.gated(late, *w)          # after the copy on the same stream
    side.synchronize()
    assert torch.equal(got, want)
    late.zero_()
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
    got = gp.gated(late, *w, stream=side)
    y = gp.linear(got, wd, b, stream=side)
    d = gp.linear_backward(y, got, wd, bias_grad=True, stream=side)
    e = gp.gated_backward(got, late, *w, (want, want), stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(y, gp.linear(want, wd, b))
    for a, c in zip(d, gp.linear_backward(y, got, wd, bias_grad=True)):
        assert torch.equal(a, c)
    for a, c in zip(e, gp.gated_backward(want, x, *w, (want, want))):
        assert torch.equal(a, c)


def test_two_threads():
    """Two host threads on streams of their own."""
    import threading
    sizes = [(40, 520, 264), (700, 640, 520)]
    ops = [block_operands(*s, 7 + i) for i, s in enumerate(sizes)]
    want = [[t.clone() for t in block_pass(*o)] for o in ops]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = block_pass(*ops[i])
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("tile,splits", [(16, 1), (32, 4), (64, 2), (129, 2), (128, 0)])
def test_a_lost_load_is_reported(tile, splits):
    """A load that never comes: the waits give up, the status says so, and the next call is right."""
    x, w, _, _, _ = block_operands(100, 384, 1500, 4)
    want = gp.linear(x, w[0], tile=tile, k_splits=splits)
    got = torch.full_like(want, 7.0)
    gp.linear(x, w[0], out=got, tile=tile, k_splits=splits, timeout_ns=5_000_000, inject_lost_load=True)
    assert gp.gemm_stats(sync=True)["status"] == gp.GP_ERR_TIMEOUT
    # tiles that came to their end are right, the others are as they were
    assert bool(((got == want) | (got == 7.0)).all()) and bool((got == 7.0).any())
    if tile != 129:
        h = torch.full((100, 384), 7.0, dtype=BF16, device="cuda")
        gp.gated(x, *w, out=h, tile=tile, k_splits=splits, timeout_ns=5_000_000, inject_lost_load=True)
        assert gp.gemm_stats(sync=True)["status"] == gp.GP_ERR_TIMEOUT
    assert torch.equal(gp.linear(x, w[0], tile=tile, k_splits=splits), want)
    status_ok()


def test_lost_load_not_where_two_ctas_share_a_tile():
    x, w, _, _, _ = block_operands(600, 384, 200, 4)
    with pytest.raises(gp.GemmError):
        gp.linear(x, w[0], tile=256, inject_lost_load=True)
    with pytest.raises(gp.GemmError):
        gp.gated(x, *w, keep="fp8", inject_lost_load=True)


def test_input_gradient_without_x():
    x, w, wd, b, r = block_operands(70, 200, 136, 6)
    z = torch.ones(70, 200, dtype=BF16, device="cuda")
    dx, none, _ = gp.linear_backward(z, None, w[0], weight_grad=False)
    assert none is None and torch.equal(dx, gp.linear_backward(z, x, w[0])[0])
    got = gp.gated_backward(z, None, *w, (z, z), weight_grad=False)
    assert got[1] is None and got[2] is None and torch.equal(got[0], gp.gated_backward(z, x, *w, (z, z))[0])
    none, dw, _ = gp.linear_backward(z, x, w[0], input_grad=False)
    assert none is None and torch.equal(dw, gp.linear_backward(z, x, w[0])[1])
    assert gp.linear_backward(z, None, w[0], input_grad=False, weight_grad=False) == (None, None, None)


def test_where_weight_gradients_go():
    """out and addend in every combination, in 16 bits and FP32, rows apart or not."""
    rng = np.random.default_rng(12)
    M, N, K = 90, 130, 70
    dy, x, w = (ref.matrix(rng, r, c, BF16, whole=2) for r, c in ((M, N), (M, K), (N, K)))
    z = torch.ones(M, N, dtype=BF16, device="cuda")
    plain = (dy.double().t() @ x.double())
    for dtype in (BF16, F32):
        for pad in (0, 1, 10):
            wide = [torch.full((N, K + pad), 5.0, dtype=dtype, device="cuda") for _ in range(4)]
            a, b, c, d = (t[:, :K] for t in wide)
            got = gp.linear_backward(dy, x, w, input_grad=False, out=a)[1]
            assert got is a and torch.equal(a, plain.to(dtype))
            got = gp.linear_backward(dy, x, w, input_grad=False, out=a, addend=b)[1]
            assert got is a and torch.equal(a, (plain + 5).to(dtype))
            got = gp.linear_backward(dy, x, w, input_grad=False, addend=b)[1]
            assert got.dtype is dtype and torch.equal(got, (plain + 5).to(dtype)) and bool((b == 5).all())
            _, g, u = gp.gated_backward(dy, x, w, w, (z, z), activation="relu", input_grad=False, out=(c, d), addend=(b, b))
            assert g is c and u is d and torch.equal(g, (plain + 5).to(dtype)) and torch.equal(u, g)
            assert all(bool((t[:, K:] == 5).all()) for t in wide)
    with pytest.raises(ValueError):
        gp.gated_backward(dy, x, w, w, (z, z), input_grad=False, out=(c, c))


def test_outputs_apart_from_what_is_read():
    """An output that overlaps an operand is refused; one beside it in the same rows, or the addend itself, is not."""
    rng = np.random.default_rng(13)
    M, N, K = 70, 64, 64
    x, w, u, dy, b = (ref.matrix(rng, r, c, BF16, whole=2) for r, c in ((M, K), (N, K), (N, K), (M, N), (1, N)))
    z = torch.ones(M, N, dtype=BF16, device="cuda")
    square = ref.matrix(rng, K, K, BF16, whole=2)
    tall = torch.zeros(M + N + 1, N, dtype=BF16, device="cuda")
    for call in (lambda: gp.linear(x, w, out=x), lambda: gp.linear(square, w, out=w), lambda: gp.gated(x, w, u, out=x),
                 lambda: gp.gated(square, w, u, out=u), lambda: gp.gated(square, w, u, out=w),
                 lambda: gp.linear(x, w, out=tall[1:M + 1], residual=tall[:M]),
                 lambda: gp.linear(x, w, tall[5], out=tall[:M]),
                 lambda: gp.linear(x, w, out=tall.flatten()[3:3 + M * N].view(M, N), residual=tall[:M]),
                 lambda: gp.linear_backward(dy, x, w, out=x[:N]), lambda: gp.linear_backward(dy, x, w, out=dy[1:N + 1]),
                 lambda: gp.linear_backward(dy, x, w, out=tall[:N], addend=tall[1:N + 1]),
                 lambda: gp.gated_backward(dy, x, w, u, (z, z), out=(tall[:N], x[:N])),
                 lambda: gp.gated_backward(dy, x, w, u, (z, z), out=(tall[:N], tall[1:N + 1])),
                 lambda: gp.gated_backward(dy, x, w, u, (z, z), out=(tall[:N], w), addend=(w, tall[:N]))):
        with pytest.raises(ValueError, match="overlaps"):
            call()
    wide = torch.zeros(M, K + N + 8, dtype=BF16, device="cuda")
    wide[:, :K].copy_(x)
    want = (x.double() @ w.double().t()).to(BF16)
    assert torch.equal(gp.linear(wide[:, :K], w, out=wide[:, K:K + N]), want) and torch.equal(wide[:, :K], x)
    dw = torch.zeros(N, 2 * K, dtype=F32, device="cuda")
    halves = (dw[:, :K], dw[:, K:])
    gp.gated_backward(dy, x, w, u, (z, z), activation="relu", input_grad=False, out=halves, addend=halves)
    plain = (dy.double().t() @ x.double()).float()
    assert torch.equal(dw, torch.cat((plain, plain), 1))
    # the weight itself as dW and addend: it is read for dx before
    want = ((dy.double() @ w.double()).to(BF16), (w.double() + plain.double()).to(BF16))
    got = gp.linear_backward(dy, x, w, out=w, addend=w)
    assert got[1] is w and torch.equal(got[0], want[0]) and torch.equal(w, want[1])
    status_ok()


def test_kept_codes_of_any_strides():
    x, w, _, _, _ = block_operands(70, 300, 136, 9)
    _, kept = gp.gated(x, *w, keep="fp8")
    dh = torch.ones(70, 300, dtype=BF16, device="cuda")
    want = gp.gated_backward(dh, x, *w, kept)
    data = [torch.zeros(70, 336, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :300] for _ in range(2)]
    for a, b in zip(data, kept[::2]):
        a.copy_(b)
    for scales in (lambda s: s.contiguous(), lambda s: s.repeat_interleave(3, 1)[:, ::3]):
        got = gp.gated_backward(dh, x, *w, (data[0], scales(kept[1]), data[1], scales(kept[3])))
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Outputs and inputs of more than 2^31 values: rows from all over against the formulas."""
    M, N, K = 70000, 33000, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w = (torch.randint(-2, 3, s, generator=g, device="cuda").to(BF16) for s in ((M, K), (N, K)))
    rows = torch.tensor([0, 1, 32767, 65077, 65078, M - 2, M - 1], device="cuda")
    y, (data, scales) = gp.linear(x, w, keep="fp8")
    status_ok()
    z = x[rows].double() @ w.double().t()
    assert torch.equal(y[rows], z.to(BF16))
    code, s = fp8_ref.quantize(z.cpu().numpy(), "rows", "e4m3")
    assert fp8_ref.same_codes(fp8_ref.codes(data.view(torch.uint8)[rows].view(torch.float8_e4m3fn)), code, "e4m3")
    assert np.array_equal(scales[rows].cpu().numpy(), s)
    dx, _, db = gp.linear_backward(y, None, w, weight_grad=False, bias_grad=True)
    status_ok()
    assert torch.equal(dx[rows], (y[rows].double() @ w.double()).to(BF16))
    want = torch.zeros(N, dtype=torch.float64, device="cuda")
    for i in range(0, M, 10000):
        want += y[i:i + 10000].double().sum(0)
    # whole numbers of 256 at most in a sum of 2^24 at most: exact in FP32
    assert float(y.abs().max()) <= 256 and torch.equal(db.double(), want)
    got = gp.gated_backward(y, None, w, w, (data, scales, data, scales), activation="relu", product=True, input_grad=False,
                            weight_grad=False)[3]
    status_ok()
    held = torch.from_numpy(fp8_ref.values(code, s, "e4m3").astype(np.float32)).cuda()   # (a code times its scale in FP32)
    assert torch.equal(got[rows], (held.clamp(min=0) * held).to(BF16))
    del y, data, scales, got
    torch.cuda.empty_cache()


def test_refusals():
    x, w, wd, b, r = block_operands(20, 64, 40, 6)
    z = torch.zeros(20, 64, dtype=BF16, device="cuda")
    data, scales = gp.quantize_fp8(z)
    blocks = gp.quantize_fp8(z, "blocks")
    cases = [
        lambda: gp.linear(x.float(), w[0]), lambda: gp.linear(x, w[0].half()), lambda: gp.linear(x, w[0].cpu()),
        lambda: gp.linear(x, wd), lambda: gp.linear(x[0], w[0]), lambda: gp.linear(x.t(), w[0].t()),
        lambda: gp.linear(x, w[0], b), lambda: gp.linear(x, w[0], z[0].half()), lambda: gp.linear(x, w[0], activation="tanh"),
        lambda: gp.linear(x, w[0], keep="fp16"), lambda: gp.linear(x, w[0], residual=r), lambda: gp.linear(x, w[0], residual=z.float()),
        lambda: gp.linear(x, w[0], out_dtype=F16), lambda: gp.linear(x, w[0], out=z, out_dtype=F32),
        lambda: gp.linear(x, w[0], out=z.half()), lambda: gp.linear(x, w[0], out=z[:10]),
        lambda: gp.gated(x, w[0], wd), lambda: gp.gated(x, w[0], w[1][:10]), lambda: gp.gated(x, *w, activation="swish"),
        lambda: gp.gated(x, *w, out=z.float()), lambda: gp.gated(x, *w, keep=1),
        lambda: gp.linear_backward(z, x, wd), lambda: gp.linear_backward(z, x[:4], w[0], weight_grad=False),
        lambda: gp.linear_backward(z, wd, w[0], weight_grad=False), lambda: gp.linear_backward(z[:4], x, w[0]),
        lambda: gp.linear_backward(z, x, w[0], activation="gelu"), lambda: gp.linear_backward(z, x, w[0], kept=(z,)),
        lambda: gp.linear_backward(z, x, w[0], activation="gelu", kept=(z.half(),)),
        lambda: gp.linear_backward(z, x, w[0], activation="gelu", kept=(z[:, :32],)),
        lambda: gp.linear_backward(z, x, w[0], activation="gelu", kept=(data, scales[:1])),
        lambda: gp.linear_backward(z, x, w[0], activation="gelu", kept=(data, blocks[1])),
        lambda: gp.linear_backward(z, x, w[0], activation="gelu", kept=(z, scales)),
        lambda: gp.linear_backward(z, x, w[0], activation="gelu", kept=(data, scales, data)),
        lambda: gp.linear_backward(z, x, w[0], weight_grad=False, addend=w[0]),
        lambda: gp.linear_backward(z, x, w[0], addend=w[0], out_dtype=F32), lambda: gp.linear_backward(z, x, w[0], out=wd),
        lambda: gp.linear_backward(z, x.half(), w[0]), lambda: gp.linear_backward(z, x, w[0], addend=(w[0], w[1])),
        lambda: gp.gated_backward(z, x, *w, None), lambda: gp.gated_backward(z, x, *w, (z,)), lambda: gp.gated_backward(z, x, *w, z),
        lambda: gp.gated_backward(z, x, *w, (data, scales, z, scales)), lambda: gp.gated_backward(z, x, w[0], wd, (z, z)),
        lambda: gp.gated_backward(z, x, *w, (z, z), addend=w[0]), lambda: gp.gated_backward(z, x, *w, (z, z), addend=(w[0], None)),
        lambda: gp.gated_backward(z, x, *w, (z, z), out=[w[0]]), lambda: gp.gated_backward(z, x, *w, (z, z), weight_grad=False, out=w),
    ]
    for i, call in enumerate(cases):
        with pytest.raises(ValueError):
            call()
            print("case", i)
    for call in (lambda: gp.linear(None, w[0]), lambda: gp.linear_backward(z, None, w[0]), lambda: gp.gated_backward(z, None, *w, (z, z)), lambda: gp.linear(x, "w"), lambda: gp.linear(x, w[0], out_dtype=3),
                 lambda: gp.gated_backward(z, x, *w, (z, "z"))):
        with pytest.raises((TypeError, ValueError)):
            call()
    # what the library refuses: rows that overlap, unknown tiles
    wide = torch.zeros(2, 64, dtype=BF16, device="cuda")[:1].expand(20, 64)
    for call in (lambda: gp.linear(wide, w[0].new_zeros(8, 64)), lambda: gp.linear(x, w[0], tile=48),
                 lambda: gp.linear(x, w[0], tile=16, k_splits=8), lambda: gp.linear_backward(z, x, w[0], tile=32)):
        with pytest.raises((gp.GemmError, ValueError)):
            call()
    assert torch.equal(gp.linear(x, w[0]), gp.linear(x, w[0]))      # (still in order)
    status_ok()


def test_gradients_against_differences():
    """dx, dW and db against the quotient of differences of the forward calls, in directions of their own."""
    rng = np.random.default_rng(8)
    M, N, K = 40, 72, 56

    def normal(*s):
        return torch.from_numpy(rng.standard_normal(s)).cuda()

    for act in ref.ACTS[2:]:
        x, w, u, b = normal(M, K) / 4, normal(N, K) / 4, normal(N, K) / 4, normal(N)
        dy = normal(M, N)
        low = [t.to(F16) for t in (x, w, u, b, dy)]
        z = low[0].double() @ low[1].double().t() + low[3].double()
        dx, dw, db = gp.linear_backward(low[4], low[0], low[1], activation=act, kept=(z.to(F16),), bias_grad=True)

        def loss(x, w, b):
            z = ref.f64(x) @ ref.f64(w).T + ref.f64(b)
            return float((ref.value(z, act) * ref.f64(low[4])).sum())

        base = [low[0].double(), low[1].double(), low[3].double()]
        for i, g in enumerate((dx, dw, db)):
            d = torch.from_numpy(rng.standard_normal(tuple(base[i].shape))).cuda()
            step = 1e-5
            plus, minus = [list(base), list(base)]
            plus[i], minus[i] = base[i] + step * d, base[i] - step * d
            want = (loss(*plus) - loss(*minus)) / (2 * step)
            got = float((g.double() * d).sum())
            # each factor was rounded to 11 bits three times at most (z, dz, the gradient): that many units of the sum of
            # magnitudes of what was added up
            scale = float((g.double() * d).abs().sum()) + abs(want)
            assert abs(got - want) <= 3 * 2.0 ** -11 * 4 * scale, (act, i, got, want)


# ---------------------------------------------------------------------------
# sums longer than one accumulator takes (4096 products in FP16, 32768 in BF16, 768 where FP32 leaves)
# ---------------------------------------------------------------------------
LONGEST = {F16: 4096, BF16: 32768}


def one_sign(g, rows, cols, dtype):
    return (torch.rand(rows, cols, generator=g, device="cuda") * 0.5 + 0.5).mul_(2.0 ** -5).to(dtype)


@pytest.mark.parametrize("dtype,K", [(F16, 1 << 20), (BF16, 1 << 22)])
def test_long_sums_of_one_sign(dtype, K):
    """What the tensor cores cut of a sum does not grow with its length: at most 2^-23 of the sum per product of one
    accumulator (half a spacing of the output for as many as it takes), 2^-24 for each of the parts, and the rounding.  A
    product of two sums (1 + a)(1 + b) is off by 2 share + share^2.  What lies past the type's range is infinite."""
    g = torch.Generator(device="cuda").manual_seed(2)
    share = LONGEST[dtype] * 2.0 ** -23 + (K // LONGEST[dtype] + 1) * 2.0 ** -24

    def close(got, want, sums=1):
        off = (1 + share) ** sums - 1
        past = want >= ref.LARGEST[dtype] * (1 + off)
        assert bool(torch.isinf(got[past]).all())
        far = float(((got.double() - want).abs() / want)[~past].max()) if not bool(past.all()) else 0.0
        assert far <= off + ref.UNIT[dtype] * (1 + off), far

    x, w = one_sign(g, 8, K, dtype), one_sign(g, 24, K, dtype)
    want = x.double() @ w.double().t()
    for tile, splits in ((0, 0), (16, 1), (32, 2), (64, 1), (129, 1), (128, 0), (256, 0)):
        y, (z,) = gp.linear(x, w, keep="real", tile=tile, k_splits=splits)
        close(y, want)
        close(z, want)
        if tile != 129:
            h, (gate, up) = gp.gated(x, w, w * 0.5, activation=None, keep="real", tile=tile, k_splits=splits)
            close(h, want * want * 0.5, 2)
            close(gate, want)
            close(up, want * 0.5)
            close(gp.gated(x, w, w * 2.0 ** -6, activation=None, tile=tile, k_splits=splits), want * want * 2.0 ** -6, 2)
    del x, w
    dy, x = one_sign(g, K, 8, dtype), one_sign(g, K, 24, dtype)      # K tokens
    want = dy.double().t() @ x.double()
    z = torch.ones_like(dy)
    for tile, splits in ((0, 0), (64, 1), (129, 1), (128, 0), (256, 0)):
        close(gp.linear_backward(dy, x, x[:8], input_grad=False, tile=tile, k_splits=splits)[1], want)
        _, dg, du = gp.gated_backward(dy, x, x[:8], x[:8], (z, z), activation="relu", input_grad=False, tile=tile, k_splits=splits)
        close(dg, want)
        close(du, want)
    half = K // 2
    dy, w = one_sign(g, 8, half, dtype), one_sign(g, half, 24, dtype)
    want = dy.double() @ w.double()
    z = torch.ones_like(dy)
    for tile, splits in ((0, 0), (16, 1), (64, 2), (129, 1), (128, 0), (256, 0)):
        close(gp.linear_backward(dy, None, w, weight_grad=False, tile=tile, k_splits=splits)[0], want)
        got = gp.gated_backward(dy, None, w, w, (z, z), activation="relu", weight_grad=False, tile=tile, k_splits=splits)[0]
        close(got, 2 * want)                                         # two products, one sum
    status_ok()


@pytest.mark.parametrize("tile", [0, 64, 129, 128, 256])
@pytest.mark.parametrize("K", [4096, 4097, 4160, 8200, 12300])
def test_long_sums_of_whole_numbers_are_exact(tile, K):
    """Around the lengths that one accumulator takes, ragged outputs: every part is added once."""
    M, N = 200, 328
    check_linear(M, N, K, F16, whole=1, bias=F16, residual=True, tile=tile)
    check_linear(M, N + 1, K, F16, whole=1, keep="real", tile=tile, ld=N + 8)
    if tile != 129:
        check_gated(M, N, K, F16, act=None, keep="real", tile=tile)
        check_gated(M, N + 3, K, F16, tile=tile)
    rng = np.random.default_rng(K)
    dy, x, w = (ref.matrix(rng, r, c, F16, whole=1) for r, c in ((K, M), (K, N), (M, N)))
    add = ref.matrix(rng, M, N, F16, whole=2)
    _, dw, _ = gp.linear_backward(dy, x, w, input_grad=False, addend=add, tile=tile)
    assert torch.equal(dw, (dy.double().t() @ x.double() + add.double()).to(F16))
    relu = torch.ones_like(dy)
    _, dg, du = gp.gated_backward(dy, x, w, w, (relu, relu + 1), activation="relu", input_grad=False, tile=tile)
    assert torch.equal(du, (dy.double().t() @ x.double()).to(F16))
    assert torch.equal(dg, (2 * (dy.double().t() @ x.double())).to(F16))
    dy, w = ref.matrix(rng, M, K, F16, whole=1), ref.matrix(rng, K, N, F16, whole=1)
    assert torch.equal(gp.linear_backward(dy, None, w, weight_grad=False, tile=tile)[0], (dy.double() @ w.double()).to(F16))
    half = K // 2
    dy, w, u = ref.matrix(rng, M, half, F16, whole=1), ref.matrix(rng, half, N, F16, whole=1), ref.matrix(rng, half, N, F16, whole=1)
    relu = torch.ones_like(dy)
    got = gp.gated_backward(dy, None, w, u, (relu, relu), activation="relu", weight_grad=False, tile=tile)[0]
    assert torch.equal(got, (dy.double() @ (w.double() + u.double())).to(F16))
    status_ok()


def test_long_sums_cut_in_halves():
    """More tiles than pairs of CTAs, the last of them as halves of their columns, over more than one accumulator's sum."""
    for M, N in ((2560, 2304), (2300, 2500)):
        assert check_linear(M, N, 4200, F16, whole=1, residual=True, tile=256)["half_tiles"] > 0
        assert check_gated(M, N // 2, 4200, F16, keep="real", tile=256)["half_tiles"] > 0


@pytest.mark.parametrize("act", ref.ACTS[1:])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_slopes_far_from_zero(act, dtype):
    """Large kept values, and FP16's that were past its range: an activation's slope there is its limit, 1 or 0, and the
    activation z or 0 (sigmoid: 1 or 0).  A NaN stays one.  Exact, as both are."""
    values = [3e4, 6e4, float("inf")] if dtype is F16 else [1e5, 7e18, 1e20, 3e38, float("inf")]
    z = torch.tensor([v for x in values for v in (x, -x)] + [float("nan")], dtype=dtype, device="cuda")
    n, up = z.numel(), z > 0
    for N in (n, 136):                           # (rows whose four values a lane takes one by one or together)
        wide = torch.ones(3, N, dtype=dtype, device="cuda")
        wide[:, :n] = z
        dy = torch.full((3, N), 0.5, dtype=dtype, device="cuda")
        w = torch.eye(N, dtype=dtype, device="cuda")
        db = gp.linear_backward(dy, None, w, activation=act, kept=(wide,), bias_grad=True, input_grad=False, weight_grad=False)[2]
        slope = torch.zeros(n, device="cuda") if act == "sigmoid" else up.float()
        assert torch.equal(db[:n - 1], 1.5 * slope[:-1]) and bool(torch.isnan(db[n - 1])), db
        h = gp.gated_backward(dy, None, w, w, (wide, torch.full_like(wide, 0.25)), activation=act, product=True, input_grad=False,
                              weight_grad=False)[3]
        value = torch.where(up, torch.ones_like(z) if act == "sigmoid" else z, torch.zeros_like(z))
        assert torch.equal(h[:, :n - 1], (value * 0.25)[:-1].expand(3, n - 1)) and bool(torch.isnan(h[:, n - 1]).all())
        status_ok()


@pytest.mark.parametrize("tile", [64, 128])
@pytest.mark.parametrize("lost", [1, 2, 3])
def test_a_lost_load_in_either_product_of_a_backward_call_is_reported(lost, tile):
    """The status of a call that makes two products is that of both, the first one's too."""
    x, w, _, _, _ = block_operands(300, 384, 1500, 4)
    dy = ref.matrix(np.random.default_rng(5), 300, 384, BF16)
    z = torch.ones_like(dy)
    calls = (lambda **kw: gp.linear_backward(dy, x, w[0], activation="relu", kept=(z,), tile=tile, **kw),
             lambda **kw: gp.gated_backward(dy, x, *w, (z, z), tile=tile, **kw))
    for call in calls:
        want = call()
        status_ok()
        got = call(timeout_ns=5_000_000, inject_lost_load=lost)
        st = gp.gemm_stats(sync=True)
        assert st["status"] == gp.GP_ERR_TIMEOUT and st["device_status"] != 0
        assert gp.gemm_stats(sync=True)["status"] == gp.GP_ERR_TIMEOUT       # (asked again)
        if lost == 1:
            assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]) if a is not None)
        if lost == 2:
            assert torch.equal(got[0], want[0])
        again = call()                                                        # a record of its own
        status_ok()
        assert all(torch.equal(a, b) for a, b in zip(again, want) if a is not None)
    # one product alone
    gp.linear_backward(dy, None, w[0], weight_grad=False, tile=tile, timeout_ns=5_000_000, inject_lost_load=1)
    assert gp.gemm_stats(sync=True)["status"] == gp.GP_ERR_TIMEOUT
    gp.linear_backward(dy, x, w[0], input_grad=False, tile=tile)
    status_ok()
    gp.linear_backward(dy, x, w[0], input_grad=False, tile=tile, timeout_ns=5_000_000, inject_lost_load=2)
    assert gp.gemm_stats(sync=True)["status"] == gp.GP_ERR_TIMEOUT
    gp.linear_backward(dy, x, w[0], tile=tile, inject_lost_load=0)
    status_ok()


def test_the_plan_is_what_runs():
    """gemm_ffn_plan and the record of the call agree, for 16-bit, FP32 and coded outputs of every product."""
    def same(planned):
        ran = status_ok()
        assert {k: v for k, v in planned.items() if ran[k] != v} == {}, ran

    rng = np.random.default_rng(1)
    for M, N, K in ((1, 4096, 4096), (40, 1000, 520), (130, 264, 4100), (700, 1100, 264), (300, 300, 9000)):
        for dtype in (F16, BF16):
            x, w, u, dy = (ref.matrix(rng, r, c, dtype) for r, c in ((M, K), (N, K), (N, K), (M, N)))
            z = torch.ones_like(dy)
            for out in (None, F32):
                for keep in (None, "real", "fp8"):
                    gp.linear(x, w, keep=keep, out_dtype=out)
                    same(gp.ffn_plan("linear", M, N, K, dtype=dtype, out_dtype=out, kept=keep == "fp8"))
                gp.linear_backward(dy, x, w, input_grad=False, out_dtype=out)
                same(gp.ffn_plan("weight_grad", M, N, K, dtype=dtype, out_dtype=out))
                gp.gated_backward(dy, x, w, u, (z, z), input_grad=False, out_dtype=out)
                same(gp.ffn_plan("weight_grad", M, N, K, dtype=dtype, out_dtype=out, count=2))
            for keep in (None, "real", "fp8"):
                gp.gated(x, w, u, keep=keep)
                same(gp.ffn_plan("gated", M, N, K, dtype=dtype, kept=keep == "fp8"))
            gp.linear_backward(dy, x, w, weight_grad=False)
            same(gp.ffn_plan("input_grad", M, N, K, dtype=dtype))
            gp.gated_backward(dy, x, w, u, (z, z), weight_grad=False)
            same(gp.ffn_plan("input_grad", M, N, K, dtype=dtype, count=2))


@pytest.mark.parametrize("M", [1, 16])
def test_few_rows_by_eight_ctas(M):
    assert check_linear(M, 300, 4096, BF16, "silu", bias=BF16, k_splits=8)["k_splits"] == 8
    assert check_gated(M, 300, 4096, BF16, k_splits=8)["k_splits"] == 8
    check_linear_backward(M, 4096, 300, BF16, k_splits=8)


def test_a_refused_argument_launches_nothing():
    """Every argument is looked at before rows are laid out or a product runs: the record is still the call's before."""
    rng = np.random.default_rng(14)
    M, N, K = 40, 72, 61
    x, w, u, dy = (ref.matrix(rng, r, c, BF16) for r, c in ((M, K), (N, K), (N, K), (M, N)))     # rows off 16-byte boundaries
    z = torch.ones_like(dy)
    a, b = ref.matrix(rng, 8, 64, BF16), ref.matrix(rng, 16, 64, BF16)
    gp.linear(a, b)
    before = status_ok()
    wrong = torch.zeros(N, K + 1, dtype=BF16, device="cuda")
    wide = torch.zeros(N, K, dtype=F32, device="cuda")
    for call in (lambda: gp.linear(x, w[:, :K - 1]), lambda: gp.linear(x, w, z[0, :5]), lambda: gp.linear(x, w, out=wrong),
                 lambda: gp.linear(x, w, residual=wrong), lambda: gp.linear(x, w, out_dtype=F16), lambda: gp.linear(x, w.half()),
                 lambda: gp.gated(x, w, u[:5]), lambda: gp.gated(x, w, u.half()), lambda: gp.gated(x, w, u, out=wrong),
                 lambda: gp.linear_backward(dy, x, w, out=wrong), lambda: gp.linear_backward(dy, x, w, out=x[:N]),
                 lambda: gp.linear_backward(dy, x, w, addend=wrong), lambda: gp.linear_backward(dy, x, w, out_dtype=F16),
                 lambda: gp.linear_backward(dy, x, w.half()), lambda: gp.linear_backward(dy, x, w, out=wide, addend=w),
                 lambda: gp.linear_backward(dy, x, w, activation="gelu", kept=(w,)),
                 lambda: gp.linear_backward(dy, x, w, activation="gelu", kept=(z,), bias_grad=True, out=wrong),
                 lambda: gp.gated_backward(dy, x, w, u, (z, w)), lambda: gp.gated_backward(dy, x, w, u, (z, z), out=(wide, wide)),
                 lambda: gp.gated_backward(dy, x, w, u, (z, z), out=(wrong, w)),
                 lambda: gp.gated_backward(dy, x, w, u.half(), (z, z)), lambda: gp.gated_backward(dy, x, w, u, (z, z), out_dtype=F16)):
        with pytest.raises(ValueError):
            call()
        assert status_ok() == before
    got = gp.linear_backward(dy, x, w, activation="relu", kept=(z,), out=wide)[1]        # and an FP32 output of such rows
    assert got is wide and torch.equal(wide, gp.linear_backward(dy, x, w, activation="relu", kept=(z,), out_dtype=F32)[1])


def test_refused_arguments_raise_value_errors():
    """What the calls look at themselves is a ValueError: codes off 16-byte boundaries, rows that overlap, options out of range."""
    x, w, wd, b, r = block_operands(20, 64, 40, 6)
    z = torch.ones(20, 64, dtype=BF16, device="cuda")
    data, scales = gp.quantize_fp8(z)
    off = torch.zeros(20, 65, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    late = torch.zeros(20 * 64 + 8, dtype=torch.uint8, device="cuda")[8:].view(20, 64).view(torch.float8_e4m3fn)
    lines = {n: torch.zeros(1, n, dtype=BF16, device="cuda").expand(20, n) for n in (40, 64)}
    one = torch.zeros(1, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).expand(20, 64)
    for call in (lambda q: gp.linear_backward(z, x, w[0], activation="gelu", kept=(q, scales)),
                 lambda q: gp.gated_backward(z, x, *w, (q, scales, data, scales)),
                 lambda q: gp.gated_backward(z, x, *w, (data, scales, q, scales))):
        for q in (off[:, :64], late, one):
            with pytest.raises(ValueError, match="rows of the"):
                call(q)
    for call in (lambda: gp.linear(lines[40], w[0]), lambda: gp.gated(lines[40], *w), lambda: gp.linear(x, w[0], residual=lines[64]),
                 lambda: gp.linear(x, w[0], out=lines[64]), lambda: gp.gated(x, *w, out=lines[64]),
                 lambda: gp.linear_backward(lines[64], x, w[0]), lambda: gp.linear_backward(lines[64], x, w[0], bias_grad=True),
                 lambda: gp.linear_backward(z, x, w[0], activation="gelu", kept=(lines[64],)),
                 lambda: gp.linear_backward(z, x, w[0], out=torch.zeros(1, 40, dtype=BF16, device="cuda").expand(64, 40)),
                 lambda: gp.gated_backward(lines[64], x, *w, (z, z)), lambda: gp.gated_backward(z, x, *w, (z, lines[64]))):
        with pytest.raises(ValueError, match="overlap"):
            call()
    for options in (dict(timeout_ns=-1), dict(tile=1 << 40), dict(tile=64.0), dict(k_splits="2"), dict(timeout_ns=1 << 64)):
        for call in (lambda: gp.linear(x, w[0], **options), lambda: gp.gated(x, *w, **options),
                     lambda: gp.linear_backward(z, x, w[0], **options), lambda: gp.gated_backward(z, x, *w, (z, z), **options)):
            with pytest.raises(ValueError):
                call()
    # what is not read may be anything of its shape
    flat = torch.zeros(1, 40, dtype=BF16, device="cuda").expand(64, 40)
    assert torch.equal(gp.linear_backward(z, x, flat, input_grad=False)[1], gp.linear_backward(z, x, w[0], input_grad=False)[1])
    # a single row's stride says nothing
    gp.linear_backward(z[:1], x[:1], w[0], activation="gelu", kept=(data[:1], scales[:1]))
    status_ok()


def test_outputs_given_count_as_changed():
    """Writing to `out` moves its version, so that autograd refuses values that it kept of it; results carry no graph."""
    x, w, wd, b, r = block_operands(20, 64, 40, 6)
    z = torch.ones(20, 64, dtype=BF16, device="cuda")
    outs = [torch.zeros(20, 64, dtype=BF16, device="cuda"), torch.zeros(20, 64, dtype=BF16, device="cuda")]
    outs += [torch.zeros(64, 40, dtype=F32, device="cuda") for _ in range(3)]
    calls = (lambda: gp.linear(x, w[0], out=outs[0]), lambda: gp.gated(x, *w, out=outs[1]),
             lambda: gp.linear_backward(z, x, w[0], out=outs[2]), lambda: gp.gated_backward(z, x, *w, (z, z), out=outs[3:]))
    written = ([0], [1], [2], [3, 4])
    for call, which in zip(calls, written):
        before = [t._version for t in outs]
        read = [t._version for t in (x, w[0], w[1], z)]
        call()
        assert [t._version - v for t, v in zip(outs, before)] == [int(i in which) for i in range(5)]
        assert [t._version for t in (x, w[0], w[1], z)] == read
    leaf = torch.ones(20, 64, device="cuda", requires_grad=True)
    buf = torch.zeros(20, 64, dtype=BF16, device="cuda")
    y = (leaf * buf).sum()                       # autograd keeps buf
    gp.linear(x, w[0], out=buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    leaf = w[0].clone().requires_grad_()
    assert not gp.linear(x, leaf).requires_grad
    with torch.inference_mode():
        frozen = torch.zeros(20, 64, dtype=BF16, device="cuda")
        assert gp.linear(x, w[0], out=frozen) is frozen
    assert gp.linear(x, w[0], out=frozen) is frozen and torch.equal(frozen, gp.linear(x, w[0]))
    status_ok()


# ---------------------------------------------------------------------------
# 128 rows by a cluster (tile 129), which the planner takes for some sizes between
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("splits", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 200, 700), (100, 1000, 333), (129, 264, 520), (200, 128, 1300), (513, 700, 1300)])
def test_linear_128_rows_by_a_cluster(M, N, K, splits):
    assert check_linear(M, N, K, BF16, "silu", bias=BF16, residual=True, tile=129, k_splits=splits)["bn"] == 128
    check_linear(M, N, K, F16, None, keep="real", out_dtype=F32, tile=129, k_splits=splits)
    check_linear(M, N, K, F16, whole=2, residual=True, out_dtype=F32, tile=129, k_splits=splits)


# rows of the weight's gradient: ends of 1 to 63, 64, and 65 to 127 past the last 128, and fewer than 64 in all
ENDS = [1, 40, 63, 64, 65, 100, 127, 128, 129, 191, 192, 193, 255, 300, 512]


@pytest.mark.parametrize("splits", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("N", ENDS)
def test_backward_128_rows_by_a_cluster(N, splits):
    for M, K in ((20, 128), (300, 65), (600, 333)):
        check_linear_backward(M, N, K, BF16, tile=129, k_splits=splits, out_dtype=F32, add=True)
        check_linear_backward(M, N, K, F16, "silu", "fp8", tile=129, k_splits=splits)
        check_gated_backward(M, N, K, BF16, tile=129, k_splits=splits)


@pytest.mark.parametrize("tile", [64, 129])
@pytest.mark.parametrize("splits", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("N", ENDS)
def test_backward_by_a_cluster_whole_numbers_are_exact(N, splits, tile):
    """One product and two in a launch, ends of either operand, sums in one part and in many."""
    rng = np.random.default_rng(N)
    for M, K in ((20, 128), (130, 65), (1000, 190), (2000, 8)):
        dy, x, w, u = (ref.matrix(rng, r, c, BF16, whole=2) for r, c in ((M, N), (M, K), (N, K), (N, K)))
        a, b, c, d = (t.double() for t in (dy, x, w, u))
        add = ref.matrix(rng, N, K, F32, whole=3)
        dx, dw, _ = gp.linear_backward(dy, x, w, out_dtype=F32, addend=add, tile=tile, k_splits=splits)
        plan = status_ok()
        assert plan["layout"] == 1 and plan["bn"] == min(tile, 128)
        assert torch.equal(dw.double(), a.t() @ b + add.double()) and torch.equal(dx, (a @ c).to(BF16))
        z = torch.ones_like(dy)
        dx, dg, du = gp.gated_backward(dy, x, w, u, (z, z + 1), activation="relu", out_dtype=F32, tile=tile, k_splits=splits)
        assert torch.equal(dg.double(), 2 * (a.t() @ b)) and torch.equal(du.double(), a.t() @ b)
        assert torch.equal(dx, (a @ (2 * c + d)).to(BF16))
        dx, dg, du = gp.gated_backward(dy, x, w, u, (z, z + 1), activation="relu", tile=tile, k_splits=splits)
        assert torch.equal(dg, (2 * (a.t() @ b)).to(BF16)) and torch.equal(du, (a.t() @ b).to(BF16))
    status_ok()


def test_sizes_where_the_planner_takes_128_rows_by_a_cluster():
    for op, M, N, K, count in (("weight_grad", 6458, 902, 692, 1), ("input_grad", 199, 4631, 3884, 1), ("input_grad", 512, 2048, 1024, 2)):
        p = gp.ffn_plan(op, M, N, K, count=count)
        assert p["layout"] == 1 and p["bn"] == 128, (op, M, N, K, p)
    check_linear_backward(6458, 902, 692, BF16)
    check_linear_backward(199, 4631, 3884, F16, weight_grad=False)
    check_gated_backward(512, 2048, 1024, BF16)
