"""gemm_fp8 against the product in float64 of the values that codes and scales
stand for, element by element within a bound derived from the arithmetic
(fp8_ref.gemm_bound): sizes around the tiles, every format and kind of scales,
strides, addends, values that are not finite, and refusals."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
import software_pipelined_tiled_pipeline_gb300 as gp

pytestmark = pytest.mark.gpu

GUARD = 512


def guarded(rows, cols, out, ld=None):
    """A NaN-filled output inside a NaN-filled buffer, and the buffer."""
    ld = ld or cols
    buf = torch.full((rows * ld + 2 * GUARD,), float("nan"), dtype=ref.REAL[out], device="cuda")
    return buf[GUARD:GUARD + rows * ld].view(rows, ld)[:, :cols], buf


def outside_untouched(buf, rows, cols, ld):
    body = buf[GUARD:GUARD + rows * ld].view(rows, ld)
    return bool(torch.isnan(buf[:GUARD]).all() and torch.isnan(buf[GUARD + rows * ld:]).all()
                and torch.isnan(body[:, cols:]).all())


def check(a, b, out="bf16", addend=None, ld=None, **kw):
    M, N = a.code.shape[0], b.code.shape[0]
    C, buf = guarded(M, N, out, ld)
    add = None
    if addend is not None:
        add = torch.from_numpy(addend).cuda().to(ref.REAL[out])
        addend = ref.f64(add)
    gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out=C, addend=add, **kw)
    st = gp.gemm_stats(sync=True)
    assert st["status"] == 0, (gp.strerror(st["status"]), st["device_status"], st["cuda_error"])
    x, y = a.values, b.values
    want = x @ y.T + (0 if addend is None else addend)
    got = ref.f64(C)
    bound = ref.gemm_bound(x, y, want, out, addend)
    got, want = ref.past_the_range(got, want, bound, out)
    worst = np.max(np.abs(got - want) / bound) if want.size else 0.0
    assert worst <= 1.0, "%g of the bound at %s (plan %s)" % (
        worst, np.unravel_index(np.argmax(np.abs(got - want) / bound), want.shape), st["plan"])
    assert outside_untouched(buf, M, N, ld or N), "write outside C"
    return C, st["plan"]


SHAPES = [(1, 1, 1), (1, 16, 16), (1, 300, 4096), (2, 129, 128), (16, 128, 130), (17, 127, 257), (31, 1000, 520),
          (33, 257, 129), (64, 640, 1024), (65, 200, 384), (128, 128, 128), (129, 130, 1000), (300, 70, 257),
          (70, 300, 2057), (511, 385, 640), (260, 1030, 300), (1000, 776, 2056), (5, 4096, 8192), (4100, 3, 700),
          (500, 600, 8200), (2100, 2300, 256), (3, 700, 513), (4, 129, 4100), (300, 2, 777),
          (1, 41, 20001), (4, 40, 9000), (2, 64, 17000), (8, 700, 2050)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kinds", [("rows", "blocks"), ("rows", "rows"), ("blocks", "rows"), ("blocks", "blocks")])
def test_shapes_and_scales(M, N, K, kinds):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a = ref.Fp8(M, K, kinds[0], "e4m3", rng)
    b = ref.Fp8(N, K, kinds[1], "e4m3", rng, order="rows")
    check(a, b, out=["bf16", "f16", "f32"][(M + N + K) % 3] if K < 200 else "bf16")


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3", "e5m2"])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(9, 200, 400), (300, 260, 520)])
def test_formats_and_output_types(fa, fb, out, M, N, K):
    rng = np.random.default_rng(11)
    a = ref.Fp8(M, K, "rows", fa, rng, spread_log2=0.5)
    b = ref.Fp8(N, K, "blocks", fb, rng, spread_log2=0.5)
    check(a, b, out)
    check(a, b, out, addend=rng.standard_normal((M, N)) * 5)


@pytest.mark.parametrize("bn", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kinds", [("rows", "blocks"), ("blocks", "rows"), ("rows", "rows"), ("blocks", "blocks")])
def test_every_width(bn, kinds):
    rng = np.random.default_rng(bn)
    a, b = ref.Fp8(200, 700, kinds[0], "e4m3", rng), ref.Fp8(333, 700, kinds[1], "e5m2", rng)
    check(a, b, bn=bn)


@pytest.mark.parametrize("order", ["groups", "rows", "strided"])
def test_strides(order):
    rng = np.random.default_rng(3)
    for M, N, K in [(40, 150, 300), (200, 300, 300)]:
        a = ref.Fp8(M, K, "rows", "e4m3", rng).put(order, pad=512)
        b = ref.Fp8(N, K, "blocks", "e4m3", rng).put(order, pad=320)
        for out, ld in (("bf16", N + 1), ("f32", N + 3), ("f16", N + 4)):
            check(a, b, out, ld=ld)


@pytest.mark.parametrize("M,N", [(3, 200), (200, 3), (300, 301)])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
def test_addend_in_place(M, N, out):
    rng = np.random.default_rng(4)
    a, b = ref.Fp8(M, 260, "rows", "e4m3", rng), ref.Fp8(N, 260, "rows", "e4m3", rng)
    C0 = torch.from_numpy(rng.standard_normal((M, N + 5))).cuda().to(ref.REAL[out])[:, :N]
    apart = gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out_dtype=ref.REAL[out], addend=C0)
    C = C0.clone(memory_format=torch.preserve_format)
    wide = torch.zeros((M, N + 5), dtype=C.dtype, device="cuda")
    wide[:, :N] = C0
    here = wide[:, :N]
    assert gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out=here, addend=here) is here
    assert torch.equal(here, apart)
    assert bool((wide[:, N:] == 0).all())


@pytest.mark.parametrize("M,N,K", [(8, 256, 512), (256, 384, 1024), (300, 520, 4096)])
def test_whole_numbers_are_exact(M, N, K):
    # codes of small whole numbers and scales of powers of two: every sum is exact in FP32, in any order
    rng = np.random.default_rng(6)
    a, b = ref.Fp8(M, K, "rows", "e4m3", rng), ref.Fp8(N, K, "blocks", "e4m3", rng)
    for m in (a, b):
        m.code = ref.encode(rng.integers(-2, 3, m.code.shape), "e4m3")
        m.s = np.exp2(rng.integers(-1, 2, m.s.shape)).astype(np.float32)
        m.put()
    C = gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out_dtype=torch.float32)
    assert np.array_equal(ref.f64(C), a.values @ b.values.T)


@pytest.mark.parametrize("M,N,K", [(5, 300, 1000), (300, 260, 1000)])
def test_each_k_block_counts_once(M, N, K):
    # one K block at a time holds the only nonzero values
    rng = np.random.default_rng(7)
    for kb in range(-(-K // 128)):
        x = np.zeros((M, K))
        x[:, kb * 128:(kb + 1) * 128] = rng.standard_normal((M, min(128, K - kb * 128)))
        check(ref.Fp8(M, K, "rows", "e4m3", rng, data=x), ref.Fp8(N, K, "blocks", "e4m3", rng))


@pytest.mark.parametrize("M,N", [(20, 200), (200, 20), (260, 270)])
def test_not_a_number_and_infinity_stay_in_their_rows(M, N):
    rng = np.random.default_rng(8)
    K = 384
    x = rng.standard_normal((M, K))
    x[3, 200], x[M - 1, 5] = np.nan, np.inf
    a = ref.Fp8(M, K, "rows", "e4m3", rng, data=x)
    b = ref.Fp8(N, K, "blocks", "e4m3", rng)
    C = ref.f64(gp.gemm_fp8(a.data, a.scales, b.data, b.scales))
    bad = np.isnan(C)
    assert bad[[3, M - 1]].all() and bad.sum() == 2 * N
    good = [r for r in range(M) if r not in (3, M - 1)]
    want = a.values[good] @ b.values.T
    assert np.all(np.abs(C[good] - want) <= ref.gemm_bound(a.values[good], b.values, want, "bf16"))


def test_rows_of_zeros():
    rng = np.random.default_rng(9)
    x = rng.standard_normal((50, 300))
    x[7] = 0.0
    a, b = ref.Fp8(50, 300, "rows", "e4m3", rng, data=x), ref.Fp8(140, 300, "blocks", "e4m3", rng)
    C, _ = check(a, b)
    assert bool((C[7] == 0).all())


def test_k_of_zero():
    a = torch.empty((5, 0), dtype=torch.float8_e4m3fn, device="cuda")
    b = torch.empty((7, 0), dtype=torch.float8_e4m3fn, device="cuda")
    sa, sb = torch.empty((5, 0), device="cuda"), torch.empty((1, 0), device="cuda")
    add = torch.randn(5, 7, device="cuda").to(torch.bfloat16)
    for out in (torch.float16, torch.bfloat16, torch.float32):
        assert bool((gp.gemm_fp8(a, sa, b, sb, out_dtype=out) == 0).all())
    assert torch.equal(gp.gemm_fp8(a, sa, b, sb, addend=add), add)


def test_empty_outputs():
    rng = np.random.default_rng(2)
    b = ref.Fp8(7, 64, "blocks", "e4m3", rng)
    a = torch.empty((0, 64), dtype=torch.float8_e4m3fn, device="cuda")
    assert gp.gemm_fp8(a, torch.empty((0, 1), device="cuda"), b.data, b.scales).shape == (0, 7)


def test_offsets_past_32_bits():
    rng = np.random.default_rng(10)
    M, N, K = 70, 130, 300
    a, b = ref.Fp8(M, K, "rows", "e4m3", rng), ref.Fp8(N, K, "blocks", "e4m3", rng)
    ld = 1 << 26                                       # 70 rows: 4.7e9 elements
    wide = torch.empty((M, ld), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    wide[:, :K].copy_(a.data)
    C = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")[:, :N]
    gp.gemm_fp8(wide[:, :K], a.scales, b.data, b.scales, out=C)
    assert torch.equal(C, gp.gemm_fp8(a.data, a.scales, b.data, b.scales))


def test_same_bits_every_time_and_on_another_stream():
    rng = np.random.default_rng(12)
    a, b = ref.Fp8(37, 4096, "rows", "e4m3", rng), ref.Fp8(640, 4096, "blocks", "e4m3", rng)
    first = gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out_dtype=torch.float32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for i in range(40):
        outs.append(gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out_dtype=torch.float32,
                                stream=side if i % 2 else None))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


def test_replays_in_a_graph():
    rng = np.random.default_rng(13)
    a, b = ref.Fp8(5, 4096, "rows", "e4m3", rng), ref.Fp8(512, 4096, "blocks", "e4m3", rng)
    want = gp.gemm_fp8(a.data, a.scales, b.data, b.scales)
    C = torch.zeros_like(want)
    s = torch.cuda.Stream()
    gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out=C, stream=s)   # a first call, outside the capture
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out=C)
    for _ in range(3):
        C.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want)


@pytest.mark.parametrize("M,N,K", [(3, 512, 4096), (200, 300, 1024), (300, 2000, 1024)])
def test_lost_load_reports_timeout_and_the_context_survives(M, N, K):
    rng = np.random.default_rng(14)
    a, b = ref.Fp8(M, K, "rows", "e4m3", rng), ref.Fp8(N, K, "blocks", "e4m3", rng)
    gp.gemm_fp8(a.data, a.scales, b.data, b.scales, timeout_ns=50_000_000, inject_lost_load=True)
    st = gp.gemm_stats(sync=True)
    assert st["status"] == gp.GP_ERR_TIMEOUT and st["device_status"] & 0xFF == 1
    for _ in range(2):
        check(a, b)


def test_refusals():
    rng = np.random.default_rng(15)
    a, b = ref.Fp8(5, 256, "rows", "e4m3", rng), ref.Fp8(6, 256, "rows", "e4m3", rng)
    with pytest.raises(ValueError):
        gp.gemm_fp8(a.data.view(torch.uint8), a.scales, b.data, b.scales)
    with pytest.raises(ValueError):
        gp.gemm_fp8(a.data, a.scales.double(), b.data, b.scales)
    with pytest.raises(ValueError):
        gp.gemm_fp8(a.data, a.scales[:, :1], b.data, b.scales)
    with pytest.raises(ValueError):
        gp.gemm_fp8(a.data[:, :128], a.scales[:, :1], b.data, b.scales)
    with pytest.raises(ValueError):
        gp.gemm_fp8(a.data, a.scales.cpu(), b.data, b.scales)
    with pytest.raises(ValueError):
        gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out=torch.empty(5, 7, device="cuda"))
    with pytest.raises(ValueError):
        gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        gp.gemm_fp8(a.data, a.scales, b.data, b.scales, addend=torch.empty(5, 6, device="cuda"))
    with pytest.raises(ValueError):
        gp.gemm_fp8(a.data.t(), a.scales, b.data, b.scales)
    with pytest.raises(gp.GemmError) as err:            # rows that do not begin on 16-byte boundaries
        gp.gemm_fp8(torch.empty(5, 250, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), a.scales,
                    b.data[:, :250], b.scales)
    assert err.value.code == gp.GP_ERR_UNSUPPORTED


def test_out_of_another_type_than_asked_for_is_refused():
    rng = np.random.default_rng(16)
    a, b = ref.Fp8(5, 256, "rows", "e4m3", rng), ref.Fp8(6, 256, "rows", "e4m3", rng)
    args = (a.data, a.scales, b.data, b.scales)
    for have in (torch.float16, torch.bfloat16, torch.float32):
        out = torch.full((5, 6), 3.0, dtype=have, device="cuda")
        for want in (torch.float16, torch.bfloat16, torch.float32):
            if want is have:
                continue
            with pytest.raises(ValueError):
                gp.gemm_fp8(*args, out=out, out_dtype=want)
            with pytest.raises(ValueError):
                gp.gemm_fp8(*args, out=out, out_dtype=want, stream=torch.cuda.Stream())
        assert bool((out == 3).all())
        fresh = gp.gemm_fp8(*args, out_dtype=have)
        assert fresh.dtype is have
        for kw in (dict(), dict(out_dtype=have)):       # out's own type, named or not
            assert gp.gemm_fp8(*args, out=out, **kw) is out and torch.equal(out, fresh)
            out.fill_(3.0)
    assert gp.gemm_fp8(*args).dtype is torch.bfloat16


def tile_regions(M, N, plan):
    """(rows, columns) of C of each output tile, in the kernel's order."""
    P, Q = (N, M) if plan["layout"] else (M, N)
    bm, bn, group = plan["bm"], plan["bn"], plan["raster_gm"]
    p_blocks, q_blocks = -(-P // bm), -(-Q // bn)
    for first in range(0, p_blocks, group):
        for qb in range(q_blocks):
            for pb in range(first, min(first + group, p_blocks)):
                p, q = slice(pb * bm, (pb + 1) * bm), slice(qb * bn, (qb + 1) * bn)
                yield (q, p) if plan["layout"] else (p, q)


@pytest.mark.parametrize("which", [1, 2])
@pytest.mark.parametrize("M,N,K,bn", [(3, 512, 4096, 0), (3, 1024, 2048, 0), (20, 4096, 1024, 0), (200, 300, 1024, 16),
                                      (200, 300, 1024, 32), (200, 300, 1024, 64), (200, 300, 1024, 128),
                                      (2100, 2300, 512, 64)])
def test_a_tile_with_a_lost_load_is_not_written(M, N, K, bn, which):
    # the first or last tile, whose K loop may be shared by a cluster: none of its CTAs writes sums that lack a share
    rng = np.random.default_rng(17)
    a, b = ref.Fp8(M, K, "rows", "e4m3", rng), ref.Fp8(N, K, "blocks", "e4m3", rng)
    C, buf = guarded(M, N, "f32")
    gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out=C, bn=bn, timeout_ns=20_000_000, inject_lost_load=which)
    st = gp.gemm_stats(sync=True)
    assert st["status"] == gp.GP_ERR_TIMEOUT
    assert outside_untouched(buf, M, N, N)
    if bn == 0:
        assert st["plan"]["k_splits"] == {512: 8, 1024: 4, 4096: 2}[N]
    x, y = a.values, b.values
    want = x @ y.T
    near = np.abs(ref.f64(C) - want) <= ref.gemm_bound(x, y, want, "f32")
    regions = list(tile_regions(M, N, st["plan"]))
    assert len(regions) == st["plan"]["tiles"]
    for i, at in enumerate(regions):
        untouched = bool(torch.isnan(C[at]).all())
        if i == (0 if which == 2 else len(regions) - 1):
            assert untouched, "the tile without a load was written"
        else:
            assert untouched or near[at].all()


@pytest.mark.parametrize("no_split", [True, False])
def test_a_lost_load_does_not_hold_the_gpu_for_the_rest_of_a_long_k_loop(no_split):
    # the first of 1024 K blocks never comes: each later wait would take its tries' 100 us again
    M, N, K = 3, 128, 131072
    q = torch.zeros((M + N, K), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.ones((M + N, K // 128), device="cuda")
    args = (q[:M], s[:M], q[M:], s[M:])
    out = torch.full((M, N), float("nan"), device="cuda")
    gp.gemm_fp8(*args, out=out, no_split=no_split)
    torch.cuda.synchronize()
    assert bool((out == 0).all())
    out.fill_(float("nan"))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    gp.gemm_fp8(*args, out=out, no_split=no_split, timeout_ns=20_000_000, inject_lost_load=2)
    end.record()
    st = gp.gemm_stats(sync=True)
    assert st["status"] == gp.GP_ERR_TIMEOUT and st["plan"]["k_splits"] == (1 if no_split else 8)
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[next(tile_regions(M, N, st["plan"]))]).all())
    assert 20 <= begin.elapsed_time(end) <= 80           # ms: the limit, and a batch of tries after it


def check_with_addend(a, b, out, ld, rng, **kw):
    """The product with an addend of its own and with the output as addend: the same bits, and within the bound."""
    M, N = a.code.shape[0], b.code.shape[0]
    add = rng.standard_normal((M, N)) * 5
    apart, plan = check(a, b, out, addend=add, ld=ld, **kw)
    C, buf = guarded(M, N, out, ld)
    C.copy_(torch.from_numpy(add).cuda())
    assert gp.gemm_fp8(a.data, a.scales, b.data, b.scales, out=C, addend=C, **kw) is C
    assert torch.equal(C, apart) and outside_untouched(buf, M, N, ld)
    return plan


@pytest.mark.parametrize("bn", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("kinds,K,swapped", [(("rows", "blocks"), 700, (0, 0)), (("rows", "rows"), 300, (0, 0)),
                                             (("blocks", "rows"), 4100, (1, 1))])
def test_addends_at_every_width(bn, out, kinds, K, swapped):
    # whole tiles and ragged ones, rows on and off the alignment of whole stores; the operand with block scales takes
    # the N side of wide tiles, so that both roles come about
    rng = np.random.default_rng(bn + K)
    M, N = 300, 520
    a, b = ref.Fp8(M, K, kinds[0], "e4m3", rng, spread_log2=0.5), ref.Fp8(N, K, kinds[1], "e5m2", rng, spread_log2=0.5)
    for ld in (N, N + 2, N + 3):
        plan = check_with_addend(a, b, out, ld, rng, bn=bn, no_split=True)
        assert plan["bn"] == bn and plan["k_splits"] == 1 and plan["cta_pair"] == (bn == 256)
        if bn >= 128:
            assert plan["layout"] == swapped[bn == 256]


# (M, N, K): the plan on 152 SMs -- 1 where B takes the M side, width, CTAs per tile
FEW_ROWS = [((1, 4096, 4096), (1, 16, 4)), ((1, 300, 4096), (1, 16, 8)), ((9, 2048, 1024), (1, 16, 2)),
            ((33, 4000, 1024), (1, 16, 1)), ((50, 8192, 1024), (1, 32, 1)), ((5, 130, 1024), (0, 16, 2)),
            ((200, 9, 4096), (0, 16, 8)), ((640, 33, 2056), (0, 16, 4)), ((1030, 60, 4096), (0, 32, 4)),
            ((1, 128, 512), (0, 16, 1))]


@pytest.mark.parametrize("shape,plan", FEW_ROWS)
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
def test_few_rows_in_every_plan(shape, plan, out):
    M, N, K = shape
    rng = np.random.default_rng(M + N)
    a = ref.Fp8(M, K, "rows", "e4m3", rng, spread_log2=0.5)
    b = ref.Fp8(N, K, "blocks" if M % 2 else "rows", "e4m3", rng, spread_log2=0.5)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for ld in (N, N + 3):
        got = check(a, b, out, ld=ld)[1], check_with_addend(a, b, out, ld, rng)
        for p in got:
            assert sms != 152 or (p["layout"], p["bn"], p["k_splits"]) == plan
    whole = check(a, b, out, no_split=True)[1]
    assert whole["k_splits"] == 1


# width forced, kinds of scales, (M, N, K): the plan on 152 SMs -- 1 where B takes the M side, CTAs per tile
CLUSTERS = [(16, "rb", (100, 200, 8192), (0, 8)), (16, "rb", (700, 150, 8192), (0, 2)), (16, "rb", (20, 2400, 8192), (1, 2)),
            (32, "rb", (100, 200, 8192), (0, 8)), (32, "rr", (700, 150, 8192), (0, 4)), (32, "rb", (300, 500, 8192), (0, 2)),
            (32, "rb", (20, 1100, 8192), (1, 8)), (32, "rb", (20, 2400, 8192), (1, 4)), (32, "rr", (260, 1000, 8192), (1, 2)),
            (64, "rb", (100, 200, 8192), (0, 8)), (64, "rb", (300, 500, 8192), (0, 4)), (64, "rr", (260, 1000, 8192), (0, 2)),
            (64, "rb", (60, 2000, 8192), (1, 8)), (64, "rb", (20, 2400, 8192), (1, 4)), (64, "rb", (60, 9000, 8192), (1, 2)),
            (128, "rb", (100, 200, 8192), (0, 8)), (128, "rb", (260, 1000, 8192), (0, 4)), (128, "rb", (60, 9000, 8192), (0, 2)),
            (128, "br", (300, 500, 32768), (1, 8)), (128, "br", (500, 600, 16384), (1, 4)), (128, "br", (900, 1100, 8192), (1, 2))]


@pytest.mark.parametrize("bn,kinds,shape,plan", CLUSTERS)
def test_clusters_of_every_width_and_role(bn, kinds, shape, plan):
    M, N, K = shape
    rng = np.random.default_rng(bn + M)
    kind = {"r": "rows", "b": "blocks"}
    a = ref.Fp8(M, K, kind[kinds[0]], "e4m3", rng, spread_log2=0.5)
    b = ref.Fp8(N, K, kind[kinds[1]], "e4m3", rng, spread_log2=0.5)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for out in ("f16", "bf16", "f32"):
        got = check(a, b, out, bn=bn)[1], check_with_addend(a, b, out, N + (out == "f16"), rng, bn=bn)
        for p in got:
            assert p["bn"] == bn
            assert sms != 152 or (p["layout"], p["k_splits"]) == plan
