"""Host-side checks of the 8-bit operators' C ABI (no GPU): argument errors are
reported before anything is launched, struct layouts match the header, the
plan follows its rules, and the tests' own plain formats agree with torch's."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import fp8_ref as ref
from software_pipelined_tiled_pipeline_gb300 import build as gbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 0x10000


@pytest.fixture(scope="module")
def gp():
    gbuild.build()
    import software_pipelined_tiled_pipeline_gb300 as mod
    mod.lib()
    return mod


def matrix(data=PTR, scales=PTR, ld=256, row=1, col=64, fmt=0, group=1):
    from software_pipelined_tiled_pipeline_gb300 import _binding as b
    return b.GpFp8Matrix(data, scales, ld, row, col, fmt, group)


def gemm(gp, A=None, B=None, C=PTR, ldc=64, add=None, ld_add=64, M=64, N=64, K=256, out=1, opts=None):
    return gp.lib().gemm_fp8(A or matrix(), B or matrix(), C, ldc, add, ld_add, M, N, K, out, None, opts)


@pytest.mark.parametrize("args,code", [
    (dict(M=-1), "ARG"), (dict(K=-1), "ARG"), (dict(N=1 << 31), "SIZE"), (dict(K=1 << 31), "SIZE"), (dict(M=(1 << 31) - 200), "SIZE"),
    (dict(out=3), "ARG"), (dict(C=None), "ARG"), (dict(ldc=63), "ARG"), (dict(add=PTR, ld_add=63), "ARG"),
    (dict(A=matrix(data=None)), "ARG"), (dict(B=matrix(scales=None)), "ARG"), (dict(A=matrix(fmt=2)), "ARG"),
    (dict(B=matrix(group=64)), "ARG"), (dict(A=matrix(ld=240)), "ARG"), (dict(A=matrix(ld=260)), "UNSUPPORTED"),
    (dict(B=matrix(data=PTR + 8)), "UNSUPPORTED"), (dict(B=matrix(scales=PTR + 2)), "UNSUPPORTED"),
    (dict(C=PTR + 1), "UNSUPPORTED"), (dict(C=PTR + 2, out=2), "UNSUPPORTED"),
    (dict(add=PTR + 1), "UNSUPPORTED"),
])
def test_gemm_argument_errors_need_no_device(gp, args, code):
    assert gemm(gp, **args) == getattr(gp, "GP_ERR_" + code)
    assert gp.gemm_stats(sync=False)["status"] == getattr(gp, "GP_ERR_" + code)


def test_gemm_null_matrix_and_forced_width(gp):
    from software_pipelined_tiled_pipeline_gb300 import _binding as b
    f = gp.lib().gemm_fp8
    assert f(None, matrix(), PTR, 64, None, 0, 64, 64, 256, 1, None, None) == gp.GP_ERR_ARG
    assert gemm(gp, opts=b.GpFp8Options(0, 48, 0, 0)) == gp.GP_ERR_UNSUPPORTED
    assert gemm(gp, opts=b.GpFp8Options(0, 256, 0, 1)) == gp.GP_ERR_UNSUPPORTED     # two CTAs share a tile


def test_empty_output_needs_no_device(gp):
    f = gp.lib().gemm_fp8
    assert f(None, None, None, 0, None, 0, 0, 64, 256, 1, None, None) == gp.GP_OK
    assert f(None, None, None, 0, None, 0, 64, 0, 256, 1, None, None) == gp.GP_OK
    assert gp.lib().fp8_quantize(None, 0, 0, 128, 0, matrix(), None, None) == gp.GP_OK
    assert gp.lib().fp8_rmsnorm(None, 0, None, 0, None, 0, 0.0, 0, 64, 0, None, 0, None, None, 0, None, None) == gp.GP_OK
    assert gp.lib().fp8_rmsnorm_backward(None, 0, None, 0, None, 0, None, 0, None, 0, 64, 0, None, 0, None, None, 0, None) == gp.GP_OK


def quantize(gp, x=PTR, ldx=256, rows=64, cols=256, type=1, q=None, qt=None):
    return gp.lib().fp8_quantize(x, ldx, rows, cols, type, q, qt, None)


@pytest.mark.parametrize("args,code", [
    (dict(), "ARG"),                                             # neither q nor qt
    (dict(q=matrix(), rows=-1), "ARG"), (dict(q=matrix(), cols=1 << 31), "SIZE"), (dict(q=matrix(), type=3), "ARG"),
    (dict(q=matrix(), x=None), "ARG"), (dict(q=matrix(), ldx=255), "ARG"), (dict(q=matrix(), x=PTR + 1), "UNSUPPORTED"),
    (dict(q=matrix(ld=240)), "ARG"), (dict(qt=matrix(ld=48)), "ARG"), (dict(qt=matrix(ld=72)), "UNSUPPORTED"),
    (dict(q=matrix(data=None)), "ARG"), (dict(q=matrix(), qt=matrix(fmt=1)), "ARG"),
    (dict(q=matrix(), qt=matrix(group=128)), "ARG"), (dict(q=matrix(group=2)), "ARG"),
])
def test_quantize_argument_errors_need_no_device(gp, args, code):
    assert quantize(gp, **args) == getattr(gp, "GP_ERR_" + code)


def norm(gp, x=PTR, ldx=256, res=None, ld_res=256, w=PTR, wtype=1, eps=1e-6, rows=4, cols=256, type=1, h=None, ld_h=256,
         rstd=PTR, y=None, ld_y=256, q=None):
    return gp.lib().fp8_rmsnorm(x, ldx, res, ld_res, w, wtype, eps, rows, cols, type, h, ld_h, rstd, y, ld_y, q, None)


@pytest.mark.parametrize("args,code", [
    (dict(x=None), "ARG"), (dict(w=None), "ARG"), (dict(type=5), "ARG"), (dict(wtype=-1), "ARG"), (dict(eps=-1.0), "ARG"),
    (dict(eps=float("nan")), "ARG"), (dict(rows=-1), "ARG"), (dict(cols=1 << 31), "SIZE"), (dict(cols=(1 << 30) + 1), "SIZE"), (dict(ldx=255), "ARG"),
    (dict(res=PTR, ld_res=255), "ARG"), (dict(h=PTR, ld_h=4), "ARG"), (dict(y=PTR, ld_y=4), "ARG"),
    (dict(h=PTR + 1), "UNSUPPORTED"), (dict(rstd=PTR + 2), "UNSUPPORTED"), (dict(q=matrix(group=128)), "ARG"),
    (dict(q=matrix(ld=248)), "ARG"), (dict(q=matrix(data=PTR + 4)), "UNSUPPORTED"),
])
def test_norm_argument_errors_need_no_device(gp, args, code):
    assert norm(gp, **args) == getattr(gp, "GP_ERR_" + code)


def backward(gp, dy=PTR, ld_dy=256, h=PTR, ld_h=256, dres=None, ld_dres=256, w=PTR, wtype=1, rstd=PTR, rows=4, cols=256,
             type=1, dx=PTR, ld_dx=256, dw=PTR, work=PTR, work_bytes=1 << 30):
    return gp.lib().fp8_rmsnorm_backward(dy, ld_dy, h, ld_h, dres, ld_dres, w, wtype, rstd, rows, cols, type, dx, ld_dx, dw,
                                         work, work_bytes, None)


@pytest.mark.parametrize("args,code", [
    (dict(dy=None), "ARG"), (dict(h=None), "ARG"), (dict(w=None), "ARG"), (dict(rstd=None), "ARG"), (dict(dx=None), "ARG"),
    (dict(ld_dy=8), "ARG"), (dict(ld_h=8), "ARG"), (dict(dres=PTR, ld_dres=8), "ARG"), (dict(ld_dx=8), "ARG"),
    (dict(type=4), "ARG"), (dict(wtype=4), "ARG"), (dict(rows=1 << 31), "SIZE"), (dict(dw=PTR + 1), "UNSUPPORTED"),
    (dict(dx=PTR + 1), "UNSUPPORTED"), (dict(work=None, rows=4000), "ARG"), (dict(work=PTR + 4), "UNSUPPORTED"),
])
def test_backward_argument_errors_need_no_device(gp, args, code):
    assert backward(gp, **args) == getattr(gp, "GP_ERR_" + code)


def test_backward_workspace(gp):
    size = ctypes.c_int64(-1)
    f = gp.lib().fp8_rmsnorm_backward_workspace
    for rows, cols in [(0, 64), (64, 0), (1, 1), (200, 2056)]:      # (few rows need none)
        assert f(rows, cols, 152, size) == gp.GP_OK and size.value == 0
    for rows, cols in [(5000, 1), (2000, 2056), (8192, 8192), (5, 20000), (4000, 20000)]:
        assert f(rows, cols, 152, size) == gp.GP_OK
        # whole rows of FP32 sums: never more than a block for each row, each with at most four rows side by side
        assert size.value % (4 * cols) == 0 and 1 <= size.value // (4 * cols) <= 4 * rows
    assert f(-1, 4, 152, size) == gp.GP_ERR_ARG and f(4, 4, -1, size) == gp.GP_ERR_ARG
    assert f(4, 4, 152, None) == gp.GP_ERR_ARG and f(4, (1 << 30) + 1, 152, size) == gp.GP_ERR_SIZE


def test_struct_layout_matches_the_header(tmp_path):
    from software_pipelined_tiled_pipeline_gb300 import _binding as b
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    checks = [("gp_fp8_matrix", b.GpFp8Matrix), ("gp_fp8_options", b.GpFp8Options)]
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "gemm_fp8.h"', "int main(void) {"]
    for cname, cls in checks:
        lines.append('  printf("%zu\\n", sizeof(' + cname + '));')
        lines += ['  printf("%%zu\\n", offsetof(%s, %s));' % (cname, f) for f, _ in cls._fields_]
    (tmp_path / "s.c").write_text("\n".join(lines + ["  return 0;\n}"]))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "s.c"), "-o", str(tmp_path / "s")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for _, cls in checks:
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def test_plan_errors(gp):
    from software_pipelined_tiled_pipeline_gb300 import _binding as b
    f, p = gp.lib().gemm_fp8_plan, b.GpPlan()
    assert f(64, 64, 64, 1, 128, 152, None, None) == gp.GP_ERR_ARG
    assert f(64, 64, 64, 2, 128, 152, None, p) == gp.GP_ERR_ARG
    assert f(64, 64, 64, 1, 128, -1, None, p) == gp.GP_ERR_ARG
    assert f(-1, 64, 64, 1, 128, 152, None, p) == gp.GP_ERR_ARG
    assert f(64, 1 << 31, 64, 1, 128, 152, None, p) == gp.GP_ERR_SIZE
    assert f((1 << 31) - 1, (1 << 31) - 1, 64, 1, 128, 152, None, p) == gp.GP_ERR_SIZE


@pytest.mark.parametrize("M,N,swapped", [(1, 4096, 1), (17, 4096, 1), (4096, 1, 0), (4096, 30, 0), (48, 8192, 1)])
def test_the_narrow_operand_takes_the_n_side(gp, M, N, swapped):
    p = gp.gemm_fp8_plan(M, N, 4096, sms=152)
    assert p["layout"] == swapped
    assert p["bn"] >= min(M, N) and p["dtype"] == 16


def test_plan_invariants_over_many_shapes(gp):
    rng = np.random.default_rng(5)
    for _ in range(400):
        M, N, K = (int(np.exp(rng.uniform(0, np.log(9000)))) for _ in range(3))
        a, b = rng.choice(["rows", "blocks"], 2)
        p = gp.gemm_fp8_plan(M, N, K, a, b, sms=152)
        P, Q = (N, M) if p["layout"] else (M, N)
        assert p["k_tiles"] == -(-K // 128)
        assert p["tiles"] == -(-P // p["bm"]) * -(-Q // p["bn"])
        assert 1 <= p["grid"] <= 152 and p["grid"] % p["k_splits"] == 0
        assert p["k_splits"] == 1 or p["tiles"] * p["k_splits"] == p["grid"]
        assert p["smem_bytes"] <= 232448 and p["tmem_cols"] <= 512
        assert p["stages"] >= 2
        assert p["dp_tiles"] + p["sk_tiles"] == p["tiles"]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_plain_formats_agree_with_torch(fmt):
    # every code's value, and the nearest code of values all over the range (finite ones: torch does not saturate)
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(ref.TORCH[fmt])
    np.testing.assert_array_equal(every.float().numpy().astype(np.float64), ref.TABLE[fmt])
    rng = np.random.default_rng(1)
    x = (rng.standard_normal(20000) * np.exp2(rng.uniform(-20, 8 if fmt == "e4m3" else 15, 20000))).astype(np.float32)
    x = x[np.abs(x) <= ref.FMAX[fmt]]
    pos = ref.TABLE[fmt][:128]
    pos = pos[np.isfinite(pos)]
    mid = ((pos[1:] + pos[:-1]) / 2).astype(np.float32)
    x = np.concatenate([x, mid, -mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9))])
    x = x[np.abs(x) <= ref.FMAX[fmt]]
    want = torch.from_numpy(x).to(ref.TORCH[fmt]).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(x, fmt), want)


def test_few_tiles_share_their_k_loops_in_clusters(gp):
    # as many CTAs per tile as keep all clusters resident, at least four K blocks each
    for M, N, K, tiles, splits in ((9, 4096, 4096, 32, 4), (9, 8192, 8192, 64, 2), (9, 2048, 8192, 16, 8),
                                   (9, 152 * 128, 4096, 152, 1)):
        p = gp.gemm_fp8_plan(M, N, K, sms=152)
        assert (p["tiles"], p["k_splits"], p["grid"]) == (tiles, splits, tiles * splits), (M, N, K, p)
        assert p["workspace_bytes"] == 0 and p["sk_tiles"] == 0
    assert gp.gemm_fp8_plan(9, 4096, 4096, sms=152, no_split=True)["k_splits"] == 1
    # pairs run whole tiles
    p = gp.gemm_fp8_plan(4096, 4096, 4096, sms=152)
    assert (p["cta_pair"], p["bm"], p["bn"], p["k_splits"], p["grid"]) == (1, 256, 256, 1, 152)


def test_plan_of_few_sms(gp):
    # a plan that no SM count allows is refused: tiles of 256 take pairs of CTAs, so two SMs
    from software_pipelined_tiled_pipeline_gb300 import _binding as b
    p = b.GpPlan()
    for sms in (1, 2, 3, 5, 8):
        for bn in (0, 16, 32, 64, 128, 256):
            for M, N, K in ((64, 64, 64), (1, 4096, 4096), (512, 512, 512), (5000, 3000, 700)):
                for groups in ((1, 128), (1, 1), (128, 1)):
                    rc = gp.lib().gemm_fp8_plan(M, N, K, *groups, sms, b.GpFp8Options(0, bn, 0, 0), p)
                    if sms == 1 and bn == 256:
                        assert rc == gp.GP_ERR_UNSUPPORTED
                        continue
                    assert rc == gp.GP_OK
                    d = p.as_dict()
                    assert 1 <= d["grid"] <= sms and d["grid"] % (2 if d["cta_pair"] else d["k_splits"]) == 0
                    assert bn in (0, d["bn"])


PTXAS = """ptxas info    : Compiling entry function '_ZN2gp15fp8_ring_kernelILi256ELb0ELb1ELb0EEEv' for 'sm_103a'
ptxas info    : Function properties for _ZN2gp15fp8_ring_kernelILi256ELb0ELb1ELb0EEEv
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 2 barriers
ptxas info    : Compiling entry function '_ZN2gp15fp8_ring_kernelILi16ELb1ELb0ELb0EEEv' for 'sm_103a'
ptxas info    : Used 122 registers, used 2 barriers
"""


def test_build_refuses_a_register_split_that_cannot_launch():
    # the wide kernels' warps trade registers; with others than 168 at launch every call would be refused
    gbuild.check_launch_registers("k_fp8_gemm.cu", PTXAS % 168)
    gbuild.check_launch_registers("k_fp8_quant.cu", "")              # (no such kernel there)
    for wrong in (160, 128):
        with pytest.raises(RuntimeError, match="compiled to %d registers" % wrong):
            gbuild.check_launch_registers("k_fp8_gemm.cu", PTXAS % wrong)
    with pytest.raises(RuntimeError):
        gbuild.check_launch_registers("k_umma.cu", PTXAS % 128)      # its kernel is missing from the output
    for src, constant, threads in (("k_fp8_gemm.cu", r"kLaunchRegs = (\d+);", None),
                                   ("k_umma.cu", r"kOvLaunchRegs = 65536 / kOvThreads;", r"kOvThreads = (\d+);")):
        text = open(os.path.join(gbuild.CSRC, src)).read()
        found = re.search(constant, text)
        regs = int(found.group(1)) if threads is None else 65536 // int(re.search(threads, text).group(1))
        assert regs == gbuild.LAUNCH_REGISTERS[src][1]


@pytest.mark.parametrize("kinds", [("columns", "blocks"), ("rows", "tiles"), (128, "rows")])
def test_plan_refuses_unknown_scales(gp, kinds):
    with pytest.raises(ValueError):
        gp.gemm_fp8_plan(64, 64, 64, *kinds)
