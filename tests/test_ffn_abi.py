"""Host-side checks of the feed-forward operators (no GPU): argument errors are
reported before anything is launched, struct layouts match the header, the plan
follows its rules, and the Python calls refuse what they cannot take."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import ffn_ref
from software_pipelined_tiled_pipeline_gb300 import _binding as b
from software_pipelined_tiled_pipeline_gb300 import build as gbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 0x10000
STRUCTS = {"gp_linear": b.GpLinear, "gp_gated": b.GpGated, "gp_input_grad": b.GpInputGrad, "gp_weight_grad": b.GpWeightGrad,
           "gp_act_backward": b.GpActBackward, "gp_gated_backward": b.GpGatedBackward, "gp_ffn_options": b.GpFfnOptions}


@pytest.fixture(scope="module")
def gp():
    gbuild.build()
    import software_pipelined_tiled_pipeline_gb300 as mod
    mod.lib()
    return mod


def codes(data=PTR, scales=PTR, ld=256, row=1, col=64, fmt=0, group=1):
    return b.GpFp8Matrix(data, scales, ld, row, col, fmt, group)


def fill(struct, **values):
    s = struct()
    for k, v in values.items():
        if isinstance(v, tuple):
            setattr(s, k, type(getattr(s, k))(*v))
        else:
            setattr(s, k, v)
    return s


def linear(gp, opts=None, **over):
    return gp.lib().gemm_linear(fill(b.GpLinear, **dict(dict(x=PTR, weight=PTR, y=PTR, M=64, N=200, K=256, ldx=256, ldw=256,
                                                             ldy=200, ld_res=200, ldz=200, type=1, out_type=1, bias_type=1),
                                                        **over)), None, opts)


def gated(gp, opts=None, **over):
    return gp.lib().gemm_gated(fill(b.GpGated, **dict(dict(x=PTR, gate=PTR, up=PTR, h=PTR, M=64, N=200, K=256, ldx=256, ld_gate=256,
                                                           ld_up=256, ldh=200, ld_zg=200, ld_zu=200, type=1, activation=4),
                                                      **over)), None, opts)


def input_grad(gp, opts=None, **over):
    return gp.lib().gemm_input_grad(fill(b.GpInputGrad, **dict(dict(dz=(PTR, PTR), weight=(PTR, PTR), dx=PTR, M=64, N=200, K=256,
                                                                    ld_dz=(200, 200), ldw=(256, 256), ld_dx=256, type=1, out_type=1,
                                                                    count=2), **over)), None, opts)


def weight_grad(gp, opts=None, **over):
    return gp.lib().gemm_weight_grad(fill(b.GpWeightGrad, **dict(dict(dz=(PTR, PTR), x=PTR, dw=(PTR, 2 * PTR), M=64, N=200, K=256,
                                                                      ld_dz=(200, 200), ldx=256, ld_add=(256, 256), ld_dw=(256, 256),
                                                                      type=1, out_type=2, count=2), **over)), None, opts)


def act_backward(gp, **over):
    return gp.lib().ffn_act_backward(fill(b.GpActBackward, **dict(dict(dy=PTR, z=PTR, dz=PTR, dbias=PTR, workspace=PTR,
                                                                       workspace_bytes=1 << 30, M=64, N=200, ld_dy=200, ldz=200,
                                                                       ld_dz=200, type=1, activation=2), **over)), None)


def gated_backward(gp, **over):
    return gp.lib().ffn_gated_backward(fill(b.GpGatedBackward, **dict(dict(dh=PTR, z_gate=PTR, z_up=PTR, dgate=PTR, dup=2 * PTR, h=PTR,
                                                                           M=64, N=200, ld_dh=200, ld_zg=200, ld_zu=200,
                                                                           ld_dgate=200, ld_dup=200, ldh=200, type=1, activation=4),
                                                                      **over)), None)


BIG = (1 << 31) - 200


@pytest.mark.parametrize("call,args,code", [
    (linear, dict(M=-1), "ARG"), (linear, dict(K=BIG), "SIZE"), (linear, dict(N=1 << 32), "SIZE"), (linear, dict(type=2), "ARG"),
    (linear, dict(out_type=0), "ARG"), (linear, dict(activation=6), "ARG"), (linear, dict(x=None), "ARG"),
    (linear, dict(weight=None), "ARG"), (linear, dict(y=None), "ARG"), (linear, dict(ldx=255), "ARG"), (linear, dict(ldw=8), "ARG"),
    (linear, dict(ldy=199), "ARG"), (linear, dict(residual=PTR, ld_res=199), "ARG"), (linear, dict(z=PTR, ldz=100), "ARG"),
    (linear, dict(bias=PTR, bias_type=0), "ARG"), (linear, dict(bias=PTR + 1), "UNSUPPORTED"),
    (linear, dict(bias=PTR + 2, bias_type=2), "UNSUPPORTED"), (linear, dict(x=PTR + 8), "UNSUPPORTED"),
    (linear, dict(weight=PTR + 2), "UNSUPPORTED"), (linear, dict(ldx=257), "UNSUPPORTED"), (linear, dict(ldw=260), "UNSUPPORTED"),
    (linear, dict(y=PTR + 1), "UNSUPPORTED"), (linear, dict(out_type=2, y=PTR + 2), "UNSUPPORTED"),
    (linear, dict(residual=PTR + 1), "UNSUPPORTED"), (linear, dict(q=codes(ld=192)), "ARG"), (linear, dict(q=codes(fmt=1)), "ARG"),
    (linear, dict(q=codes(group=128)), "ARG"), (linear, dict(q=codes(scales=None)), "ARG"), (linear, dict(q=codes(ld=216)), "UNSUPPORTED"),
    (linear, dict(q=codes(data=PTR + 8)), "UNSUPPORTED"), (linear, dict(q=codes(), z=PTR), "ARG"),
    (gated, dict(M=-1), "ARG"), (gated, dict(N=BIG), "SIZE"), (gated, dict(type=2), "ARG"), (gated, dict(activation=-1), "ARG"),
    (gated, dict(up=None), "ARG"), (gated, dict(gate=PTR + 4), "UNSUPPORTED"), (gated, dict(ld_up=252), "ARG"),
    (gated, dict(ld_gate=268), "UNSUPPORTED"), (gated, dict(h=None), "ARG"), (gated, dict(z_gate=PTR), "ARG"),
    (gated, dict(z_gate=PTR, z_up=PTR, ld_zu=10), "ARG"), (gated, dict(q_gate=codes()), "ARG"),
    (gated, dict(q_gate=codes(), q_up=codes(ld=64)), "ARG"), (gated, dict(q_gate=codes(), q_up=codes(), z_gate=PTR, z_up=PTR), "ARG"),
    (input_grad, dict(count=0), "ARG"), (input_grad, dict(count=3), "ARG"), (input_grad, dict(dz=(PTR, None)), "ARG"),
    (input_grad, dict(weight=(PTR, PTR + 2)), "UNSUPPORTED"), (input_grad, dict(ld_dz=(200, 204)), "UNSUPPORTED"),
    (input_grad, dict(ldw=(248, 256)), "ARG"), (input_grad, dict(dx=None), "ARG"), (input_grad, dict(ld_dx=255), "ARG"),
    (input_grad, dict(out_type=0), "ARG"), (input_grad, dict(M=-4), "ARG"),
    (weight_grad, dict(x=None), "ARG"), (weight_grad, dict(dw=(PTR, None)), "ARG"), (weight_grad, dict(addend=(PTR, None)), "ARG"),
    (weight_grad, dict(addend=(PTR, PTR + 2)), "UNSUPPORTED"), (weight_grad, dict(ld_add=(8, 256), addend=(PTR, PTR)), "ARG"),
    (weight_grad, dict(dz=(PTR + 8, PTR)), "UNSUPPORTED"), (weight_grad, dict(ldx=250), "ARG"), (weight_grad, dict(type=3), "ARG"),
    (act_backward, dict(dy=None), "ARG"), (act_backward, dict(z=None), "ARG"), (act_backward, dict(q=codes()), "ARG"),
    (act_backward, dict(z=None, q=codes(ld=64)), "ARG"), (act_backward, dict(ld_dy=100), "ARG"), (act_backward, dict(ld_dz=100), "ARG"),
    (act_backward, dict(workspace=PTR + 4), "UNSUPPORTED"), (act_backward, dict(dbias=PTR + 2), "UNSUPPORTED"),
    (act_backward, dict(type=2), "ARG"), (act_backward, dict(activation=9), "ARG"), (act_backward, dict(N=BIG), "SIZE"),
    (gated_backward, dict(z_up=None), "ARG"), (gated_backward, dict(q_gate=codes(), q_up=codes()), "ARG"),
    (gated_backward, dict(z_gate=None, z_up=None), "ARG"), (gated_backward, dict(dgate=None), "ARG"),
    (gated_backward, dict(z_gate=None, z_up=None, q_gate=codes(), q_up=codes(fmt=1)), "ARG"), (gated_backward, dict(ldh=1), "ARG"),
    (weight_grad, dict(dw=(PTR, PTR)), "ARG"), (gated_backward, dict(dup=PTR), "ARG"), (gated, dict(z_gate=PTR, z_up=PTR), "ARG"),
    (gated_backward, dict(dup=PTR + 1), "UNSUPPORTED"), (gated_backward, dict(M=-1), "ARG"),
])
def test_argument_errors_need_no_device(gp, call, args, code):
    assert call(gp, **args) == getattr(gp, "GP_ERR_" + code)
    assert gp.gemm_stats(sync=False)["status"] == getattr(gp, "GP_ERR_" + code)


def test_null_arguments(gp):
    L = gp.lib()
    for f in (L.gemm_linear, L.gemm_gated, L.gemm_input_grad, L.gemm_weight_grad):
        assert f(None, None, None) == gp.GP_ERR_ARG
    assert L.ffn_act_backward(None, None) == gp.GP_ERR_ARG and L.ffn_gated_backward(None, None) == gp.GP_ERR_ARG


def test_forced_tiles(gp):
    def opts(tile, lose=0, splits=0):
        return b.GpFfnOptions(0, tile, splits, lose)
    assert linear(gp, opts(32, splits=3)) == gp.GP_ERR_UNSUPPORTED and linear(gp, opts(16, splits=8)) == gp.GP_ERR_UNSUPPORTED
    assert linear(gp, opts(48)) == gp.GP_ERR_UNSUPPORTED and linear(gp, opts(256, 1)) == gp.GP_ERR_UNSUPPORTED
    assert linear(gp, opts(16), q=codes()) == gp.GP_ERR_UNSUPPORTED
    assert gated(gp, opts(128), q_gate=codes(), q_up=codes()) == gp.GP_ERR_UNSUPPORTED
    assert gated(gp, opts(0, 1), q_gate=codes(), q_up=codes()) == gp.GP_ERR_UNSUPPORTED
    assert weight_grad(gp, opts(32)) == gp.GP_ERR_UNSUPPORTED and weight_grad(gp, opts(16)) == gp.GP_ERR_UNSUPPORTED
    assert input_grad(gp, opts(96)) == gp.GP_ERR_UNSUPPORTED


def test_empty_outputs_need_no_device(gp):
    for over in (dict(M=0), dict(N=0)):
        assert linear(gp, x=None, y=None, **over) == gp.GP_OK and gated(gp, x=None, h=None, **over) == gp.GP_OK
    assert input_grad(gp, M=0, dx=None) == gp.GP_OK and input_grad(gp, K=0, dx=None) == gp.GP_OK
    assert weight_grad(gp, N=0, x=None) == gp.GP_OK and weight_grad(gp, K=0, x=None) == gp.GP_OK
    assert act_backward(gp, N=0, dy=None) == gp.GP_OK and act_backward(gp, M=0, dbias=None) == gp.GP_OK
    assert gated_backward(gp, M=0, dh=None, z_up=None) == gp.GP_OK
    assert gp.lib().ffn_pack_rows(None, 0, None, 0, 0, 5, None) == gp.GP_OK


def test_pack_refusals(gp):
    f = gp.lib().ffn_pack_rows
    assert f(None, 5, PTR, 8, 4, 5, None) == gp.GP_ERR_ARG and f(PTR, 4, PTR, 8, 4, 5, None) == gp.GP_ERR_ARG
    assert f(PTR, 5, PTR, 12, 4, 5, None) == gp.GP_ERR_UNSUPPORTED and f(PTR, 5, PTR + 8, 8, 4, 5, None) == gp.GP_ERR_UNSUPPORTED
    assert f(PTR + 1, 5, PTR, 8, 4, 5, None) == gp.GP_ERR_UNSUPPORTED and f(PTR, 5, PTR, 8, -1, 5, None) == gp.GP_ERR_ARG


def test_bias_workspace(gp):
    size = ctypes.c_int64(-1)
    f = gp.lib().ffn_act_backward_workspace
    for M, N in [(0, 64), (64, 0), (1, 1), (16, 5000), (200, 2056), (128, 100)]:       # what a cluster adds up needs none
        assert f(M, N, 152, size) == gp.GP_OK and size.value == 0
    for M, N in [(1000, 1), (8192, 1000), (4096, 100)]:
        assert f(M, N, 152, size) == gp.GP_OK
        parts, left = divmod(size.value, 4 * N)
        assert left == 0 and 2 <= parts <= (M + 127) // 128        # eight parts of two rows for each warp at least
    assert f(-1, 4, 152, size) == gp.GP_ERR_ARG and f(4, 4, -1, size) == gp.GP_ERR_ARG and f(4, 4, 152, None) == gp.GP_ERR_ARG


def test_struct_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "gemm_ffn.h"', "int main(void) {"]
    want = []
    for name, cls in STRUCTS.items():
        lines.append('printf("%%zu\\n", sizeof(%s));' % name)
        want.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            lines.append('printf("%%zu\\n", offsetof(%s, %s));' % (name, field))
            want.append(getattr(cls, field).offset)
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = str(tmp_path / "layout")
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out] == want


def test_header_constants():
    text = open(os.path.join(ROOT, "include", "gemm_ffn.h")).read()
    for name, value in b.ACTIVATIONS.items():
        assert int(re.search(r"GP_ACT_%s = (\d+)" % name.upper(), text).group(1)) == value
    assert int(re.search(r"GP_PLAN_FFN (\d+)", text).group(1)) == b.GP_PLAN_FFN


@pytest.mark.parametrize("op", ["linear", "gated", "input_grad", "weight_grad"])
def test_plan_invariants(gp, op):
    rng = np.random.default_rng(5)
    for _ in range(300):
        M, N, K = (int(2 ** rng.uniform(0, 14)) for _ in range(3))
        kept, count = bool(rng.integers(2)), int(rng.integers(1, 3))
        sms = int(rng.choice([1, 2, 100, 152]))
        if op == "gated" and kept and sms == 1:
            with pytest.raises(gp.GemmError):
                gp.ffn_plan(op, M, N, K, count=count, kept=kept, sms=sms)
            continue
        p = gp.ffn_plan(op, M, N, K, count=count, kept=kept, sms=sms)
        rows, cols = (N, K) if op == "weight_grad" else (M, K if op == "input_grad" else N)
        if p["layout"]:
            assert not kept or op in ("input_grad", "weight_grad")
            assert p["tiles"] == -(-cols // p["bm"]) * -(-rows // p["bn"]) * (count if op == "weight_grad" else 1)
            assert p["grid"] == p["tiles"] * p["k_splits"] and (p["bn"] >= 64 or op != "weight_grad")
            assert p["k_splits"] == 1 or (p["grid"] <= sms and p["k_tiles"] >= 4 * p["k_splits"])
        else:
            assert p["tiles"] == -(-rows // p["bm"]) * -(-cols // p["bn"]) * (count if op == "weight_grad" else 1)
            assert p["k_splits"] == 1 and 1 <= p["grid"] <= sms and p["grid"] % (2 if p["cta_pair"] else 1) == 0
        assert p["smem_bytes"] <= 232448 and p["ring_bytes"] == p["stages"] * p["stage_bytes"] and p["tmem_cols"] <= 512


def test_plan_refusals(gp):
    p = b.GpPlan()
    f = gp.lib().gemm_ffn_plan
    assert f(4, 8, 8, 8, 1, 0, 0, None, p) == gp.GP_ERR_ARG and f(0, 8, 8, 8, 3, 0, 0, None, p) == gp.GP_ERR_ARG
    assert f(0, 8, 8, 8, 1, 0, 0, None, None) == gp.GP_ERR_ARG and f(0, -8, 8, 8, 1, 0, 0, None, p) == gp.GP_ERR_ARG
    assert f(0, 0, 8, 8, 1, 0, 0, None, p) == gp.GP_ERR_ARG and f(0, BIG, 8, 8, 1, 0, 0, None, p) == gp.GP_ERR_SIZE
    assert f(0, BIG - 256, BIG - 256, 8, 1, 0, 0, None, p) == gp.GP_ERR_SIZE


def test_python_refusals_need_no_device(gp):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: gp.linear(x, x), lambda: gp.gated(x, x, x), lambda: gp.linear_backward(x, x, x),
                 lambda: gp.gated_backward(x, x, x, x, (x, x))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


@pytest.mark.parametrize("act", ffn_ref.ACTS)
def test_the_plain_slopes_are_the_values_differences(act):
    z = np.array([-9.0, -3.3, -1.0, -0.2, 0.3, 1.0, 2.7, 8.0])
    h = 1e-5
    d = (ffn_ref.value(z + h, act) - ffn_ref.value(z - h, act)) / (2 * h)
    # the third derivative (below 4) times h^2 / 6, and the values' rounding (2^-53 of 9) over h
    assert np.allclose(d, ffn_ref.slope(z, act), rtol=0, atol=4 * h * h / 6 + 9 * 2.0 ** -53 / h)


def test_plan_tells_codes_from_wide_outputs(gp):
    """FP32 outputs go to the cluster kernels too, values kept in 8 bits do not; long sums into 16 bits are held, by type."""
    f32, f16, bf16 = torch.float32, torch.float16, torch.bfloat16
    for M in (1, 40, 100):
        kernels = [gp.ffn_plan("linear", M, 4096, 4096, sms=152, out_dtype=t)["kernel"] for t in (None, f32)]
        assert kernels == ["ffn_few", "ffn_few"]
        assert gp.ffn_plan("linear", M, 4096, 4096, sms=152, kept=True)["kernel"] == "ffn_ring"
        assert gp.ffn_plan("linear", M, 4096, 4096, sms=152, kept=True, out_dtype=f32)["kernel"] == "ffn_ring"
    assert gp.ffn_plan("linear", 1, 4096, 4096, sms=152, out_dtype=f32, tile=16)["bn"] == 16
    with pytest.raises(gp.GemmError):
        gp.ffn_plan("linear", 1, 4096, 4096, sms=152, kept=True, tile=16)
    for dtype, longest in ((f16, 4096), (bf16, 32768)):
        for tile in (128, 256):
            threads = [gp.ffn_plan("linear", 4096, 4096, K, sms=152, dtype=dtype, tile=tile)["threads"] for K in (longest, longest + 1)]
            held = gp.ffn_plan("linear", 4096, 4096, 64, sms=152, out_dtype=f32, dtype=dtype, tile=tile)["threads"]
            assert threads[1] == held and (tile == 128 or threads[0] < held)
    # both products of a pair's input gradient are one sum
    one, two = (gp.ffn_plan("input_grad", 4096, 4096, 4096, sms=152, dtype=f16, count=c, tile=256)["threads"] for c in (1, 2))
    assert one == 384 and two == 640
    p = b.GpPlan()
    for op, kept in ((0, -1), (0, 8), (1, 2), (1, 3)):
        assert gp.lib().gemm_ffn_plan(op, 8, 8, 8, 1, kept, 0, None, p) == gp.GP_ERR_ARG
    for bad in (dict(dtype=f32), dict(out_dtype=f16), dict(dtype=f16, out_dtype=bf16)):
        with pytest.raises(ValueError):
            gp.ffn_plan("linear", 8, 8, 8, **bad)


@pytest.mark.parametrize("op", ["linear", "gated", "input_grad", "weight_grad"])
def test_the_planner_chooses_a_tile_that_takes_the_forced_split(gp, op):
    for M in (1, 5, 16, 17, 64):
        for splits in (1, 2, 4, 8):
            p = gp.ffn_plan(op, M, 4096, 4096, sms=152, k_splits=splits)
            assert p["k_splits"] == (splits if p["layout"] else 1)
            assert op == "weight_grad" or p["layout"] == 1        # (few rows go to clusters)
            assert p["bn"] != 16 or splits <= 4
