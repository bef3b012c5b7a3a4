"""libnvfp4_ffn.so on the CPU: it exports what include/nvfp4_ffn.h declares, sizes its buffers, says how it computes a
product, and refuses what the header rules out before any HIP call (no GPU needed: every call here returns before one).
The oracle of the GPU tests is pinned here as well, and its gradients are checked against differences."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import moe_matmul_amd as mm
import oracle.ffn_oracle as FO
from ffn_cases import LINEAR, PRODUCT_KINDS, GATED, parts_of
from moe_matmul_amd import _ffn_binding as c
from moe_matmul_amd import ffn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # an address that no refused call reads
INVALID, MISALIGNED, WORKSPACE = mm.NVFP4_ERR_INVALID, mm.NVFP4_ERR_MISALIGNED, mm.NVFP4_ERR_WORKSPACE
F32, F16, BF16 = 0, 1, 2


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "nvfp4_ffn.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(nvfp4_ffn_\w+)\s*\(", text)))
    lib = c.load_ffn_library()
    assert "nvfp4_ffn_gated" in names and names == sorted(c._SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", c.FFN_LIB_PATH], capture_output=True, text=True).stdout
    assert sorted(set(re.findall(r"\bT (nvfp4_\w+)", out))) == names
    assert all(hasattr(lib, n) for n in names)


def refused(code, call, *args):
    with pytest.raises(c.Nvfp4FfnError) as e:
        call(*args)
    assert e.value.code == code


def with_(call, names, base, code, **changes):
    """call with base's values but for the changes is refused with that code."""
    refused(code, call, *[{**base, **changes}[n] for n in names.split()])


def plan_of(experts=4, topk=2, offsets=P, row_slots=P):
    return ctypes.byref(c.nvfp4_ffn_plan(experts, topk, offsets, row_slots))


NORM = "x dtype rows n x_stride residual residual_stride weight weight_f32 eps sum y codes scales rstd stream"
NORM_OK = dict(x=P, dtype=BF16, rows=4, n=64, x_stride=64, residual=P, residual_stride=64, weight=P, weight_f32=1,
               eps=1e-6, sum=P, y=P, codes=P, scales=P, rstd=P, stream=0)


@pytest.mark.parametrize("code,bad", [
    (INVALID, dict(dtype=3)), (INVALID, dict(dtype=-1)), (INVALID, dict(rows=-1)), (INVALID, dict(rows=1 << 31)),
    (INVALID, dict(n=0)), (INVALID, dict(n=65537)), (INVALID, dict(n=48, x_stride=48, residual_stride=48)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=math.nan)), (INVALID, dict(scales=0)), (INVALID, dict(codes=0)),
    (INVALID, dict(y=0, codes=0, scales=0, rstd=0)), (INVALID, dict(x=0)), (INVALID, dict(x_stride=63)),
    (INVALID, dict(residual_stride=63)), (INVALID, dict(sum=0)), (MISALIGNED, dict(x=P + 1)),
    (MISALIGNED, dict(weight=P + 2)), (MISALIGNED, dict(codes=P + 4)), (MISALIGNED, dict(rstd=P + 2)),
    (MISALIGNED, dict(sum=P + 1)), (MISALIGNED, dict(residual=P + 1)), (MISALIGNED, dict(y=P + 1))])
def test_rmsnorm_refuses(code, bad):
    with_(c.nvfp4_ffn_rmsnorm, NORM, NORM_OK, code, **bad)


def test_calls_without_rows_launch_nothing():
    c.nvfp4_ffn_rmsnorm(*[{**NORM_OK, "rows": 0, "x": 0}[n] for n in NORM.split()])
    c.nvfp4_ffn_quantize8(0, BF16, 0, 64, 64, 0, 0, 0)
    c.nvfp4_ffn_dequantize8(0, 0, 0, 64, 0, BF16, 64, 0)
    c.nvfp4_ffn_linear(0, 64, 0, 0, 0, 0, 0, 0, 0, 0, BF16, 0, 64, 64, None, 1, 0, 0, 0)
    c.nvfp4_ffn_gated(0, 64, 0, 2, 0, 0, 0, 0, BF16, 0, 64, 64, None, 1, 0, 0, 0)
    c.nvfp4_ffn_linear_dx(0, 64, 0, 0, BF16, 0, 64, 64, None, 1, 0, 0, 0)
    c.nvfp4_ffn_linear_dz(0, 64, 0, 0, 0, 0, 0, BF16, 0, 64, None, 0, 0, 0)
    c.nvfp4_ffn_gated_dz(0, 64, 0, 0, 0, 2, 0, BF16, 0, 64, None, 0)
    c.nvfp4_ffn_gather(0, 0, 0, 0, BF16, 0, 64, plan_of(), 0, 0)


BACK = "dy dy_stride s s_stride dtype rows n weight weight_f32 rstd dsum dsum_stride dx dweight ws ws_bytes stream"
BACK_OK = dict(dy=P, dy_stride=64, s=P, s_stride=64, dtype=BF16, rows=4, n=64, weight=P, weight_f32=0, rstd=P, dsum=P,
               dsum_stride=64, dx=P, dweight=P, ws=P, ws_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("code,bad", [
    (INVALID, dict(dtype=3)), (INVALID, dict(rows=-1)), (INVALID, dict(n=0)), (INVALID, dict(n=65537)), (INVALID, dict(dy=0)),
    (INVALID, dict(s=0)), (INVALID, dict(rstd=0)), (INVALID, dict(dx=0)), (INVALID, dict(weight=0)),
    (INVALID, dict(dy_stride=63)), (INVALID, dict(s_stride=63)), (INVALID, dict(dsum_stride=63)),
    (MISALIGNED, dict(dy=P + 1)), (MISALIGNED, dict(dx=P + 1)), (MISALIGNED, dict(dweight=P + 1)),
    (MISALIGNED, dict(ws=P + 16)), (WORKSPACE, dict(ws=0)), (WORKSPACE, dict(ws_bytes=4 * 64 * 4 - 1))])
def test_rmsnorm_backward_refuses(code, bad):
    assert c.nvfp4_ffn_rmsnorm_workspace_bytes(4, 64) == 4 * 64 * 4
    with_(c.nvfp4_ffn_rmsnorm_backward, BACK, BACK_OK, code, **bad)


def test_rows8_refuse():
    for dtype, rows, n, stride in ((3, 4, 64, 64), (BF16, -1, 64, 64), (BF16, 4, 48, 48), (BF16, 4, 0, 0),
                                   (BF16, 4, 64, 63), (BF16, 4, 1 << 21, 1 << 21)):
        refused(INVALID, c.nvfp4_ffn_quantize8, P, dtype, rows, n, stride, P, P, 0)
        refused(INVALID, c.nvfp4_ffn_dequantize8, P, P, rows, n, P, dtype, stride, 0)
    for args in ((0, P, P), (P, 0, P), (P, P, 0)):
        refused(INVALID, c.nvfp4_ffn_quantize8, args[0], BF16, 4, 64, 64, *args[1:], 0)
        refused(INVALID, c.nvfp4_ffn_dequantize8, *args[1:], 4, 64, args[0], BF16, 64, 0)
    refused(MISALIGNED, c.nvfp4_ffn_quantize8, P + 1, BF16, 4, 64, 64, P, P, 0)
    refused(MISALIGNED, c.nvfp4_ffn_quantize8, P, BF16, 4, 64, 64, P + 4, P, 0)


LINEAR_ARGS = "x x_stride w bias bias_f32 act residual residual_stride z y dtype rows n k plan clear ws ws_bytes stream"
LINEAR_OK = dict(x=P, x_stride=64, w=P, bias=P, bias_f32=0, act=2, residual=P, residual_stride=64, z=P, y=P, dtype=BF16,
                 rows=4, n=64, k=64, plan=None, clear=1, ws=0, ws_bytes=0, stream=0)


@pytest.mark.parametrize("code,bad", [
    (INVALID, dict(dtype=F32)), (INVALID, dict(dtype=3)), (INVALID, dict(act=4)), (INVALID, dict(act=-1)),
    (INVALID, dict(rows=-1)), (INVALID, dict(rows=1 << 31)), (INVALID, dict(n=60)), (INVALID, dict(n=0)),
    (INVALID, dict(n=1 << 21, residual_stride=1 << 21)), (INVALID, dict(k=60)), (INVALID, dict(k=0)), (INVALID, dict(x=0)), (INVALID, dict(w=0)),
    (INVALID, dict(y=0)), (INVALID, dict(x_stride=56)), (INVALID, dict(x_stride=1 << 22)),
    (INVALID, dict(residual_stride=56)), (INVALID, dict(n=1 << 16, k=1 << 15, x_stride=1 << 15, residual_stride=1 << 16)),
    (MISALIGNED, dict(x=P + 8)), (MISALIGNED, dict(w=P + 8)), (MISALIGNED, dict(y=P + 8)), (MISALIGNED, dict(bias=P + 8)),
    (MISALIGNED, dict(z=P + 8)), (MISALIGNED, dict(residual=P + 8)), (MISALIGNED, dict(x_stride=68)),
    (MISALIGNED, dict(residual_stride=68)), (WORKSPACE, dict(rows=33, n=4096, k=7168, x_stride=7168, residual_stride=4096)),
    (WORKSPACE, dict(rows=33, n=4096, k=7168, x_stride=7168, residual_stride=4096, ws=P, ws_bytes=1 << 10)),
    (MISALIGNED, dict(rows=33, n=4096, k=7168, x_stride=7168, residual_stride=4096, ws=P + 128, ws_bytes=1 << 30))])
def test_linear_refuses(code, bad):
    with_(c.nvfp4_ffn_linear, LINEAR_ARGS, LINEAR_OK, code, **bad)


@pytest.mark.parametrize("code,bad", [
    (INVALID, dict(experts=0)), (INVALID, dict(experts=513)), (INVALID, dict(offsets=0)), (MISALIGNED, dict(offsets=P + 2))])
def test_plans_are_refused(code, bad):
    bad = plan_of(**bad)
    with_(c.nvfp4_ffn_linear, LINEAR_ARGS, LINEAR_OK, code, plan=bad)
    refused(code, c.nvfp4_ffn_gated, P, 64, P, 2, P, 0, 0, 0, BF16, 4, 64, 64, bad, 1, 0, 0, 0)
    refused(code, c.nvfp4_ffn_linear_dx, P, 64, P, P, BF16, 4, 64, 64, bad, 1, 0, 0, 0)
    refused(code, c.nvfp4_ffn_linear_dw, P, 64, P, 64, P, 0, BF16, 4, 64, 64, bad, 0, 0, 0)
    refused(code, c.nvfp4_ffn_linear_dz, P, 64, P, 2, P, 0, 0, BF16, 4, 64, bad, 0, 0, 0)
    refused(code, c.nvfp4_ffn_gated_dz, P, 64, P, 0, 0, 2, P, BF16, 4, 64, bad, 0)
    refused(code, c.nvfp4_ffn_gather, P, 64, 0, 0, BF16, 4, 64, bad, P, 0)


@pytest.mark.parametrize("code,bad", [
    (INVALID, dict(topk=0)), (INVALID, dict(topk=17)), (INVALID, dict(topk=3)), (INVALID, dict(row_slots=0)),
    (MISALIGNED, dict(row_slots=P + 2))])
def test_plans_that_gather_are_refused(code, bad):
    refused(code, c.nvfp4_ffn_gated, P, 64, P, 2, P, 0, 0, 0, BF16, 4, 64, 64, plan_of(**bad), 1, 0, 0, 0)


@pytest.mark.parametrize("tokens", [-1, 1 << 30, 1 << 31, 1 << 62, (1 << 63) - 1])
def test_gather_refuses_more_rows_than_there_can_be(tokens):
    """1 << 62 tokens of four slots are 0 rows in 64 bits."""
    refused(INVALID, c.nvfp4_ffn_gather, P, 64, 0, 0, BF16, tokens, 64, plan_of(topk=4), P, 0)


GATED_ARGS = "x x_stride w act h kept codes scales dtype rows inner k plan clear ws ws_bytes stream"
GATED_OK = dict(x=P, x_stride=64, w=P, act=2, h=P, kept=P, codes=P, scales=P, dtype=F16, rows=4, inner=64, k=64, plan=None,
                clear=1, ws=0, ws_bytes=0, stream=0)


@pytest.mark.parametrize("code,bad", [
    (INVALID, dict(dtype=F32)), (INVALID, dict(act=0)), (INVALID, dict(act=4)), (INVALID, dict(rows=-1)),
    (INVALID, dict(inner=60)), (INVALID, dict(inner=40)), (INVALID, dict(inner=1 << 20)), (INVALID, dict(k=4)),
    (INVALID, dict(codes=0)), (INVALID, dict(scales=0)), (INVALID, dict(x=0)), (INVALID, dict(w=0)), (INVALID, dict(h=0)),
    (INVALID, dict(x_stride=56)), (MISALIGNED, dict(x=P + 8)), (MISALIGNED, dict(w=P + 8)), (MISALIGNED, dict(h=P + 8)),
    (MISALIGNED, dict(kept=P + 8)), (MISALIGNED, dict(codes=P + 4)), (MISALIGNED, dict(x_stride=68)),
    (INVALID, dict(rows=1 << 26, x_stride=1 << 10, plan=plan_of()))])
def test_gated_refuses(code, bad):
    with_(c.nvfp4_ffn_gated, GATED_ARGS, GATED_OK, code, **bad)


def test_gradients_refuse():
    dx, dw, dz, gdz = c.nvfp4_ffn_linear_dx, c.nvfp4_ffn_linear_dw, c.nvfp4_ffn_linear_dz, c.nvfp4_ffn_gated_dz
    for dtype, rows, n, k in ((F32, 4, 64, 64), (BF16, -1, 64, 64), (BF16, 4, 60, 64), (BF16, 4, 64, 60)):
        refused(INVALID, dx, P, 64, P, P, dtype, rows, n, k, None, 1, 0, 0, 0)
        refused(INVALID, dw, P, 64, P, 64, P, 0, dtype, rows, n, k, None, 0, 0, 0)
    for a, b, d, stride in ((0, P, P, 64), (P, 0, P, 64), (P, P, 0, 64), (P, P, P, 56)):
        refused(INVALID, dx, a, stride, b, d, BF16, 4, 64, 64, None, 1, 0, 0, 0)
        refused(INVALID, dw, a, stride, b, 64, d, 0, BF16, 4, 64, 64, None, 0, 0, 0)
    refused(MISALIGNED, dx, P + 8, 64, P, P, BF16, 4, 64, 64, None, 1, 0, 0, 0)
    refused(MISALIGNED, dx, P, 68, P, P, BF16, 4, 64, 64, None, 1, 0, 0, 0)
    refused(MISALIGNED, dw, P, 64, P, 68, P, 0, BF16, 4, 64, 64, None, 0, 0, 0)
    refused(MISALIGNED, dw, P, 64, P, 64, P + 8, 1, BF16, 4, 64, 64, None, 0, 0, 0)
    refused(WORKSPACE, dw, P, 64, P, 64, P, 0, BF16, 8192, 64, 64, None, 0, 0, 0)
    for args in ((P, 64, 0, 2, P, 0), (P, 64, P, 2, 0, 0), (0, 64, P, 2, P, 0), (P, 56, P, 2, P, 0), (P, 64, P, 5, P, 0)):
        refused(INVALID, dz, *args, 0, BF16, 4, 64, None, 0, 0, 0)
    refused(WORKSPACE, dz, P, 64, P, 2, P, P, 0, BF16, 4, 64, None, 0, 0, 0)
    refused(MISALIGNED, dz, P, 64, P, 2, P, P + 1, 0, BF16, 4, 64, None, 0, 0, 0)
    for args in ((P, 64, 0, 0, 0, 2, P), (P, 64, P, 0, 0, 0, P), (0, 64, P, 0, 0, 2, P), (P, 64, P, 0, 0, 2, 0), (P, 56, P, 0, 0, 2, P)):
        refused(INVALID, gdz, *args, BF16, 4, 64, None, 0)
    refused(INVALID, gdz, P, 40, 0, P, P, 2, P, BF16, 4, 40, None, 0)
    refused(MISALIGNED, gdz, P, 64, P + 8, 0, 0, 2, P, BF16, 4, 64, None, 0)
    names = "dh dh_stride x x_stride w act dz dtype rows inner k plan ws ws_bytes stream"
    ok = dict(dh=P, dh_stride=64, x=P, x_stride=64, w=P, act=2, dz=P, dtype=BF16, rows=4, inner=64, k=64, plan=None, ws=0, ws_bytes=0, stream=0)
    for code, bad in ((INVALID, dict(dh=0)), (INVALID, dict(x=0)), (INVALID, dict(w=0)), (INVALID, dict(dz=0)), (INVALID, dict(act=0)),
                      (INVALID, dict(dtype=F32)), (INVALID, dict(dh_stride=56)), (INVALID, dict(x_stride=56)), (INVALID, dict(inner=60)),
                      (INVALID, dict(k=60)), (INVALID, dict(rows=-1)), (INVALID, dict(plan=plan_of(topk=3))), (MISALIGNED, dict(dh=P + 8)),
                      (MISALIGNED, dict(dz=P + 8)), (MISALIGNED, dict(dh_stride=68)), (WORKSPACE, dict(rows=33, inner=2048, dh_stride=2048, k=7168, x_stride=7168))):
        with_(c.nvfp4_ffn_gated_again, names, ok, code, **bad)
    gather = c.nvfp4_ffn_gather
    refused(INVALID, gather, P, 64, 0, 0, BF16, 4, 64, None, P, 0)
    refused(INVALID, gather, 0, 64, P, P, BF16, 4, 40, plan_of(), P, 0)
    refused(INVALID, gather, 0, 64, P, 0, BF16, 4, 64, plan_of(), P, 0)
    refused(INVALID, gather, P, 64, 0, 0, F32, 4, 64, plan_of(), P, 0)
    refused(INVALID, gather, P, 64, 0, 0, BF16, 4, 64, plan_of(topk=17), P, 0)
    refused(MISALIGNED, gather, P, 68, 0, 0, BF16, 4, 64, plan_of(), P, 0)


def test_sizes_of_what_is_none():
    assert c.nvfp4_ffn_product_workspace_bytes(0, 64, 64, 0) == 0
    assert c.nvfp4_ffn_product_workspace_bytes(4, 60, 64, 0) == 0
    assert c.nvfp4_ffn_product_workspace_bytes(4, 64, 64, 513) == 0
    assert c.nvfp4_ffn_dw_workspace_bytes(-1, 64, 64, 0) == 0
    assert c.nvfp4_ffn_dz_workspace_bytes(4, 4, 0) == 0
    assert c.nvfp4_ffn_rmsnorm_workspace_bytes(4, 65537) == 0
    assert c.nvfp4_ffn_product_parts(4, 4, 64, 64, 0) == [] and c.nvfp4_ffn_product_parts(0, 0, 64, 64, 0) == []


@pytest.mark.parametrize("kind", PRODUCT_KINDS)
def test_parts_cover_the_rows_and_fit_the_workspace(kind):
    for rows in (1, 8, 9, 33, 64, 65, 257, 2051, 4096, 4099, 70000):
        for n, k in ((8, 8), (64, 8192), (4096, 64), (4104, 2048), (2048, 7168)):
            for experts in (0, 1, 8, 64):
                parts = c.nvfp4_ffn_product_parts(kind, rows, n, k, experts)
                out_rows, cols = (n, k) if kind == c.NVFP4_FFN_DW else (rows, k if kind == c.NVFP4_FFN_DX else n)
                assert sum(p[0] for p in parts) == out_rows and (len(parts) == 1 or not experts)
                if kind == c.NVFP4_FFN_DW:
                    have = c.nvfp4_ffn_dw_workspace_bytes(rows, n, k, experts)
                    out_rows *= max(experts, 1)
                else:
                    have = c.nvfp4_ffn_product_workspace_bytes(rows, cols, k + n - cols, experts)
                for r, tile, _, splits in parts:
                    assert 1 <= splits <= 16
                    r *= max(experts, 1) if kind == c.NVFP4_FFN_DW else 1
                    assert splits == 1 or r * cols * 4 * splits <= have


@pytest.mark.parametrize("rows,n,k", [(1 << 30, 8, 64), ((1 << 31) - (1 << 15), 8, 8), (1 << 25, 8192, 64), (1 << 24, 30000, 8)])
@pytest.mark.parametrize("experts", [0, 8])
def test_products_of_the_most_rows_fit_one_launch(rows, n, k, experts):
    for kind in (c.NVFP4_FFN_FORWARD, c.NVFP4_FFN_FORWARD_CODES):
        for r, tile, cols, splits in c.nvfp4_ffn_product_parts(kind, rows, n, k, experts):
            assert (r // tile + experts + 1) * -(-n // cols) * splits + 64 < 1 << 23


def test_gpu_cases_reach_every_kernel():
    """Every tile, with one part of k and with several, few rows, and ragged rows in two launches, by the products that
    can have them; for a device of 256 compute units, as every test of the package assumes."""
    seen = {kind: set() for kind in PRODUCT_KINDS}
    two = set()
    for kind, parts in parts_of(LINEAR, GATED):
        two |= {kind} if len(parts) > 1 else set()
        seen[kind] |= {(tile, cols, splits > 1) for _, tile, cols, splits in parts}
    shapes = {(128, 128), (256, 128), (256, 256)}
    want = {(*s, False) for s in shapes} | {(128, 128, True)}
    for kind in PRODUCT_KINDS:
        rows64 = {(64, 128, False), (64, 128, True), (320, 128, False), (320, 256, False)} if kind != c.NVFP4_FFN_DW else set()
        few = {(0, 0, False)} if kind == c.NVFP4_FFN_FORWARD else set()
        missing = (want | rows64 | few) - seen[kind]
        assert not missing, (kind, missing)
    assert {c.NVFP4_FFN_FORWARD, c.NVFP4_FFN_DX, c.NVFP4_FFN_DW} <= two


# ---- what Python checks --------------------------------------------------------------

def test_python_refuses_what_is_not_on_a_gpu_or_not_known():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, 64, dtype=torch.bfloat16)
    for call in (lambda: ffn.rmsnorm(x), lambda: ffn.quantize8(x), lambda: ffn.linear(x, w), lambda: ffn.gated(x, w),
                 lambda: ffn.dequantize8(ffn.Rows8(x, x)), lambda: ffn.rmsnorm_backward(x, x, None, x[:, 0]),
                 lambda: ffn.linear_backward(x, x, w), lambda: ffn.gated_backward(x, x, w)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for name in ("tanh", "SiLU", 3):
        with pytest.raises(ValueError, match="activation"):
            ffn._activation(name)
    with pytest.raises(ValueError, match="activation"):
        ffn._activation(None, gated=True)


# ---- the oracle --------------------------------------------------------------------------

def test_oracle_rows8_pins():
    v = torch.zeros(1, 64, dtype=torch.float64)
    v[0, :6] = torch.tensor([448.0, -1.0, 0.5, 2.0 ** -9, 3 * 2.0 ** -10, 17.0])
    v[0, 32], v[0, 33] = 449.0, math.inf
    codes, scales = FO.rows8(v)
    # 448: 0x7E; -1: 0xB8; half a step below 2^-6: ties to even; 17 between 16 and 18: the even mantissa
    assert codes[0, :6].tolist() == [0x7E, 0xB8, 0x30, 1, 2, 0x58] and scales.tolist() == [[127, 255]]
    got = FO.values8(codes, scales)
    assert got[0, :6].tolist() == [448.0, -1.0, 0.5, 2.0 ** -9, 2.0 ** -8, 16.0] and bool(got[0, 32:].isnan().all())
    for top, byte in ((448.0, 127), (448.5, 128), (896.0, 128), (224.0, 126), (225.0, 127), (2.0 ** -140, 1), (0.0, 1)):
        assert FO.rows8(torch.full((1, 32), top, dtype=torch.float64))[1].item() == byte


def test_oracle_codes_are_torchs():
    v = torch.randn(50, 64, dtype=torch.float64) * torch.logspace(-6, 6, 50, dtype=torch.float64).unsqueeze(1)
    codes, scales = FO.rows8(v)
    q = v.unflatten(1, (-1, 32)) / torch.exp2(scales.double() - 127).unsqueeze(-1)
    assert torch.equal(q.float().to(torch.float8_e4m3fn).view(torch.uint8).flatten(1), codes)
    assert float(q.abs().max()) <= 448 and float(q.abs().amax(-1).min()) > 224


def differences(f, x, h=1e-5):
    """Gradient of the scalar f at x by central differences."""
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        up = f()
        flat[i] = keep - h
        out[i] = (up - f()) / (2 * h)
        flat[i] = keep
    return g


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu"])
def test_oracle_gradients_against_differences(act):
    g = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, dy = r(3, 5), r(4, 5), r(4), r(3, 4)
    y, z = FO.linear(x, w, b, act)
    dx, dw, db, _ = FO.linear_backward(dy, x, w, z, act)
    loss = lambda: float((FO.linear(x, w, b, act)[0] * dy).sum())  # noqa: E731
    for got, at in ((dx, x), (dw, w), (db, b)):
        assert torch.allclose(got, differences(loss, at), atol=1e-8, rtol=1e-7)
    if act is not None:
        dh = r(3, 2)
        dz = FO.gated_dz(dh, FO.gated(x, w, act)[1], act)
        loss = lambda: float((FO.gated(x, w, act)[0] * dh).sum())  # noqa: E731
        assert torch.allclose(dz @ w, differences(loss, x), atol=1e-8, rtol=1e-7)
        assert torch.allclose(dz.T @ x, differences(loss, w), atol=1e-8, rtol=1e-7)


def test_oracle_norm_gradients_against_differences():
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    s, w, dy, dsum = r(3, 6), r(6), r(3, 6), r(3, 6)
    _, rstd = FO.rmsnorm(s, w, 1e-3)
    dx, dw = FO.rmsnorm_backward(dy, s, w, rstd, dsum)
    loss = lambda: float((FO.rmsnorm(s, w, 1e-3)[0] * dy).sum() + (s * dsum).sum())  # noqa: E731
    assert torch.allclose(dx, differences(loss, s), atol=1e-8, rtol=1e-7)
    assert torch.allclose(dw, differences(loss, w), atol=1e-8, rtol=1e-7)


def test_oracle_limits():
    z = torch.tensor([-math.inf, math.inf, math.nan, -1000.0, 1000.0], dtype=torch.float64)
    for kind in ("relu", "silu", "gelu"):
        a, s = FO.activation(z, kind), FO.slope(z, kind)
        assert a[0] == 0 and a[1] == math.inf and a[2].isnan() and a[3] == 0 and a[4] == 1000
        assert abs(s[0]) < 1e-290 and s[1] == 1 and s[2].isnan() and abs(s[3]) < 1e-290 and s[4] == 1
