"""Forms of the block's entry points on the CPU: what they refuse, and how products are computed (no GPU needed)."""
import pytest

import ffn_cases
import ffn_parts_cases
import moe_matmul_amd as mm
from moe_matmul_amd import _ffn_binding as c

P = 0x10000  # an address that no refused call reads
INVALID, MISALIGNED, WORKSPACE = mm.NVFP4_ERR_INVALID, mm.NVFP4_ERR_MISALIGNED, mm.NVFP4_ERR_WORKSPACE

DX = dict(dz=P, dz_stride=64, w=P, dx=P, dx_f32=1, dtype=2, rows=4, n=64, k=64, plan=None, clear=1, ws=0, ws_bytes=0, stream=0)


@pytest.mark.parametrize("code,bad", [
    (INVALID, dict(dtype=0)), (INVALID, dict(rows=-1)), (INVALID, dict(n=60)), (INVALID, dict(k=60)), (INVALID, dict(dz=0)),
    (INVALID, dict(w=0)), (INVALID, dict(dx=0)), (INVALID, dict(dz_stride=56)), (INVALID, dict(dz_stride=1 << 22)),
    (MISALIGNED, dict(dz=P + 8)), (MISALIGNED, dict(dx=P + 8)), (MISALIGNED, dict(dz_stride=68)),
    (WORKSPACE, dict(rows=33, n=8192, dz_stride=8192, k=512))])
@pytest.mark.parametrize("f32", [0, 1])
def test_gradients_of_rows_refuse(code, bad, f32):
    with pytest.raises(c.Nvfp4FfnError) as e:
        c.nvfp4_ffn_linear_dx_ex(*{**DX, "dx_f32": f32, **bad}.values())
    assert e.value.code == code
    c.nvfp4_ffn_linear_dx_ex(*{**DX, "rows": 0}.values())


@pytest.mark.parametrize("n,k", [(2048, 512), (1024, 2048), (14336, 4096)])
def test_few_rows_of_experts_are_few_in_all(n, k):
    """The kernel of few rows takes an expert's eight at a time, one after the other: what all may be one expert's has to
    be few itself."""
    few = [(0, 0)]
    for experts in (2, 8, 16, 17, 64, 256, 512):
        for rows in (1, 2 * experts, 4 * experts, 4 * experts + 1, 63, 64, 65, 128, 1000, 2048):
            parts = c.nvfp4_ffn_product_parts(c.NVFP4_FFN_FORWARD, rows, n, k, experts)
            assert ([p[1:3] for p in parts] == few) == (rows <= min(64, 4 * experts)), (experts, rows, parts)


def test_gpu_cases_reach_every_tile_with_and_without_parts():
    """For a device of 256 compute units. (Dense rows in tiles of 320 x 256 never come in parts: they are there for rows
    that leave a part of a round in all others, and parts fill rounds.)"""
    seen = set()
    for size in ffn_cases.LINEAR + ffn_parts_cases.LINEAR:
        seen |= ffn_parts_cases.linear_kernels(*size)
    for size in ffn_cases.GATED + ffn_parts_cases.GATED:
        seen |= ffn_parts_cases.gated_kernels(*size)
    for size in ffn_parts_cases.EXPERTS:
        seen |= ffn_parts_cases.experts_kernels(*size)
    tall = [(64, 128), (128, 128), (256, 128), (256, 256), (320, 128), (320, 256)]
    want = {(name, by_experts, *tile, parts) for name in ("linear", "gated", "codes", "dx", "dw") for by_experts in (False, True)
            for tile in (tall[1:4] if name == "dw" else tall) for parts in (False, True)}
    want -= {(name, False, 320, 256, True) for name in ("linear", "gated", "codes", "dx")}
    want |= {(name, by_experts, 0, 0, False) for name in ("linear", "gated") for by_experts in (False, True)}
    assert not want - seen, sorted(want - seen)
