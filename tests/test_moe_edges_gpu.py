"""Edges of the operators around the grouped GEMM, on the GPU against the float64
oracle: tables that do not fit together, logits whose scores leave fp32, factors
of a layer, groups beyond the grouped GEMM's limits, choice values a few 2^-24
apart. Helpers and tolerances are those of test_moe_gpu.py.
"""
import sys

import numpy as np
import pytest
import torch

import moe_matmul_amd as mm
import oracle.moe_oracle as MO
from moe_matmul_amd import _moe_binding as c
from moe_matmul_amd import moe
from test_moe_gpu import H, TYPES, check_rows, close, f64, gpu, operand, rng_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def announce(request):
    print(f"[gpu-case] {request.node.name}", flush=True)
    sys.stdout.flush()
    yield
    torch.cuda.synchronize()


# ---- tables that do not fit together ---------------------------------------------

@pytest.mark.parametrize("tokens,topk,experts,k", [(40, 3, 7, 96), (4500, 8, 20, 1056)])  # scales in one launch, and in two
@pytest.mark.parametrize("other", ["none", "beyond", "next"])
def test_dispatch_takes_experts_from_rows(tokens, topk, experts, k, other):
    """Ids that were rewritten after the plan change nothing; slots whose row is none of the rows store nothing."""
    rng = rng_of(tokens, topk, experts, k)
    ids = rng.integers(-1, experts, (tokens, topk)).astype(np.int32)
    x = gpu(rng.standard_normal((tokens, k)), torch.bfloat16)
    p = moe.plan(gpu(ids), experts)
    slots = tokens * topk
    room = c.nvfp4_moe_sf_bytes(slots, experts, k)
    a = torch.full((slots + 2, k // 2), 0xAB, dtype=torch.uint8, device="cuda")
    store = torch.full((room + 1024,), 0xCD, dtype=torch.uint8, device="cuda")
    rewritten = gpu({"none": np.full_like(ids, -1), "beyond": np.full_like(ids, 2 ** 31 - 1), "next": ids + 1}[other])
    need = c.nvfp4_moe_dispatch_workspace_bytes(tokens, topk, k)
    assert (need > 0) == (slots * k > 2 ** 25)
    workspace = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")

    def dispatch(slot_rows):
        c.nvfp4_moe_dispatch(x.data_ptr(), c.NVFP4_MOE_BF16, tokens, topk, k, k, 1.0, rewritten.data_ptr(), slot_rows.data_ptr(),
                             p.row_slots.data_ptr(), p.offsets.data_ptr(), p.atoms.data_ptr(), experts, a[1].data_ptr(),
                             store[512:].data_ptr(), workspace.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
    dispatch(p.slot_rows)
    offsets, atoms, _, row_slots = MO.plan(ids, experts)
    rows = int(offsets[-1])
    an, sn, xn = a.cpu().numpy(), store.cpu().numpy(), f64(x)
    for e in range(experts):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            check_rows(an[1 + lo:1 + hi], sn[512:], xn[row_slots[lo:hi] // topk], k, atom=int(atoms[e]))
    assert (an[0] == 0xAB).all() and (an[1 + rows:] == 0xAB).all() and (sn[:512] == 0xCD).all() and (sn[512 + room:] == 0xCD).all()
    a.fill_(0xAB)
    beyond = rng.choice(np.array([-1, -2 ** 31, slots, slots + 1, 2 ** 31 - 1]), ids.shape).astype(np.int32)
    dispatch(gpu(beyond))
    assert (a == 0xAB).all() and (store[:512] == 0xCD).all() and (store[512 + room:] == 0xCD).all()


def test_a_plan_keeps_its_ids():
    """What a plan was made from may be rewritten: by the next layer's routing, say."""
    rng = rng_of(31)
    ids = rng.integers(-1, 6, (50, 3)).astype(np.int32)
    x = gpu(rng.standard_normal((150, 64)), torch.float16)
    w, alpha = rng.standard_normal((50, 3)).astype(np.float32), rng.uniform(0.5, 2, 5).astype(np.float32)
    buffer = gpu(ids)
    p = moe.plan(buffer, 5)
    buffer.copy_((buffer + 1).clamp(max=4))
    rows = MO.plan(ids, 5)[2]
    assert np.array_equal(p.ids.cpu().numpy(), np.where(ids < 5, ids, -1))
    want, size = MO.combine(f64(x), w, rows, alpha, ids)
    close(moe.combine(x, gpu(w), p, alpha=gpu(alpha), dtype=torch.float32), want, 6 * H[torch.float32] * size, torch.float32)
    a, sfa = moe.quantize(x[:50], plan=p)
    values = f64(moe.dequantize(a, sfa, plan=p))
    codes, scales = MO.quantize(f64(x[:50]))
    for t, j in zip(*np.nonzero(rows >= 0)):
        assert np.array_equal(values[rows[t, j]], MO.values(codes[t:t + 1], scales[t:t + 1])[0])
    dy = gpu(rng.standard_normal((50, 64)), torch.float32)
    want, want_w, size = MO.combine_backward(f64(dy), f64(x), w, rows, alpha, ids)
    dc, dw = moe.combine_backward(dy, x, gpu(w), p, alpha=gpu(alpha), dc=torch.zeros_like(x))
    named = np.flatnonzero(~np.isnan(want).any(axis=1))
    close(dc[gpu(named)], want[named], 3 * H[torch.float32] * np.abs(want[named]), torch.float16)
    close(dw, want_w, 13 * H[torch.float32] * size, torch.float32)
