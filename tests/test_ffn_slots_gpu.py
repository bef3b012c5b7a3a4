"""The gradient of a token's row by experts is one sum, over its slots and their columns: rounded once."""
import pytest
import torch

import oracle.ffn_oracle as FO
from moe_matmul_amd import _ffn_binding as c
from moe_matmul_amd import ffn, moe
from test_ffn_gpu import announce, close, pick, rng, same, H  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,topk,experts,inner,hidden", [(3, 2, 4, 32, 64), (70, 4, 8, 96, 136), (900, 2, 3, 160, 520), (300, 16, 64, 64, 72),
                                                              (50, 1, 4, 64, 72)])
def test_whole_numbers(tokens, topk, experts, inner, hidden, dtype):
    """Small whole numbers: dz is exact in 16 bits and every partial sum in 32, but a slot's sum is not in 16 (it is
    odd, and beyond 2^8 or 2^11); what is left of a token's slots once they are added often is."""
    g = torch.Generator("cuda").manual_seed(tokens)
    ints = lambda top, *s: torch.randint(-top, top + 1, s, device="cuda", generator=g).to(dtype)  # noqa: E731
    p = moe.plan(pick(rng(tokens, topk), tokens, topk, experts, 0.1), experts)
    x, w, dh = ints(3, tokens, hidden), ints(7, experts, 2 * inner, hidden), ints(7, p.rows, inner)
    kept = ints(31, p.rows, 2 * inner)
    dx, _ = ffn.gated_backward(dh, x, w, kept, activation="relu", plan=p)
    f, ends = torch.Tensor.double, p.offsets.tolist()
    dz, want, lost = FO.gated_dz(f(dh), f(kept), "relu"), torch.zeros(tokens, hidden, device="cuda", dtype=torch.float64), 0
    same(dz.to(dtype).double().float(), dz.float())
    for e in range(experts):
        at = slice(ends[e], ends[e + 1])
        row = dz[at] @ f(w[e])
        lost += int((row.to(dtype).double() != row).sum())
        want.index_add_(0, p.row_slots[at].long() // topk, row)
    assert lost and float(want.abs().max()) < 2 ** 24
    same(dx, want.to(dtype))


@pytest.mark.parametrize("experts", [0, 3])
@pytest.mark.parametrize("rows,n,k", [(1, 64, 72), (9, 4096, 64), (300, 264, 1000), (33, 8192, 512), (2051, 512, 2048), (8195, 512, 8192)])
def test_rows_gradient_in_fp32(rows, n, k, experts):
    """nvfp4_ffn_linear_dx_ex by tiles, parts of k and two launches: its fp32 rows rounded are the 16-bit ones."""
    r = rng(rows, n, k, experts)
    lead = (experts,) if experts else ()
    dz, w = r(rows, n).bfloat16(), (r(*lead, n, k) * n ** -0.5).bfloat16()
    p = moe.plan((torch.arange(rows, device="cuda", dtype=torch.int32) % 4 - 1).view(-1, 1), experts) if experts else None
    need = c.nvfp4_ffn_product_workspace_bytes(rows, k, n, experts)
    room = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    out = []
    for f32 in (0, 1):
        dx = torch.full((rows, k), 7.0, device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
        c.nvfp4_ffn_linear_dx_ex(dz.data_ptr(), n, w.data_ptr(), dx.data_ptr(), f32, 2, rows, n, k, ffn._plan(p), 1, room.data_ptr(), need,
                                 torch.cuda.current_stream().cuda_stream)
        out.append(dx)
    same(out[1].bfloat16(), out[0])
    for e, at in enumerate([slice(0, rows)] if p is None else [slice(a, b) for a, b in zip(p.offsets.tolist(), p.offsets.tolist()[1:])]):
        d, v = dz[at].double(), (w if p is None else w[e]).double()
        close(out[1][at], d @ v, (n + 16) * H * (d.abs() @ v.abs()))
    if p is not None:
        assert bool((out[1][p.offsets.tolist()[-1]:] == 0).all())
