"""Products of rows that lie far apart, on the GPU: the largest stride that is taken, where the last rows of a tile of 320
would be beyond 32-bit offsets from its first. What lies between the rows is NaN.

Tolerances as in test_ffn_gpu.py: sums of exact products by (k + 16) half steps of fp32 of their terms' magnitude, and
what follows them; outputs are rounded once more."""
import math

import pytest
import torch

import oracle.ffn_oracle as FO
from moe_matmul_amd import _ffn_binding as c
from moe_matmul_amd import ffn, moe
from test_ffn_gpu import H, H16, TINY, act_error, announce, close, linear_bounds, rng  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = (1 << 22) - 8
f = torch.Tensor.double


def far_apart(v, stride):
    room = torch.full((v.shape[0] * stride,), math.nan, device="cuda", dtype=v.dtype)
    out = room.as_strided(v.shape, (stride, 1))
    out.copy_(v)
    return out


def tall(kind, rows, n, k, experts):
    return all(p[1] == 320 for p in c.nvfp4_ffn_product_parts(kind, rows, n, k, experts))


@pytest.mark.parametrize("stride", [3365960, 3365968, FAR])
@pytest.mark.parametrize("rows,n,k", [(640, 16384, 520), (1280, 13120, 64), (320, 13120, 8192)])
def test_linear(rows, n, k, stride):
    assert tall(c.NVFP4_FFN_FORWARD, rows, n, k, 0)
    r = rng(rows, n, k)
    x, w, residual = r(rows, k).bfloat16(), (r(n, k) * k ** -0.5).bfloat16(), r(rows, n).bfloat16()
    y, z = ffn.linear(far_apart(x, stride), w, residual=residual, activation="silu", save=True)
    want, want_z, by, bz = linear_bounds(f(x), f(w), None, "silu", f(residual))
    close(z, want_z, bz)
    close(y, want, by)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,inner,k", [(640, 8192, 520), (1280, 6560, 64)])
def test_gated_and_its_gradients_without_what_was_kept(rows, inner, k, dtype):
    assert tall(c.NVFP4_FFN_FORWARD, rows, 2 * inner, k, 0)
    r = rng(rows, inner, k)
    x, w, dh = r(rows, k).to(dtype), (r(2 * inner, k) * k ** -0.5).to(dtype), r(rows, inner).to(dtype)
    far = far_apart(x, FAR)
    h, kept = ffn.gated(far, w, save="rows")
    want, z = FO.gated(f(x), f(w))
    bz = (k + 16) * H * (f(x).abs() @ f(w).abs().T)
    close(kept, z, bz)
    (g, u), (bg, bu) = z.chunk(2, 1), bz.chunk(2, 1)
    close(h, want, act_error(g, bg, "silu") * (u.abs() + bu) + FO.activation(g, "silu").abs() * bu + 2 * H * want.abs())
    dx, dw = ffn.gated_backward(dh, far, w)
    d = f(dh).abs()
    dz = FO.gated_dz(f(dh), z)
    err = H16[dtype] * dz.abs() + 512 * H * torch.cat((d * u.abs(), d * FO.activation(g, "silu").abs()), 1) + TINY[dtype]
    err = err + torch.cat((d * (1.13 * bu + 1.13 * bg * (u.abs() + bu)), d * 1.13 * bg), 1)
    a = dz.abs() + err
    close(dx, dz @ f(w), (2 * inner + 16) * H * (a @ f(w).abs()) + err @ f(w).abs())
    close(dw, dz.T @ f(x), (rows + 16) * H * (a.T @ f(x).abs()) + err.T @ f(x).abs())


@pytest.mark.parametrize("rows,n,k", [(620, 2048, 14336), (1280, 6144, 4096)])
def test_gradients_of_a_product_whose_dy_lies_apart(rows, n, k):
    """Without an activation dy takes the place of dz, where it lies."""
    assert tall(c.NVFP4_FFN_DX, rows, n, k, 0)
    r = rng(rows, n, k)
    x, w, dy = r(rows, k).bfloat16(), (r(n, k) * k ** -0.5).bfloat16(), r(rows, n).bfloat16()
    dx, dw, _ = ffn.linear_backward(far_apart(dy, FAR), x, w)
    close(dx, f(dy) @ f(w), (n + 16) * H * (f(dy).abs() @ f(w).abs()))
    close(dw, f(dy).T @ f(x), (rows + 16) * H * (f(dy).abs().T @ f(x).abs()))


def test_by_experts():
    """Experts of 320 and of 640 rows, whose tiles would be of 320: forward and gradients, each row far from the next."""
    rows, n, k, experts = 1480, 8192, 64, 3
    assert tall(c.NVFP4_FFN_FORWARD, rows, n, k, experts) and tall(c.NVFP4_FFN_DX, rows, 2048, 4096, experts)
    counts = [640, 320, 520]
    p = moe.plan(torch.repeat_interleave(torch.arange(3), torch.tensor(counts)).to("cuda", torch.int32).view(-1, 1), experts)
    r, ends = rng(7), [0, 640, 960, 1480]
    x, w = r(rows, k).bfloat16(), (r(experts, n, k) * k ** -0.5).bfloat16()
    y = ffn.linear(far_apart(x, FAR), w, plan=p)
    dy, w2, x2 = r(rows, 2048).bfloat16(), (r(experts, 2048, 4096) / 64).bfloat16(), r(rows, 4096).bfloat16()
    dx, dw, _ = ffn.linear_backward(far_apart(dy, FAR), x2, w2, plan=p)
    for e in range(experts):
        at = slice(ends[e], ends[e + 1])
        close(y[at], f(x[at]) @ f(w[e]).T, (k + 16) * H * (f(x[at]).abs() @ f(w[e]).abs().T))
        close(dx[at], f(dy[at]) @ f(w2[e]), (2048 + 16) * H * (f(dy[at]).abs() @ f(w2[e]).abs()))
        close(dw[e], f(dy[at]).T @ f(x2[at]), (counts[e] + 16) * H * (f(dy[at]).abs().T @ f(x2[at]).abs()))
