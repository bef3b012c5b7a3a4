"""Gated projections and their gradients with ReLU and GELU at every size: test_ffn_gpu.py has SiLU in place of one or
both of them at the larger ones. Tolerances as there, and one term more for ReLU where both projections are computed
again from x: its slope jumps from 0 to 1 at 0, so where the sum's error bg reaches over 0 (|g| <= bg) the slope is off by
up to 1, and dg = dh u act'(g) by up to |dh| (|u| + bu). (Of what was kept the slope is that of the kept value.)"""
import pytest
import torch

import oracle.ffn_oracle as FO
from ffn_cases import GATED
from moe_matmul_amd import ffn
from test_ffn_gpu import H, H16, TINY, TYPES, act_error, announce, close, rng, same  # noqa: F401

pytestmark = pytest.mark.gpu

ACTS = ("relu", "silu", "gelu")
# the sizes beyond the ninth with an activation whose place SiLU has there
CASES = [(size, act) for i, size in enumerate(GATED) for act in ("relu", "gelu") if i > 8 and (i + ACTS.index(act)) % 3]


def check_gated(m, inner, k, act, dtype):
    t, n, r = TYPES[dtype], 2 * inner, rng(m, inner, k, dtype)
    x, w, dh = r(m, k).to(t), (r(n, k) * k ** -0.5).to(t), r(m, inner).to(t)
    f = torch.Tensor.double
    h, kept = ffn.gated(x, w, activation=act, save="rows")
    want, z = FO.gated(f(x), f(w), act)
    bz = (k + 16) * H * (f(x).abs() @ f(w).abs().T)
    close(kept, z, bz)
    (g, u), (bg, bu) = z.chunk(2, 1), bz.chunk(2, 1)
    bh = act_error(g, bg, act) * (u.abs() + bu) + FO.activation(g, act).abs() * bu + 2 * H * want.abs()
    close(h, want, bh)
    same(ffn.gated(x, w, activation=act), h)
    keeps = [("rows", kept, x)]
    if inner % 32 == 0 and k % 32 == 0:
        h8, kept8 = ffn.gated(x, w, activation=act, save="rows8")
        close(h8, want, bh)
        scale = torch.exp2(kept8.scales.double() - 127).repeat_interleave(32, 1)
        close(FO.values8(*kept8).float(), z, bz * 1.1 + 2.0 ** -4 * z.abs() + scale * 2.0 ** -10)
        keeps.append(("rows8", kept8, ffn.quantize8(x)))
    keeps.append(("none", None, x))
    d = f(dh).abs()
    for name, k_, x_ in keeps:
        dx, dw = ffn.gated_backward(dh, x_, w, k_, activation=act)
        zk = z if k_ is None else f(kept) if name == "rows" else FO.values8(*k_)
        xk = FO.values8(*x_) if isinstance(x_, ffn.Rows8) else f(x_)
        dz = FO.gated_dz(f(dh), zk, act)
        gk, uk = zk.chunk(2, 1)
        err = H16[t] * dz.abs() + 512 * H * torch.cat((d * uk.abs(), d * FO.activation(gk, act).abs()), 1) + TINY[t]
        if k_ is None:
            jump = d * (u.abs() + bu) * (g.abs() <= bg) if act == "relu" else torch.zeros_like(d)
            err = err + torch.cat((d * (1.13 * bu + 1.13 * bg * (u.abs() + bu)) + jump, d * 1.13 * bg), 1)
        a = dz.abs() + err
        close(dx, dz @ f(w), (n + 16) * H * (a @ f(w).abs()) + err @ f(w).abs())
        close(dw, dz.T @ xk, (m + 16) * H * (a.T @ xk.abs()) + err.T @ xk.abs())


@pytest.mark.parametrize("size,act", CASES, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else v)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated_and_its_gradients(size, act, dtype):
    check_gated(*size, act, dtype)
