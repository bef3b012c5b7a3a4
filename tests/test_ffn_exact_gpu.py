"""What can be told to the last bit: directional derivatives of products of whole numbers, through the kernels' own
forward products, and activations of infinities and far values. Tolerances of activations and slopes as in
test_ffn_gpu.py; the 256 half steps H of an activation's own evaluation are:
* e^x by 2^x: log2 e is rounded, 0.23 |x| H of the result, the product with it, |x| H, the power 2 H; SiLU's x is z, above
  -87 where z e^z is above 2^-119: 109 H, and a reciprocal, a sum and a product, 4 H
* GELU's x is -z^2 / 2, above -80 where z Phi(z) is: 98 H, the square's rounding |x| H more, 80 H, and Phi's polynomial
  (0.75 H and 9 roundings of terms that nearly all are positive, a reciprocal) and three products, 20 H
Below 2^-119 a result may be 0."""
import math

import pytest
import torch

import oracle.ffn_oracle as FO
from moe_matmul_amd import ffn, moe
from test_ffn_gpu import H, announce, close, same  # noqa: F401

pytestmark = pytest.mark.gpu

f = torch.Tensor.double


@pytest.mark.parametrize("m,n,k", [(3, 16, 24), (8, 136, 200), (70, 72, 40), (300, 136, 64), (700, 200, 520)])
@pytest.mark.parametrize("experts", [0, 3])
def test_gradients_are_the_slopes_of_the_forward_product(m, n, k, experts):
    """A change of one element of a row of x, by 1 or 2, changes its row of y by that multiple of w's column: at most 6 in
    magnitude, exact, as dx is (at most 9 * 200 < 2^11 in fp16) and dw in fp32. So along any such change of all rows y's
    is dx's, to the last bit, and alike for w. The sums in float64 are of whole numbers."""
    g = torch.Generator("cuda").manual_seed(m + experts)
    ints = lambda *s: torch.randint(-3, 4, s, device="cuda", generator=g).half()  # noqa: E731
    lead = (experts,) if experts else ()

    def one_in_a_row(*s):
        at = torch.randint(s[-1], s[:-1], device="cuda", generator=g).unsqueeze(-1)
        return torch.zeros(*s, device="cuda", dtype=torch.float16).scatter_(-1, at, 1 + torch.rand(at.shape, device="cuda", generator=g).round().half())

    p = moe.plan((torch.arange(m, device="cuda", dtype=torch.int32) % (experts + 1) - 1).view(-1, 1), experts) if experts else None
    x, w, dy, d, e = ints(m, k), ints(*lead, n, k), ints(m, n), one_in_a_row(m, k), one_in_a_row(*lead, n, k)
    dw = torch.empty(*lead, n, k, device="cuda")
    dx, _, _ = ffn.linear_backward(dy, x, w, plan=p, dw=dw)
    assert float(dx.abs().max()) > 8 and float(dw.abs().max()) > 8
    for got, change, y in ((dx, d, ffn.linear(d, w, plan=p)), (dw, e, ffn.linear(x, e, plan=p))):
        assert float((f(got) * f(change)).sum()) == float((f(dy) * f(y)).sum())
    if p is None:  # and row by row
        y = ffn.linear(d, w)
        assert torch.equal((f(dx) * f(d)).sum(1), (f(dy) * f(y)).sum(1))
        y = ffn.linear(x, e)
        assert torch.equal((f(dw) * f(e)).sum(1), (f(dy) * f(y)).sum(0))


LIMITS = [-math.inf, math.inf, math.nan, -60000.0, 60000.0, -2000.0, 2000.0, -110.0, -104.5, -103.5, -100.0, -90.0, -16.0, -15.5, -14.0, -12.5,
          -1e-3, -0.0, 0.0, 1e-3, 15.5, 90.0, 110.0, 6e-5]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("rows", [8, 24, 600])
def test_activations_at_their_limits(rows, act, dtype):
    """Products of one element a row, the others 0 on both sides: z is what was given, infinities among it, and NaN is
    where NaN was given and nowhere else. By the kernels of few rows, of tiles and of parts."""
    z = torch.tensor(LIMITS, device="cuda").to(dtype).repeat(-(-rows // len(LIMITS)) + 1)
    for at in range(0, len(LIMITS), min(rows, len(LIMITS))):
        mine = z[at:at + rows]
        for k in (8, 4096):
            x, w = torch.zeros(rows, k, device="cuda", dtype=dtype), torch.zeros(64, k, device="cuda", dtype=dtype)
            x[:, 0], w[:, 0] = mine, 1
            given = mine.view(-1, 1).expand(-1, 64)
            y, kept = ffn.linear(x, w, activation=act, save=True)
            assert torch.equal(kept.nan_to_num(nan=7.0, posinf=math.inf, neginf=-math.inf), given.nan_to_num(nan=7.0, posinf=math.inf, neginf=-math.inf))
            assert torch.equal(kept.isnan(), given.isnan())
            want = FO.activation(f(given), act)
            close(y, want, 256 * H * want.abs() + 2.0 ** -119)
            # the gate has z, the other projection 1: h is the activation, dz its slope and its value
            x[:, 1], w[32:, 0], w[32:, 1] = 1, 0, 1
            want = want[:, :32]
            h, kept = ffn.gated(x, w, activation=act, save="rows")
            fine = torch.isfinite(mine)  # infinity times w's 0 is NaN in the other projection
            close(h[fine], want[fine], 258 * H * want[fine].abs() + 2.0 ** -119)
            one = torch.ones(rows, 32, device="cuda", dtype=dtype)
            g64 = f(given)[fine, :32]
            for k_ in (kept, None):
                _, dw = ffn.gated_backward(one[fine], x[fine], w, None if k_ is None else k_[fine], activation=act,
                                           dw=torch.empty(64, k, device="cuda"))
                # x's column 1 is 1 in every row: dw's column 1 has the sums of the slopes and of the activations
                half = torch.finfo(dtype).eps / 2
                slope, value = FO.slope(g64, act), FO.activation(g64, act)
                n = g64.shape[0] + 16
                for got, v, err in ((dw[:32, 1], slope, 512 * H), (dw[32:, 1], value, 256 * H)):
                    terms = v.abs() + err * (v.abs() + 1) + 2.0 ** -24
                    close(got, v.sum(0), ((half + n * H) * terms + err * (v.abs() + 1) + 2.0 ** -24).sum(0))
