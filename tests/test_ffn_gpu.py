"""GPU parity of the feed-forward block in 16 bits (moe_matmul_amd.ffn) against the float64 oracle of
oracle/ffn_oracle.py.

Tolerances. H(t) is half a step of a type relative to the value: fp32 2^-24, fp16 2^-11, bf16 2^-8, E4M3 2^-4
(eps / 2); H alone is fp32's. Rows in 8 bits by themselves, and sums of the residual, are equal. fp32 results:
* products: exact products, at most k + 16 roundings of partial sums: (k + 16) H of the terms' magnitude, the bias
  among them.
* activations: slopes are at most 1.13, so 1.13 of their argument's error; their own evaluation 256 H of the value
  (erfc's argument is rounded, and erfc(t) falls by 2 t relative to itself: 2 t^2 H, t <= 10), and 2^-119, below
  which a result may be 0. A product of two: the errors times the other factor.
* slopes: sums and products of a few such, bounded by 1.13: 512 H.
* gradients of products take dz in 16 bits: H(t) of the terms' magnitude besides the sum's (n + 16) H.
* norm: squares in fp64, so rstd within 2 H; y two more products: 6 H. Gradient: two rounded products a term, sums of n
  in chains of 32 and 11 levels: 64 H of the terms' magnitude; dweight: chains of at most rows / 256 + 40 roundings.
* column sums: chains of 8, 8 and rows / 64 / 32 + 16 roundings: (rows / 2048 + 40) H of the terms' magnitude.
"""
import ctypes
import math
import sys
import zlib

import pytest
import torch

import oracle.ffn_oracle as FO
from ffn_cases import GATED, LINEAR
from moe_matmul_amd import _ffn_binding as c
from moe_matmul_amd import ffn, moe

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
H16 = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
H = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
ACTS = [None, "relu", "silu", "gelu"]


@pytest.fixture(autouse=True)
def announce(request):
    print(f"[gpu-case] {request.node.name}", flush=True)
    sys.stdout.flush()
    # what is allocated next holds NaN: an operator that reads what it has not written shows
    held = [torch.full((n,), math.nan, device="cuda") for n in (1 << 10, 1 << 12, 1 << 14, 1 << 16, 1 << 22, 1 << 25) for _ in range(8)]
    del held
    yield
    torch.cuda.synchronize()


def rng(*key):
    g = torch.Generator("cuda")
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return lambda *shape: torch.randn(*shape, device="cuda", generator=g)


def close(got, want, bound=0.0):
    """Within bound + half a step of got's type, NaN and infinities alike; beyond the type's range infinite."""
    t = got.dtype
    assert got.shape == want.shape
    g = got.double()
    assert torch.equal(g.isnan(), want.isnan())
    big = torch.finfo(t).max
    ok = ~want.isnan()
    g, w = g[ok].clamp(-big, big), want[ok].clamp(-big, big)
    bound = bound.expand_as(want)[ok] if isinstance(bound, torch.Tensor) else bound
    worst = (g - w).abs() - (bound * (1 + H16[t]) + H16[t] * w.abs() + TINY[t])
    assert worst.numel() == 0 or float(worst.max()) <= 0, f"off by {float(worst.max())} beyond the tolerance"


def same(a, b):
    """Bit for bit."""
    assert a.dtype == b.dtype and a.shape == b.shape
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    assert torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def act_error(z, bz, kind):
    """Error of act(z) for an error bz of z."""
    return 1.13 * bz + 256 * H * FO.activation(z, kind).abs() + 2.0 ** -119 if kind else bz


def linear_bounds(x, w, b, kind, residual):
    """(y, z, their errors before the last rounding)."""
    y, z = FO.linear(x, w, b, kind, residual)
    bz = (x.shape[1] + 16) * H * (x.abs() @ w.abs().T + (0 if b is None else b.abs()))
    by = act_error(z, bz, kind) + 2 * H * y.abs() + (0 if residual is None else H * residual.abs())
    return y, z, by, bz


# ---- rows in 8 bits ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,n", [(1, 32), (3, 96), (64, 64), (1000, 2048), (257, 7168), (5, 1 << 20)])
def test_rows8(rows, n, dtype):
    r = rng(rows, n, dtype)
    x = (r(rows, n) * torch.exp2(r(rows, n // 32).mul(6).round().repeat_interleave(32, 1))).to(TYPES[dtype])
    got = ffn.quantize8(x)
    codes, scales = FO.rows8(x.double())
    assert torch.equal(got.scales, scales) and torch.equal(got.codes & 127, codes & 127)
    number = (codes & 127 != 0) & (codes & 127 != 127)  # signs, but for those of 0 and NaN (of values beyond fp16)
    assert torch.equal(got.codes[number], codes[number])
    for t in TYPES.values():
        want = FO.values8(codes, scales)
        assert torch.equal(ffn.dequantize8(got, dtype=t).nan_to_num(nan=3.0), want.to(t).nan_to_num(nan=3.0))
    wide = torch.full((rows, n + 24), math.nan, device="cuda", dtype=TYPES[dtype])
    wide[:, 8:8 + n] = x
    again = ffn.quantize8(wide[:, 8:8 + n])
    same(again.codes, got.codes)
    same(again.scales, got.scales)
    out = torch.full((rows, n + 8), 7.0, device="cuda", dtype=TYPES[dtype])
    ffn.dequantize8(got, out=out[:, :n])
    same(out[:, :n], ffn.dequantize8(got, dtype=TYPES[dtype]))
    assert bool((out[:, n:] == 7).all())


def test_rows8_borders():
    """Ties between codes, E4M3's subnormals, largest elements on both sides of 448 times a power of two, the smallest
    scale, infinities and NaN."""
    grid = FO.values8(torch.arange(127, device="cuda", dtype=torch.uint8).repeat_interleave(32).view(1, -1),
                      torch.full((1, 127), 127, device="cuda", dtype=torch.uint8))[0, ::32]
    ties = (grid[1:] + grid[:-1]) / 2
    for v in (grid, ties, ties * (1 + 2.0 ** -20), ties * (1 - 2.0 ** -20)):
        x = torch.zeros(v.numel(), 32, device="cuda", dtype=torch.float64)
        x[:, 0], x[:, 5], x[:, 17] = v, 448, -v
        x = x.float()
        got, want = ffn.quantize8(x), FO.rows8(x.double())
        assert torch.equal(got.scales, want[1]) and torch.equal(FO.values8(*got), FO.values8(*want))
    tops = torch.tensor([448, 448 * (1 + 2.0 ** -23), 449, 896, 897, 2.0 ** -118, 448 * 2.0 ** -126, 2.0 ** -126, 2.0 ** -149, 0,
                         3e38, math.inf, -math.inf, math.nan], dtype=torch.float64, device="cuda")
    x = torch.zeros(tops.numel(), 64, device="cuda")
    x[:, 3], x[:, 4] = tops.float(), tops.float() / 3
    x[:, 40] = 1
    got, want = ffn.quantize8(x), FO.rows8(x.double())
    assert torch.equal(got.scales, want[1])
    assert torch.equal(FO.values8(*got).nan_to_num(nan=12345.0), FO.values8(*want).nan_to_num(nan=12345.0))
    v = ffn.dequantize8(got, dtype=torch.float32)
    assert bool(v[-3:, :32].isnan().all()) and bool((v[:, 32:].sum(1) == 1).all())


# ---- the norm --------------------------------------------------------------------------

NORM = [(1, 1), (1, 7168), (3, 5), (2, 64), (7, 96), (300, 512), (600, 513), (1, 8200), (3, 16384), (700, 1000), (2, 65536), (65, 65535),
        (1030, 2048), (4, 33)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,n", NORM)
def test_rmsnorm(rows, n, dtype):
    t, r = TYPES[dtype], rng(rows, n, dtype)
    x, residual, weight = (r(rows, n) * 3).to(t), r(rows, n).to(t), r(n)
    dy, dsum = r(rows, n).to(t), r(rows, n).to(t)
    for use_residual, w in ((True, weight), (False, weight.to(t)), (True, None)):
        got = ffn.rmsnorm(x, w, residual=residual if use_residual else None, eps=1e-5)
        total = (x.float() + residual.float()).to(t) if use_residual else x
        same(got.sum, total)
        w64 = None if w is None else w.double()
        y, rstd = FO.rmsnorm(total.double(), w64, 1e-5)
        close(got.rstd, rstd, 2 * H * rstd.abs())
        close(got.y, y, 6 * H * y.abs())
        s, d = total.double(), dy.double()
        dx, dweight = ffn.rmsnorm_backward(dy, got.sum, w, got.rstd, dsum=dsum if use_residual else None)
        want, want_w = FO.rmsnorm_backward(d, s, w64, rstd, dsum.double() if use_residual else None)
        g, h = (d if w is None else d * w64).abs(), (s * rstd.unsqueeze(1)).abs()
        terms = rstd.unsqueeze(1) * (g + h * (g * h).mean(1, keepdim=True)) + (dsum.double().abs() if use_residual else 0)
        close(dx, want, 64 * H * terms)
        if w is None:
            assert dweight is None
        else:
            assert dweight.dtype == w.dtype
            close(dweight, want_w, (rows / 256 + 40) * H * (d * s * rstd.unsqueeze(1)).abs().sum(0))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,n", [(1, 32), (5, 96), (300, 7168), (1200, 512), (3, 65536)])
def test_rmsnorm_in_8_bits(rows, n, dtype):
    t, r = TYPES[dtype], rng(rows, n, dtype, 8)
    x, residual, weight = (r(rows, n) * 3).to(t), r(rows, n).to(t), r(n)
    got = ffn.rmsnorm(x, weight, residual=residual, rows8=True)
    alone = ffn.rmsnorm(x, weight, residual=residual, rows=False, rows8=True)
    assert alone.y is None
    same(alone.y8.codes, got.y8.codes)
    same(alone.y8.scales, got.y8.scales)
    if t == torch.float32:  # what is in 8 bits is then y itself
        codes, scales = FO.rows8(got.y.double())
        assert torch.equal(got.y8.scales, scales) and torch.equal(FO.values8(*got.y8), FO.values8(codes, scales))
    else:  # codes of a y that is 6 H off: those of both ends, or between
        y = FO.rmsnorm(got.sum.double(), weight.double(), 1e-6)[0]
        (cl, sl), (ch, sh) = FO.rows8(y * (1 - 6 * H)), FO.rows8(y * (1 + 6 * H))
        ends = torch.stack((FO.values8(cl, sl), FO.values8(ch, sh)))
        v = FO.values8(*got.y8)
        sure = (sl == sh).repeat_interleave(32, 1)
        assert bool(((v >= ends.amin(0)) & (v <= ends.amax(0)) | ~sure).all()) and float((~sure).double().mean()) < 0.01
        assert float((v - y).norm() / y.norm()) < 2.0 ** -4


def test_rmsnorm_edges():
    one = torch.ones(64, device="cuda")
    for t in (torch.float32, torch.bfloat16):  # elements whose squares leave fp32
        for scale in (1e30, 1e-30):
            x = (torch.arange(1, 129, device="cuda").view(2, 64) * scale).to(t)
            got = ffn.rmsnorm(x, one, eps=0.0)
            y, rstd = FO.rmsnorm(x.double(), one.double(), 0.0)
            close(got.y, y, 6 * H * y.abs())
            close(got.rstd, rstd, 2 * H * rstd)
    x = torch.zeros(3, 64, device="cuda", dtype=torch.bfloat16)
    x[1, 5], x[2, 6] = math.nan, math.inf
    got = ffn.rmsnorm(x, one)
    assert bool((got.y[0] == 0).all()) and bool(got.y[1].isnan().all()) and bool(got.y[2, 6].isnan()) and float(got.rstd[2]) == 0
    # in place of x or the residual nothing is written; rows apart, and from an odd element on
    base = torch.full((5, 200), math.nan, device="cuda", dtype=torch.float16)
    x = rng(3)(5, 64).half()
    base[:, 3:67], base[:, 100:164] = x, x * 2
    got, want = ffn.rmsnorm(base[:, 3:67], one, residual=base[:, 100:164]), ffn.rmsnorm(x, one, residual=x * 2)
    close(got.y, want.y.double(), 2.0 ** -10 * want.y.double().abs())
    same(got.sum, want.sum)
    empty = ffn.rmsnorm(x[:0], one, rows8=True)
    assert empty.y.shape == (0, 64) and empty.y8.scales.shape == (0, 2)
    dx, dw = ffn.rmsnorm_backward(x[:0], x[:0], one, empty.rstd)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


def test_rmsnorm_gradient_against_differences():
    """The kernels' own forward pass in fp32, whose central differences of step 2^-6 are within 2^-12 of its slope's
    scale (third derivatives) and 2^-24 * 2^6 of its value's (rounding)."""
    r = rng(77)
    x, w, dy = r(2, 40), r(40), r(2, 40)
    n = ffn.rmsnorm(x, w)
    dx, dw = ffn.rmsnorm_backward(dy, n.sum, w, n.rstd)
    loss = lambda: float((ffn.rmsnorm(x, w).y.double() * dy.double()).sum())  # noqa: E731
    scale = float(dy.double().abs().sum())
    for at, g in ((x, dx), (w, dw)):
        flat = at.view(-1)
        for i in range(0, flat.numel(), 7):
            keep = flat[i].clone()
            flat[i] = keep + 2.0 ** -6
            up = loss()
            flat[i] = keep - 2.0 ** -6
            down = loss()
            flat[i] = keep
            assert abs((up - down) * 2.0 ** 5 - float(g.view(-1)[i])) < 2.0 ** -12 * scale


# ---- products -----------------------------------------------------------------------------

def setting(i):
    """One of the epilogues' combinations for the i-th size."""
    return dict(act=ACTS[i % 4], bias=(None, "fp32", "same")[i % 3], residual=i % 5 in (1, 2))


@pytest.mark.parametrize("i", range(len(LINEAR)), ids=lambda i: "x".join(map(str, LINEAR[i])))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_linear_and_its_gradients(i, dtype):
    (m, n, k), t, how = LINEAR[i], TYPES[dtype], setting(i + (dtype == "fp16"))
    r = rng(m, n, k, dtype)
    x, w, dy = r(m, k).to(t), (r(n, k) * k ** -0.5).to(t), r(m, n).to(t)
    bias = None if how["bias"] is None else r(n) if how["bias"] == "fp32" else r(n).to(t)
    residual = r(m, n).to(t) if how["residual"] else None
    f = lambda v: None if v is None else v.double()  # noqa: E731
    y, z = ffn.linear(x, w, bias=bias, activation=how["act"], residual=residual, save=True)
    same(ffn.linear(x, w, bias=bias, activation=how["act"], residual=residual), y)
    want, want_z, by, bz = linear_bounds(f(x), f(w), f(bias), how["act"], f(residual))
    close(z, want_z, bz)
    close(y, want, by)
    dx, dw, dbias = ffn.linear_backward(dy, x, w, bias=bias, z=z, activation=how["act"])
    wx, ww, wb, dz = FO.linear_backward(f(dy), f(x), f(w), f(z), how["act"])
    a, hz = dz.abs(), H16[t] if how["act"] else 0.0
    slack = 512 * H * f(dy).abs() if how["act"] else torch.zeros_like(dz)
    tiny = TINY[t] if how["act"] else 0.0
    err = hz * a + slack + tiny
    close(dx, wx, (n + 16) * H * (a @ f(w).abs()) + err @ f(w).abs())
    close(dw, ww, (m + 16) * H * (a.T @ f(x).abs()) + err.T @ f(x).abs())
    if bias is None:
        assert dbias is None
    else:
        assert dbias.dtype == bias.dtype
        close(dbias, wb, (m / 2048 + 40) * H * a.sum(0) + slack.sum(0))
    dw32 = torch.full((n, k), 7.0, device="cuda")
    assert ffn.linear_backward(dy, x, w, z=z, activation=how["act"], dw=dw32)[1] is dw32
    close(dw32, ww, (m + 16) * H * (a.T @ f(x).abs()) + err.T @ f(x).abs())
    same(dw32.to(t), dw)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("i", range(len(GATED)), ids=lambda i: "x".join(map(str, GATED[i])))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated_and_its_gradients(i, dtype, act):
    if (i + ("relu", "silu", "gelu").index(act)) % 3 and i > 8:
        act = "silu"
    (m, inner, k), t = GATED[i], TYPES[dtype]
    r, n = rng(m, inner, k, dtype), 2 * inner
    x, w, dh = r(m, k).to(t), (r(n, k) * k ** -0.5).to(t), r(m, inner).to(t)
    f = lambda v: v.double()  # noqa: E731
    h, kept = ffn.gated(x, w, activation=act, save="rows")
    want, z = FO.gated(f(x), f(w), act)
    bz = (k + 16) * H * (f(x).abs() @ f(w).abs().T)
    close(kept, z, bz)
    (g, u), (bg, bu) = z.chunk(2, 1), bz.chunk(2, 1)
    ba = act_error(g, bg, act)
    bh = ba * (u.abs() + bu) + FO.activation(g, act).abs() * bu + 2 * H * want.abs()
    close(h, want, bh)
    close(ffn.gated(x, w, activation=act), want, bh)
    keeps = [("rows", kept, x)]
    if inner % 32 == 0 and k % 32 == 0:
        h8, kept8 = ffn.gated(x, w, activation=act, save="rows8")
        close(h8, want, bh)
        values = FO.values8(*kept8)
        # E4M3's half step of the value, or of its smallest normal number under the block's scale
        close(values.float(), z, bz * 1.1 + 2.0 ** -4 * z.abs() + torch.exp2(kept8.scales.double() - 127).repeat_interleave(32, 1) * 2.0 ** -10)
        keeps.append(("rows8", kept8, ffn.quantize8(x)))
    keeps.append(("none", None, x))
    for name, k_, x_ in keeps:
        dx, dw = ffn.gated_backward(dh, x_, w, k_, activation=act)
        zk = z if k_ is None else f(kept) if name == "rows" else FO.values8(*k_)
        xk = FO.values8(*x_) if isinstance(x_, ffn.Rows8) else f(x_)
        dz = FO.gated_dz(f(dh), zk, act)
        gk, uk = zk.chunk(2, 1)
        size = torch.cat((f(dh).abs() * uk.abs(), f(dh).abs() * FO.activation(gk, act).abs()), 1)
        err = H16[t] * dz.abs() + 512 * H * size + TINY[t]
        if k_ is None:
            # g and u of fp32 sums: their errors through dh u act'(g) and dh act(g); slopes of slopes are at most 1.13 too
            d = f(dh).abs()
            err = err + torch.cat((d * (1.13 * bu + 1.13 * bg * (u.abs() + bu)), d * 1.13 * bg), 1)
        a = dz.abs() + err
        close(dx, dz @ f(w), (n + 16) * H * (a @ f(w).abs()) + err @ f(w).abs())
        close(dw, dz.T @ xk, (m + 16) * H * (a.T @ xk.abs()) + err.T @ xk.abs())
        dw32 = torch.empty(n, k, device="cuda")
        ffn.gated_backward(dh, x_, w, k_, activation=act, dw=dw32)
        same(dw32.to(t), dw)


# ---- by experts --------------------------------------------------------------------------------

def pick(r, tokens, topk, experts, dropped=0.0, only=None):
    ids = torch.rand(tokens, experts, device="cuda").argsort(1)[:, :topk].to(torch.int32) if only is None else \
        torch.full((tokens, topk), only, device="cuda", dtype=torch.int32)
    return torch.where(r(tokens, topk).abs() < dropped, -1, ids).to(torch.int32)


# tokens, topk, experts, inner, hidden, share of slots dropped, the only expert
EXPERTS = [(1, 1, 1, 32, 32, 0.0, None), (5, 2, 4, 32, 64, 0.0, None), (1, 4, 8, 64, 4096, 0.0, None), (33, 2, 8, 96, 160, 0.3, None),
           (64, 2, 3, 64, 96, 0.0, 1), (300, 4, 64, 64, 128, 0.2, None), (257, 3, 5, 160, 288, 0.0, None), (100, 2, 512, 32, 32, 0.0, None),
           (700, 2, 4, 256, 512, 0.1, None), (40, 1, 2, 512, 2048, 2.0, None), (20, 1, 2, 64, 64, 99.0, None), (1500, 2, 8, 512, 1024, 0.1, None),
           (2100, 2, 2, 1024, 512, 0.0, 0)]


@pytest.mark.parametrize("i", range(len(EXPERTS)), ids=lambda i: "-".join(map(str, EXPERTS[i])))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_experts(i, dtype):
    """The gated projections and a product with bias, activation and residual by a plan, with their gradients, against
    each expert's rows by themselves."""
    tokens, topk, experts, inner, hidden, dropped, only = EXPERTS[i]
    t, r = TYPES[dtype], rng(*EXPERTS[i], dtype)
    x = r(tokens, hidden).to(t)
    w1, w2 = (r(experts, 2 * inner, hidden) * hidden ** -0.5).to(t), (r(experts, hidden, inner) * inner ** -0.5).to(t)
    bias = r(experts, hidden).to(t)
    p = moe.plan(pick(r, tokens, topk, experts, dropped, only), experts)
    rows = p.rows
    h, kept = ffn.gated(x, w1, plan=p, save="rows")
    h8, kept8 = ffn.gated(x, w1, plan=p, save="rows8")
    residual, dy = r(rows, hidden).to(t), r(rows, hidden).to(t)
    y, z = ffn.linear(h, w2, bias=bias, activation="gelu", residual=residual, plan=p, save=True)
    dh, dw2, dbias = ffn.linear_backward(dy, h, w2, bias=bias, z=z, activation="gelu", plan=p)
    dx, dw1 = ffn.gated_backward(dh, x, w1, kept, plan=p)
    x8 = ffn.quantize8(x)
    dx8, dw8 = ffn.gated_backward(dh, x8, w1, kept8, plan=p)
    dxn, dwn = ffn.gated_backward(dh, x, w1, None, plan=p)
    assert h.shape == (rows, inner) and dx.shape == (tokens, hidden)
    f = lambda v: v.double()  # noqa: E731
    offsets = p.offsets.tolist()
    sum_x, sum_x8, mag = torch.zeros(tokens, hidden, device="cuda", dtype=torch.float64), None, None
    sum_x8, mag, mag8 = sum_x.clone(), sum_x.clone(), sum_x.clone()
    for e in range(experts):
        at = slice(offsets[e], offsets[e + 1])
        token = p.row_slots[at].long() // topk
        want, zg = FO.gated(f(x)[token], f(w1[e]))
        bz = (hidden + 16) * H * (f(x)[token].abs() @ f(w1[e]).abs().T)
        (g, u), (bg, bu) = zg.chunk(2, 1), bz.chunk(2, 1)
        bh = act_error(g, bg, "silu") * (u.abs() + bu) + FO.activation(g, "silu").abs() * bu + 2 * H * want.abs()
        close(kept[at], zg, bz)
        close(h[at], want, bh)
        close(h8[at], want, bh)
        wy, wz, by, bzz = linear_bounds(f(h[at]), f(w2[e]), f(bias[e]), "gelu", f(residual[at]))
        close(z[at], wz, bzz)
        close(y[at], wy, by)
        wx, ww, wb, dz = FO.linear_backward(f(dy[at]), f(h[at]), f(w2[e]), f(z[at]), "gelu")
        err = H16[t] * dz.abs() + 512 * H * f(dy[at]).abs() + TINY[t]
        a = dz.abs() + err
        m = dz.shape[0]
        close(dh[at], wx, (hidden + 16) * H * (a @ f(w2[e]).abs()) + err @ f(w2[e]).abs())
        close(dw2[e], ww, (m + 16) * H * (a.T @ f(h[at]).abs()) + err.T @ f(h[at]).abs())
        close(dbias[e], wb, (m / 2048 + 40) * H * a.sum(0) + 512 * H * f(dy[at]).abs().sum(0))
        for zk, xk, got_w, total, size in ((f(kept[at]), f(x)[token], dw1, sum_x, mag),
                                           (FO.values8(kept8.codes[at], kept8.scales[at]), FO.values8(*x8)[token], dw8, sum_x8, mag8)):
            dz = FO.gated_dz(f(dh[at]), zk)
            gk, uk = zk.chunk(2, 1)
            terms = torch.cat((f(dh[at]).abs() * uk.abs(), f(dh[at]).abs() * FO.activation(gk, "silu").abs()), 1)
            err = H16[t] * dz.abs() + 512 * H * terms + TINY[t]
            a = dz.abs() + err
            close(got_w[e], dz.T @ xk, (m + 16) * H * (a.T @ xk.abs()) + err.T @ xk.abs())
            row = dz @ f(w1[e])
            total.index_add_(0, token, row)
            # each row's error, its rounding to 16 bits, and the sum's roundings
            size.index_add_(0, token, (2 * inner + 16) * H * (a @ f(w1[e]).abs()) + err @ f(w1[e]).abs() + (H16[t] + 4 * topk * H) * row.abs() + TINY[t])
    close(dx, sum_x, mag * (1 + H16[t]))
    close(dx8, sum_x8, mag8 * (1 + H16[t]))
    assert float((dxn - dx).double().norm()) <= 2.0 ** -6 * float(dx.double().norm())
    assert float((dwn - dw1).double().norm()) <= 2.0 ** -6 * float(dw1.double().norm())
    end = offsets[-1]
    for v in (h, kept, y, z, dh):
        assert bool((v[end:] == 0).all())
    assert bool((FO.values8(*kept8)[end:] == 0).all())
    # given outputs keep the rows of no expert
    for call, width in ((lambda o: ffn.gated(x, w1, plan=p, out=o), inner), (lambda o: ffn.linear(h, w2, plan=p, out=o), hidden)):
        out = torch.full((rows, width), math.nan, device="cuda", dtype=t)
        call(out)
        assert bool(out[end:].isnan().all()) and not bool(out[:end].isnan().any())
    out = torch.empty(rows, inner, device="cuda", dtype=t)
    same(ffn.gated(x, w1, plan=p, out=out, save="rows")[1], kept)
    again8 = ffn.gated(x, w1, plan=p, out=out, save="rows8")[1]
    same(again8.codes, kept8.codes)
    assert bool((FO.values8(*again8)[end:] == 0).all())
    out = torch.empty(rows, hidden, device="cuda", dtype=t)
    same(ffn.linear(h, w2, bias=bias, activation="gelu", residual=residual, plan=p, out=out, save=True)[1], z)


@pytest.mark.parametrize("rows", [1, 2, 7, 8])
@pytest.mark.parametrize("k", [8, 56, 1992, 2048, 2056, 8184, 8192, 8200, 16384, 24616])
def test_few_rows_of_any_length(rows, k):
    """One chunk of k, several, and ragged last ones; captured by the first call of its kind."""
    r = rng(rows, k)
    x, w = r(rows, k).bfloat16(), (r(48, k) * k ** -0.5).bfloat16()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = ffn.linear(x, w), ffn.gated(x, w)
    graph.replay()
    f = lambda v: v.double()  # noqa: E731
    bz = (k + 16) * H * (f(x).abs() @ f(w).abs().T)
    z = f(x) @ f(w).T
    close(y, z, bz)
    (g, u), (bg, bu) = z.chunk(2, 1), bz.chunk(2, 1)
    want = FO.gated(f(x), f(w))[0]
    close(h, want, act_error(g, bg, "silu") * (u.abs() + bu) + FO.activation(g, "silu").abs() * bu + 2 * H * want.abs())
    p = moe.plan(torch.arange(rows, device="cuda", dtype=torch.int32).view(-1, 1) % 3, 3)
    w3 = torch.stack((w, w * 2, w * 4))
    rows_of = p.row_slots.long()
    scale = torch.tensor([1.0, 2.0, 4.0], device="cuda", dtype=torch.float64)[rows_of % 3].unsqueeze(1)
    same(ffn.linear(x[rows_of].contiguous(), w3, plan=p), (f(ffn.linear(x, w))[rows_of] * scale).bfloat16())


# tokens, topk, experts, inner, hidden, share of slots dropped, the only expert: up to 4 rows an expert, of which many or
# few have any, some more than one pass takes, and k that 16 waves and fewer share
FEW = [(1, 8, 64, 1024, 256, 0.0, None), (3, 8, 256, 264, 520, 0.3, None), (64, 4, 64, 504, 72, 0.0, None), (60, 4, 300, 136, 2048, 0.1, None),
       (13, 4, 16, 4096, 1000, 0.0, None), (1, 1, 8, 8, 8, 0.0, None), (32, 4, 32, 2056, 2056, 0.5, None), (50, 1, 64, 512, 136, 0.2, 63),
       (2, 16, 256, 8, 24576, 0.0, None), (30, 1, 16, 1032, 40, 99.0, None), (1, 1, 1, 28680, 136, 0.0, None), (8, 1, 1, 40000, 1024, 0.0, None)]


@pytest.mark.parametrize("i", range(len(FEW)), ids=lambda i: "-".join(map(str, FEW[i])))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_few_rows_of_many_experts(i, dtype):
    tokens, topk, experts, inner, hidden, dropped, only = FEW[i]
    t, r = TYPES[dtype], rng(*FEW[i], dtype)
    x = r(tokens, hidden).to(t)
    w1, w2 = (r(experts, 2 * inner, hidden) * hidden ** -0.5).to(t), (r(experts, hidden, inner) * inner ** -0.5).to(t)
    bias = r(experts, hidden)
    p = moe.plan(pick(r, tokens, topk, experts, dropped, only), experts)
    h, kept = ffn.gated(x, w1, plan=p, save="rows")
    residual, dh = r(p.rows, hidden).to(t), r(p.rows, inner).to(t)
    y = ffn.linear(h, w2, bias=bias, activation="silu", residual=residual, plan=p)
    dx, dw = ffn.gated_backward(dh, x, w1, None, plan=p)
    f = lambda v: v.double()  # noqa: E731
    offsets = p.offsets.tolist()
    for e in range(experts):
        at = slice(offsets[e], offsets[e + 1])
        m = at.stop - at.start
        if not m:
            assert bool((dw[e] == 0).all())
            continue
        xe = f(x)[p.row_slots[at].long() // topk]
        want, zg = FO.gated(xe, f(w1[e]))
        bz = (hidden + 16) * H * (xe.abs() @ f(w1[e]).abs().T)
        (g, u), (bg, bu) = zg.chunk(2, 1), bz.chunk(2, 1)
        close(kept[at], zg, bz)
        close(h[at], want, act_error(g, bg, "silu") * (u.abs() + bu) + FO.activation(g, "silu").abs() * bu + 2 * H * want.abs())
        wy, _, by, _ = linear_bounds(f(h[at]), f(w2[e]), f(bias[e]), "silu", f(residual[at]))
        close(y[at], wy, by)
        # dz by way of dw: its rounding and its slopes' error as in the tests above
        d = f(dh[at]).abs()
        dz = FO.gated_dz(f(dh[at]), zg)
        size = torch.cat((d * u.abs(), d * FO.activation(g, "silu").abs()), 1)
        err = H16[t] * dz.abs() + 512 * H * size + TINY[t] + torch.cat((d * (1.13 * bu + 1.13 * bg * (u.abs() + bu)), d * 1.13 * bg), 1)
        close(dw[e], dz.T @ xe, (m + 16) * H * ((dz.abs() + err).T @ xe.abs()) + err.T @ xe.abs())
    end = offsets[-1]
    assert bool((h[end:] == 0).all()) and bool((kept[end:] == 0).all()) and bool((y[end:] == 0).all())


@pytest.mark.parametrize("counts,n,k,tiles", [
    ([320, 321, 0, 640, 641, 1, 33], 4096, 520, [320, 128]), ([320, 321, 0, 640, 641, 1, 33], 6144, 64, [320, 256]),
    ([64, 65, 0, 128, 129, 1, 33], 272, 64, [64, 128]), ([256, 257, 512, 513, 31, 2335], 2048, 64, [256, 256])])
def test_an_experts_tiles_share_its_rows(counts, n, k, tiles):
    """Rows of experts at the tiles' heights and beside them."""
    r, rows = rng(tuple(counts), n, k), sum(counts)
    assert c.nvfp4_ffn_product_parts(c.NVFP4_FFN_FORWARD, rows, n, k, len(counts))[0][1:3] == tuple(tiles)
    ids = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))[torch.randperm(rows)]
    p = moe.plan(ids.to("cuda", torch.int32).view(-1, 1), len(counts))
    x, w = r(rows, k).bfloat16(), (r(len(counts), n, k) * k ** -0.5).bfloat16()
    residual, dy = r(rows, n).bfloat16(), r(rows, n).bfloat16()
    y = ffn.linear(x, w, residual=residual, plan=p)
    h = ffn.gated(x, w, plan=p)
    dx, dw, _ = ffn.linear_backward(dy, x, w, plan=p)
    f = lambda v: v.double()  # noqa: E731
    offsets = p.offsets.tolist()
    assert [b - a for a, b in zip(offsets, offsets[1:])] == counts
    for e in range(len(counts)):
        at = slice(offsets[e], offsets[e + 1])
        want, _, by, _ = linear_bounds(f(x[at]), f(w[e]), None, None, f(residual[at]))
        close(y[at], want, by)
        xs = f(x)[p.row_slots[at].long()]
        want, z = FO.gated(xs, f(w[e]))
        (g, u), (bg, bu) = z.chunk(2, 1), ((k + 16) * H * (xs.abs() @ f(w[e]).abs().T)).chunk(2, 1)
        close(h[at], want, act_error(g, bg, "silu") * (u.abs() + bu) + FO.activation(g, "silu").abs() * bu + 2 * H * want.abs())
        close(dx[at], f(dy[at]) @ f(w[e]), (n + 16) * H * (f(dy[at]).abs() @ f(w[e]).abs()))
        close(dw[e], f(dy[at]).T @ f(x[at]), (counts[e] + 16) * H * (f(dy[at]).abs().T @ f(x[at]).abs()))


def test_a_plan_of_one_expert_is_dense():
    r = rng(5)
    x, w = r(300, 96).bfloat16(), r(1, 128, 96).bfloat16()
    p = moe.plan(torch.zeros(300, 1, dtype=torch.int32, device="cuda"), 1)
    same(ffn.gated(x, w, plan=p), ffn.gated(x, w[0]))
    same(ffn.linear(x, w, plan=p), ffn.linear(x, w[0]))


def test_tables_that_name_nothing_are_harmless():
    """Offsets beyond the rows or falling, slots out of range: nothing outside the outputs is written, and rows whose
    slot is none are those of a token of zeros."""
    r = rng(6)
    experts, tokens, topk, k, inner = 4, 40, 2, 64, 32
    x, w = r(tokens, k).bfloat16(), r(experts, 2 * inner, k).bfloat16()
    for offsets in ([0, 20, 40, 60, 500], [-7, 20, 10, 30, 80], [80, 60, 40, 20, 0], [0, 0, 0, 0, 80]):
        p = moe.plan(pick(r, tokens, topk, experts), experts)
        p.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
        p.row_slots[3], p.row_slots[5] = 1 << 30, -5
        room = torch.full((p.rows + 128, inner), 7.0, device="cuda", dtype=torch.bfloat16)
        ffn.gated(x, w, plan=p, out=room[64:-64])
        assert bool((room[:64] == 7).all()) and bool((room[-64:] == 7).all())
        dw = torch.full((experts + 2, 2 * inner, k), 7.0, device="cuda")
        ffn.gated_backward(r(p.rows, inner).bfloat16(), x, w, None, plan=p, dw=dw[1:-1])
        ffn.linear_backward(r(p.rows, 2 * inner).bfloat16(), r(p.rows, k).bfloat16(), w, bias=r(experts, 2 * inner), plan=p)
        assert bool((dw[0] == 7).all()) and bool((dw[-1] == 7).all())
    p = moe.plan(torch.zeros(tokens, 1, dtype=torch.int32, device="cuda"), experts)
    p.row_slots[3] = 1 << 20
    h = ffn.gated(x, w, plan=p)
    assert bool((h[3] == 0).all()) and not bool((h[4] == 0).all())


def test_tables_that_name_too_many_rows_stay_in_the_workspace():
    """Experts that overlap have more chunks of rows than the sums of bias gradients have room for, beside a launch that
    is rounded up (32768 chunks and more)."""
    rows, n, experts = 64 * 32768 + 128, 8, 4
    offsets = torch.tensor([0, rows, 0, rows, 0], dtype=torch.int32, device="cuda")
    plan = c.nvfp4_ffn_plan(experts, 1, offsets.data_ptr(), 0)
    dy, z = torch.ones(rows, n, device="cuda").bfloat16(), torch.ones(rows, n, device="cuda").bfloat16()
    dz, dbias = torch.zeros_like(z), torch.zeros(experts, n, device="cuda")
    need = c.nvfp4_ffn_dz_workspace_bytes(rows, n, experts)
    room = torch.full((need // 4 + 40000 * n,), 7.0, device="cuda")
    c.nvfp4_ffn_linear_dz(dy.data_ptr(), n, z.data_ptr(), c.NVFP4_FFN_RELU, dz.data_ptr(), dbias.data_ptr(), 1, 2, rows, n,
                          ctypes.byref(plan), room.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert bool((room[need // 4:] == 7).all())


# ---- strides, values that are none, types -----------------------------------------------------

@pytest.mark.parametrize("m,n,k", [(5, 48, 24), (70, 144, 200), (600, 272, 72), (2051, 512, 2048)])
def test_rows_apart_and_what_lies_between(m, n, k):
    """Rows in wider ones whose other elements are NaN, before, between and after."""
    r = rng(m, n, k, 3)

    def inside(v):
        wide = torch.full((v.shape[0] + 2, v.shape[1] + 24), math.nan, device="cuda", dtype=v.dtype)
        wide[1:-1, 8:8 + v.shape[1]] = v
        return wide[1:-1, 8:8 + v.shape[1]]

    x, w, residual, dy = r(m, k).bfloat16(), r(n, k).bfloat16(), r(m, n).bfloat16(), r(m, n).bfloat16()
    y, z = ffn.linear(x, w, residual=residual, activation="silu", save=True)
    same(ffn.linear(inside(x), w, residual=inside(residual), activation="silu"), y)
    for a, b in zip(ffn.linear_backward(inside(dy), inside(x), w, z=z, activation="silu", bias=w[:, 0].contiguous()),
                    ffn.linear_backward(dy, x, w, z=z, activation="silu", bias=w[:, 0].contiguous())):
        same(a, b)
    h = ffn.gated(x, w)
    same(ffn.gated(inside(x), w), h)
    for a, b in zip(ffn.gated_backward(inside(dy[:, :n // 2]), inside(x), w), ffn.gated_backward(dy[:, :n // 2].contiguous(), x, w)):
        same(a, b)


@pytest.mark.parametrize("m", [1, 20, 300])
def test_values_that_are_none_stay_in_their_row_and_column(m):
    r, n, k = rng(m, 9), 136, 200
    x, w = r(m, k).half(), r(n, k).half()
    clean = ffn.linear(x, w)
    x2, w2 = x.clone(), w.clone()
    x2[m // 2, 3], w2[7, 11] = math.nan, math.inf
    y = ffn.linear(x2, w2)
    assert bool(y[m // 2].isnan().all())
    rows = torch.arange(m, device="cuda") != m // 2
    cols = torch.arange(n, device="cuda") != 7
    same(y[rows][:, cols], clean[rows][:, cols])
    assert bool(y[rows][:, 7].isinf().all())
    dx, dw, _ = ffn.linear_backward(y.nan_to_num(0, 0, 0), x2, w)
    assert bool(dw[:, 3].isnan().all()) and not bool(dw[:, :3].isnan().any()) and not bool(dx.isnan().any())


def test_activations_at_their_limits():
    """Sums of one product each, so that z is what was given: infinities, far and small values."""
    z = torch.tensor([-math.inf, math.inf, math.nan, -2000.0, 2000.0, -110.0, -100.0, -90.0, -16.0, -14.0, -12.5, -1e-3, 0.0, 1e-3,
                      15.5, 90.0, 110.0, 6e-5], device="cuda").half()
    x = torch.zeros(z.numel(), 8, device="cuda", dtype=torch.float16)
    x[:, 0] = z
    w = torch.zeros(8, 8, device="cuda", dtype=torch.float16)
    w[:, 0] = 1
    z64 = x[:, :1].double().expand(-1, 8)
    for kind in ("relu", "silu", "gelu"):
        y, kept = ffn.linear(x, w, activation=kind, save=True)
        # infinity times a 0 of w is NaN: those rows by what the sum was
        inf = kept.isinf() | kept.isnan()
        want = FO.activation(torch.where(inf, kept.double(), z64), kind)
        close(y, want, 256 * H * want.abs() + 2.0 ** -119)
        dz = torch.empty_like(kept)
        dy = torch.ones_like(kept)
        kept2 = z.view(-1, 1).expand(-1, 8).contiguous()
        c.nvfp4_ffn_linear_dz(dy.data_ptr(), 8, kept2.data_ptr(), ffn._ACTIVATIONS[kind], dz.data_ptr(), 0, 0, 1, z.numel(), 8, None, 0, 0,
                              torch.cuda.current_stream().cuda_stream)
        close(dz, FO.slope(kept2.double(), kind), 512 * H)


def test_products_add_up():
    """Small whole numbers: products are exact, so dx and dw are the slopes of y along x and w to the last bit."""
    g = torch.Generator("cuda").manual_seed(3)
    ints = lambda *s: torch.randint(-3, 4, s, device="cuda", generator=g).bfloat16()  # noqa: E731
    for m, n, k in ((3, 16, 24), (70, 72, 40), (300, 136, 64)):
        x, w, dy, d, e = ints(m, k), ints(n, k), ints(m, n), ints(m, k), ints(n, k)
        dw = torch.empty(n, k, device="cuda")
        dx, _, _ = ffn.linear_backward(dy, x, w, dw=dw)
        f = lambda v: v.double()  # noqa: E731
        # y is below 2^8 * 9 and rounded, so the slopes go by the exact product of the change
        same(dx, (f(dy) @ f(w)).bfloat16())
        assert float((f(dx) * f(d)).sum() - (f(dy) * (f(d) @ f(w).T)).sum()) == float(((f(dx) - f(dy) @ f(w)) * f(d)).sum())
        assert float((f(dw) * f(e)).sum()) == float((f(dy) * (f(x) @ f(e).T)).sum())


def test_no_rows():
    w = torch.ones(64, 96, device="cuda", dtype=torch.bfloat16)
    x, dy = w[:0], torch.ones(0, 64, device="cuda", dtype=torch.bfloat16)
    assert ffn.linear(x, w).shape == (0, 64) and ffn.gated(x, w).shape == (0, 32)
    dx, dw, db = ffn.linear_backward(dy, x, w, bias=w[:, 0].contiguous())
    assert dx.shape == (0, 96) and bool((dw == 0).all()) and bool((db == 0).all())
    dx, dw = ffn.gated_backward(dy[:, :32].contiguous(), x, w)
    assert dx.shape == (0, 96) and bool((dw == 0).all())
    p = moe.plan(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 3)
    w3 = torch.ones(3, 64, 96, device="cuda", dtype=torch.bfloat16)
    assert ffn.gated(x, w3, plan=p).shape == (0, 32)
    dx, dw, db = ffn.linear_backward(dy, x, w3, bias=torch.ones(3, 64, device="cuda"), plan=p)
    assert bool((dw == 0).all()) and db.shape == (3, 64) and bool((db == 0).all())
    assert ffn.quantize8(x).codes.shape == (0, 96) and ffn.dequantize8(ffn.quantize8(x)).shape == (0, 96)


def test_refusals():
    b = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x, w, p = b(8, 64), b(32, 64), moe.plan(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 3)
    w3 = b(3, 32, 64)
    for call in (
            lambda: ffn.linear(x.float(), w.float()), lambda: ffn.linear(x, w.half()), lambda: ffn.linear(x, w[:, :32]),
            lambda: ffn.linear(x, w3), lambda: ffn.linear(x, w, plan=p), lambda: ffn.linear(b(7, 64), w3, plan=p),
            lambda: ffn.linear(x, b(4, 32, 64), plan=p), lambda: ffn.linear(x, w, bias=b(31)), lambda: ffn.linear(x, w, bias=b(32).half()),
            lambda: ffn.linear(x, w, residual=b(8, 31)), lambda: ffn.linear(x, w, residual=b(8, 32).float()),
            lambda: ffn.linear(x, w, out=b(8, 31)), lambda: ffn.linear(x, w, activation="tanh"), lambda: ffn.linear(x.t(), w),
            lambda: ffn.linear(x[:1].expand(8, 64), w), lambda: ffn.linear(x.cpu(), w), lambda: ffn.linear(x, w.cpu()),
            lambda: ffn.linear_backward(b(8, 32), x, w, activation="silu"), lambda: ffn.linear_backward(b(8, 31), x, w),
            lambda: ffn.linear_backward(b(8, 32), b(7, 64), w), lambda: ffn.linear_backward(b(8, 32), x, w, dw=b(31, 64)),
            lambda: ffn.linear_backward(b(8, 32), x, w, dw=b(32, 64).half()), lambda: ffn.linear_backward(b(8, 32), x, w3, plan=p, bias=b(32)),
            lambda: ffn.linear_backward(b(8, 32), x, w, z=b(8, 31), activation="relu"),
            lambda: ffn.gated(x, b(31, 64)), lambda: ffn.gated(x, w, activation=None), lambda: ffn.gated(x, w, save="8"),
            lambda: ffn.gated(x, b(48, 64), save="rows8"), lambda: ffn.gated(x, w3, plan=p), lambda: ffn.gated(x, w, out=b(8, 32)),
            lambda: ffn.gated_backward(b(8, 16), x, w, b(8, 31)), lambda: ffn.gated_backward(b(8, 15), x, w),
            lambda: ffn.gated_backward(b(8, 16), b(7, 64), w), lambda: ffn.gated_backward(b(8, 16), ffn.quantize8(b(7, 64)), w),
            lambda: ffn.rmsnorm(x, b(63)), lambda: ffn.rmsnorm(x, residual=b(8, 63)), lambda: ffn.rmsnorm(x, rows=False),
            lambda: ffn.rmsnorm(b(8, 40), rows8=True), lambda: ffn.rmsnorm(x.double()), lambda: ffn.quantize8(b(8, 40)),
            lambda: ffn.quantize8(x.double()), lambda: ffn.rmsnorm_backward(x, x, None, b(8)),
            lambda: ffn.dequantize8(ffn.quantize8(x), out=b(8, 63))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ffn.linear(b(8, 60), b(32, 60)), lambda: ffn.linear(b(8, 64), b(30, 64)), lambda: ffn.linear(b(8, 68)[:, :64], w),
                 lambda: ffn.linear(b(8, 80)[:, 4:68], w), lambda: ffn.gated(x, b(24, 64)), lambda: ffn.rmsnorm(x, eps=-1.0)):
        with pytest.raises(c.Nvfp4FfnError):
            call()


# ---- streams, graphs, a run together --------------------------------------------------------------

def block(s, p):
    """A training step of a feed-forward block: norm, gated projections, down projection, and all gradients; with a plan
    by experts and combined."""
    norm = ffn.rmsnorm(s["x"], s["norm"], residual=s["stream"], rows8=True)
    h, kept = ffn.gated(norm.y, s["w1"], plan=p, save="rows8")
    y = ffn.linear(h, s["w2"], plan=p, residual=None if p else norm.sum)
    out = moe.combine(y, s["weights"], p, residual=norm.sum, dtype=y.dtype) if p else y
    dout = s["dout"]
    dy = moe.combine_backward(dout, y, s["weights"], p)[0] if p else dout
    dh, dw2, _ = ffn.linear_backward(dy, h, s["w2"], plan=p)
    dnorm, dw1 = ffn.gated_backward(dh, norm.y8, s["w1"], kept, plan=p)
    dx, dweight = ffn.rmsnorm_backward(dnorm, norm.sum, s["norm"], norm.rstd, dsum=dout)
    return dict(out=out, dx=dx, dweight=dweight, dw1=dw1, dw2=dw2)


def block_state(seed, experts, tokens=70, hidden=256, inner=96, t=torch.bfloat16):
    r = rng(seed, experts)
    lead = (experts,) if experts else ()
    return dict(x=r(tokens, hidden).to(t), stream=r(tokens, hidden).to(t), norm=1 + 0.1 * r(hidden), dout=r(tokens, hidden).to(t),
                w1=(r(*lead, 2 * inner, hidden) * hidden ** -0.5).to(t), w2=(r(*lead, hidden, inner) * inner ** -0.5).to(t),
                weights=r(tokens, 2).abs(), ids=pick(r, tokens, 2, experts, 0.1) if experts else None)


def plan_of(s):
    return None if s["ids"] is None else moe.plan(s["ids"], s["w1"].shape[0])


@pytest.mark.parametrize("experts", [0, 4])
def test_a_block_against_torchs_gradients(experts):
    """All gradients of a block at once, against torch's own differentiation in fp64 of the same formulas. 8-bit rows are
    off by up to 2^-4 and about 2^-5.3 in the mean square; a gradient goes through one of x and one of g, u: 2^-4 in all."""
    s = block_state(1, experts)
    p = plan_of(s)
    got = block(s, p)
    leaf = {k: s[k].double().requires_grad_() for k in ("x", "norm", "w1", "w2")}
    total = (s["x"].float() + s["stream"].float()).bfloat16().double() + (leaf["x"] - leaf["x"].detach())
    n = total / (total.square().mean(1, keepdim=True) + 1e-6).sqrt() * leaf["norm"]
    if experts:
        out = total
        for e in range(experts):
            token, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
            g, u = (n[token] @ leaf["w1"][e].T).chunk(2, 1)
            y = (torch.nn.functional.silu(g) * u) @ leaf["w2"][e].T
            out = out.index_add(0, token, y * s["weights"].double()[token, slot].unsqueeze(1))
    else:
        g, u = (n @ leaf["w1"].T).chunk(2, 1)
        out = total + (torch.nn.functional.silu(g) * u) @ leaf["w2"].T
    out.backward(s["dout"].double())
    want = dict(out=out.detach(), dx=leaf["x"].grad, dweight=leaf["norm"].grad, dw1=leaf["w1"].grad, dw2=leaf["w2"].grad)
    for name, v in want.items():
        off = float((got[name].double() - v).norm() / v.norm())
        assert off < (2.0 ** -7 if name in ("out", "dw2") else 2.0 ** -4), (name, off)


@pytest.mark.parametrize("experts", [0, 4])
def test_a_captured_step_replays_on_new_inputs(experts):
    states = [block_state(i, experts) for i in range(4)]
    want = [{k: v.clone() for k, v in block(s, plan_of(s)).items()} for s in states]
    s = {k: None if v is None else v.clone() for k, v in states[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(s, plan_of(s))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(s, plan_of(s))
    for i in (1, 2, 3, 1, 0):
        for k, v in states[i].items():
            if v is not None:
                s[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for k in out:
            same(out[k], want[i][k])
        block(states[(i + 1) % 4], plan_of(states[(i + 1) % 4]))


@pytest.mark.parametrize("experts", [0, 4])
def test_steps_on_two_streams_at_once(experts):
    states = [block_state(10 + i, experts, tokens=200, hidden=512, inner=256) for i in range(2)]
    want = [block(s, plan_of(s)) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = block(states[i], plan_of(states[i]))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for k in w:
            same(g[k], w[k])


def apart(t, gap=24):
    """The same rows, further apart, in memory of NaN."""
    room = torch.full((t.shape[0], t.shape[1] + gap), math.nan, device="cuda", dtype=t.dtype)
    room[:, :t.shape[1]] = t
    return room[:, :t.shape[1]]


@pytest.mark.parametrize("tokens,hidden,inner", [(3, 64, 32), (70, 256, 160), (600, 512, 288)])
@pytest.mark.parametrize("experts", [0, 3])
def test_less_usual_forms_are_the_usual_ones(tokens, hidden, inner, experts):
    """Operands whose rows lie apart, rows in 8 bits in place of 16, gradients without what was kept, one tensor in two
    places: bit for bit as the usual call on the same values."""
    r = rng(tokens, hidden, inner, experts)
    lead = (experts,) if experts else ()
    p = moe.plan(pick(r, tokens, 2, experts, 0.2), experts) if experts else None
    rows = p.rows if experts else tokens
    x, w1 = r(tokens, hidden).bfloat16(), (r(*lead, 2 * inner, hidden) * hidden ** -0.5).bfloat16()
    w2, bias = (r(*lead, hidden, inner) * inner ** -0.5).bfloat16(), r(*lead, hidden).bfloat16()
    dh, dy, residual = r(rows, inner).bfloat16(), r(rows, hidden).bfloat16(), r(rows, hidden).bfloat16()
    q = ffn.quantize8(x)
    x = ffn.dequantize8(q)
    h, kept = ffn.gated(x, w1, plan=p, save="rows")
    for a, b in zip(ffn.gated(apart(x), w1, plan=p, save="rows"), (h, kept)):
        same(a, b)
    for k in (kept, None, ffn.gated(x, w1, plan=p, save="rows8")[1]):
        want = ffn.gated_backward(dh, x, w1, k, plan=p)
        for form in ((dh, q), (apart(dh), apart(x)), (apart(dh, 8), q)):
            for a, b in zip(ffn.gated_backward(*form, w1, k, plan=p), want):
                same(a, b)
    how = dict(bias=bias, activation="gelu", plan=p)
    y, z = ffn.linear(h, w2, residual=residual, save=True, **how)
    for a, b in zip(ffn.linear(apart(h), w2, residual=apart(residual, 8), save=True, **how), (y, z)):
        same(a, b)
    want = ffn.linear_backward(dy, h, w2, z=z, **how)
    for a, b in zip(ffn.linear_backward(apart(dy), apart(h), w2, z=z, **how), want):
        same(a, b)
    h8 = ffn.quantize8(h)
    for a, b in zip(ffn.linear_backward(dy, h8, w2, z=z, **how), ffn.linear_backward(dy, ffn.dequantize8(h8), w2, z=z, **how)):
        same(a, b)
    # without an activation dy takes the place of dz, and lies apart itself
    for a, b in zip(ffn.linear_backward(apart(dy), h, w2, bias=bias, plan=p), ffn.linear_backward(dy, h, w2, bias=bias, plan=p)):
        same(a, b)
    weight = r(hidden)
    n = ffn.rmsnorm(x, weight, residual=x, rows8=True)
    same(n.sum, (x.float() * 2).bfloat16())
    m = ffn.rmsnorm(apart(x), weight, residual=apart(x, 8), rows=False, rows8=True)
    same(m.y8.codes, n.y8.codes)
    same(m.y8.scales, n.y8.scales)
    same(m.sum, n.sum)
    assert m.y is None
    dn = r(tokens, hidden).bfloat16()
    want = ffn.rmsnorm_backward(dn, n.sum, weight, n.rstd, dsum=dn)
    for a, b in zip(ffn.rmsnorm_backward(apart(dn), apart(n.sum, 8), weight, n.rstd, dsum=apart(dn, 16)), want):
        same(a, b)
    same(ffn.rmsnorm_backward(dn, n.sum, None, n.rstd)[0], ffn.rmsnorm_backward(dn, n.sum, torch.ones_like(weight), n.rstd)[0])
    room = torch.full((tokens, hidden + 8), 7.0, device="cuda")
    ffn.dequantize8(q, out=room[:, :hidden])
    assert bool((room[:, hidden:] == 7).all()) and torch.equal(room[:, :hidden].bfloat16(), x)


def test_the_stream_argument():
    r = rng(4)
    x, w = r(300, 256).bfloat16(), r(512, 256).bfloat16()
    want = ffn.gated(x, w)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (st, st.cuda_stream):
        got = ffn.gated(x, w, stream=stream)
        st.synchronize()
        same(got, want)
    n = ffn.rmsnorm(x, stream=st)
    dx, _ = ffn.rmsnorm_backward(x, n.sum, None, n.rstd, stream=st)
    dx2, dw, _ = ffn.linear_backward(r(300, 512).bfloat16(), x, w, stream=st)
    q = ffn.dequantize8(ffn.quantize8(x, stream=st), stream=st)
    st.synchronize()
    assert dx.shape == x.shape and dx2.shape == x.shape and q.shape == x.shape and dw.shape == w.shape


def test_an_operand_beyond_32_bit_offsets():
    """Rows from 2^31 bytes on: 140000 rows of 16384, read in place at the far end."""
    rows, k = 140000, 16384
    x = torch.zeros(rows, k, device="cuda", dtype=torch.bfloat16)
    r = rng(12)
    w = (r(64, k) * k ** -0.5).bfloat16()
    x[-300:] = r(300, k).bfloat16()
    x[:5] = r(5, k).bfloat16()
    y = ffn.linear(x, w)
    for at in (slice(0, 5), slice(rows - 300, rows)):
        part = x[at].contiguous()
        close(y[at], part.double() @ w.double().T, (k + 16) * H * (part.double().abs() @ w.double().abs().T))
    assert bool((y[5:-300] == 0).all())
    dw = torch.empty(64, k, device="cuda")
    dx, _, _ = ffn.linear_backward(y, x, w, dw=dw)
    f = lambda v: v.double()  # noqa: E731
    ends = torch.cat((torch.arange(5), torch.arange(rows - 300, rows))).cuda()
    close(dw, f(y[ends]).T @ f(x[ends]), (rows + 16) * H * (f(y[ends]).abs().T @ f(x[ends]).abs()))
    close(dx[-300:], f(y[-300:]) @ f(w), 80 * H * (f(y[-300:]).abs() @ f(w).abs()))
    q = ffn.quantize8(x)
    same(q.codes[-3:], ffn.quantize8(x[-3:].contiguous()).codes)
    n = ffn.rmsnorm(x)
    same(n.y[-3:], ffn.rmsnorm(x[-3:].contiguous()).y)
