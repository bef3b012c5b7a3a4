"""GPU parity of the operators around the grouped GEMM (moe_matmul_amd.moe)
against the float64 oracle of oracle/moe_oracle.py.

Tolerances. H(t) is half a step of a type relative to the value: fp32 2^-24, fp16
2^-11, bf16 2^-8 (eps / 2). Whole numbers, NVFP4 codes and scales, and values
that fit their type are equal. fp32 results:
* weights: exp within 3 H, two divisions and a product 3 H, a sum of up to 512
  positive terms in chains of 32 and 6 levels 40 H: 64 H of the value, and what
  underflows (2^-126).
* d logits: four such factors: 256 H of the magnitude of the terms, and a half
  step of the result's type.
* combine: one rounding of weight * alpha and one for each slot: (topk + 2) H of
  the terms' magnitude, and a half step. d weights: chains of n / 256 and 10
  levels: (n / 256 + 12) H of the terms' magnitude.
* products of a few tokens: exact products, at most k + 8 roundings of partial
  sums, so (k + 16) H of the terms' magnitude (the scaling of bf16 rows adds
  2^-39 of the largest element, within the 16); silu(g) u carries the errors of g
  (slope at most 1.1) and u, and 16 H of its own.
"""
import sys

import numpy as np
import pytest
import torch

import moe_matmul_amd as mm
import oracle.moe_oracle as MO
from moe_matmul_amd import _moe_binding as c
from moe_matmul_amd import moe

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
H = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}  # least result step that counts


@pytest.fixture(autouse=True)
def announce(request):
    print(f"[gpu-case] {request.node.name}", flush=True)
    sys.stdout.flush()
    yield
    torch.cuda.synchronize()


def rng_of(*key):
    return np.random.default_rng([int(k) for k in key])


def gpu(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, want, bound, dtype):
    """Within bound + half a step of dtype, NaN and infinities alike."""
    g = f64(got)
    assert g.shape == want.shape
    assert np.array_equal(np.isnan(g), np.isnan(want))
    ok = ~np.isnan(want)
    big = float(torch.finfo(dtype).max)
    g, w = np.clip(g[ok], -big, big), np.clip(want[ok], -big, big)
    limit = np.broadcast_to(bound, want.shape)[ok] * (1 + H[dtype]) + H[dtype] * np.abs(w) + TINY[dtype]
    worst = np.max(np.abs(g - w) - limit, initial=-1.0)
    assert worst <= 0, f"off by {worst} beyond the tolerance"


# ---- routing ---------------------------------------------------------------------

ROUTE = [
    # tokens, experts, topk, dtype, options
    (1, 8, 2, "fp32", {}), (1, 256, 8, "fp32", dict(score="sigmoid", bias=True, groups=8, topk_groups=4, group_best=2)),
    (3, 1, 1, "bf16", {}), (65, 2, 2, "fp16", dict(score="sigmoid")), (64, 5, 3, "bf16", dict(renormalize=False)),
    (1000, 64, 6, "fp32", dict(renormalize=False)), (257, 100, 8, "bf16", dict(scale=2.5)),
    (33, 511, 16, "fp16", dict(score="sigmoid", renormalize=False)), (40, 512, 16, "fp32", dict(bias=True)),
    (9000, 60, 4, "bf16", dict(score="sigmoid", bias=True)), (70, 48, 5, "fp32", dict(groups=3, topk_groups=2, group_best=2)),
    (70, 512, 8, "bf16", dict(score="sigmoid", bias=True, groups=64, topk_groups=7, group_best=2)),
    (70, 64, 1, "fp16", dict(groups=64, topk_groups=1)), (50, 24, 12, "fp32", dict(groups=2, topk_groups=1, group_best=1)),
    (130, 160, 9, "bf16", dict(groups=5, topk_groups=2, group_best=2, bias=True, renormalize=False)),
    (17000, 16, 2, "fp32", {}), (5, 330, 16, "bf16", dict(groups=33, topk_groups=5, group_best=2)),
]


def route_case(tokens, experts, topk, dtype, options, seed=0):
    rng = rng_of(tokens, experts, topk, seed)
    x = gpu(rng.standard_normal((tokens, experts)) * 2, TYPES[dtype])
    how = dict(options)
    bias = rng.standard_normal(experts).astype(np.float32) * 0.1 if how.pop("bias", False) else None
    return x, bias, how


def check_route(x, topk, bias, how):
    ids, w = moe.route(x, topk, bias=None if bias is None else gpu(bias), **how)
    want_ids, want_w = MO.route(f64(x), topk, bias=None if bias is None else bias.astype(np.float64), **how)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    close(w, want_w, 64 * H[torch.float32] * np.abs(np.nan_to_num(want_w)), torch.float32)
    return ids, w


@pytest.mark.parametrize("tokens,experts,topk,dtype,options", ROUTE)
def test_route(tokens, experts, topk, dtype, options):
    x, bias, how = route_case(tokens, experts, topk, dtype, options)
    check_route(x, topk, bias, how)


@pytest.mark.parametrize("options", [{}, dict(score="sigmoid", bias=True), dict(groups=4, topk_groups=2, group_best=2),
                                     dict(renormalize=False), dict(score="sigmoid", renormalize=False)])
@pytest.mark.parametrize("dtype", TYPES)
def test_route_at_the_edges(dtype, options):
    """Masked experts and rows, ties, both zeros, the type's lowest and highest value, infinities and NaN."""
    t = TYPES[dtype]
    lowest, highest = torch.finfo(t).min, torch.finfo(t).max
    x = torch.randn(64, 16, generator=torch.Generator().manual_seed(5)).to(t)
    inf = float("inf")
    x[0] = -inf                                   # no expert left
    x[1] = -inf
    x[1, 11] = 0.5                                # one
    x[2, ::2] = -inf
    x[3] = 1.0                                    # all equal: the lowest indices
    x[4, :] = torch.tensor([0.0, -0.0] * 8)       # zeros are equal
    x[5] = lowest
    x[6] = lowest
    x[6, 3] = -inf
    x[7, 5] = highest
    x[8] = x[8, 0]
    x[8, 9] = float("nan")
    x[9] = float("nan")
    x[10, 2] = inf
    x[11, 4:] = -inf                              # fewer experts than slots
    x[12, :8] = x[12, 8:]
    x = x.cuda()
    how = dict(options)
    bias = rng_of(7).standard_normal(16).astype(np.float32) if how.pop("bias", False) else None
    if bias is not None:
        bias[6] = -np.inf                         # never chosen
    ids, w = check_route(x, 6, bias, how)
    assert (ids[0] == -1).all() and (w[0] == 0).all()
    assert torch.isnan(w[8]).any() and not torch.isnan(w[:8]).any()


@pytest.mark.parametrize("experts,topk,dtype,options", [
    (64, 6, "bf16", dict(score="sigmoid", bias=True)), (40, 4, "fp32", dict(groups=4, topk_groups=2, group_best=1)),
    (128, 8, "fp32", dict(score="sigmoid", bias=True, groups=8, topk_groups=4, group_best=2, renormalize=False)),
    (60, 10, "fp16", dict(groups=20, topk_groups=7, group_best=2, bias=True))])
def test_route_of_many_tokens_is_that_of_few(experts, topk, dtype, options):
    """Scores that are nearly or exactly equal, far apart, masked and not finite: in one call of 140000 tokens, and in
    calls of 2000 (which the oracle checks above)."""
    g = torch.Generator("cuda").manual_seed(experts)
    x = torch.randn(140000, experts, device="cuda", generator=g)
    x[1::5] = x[1::5] * 1e-5 + 0.5
    x[2::5] = x[2::5] * 20
    x[3::10, ::2] = x[3::10, 1::2]
    x.masked_fill_(torch.rand(x.shape, device="cuda", generator=g) < 0.05, float("-inf"))
    x[:200, 3], x[100:300, 5], x[400] = float("inf"), float("nan"), float("-inf")
    x = x.to(TYPES[dtype])
    how = dict(options)
    bias = torch.randn(experts, device="cuda", generator=g) * 1e-6 if how.pop("bias", False) else None
    ids, w = moe.route(x, topk, bias=bias, **how)
    for i in range(0, 140000, 2000):
        few_ids, few_w = moe.route(x[i:i + 2000], topk, bias=bias, **how)
        assert torch.equal(ids[i:i + 2000], few_ids)
        close(w[i:i + 2000], f64(few_w), 64 * H[torch.float32] * np.abs(np.nan_to_num(f64(few_w))), torch.float32)


def test_route_strides_alignment_and_outputs():
    base = torch.randn(40, 3 + 61 + 4, device="cuda").to(torch.bfloat16)
    x = base[:, 3:64]                             # odd offset, odd width, rows 68 apart
    ids = torch.full((40, 5), 77, dtype=torch.int32, device="cuda")
    w = torch.full((40, 5), float("nan"), device="cuda")
    got = moe.route(x, 5, ids=ids, weights=w)
    assert got[0] is ids and got[1] is w
    want_ids, want_w = MO.route(f64(x), 5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    close(w, want_w, 64 * H[torch.float32] * want_w, torch.float32)
    with pytest.raises(ValueError):
        moe.route(x.t(), 2)
    with pytest.raises(ValueError):
        moe.route(x, 5, ids=ids.long())
    with pytest.raises(ValueError):
        moe.route(x.double(), 5)
    with pytest.raises(ValueError):
        moe.route(x, 5, score="tanh")
    with pytest.raises(c.Nvfp4MoeError):
        moe.route(x, 62)
    assert moe.route(x[:0], 5)[0].shape == (0, 5)


@pytest.mark.parametrize("tokens,experts,topk,dtype,options", [r for r in ROUTE if not r[4].get("bias") and "groups" not in r[4]])
def test_route_backward(tokens, experts, topk, dtype, options):
    x, _, how = route_case(tokens, experts, topk, dtype, options, seed=1)
    ids, _ = moe.route(x, topk, **how)
    dw = torch.randn(tokens, topk, device="cuda")
    d = moe.route_backward(x, ids, dw, **how)
    want, size = MO.route_backward(f64(x), ids.cpu().numpy(), f64(dw), **how)
    close(d, want, 256 * H[torch.float32] * size, x.dtype)


def test_route_backward_of_masked_rows_and_strides():
    base = torch.randn(37, 50, device="cuda")
    x = base[:, 5:34]
    x[3] = float("-inf")
    x[4, 2:] = float("-inf")
    ids, _ = moe.route(x, 4, renormalize=False)
    dw = torch.randn(37, 4, device="cuda")
    dw[3] = float("nan")                          # of slots without an expert: not used
    dw[4, 2:] = float("nan")
    store = torch.full((37, 40), 9.0, device="cuda")
    d = moe.route_backward(x, ids, dw, renormalize=False, dlogits=store[:, 3:32])
    want, size = MO.route_backward(f64(x), ids.cpu().numpy(), f64(dw), renormalize=False)
    close(d, want, 256 * H[torch.float32] * size, torch.float32)
    assert (store[:, :3] == 9).all() and (store[:, 32:] == 9).all() and (d[3] == 0).all()


def test_route_backward_against_differences():
    """Of the kernel's own forward pass, at logits where the choice does not change."""
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            how = dict(score=score, renormalize=renormalize, scale=1.5)
            x = torch.arange(12, device="cuda").float().view(1, 12).mul(0.37).sin().mul(3).repeat(24, 1)
            dw = torch.randn(1, 5, device="cuda").repeat(24, 1)
            h = 2.0 ** -7
            step = torch.cat((torch.eye(12), -torch.eye(12))).cuda() * h
            ids, w = moe.route(x + step, 5, **how)
            assert (ids == ids[0]).all()
            loss = (w.double() * dw.double()).sum(1)
            diff = (loss[:12] - loss[12:]) / (2 * h)
            d = moe.route_backward(x[:1].contiguous(), ids[:1].contiguous(), dw[:1].contiguous(), **how)
            # central differences: h^2 / 6 of the third derivative (below 1.5 |dw| for these functions), and 64 H of the
            # weights (at most 1.5 times |dw|) over h
            size = float(dw[0].abs().sum()) * 1.5
            assert float((d[0].double() - diff).abs().max()) < h * h / 6 * size * 8 + 64 * 2.0 ** -24 * size * 2 / h


# ---- the plan --------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 8, 256), (63, 1, 7), (65, 3, 512), (1300, 3, 17), (4096, 2, 12), (2048, 8, 64), (8192, 2, 300),
                                                 (16385, 1, 5), (5000, 8, 256), (40000, 4, 33)])
def test_plan(tokens, topk, experts):
    rng = rng_of(tokens, topk, experts)
    ids = rng.integers(-2, experts + 2, (tokens, topk)).astype(np.int32)
    ids[rng.random(tokens) < 0.1] = rng.integers(0, experts)  # a run of one expert
    p = moe.plan(gpu(ids), experts)
    offsets, atoms, slot_rows, row_slots = MO.plan(ids, experts)
    for got, want in ((p.offsets, offsets), (p.atoms, atoms), (p.slot_rows, slot_rows), (p.row_slots, row_slots)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert c.nvfp4_moe_sf_bytes(tokens * topk, experts, 64) >= int(atoms[-1]) * 512


def test_plan_without_slots_and_its_tables():
    b, sfb = torch.zeros(3, 16, 32, dtype=torch.uint8, device="cuda"), torch.zeros(3, 512, dtype=torch.uint8, device="cuda")
    for ids in (np.zeros((0, 2), dtype=np.int32), np.full((4, 2), -1, dtype=np.int32), np.array([[2, 0], [2, 2]], dtype=np.int32)):
        rows = ids.size
        a = torch.zeros(rows, 32, dtype=torch.uint8, device="cuda")
        sfa = torch.zeros(c.nvfp4_moe_sf_bytes(rows, 3, 64), dtype=torch.uint8, device="cuda")
        q = moe.Product(a, sfa, b, sfb, torch.zeros(rows, 16, dtype=torch.float16, device="cuda"))
        p = moe.plan(gpu(ids), 3, (q,))
        offsets, atoms, _, _ = MO.plan(ids, 3)
        assert np.array_equal(p.offsets.cpu().numpy(), offsets) and np.array_equal(p.atoms.cpu().numpy(), atoms)
        raw = q._tables.cpu().numpy()
        at = [t - q.tables[0] for t in q.tables]
        sizes = raw[at[0]:at[0] + 48].view(np.int32).reshape(3, 4)
        assert np.array_equal(sizes, [[offsets[e + 1] - offsets[e], 16, 64, 1] for e in range(3)])
        abc = raw[at[1]:at[1] + 72].view(np.uint64).reshape(3, 3)
        sf = raw[at[2]:at[2] + 48].view(np.uint64).reshape(3, 2)
        for e in range(3):
            assert abc[e].tolist() == [a.data_ptr() + int(offsets[e]) * 32, b.data_ptr() + e * 16 * 32,
                                       q.out.data_ptr() + int(offsets[e]) * 32]
            assert sf[e].tolist() == [sfa.data_ptr() + int(atoms[e]) * 512, sfb.data_ptr() + e * 512]


# ---- NVFP4 ---------------------------------------------------------------------------------

def check_rows(a, sfa, v, k, atom=0):
    codes, scales = MO.quantize(v)
    got_codes, got_scales = MO.unpack_rows(a, sfa, v.shape[0], k, atom)
    assert np.array_equal(got_scales, scales)
    assert np.array_equal(got_codes, codes)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,k", [(1, 32), (3, 96), (15, 64), (16, 4096), (33, 7168 // 32 * 32), (127, 288), (128, 256), (129, 544),
                                 (300, 1056)])
def test_quantize(dtype, m, k):
    rng = rng_of(m, k)
    x = gpu(rng.standard_normal((m, k)) * np.exp(rng.uniform(-6, 6, (m, 1))), TYPES[dtype])
    a, sfa = moe.quantize(x)
    check_rows(a.cpu().numpy(), sfa.cpu().numpy(), f64(x), k)
    for out in TYPES.values():
        codes, scales = MO.quantize(f64(x))
        assert np.array_equal(f64(moe.dequantize(a, sfa, dtype=out)), MO.values(codes, scales))


@pytest.mark.parametrize("dtype,l,m,k", [("bf16", 1, 4099, 2080), ("fp16", 41, 131, 1632), ("fp32", 260, 33, 992)])
def test_quantize_of_many_rows(dtype, l, m, k):
    x = torch.randn(l, m, k, device="cuda", generator=torch.Generator("cuda").manual_seed(m)).to(TYPES[dtype])
    x[:, ::5] *= 1e-3
    a, sfa = moe.quantize(x)
    an, sn, xn = a.cpu().numpy(), sfa.cpu().numpy(), f64(x)
    for li in sorted({0, l // 2, l - 1}):
        check_rows(an[li], sn, xn[li], k, atom=li * -(-m // 128))
    values = moe.dequantize(a, sfa, dtype=torch.float32)
    for li in sorted({0, l // 2, l - 1}):
        rows = MO.unpack_rows(an[li], sn, m, k, li * -(-m // 128))
        assert np.array_equal(f64(values[li]), MO.values(*rows))


def test_dequantize_of_many_rows():
    """The way back of 2^26 elements and a few, to all types, against single batches' way back."""
    x = torch.randn(63, 1031, 1056, device="cuda", dtype=torch.float16, generator=torch.Generator("cuda").manual_seed(3))
    a, sfa = moe.quantize(x)
    per = mm.nvfp4_sf_bytes(1031, 1056)
    for out in TYPES.values():
        values = moe.dequantize(a, sfa, dtype=out)
        for li in (0, 1, 40, 62):
            assert torch.equal(values[li], moe.dequantize(a[li].clone(), sfa[li * per:(li + 1) * per].clone(), dtype=out))


def test_quantize_at_the_borders():
    """Quotients on and next to every border of both roundings, zeros, the smallest and largest scales, and saturation."""
    rows = []
    for s in list(MO.E4M3[1:12]) + [0.75, 1.0, 1.125, 1.875, 100.0, 448.0]:
        for top in (6 * s, np.nextafter(np.float32(6 * s), np.float32(0)), np.nextafter(np.float32(6 * s), np.float32(1e9))):
            for mid in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
                b = np.float32(mid * s)
                near = [b, np.nextafter(b, np.float32(0)), np.nextafter(b, np.float32(1e9))]
                rows.append([top] + near + [-v for v in near] + [0.0, -0.0] + [top / 3] * 7)
    middle = (MO.E4M3[1:] + MO.E4M3[:-1]) / 2 * 6
    for t in middle:
        for top in (t, np.nextafter(np.float32(t), np.float32(0)), np.nextafter(np.float32(t), np.float32(1e9))):
            rows.append([top, top / 2, -top] + [top * 0.3] * 13)
    rows += [[0.0] * 16, [-0.0] * 16, [1e-30] * 16, [2.0 ** -149] * 16, [3000.0, 1.0] * 8, [3e38, -1e38] * 8, [2688.0, 2689.0] * 8]
    v = np.array(rows, dtype=np.float32)
    v = np.repeat(v, 2, axis=0).reshape(-1, 32)   # two blocks a row
    a, sfa = moe.quantize(gpu(v))
    check_rows(a.cpu().numpy(), sfa.cpu().numpy(), v, 32)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_non_finite_and_scaled(dtype):
    x = torch.randn(20, 64, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype])
    x[0, 3], x[1, 20], x[2, 63] = float("inf"), float("nan"), float("-inf")
    for scale in (1.0, 0.3, 1024.0):
        v = (x.float() * np.float32(scale)).numpy()
        a, sfa = moe.quantize(x.cuda(), scale=scale)
        check_rows(a.cpu().numpy(), sfa.cpu().numpy(), v, 64)
    values = f64(moe.dequantize(*moe.quantize(x.cuda())))
    assert np.isnan(values[0, :16]).all() and np.isnan(values[1, 16:32]).all() and np.isnan(values[2, 48:]).all()
    assert np.isfinite(values[3:]).all()


def test_quantize_batches_strides_and_guards():
    base = torch.randn(3, 150, 80, device="cuda").half()
    x = base[:, 10:143, 5:69]                     # 133 rows of 64, odd offset
    a = torch.full((3, 133, 32), 0xAB, dtype=torch.uint8, device="cuda")
    need = mm.nvfp4_sf_bytes(133, 64, 3)
    store = torch.full((need + 512,), 0xCD, dtype=torch.uint8, device="cuda")
    moe.quantize(x, a=a, sfa=store[256:256 + need])
    sf = store.cpu().numpy()
    assert (sf[:256] == 0xCD).all() and (sf[256 + need:] == 0xCD).all()
    for li in range(3):
        check_rows(a[li].cpu().numpy(), sf[256:], f64(x[li]), 64, atom=2 * li)
    back = moe.dequantize(a, store[256:256 + need].clone())
    codes, scales = MO.quantize(f64(x[1]))
    assert np.array_equal(f64(back[1]), MO.values(codes, scales))
    one = moe.quantize(x[0].t().contiguous().t()[:, :0])[0]
    assert one.shape == (133, 0)
    with pytest.raises(ValueError):
        moe.quantize(x[..., :48])
    with pytest.raises(ValueError):
        moe.quantize(x.transpose(1, 2)[:, :64, :64])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,topk,experts,k,dropped", [(1, 1, 1, 32, 0), (1, 8, 256, 7168, 0), (33, 8, 256, 96, 0.2), (130, 2, 3, 160, 0),
                                                           (700, 4, 8, 1088, 0.5), (257, 3, 16, 320, 1.0), (64, 16, 40, 64, 0),
                                                           (4111, 8, 20, 1056, 0.01), (8200, 3, 300, 1440, 0.02)])
def test_dispatch(dtype, tokens, topk, experts, k, dropped):
    rng = rng_of(tokens, topk, experts, k)
    ids = np.argsort(rng.random((tokens, experts)), axis=1)[:, :topk].astype(np.int32) if topk <= experts else None
    ids[rng.random(ids.shape) < dropped] = -1
    x = gpu(rng.standard_normal((tokens, k)), TYPES[dtype])
    p = moe.plan(gpu(ids), experts)
    a, sfa = moe.quantize(x, plan=p)
    offsets, atoms, _, row_slots = MO.plan(ids, experts)
    an, sn, xn = a.cpu().numpy(), sfa.cpu().numpy(), f64(x)
    for e in range(experts):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            check_rows(an[lo:hi], sn, xn[row_slots[lo:hi] // topk], k, atom=int(atoms[e]))
    out = torch.full((tokens * topk, k), -7.0, dtype=torch.float16, device="cuda")
    moe.dequantize(a, sfa, plan=p, out=out)
    rows = int(offsets[-1])
    if rows:
        codes, scales = MO.quantize(xn[row_slots[:rows] // topk])
        assert np.array_equal(f64(out[:rows]), MO.values(codes, scales))
    assert (out[rows:] == -7).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,topk,experts,k", [(1, 2, 8, 32), (9, 8, 64, 288), (400, 2, 5, 2048), (300, 4, 16, 96),
                                                   (1031, 4, 7, 2080)])
def test_swiglu(dtype, tokens, topk, experts, k):
    """Equal codes and scales: activations next to a border are decided in fp64 (the oracle's)."""
    rng = rng_of(tokens, topk, experts, k)
    ids = rng.integers(-1, experts, (tokens, topk)).astype(np.int32)
    x = gpu(rng.standard_normal((tokens * topk, 2 * k)) * 2, TYPES[dtype])
    alpha = rng.uniform(0.3, 2, experts).astype(np.float32)
    p = moe.plan(gpu(ids), experts)
    offsets, atoms, _, _ = MO.plan(ids, experts)
    for al in (None, alpha):
        a, sfa = moe.swiglu_quantize(x, plan=p, alpha=None if al is None else gpu(al), scale=0.75)
        an, sn = a.cpu().numpy(), sfa.cpu().numpy()
        for e in range(experts):
            lo, hi = offsets[e], offsets[e + 1]
            if lo < hi:
                v = MO.swiglu(f64(x)[lo:hi], 1.0 if al is None else float(al[e]), 0.75)
                check_rows(an[lo:hi], sn, v, k, atom=int(atoms[e]))
    a, sfa = moe.swiglu_quantize(x)
    check_rows(a.cpu().numpy(), sfa.cpu().numpy(), MO.swiglu(f64(x)), k)


def test_swiglu_at_the_edges():
    x = torch.zeros(20, 64, device="cuda")
    x[0] = 0
    x[1, :32], x[1, 32:] = -200.0, 5.0            # silu underflows
    x[2, :32], x[2, 32:] = 200.0, 3.0             # silu(g) = g
    x[3, :32], x[3, 32:] = 1e30, 1e30             # beyond fp32
    x[4, 3] = float("nan")
    x[5, 40] = float("inf")
    x[6] = -0.0
    x[7, :32], x[7, 32:] = -88.0, 1e38
    a, sfa = moe.swiglu_quantize(x)
    v = f64(moe.dequantize(a, sfa))
    assert (v[0] == 0).all() and (v[1] == 0).all() and (v[6] == 0).all()
    codes, scales = MO.quantize(MO.swiglu(f64(x[2:3])))
    assert np.array_equal(v[2:3], MO.values(codes, scales))
    assert np.isnan(v[3]).all() and np.isnan(v[4, :16]).all() and (v[4, 16:] == 0).all() and np.isnan(v[5, :16]).all()
    codes, scales = MO.quantize(MO.swiglu(f64(x[7:8])))
    assert np.array_equal(v[7:8], MO.values(codes, scales))


@pytest.mark.parametrize("scale", [1e-20, 1.0, 1e20, 0.0])
def test_swiglu_whose_factors_leave_the_range(scale):
    """Products of alpha, scale and an operand below and beyond what fp32 has, where the activation is an ordinary number."""
    alphas = [1e-30, 1e-25, 1e-19, 1e19, 1e25, 0.0]
    ids = torch.arange(len(alphas), dtype=torch.int32).repeat_interleave(12).view(-1, 1)
    p = moe.plan(ids.cuda(), len(alphas))
    x = np.zeros((12 * len(alphas), 128), dtype=np.float32)
    rng = rng_of(int(np.log2(scale)) + 999 if scale else 0)
    for i, alpha in enumerate(np.repeat(np.array(alphas, dtype=np.float32), 12)):
        al = float(alpha) or 1.0
        for kb in range(4):  # of each block: g alpha, and what v is to be
            g = np.float64(rng.choice([-60.0, -3.0, 1e-3, 1.0, 40.0, 1e12])) * rng.uniform(0.5, 1, 16)
            v = np.float64(rng.choice([0.05, 1.0, 300.0])) * rng.standard_normal(16)
            u = v / (g / (1 + np.exp(-g)) * al * (np.float64(np.float32(scale)) or 1.0))
            x[i, kb * 16:kb * 16 + 16] = np.clip(g / al, -1e38, 1e38)
            x[i, 64 + kb * 16:80 + kb * 16] = np.clip(u, -1e38, 1e38)
    a, sfa = moe.swiglu_quantize(gpu(x), plan=p, alpha=gpu(np.array(alphas, dtype=np.float32)), scale=scale)
    an, sn, atoms = a.cpu().numpy(), sfa.cpu().numpy(), p.atoms.cpu().numpy()
    for e, alpha in enumerate(np.array(alphas, dtype=np.float32)):
        v = MO.swiglu(x[e * 12:e * 12 + 12].astype(np.float64), float(alpha), float(np.float32(scale)))
        v = np.where(np.abs(v) < 2.0 ** 128, v, np.inf)
        check_rows(an[e * 12:e * 12 + 12], sn, v, 64, atom=int(atoms[e]))


# ---- the combine ----------------------------------------------------------------------------

COMBINE = [(1, 1, 8), (1, 8, 7168), (5, 3, 24), (33, 2, 520), (64, 16, 264), (100, 8, 1032), (7, 9, 2056), (40, 4, 48)]


def combine_case(tokens, topk, n, kind, seed=0):
    rng = rng_of(tokens, topk, n, seed)
    rows = rng.permutation(tokens * topk).astype(np.int32).reshape(tokens, topk)
    rows[rng.random(rows.shape) < 0.2] = -1
    x = rng.standard_normal((tokens * topk, n))
    x[np.setdiff1d(np.arange(tokens * topk), rows)] = np.nan  # rows that no slot names are not read
    w = rng.standard_normal((tokens, topk)).astype(np.float32)
    w[rows < 0] = np.nan                                      # nor are those slots' weights
    ids = rng.integers(0, 6, rows.shape).astype(np.int32)
    alpha = rng.uniform(0.5, 2, 6).astype(np.float32)
    return gpu(x, kind), rows, w, ids, alpha


@pytest.mark.parametrize("types", [("fp16", "bf16"), ("bf16", "fp32"), ("fp32", "fp16")])
@pytest.mark.parametrize("tokens,topk,n", COMBINE)
def test_combine(tokens, topk, n, types):
    x, rows, w, ids, alpha = combine_case(tokens, topk, n, TYPES[types[0]])
    out_type = TYPES[types[1]]
    y = moe.combine(x, gpu(w), gpu(rows), dtype=out_type)
    want, size = MO.combine(f64(x), w, rows)
    close(y, want, (topk + 2) * H[torch.float32] * size, out_type)
    residual = torch.randn(tokens, n, device="cuda").to(out_type)
    y = moe.combine(x, gpu(w), gpu(rows), alpha=gpu(alpha), ids=gpu(ids), residual=residual)
    want, size = MO.combine(f64(x), w, rows, alpha, ids, f64(residual))
    close(y, want, (topk + 3) * H[torch.float32] * size, out_type)


@pytest.mark.parametrize("types", [("fp16", "bf16"), ("bf16", "fp32"), ("fp32", "fp16")])
@pytest.mark.parametrize("tokens,topk,n", COMBINE)
def test_combine_backward(tokens, topk, n, types):
    x, rows, w, ids, alpha = combine_case(tokens, topk, n, TYPES[types[0]], seed=1)
    dy = torch.randn(tokens, n, device="cuda").to(TYPES[types[1]])
    for al in (None, alpha):
        dc0 = torch.full_like(x, 3.0)
        dc, dw = moe.combine_backward(dy, x, gpu(w), gpu(rows), alpha=None if al is None else gpu(al),
                                      ids=None if al is None else gpu(ids), dc=dc0)
        want, want_w, size = MO.combine_backward(f64(dy), f64(x), w, rows, al, None if al is None else ids)
        named = ~np.isnan(want).any(axis=1)
        assert (f64(dc)[~named] == 3).all()
        close(dc[gpu(np.flatnonzero(named))], want[named], 3 * H[torch.float32] * np.abs(want[named]), x.dtype)
        close(dw, want_w, (n / 256 + 12) * H[torch.float32] * size, torch.float32)


def test_combine_slots_in_order_strides_and_refusals():
    store = torch.randn(12, 100, device="cuda").half()
    x = store[:, 3:67]                            # odd offset
    ids = torch.tensor([[0, -1, 2], [1, 1, -5], [-1, -1, -1], [0, 1, 2]], dtype=torch.int32, device="cuda")
    w = torch.rand(4, 3, device="cuda")
    y = moe.combine(x, w, ids=ids, dtype=torch.float32)
    want, size = MO.combine(f64(x), f64(w), np.arange(12).reshape(4, 3), ids=ids.cpu().numpy())
    close(y, want, 5 * H[torch.float32] * size, torch.float32)
    assert (y[2] == 0).all()
    y = moe.combine(x, None, torch.arange(12, dtype=torch.int32, device="cuda").view(4, 3), dtype=torch.float32)
    close(y, f64(x).reshape(4, 3, 64).sum(1), 5 * H[torch.float32] * np.abs(f64(x)).reshape(4, 3, 64).sum(1), torch.float32)
    for bad in (lambda: moe.combine(x, w[:3], ids=ids), lambda: moe.combine(x, w, alpha=w[0]), lambda: moe.combine(x[:5], w),
                lambda: moe.combine(x, w.double()), lambda: moe.combine(x, None), lambda: moe.combine(x.long(), w)):
        with pytest.raises(ValueError):
            bad()


def test_combine_of_slots_without_rows_or_experts():
    """Rows and experts that are not there add nothing, and what they name gets gradients of 0."""
    x = torch.randn(8, 72, device="cuda")
    alpha = torch.tensor([2.0, 3.0, 5.0], device="cuda")
    ids = torch.tensor([[0, 3, 1], [-1, 2, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 7.0, 1.0], [float("inf"), 2.0, float("nan")]], device="cuda")
    dy = torch.full((2, 72), float("inf"), device="cuda")
    dy[0] = 1.0
    dy[1, 0] = 2.0
    f = f64(x)
    want = np.stack([0.5 * 2 * f[0] + 3 * f[2], 2 * 5 * f[4]])
    close(moe.combine(x[:6], w, ids=ids, alpha=alpha), want, 4 * H[torch.float32] * np.abs(f).max() * 8, torch.float32)
    dc = torch.full_like(x, 9.0)
    _, dw = moe.combine_backward(dy, x[:6], w, ids=ids, alpha=alpha, dc=dc[:6])
    assert (dc[[1, 3, 5]] == 0).all() and (dc[6:] == 9).all() and (dc[0] == 1).all() and (dc[2] == 3).all()
    assert dc[4, 0] == 20 and (dw[[0, 1, 1], [1, 0, 2]] == 0).all()
    rows = torch.tensor([[8, 0, -7], [2 ** 31 - 1, 7, -2 ** 31]], dtype=torch.int32, device="cuda")
    ones = torch.ones_like(w)
    assert torch.equal(moe.combine(x, ones, rows), x[[0, 7]])
    dc, dw = moe.combine_backward(torch.ones_like(dy), x, ones, rows, dc=torch.full_like(x, 9.0))
    assert (dc[[0, 7]] == 1).all() and (dc[1:7] == 9).all() and (dw[[0, 0, 1, 1], [0, 2, 0, 2]] == 0).all()


def test_combine_backward_against_differences():
    """Of the kernel's own forward pass in fp32 (a sum of products: differences are exact but for rounding)."""
    x, rows, w, ids, alpha = combine_case(6, 3, 16, torch.float32, seed=3)
    x = torch.nan_to_num(x)
    w = np.nan_to_num(w)
    dy = torch.randn(6, 16, device="cuda")
    dc, dw = moe.combine_backward(dy, x, gpu(w), gpu(rows), alpha=gpu(alpha), ids=gpu(ids), dc=torch.zeros_like(x))
    f = lambda x, w: float((moe.combine(x, gpu(w), gpu(rows), alpha=gpu(alpha), ids=gpu(ids)).double() * dy.double()).sum())  # noqa: E731
    size = float(MO.combine(f64(x), w, rows, alpha, ids)[1].max()) * 16 * 6 * 4
    for i, j in ((0, 0), (5, 7), (11, 15), (17, 3)):
        step = torch.zeros_like(x)
        step[i, j] = 1.0
        assert abs((f(x + step, w) - f(x - step, w)) / 2 - float(dc[i, j])) < 8 * H[torch.float32] * (size + 10)
    for t, j in ((0, 0), (2, 1), (5, 2)):
        step = np.zeros_like(w)
        step[t, j] = 1.0
        assert abs((f(x, w + step) - f(x, w - step)) / 2 - float(dw[t, j])) < 8 * H[torch.float32] * (size + 50)


# ---- a few tokens ------------------------------------------------------------------------------

def operand(rng, experts, n, k, low=0x20, high=0x50):
    codes = rng.integers(0, 16, (experts, n, k), dtype=np.uint8)
    scales = rng.integers(low, high, (experts, n, k // 16), dtype=np.uint8)
    packed = [MO.pack(codes[e], scales[e]) for e in range(experts)]
    w = np.stack([MO.values(codes[e], scales[e]) for e in range(experts)]) if experts else None
    return gpu(np.stack([p[0] for p in packed])), gpu(np.stack([p[1] for p in packed])), w


def few_bound(want, size, k):
    return (k + 16) * H[torch.float32] * size


def swiglu_of(y, bound):
    """silu(g) u of the halves, and how far it may be off."""
    g, u = np.split(y, 2, axis=-1)
    bg, bu = np.split(bound, 2, axis=-1)
    silu = g / (1 + np.exp(-g))
    want = silu * u
    return want, 1.1 * bg * (np.abs(u) + bu) + np.abs(silu) * bu + 16 * H[torch.float32] * np.abs(want)


FEW = [
    # tokens, topk, experts, n, k
    (1, 1, 1, 8, 32), (1, 8, 32, 256, 7168), (1, 3, 4, 40, 64), (2, 2, 8, 512, 1024), (3, 8, 256, 64, 96), (13, 2, 8, 264, 2080),
    (17, 1, 2, 136, 288), (16, 4, 4, 128, 4128), (40, 2, 3, 72, 160), (64, 8, 16, 96, 544), (5, 16, 20, 1000, 512), (130, 1, 1, 48, 256),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tokens,topk,experts,n,k", FEW)
def test_few_tokens(tokens, topk, experts, n, k, dtype):
    rng = rng_of(tokens, topk, experts, n, k)
    ids = rng.integers(-1, experts + 1, (tokens, topk)).astype(np.int32)  # a token may name an expert twice
    b, sfb, w = operand(rng, experts, n, k)
    alpha = rng.uniform(0.25, 2, experts).astype(np.float32)
    for per_slot in (False, True):
        x = gpu(rng.standard_normal((tokens, topk, k) if per_slot else (tokens, k)) * 0.1, TYPES[dtype])
        for al, out in ((alpha, torch.float32), (None, TYPES[dtype])):
            y = moe.few_tokens(x, gpu(ids), b, sfb, alpha=None if al is None else gpu(al), dtype=out)
            want, size = MO.few(f64(x), ids, w, al)
            close(y, want, few_bound(want, size, k), out)
        assert (y.cpu()[torch.from_numpy((ids < 0) | (ids >= experts))] == 0).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tokens,topk,experts,n,k", [(1, 8, 16, 512, 2048), (1, 1, 1, 16, 32), (3, 2, 4, 144, 96), (20, 2, 6, 208, 1056),
                                                     (16, 1, 1, 128, 512), (9, 3, 64, 48, 320)])
def test_few_tokens_swiglu(tokens, topk, experts, n, k, dtype):
    rng = rng_of(tokens, topk, experts, n, k, 1)
    ids = rng.integers(-1, experts, (tokens, topk)).astype(np.int32)
    b, sfb, w = operand(rng, experts, n, k)
    x = gpu(rng.standard_normal((tokens, k)) * (0.5 / np.sqrt(k)), TYPES[dtype])
    alpha = rng.uniform(0.25, 2, experts).astype(np.float32)
    y = moe.few_tokens(x, gpu(ids), b, sfb, alpha=gpu(alpha), swiglu=True, dtype=torch.float32)
    want, bound = swiglu_of(*(lambda v, s: (v, few_bound(v, s, k)))(*MO.few(f64(x), ids, w, alpha)))
    close(y, want, bound, torch.float32)


def test_few_tokens_wide_ranges_and_non_finite():
    """bf16 rows at both ends of their range, rows of zeros, infinities and NaN in one row only, poisoned padding."""
    rng = rng_of(99)
    b, sfb, w = operand(rng, 2, 64, 416)
    x = rng.standard_normal((9, 416))
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = 0
    x[3, 5] *= 1e8
    x[4] *= np.exp2(rng.uniform(-30, 0, 416))
    x[7, 9], x[8, 9] = np.inf, np.nan
    t = gpu(x, torch.bfloat16)
    ids = np.array([[0], [1], [0], [1], [0], [1], [0], [1], [0]], dtype=np.int32)
    y = moe.few_tokens(t, gpu(ids), b, sfb, dtype=torch.float32)
    want, size = MO.few(f64(t[:7]), ids[:7], w)
    close(y[:7], want, few_bound(want, size, 416), torch.float32)
    assert not torch.isfinite(y[7]).any() or (w[1][:, 9] == 0).any()
    assert torch.isnan(y[8]).all()


def test_few_tokens_long_rows_scale_as_they_go():
    """Rows longer than a stage of shared memory, their large elements late."""
    rng = rng_of(5)
    k = 16384 + 96
    b, sfb, w = operand(rng, 1, 32, k)
    x = rng.standard_normal((3, k))
    x[0, -40:] *= 1e6
    x[1, :40] *= 1e6
    x[2] *= np.linspace(1e-3, 1e3, k)
    for tokens in (1, 3):
        t = gpu(x[:tokens], torch.bfloat16)
        ids = np.zeros((tokens, 1), dtype=np.int32)
        y = moe.few_tokens(t, gpu(ids), b, sfb, dtype=torch.float32)
        want, size = MO.few(f64(t), ids, w)
        close(y, want, few_bound(want, size, k), torch.float32)


def test_few_tokens_strides_duplicates_and_refusals():
    rng = rng_of(6)
    b, sfb, w = operand(rng, 4, 40, 96)
    store = torch.randn(7, 120, device="cuda").bfloat16()
    x = store[:, 5:101]                           # not 16-byte aligned
    ids = np.array([[1, 1], [1, 1], [3, 0], [0, 3], [2, 9], [-1, -1], [1, 2]], dtype=np.int32)
    y = moe.few_tokens(x, gpu(ids), b, sfb, dtype=torch.float32)
    want, size = MO.few(f64(x), ids, w)
    close(y, want, few_bound(want, size, 96), torch.float32)
    assert moe.few_tokens(x[:0], gpu(ids[:0]), b, sfb).shape == (0, 2, 40)
    for bad in (lambda: moe.few_tokens(x, gpu(ids), b, sfb[:, :-1]), lambda: moe.few_tokens(x[:, :64], gpu(ids), b, sfb),
                lambda: moe.few_tokens(x[:6], gpu(ids), b, sfb), lambda: moe.few_tokens(x, gpu(ids).long(), b, sfb),
                lambda: moe.few_tokens(x, gpu(ids), b, sfb, alpha=torch.ones(3, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(c.Nvfp4MoeError):
        moe.few_tokens(x.float(), gpu(ids), b, sfb)
    with pytest.raises(c.Nvfp4MoeError):
        moe.few_tokens(x, gpu(ids), b, sfb, swiglu=True)   # halves of 20 rows


def test_few_tokens_no_k_gives_zeros():
    b = torch.zeros(2, 16, 0, dtype=torch.uint8, device="cuda")
    sfb = torch.zeros(2, 0, dtype=torch.uint8, device="cuda")
    x = torch.zeros(3, 0, dtype=torch.float16, device="cuda")
    ids = gpu(np.array([[0], [1], [-1]], dtype=np.int32))
    out = torch.full((3, 1, 16), 5.0, dtype=torch.float16, device="cuda")
    c.nvfp4_moe_few_tokens(0, c.NVFP4_MOE_F16, 0, 0, ids.data_ptr(), 3, 1, 2, 16, 0, 0, 0, 0, 0, out.data_ptr(), c.NVFP4_MOE_F16,
                           torch.cuda.current_stream().cuda_stream)
    assert (out == 0).all() and x.numel() == b.numel() == sfb.numel() == 0


# ---- together -------------------------------------------------------------------------------------

def layer_case(tokens, experts, topk, hidden, inner, dtype, seed=0):
    rng = rng_of(tokens, experts, hidden, seed)
    b1, sfb1, w1 = operand(rng, experts, 2 * inner, hidden, 0x18, 0x20)
    b2, sfb2, w2 = operand(rng, experts, hidden, inner, 0x18, 0x20)
    x = gpu(rng.standard_normal((tokens, hidden)), TYPES[dtype])
    logits = gpu(rng.standard_normal((tokens, experts)), TYPES[dtype])
    return moe.FeedForward(b1, sfb1, b2, sfb2), w1, w2, x, logits


@pytest.mark.parametrize("tokens,experts,topk,hidden,inner,dtype", [(1, 8, 2, 256, 128, "bf16"), (5, 4, 2, 512, 96, "fp16"),
                                                                    (150, 6, 3, 256, 160, "bf16"), (700, 3, 1, 128, 64, "fp16")])
def test_layer(tokens, experts, topk, hidden, inner, dtype):
    """Both forms of the layer against the steps' definitions. Every step's own error is tested above; here the codes
    of intermediate rows may differ where a product's last bit does, so the outputs are compared as a whole: a code's
    step is at most a third of its value, and the few that differ keep the relative norm below 2^-6."""
    layer, w1, w2, x, logits = layer_case(tokens, experts, topk, hidden, inner, dtype)
    ids, w = moe.route(logits, topk)
    xn, idn, wn = f64(x), ids.cpu().numpy(), f64(w)

    def reference(quantized):
        nv = lambda v: MO.values(*MO.quantize(v)) if quantized else v  # noqa: E731
        y = np.zeros_like(xn)
        for t in range(tokens):
            for j in range(topk):
                e = idn[t, j]
                h = nv(xn[t:t + 1]) @ w1[e].T
                h = nv(MO.swiglu(h.astype(np.float16) if quantized else h))
                y[t] += wn[t, j] * (h @ w2[e].T)[0]
        return y
    residual = torch.randn_like(x)
    for run, quantized in ((layer.grouped, True), (layer.few, False)):
        if quantized or tokens * topk <= 1024:
            want = reference(quantized)
            got = f64(run(x, ids, w))
            assert np.linalg.norm(got - want) <= 2.0 ** -6 * np.linalg.norm(want)
            both = f64(run(x, ids, w, residual=residual))
            want = want + f64(residual)
            assert np.linalg.norm(both - want) <= 2.0 ** -6 * np.linalg.norm(want)
    assert layer(x, ids, w).shape == x.shape


def test_layer_in_a_graph_replays_on_new_data():
    """Captured once, replayed between other work and synchronisations, with inputs that change the plan."""
    layer, _, _, x, logits = layer_case(96, 4, 2, 256, 128, "bf16", seed=2)
    xs = [torch.randn_like(x) for _ in range(3)]
    ls = [torch.randn_like(logits) for _ in range(3)]
    ls[1][:, 2] = float("-inf")

    def both(x, logits):
        ids, w = moe.route(logits, 2)
        return layer.grouped(x, ids, w), layer.few(x, ids, w), moe.route_backward(logits, ids, w)
    want = [[t.clone() for t in both(a, b)] for a, b in zip(xs, ls)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(x, logits)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both(x, logits)
    for turn in range(6):
        i = turn % 3
        x.copy_(xs[i])
        logits.copy_(ls[i])
        g.replay()
        torch.cuda.synchronize()
        torch.randn(1 << 16, device="cuda").sort()
        for got, ref in zip(out, want[i]):
            assert torch.equal(got, ref)


def test_other_streams_and_determinism():
    """A call on a stream of its own, behind work there, gives what the current stream gives; twice the same bits."""
    layer, _, _, x, logits = layer_case(40, 4, 2, 512, 128, "bf16", seed=3)
    ids, w = moe.route(logits, 2)
    want = layer.grouped(x, ids, w), layer.few(x, ids, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    later = torch.empty_like(x)
    with torch.cuda.stream(side):
        torch.randn(1 << 22, device="cuda").sort()
        later.copy_(x)
    got = layer.grouped(later, ids, w, stream=side), layer.few(later, ids, w, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    dc1 = moe.combine_backward(x, torch.randn(80, 512, device="cuda", generator=torch.Generator("cuda").manual_seed(1)), w,
                               torch.arange(80, dtype=torch.int32, device="cuda").view(40, 2))
    dc2 = moe.combine_backward(x, torch.randn(80, 512, device="cuda", generator=torch.Generator("cuda").manual_seed(1)), w,
                               torch.arange(80, dtype=torch.int32, device="cuda").view(40, 2))
    assert all(torch.equal(a, b) for a, b in zip(dc1, dc2))


def test_what_a_call_on_another_stream_allocates_is_that_streams():
    """Memory of the current stream may still be in use there, and may be used there again at once."""
    layer, _, _, x, logits = layer_case(2000, 4, 2, 512, 256, "bf16", seed=4)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        ids, w = moe.route(logits, 2)
        torch.cuda.synchronize()
        y = layer.grouped(x, ids, w, stream=stream)
        a, sfa = moe.quantize(x, stream=stream)
        side.synchronize()
        at = {y.data_ptr(), a.data_ptr()}
        del y, a, sfa
        assert not at & {torch.empty(2000, n, dtype=torch.uint8, device="cuda").data_ptr() for n in (1024, 256)}
        before = torch.cuda.memory_reserved()
        with torch.cuda.stream(side):
            layer.grouped(x, ids, w)   # finds what the calls before left there
        assert torch.cuda.memory_reserved() == before
    torch.cuda.synchronize()


def test_products_and_layers_refuse_what_does_not_fit():
    layer, _, _, x, logits = layer_case(8, 4, 2, 256, 128, "bf16", seed=5)
    ids, w = moe.route(logits, 2)
    for bad in (lambda: layer.grouped(x[:, :128], ids, w), lambda: layer.grouped(x[:7], ids, w), lambda: layer.grouped(x, ids.long(), w),
                lambda: layer.grouped(x, ids, w.double()), lambda: layer.grouped(x, ids, w[:7]), lambda: layer.grouped(x.cpu(), ids, w),
                lambda: layer.grouped(x, ids, w, residual=x.float()), lambda: layer.grouped(x.t(), ids, w), lambda: layer.few(x[:7], ids, w),
                lambda: layer.few(x.float(), ids, w), lambda: moe.FeedForward(layer.b1, layer.sfb1, layer.b1, layer.sfb1),
                lambda: moe.FeedForward(layer.b1, layer.sfb1, layer.b2, layer.sfb2, alpha1=w[0])):
        with pytest.raises((ValueError, moe.c.Nvfp4MoeError)):
            bad()
    a, sfa = moe.quantize(x)
    q = moe.Product(a, torch.zeros(moe.c.nvfp4_moe_sf_bytes(8, 4, 256), dtype=torch.uint8, device="cuda"), layer.b1, layer.sfb1,
                    torch.zeros(8, 256, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="plan"):
        q.run()
    assert layer.grouped(x[:0], ids[:0], w[:0]).shape == (0, 256)
