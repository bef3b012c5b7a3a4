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


# ---- sigmoid scores that leave fp32 ------------------------------------------------

@pytest.mark.parametrize("topk", [1, 2, 8, 13])
@pytest.mark.parametrize("dtype", TYPES)
def test_sigmoid_renormalised_far_below_zero(dtype, topk):
    """Logits of -80 .. -120, where sigmoids are denormal or 0 in fp32, of -700, and mixed with ordinary ones."""
    rng = rng_of(topk, 80)
    x = rng.uniform(-120, -80, (96, 16))
    x[1::4] = rng.uniform(-95, -2, (24, 16))          # some of a token below 2^-126
    x[2::4] = rng.uniform(-700, -600, (24, 16))
    x[3::4] = rng.uniform(-100, 3, (24, 16))
    x[0] = -90.0
    x[4, 3:] = -np.inf
    x[5, 1:] = -np.inf
    x[8, :2] = -90.0, -91.0
    x[8, 2:] = -110.0
    x = gpu(x, TYPES[dtype])
    how = dict(score="sigmoid", scale=2.5)
    for bias in (None, gpu(np.zeros(16, dtype=np.float32))):
        ids, w = moe.route(x, topk, bias=bias, **how)
        want_ids, want_w = MO.route(f64(x), topk, **how)
        if bias is None:
            assert np.array_equal(ids.cpu().numpy(), want_ids)
        else:  # scores this small count as equal beside a bias: weights of what was chosen
            s = np.take_along_axis(MO.scores(f64(x), "sigmoid"), np.maximum(ids.cpu().numpy(), 0).astype(np.int64), 1)
            s = np.where(ids.cpu().numpy() >= 0, s, 0)
            want_w = 2.5 * s / s.sum(1, keepdims=True)
        close(w, want_w, 64 * H[torch.float32] * want_w, torch.float32)
    if topk == 2:
        assert abs(float(w[8].sum()) - 2.5) < 1e-5 and abs(float(w[8, 0]) / 2.5 - 0.7310586) < 1e-5
    ids, _ = moe.route(x, topk, **how)
    dw = gpu(rng.standard_normal((96, topk)).astype(np.float32) * 4)
    d = moe.route_backward(x, ids, dw, **how)
    want, size = MO.route_backward(f64(x), ids.cpu().numpy(), f64(dw), **how)
    close(d, want, 256 * H[torch.float32] * size, x.dtype)


def test_sigmoid_renormalised_gradient_against_differences():
    """Of the kernel's own forward pass, at logits around -90."""
    x = -90 + torch.arange(12, device="cuda").float().view(1, 12).mul(0.37).sin().mul(3).repeat(24, 1)
    dw = torch.randn(1, 5, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).repeat(24, 1)
    h = 2.0 ** -7
    step = torch.cat((torch.eye(12), -torch.eye(12))).cuda() * h
    ids, w = moe.route(x + step, 5, score="sigmoid", scale=1.5)
    assert (ids == ids[0]).all()
    loss = (w.double() * dw.double()).sum(1)
    diff = (loss[:12] - loss[12:]) / (2 * h)
    d = moe.route_backward(x[:1].contiguous(), ids[:1].contiguous(), dw[:1].contiguous(), score="sigmoid", scale=1.5)
    # h^2 / 6 of the third derivative (below 8 times the weights' size), and 64 H of the weights over h
    size = float(dw[0].abs().sum()) * 1.5
    assert float(d.abs().max()) > 0.01
    assert float((d[0].double() - diff).abs().max()) < h * h / 6 * size * 8 + 64 * 2.0 ** -24 * size * 2 / h


# ---- the layer ---------------------------------------------------------------------

def layer_of(tokens, experts, hidden, inner, dtype, low=0x18, high=0x20, alpha1=None, alpha2=None, **how):
    rng = rng_of(tokens, experts, hidden, inner)
    b1, sfb1, w1 = operand(rng, experts, 2 * inner, hidden, low, high)
    b2, sfb2, w2 = operand(rng, experts, hidden, inner, low, high)
    x = gpu(rng.standard_normal((tokens, hidden)), TYPES[dtype])
    layer = moe.FeedForward(b1, sfb1, b2, sfb2, alpha1=None if alpha1 is None else gpu(alpha1),
                            alpha2=None if alpha2 is None else gpu(alpha2), **how)
    return layer, w1, w2, x


def layer_reference(layer, x, ids, w, w1, w2, quantized, alpha1=None, alpha2=None, scale1=1.0, scale2=1.0):
    """The layer by its steps' definitions. Products of the grouped form are rounded to fp16 and divided by the rows'
    factor afterwards."""
    xn, y = f64(x), np.zeros((x.shape[0], x.shape[1]))
    one = np.ones(w1.shape[0], dtype=np.float32)
    alpha1, alpha2 = one if alpha1 is None else alpha1, one if alpha2 is None else alpha2
    nv = lambda v: MO.values(*MO.quantize(v)) if quantized else v  # noqa: E731
    half = lambda v: v.astype(np.float16).astype(np.float64) if quantized else v  # noqa: E731
    rows = nv((xn * scale1).astype(np.float32)) if quantized else xn
    s1, s2 = (scale1, scale2) if quantized else (1.0, 1.0)
    for e in range(w1.shape[0]):
        t, j = np.nonzero(ids == e)
        if t.size:
            h = MO.swiglu(half(rows[t] @ w1[e].T), float(alpha1[e]) / s1, s2)
            np.add.at(y, t, w[t, j].astype(np.float64)[:, None] * float(alpha2[e]) / s2 * half(nv(h) @ w2[e].T))
    return y


def near(got, want):
    """Every step's own error is tested with the step; where a product's last bit differs, a code next to a border may,
    by a third of its value at most: the few that do keep the relative norm below 2^-6."""
    got = f64(got)
    assert np.isfinite(got).all()
    assert np.linalg.norm(got - want) <= 2.0 ** -6 * np.linalg.norm(want)


@pytest.mark.parametrize("tokens,experts,topk,hidden,inner,dtype", [
    (2, 5, 2, 256, 128, "fp16"), (70, 5, 2, 256, 128, "fp32"), (300, 7, 3, 512, 96, "bf16"), (600, 40, 4, 256, 64, "bf16"),
    (90, 160, 6, 128, 64, "fp32"), (130, 300, 8, 128, 64, "fp16")])
def test_layer_with_factors(tokens, experts, topk, hidden, inner, dtype):
    """Factors that differ from expert to expert and between the products, in both forms, and in what a call chooses."""
    rng = rng_of(tokens, experts, 5)
    alpha1, alpha2 = rng.uniform(0.25, 1.5, experts).astype(np.float32), rng.uniform(0.125, 2, experts).astype(np.float32)
    layer, w1, w2, x = layer_of(tokens, experts, hidden, inner, dtype, alpha1=alpha1, alpha2=alpha2)
    ids, w = moe.route(gpu(rng.standard_normal((tokens, experts)), torch.float32), topk)
    idn, wn = ids.cpu().numpy(), f64(w)
    few = tokens * topk <= 3 * experts and dtype != "fp32"
    for run, quantized in ((layer.grouped, True), (layer, not few)) + (((layer.few, False),) if dtype != "fp32" else ()):
        residual = torch.randn_like(x)
        want = layer_reference(layer, x, idn, wn, w1, w2, quantized, alpha1, alpha2)
        near(run(x, ids, w), want)
        near(run(x, ids, w, residual=residual), want + f64(residual))


@pytest.mark.parametrize("rows,experts,hidden,inner,tiles", [
    (4, 32, 2048, 64, (2, 1)), (4, 32, 256, 1024, (1, 2)), (100, 4, 2048, 64, (2, 2)), (100, 32, 256, 1024, (0, 2)),
    (256, 32, 2048, 64, (2, 0))])
def test_layer_by_every_tile(rows, experts, hidden, inner, tiles):
    """Layers whose products take each of the tile configurations that the layer chooses from."""
    layer, w1, w2, x = layer_of(rows * experts // 2, experts, hidden, inner, "bf16")
    slots = rows * experts
    assert (layer._tile(slots, 2 * inner), layer._tile(slots, hidden)) == tiles
    ids = np.argsort(rng_of(rows, 3).random((x.shape[0], experts)), axis=1)[:, :2].astype(np.int32)
    w = rng_of(rows, 4).uniform(0.1, 1, ids.shape).astype(np.float32)
    y = layer.grouped(x, gpu(ids), gpu(w))
    some = np.unique(np.concatenate(([0, 1, x.shape[0] - 1], rng_of(rows, 5).integers(0, x.shape[0], 60))))
    near(y[gpu(some)], layer_reference(layer, x[gpu(some)], ids[some], w[some], w1, w2, True))
    assert torch.equal(y, layer.grouped(x, gpu(ids), gpu(w)))


def test_product_after_a_plan():
    """The grouped GEMM by the public way: dispatch, a plan with its product, run."""
    rng = rng_of(55)
    b, sfb, w = operand(rng, 5, 136, 192)
    x = gpu(rng.standard_normal((90, 192)), torch.float16)
    ids = rng.integers(-1, 6, (90, 2)).astype(np.int32)
    a = torch.empty(180, 96, dtype=torch.uint8, device="cuda")
    sfa = torch.empty(c.nvfp4_moe_sf_bytes(180, 5, 192), dtype=torch.uint8, device="cuda")
    out = torch.full((180, 136), 7.0, dtype=torch.float16, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    q = moe.Product(a, sfa, b, sfb, out)
    p = moe.plan(gpu(ids), 5, (q,))
    moe.quantize(x, plan=p, a=a, sfa=sfa)
    values = MO.values(*MO.quantize(f64(x)))
    rows = MO.plan(ids, 5)[2]
    for config in (-1, 0, 1, 2, 3, 4):
        out.fill_(7.0)
        assert q.run(config, status) is out and int(status) == 0
        got = f64(out)
        for t, j in zip(*np.nonzero(rows >= 0)):
            want, size = w[ids[t, j]] @ values[t], np.abs(w[ids[t, j]]) @ np.abs(values[t])
            assert (np.abs(got[rows[t, j]] - want) <= 1e-5 * size + 2 * 2.0 ** -11 * np.abs(want)).all()
        assert (got[int((rows >= 0).sum()):] == 7).all()


# ---- slots without an expert -------------------------------------------------------

def test_combine_takes_the_number_of_experts():
    """Without factors, too, a slot whose id is none of the experts' adds nothing and gets gradients of 0."""
    x = torch.randn(8, 72, device="cuda")
    ids = torch.tensor([[0, 3, 1, -1], [2, 2 ** 31 - 1, -2 ** 31, 5]], dtype=torch.int32, device="cuda")
    nan, inf = float("nan"), float("inf")
    w = torch.tensor([[0.5, nan, 1.0, inf], [2.0, nan, inf, nan]], device="cuda")
    f = f64(x)
    want = np.stack([0.5 * f[0] + f[2], 2 * f[4]])
    close(moe.combine(x, w, ids=ids, experts=3), want, 6 * H[torch.float32] * 2 * np.abs(f).max(), torch.float32)
    dy = torch.ones(2, 72, device="cuda")
    dc, dw = moe.combine_backward(dy, x, w, ids=ids, experts=3, dc=torch.full_like(x, 9.0))
    assert (dc[[1, 3, 5, 6, 7]] == 0).all() and (dc[0] == 0.5).all() and (dc[2] == 1).all() and (dc[4] == 2).all()
    assert (dw[[0, 0, 1, 1, 1], [1, 3, 1, 2, 3]] == 0).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("tokens", [3, 40])
def test_layer_slots_without_an_expert(tokens):
    """Both forms: ids below 0 and beyond the experts, whose weights are NaN or infinite."""
    layer, w1, w2, x = layer_of(tokens, 6, 256, 128, "bf16")
    rng = rng_of(tokens, 77)
    ids = rng.integers(0, 6, (tokens, 3)).astype(np.int32)
    bad = rng.random(ids.shape) < 0.4
    ids[bad] = rng.choice(np.array([-1, 6, 7, 2 ** 31 - 1, -2 ** 31]), int(bad.sum()))
    w = rng.uniform(0.1, 1, ids.shape).astype(np.float32)
    w[bad] = rng.choice(np.array([np.nan, np.inf, -np.inf, 1.0], dtype=np.float32), int(bad.sum()))
    ids[0], w[0] = 6, np.nan                          # a token without any
    for run, quantized in ((layer.grouped, True), (layer.few, False), (layer, tokens * 3 > 18)):
        near(run(x, gpu(ids), gpu(w)), layer_reference(layer, x, ids, w, w1, w2, quantized))


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_whose_products_need_a_factor_on_their_rows(dtype):
    """Block scales near 448 and a factor of a weight tensor, as checkpoints have them: products of rows as they are leave
    fp16. Factors on the rows that bring them back leave the layer's two forms the same function."""
    rng = rng_of(8)
    alpha1, alpha2 = rng.uniform(2e-5, 6e-5, 6).astype(np.float32), rng.uniform(2e-5, 6e-5, 6).astype(np.float32)
    scales = dict(scale1=2.0 ** -4, scale2=2.0 ** -2)
    layer, w1, w2, x = layer_of(64, 6, 512, 256, dtype, low=0x60, high=0x7F, alpha1=alpha1, alpha2=alpha2, **scales)
    ids = rng.integers(0, 6, (64, 2)).astype(np.int32)
    w = rng.uniform(0.1, 1, ids.shape).astype(np.float32)
    x *= 3
    plain = moe.FeedForward(layer.b1, layer.sfb1, layer.b2, layer.sfb2, alpha1=gpu(alpha1), alpha2=gpu(alpha2))
    assert not torch.isfinite(plain.grouped(x, gpu(ids), gpu(w))).all()
    want = layer_reference(layer, x, ids, w, w1, w2, True, alpha1, alpha2, **scales)
    near(layer.grouped(x, gpu(ids), gpu(w)), want)
    if dtype != "fp32":
        few = layer_reference(layer, x, ids, w, w1, w2, False, alpha1, alpha2)
        near(layer.few(x, gpu(ids), gpu(w)), few)
        # rows, weights' products and activations in 4 bits against 16: a sixth of each value at most
        assert np.linalg.norm(want - few) < 0.25 * np.linalg.norm(few)


def test_layer_factors_of_rows_alone():
    """Without the experts' factors, and of a factor that is no power of two."""
    scales = dict(scale1=24.0, scale2=0.3)
    layer, w1, w2, x = layer_of(50, 4, 256, 96, "bf16", **scales)
    rng = rng_of(9)
    ids = rng.integers(0, 4, (50, 2)).astype(np.int32)
    w = rng.uniform(0.1, 1, ids.shape).astype(np.float32)
    near(layer.grouped(x, gpu(ids), gpu(w)), layer_reference(layer, x, ids, w, w1, w2, True, **scales))
    near(layer.few(x, gpu(ids), gpu(w)), layer_reference(layer, x, ids, w, w1, w2, False))
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e39, 1e-46):
        with pytest.raises(ValueError, match="scale"):
            moe.FeedForward(layer.b1, layer.sfb1, layer.b2, layer.sfb2, scale2=bad)


# ---- more rows than a group of the grouped GEMM holds ----------------------------------

def test_layer_in_parts(monkeypatch):
    """A layer whose rows might not fit one group takes its tokens in parts, and gives what each part gives."""
    layer, w1, w2, x = layer_of(300, 5, 256, 64, "bf16")
    rng = rng_of(300, 1)
    ids, w = gpu(rng.integers(-1, 5, (300, 2)).astype(np.int32)), gpu(rng.uniform(0.1, 1, (300, 2)).astype(np.float32))
    residual = torch.randn_like(x)
    assert layer._most_tokens(2) > 1 << 20
    monkeypatch.setattr(moe.FeedForward, "_most_tokens", lambda self, topk: 128)
    y = layer.grouped(x, ids, w, residual=residual)
    monkeypatch.undo()
    for lo in (0, 128, 256):
        part = slice(lo, lo + 128)
        assert torch.equal(y[part], layer.grouped(x[part], ids[part], w[part], residual=residual[part]))


def test_layer_of_an_expert_with_more_rows_than_a_group_holds():
    """262200 rows of 8192 bytes on one expert: the grouped GEMM refuses such a group and leaves its rows as they were."""
    tokens, hidden = 262200, 16384
    layer, w1, w2, _ = layer_of(1, 2, hidden, 32, "bf16")
    x = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    ids = torch.zeros(tokens, 1, dtype=torch.int32, device="cuda")
    ids[5] = 1
    w = torch.rand(tokens, 1, device="cuda") + 0.5
    y = layer.grouped(x, ids, w)
    for some in (slice(0, 8), slice(tokens // 2 - 4, tokens // 2 + 4), slice(tokens - 8, tokens)):
        near(y[some], layer_reference(layer, x[some], ids[some].cpu().numpy(), f64(w[some]), w1, w2, True))


def test_product_of_a_group_that_is_refused():
    """Its rows are NaN where no status is asked for, and as they were where one is."""
    b, sfb, w = operand(rng_of(3), 2, 16, 16384)
    rows = 262200
    a = torch.zeros(rows, 8192, dtype=torch.uint8, device="cuda")
    sfa = torch.zeros(c.nvfp4_moe_sf_bytes(rows, 2, 16384), dtype=torch.uint8, device="cuda")
    q = moe.Product(a, sfa, b, sfb, torch.full((rows, 16), 7.0, dtype=torch.float16, device="cuda"))
    ids = torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
    ids[-40:] = 1
    moe.plan(ids, 2, (q,))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = q.run(status=status)
    assert int(status) == 1 and (out[:-40] == 7).all() and (out[-40:] == 0).all()
    out = q.run()
    assert torch.isnan(out[:-40]).all() and (out[-40:] == 0).all()


# ---- a few tokens -----------------------------------------------------------------------

@pytest.mark.parametrize("swiglu", [False, True])
def test_few_tokens_factors_beside_rows_of_any_size(swiglu):
    """Rows whose largest element is at either end of bf16's range with factors at the other: results that are ordinary
    numbers, and rows of weights that are 0."""
    rng = rng_of(12)
    b, sfb, w = operand(rng, 6, 64, 160)
    b[:, 5] = 0
    w[:, 5] = 0
    sizes = np.array([2.0 ** 120, 2.0 ** -110, 2.0 ** 100, 2.0 ** -90, 1.0, 2.0 ** -110])
    alpha = (rng.uniform(1, 2, 6) / sizes / 64).astype(np.float32)
    alpha[2] = 2.0 ** 90                              # results beyond fp32, but for the row of zeros
    alpha[5] = 2.0 ** -13 * 1.37                      # results of about 2^-118
    x = rng.standard_normal((6, 160)) * sizes[:, None]
    t = gpu(x, torch.bfloat16)
    ids = np.arange(6, dtype=np.int32)[:, None]
    y = moe.few_tokens(t, gpu(ids), b, sfb, alpha=gpu(alpha), swiglu=swiglu, dtype=torch.float32)
    want, size = MO.few(f64(t), ids, w, alpha)
    if swiglu:
        some = [0, 1, 3, 4, 5]
        bound = (160 + 16) * H[torch.float32] * size
        g, u = np.split(want, 2, axis=-1)
        bg, bu = np.split(bound, 2, axis=-1)
        silu = g / (1 + np.exp(-np.clip(g, -700, None)))
        close(y[some], (silu * u)[some], (1.1 * bg * (np.abs(u) + bu) + np.abs(silu) * bu + 16 * H[torch.float32] * np.abs(silu * u))[some],
              torch.float32)
    else:
        close(y, want, (160 + 16) * H[torch.float32] * np.minimum(size, 1e300), torch.float32)
        assert (y[:, 0, 5] == 0).all()


# ---- combine ----------------------------------------------------------------------------

@pytest.mark.parametrize("kind", TYPES)
def test_combine_of_no_rows(kind):
    """Experts' rows that are none: the residual alone, and gradients of 0."""
    x = torch.empty(0, 72, dtype=TYPES[kind], device="cuda")
    rows = torch.tensor([[-1, -1], [0, 7], [-1, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    w = torch.full((3, 2), float("nan"), device="cuda")
    residual = torch.randn(3, 72, device="cuda").to(TYPES[kind])
    assert torch.equal(moe.combine(x, w, rows, residual=residual), residual)
    assert (moe.combine(x, w, rows) == 0).all()
    dc, dw = moe.combine_backward(residual, x, w, rows)
    assert dc.shape == (0, 72) and (dw == 0).all()


@pytest.mark.parametrize("strided", [False, True])
def test_combine_gradient_of_rows_that_no_slot_has(strided):
    """0, in a gradient that the call allocates (whatever its memory held)."""
    rng = rng_of(44)
    ids = rng.integers(-1, 4, (64, 3)).astype(np.int32)
    store = gpu(rng.standard_normal((192, 80)), torch.float16)
    x = store[:, 8:72] if strided else store[:, :64].contiguous()
    w, dy = gpu(rng.uniform(0.1, 1, (64, 3)).astype(np.float32)), gpu(rng.standard_normal((64, 64)), torch.float32)
    p = moe.plan(gpu(ids), 4)
    want = MO.combine_backward(f64(dy), f64(x), f64(w), MO.plan(ids, 4)[2])[0]
    want = np.where(np.isnan(want), 0, want)
    for _ in range(3):
        for n in (192 * 64, 192 * 80):
            torch.full((n,), float("nan"), dtype=torch.float16, device="cuda")  # freed at once: what comes next may lie there
        dc, _ = moe.combine_backward(dy, x, w, p)
        assert dc.stride() == x.stride()
        close(dc, want, 3 * H[torch.float32] * np.abs(want), torch.float16)


# ---- choice values that are nearly equal ------------------------------------------------

def choice_values(x, how, bias):
    s = MO.scores(x, how["score"])
    return np.where(np.isneginf(x), -np.inf, s + (0 if bias is None else bias.astype(np.float64)))


def told_apart(values, count):
    """Tokens whose `count` largest values, and the next, differ from each other by more than 2^-41 or not at all (the
    kernels take what is within 2^-42 for equal)."""
    top = np.sort(values, axis=1)[:, ::-1][:, :count + 1]
    gap = top[:, :-1] - top[:, 1:]
    return ~((gap > 0) & (gap < 2.0 ** -41)).any(axis=1)


@pytest.mark.parametrize("step", [2.0 ** -24, 2.0 ** -23, 2.0 ** -22, 2.0 ** -21, 2.0 ** -20, 2.0 ** -19, 2.0 ** -18, 2.0 ** -17])
@pytest.mark.parametrize("score,experts,topk,dtype", [("sigmoid", 64, 6, "fp32"), ("softmax", 64, 6, "fp32"), ("sigmoid", 256, 8, "bf16"),
                                                      ("softmax", 40, 3, "fp32"), ("softmax", 8, 1, "fp16")])
def test_route_choice_values_around_the_margin(score, experts, topk, dtype, step):
    """Neighbouring choice values a few `step` apart, by the logits and by the bias: the ids are the exact values'."""
    rng = rng_of(experts, topk, int(-np.log2(step)))
    tokens = 1500
    slope = 0.24 if score == "sigmoid" else 1.0 / experts
    x = 0.3 + rng.integers(-3, 4, (tokens, experts)) * (step / slope)     # all scores nearly the same
    bias = (rng.integers(-4, 5, experts) * step * rng.choice([0.5, 1.0, 1.5], experts)).astype(np.float32)
    x[1::3] = rng.standard_normal((len(x[1::3]), experts))                # scores apart, the bias makes up for it
    x[2::3] = rng.standard_normal((len(x[2::3]), 1)) + rng.standard_normal((len(x[2::3]), experts)) * step * 8
    x[5::30, ::2] = x[5::30, 1::2]
    x[rng.random(x.shape) < 0.03] = -np.inf
    x = gpu(x, TYPES[dtype])
    how = dict(score=score)
    told = told_apart(choice_values(f64(x), how, bias), topk)
    assert told.mean() > 0.9
    want_ids, want_w = MO.route(f64(x), topk, bias=bias.astype(np.float64), **how)
    for many in (1, 90):                                                  # many lanes a token, and few
        ids, w = moe.route(x.repeat(many, 1), topk, bias=gpu(bias), **how)
        got = ids[-tokens:].cpu().numpy()
        assert np.array_equal(got[told], want_ids[told])
        assert torch.equal(ids[:tokens], ids[-tokens:])
        close(w[-tokens:][gpu(np.flatnonzero(told))], want_w[told], 64 * H[torch.float32] * want_w[told], torch.float32)


def test_route_bias_that_makes_up_for_the_scores():
    """Each token's own scores all over [0, 1], lifted by the bias to values that differ by 2^-22 or so: the margin where the
    scores' own errors are largest and differ."""
    for score, experts in (("sigmoid", 64), ("softmax", 24)):
        rng = rng_of(experts, 9)
        x = rng.standard_normal((1, experts)).astype(np.float32) * 2
        bias = (0.75 - MO.scores(x.astype(np.float64), score)[0] + rng.integers(-6, 7, experts) * 2.0 ** -24).astype(np.float32)
        x = np.repeat(x, 1200, axis=0)
        x += rng.integers(-3, 4, x.shape).astype(np.float32) * np.float32(2.0 ** -22)
        told = told_apart(choice_values(x.astype(np.float64), dict(score=score), bias), 6)
        assert told.mean() > 0.9
        ids, _ = moe.route(gpu(x), 6, bias=gpu(bias), score=score)
        want, _ = MO.route(x.astype(np.float64), 6, bias=bias.astype(np.float64), score=score)
        assert np.array_equal(ids.cpu().numpy()[told], want[told])


@pytest.mark.parametrize("experts,topk,how", [
    (40, 4, dict(score="softmax", groups=4, topk_groups=2, group_best=1)),
    (128, 8, dict(score="sigmoid", groups=8, topk_groups=4, group_best=2)),
    (60, 10, dict(score="softmax", groups=20, topk_groups=7, group_best=2))])
def test_route_groups_that_are_nearly_equal(experts, topk, how):
    """The same inputs as of the calls of many tokens against few, here against the oracle."""
    rng = rng_of(experts, 10)
    x = rng.standard_normal((900, experts))
    x[1::3] = x[1::3] * 1e-5 + 0.5
    x[2::6, ::2] = x[2::6, 1::2]
    x = x.astype(np.float32)
    bias = (rng.standard_normal(experts) * 1e-6).astype(np.float32)
    values = choice_values(x.astype(np.float64), how, bias)
    best = np.sort(values.reshape(900, how["groups"], -1), axis=2)[:, :, ::-1][:, :, :how["group_best"]].sum(2)
    told = told_apart(values, experts - 1) & told_apart(best, how["groups"] - 1)
    assert told.mean() > 0.9
    ids, _ = moe.route(gpu(x), topk, bias=gpu(bias), **how)
    want, _ = MO.route(x.astype(np.float64), topk, bias=bias.astype(np.float64), **how)
    assert np.array_equal(ids.cpu().numpy()[told], want[told])


# ---- more tiles than a launch can have -------------------------------------------------

def test_quantize_of_more_tiles_than_a_launch_holds():
    """2^22 batches and a few of 32 rows of 32, whose tiles would be more than 2^32 threads: to their codes and back."""
    l = (1 << 22) + 9
    x = torch.empty(l, 32, 32, dtype=torch.float16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(6))
    a, sfa = moe.quantize(x)
    values = moe.dequantize(a, sfa)
    for li in (0, 1, 8, 9, 1 << 21, l - 10, l - 9, l - 2, l - 1):
        codes, scales = MO.quantize(f64(x[li]))
        got_codes, got_scales = MO.unpack_rows(a[li].cpu().numpy(), sfa[li * 512:li * 512 + 512].cpu().numpy(), 32, 32)
        assert np.array_equal(got_codes, codes) and np.array_equal(got_scales, scales)
        assert np.array_equal(f64(values[li]), MO.values(codes, scales))
