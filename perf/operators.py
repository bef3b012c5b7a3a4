"""Speed and agreement of the mixture-of-experts operators around the grouped GEMM.

Five operators, each in the forms that a layer of experts needs:

* ``route``    - scores, choice of experts and weights; its gradient
* ``dispatch`` - rows sorted by expert, quantised to NVFP4 on the way
* ``quantize`` / ``swiglu`` - rows to NVFP4, plain or after the gated activation
* ``combine``  - weighted sum of the experts' rows; its gradient
* ``few``      - the experts' products of a few tokens, activations unquantised

and ``layer``, which runs them together around the grouped GEMM.

With ``own`` false, ``run`` computes each from elementary torch operations;
with ``own`` true it calls ``moe_matmul_amd.moe``. NVFP4 operands come back as
the values they stand for (E2M1 code times E4M3 scale: exact in fp16).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
DEVICE = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a serving step: latency of a biased, grouped choice of 8 in 256 experts
        dict(name="route_token", op="route", tokens=1, experts=256, topk=8, dtype="fp32", score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_best=2, renormalize=True, scale=2.5, masked=0.0, backward=False),
        # the same choice for a long prompt
        dict(name="route_prompt", op="route", tokens=16384, experts=256, topk=8, dtype="bf16", score="sigmoid",
             bias=True, groups=8, topk_groups=4, group_best=2, renormalize=True, scale=2.5, masked=0.0, backward=False),
        # a training batch: softmax scores as they are, forward and the dense gradient of the logits;
        # some experts are masked out, an odd number of tokens
        dict(name="route_train", op="route", tokens=65537, experts=64, topk=6, dtype="fp32", score="softmax",
             bias=False, groups=1, topk_groups=1, group_best=1, renormalize=False, scale=1.0, masked=0.05,
             backward=True),
        # a serving step of 33 sequences, spread over many experts (mostly one row or none each)
        dict(name="dispatch_step", op="dispatch", tokens=33, experts=256, topk=8, k=7168, dtype="bf16", dropped=0.0),
        # a prompt; a few slots have no expert on this device
        dict(name="dispatch_prompt", op="dispatch", tokens=4096, experts=64, topk=8, k=7168, dtype="bf16",
             dropped=0.05),
        # rows of a prompt before a product
        dict(name="quantize_rows", op="quantize", tokens=16384, k=7168, dtype="bf16"),
        # gate and up halves of the experts' first product, to the operand of the second
        dict(name="swiglu_rows", op="swiglu", tokens=8195, experts=32, topk=2, k=2048, dtype="fp16"),
        # experts' rows back to tokens, a prompt
        dict(name="combine_prompt", op="combine", tokens=8192, experts=64, topk=8, n=7168, dtype="bf16", dropped=0.05,
             backward=False),
        # its gradients, a training batch
        dict(name="combine_train", op="combine", tokens=4099, experts=32, topk=4, n=4096, dtype="bf16", dropped=0.0,
             backward=True),
        # one token through the first product of its eight experts: weight streaming
        dict(name="few_token", op="few", tokens=1, experts=32, topk=8, n=4096, k=7168, dtype="bf16", swiglu=True,
             per_slot=False),
        # a small serving batch through the second product
        dict(name="few_step", op="few", tokens=13, experts=8, topk=2, n=7168, k=2048, dtype="bf16", swiglu=False,
             per_slot=True),
        # the whole layer on a prompt: route, dispatch, product, activation, product, combine
        dict(name="layer_prompt", op="layer", tokens=1024, experts=8, topk=2, hidden=7168, inner=2048, dtype="bf16"),
    ]


def _spread(rng, low, high, step=1):
    """A multiple of ``step`` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high // step * step, max(-(-low // step) * step, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(["route", "route", "dispatch", "quantize", "swiglu", "combine", "few", "few", "layer"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _spread(rng, 4, 512 // groups if groups > 1 else 512)
        experts = groups * per
        kept = rng.randint(1, groups)
        topk = rng.randint(1, min(16, kept * per))
        return dict(op=op, tokens=_spread(rng, 1, 4_000_000 // max(experts, 64)), experts=experts, topk=topk,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, topk_groups=kept, group_best=rng.choice([1, 2]),
                    renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.1, 0.6]),
                    backward=rng.random() < 0.5)
    experts = _spread(rng, 4, 256)
    topk = rng.randint(1, min(8, experts))
    if op == "dispatch":
        k = _spread(rng, 64, 8192, 32)
        return dict(op=op, tokens=_spread(rng, 1, max(1, 200_000_000 // (k * topk))), experts=experts, topk=topk, k=k,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), dropped=rng.choice([0.0, 0.0, 0.1, 0.9]))
    if op == "quantize":
        k = _spread(rng, 32, 16384, 32)
        return dict(op=op, tokens=_spread(rng, 1, 100_000_000 // k), k=k, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "swiglu":
        k = _spread(rng, 32, 8192, 32)
        return dict(op=op, tokens=_spread(rng, 1, max(1, 30_000_000 // (k * topk))), experts=experts, topk=topk, k=k,
                    dtype=dtype)
    if op == "combine":
        n = _spread(rng, 8, 16384, 8)
        backward = rng.random() < 0.5
        return dict(op=op, tokens=_spread(rng, 1, max(1, (60_000_000 if backward else 400_000_000) // (n * topk))),
                    experts=experts, topk=topk, n=n, dtype=dtype, dropped=rng.choice([0.0, 0.0, 0.1, 0.9]),
                    backward=backward)
    if op == "few":
        experts = _spread(rng, 4, 32)
        topk = rng.randint(1, min(8, experts))
        n, k = _spread(rng, 64, 4096, 16), _spread(rng, 64, 7168, 32)
        return dict(op=op, tokens=_spread(rng, 1, 32), experts=experts, topk=topk, n=n, k=k, dtype=dtype,
                    swiglu=rng.random() < 0.5, per_slot=rng.random() < 0.5)
    experts = _spread(rng, 4, 16)
    return dict(op="layer", tokens=_spread(rng, 1, 512), experts=experts, topk=rng.randint(1, min(4, experts)),
                hidden=_spread(rng, 256, 4096, 64), inner=_spread(rng, 128, 1024, 64), dtype=dtype)


# ---------------------------------------------------------------- inputs

def _sf_bytes(rows, k):
    return (rows + 127) // 128 * 128 * ((k + 63) // 64) * 4


def _pick(g, tokens, experts, topk):
    """Distinct experts for each token, some experts more popular than others."""
    liked = torch.randn(experts, generator=g, device=DEVICE)
    noise = -torch.log(-torch.log(torch.rand(tokens, experts, generator=g, device=DEVICE).clamp(1e-7, 1 - 1e-7)))
    return torch.topk(liked * 0.5 + noise, topk, dim=1).indices.to(torch.int32)


def _drop(g, ids, share):
    return torch.where(torch.rand(ids.shape, generator=g, device=DEVICE) < share, -1, ids) if share else ids


def _activations(g, shape, dtype):
    """Roughly normal, with a few channels much larger than the rest."""
    x = torch.randn(shape, generator=g, device=DEVICE)
    x = x * (1 + 15 * (torch.rand(shape[-1], generator=g, device=DEVICE) < 0.01))
    return x.to(DTYPES[dtype])


def _operand(g, experts, rows, k):
    """NVFP4 weights of ``experts`` products: random codes, scales that give entries of about 1/sqrt(k)."""
    codes = torch.randint(0, 256, (experts, rows, k // 2), generator=g, device=DEVICE, dtype=torch.uint8)
    # E4M3 bytes of exponent field e and any mantissa: (1 + m/8) * 2^(e - 7)
    e = max(1, min(14, 7 + round(math.log2(1 / (2.8 * math.sqrt(k))))))
    sf = torch.randint(e * 8, (e + 1) * 8, (experts, _sf_bytes(rows, k)), generator=g, device=DEVICE, dtype=torch.uint8)
    return codes, sf


def _weights(g, ids):
    w = torch.rand(ids.shape, generator=g, device=DEVICE) + 0.05
    return w / w.sum(1, keepdim=True)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    c, s = case, dict(case=case)
    op = c["op"]
    if op == "route":
        x = torch.randn(c["tokens"], c["experts"], generator=g, device=DEVICE) * 1.5
        if c["masked"]:
            x.masked_fill_(torch.rand(x.shape, generator=g, device=DEVICE) < c["masked"], float("-inf"))
        s["logits"] = x.to(DTYPES[c["dtype"]])
        s["bias"] = torch.randn(c["experts"], generator=g, device=DEVICE) * 0.05 if c["bias"] else None
        s["dweights"] = torch.randn(c["tokens"], c["topk"], generator=g, device=DEVICE)
    elif op == "dispatch":
        s["ids"] = _drop(g, _pick(g, c["tokens"], c["experts"], c["topk"]), c["dropped"])
        s["x"] = _activations(g, (c["tokens"], c["k"]), c["dtype"])
        s["values"] = torch.zeros(c["tokens"] * c["topk"], c["k"], device=DEVICE, dtype=torch.float16)
    elif op == "quantize":
        s["x"] = _activations(g, (c["tokens"], c["k"]), c["dtype"])
    elif op == "swiglu":
        s["ids"] = _pick(g, c["tokens"], c["experts"], c["topk"])
        s["c"] = _activations(g, (c["tokens"] * c["topk"], 2 * c["k"]), c["dtype"])
        s["alpha"] = torch.rand(c["experts"], generator=g, device=DEVICE) + 0.5
    elif op == "combine":
        s["ids"] = _drop(g, _pick(g, c["tokens"], c["experts"], c["topk"]), c["dropped"])
        s["weights"] = _weights(g, s["ids"])
        s["rows"] = _slot_rows(s["ids"], c["experts"])[0]
        s["c"] = _activations(g, (c["tokens"] * c["topk"], c["n"]), "fp16")
        s["dy"] = _activations(g, (c["tokens"], c["n"]), c["dtype"])
        s["dc"] = torch.zeros_like(s["c"])
    elif op == "few":
        s["ids"] = _pick(g, c["tokens"], c["experts"], c["topk"])
        s["x"] = _activations(g, (c["tokens"], c["topk"], c["k"]) if c["per_slot"] else (c["tokens"], c["k"]), c["dtype"])
        s["b"], s["sfb"] = _operand(g, c["experts"], c["n"], c["k"])
        s["alpha"] = torch.rand(c["experts"], generator=g, device=DEVICE) + 0.5
    else:
        s["x"] = torch.randn(c["tokens"], c["hidden"], generator=g, device=DEVICE).to(DTYPES[c["dtype"]])
        s["logits"] = torch.randn(c["tokens"], c["experts"], generator=g, device=DEVICE).to(DTYPES[c["dtype"]])
        s["b1"], s["sfb1"] = _operand(g, c["experts"], 2 * c["inner"], c["hidden"])
        s["b2"], s["sfb2"] = _operand(g, c["experts"], c["hidden"], c["inner"])
    return s


# ---------------------------------------------------------------- plain forms

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _softmax(x):
    """Over the last axis; a row that is masked out whole gives zeros."""
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _score(x, kind):
    return _softmax(x) if kind == "softmax" else 1 / (1 + torch.exp(-x))


def _choose(c, logits, bias):
    """Expert ids by falling choice value, ties to the lowest id, -1 where no expert is left.

    Values that border on each other decide the order, so they are held in 64 bits."""
    x = logits.double()
    v = x if bias is None and c["groups"] == 1 else _score(x, c["score"])
    if bias is not None:
        v = v + bias.double()
    v = torch.where(x == -math.inf, -math.inf, v)
    if c["groups"] > 1:
        parts = v.view(v.shape[0], c["groups"], -1)
        best = torch.sort(parts, dim=2, descending=True).values[:, :, :c["group_best"]]
        found = best > -math.inf
        of = torch.where(found, best, torch.zeros_like(best)).sum(2)
        of = torch.where(found.any(2), of, -math.inf)
        kept = torch.sort(of, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros_like(of, dtype=torch.bool).scatter(1, kept, True)
        v = torch.where(keep.unsqueeze(2), parts, -math.inf).view_as(v)
    top, ids = torch.sort(v, dim=1, descending=True, stable=True)
    top, ids = top[:, :c["topk"]], ids[:, :c["topk"]]
    return torch.where(top == -math.inf, -1, ids).to(torch.int32)


def _route_weights(c, x, ids):
    """(weights, scores of the chosen, their sum, scores of all) in x's type."""
    p = _score(x, c["score"])
    chosen = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0).long()), torch.zeros((), dtype=x.dtype, device=x.device))
    total = chosen.sum(1, keepdim=True) if c["renormalize"] else torch.ones_like(chosen[:, :1])
    total = torch.where(total == 0, torch.ones_like(total), total)
    return chosen / total * c["scale"], chosen, total, p


def _route_gradient(c, x, ids, dweights):
    """d logits, in x's type."""
    _, chosen, total, p = _route_weights(c, x, ids)
    dw = torch.where(ids >= 0, dweights.to(x.dtype), torch.zeros((), dtype=x.dtype, device=x.device)) * c["scale"]
    if c["renormalize"]:
        dw = (dw - (dw * chosen / total).sum(1, keepdim=True)) / total
    # ids of -1 add zero to expert 0
    dp = torch.zeros_like(p).scatter_add(1, ids.clamp(min=0).long(), torch.where(ids >= 0, dw, torch.zeros_like(dw)))
    if c["score"] == "sigmoid":
        return dp * p * (1 - p)
    return p * (dp - (dp * p).sum(1, keepdim=True))


def _slot_rows(ids, experts):
    """Rows sorted by expert, in slot order within one: (row of each slot, slot of each row, row offset of each expert)."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= experts), experts, flat)
    key, order = torch.sort(key, stable=True)
    rows = torch.arange(flat.numel(), device=flat.device)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=flat.device))
    used = rows < offsets[-1]
    slot_rows = torch.empty_like(flat).scatter(0, order, torch.where(used, rows, -1))
    row_slots = torch.where(used, order, -1)
    return slot_rows.view(ids.shape).to(torch.int32), row_slots.to(torch.int32), offsets.to(torch.int32)


def _nvfp4(v):
    """The values that NVFP4 operands of the rows ``v`` stand for, in fp32.

    Quotients on a border between two codes decide which it is, so they are held in 64 bits."""
    blocks = v.reshape(v.shape[0], -1, 16).double()
    scales = torch.arange(127, dtype=torch.uint8, device=v.device).view(torch.float8_e4m3fn).double()
    top, borders = blocks.abs().amax(2, keepdim=True), (scales[1:] + scales[:-1]) * 3  # six times the middle of two
    below, above = torch.bucketize(top, borders), torch.bucketize(top, borders, right=True)
    scale = scales[torch.where(below % 2 == 0, below, above)]  # the even code where both are as near
    q = torch.where(scale == 0, torch.zeros_like(blocks), blocks / scale)
    a = q.abs()
    # nearest E2M1 value, ties to the even code
    code = ((a > 0.25).to(torch.int32) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    value = torch.tensor(E2M1, device=v.device)[code.long()]
    return (torch.where(q < 0, -value, value) * scale.float()).view(v.shape)


def _silu_mul(c):
    gate, up = c.chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _unpack(codes, sf, dtype=torch.float32):
    """[experts, rows, k] values of packed codes and tiled scales."""
    experts, rows, half = codes.shape
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=codes.device, dtype=dtype)
    v = table[torch.stack((codes & 15, codes >> 4), dim=3).view(experts, rows, 2 * half).long()]
    # a scale atom is [32 rows][4 blocks of 32 rows][4 scales along k]
    atoms = sf.view(torch.float8_e4m3fn).to(dtype).view(experts, (rows + 127) // 128, -1, 32, 4, 4)
    scale = atoms.permute(0, 1, 4, 3, 2, 5).reshape(experts, (rows + 127) // 128 * 128, -1)[:, :rows, :half // 8]
    return (v.view(experts, rows, half // 8, 16) * scale.unsqueeze(3)).view(experts, rows, 2 * half)


def _few(x, ids, w, alpha, swiglu):
    """x [tokens, k] or [tokens, topk, k] times the chosen experts' weights: [tokens, topk, n]."""
    tokens, topk = ids.shape
    at = torch.arange(tokens * topk, device=ids.device).view(tokens, topk)
    at = at if x.dim() == 3 else at // topk
    y = torch.matmul(x.reshape(-1, x.shape[-1]), w.transpose(1, 2))[ids.long(), at]
    y = y * alpha[ids.long()].unsqueeze(2)
    return _silu_mul(y) if swiglu else y


def _layer(c, s, wide):
    """The layer's answer; ``wide`` is the type it is computed in. Products are rounded to fp16, as the grouped GEMM
    writes them."""
    ids = _choose(_layer_route(c), s["logits"], None)
    weights = _route_weights(_layer_route(c), s["logits"].to(wide), ids)[0]
    x = (_nvfp4 if wide == torch.float32 else _nvfp4_exact)(s["x"].to(wide))
    h = torch.matmul(x, _unpack(s["b1"], s["sfb1"], wide).transpose(1, 2)).half().to(wide)
    h = _silu_mul(h).view(-1, c["inner"])
    h = (_nvfp4 if wide == torch.float32 else _nvfp4_exact)(h).view(c["experts"], c["tokens"], c["inner"])
    y = torch.matmul(h, _unpack(s["b2"], s["sfb2"], wide).transpose(1, 2)).half().to(wide)
    y = y[ids.long(), torch.arange(c["tokens"], device=ids.device).unsqueeze(1)]
    return ids, weights, (y * weights.unsqueeze(2)).sum(1)


def _layer_route(c):
    return dict(score="softmax", groups=1, topk=c["topk"], renormalize=True, scale=1.0)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        ids = _choose(c, s["logits"], s["bias"])
        x = s["logits"].float()
        out = dict(ids=ids, weights=_route_weights(c, x, ids)[0])
        if c["backward"]:
            out["dlogits"] = _route_gradient(c, x, ids, s["dweights"]).to(s["logits"].dtype)
        return out
    if op == "dispatch":
        slot_rows, row_slots, offsets = _slot_rows(s["ids"], c["experts"])
        v = _nvfp4(s["x"].float()).half()[(row_slots.clamp(min=0) // c["topk"]).long()]
        return dict(slot_rows=slot_rows, row_slots=row_slots, offsets=offsets,
                    values=torch.where(row_slots.unsqueeze(1) >= 0, v, torch.zeros_like(v)))
    if op == "quantize":
        return _nvfp4(s["x"].float()).half()
    if op == "swiglu":
        offsets = _slot_rows(s["ids"], c["experts"])[2]
        of = torch.searchsorted(offsets[1:].contiguous(), torch.arange(s["c"].shape[0], device=DEVICE, dtype=torch.int32),
                                right=True)
        # in 64 bits: an activation next to a border between two codes decides which it is
        return _nvfp4(_silu_mul(s["c"].double() * s["alpha"][of].double().unsqueeze(1))).half()
    if op == "combine":
        rows, w = s["rows"], s["weights"]
        there = (rows >= 0).unsqueeze(2)
        v = torch.where(there, s["c"][rows.clamp(min=0).long()].float(), torch.zeros((), device=DEVICE))
        if not c["backward"]:
            return (v * w.unsqueeze(2)).sum(1).to(DTYPES[c["dtype"]])
        dy = s["dy"].float().unsqueeze(1)
        # slots without a row write to one more row, which is cut off
        at = torch.where(rows >= 0, rows, s["c"].shape[0]).reshape(-1).long()
        dc = torch.zeros(s["c"].shape[0] + 1, c["n"], device=DEVICE, dtype=torch.float16)
        dc[at] = (dy * w.unsqueeze(2)).half().view(-1, c["n"])
        return dict(dc=dc[:-1], dweights=(v * dy).sum(2))
    if op == "few":
        return _few(s["x"].float(), s["ids"], _unpack(s["b"], s["sfb"]), s["alpha"], c["swiglu"]).to(s["x"].dtype)
    ids, weights, y = _layer(c, s, torch.float32)
    return dict(ids=ids, weights=weights, y=y.to(s["x"].dtype))


# ---------------------------------------------------------------- the framework's operators

def _own(s):
    from moe_matmul_amd import moe
    c = s["case"]
    op = c["op"]
    if op == "route":
        how = dict(score=c["score"], renormalize=c["renormalize"], scale=c["scale"])
        ids, weights = moe.route(s["logits"], c["topk"], bias=s["bias"], groups=c["groups"],
                                 topk_groups=c["topk_groups"], group_best=c["group_best"], **how)
        out = dict(ids=ids, weights=weights)
        if c["backward"]:
            out["dlogits"] = moe.route_backward(s["logits"], ids, s["dweights"], **how)
        return out
    if op == "dispatch":
        p = moe.plan(s["ids"], c["experts"])
        a, sfa = moe.quantize(s["x"], plan=p)
        values = moe.dequantize(a, sfa, plan=p, out=s["values"])
        return dict(slot_rows=p.slot_rows, row_slots=p.row_slots, offsets=p.offsets, values=values)
    if op == "quantize":
        a, sfa = moe.quantize(s["x"])
        return moe.dequantize(a, sfa)
    if op == "swiglu":
        p = moe.plan(s["ids"], c["experts"])
        a, sfa = moe.swiglu_quantize(s["c"], plan=p, alpha=s["alpha"])
        return moe.dequantize(a, sfa, plan=p)
    if op == "combine":
        if c["backward"]:
            dc, dweights = moe.combine_backward(s["dy"], s["c"], s["weights"], s["rows"], dc=s["dc"])
            return dict(dc=dc, dweights=dweights)
        return moe.combine(s["c"], s["weights"], s["rows"], dtype=DTYPES[c["dtype"]])
    if op == "few":
        return moe.few_tokens(s["x"], s["ids"], s["b"], s["sfb"], alpha=s["alpha"], swiglu=c["swiglu"])
    if "layer" not in s:  # a program makes its layer once, with the weights
        s["layer"] = moe.FeedForward(s["b1"], s["sfb1"], s["b2"], s["sfb2"])
    ids, weights = moe.route(s["logits"], c["topk"])
    return dict(ids=ids, weights=weights, y=s["layer"].grouped(s["x"], ids, weights))


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    t = c["tokens"]
    if op == "route":
        e, size = c["experts"], SIZE[c["dtype"]]
        passes = 3 if c["backward"] else 1  # the gradient reads the logits again and writes their like
        return dict(bytes=t * e * size * passes + t * c["topk"] * (20 if c["backward"] else 8), flops=8 * t * e * passes)
    if op == "quantize":
        return dict(bytes=t * c["k"] * (SIZE[c["dtype"]] + 2 * 9 / 16 + 2), flops=6 * t * c["k"])
    r = t * c["topk"]
    if op == "dispatch":
        r *= 1 - c["dropped"]
        return dict(bytes=t * c["k"] * SIZE[c["dtype"]] + r * c["k"] * (2 * 9 / 16 + 2) + 12 * t * c["topk"],
                    flops=6 * t * c["k"])
    if op == "swiglu":
        return dict(bytes=r * c["k"] * (2 * SIZE[c["dtype"]] + 2 * 9 / 16 + 2) + 12 * r, flops=20 * r * c["k"])
    if op == "combine":
        r *= 1 - c["dropped"]
        if c["backward"]:
            return dict(bytes=c["n"] * (t * SIZE[c["dtype"]] + 4 * r) + 12 * t * c["topk"], flops=3 * r * c["n"])
        return dict(bytes=c["n"] * (t * SIZE[c["dtype"]] + 2 * r) + 8 * t * c["topk"], flops=2 * r * c["n"])
    used = c["experts"] * (1 - (1 - c["topk"] / c["experts"]) ** t)  # experts that some token chose
    if op == "few":
        x = (r if c["per_slot"] else t) * c["k"] * SIZE[c["dtype"]]
        y = r * c["n"] // (2 if c["swiglu"] else 1) * SIZE[c["dtype"]]
        return dict(bytes=used * c["n"] * c["k"] * 9 / 16 + x + y, flops=2 * r * c["n"] * c["k"])
    h, i = c["hidden"], c["inner"]
    moved = t * h * 2 * SIZE[c["dtype"]] + r * 9 / 16 * 2 * (h + i) + r * 2 * 2 * (2 * i + h)
    return dict(bytes=used * 3 * h * i * 9 / 16 + moved, flops=2 * r * 3 * h * i)


# ---------------------------------------------------------------- the definition in 64 bits

def _power(x, least):
    """The power of two at or below each x, ``least`` at the least."""
    return (x.view(torch.int64) & 0x7FF0000000000000).view(torch.float64).clamp(min=least)


def _nvfp4_exact(v):
    """Nearest E4M3 scale of a sixth of each block's largest entry, nearest E2M1 multiple of it, ties to even."""
    b = v.double().unflatten(1, (-1, 16))
    top = b.abs().amax(2, keepdim=True)
    top = top / torch.full_like(top, 6)
    step = _power(top, 2.0 ** -6) / 8
    scale = (torch.round(top / step) * step).clamp(max=448)
    q = b / scale.clamp(min=2.0 ** -9)
    step = _power(q.abs(), 1.0) / 2
    return ((torch.round(q / step) * step).clamp(-6, 6) * scale).flatten(1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "route":
        x, e = s["logits"].double(), c["experts"]
        ids = _choose(c, s["logits"], s["bias"])
        # the weights and their gradient through torch's own differentiation of the formula
        x.requires_grad_(c["backward"])
        dead = (x.detach() == -math.inf).all(1, keepdim=True)
        p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(torch.where(dead, torch.zeros_like(x), x), 1)
        one = (ids.unsqueeze(2) == torch.arange(e, device=DEVICE)).double()  # [tokens, topk, experts]
        w = (one * p.unsqueeze(1)).sum(2)
        if c["renormalize"]:
            w = w / torch.where(w.sum(1, keepdim=True) == 0, 1.0, w.sum(1, keepdim=True))
        w = w * c["scale"]
        out = dict(ids=None, weights=w.detach())
        if c["backward"]:
            (w * s["dweights"].double()).sum().backward()
            out["dlogits"] = torch.nan_to_num(x.grad)
        return out
    if op == "dispatch":
        _, row_slots, _ = _slot_rows(s["ids"], c["experts"])
        v = _nvfp4_exact(s["x"])[(row_slots.clamp(min=0) // c["topk"]).long()]
        return dict(slot_rows=None, row_slots=None, offsets=None, values=v * (row_slots >= 0).unsqueeze(1))
    if op == "quantize":
        return _nvfp4_exact(s["x"])
    if op == "swiglu":
        counts = torch.bincount(s["ids"].reshape(-1).long(), minlength=c["experts"])
        gate, up = (s["c"].double() * torch.repeat_interleave(s["alpha"].double(), counts).unsqueeze(1)).chunk(2, 1)
        return _nvfp4_exact(gate * torch.sigmoid(gate) * up)
    if op == "combine":
        y, dc, dw = [], torch.zeros(s["c"].shape, device=DEVICE, dtype=torch.float64), []
        for j in range(c["topk"]):
            r, w = s["rows"][:, j].long(), s["weights"][:, j:j + 1].double()
            live = (r >= 0).double().unsqueeze(1)
            v = s["c"][r.clamp(min=0)].double() * live
            y.append(v * w)
            if c["backward"]:
                dc.index_add_(0, r.clamp(min=0), s["dy"].double() * w * live)
                dw.append((v * s["dy"].double()).sum(1))
        return dict(dc=dc, dweights=torch.stack(dw, 1)) if c["backward"] else sum(y)
    if op == "few":
        w, n = _unpack(s["b"], s["sfb"], torch.float64), c["n"]
        x = s["x"].double()
        out = torch.empty(c["tokens"], c["topk"], n, device=DEVICE, dtype=torch.float64)
        for t, row in enumerate(s["ids"].tolist()):
            for j, e in enumerate(row):
                out[t, j] = w[e] @ (x[t, j] if c["per_slot"] else x[t]) * s["alpha"][e].double()
        if c["swiglu"]:
            gate, up = out[..., :n // 2], out[..., n // 2:]
            out = gate * torch.sigmoid(gate) * up
        return out
    ids, weights, y = _layer(c, s, torch.float64)
    return dict(ids=None, weights=weights, y=y)
