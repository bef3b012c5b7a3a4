"""Speed and agreement of the feed-forward block in 16 bits and its training.

Four operators, dense or by the experts that a plan sorts rows by:

* ``norm``   - root-mean-square norm of a sum with the residual, its rows in 16 or in 8 bits; its gradient
* ``rows8``  - activations kept in 8 bits with a scale for 32 of them (checkpoints)
* ``linear`` - product with bias, activation and residual in its epilogue; its gradients
* ``gated``  - both projections of a gated feed-forward block, the activation and the product; its gradients,
  from activations kept in 16 or in 8 bits

With ``own`` false, ``run`` computes each from elementary torch operations in 32 bits; with ``own`` true it calls
``moe_matmul_amd.ffn``. Rows in 8 bits come back as the values that they stand for (E4M3 code times power of two).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
DEVICE = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a serving step: latency of the norm before a layer
        dict(name="norm_token", op="norm", rows=1, n=7168, dtype="bf16", residual=True, eight=False, backward=False),
        # a prompt, its rows kept in 8 bits
        dict(name="norm_prompt8", op="norm", rows=16384, n=7168, dtype="bf16", residual=True, eight=True,
             backward=False),
        # a training batch: forward, and the gradients of the sum and of the weight; an odd number of rows
        dict(name="norm_train", op="norm", rows=8195, n=4096, dtype="fp16", residual=True, eight=False, backward=True),
        # activations of a batch to 8 bits and back
        dict(name="rows8_batch", op="rows8", rows=16390, n=2048, dtype="bf16"),
        # one token through a down projection with the residual: weight streaming
        dict(name="linear_token", op="linear", rows=1, n=7168, k=2048, dtype="bf16", bias=False, activation="none",
             residual=True, experts=0, topk=1, dropped=0.0, backward=False),
        # a serving step of 33 sequences, with bias and activation
        dict(name="linear_step", op="linear", rows=33, n=4096, k=7168, dtype="fp16", bias=True, activation="gelu",
             residual=False, experts=0, topk=1, dropped=0.0, backward=False),
        # the down projection of a prompt with its residual
        dict(name="linear_prompt", op="linear", rows=4096, n=7168, k=2048, dtype="bf16", bias=False, activation="none",
             residual=True, experts=0, topk=1, dropped=0.0, backward=False),
        # a training step: forward and all gradients, ragged in rows and columns
        dict(name="linear_train", op="linear", rows=2051, n=4104, k=2048, dtype="bf16", bias=True, activation="silu",
             residual=False, experts=0, topk=1, dropped=0.0, backward=True),
        # one token through both projections of a shared expert
        dict(name="gated_token", op="gated", rows=1, hidden=7168, inner=2048, dtype="bf16", experts=0, topk=1,
             dropped=0.0, keep="none", backward=False),
        # a prompt through them
        dict(name="gated_prompt", op="gated", rows=8192, hidden=7168, inner=2048, dtype="bf16", experts=0, topk=1,
             dropped=0.0, keep="none", backward=False),
        # a training step that keeps its rows and both projections in 8 bits
        dict(name="gated_train8", op="gated", rows=4099, hidden=7168, inner=2048, dtype="bf16", experts=0, topk=1,
             dropped=0.0, keep="rows8", backward=True),
        # a training step of eight experts, two for each token, a few slots dropped
        dict(name="gated_experts", op="gated", rows=2048, hidden=4096, inner=1024, dtype="bf16", experts=8, topk=2,
             dropped=0.05, keep="rows", backward=True),
    ]


def _spread(rng, low, high, step=1):
    """A multiple of ``step`` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high // step * step, max(-(-low // step) * step, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "rows8", "linear", "linear", "linear", "gated", "gated", "gated"])
    if op == "norm":
        eight = rng.random() < 0.4
        n = _spread(rng, 64, 16384, 32 if eight else 8)
        return dict(op=op, rows=_spread(rng, 1, 100_000_000 // n), n=n, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    residual=rng.random() < 0.7, eight=eight, backward=not eight and rng.random() < 0.5)
    if op == "rows8":
        n = _spread(rng, 32, 16384, 32)
        return dict(op=op, rows=_spread(rng, 1, 100_000_000 // n), n=n, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    experts = rng.choice([0, 0, 0, 2, 4, 8, 16])
    topk = rng.randint(1, min(4, experts)) if experts else 1
    dropped = rng.choice([0.0, 0.1, 0.5]) if experts else 0.0
    backward = rng.random() < 0.5
    dtype = rng.choice(["bf16", "fp16"])
    # at most so many multiplications, and so many weights over all experts
    most = 4e10 if backward else 1e11
    if op == "linear":
        n, k = _spread(rng, 64, 8192, 8), _spread(rng, 64, 8192, 8)
        while n * k * max(experts, 1) > 2e8:
            n, k = max(64, n // 16 * 8), max(64, k // 16 * 8)
        return dict(op=op, rows=_spread(rng, 1, max(1, min(16384, int(most / (n * k * topk))))), n=n, k=k, dtype=dtype,
                    bias=rng.random() < 0.5, activation=rng.choice(["none", "none", "relu", "silu", "gelu"]),
                    residual=rng.random() < 0.4, experts=experts, topk=topk, dropped=dropped, backward=backward)
    hidden, inner = _spread(rng, 64, 8192, 32), _spread(rng, 64, 4096, 32)
    while 2 * hidden * inner * max(experts, 1) > 2e8:
        hidden, inner = max(64, hidden // 64 * 32), max(64, inner // 64 * 32)
    return dict(op=op, rows=_spread(rng, 1, max(1, min(16384, int(most / (2 * hidden * inner * topk))))), hidden=hidden,
                inner=inner, dtype=dtype, experts=experts, topk=topk, dropped=dropped,
                keep=rng.choice(["rows", "rows8", "none"]) if backward else "none", backward=backward)


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE)


def _activations(g, shape, dtype):
    """Roughly normal, with a few channels much larger than the rest."""
    x = _randn(g, *shape)
    return (x * (1 + 15 * (torch.rand(shape[-1], generator=g, device=DEVICE) < 0.01))).to(DTYPES[dtype])


def _weights(g, experts, n, k, dtype):
    """Entries of about k ** -0.5; [n, k], or [experts, n, k]."""
    return _randn(g, *((experts, n, k) if experts else (n, k))).mul_(k ** -0.5).to(DTYPES[dtype])


def _pick(g, c, s):
    """Distinct experts for each token, some more popular than others and a few slots dropped; the rows of the most
    popular one, to which a program that pads its experts' rows pads them."""
    e = c["experts"]
    if not e:
        return
    liked = _randn(g, e) * 0.5
    noise = -torch.log(-torch.log(torch.rand(c["rows"], e, generator=g, device=DEVICE).clamp(1e-7, 1 - 1e-7)))
    ids = torch.topk(liked + noise, c["topk"], dim=1).indices.to(torch.int32)
    s["ids"] = torch.where(torch.rand(ids.shape, generator=g, device=DEVICE) < c["dropped"], -1, ids)
    s["room"] = max(1, int(torch.bincount(s["ids"].reshape(-1).long() + 1, minlength=e + 1)[1:].max()))


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    c, s = case, dict(case=case)
    dtype, rows = c["dtype"], c["rows"]
    if c["op"] == "norm":
        s["x"] = _activations(g, (rows, c["n"]), dtype)
        s["residual"] = _activations(g, (rows, c["n"]), dtype) if c["residual"] else None
        s["weight"] = _randn(g, c["n"]) * 0.1 + 1
        if c["backward"]:
            s["dy"], s["dsum"] = _randn(g, rows, c["n"]).to(DTYPES[dtype]), _randn(g, rows, c["n"]).to(DTYPES[dtype])
    elif c["op"] == "rows8":
        s["x"] = _activations(g, (rows, c["n"]), dtype)
    elif c["op"] == "linear":
        _pick(g, c, s)
        rows, n = rows * c["topk"], c["n"]
        s["x"] = _activations(g, (rows, c["k"]), dtype)
        s["w"] = _weights(g, c["experts"], n, c["k"], dtype)
        s["bias"] = _randn(g, *s["w"].shape[:-1]).to(DTYPES[dtype]) if c["bias"] else None
        s["residual"] = _randn(g, rows, n).to(DTYPES[dtype]) if c["residual"] else None
        s["dy"] = _randn(g, rows, n).to(DTYPES[dtype]) if c["backward"] else None
    else:
        _pick(g, c, s)
        s["x"] = _randn(g, rows, c["hidden"]).to(DTYPES[dtype])
        s["w"] = _weights(g, c["experts"], 2 * c["inner"], c["hidden"], dtype)
        s["dh"] = _randn(g, rows * c["topk"], c["inner"]).to(DTYPES[dtype]) if c["backward"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _rows8(v):
    """The values that rows kept in 8 bits stand for: for every 32 the least power of two (2^-126 at the least) under
    which the largest is at most 448, and the E4M3 value nearest to each quotient."""
    b = v.unflatten(-1, (-1, 32))
    part, power = torch.frexp(b.abs().amax(-1, keepdim=True))  # the largest is part * 2^power, part in [0.5, 1)
    power = (power - torch.where(part <= 0.875, 9, 8)).clamp(min=-126)
    scale = torch.exp2(power.double()).to(v.dtype)
    return ((b / scale).float().to(torch.float8_e4m3fn).to(v.dtype) * scale).flatten(-2)


def _norm(v, weight):
    """(the norm of the rows v, v divided by its root mean square, one over that)"""
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * r * weight, v * r, r


def _norm_backward(dy, hat, r, weight, dsum):
    dhat = dy * weight
    return r * (dhat - hat * (dhat * hat).mean(1, keepdim=True)) + dsum, (dy * hat).sum(0)


def _cdf(z):
    """The normal distribution's."""
    return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))


def _act(z, kind):
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z * _cdf(z) if kind == "gelu" else z


def _act_slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return _cdf(z) + z * torch.exp(z * z * -0.5) * (2 * math.pi) ** -0.5 if kind == "gelu" else torch.ones_like(z)


class _Sorted:
    """Rows sorted by expert, and padded to [experts, room, ...] for batched products. Rows of slots that were dropped
    come last."""

    def __init__(self, s):
        c = s["case"]
        self.experts, self.room, self.topk = c["experts"], s["room"], c["topk"]
        flat = s["ids"].reshape(-1).long()
        key, self.slots = torch.sort(torch.where(flat < 0, self.experts, flat), stable=True)
        begin = torch.searchsorted(key, torch.arange(self.experts + 1, device=key.device))
        self.expert, self.live = key, (key < self.experts).unsqueeze(1)
        self.at = (torch.arange(key.numel(), device=key.device) - begin[key]).clamp(max=self.room - 1)

    def pad(self, rows):
        out = torch.zeros(self.experts + 1, self.room, rows.shape[1], dtype=rows.dtype, device=rows.device)
        out[self.expert, self.at] = rows
        return out[:-1]

    def rows(self, padded):
        v = padded[self.expert.clamp(max=self.experts - 1), self.at]
        return torch.where(self.live, v, torch.zeros_like(v))

    def tokens(self, rows):
        """The sum of each token's rows."""
        return torch.zeros_like(rows).index_copy(0, self.slots, rows).view(-1, self.topk, rows.shape[1]).sum(1)


def _times(a, b, order):
    """a b^T of rows by expert, or of all."""
    return torch.matmul(a, b.transpose(-1, -2)) if order else torch.matmul(a, b)


def _linear(s, order, wide):
    """y, and with a gradient to come dx, dw and dbias, in the type ``wide``."""
    c = s["case"]
    x, w = s["x"].to(wide), s["w"].to(wide)
    xs = order.pad(x) if order else x
    z = _times(xs, w, True)
    if s["bias"] is not None:
        z = z + s["bias"].to(wide).unsqueeze(-2)
    y = _act(z, c["activation"])
    y = order.rows(y) if order else y
    if s["residual"] is not None:
        y = y + (torch.where(order.live, s["residual"].to(wide), 0.0) if order else s["residual"].to(wide))
    if not c["backward"]:
        return dict(y=y)
    dz = (order.pad(s["dy"].to(wide)) if order else s["dy"].to(wide)) * _act_slope(z, c["activation"])
    dx = _times(dz, w, False)
    out = dict(y=y, dx=order.rows(dx) if order else dx, dw=_times(dz.transpose(-1, -2), xs, False))
    return out if s["bias"] is None else dict(out, dbias=dz.sum(-2))


def _gated(s, order, wide):
    """h, and with a gradient to come dx and dw, in the type ``wide``."""
    c = s["case"]
    x, w = s["x"].to(wide), s["w"].to(wide)
    take = (lambda v: order.pad(v[order.slots // c["topk"]])) if order else (lambda v: v)
    z = _times(take(x), w, True)
    g, u = z.chunk(2, -1)
    h = _act(g, "silu") * u
    out = dict(h=order.rows(h) if order else h)
    if not c["backward"]:
        return out
    if c["keep"] == "rows8":
        x = _rows8(x)
        g, u = _rows8(z).chunk(2, -1)
    dh = order.pad(s["dh"].to(wide)) if order else s["dh"].to(wide)
    dz = torch.cat((dh * u * _act_slope(g, "silu"), dh * _act(g, "silu")), -1)
    dx = _times(dz, w, False)
    return dict(out, dx=order.tokens(order.rows(dx)) if order else dx,
                dw=_times(dz.transpose(-1, -2), take(x), False))


def _compute(s, wide):
    c = s["case"]
    if c["op"] == "norm":
        total = s["x"] if s["residual"] is None else (s["x"].to(wide) + s["residual"].to(wide)).to(s["x"].dtype)
        weight = s["weight"].to(wide)
        y, hat, r = _norm(total.to(wide), weight)
        if c["eight"]:
            return dict(sum=total, y=_rows8(y))
        if not c["backward"]:
            return dict(sum=total, y=y)
        dx, dweight = _norm_backward(s["dy"].to(wide), hat, r, weight, s["dsum"].to(wide))
        return dict(sum=total, y=y, dx=dx, dweight=dweight)
    if c["op"] == "rows8":
        return dict(values=_rows8(s["x"].to(wide)))
    order = _Sorted(s) if c["experts"] else None
    return (_linear if c["op"] == "linear" else _gated)(s, order, wide)


def _plain(s):
    dtype = s["x"].dtype
    return {name: v if name == "dweight" else v.to(dtype) for name, v in _compute(s, torch.float32).items()}


# ---------------------------------------------------------------- the framework's operators

def _own(s):
    from moe_matmul_amd import ffn, moe
    c = s["case"]
    x = s["x"]
    if c["op"] == "norm":
        n = ffn.rmsnorm(x, s["weight"], residual=s["residual"], eps=EPS, rows=not c["eight"], rows8=c["eight"])
        if c["eight"]:
            return dict(sum=n.sum, y=ffn.dequantize8(n.y8, dtype=x.dtype))
        if not c["backward"]:
            return dict(sum=n.sum, y=n.y)
        dx, dweight = ffn.rmsnorm_backward(s["dy"], n.sum, s["weight"], n.rstd, dsum=s["dsum"])
        return dict(sum=n.sum, y=n.y, dx=dx, dweight=dweight)
    if c["op"] == "rows8":
        return dict(values=ffn.dequantize8(ffn.quantize8(x), dtype=x.dtype))
    plan = moe.plan(s["ids"], c["experts"]) if c["experts"] else None
    if c["op"] == "linear":
        how = dict(activation=None if c["activation"] == "none" else c["activation"], plan=plan)
        if not c["backward"]:
            return dict(y=ffn.linear(x, s["w"], bias=s["bias"], residual=s["residual"], **how))
        y, z = ffn.linear(x, s["w"], bias=s["bias"], residual=s["residual"], save=True, **how)
        dx, dw, dbias = ffn.linear_backward(s["dy"], x, s["w"], bias=s["bias"], z=z, **how)
        return dict(y=y, dx=dx, dw=dw) if dbias is None else dict(y=y, dx=dx, dw=dw, dbias=dbias)
    if not c["backward"]:
        return dict(h=ffn.gated(x, s["w"], plan=plan))
    if c["keep"] == "none":  # both projections are computed again for the gradients
        h, kept = ffn.gated(x, s["w"], plan=plan), None
    else:
        h, kept = ffn.gated(x, s["w"], plan=plan, save=c["keep"])
    rows = ffn.quantize8(x) if c["keep"] == "rows8" else x
    dx, dw = ffn.gated_backward(s["dh"], rows, s["w"], kept, plan=plan)
    return dict(h=h, dx=dx, dw=dw)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, size, rows = case, SIZE[case["dtype"]], case["rows"]
    if c["op"] == "rows8":
        return dict(bytes=rows * c["n"] * (2 * size + 2 * 33 / 32), flops=4 * rows * c["n"])
    if c["op"] == "norm":
        e = rows * c["n"]
        # x, the residual, the sum and the norm; with 8 bits their codes and the values; with gradients the sum again,
        # dy, the sum's gradient and dx
        moved = size * (1 + 2 * c["residual"]) + (2 * 33 / 32 + size if c["eight"] else size) + 4 * size * c["backward"]
        return dict(bytes=e * moved + 8 * c["n"], flops=e * (14 if c["backward"] else 5))
    experts, topk = max(c["experts"], 1), c["topk"]
    used = experts * (1 - (1 - topk * (1 - c["dropped"]) / experts) ** rows) if c["experts"] else 1  # that some row has
    live = rows * topk * (1 - c["dropped"])
    if c["op"] == "linear":
        n, k = c["n"], c["k"]
        moved = size * (used * n * k + live * (k + n * (1 + c["residual"])))
        if c["backward"]:
            moved += size * (used * n * k + experts * n * k + live * (2 * k + n))
        return dict(bytes=moved, flops=2 * live * n * k * (3 if c["backward"] else 1))
    h, i = c["hidden"], c["inner"]
    moved = size * (used * 2 * h * i + rows * h + live * i)
    if c["backward"]:
        moved += size * (used * 2 * h * i + experts * 2 * h * i + 2 * rows * h + live * i)
        moved += {"rows": 2 * size, "rows8": 2 * 33 / 32, "none": 0}[c["keep"]] * live * 2 * i
        moved += rows * h * 33 / 32 if c["keep"] == "rows8" else 0
    return dict(bytes=moved, flops=2 * live * 2 * h * i * ((4 if c["keep"] == "none" else 3) if c["backward"] else 1))


# ---------------------------------------------------------------- the definition in 64 bits

def _rows8_exact(v):
    """By the power of two itself: 2^e, e = ceil(log2(largest / 448)), and E4M3's steps of an eighth of a power of two,
    2^-9 at the least."""
    b = v.unflatten(-1, (-1, 32))
    e = torch.ceil(torch.log2(b.abs().amax(-1, keepdim=True) / 448)).clamp(min=-126)
    q = b / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step * torch.exp2(e)).flatten(-2)


def _differentiated(x, w, call, dy):
    """call(x, w) and the gradients of its products with dy, by torch's own differentiation."""
    x, w = x.requires_grad_(), w.requires_grad_()
    y = call(x, w)
    return y.detach(), *torch.autograd.grad(y, (x, w), dy)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f = lambda v: None if v is None else v.double()  # noqa: E731
    x = f(s["x"])
    if c["op"] == "rows8":
        return dict(values=_rows8_exact(x))
    if c["op"] == "norm":
        total = s["x"] if s["residual"] is None else (x + f(s["residual"])).to(s["x"].dtype)
        norm = lambda v, w: v / (v.square().mean(1, keepdim=True) + EPS).sqrt() * w  # noqa: E731
        out = dict(sum=f(total))
        if not c["backward"]:
            y = norm(f(total), f(s["weight"]))
            return dict(out, y=_rows8_exact(y.float().double()) if c["eight"] else y)
        out["y"], dx, out["dweight"] = _differentiated(f(total), f(s["weight"]), norm, f(s["dy"]))
        return dict(out, dx=dx + f(s["dsum"]))
    experts = max(c["experts"], 1)
    w = f(s["w"]).view(experts, *s["w"].shape[-2:])
    ids = s["ids"].reshape(-1) if c["experts"] else torch.zeros(c["rows"], dtype=torch.int32, device=DEVICE)
    # the slots of each expert, and where their rows lie
    slots = [torch.nonzero(ids == e).flatten() for e in range(experts)]
    begin, total = 0, ids.numel()
    act = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}
    if c["op"] == "linear":
        out = dict(y=torch.zeros(total, c["n"], dtype=torch.float64, device=DEVICE))
        if c["backward"]:
            out |= dict(dx=torch.zeros_like(x), dw=torch.zeros_like(w))
            if c["bias"]:
                out["dbias"] = torch.zeros_like(w[..., 0])
        for e, of in enumerate(slots):
            at = slice(begin, begin + of.numel())
            begin = at.stop
            b = torch.zeros_like(w[e, :, 0]) if s["bias"] is None else f(s["bias"]).view(experts, -1)[e]
            b.requires_grad_()
            call = lambda v, m: act[c["activation"]](v @ m.T + b)  # noqa: E731, B023
            if c["backward"]:
                xe, we = x[at].requires_grad_(), w[e].detach().requires_grad_()
                y = call(xe, we)
                out["dx"][at], out["dw"][e], db = torch.autograd.grad(y, (xe, we, b), f(s["dy"])[at])
                if c["bias"]:
                    out["dbias"][e] = db
            else:
                y = call(x[at], w[e])
            out["y"][at] = y.detach() if s["residual"] is None else y.detach() + f(s["residual"])[at]
    else:
        i = c["inner"]
        out = dict(h=torch.zeros(total, i, dtype=torch.float64, device=DEVICE))
        if c["backward"]:
            out |= dict(dx=torch.zeros_like(x), dw=torch.zeros_like(w))
        for e, of in enumerate(slots):
            at = slice(begin, begin + of.numel())
            begin = at.stop
            token = of // c["topk"]
            z = x[token] @ w[e].T
            out["h"][at] = torch.nn.functional.silu(z[:, :i]) * z[:, i:]
            if c["backward"]:
                kept = _rows8_exact(x[token]) if c["keep"] == "rows8" else x[token]
                z = (_rows8_exact(z.float().double()) if c["keep"] == "rows8" else z).requires_grad_()
                h = torch.nn.functional.silu(z[:, :i]) * z[:, i:]
                dz = torch.autograd.grad(h, z, f(s["dh"])[at])[0]
                out["dx"].index_add_(0, token, dz @ w[e])
                out["dw"][e] = dz.T @ kept
    if "dw" in out and not c["experts"]:
        out |= {name: out[name][0] for name in ("dw", "dbias") if name in out}
    return out
