"""A layer of experts around the NVFP4 grouped GEMM, on PyTorch tensors.

Each function checks its tensors, allocates the outputs that are not given and
enqueues one operator of ``include/nvfp4_moe.h`` (which states the mathematics,
the limits and what happens at the edges) on ``stream`` (a torch stream or a
handle), by default torch's current stream. Nothing is synchronised and nothing
read from the device, so calls can be captured in a graph. Outputs and
workspaces are allocated on that stream; its waiting for the inputs, and keeping
alive what another stream uses (``Tensor.record_stream``), are the caller's
part, as everywhere in torch.

Rows may lie apart (a slice of wider rows), but their elements have to be adjacent
and rows may not overlap: expanded tensors, such as the gradient of a sum, are
refused and need ``contiguous()`` first.

``FeedForward`` runs them together: route -> plan -> quantise -> grouped GEMM ->
gated activation -> grouped GEMM -> combine, or, for a few tokens, the experts'
products with activations as they are.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _moe_binding as c
from ._binding import nvfp4_device_group_tiles, nvfp4_grouped_gemm_device, nvfp4_sf_bytes

_TYPES = {torch.float32: c.NVFP4_MOE_F32, torch.float16: c.NVFP4_MOE_F16, torch.bfloat16: c.NVFP4_MOE_BF16}
_SCORES = {"softmax": c.NVFP4_MOE_SOFTMAX, "sigmoid": c.NVFP4_MOE_SIGMOID}


def _type(t: torch.Tensor, what: str) -> int:
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{what} must be fp32, fp16 or bf16, not {t.dtype}") from None


def _gpu(t: torch.Tensor, what: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a GPU")
    return t.device


def _like(t, what, shape, dtype, device):
    """A contiguous tensor of that shape and type, on that device."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, not "
                         f"{t.dtype} {tuple(t.shape)} {tuple(t.stride())} on {t.device}")
    return t


def _out(t, what, shape, dtype, device):
    if t is not None:
        return _like(t, what, shape, dtype, device)
    if len(shape) == 2:  # strides given: two thirds of the host's time (1.0 and 1.5 us)
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _rows(t: torch.Tensor, what: str, width=None) -> int:
    """Row stride of a 2-d tensor with adjacent columns."""
    if t.dim() != 2 or (width is not None and t.shape[1] != width):
        raise ValueError(f"{what} must have shape [rows, {'columns' if width is None else width}], not {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have adjacent columns (strides {tuple(t.stride())})")
    # a single row's stride says nothing, and broadcast rows are all the same
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{what} must have rows that do not overlap (strides {tuple(t.stride())})")
    return max(t.stride(0), t.shape[1]) if t.shape[0] > 1 else t.shape[1]


def _at(t) -> int:
    return 0 if t is None else t.data_ptr()


try:
    # the handle alone, in a tenth of the time of a Stream object
    _current_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
except AttributeError:
    _current_device = torch.cuda.current_device

    def _current_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _enqueue(call, device, *args):
    """``call(*args, current stream)`` with the tensors' device current."""
    if device.index == _current_device():
        call(*args, _current_stream(device.index))
    else:
        with torch.cuda.device(device):
            call(*args, _current_stream(device.index))


def _on_stream(fn):
    """``fn`` with its ``stream``, where one is given, current: for its calls, and for what it allocates, whose memory
    would else come from, and go back to, work of another stream that may still be under way."""
    @functools.wraps(fn)
    def call(*args, stream=None, **named):
        if stream is None:
            return fn(*args, **named)
        if not isinstance(stream, torch.cuda.Stream):
            device = next(t.device for t in (*args, *named.values()) if hasattr(t, "device"))
            stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
        with torch.cuda.stream(stream):
            return fn(*args, **named)
    return call


@functools.lru_cache(maxsize=256)
def _choice(score, topk, groups, topk_groups, group_best, renormalize, scale):
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', not {score!r}")
    return ctypes.byref(c.nvfp4_moe_choice(_SCORES[score], topk, groups, groups if topk_groups is None else topk_groups,
                                           group_best, bool(renormalize), scale))


# ---- routing ------------------------------------------------------------------

@_on_stream
def route(logits, topk, *, score="softmax", bias=None, groups=1, topk_groups=None, group_best=1, renormalize=True,
          scale=1.0, ids=None, weights=None, stream=None):
    """Expert ids (int32) and weights (fp32) [tokens, topk] of ``logits`` [tokens, experts].

    ``score`` of all logits, plus ``bias`` [experts] (fp32) for the choice alone; with ``groups``, only the
    ``topk_groups`` groups of experts whose best ``group_best`` (1 or 2) choice values sum highest stay eligible;
    ``renormalize``: divide by the sum of the chosen; times ``scale``. -inf masks an expert; slots that no expert is
    left for get id -1 and weight 0."""
    device = _gpu(logits, "logits")
    stride = _rows(logits, "logits")
    tokens, experts = logits.shape
    if bias is not None:
        _like(bias, "bias", (experts,), torch.float32, device)
    ids = _out(ids, "ids", (tokens, topk), torch.int32, device)
    weights = _out(weights, "weights", (tokens, topk), torch.float32, device)
    _enqueue(c.nvfp4_moe_route, device, logits.data_ptr(), _type(logits, "logits"), tokens, experts, stride,
             _at(bias), _choice(score, topk, groups, topk_groups, group_best, renormalize, float(scale)), ids.data_ptr(),
             weights.data_ptr())
    return ids, weights


@_on_stream
def route_backward(logits, ids, dweights, *, score="softmax", renormalize=True, scale=1.0, dlogits=None, stream=None):
    """Gradient of ``route``'s weights with respect to the logits (their type, every element written), the chosen
    ``ids`` held fixed."""
    device = _gpu(logits, "logits")
    stride = _rows(logits, "logits")
    tokens, experts = logits.shape
    topk = ids.shape[-1]
    _like(ids, "ids", (tokens, topk), torch.int32, device)
    _like(dweights, "dweights", (tokens, topk), torch.float32, device)
    if dlogits is None:
        dlogits = torch.empty((tokens, experts), dtype=logits.dtype, device=device)
    elif dlogits.dtype != logits.dtype or dlogits.device != device or dlogits.shape != logits.shape:
        raise ValueError("dlogits must have the logits' shape, type and device")
    _enqueue(c.nvfp4_moe_route_backward, device, logits.data_ptr(), _type(logits, "logits"), tokens, experts,
             stride, _choice(score, topk, 1, 1, 1, renormalize, float(scale)), ids.data_ptr(), dweights.data_ptr(),
             dlogits.data_ptr(), _rows(dlogits, "dlogits"))
    return dlogits


# ---- the plan --------------------------------------------------------------------

def _group_fits(m, n, k):
    """Whether the grouped GEMM takes a group of that size (else it leaves its rows as they are)."""
    return m < 1 << 31 and nvfp4_device_group_tiles((m, n, k, 1), (4096,) * 5) >= 0


@functools.lru_cache(maxsize=1024)
def _most_rows(n, k):
    """The most rows that a group of n columns and k elements can have: 2^31 bytes of codes, as a rule."""
    low, high = 0, 1 << 30
    if not _group_fits(1, n, k):
        raise ValueError(f"the grouped GEMM does not take weights of {n} x {k}")
    while low < high:
        mid = (low + high + 1) // 2
        low, high = (mid, high) if _group_fits(mid, n, k) else (low, mid - 1)
    return low


class Product:
    """A grouped product over rows sorted by expert, ``c[row] = a[row] . b[expert]``, and the group tables that
    ``plan`` fills for ``nvfp4_grouped_gemm_device``."""

    def __init__(self, a, sfa, b, sfb, out):
        device = _gpu(b, "b")
        experts, n, half = b.shape
        self.n, self.k, self.experts, self.device = n, 2 * half, experts, device
        rows = a.shape[0]
        self.a, self.out = _like(a, "a", (rows, half), torch.uint8, device), _like(out, "out", (rows, n), torch.float16, device)
        self.b, self.sfb = _operand(b, sfb)
        self.sfa = _like(sfa, "sfa", (max(sfa.shape[0], c.nvfp4_moe_sf_bytes(rows, experts, self.k)),), torch.uint8, device)
        # sizes int32 [experts][4], then the two address tables, each from a multiple of 16 bytes on
        self._tables = torch.empty(experts * 56 + 32, dtype=torch.uint8, device=device)
        sizes = self._tables.data_ptr()
        abc = sizes + 16 * experts
        self.tables = (sizes, abc, (abc + 24 * experts + 15) // 16 * 16)
        self.planned = False

    def entry(self):
        return c.nvfp4_moe_product(self.n, self.k, self.a.data_ptr(), self.b.data_ptr(), self.out.data_ptr(),
                                   self.sfa.data_ptr(), self.sfb.data_ptr(), *self.tables)

    @_on_stream
    def run(self, tile_config=-1, status=None, *, stream=None):
        """Enqueue the product, after a ``plan`` that this one was given to.

        An expert with more rows than the grouped GEMM takes in a group (2^31 bytes of codes) has no result. Where there
        are so many rows in all, ``status`` (int32 [1]) says how many such experts there are, their rows left as they
        were; without it their rows are NaN."""
        if not self.planned:
            raise ValueError("no plan has filled this product's tables")
        if status is None and self.a.shape[0] > _most_rows(self.n, self.k):
            self.out.fill_(float("nan"))
        _enqueue(nvfp4_grouped_gemm_device, self.device, *self.tables, self.experts, tile_config,
                 _at(status))
        return self.out


class Plan:
    """Where the rows of every slot lie: ``offsets`` and ``atoms`` [experts + 1], ``slot_rows`` and ``ids`` [tokens, topk]
    and ``row_slots`` [tokens * topk] (all int32). ``ids`` are the plan's own (-1 where a slot has no expert): those that it
    was made from may be rewritten once it is."""

    def __init__(self, tokens, topk, experts, device):
        self.tokens, self.topk, self.experts, self.device = tokens, topk, experts, device
        #: the most rows there can be (those that are there: ``offsets[experts]``, on the device)
        self.rows = self.tokens * self.topk
        self._store = torch.empty(2 * (experts + 1) + 3 * self.rows, dtype=torch.int32, device=device)
        at, rows = self._store.data_ptr(), 4 * self.rows
        slots = at + 8 * (experts + 1)
        #: addresses of offsets, atoms, slot_rows, row_slots and ids
        self.addresses = (at, at + 4 * (experts + 1), slots, slots + rows, slots + 2 * rows)

    def __getattr__(self, name):
        # the views are made when they are first asked for
        if name == "ids":
            self.ids = self._store.as_strided((self.tokens, self.topk), (self.topk, 1), 2 * (self.experts + 1 + self.rows))
        elif name in ("offsets", "atoms", "slot_rows", "row_slots"):
            n = self.experts + 1
            # (a third faster than split)
            parts = self._store.split_with_sizes((n, n, self.rows, self.rows, self.rows))
            self.offsets, self.atoms, self.row_slots = parts[0], parts[1], parts[3]
            self.slot_rows = parts[2].view(self.tokens, self.topk)
        else:
            raise AttributeError(name)
        return self.__dict__[name]


@_on_stream
def plan(ids, experts, products=(), *, stream=None) -> Plan:
    """Sort the slots of ``ids`` [tokens, topk] (int32) by expert, and fill the tables of ``products``."""
    device = _gpu(ids, "ids")
    if ids.dim() != 2:
        raise ValueError(f"ids must have shape [tokens, topk], not {tuple(ids.shape)}")
    _like(ids, "ids", ids.shape, torch.int32, device)
    p = Plan(*ids.shape, experts, device)
    entries = (c.nvfp4_moe_product * len(products))(*[q.entry() for q in products]) if products else None
    for q in products:
        if q.experts != experts or q.a.shape[0] < p.rows or q.device != device:
            raise ValueError("a product must have the plan's experts and device, and room for its rows")
    need = c.nvfp4_moe_plan_workspace_bytes(p.tokens, p.topk, experts)
    workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _enqueue(c.nvfp4_moe_plan_ex, device, ids.data_ptr(), p.tokens, p.topk, experts, *p.addresses, entries,
             len(products), _at(workspace), need)
    for q in products:
        q.planned = True
    return p


# ---- quantisation ------------------------------------------------------------------

def _operand(b, sfb):
    """Stacked weights [experts, n, k/2] with their scales [experts, nvfp4_sf_bytes(n, k)]."""
    if b.dim() != 3:
        raise ValueError(f"b must have shape [experts, n, k/2], not {tuple(b.shape)}")
    device = _gpu(b, "b")
    _like(b, "b", b.shape, torch.uint8, device)
    _like(sfb, "sfb", (b.shape[0], nvfp4_sf_bytes(b.shape[1], 2 * b.shape[2])), torch.uint8, device)
    return b, sfb


@_on_stream
def quantize(x, *, plan=None, scale=1.0, a=None, sfa=None, stream=None):
    """NVFP4 codes and tiled scales of ``x * scale``.

    Without a plan: x [m, k] or [l, m, k] -> a [..., k/2] (uint8) and sfa (uint8, ``nvfp4_sf_bytes(m, k, l)``). With
    one: x [tokens, k] -> a [tokens * topk, k/2], each token's row at the rows of its slots, and sfa of the rows
    sorted by expert."""
    device = _gpu(x, "x")
    kind = _type(x, "x")
    k = x.shape[-1]
    if k % 32:
        raise ValueError(f"rows must have a multiple of 32 elements, not {k}")
    if plan is not None:
        stride = _rows(x, "x")
        if x.shape[0] != plan.tokens or plan.device != device:
            raise ValueError(f"x must have the plan's {plan.tokens} tokens, on its device")
        a = _out(a, "a", (plan.rows, k // 2), torch.uint8, device)
        sfa = _out(sfa, "sfa", (c.nvfp4_moe_sf_bytes(plan.rows, plan.experts, k),), torch.uint8, device)
        need = c.nvfp4_moe_dispatch_workspace_bytes(plan.tokens, plan.topk, k)
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        offsets, atoms, slot_rows, row_slots, ids = plan.addresses
        _enqueue(c.nvfp4_moe_dispatch, device, x.data_ptr(), kind, plan.tokens, plan.topk, k, stride, scale,
                 ids, slot_rows, row_slots, offsets, atoms, plan.experts, a.data_ptr(), sfa.data_ptr(),
                 _at(workspace), need)
        return a, sfa
    if x.dim() not in (2, 3):
        raise ValueError(f"x must have shape [m, k] or [l, m, k], not {tuple(x.shape)}")
    l, m = (x.shape[0], x.shape[1]) if x.dim() == 3 else (1, x.shape[0])
    stride = _rows(x[0] if x.dim() == 3 and l else x.view(-1, k) if x.dim() == 3 else x, "x")
    batch = x.stride(0) if x.dim() == 3 else 0
    a = _out(a, "a", (*x.shape[:-1], k // 2), torch.uint8, device)
    sfa = _out(sfa, "sfa", (nvfp4_sf_bytes(m, k, l),), torch.uint8, device)
    if l:
        _enqueue(c.nvfp4_moe_quantize, device, x.data_ptr(), kind, l, m, k, batch, stride, scale,
                 a.data_ptr(), sfa.data_ptr())
    return a, sfa


@_on_stream
def swiglu_quantize(x, *, plan=None, alpha=None, scale=1.0, a=None, sfa=None, stream=None):
    """NVFP4 codes and scales of ``silu(g * alpha) * (u * alpha) * scale``, g and u the halves of each row of ``x``
    [rows, 2k]: rows of one group, or with a plan rows sorted by expert, ``alpha`` [experts] (fp32) by expert."""
    device = _gpu(x, "x")
    stride = _rows(x, "x")
    rows, k = x.shape[0], x.shape[1] // 2
    if x.shape[1] % 64:
        raise ValueError(f"the halves of a row must have a multiple of 32 elements (row of {x.shape[1]})")
    experts = 1 if plan is None else plan.experts
    if plan is not None and (rows != plan.rows or plan.device != device):
        raise ValueError(f"x must have the plan's {plan.rows} rows, on its device")
    if alpha is not None:
        _like(alpha, "alpha", (experts,), torch.float32, device)
    a = _out(a, "a", (rows, k // 2), torch.uint8, device)
    sfa = _out(sfa, "sfa", (nvfp4_sf_bytes(rows, k) if plan is None else c.nvfp4_moe_sf_bytes(rows, experts, k),),
               torch.uint8, device)
    _enqueue(c.nvfp4_moe_swiglu, device, x.data_ptr(), _type(x, "x"), rows, k, stride, _at(alpha), scale,
             *((0, 0) if plan is None else plan.addresses[:2]), experts, a.data_ptr(), sfa.data_ptr())
    return a, sfa


@_on_stream
def dequantize(a, sfa, *, plan=None, dtype=torch.float16, out=None, stream=None):
    """The values that NVFP4 rows stand for: a [m, k/2] or [l, m, k/2] -> [..., k]. With a plan, of rows sorted by
    expert; rows that no slot has are not written."""
    device = _gpu(a, "a")
    if a.dim() not in (2, 3) or (plan is not None and a.dim() != 2):
        raise ValueError(f"a must have shape [m, k/2] (or, without a plan, [l, m, k/2]), not {tuple(a.shape)}")
    _like(a, "a", a.shape, torch.uint8, device)
    l, m, k = a.shape[0] if a.dim() == 3 else 1, a.shape[-2], 2 * a.shape[-1]
    if plan is not None and (m != plan.rows or plan.device != device):
        raise ValueError(f"a must have the plan's {plan.rows} rows, on its device")
    need = nvfp4_sf_bytes(m, k, l) if plan is None else c.nvfp4_moe_sf_bytes(m, plan.experts, k)
    _like(sfa, "sfa", (need,), torch.uint8, device)
    if out is not None:
        dtype = out.dtype
    out = _out(out, "out", (*a.shape[:-1], k), dtype, device)
    if l:
        _enqueue(c.nvfp4_moe_dequantize, device, a.data_ptr(), sfa.data_ptr(), l, m, k,
                 *((0, 0) if plan is None else plan.addresses[:2]), 1 if plan is None else plan.experts,
                 out.data_ptr(), _type(out, "out"), k)
    return out


# ---- the combine ----------------------------------------------------------------------

def _slots(weights, rows, alpha, ids, experts, slots_of, device):
    """Checked (tokens, topk, rows, ids, number of experts or 0) of a combine's slots; ``rows`` a Plan, a tensor or
    None."""
    if isinstance(rows, Plan):
        ids, rows = rows.ids, rows.slot_rows
    given = weights if weights is not None else rows
    if given is None or given.dim() != 2:
        raise ValueError("weights or rows must have shape [tokens, topk]")
    shape = given.shape
    if weights is not None:
        _like(weights, "weights", shape, torch.float32, device)
    if rows is not None:
        _like(rows, "rows", shape, torch.int32, device)
    elif slots_of.shape[0] != shape[0] * shape[1]:
        raise ValueError(f"without rows, c must have a row for each of the {shape[0] * shape[1]} slots")
    if ids is not None:
        _like(ids, "ids", shape, torch.int32, device)
    if alpha is not None:
        if ids is None:
            raise ValueError("alpha needs ids")
        _like(alpha, "alpha", (alpha.shape[0],), torch.float32, device)
        if experts is not None and experts != alpha.shape[0]:
            raise ValueError(f"alpha has {alpha.shape[0]} experts, not {experts}")
        experts = alpha.shape[0]
    elif experts is not None and (ids is None or experts < 1):
        raise ValueError("experts needs ids, and at least one expert")
    return shape[0], shape[1], rows, ids, experts or 0


@_on_stream
def combine(x, weights, rows=None, *, alpha=None, ids=None, experts=None, residual=None, dtype=None, out=None, stream=None):
    """``out[t] = residual[t] + sum_j weights[t, j] * alpha[ids[t, j]] * x[rows[t, j]]``, summed in fp32 in slot order.

    ``x`` [rows, n]: the experts' rows; ``rows``: a Plan, int32 [tokens, topk] (-1: no row), or None where the slots'
    rows follow each other; ``weights`` fp32 [tokens, topk] or None for 1. Slots whose id is below 0, or not below the
    number of ``experts`` (that of ``alpha`` where there is one, else any), add nothing, whatever their weight holds.
    ``dtype`` of the result: that of ``out`` or ``residual``, else x's."""
    device = _gpu(x, "x")
    stride = _rows(x, "x")
    n = x.shape[1]
    tokens, topk, rows, ids, experts = _slots(weights, rows, alpha, ids, experts, x, device)
    if dtype is None:
        dtype = out.dtype if out is not None else residual.dtype if residual is not None else x.dtype
    out = _out(out, "out", (tokens, n), dtype, device)
    if residual is not None:
        _like(residual, "residual", (tokens, n), dtype, device)
    _enqueue(c.nvfp4_moe_combine, device, x.data_ptr(), _type(x, "x"), stride, x.shape[0], tokens, topk, n,
             _at(rows), _at(weights), _at(alpha), _at(ids), experts, _at(residual),
             out.data_ptr(), _type(out, "out"), n)
    return out


@_on_stream
def combine_backward(dy, x, weights, rows=None, *, alpha=None, ids=None, experts=None, dc=None, stream=None):
    """(d x, d weights) of ``combine``; rows of d x whose slots have no expert are 0, and so are rows that no slot has.
    Those are not written to a ``dc`` that is given: a program that keeps one cleared saves the clearing."""
    device = _gpu(x, "x")
    stride = _rows(x, "x")
    tokens, topk, rows, ids, experts = _slots(weights, rows, alpha, ids, experts, x, device)
    dy_stride = _rows(dy, "dy", x.shape[1])
    if dy.shape[0] != tokens or dy.device != device:
        raise ValueError(f"dy must have {tokens} rows, on {device}")
    if dc is None:
        dc = torch.empty_strided(x.shape, (stride, 1), dtype=x.dtype, device=device)
        if rows is not None or x.shape[0] > tokens * topk:  # else every row is a slot's
            dc.zero_()
    elif dc.shape != x.shape or dc.dtype != x.dtype or dc.device != device or _rows(dc, "dc") != stride:
        raise ValueError("dc must have x's shape, strides, type and device")
    dweights = torch.empty((tokens, topk), dtype=torch.float32, device=device)
    _enqueue(c.nvfp4_moe_combine_backward, device, dy.data_ptr(), _type(dy, "dy"), dy_stride, x.data_ptr(),
             _type(x, "x"), stride, x.shape[0], tokens, topk, x.shape[1], _at(rows), _at(weights), _at(alpha), _at(ids),
             experts, dc.data_ptr(), dweights.data_ptr())
    return dc, dweights


# ---- a few tokens ------------------------------------------------------------------------

@_on_stream
def few_tokens(x, ids, b, sfb, *, alpha=None, swiglu=False, dtype=None, out=None, stream=None):
    """The experts' products of a few tokens: out [tokens, topk, n] = alpha[id] * b[id] . x, and with ``swiglu``
    silu of the first half times the second, [tokens, topk, n/2].

    ``x`` (fp16 or bf16) [tokens, k], or [tokens, topk, k] with a row for each slot; ``ids`` int32 [tokens, topk];
    ``b``, ``sfb``: stacked NVFP4 weights. Slots without an expert give zeros."""
    device = _gpu(x, "x")
    if ids.dim() != 2:
        raise ValueError(f"ids must have shape [tokens, topk], not {tuple(ids.shape)}")
    tokens, topk = ids.shape
    _like(ids, "ids", ids.shape, torch.int32, device)
    b, sfb = _operand(b, sfb)
    experts, n, k = b.shape[0], b.shape[1], 2 * b.shape[2]
    if x.dim() == 3:
        _like(x, "x", (tokens, topk, k), x.dtype, device)
        stride = k
    else:
        stride = _rows(x, "x", k)
        if x.shape[0] != tokens:
            raise ValueError(f"x must have {tokens} rows, not {x.shape[0]}")
    if b.device != device:
        raise ValueError(f"b must be on {device}")
    if alpha is not None:
        _like(alpha, "alpha", (experts,), torch.float32, device)
    if dtype is None:
        dtype = x.dtype if out is None else out.dtype
    out = _out(out, "out", (tokens, topk, n // 2 if swiglu else n), dtype, device)
    _enqueue(c.nvfp4_moe_few_tokens, device, x.data_ptr(), _type(x, "x"), stride, x.dim() == 3,
             ids.data_ptr(), tokens, topk, experts, n, k, b.data_ptr(), sfb.data_ptr(), _at(alpha), bool(swiglu),
             out.data_ptr(), _type(out, "out"))
    return out


# ---- the layer ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def _layer_room(tokens, topk, experts, hidden, inner):
    """Where the parts of a grouped layer's workspace begin, its bytes, and those of the plan's and dispatch's own."""
    rows = tokens * topk
    plan_bytes = c.nvfp4_moe_plan_workspace_bytes(tokens, topk, experts)
    dispatch_bytes = c.nvfp4_moe_dispatch_workspace_bytes(tokens, topk, hidden)
    places, end = [], 0
    for size in (4 * (experts + 1), 4 * (experts + 1), 4 * rows, 4 * rows, plan_bytes, dispatch_bytes,
                 rows * hidden // 2, c.nvfp4_moe_sf_bytes(rows, experts, hidden), rows * inner * 4,
                 rows * inner // 2, c.nvfp4_moe_sf_bytes(rows, experts, inner), rows * hidden * 2,
                 *(16 * experts, 24 * experts, 16 * experts) * 2):
        places.append(end)
        end += -(-size // 256) * 256
    return places, end, plan_bytes, dispatch_bytes


class FeedForward:
    """The experts' gated feed-forward with NVFP4 weights:
    ``y[t] = sum_j w[t, j] * down[e] . (silu(gate[e] . x[t]) * (up[e] . x[t]))``, e = ids[t, j].

    ``b1``, ``sfb1``: gate rows, then up rows, [experts, 2 * inner, hidden / 2]; ``b2``, ``sfb2``: [experts, hidden,
    inner / 2]; ``alpha1``, ``alpha2``: factors on each expert's products (fp32 [experts]), as weights that were
    quantised under a factor of their own need them.

    ``scale1``, ``scale2`` are factors on the rows and on the activations before ``grouped`` quantises them; it takes
    them out again with the products' factors (``alpha1 / scale1`` and ``alpha2 / scale2`` are formed here, once, where
    a scale is not 1; powers of two lose nothing). They keep two things in range, which differ from weights to weights
    and which nothing checks: the grouped GEMM writes its products, without ``alpha``, in fp16, so ``scale * y / alpha``
    has to stay below 65504 (beyond, the layer gives infinities and NaN); and what is quantised keeps its 4 bits from
    about 0.1 (a block's largest element; below 0.006 it is 0) to 2688 (beyond, it is 2688). ``few`` quantises neither
    and needs no scale. Weights whose block scales go up to 448 have an alpha of about their largest entry / 2688: with
    entries up to 0.1, a scale of 1 holds for y up to 2.4, one of 1/16 up to 39."""

    #: Up to this many slots an expert the products of few tokens are faster than the grouped ones (8 experts of
    #: 7168x2048, 2 and 4 slots an expert: 70 and 88 us against 78 both times; 64 of 4096x1024: 104 and 139 against 127
    #: and 131).
    FEW_ROWS = 3

    def __init__(self, b1, sfb1, b2, sfb2, *, alpha1=None, alpha2=None, scale1=1.0, scale2=1.0):
        (self.b1, self.sfb1), (self.b2, self.sfb2) = _operand(b1, sfb1), _operand(b2, sfb2)
        self.experts, self.hidden, self.inner = b1.shape[0], 2 * b1.shape[2], 2 * b2.shape[2]
        if tuple(b1.shape[:2]) != (b2.shape[0], 2 * self.inner) or b2.shape[1] != self.hidden or b1.device != b2.device:
            raise ValueError(f"b1 {tuple(b1.shape)} and b2 {tuple(b2.shape)} do not fit together")
        for name, alpha in (("alpha1", alpha1), ("alpha2", alpha2)):
            if alpha is not None:
                _like(alpha, name, (self.experts,), torch.float32, b1.device)
        for name, scale in (("scale1", scale1), ("scale2", scale2)):
            if not 2.0 ** -126 <= scale <= 2.0 ** 126:
                raise ValueError(f"{name} must be a positive number within fp32's range, not {scale}")
        self.alpha1, self.alpha2, self.scale1, self.scale2 = alpha1, alpha2, float(scale1), float(scale2)
        # the grouped products' own factors
        self._gain1, self._gain2 = self._gain(alpha1, scale1), self._gain(alpha2, scale2)
        if scale1 != 1 or scale2 != 1:
            torch.cuda.current_stream(b1.device).synchronize()  # calls on any stream find them made
        self.units = torch.cuda.get_device_properties(b1.device).multi_processor_count

    def _gain(self, alpha, scale):
        """alpha / scale, in fp32 (None for 1)."""
        if scale == 1:
            return alpha
        one = torch.ones(self.experts, dtype=torch.float32, device=self.b1.device) if alpha is None else alpha
        return one / torch.full_like(one, scale)

    def __call__(self, x, ids, weights, *, residual=None, stream=None):
        """y [tokens, hidden] of ``x``'s type, by the products that suit the number of tokens: up to ``FEW_ROWS`` slots an
        expert ``few``, beyond ``grouped``, whose rows and activations are in 4 bits. The two differ by that rounding; a
        program that wants one of them whatever the batch calls it by name."""
        slots = ids.numel()
        few = slots <= min(self.FEW_ROWS * self.experts, c.NVFP4_MOE_MAX_FEW_SLOTS) and x.dtype != torch.float32
        run = self.few if few else self.grouped
        return run(x, ids, weights, residual=residual, stream=stream)

    @_on_stream
    def few(self, x, ids, weights, *, residual=None, stream=None):
        """By the products of few tokens, with ``x`` (fp16 or bf16) as it is."""
        h = few_tokens(x, ids, self.b1, self.sfb1, alpha=self.alpha1, swiglu=True)
        y = few_tokens(h, ids, self.b2, self.sfb2, alpha=self.alpha2)
        return combine(y.view(-1, self.hidden), weights, ids=ids, experts=self.experts, residual=residual, dtype=x.dtype)

    @_on_stream
    def grouped(self, x, ids, weights, *, residual=None, stream=None):
        """By the grouped GEMM, on rows and activations quantised to NVFP4. The operators are enqueued with addresses
        in one workspace: a small layer takes the host longer than the GPU (64 tokens on 16 experts of 2048x1024, with
        their routing: 87 us with tensors made and checked operator by operator, 48 like this). More tokens than a group of
        the grouped GEMM is sure to hold (2^31 bytes of codes: 599186 rows of 7168) are taken in parts."""
        device, hidden = _gpu(x, "x"), self.hidden
        layout = _type(x, "x"), _rows(x, "x", hidden)
        if device != self.b1.device:
            raise ValueError(f"x must be on {self.b1.device}")
        tokens, topk = x.shape[0], ids.shape[-1]
        _like(ids, "ids", (tokens, topk), torch.int32, device)
        _like(weights, "weights", (tokens, topk), torch.float32, device)
        if residual is not None:
            _like(residual, "residual", (tokens, hidden), x.dtype, device)
        out = torch.empty((tokens, hidden), dtype=x.dtype, device=device)
        most = self._most_tokens(topk)
        if tokens <= most:
            self._grouped(x, layout, ids, weights, residual, out)
        else:
            for part in (slice(i, i + most) for i in range(0, tokens, most)):
                self._grouped(x[part], layout, ids[part], weights[part], None if residual is None else residual[part],
                              out[part])
        return out

    def _most_tokens(self, topk):
        """The most tokens whose rows fit the grouped GEMM's groups, were they all one expert's."""
        return max(1, min(_most_rows(2 * self.inner, self.hidden), _most_rows(self.hidden, self.inner)) // max(topk, 1))

    def _grouped(self, x, layout, ids, weights, residual, out):
        device, e, hidden, inner = x.device, self.experts, self.hidden, self.inner
        (kind, stride), (tokens, topk) = layout, ids.shape
        rows = tokens * topk
        places, size, plan_bytes, dispatch_bytes = _layer_room(tokens, topk, e, hidden, inner)
        room = torch.empty(size, dtype=torch.uint8, device=device)
        base, ids_at = room.data_ptr(), ids.data_ptr()
        (offsets, atoms, slot_rows, row_slots, plan_room, dispatch_room, a1, sf1, c1, a2, sf2, c2, sizes1, abc1, scales1,
         sizes2, abc2, scales2) = [base + p for p in places]
        products = (c.nvfp4_moe_product * 2)(
            (2 * inner, hidden, a1, self.b1.data_ptr(), c1, sf1, self.sfb1.data_ptr(), sizes1, abc1, scales1),
            (hidden, inner, a2, self.b2.data_ptr(), c2, sf2, self.sfb2.data_ptr(), sizes2, abc2, scales2))

        def enqueue(stream):
            c.nvfp4_moe_plan(ids_at, tokens, topk, e, offsets, atoms, slot_rows, row_slots, products, 2, plan_room,
                             plan_bytes, stream)
            c.nvfp4_moe_dispatch(x.data_ptr(), kind, tokens, topk, hidden, stride, self.scale1, ids_at, slot_rows, row_slots,
                                 offsets, atoms, e, a1, sf1, dispatch_room, dispatch_bytes, stream)
            nvfp4_grouped_gemm_device(sizes1, abc1, scales1, e, self._tile(rows, 2 * inner), 0, stream)
            c.nvfp4_moe_swiglu(c1, c.NVFP4_MOE_F16, rows, inner, 2 * inner, _at(self._gain1), self.scale2, offsets, atoms, e,
                               a2, sf2, stream)
            nvfp4_grouped_gemm_device(sizes2, abc2, scales2, e, self._tile(rows, hidden), 0, stream)
            c.nvfp4_moe_combine(c2, c.NVFP4_MOE_F16, hidden, rows, tokens, topk, hidden, slot_rows, weights.data_ptr(),
                                _at(self._gain2), ids_at, e, _at(residual), out.data_ptr(), kind, hidden, stream)
        _enqueue(enqueue, device)

    def _tile(self, rows, n):
        """The grouped GEMM's tile configuration for ``rows`` rows spread evenly: the one whose rounds of tiles over the
        compute units take least. A round of mostly empty 128x256 tiles takes 1.5 times one of 256x128 tiles (8 experts
        of 16 rows, 4096x7168: 59 and 39 us, 7168x2048: 24 us and two rounds, 30), one of full 256x256 tiles 1.55 times
        (8 experts of 256 rows: 168 and 147, 68 us and two rounds, 73)."""
        mean = rows / self.experts
        rounds = lambda bm, bn: -(-self.experts * -(-max(int(mean), 1) // bm) * -(-n // bn) // self.units)  # noqa: E731
        if mean <= 64:
            return 1 if 3 * rounds(128, 256) < 2 * rounds(256, 128) else 2
        return 0 if 1.55 * rounds(256, 256) < rounds(256, 128) else 2
