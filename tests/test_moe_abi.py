"""libnvfp4_moe.so on the CPU: it exports what include/nvfp4_moe.h declares, sizes
its buffers, and refuses what the header rules out before any HIP call (no GPU
needed: every call here returns before one). The oracle of the GPU tests is
pinned here as well."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import moe_matmul_amd as mm
import oracle.moe_oracle as MO
import oracle.nvfp4_oracle as O
from moe_matmul_amd import _moe_binding as c
from moe_matmul_amd import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # an address that no refused call reads
INVALID, MISALIGNED, WORKSPACE = mm.NVFP4_ERR_INVALID, mm.NVFP4_ERR_MISALIGNED, mm.NVFP4_ERR_WORKSPACE


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "nvfp4_moe.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(nvfp4_moe_\w+)\s*\(", text)))
    lib = c.load_moe_library()
    assert "nvfp4_moe_route" in names and names == sorted(c._SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", c.MOE_LIB_PATH], capture_output=True, text=True).stdout
    assert sorted(set(re.findall(r"\bT (nvfp4_\w+)", out))) == names
    assert all(hasattr(lib, n) for n in names)


def choice(**kw):
    v = dict(score=0, topk=2, groups=1, topk_groups=1, group_best=1, renormalize=1, scale=1.0) | kw
    return ctypes.byref(c.nvfp4_moe_choice(*[v[n] for n, _ in c.nvfp4_moe_choice._fields_]))


def refused(code, call, *args):
    with pytest.raises(c.Nvfp4MoeError) as e:
        call(*args)
    assert e.value.code == code


@pytest.mark.parametrize("bad", [dict(score=2), dict(score=-1), dict(topk=0), dict(topk=17), dict(topk=9), dict(groups=0),
                                 dict(groups=3), dict(groups=65), dict(groups=2, topk_groups=3), dict(topk_groups=0),
                                 dict(group_best=0), dict(group_best=3), dict(groups=4, topk_groups=1, topk=3)])
def test_route_refuses_choices(bad):
    refused(INVALID, c.nvfp4_moe_route, P, 0, 4, 8, 8, 0, choice(**bad), P, P, 0)
    refused(INVALID, c.nvfp4_moe_route_backward, P, 0, 4, 8, 8, choice(**bad), P, P, P, 8, 0)


def test_route_refuses_arguments():
    route = c.nvfp4_moe_route
    ok = choice()
    for dtype, tokens, experts, stride in ((3, 4, 8, 8), (-1, 4, 8, 8), (0, -1, 8, 8), (0, 4, 0, 8), (0, 4, 513, 513),
                                           (0, 4, 8, 7), (0, 1 << 26, 8, 8)):
        refused(INVALID, route, P, dtype, tokens, experts, stride, 0, ok, P, P, 0)
    refused(INVALID, route, 0, 0, 4, 8, 8, 0, ok, P, P, 0)
    refused(INVALID, route, P, 0, 4, 8, 8, 0, ok, 0, P, 0)
    refused(INVALID, route, P, 0, 4, 8, 8, 0, None, P, P, 0)
    refused(MISALIGNED, route, P + 2, 0, 4, 8, 8, 0, ok, P, P, 0)
    refused(MISALIGNED, route, P + 1, 2, 4, 8, 8, 0, ok, P, P, 0)
    refused(MISALIGNED, route, P, 0, 4, 8, 8, P + 2, ok, P, P, 0)
    refused(MISALIGNED, route, P, 0, 4, 8, 8, 0, ok, P, P + 1, 0)
    route(0, 0, 0, 8, 8, 0, ok, 0, 0, 0)  # no tokens: nothing to do
    refused(INVALID, c.nvfp4_moe_route_backward, P, 0, 4, 8, 8, ok, P, P, P, 7, 0)
    refused(INVALID, c.nvfp4_moe_route_backward, P, 0, 4, 8, 8, ok, P, 0, P, 8, 0)


def test_plan_refuses_and_sizes_its_workspace():
    def call(tokens=4, topk=2, experts=8, ids=P, offsets=P, products=None, count=0, ws=0, ws_bytes=0):
        c.nvfp4_moe_plan(ids, tokens, topk, experts, offsets, P, P, P, products, count, ws, ws_bytes, 0)
    for bad in (dict(tokens=-1), dict(topk=0), dict(topk=17), dict(experts=0), dict(experts=513), dict(tokens=1 << 30),
                dict(ids=0), dict(offsets=0), dict(count=1), dict(count=5), dict(count=-1)):
        refused(INVALID, call, *[{**dict(tokens=4, topk=2, experts=8, ids=P, offsets=P, products=None, count=0), **bad}[n]
                                 for n in ("tokens", "topk", "experts", "ids", "offsets", "products", "count")])
    refused(MISALIGNED, call, 4, 2, 8, P + 1)
    for bad, code in ((dict(n=12), INVALID), (dict(k=48), INVALID), (dict(sizes=0), INVALID), (dict(a=P + 8), MISALIGNED),
                      (dict(sf=P + 4), MISALIGNED)):
        v = dict(n=16, k=64, a=P, b=P, c=P, sfa=P, sfb=P, sizes=P, abc=P, sf=P) | bad
        entry = (c.nvfp4_moe_product * 1)(c.nvfp4_moe_product(*[v[n] for n, _ in c.nvfp4_moe_product._fields_]))
        refused(code, call, 4, 2, 8, P, P, entry, 1)
    assert c.nvfp4_moe_plan_workspace_bytes(4096, 2, 8) == 0
    need = c.nvfp4_moe_plan_workspace_bytes(4097, 2, 8)
    assert need > 0
    refused(WORKSPACE, call, 4097, 2)
    refused(WORKSPACE, call, 4097, 2, 8, P, P, None, 0, 0x20000, need - 1)
    refused(MISALIGNED, call, 4097, 2, 8, P, P, None, 0, 0x20010, need)


def test_scale_bytes_hold_every_spread():
    rng = np.random.default_rng(0)
    for rows in (0, 1, 5, 127, 128, 129, 1000):
        for experts in (1, 3, 64):
            room = c.nvfp4_moe_sf_bytes(rows, experts, 96) // (2 * 512)
            worst = 0
            for _ in range(50):
                m = rng.multinomial(rows, rng.dirichlet(np.full(experts, 0.3)))
                worst = max(worst, int(sum(-(-v // 128) for v in m)))
            # one row in every expert but one
            m = [1] * min(experts, rows)
            if m:
                m[0] += rows - len(m)
            worst = max(worst, sum(-(-v // 128) for v in m))
            assert worst <= room <= worst + 1
    assert c.nvfp4_moe_sf_bytes(-1, 4, 64) == 0 and c.nvfp4_moe_sf_bytes(4, 0, 64) == 0


def test_quantisation_refuses():
    q = c.nvfp4_moe_quantize
    for l, m, k, stride in ((0, 4, 64, 64), (1, -1, 64, 64), (1, 4, 48, 64), (1, 4, -32, 64), (1, 4, 64, 63), (1, 1 << 31, 64, 64),
                            (4, 1 << 29, 64, 64)):
        refused(INVALID, q, P, 0, l, m, k, 0, stride, 1.0, P, P, 0)
    refused(INVALID, q, P, 3, 1, 4, 64, 0, 64, 1.0, P, P, 0)
    refused(INVALID, q, 0, 0, 1, 4, 64, 0, 64, 1.0, P, P, 0)
    refused(INVALID, q, P, 0, 1, 4, 64, 0, 64, 1.0, 0, P, 0)
    refused(MISALIGNED, q, P, 0, 1, 4, 64, 0, 64, 1.0, P + 8, P, 0)
    refused(MISALIGNED, q, P + 2, 0, 1, 4, 64, 0, 64, 1.0, P, P, 0)
    q(P, 0, 1, 0, 64, 0, 64, 1.0, P, P, 0)
    d = c.nvfp4_moe_dispatch
    for tokens, topk, k, experts in ((-1, 2, 64, 8), (4, 0, 64, 8), (4, 17, 64, 8), (4, 2, 48, 8), (4, 2, 64, 0), (4, 2, 64, 513)):
        refused(INVALID, d, P, 0, tokens, topk, k, 64, 1.0, P, P, P, P, P, experts, P, P, 0, 0, 0)
    refused(INVALID, d, P, 0, 4, 2, 64, 64, 1.0, 0, P, P, P, P, 8, P, P, 0, 0, 0)
    refused(INVALID, d, P, 0, 4, 2, 64, 64, 1.0, P, P, P, 0, P, 8, P, P, 0, 0, 0)
    large = 1 << 19  # tokens of two slots of 64 elements
    need = c.nvfp4_moe_dispatch_workspace_bytes(large, 2, 64)
    assert need > 0 and c.nvfp4_moe_dispatch_workspace_bytes(4, 2, 64) == 0
    refused(WORKSPACE, d, P, 0, large, 2, 64, 64, 1.0, P, P, P, P, P, 8, P, P, 0, 0, 0)
    refused(WORKSPACE, d, P, 0, large, 2, 64, 64, 1.0, P, P, P, P, P, 8, P, P, P, need - 1, 0)
    refused(MISALIGNED, d, P, 0, large, 2, 64, 64, 1.0, P, P, P, P, P, 8, P, P, P + 16, need, 0)
    s = c.nvfp4_moe_swiglu
    refused(INVALID, s, P, 1, 4, 64, 127, 0, 1.0, 0, 0, 1, P, P, 0)
    refused(INVALID, s, P, 1, 4, 64, 128, 0, 1.0, P, 0, 4, P, P, 0)
    refused(INVALID, s, P, 1, 4, 64, 128, 0, 1.0, 0, 0, 4, P, P, 0)
    refused(MISALIGNED, s, P, 1, 4, 64, 128, P + 2, 1.0, 0, 0, 1, P, P, 0)
    z = c.nvfp4_moe_dequantize
    refused(INVALID, z, P, P, 2, 4, 64, P, P, 4, P, 1, 64, 0)
    refused(INVALID, z, P, P, 1, 4, 64, 0, 0, 1, P, 1, 63, 0)
    refused(INVALID, z, P, P, 1, 4, 64, 0, 0, 1, 0, 1, 64, 0)


def test_combine_refuses():
    f = c.nvfp4_moe_combine
    for cd, cs, tokens, topk, n, od, os_ in ((3, 64, 4, 2, 64, 1, 64), (1, 63, 4, 2, 64, 1, 64), (1, 64, -1, 2, 64, 1, 64),
                                             (1, 64, 4, 0, 64, 1, 64), (1, 64, 4, 17, 64, 1, 64), (1, 64, 4, 2, 60, 1, 64),
                                             (1, 64, 4, 2, 64, 9, 64), (1, 64, 4, 2, 64, 1, 56)):
        refused(INVALID, f, P, cd, cs, 8, tokens, topk, n, P, P, 0, 0, 0, 0, P, od, os_, 0)
    refused(INVALID, f, P, 1, 64, 8, 4, 2, 64, P, P, P, 0, 4, 0, P, 1, 64, 0)  # alpha without ids
    refused(INVALID, f, P, 1, 64, 8, 4, 2, 64, P, P, P, P, 0, 0, P, 1, 64, 0)  # alpha of no experts
    refused(INVALID, f, P, 1, 64, 7, 4, 2, 64, 0, P, 0, 0, 0, 0, P, 1, 64, 0)  # fewer rows than slots
    refused(INVALID, f, P, 1, 64, -1, 4, 2, 64, P, P, 0, 0, 0, 0, P, 1, 64, 0)
    refused(INVALID, f, 0, 1, 64, 8, 4, 2, 64, P, P, 0, 0, 0, 0, P, 1, 64, 0)
    refused(MISALIGNED, f, P, 1, 64, 8, 4, 2, 64, P, P, 0, 0, 0, 0, P + 1, 1, 64, 0)
    refused(MISALIGNED, f, P, 1, 64, 8, 4, 2, 64, P + 2, P, 0, 0, 0, 0, P, 1, 64, 0)
    b = c.nvfp4_moe_combine_backward
    refused(INVALID, b, P, 1, 64, P, 1, 64, 8, 4, 2, 64, P, P, 0, 0, 0, P, 0, 0)
    refused(INVALID, b, P, 1, 64, P, 1, 64, 8, 4, 2, 64, P, P, 0, 0, 0, 0, P, 0)
    refused(INVALID, b, P, 1, 64, P, 1, 64, 7, 4, 2, 64, 0, P, 0, 0, 0, P, P, 0)
    refused(MISALIGNED, b, P, 1, 64, P, 1, 64, 8, 4, 2, 64, P, P, 0, 0, 0, P + 1, P, 0)


def test_few_tokens_refuses():
    def call(dtype=1, xs=64, tokens=4, topk=2, experts=8, n=64, k=64, swiglu=0, od=1, x=P, b=P, out=P, alpha=0, ids=P):
        c.nvfp4_moe_few_tokens(x, dtype, xs, 0, ids, tokens, topk, experts, n, k, b, P, alpha, swiglu, out, od, 0)
    for bad in (dict(dtype=0), dict(dtype=3), dict(od=3), dict(tokens=-1), dict(tokens=2049), dict(topk=17), dict(topk=0),
                dict(experts=0), dict(experts=513), dict(n=12), dict(n=-8), dict(n=72, swiglu=1), dict(k=48), dict(xs=63),
                dict(x=0), dict(b=0), dict(out=0), dict(ids=0), dict(n=1 << 20, k=1 << 13)):
        with pytest.raises(c.Nvfp4MoeError) as e:
            call(**bad)
        assert e.value.code == INVALID, bad
    for bad in (dict(x=P + 1), dict(b=P + 8), dict(out=P + 1), dict(alpha=P + 2), dict(ids=P + 2)):
        with pytest.raises(c.Nvfp4MoeError) as e:
            call(**bad)
        assert e.value.code == MISALIGNED, bad
    call(tokens=0)


def test_tensors_are_refused():
    x = torch.zeros(4, 8)
    for call in (lambda: moe.route(x, 2), lambda: moe.plan(torch.zeros(4, 2, dtype=torch.int32), 8), lambda: moe.quantize(x),
                 lambda: moe.swiglu_quantize(x), lambda: moe.dequantize(x, x), lambda: moe.combine(x, x),
                 lambda: moe.few_tokens(x, x, x, x), lambda: moe.FeedForward(x, x, x, x)):
        with pytest.raises(ValueError):
            call()


# ---- the oracle ---------------------------------------------------------------------

def test_oracle_quantisation_is_the_nearest_value():
    """By search over every value, and at the borders themselves."""
    rng = np.random.default_rng(1)
    v = (rng.standard_normal((200, 16)) * np.exp(rng.uniform(-9, 9, (200, 1)))).astype(np.float32)
    codes, scales = MO.quantize(v)
    for r in range(v.shape[0]):
        top = float(np.abs(v[r]).max()) / 6
        assert abs(MO.E4M3[scales[r, 0]] - min(top, 448)) == np.min(np.abs(MO.E4M3 - min(top, 448)))
        s = MO.E4M3[scales[r, 0]]
        for i in range(16):
            got = abs(O.E2M1_VALUES[codes[r, i]]) * s
            want = np.min(np.abs(MO.E2M1 * s - min(abs(float(v[r, i])), 6 * s)))
            assert abs(got - min(abs(float(v[r, i])), 6 * s)) == want
            assert (codes[r, i] >= 8) == (v[r, i] < 0 and s != 0)
    # ties: 2.5 lies between 2 (code 4) and 3 (code 5), with 6 in the block the scale is 1
    row = np.zeros((1, 16), dtype=np.float32)
    row[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    codes, scales = MO.quantize(row)
    assert codes[0, :8].tolist() == [7, 0, 2, 2, 4, 4, 6, 6] and scales[0, 0] == 0x38


def test_oracle_pack_and_unpack_are_inverse():
    rng = np.random.default_rng(2)
    codes, scales = rng.integers(0, 16, (130, 96), dtype=np.uint8), rng.integers(0, 127, (130, 6), dtype=np.uint8)
    a, sf = MO.pack(codes, scales)
    assert sf.size == mm.nvfp4_sf_bytes(130, 96)
    c2, s2 = MO.unpack_rows(a, sf, 130, 96)
    assert np.array_equal(codes, c2) and np.array_equal(scales, s2)
    assert np.array_equal(MO.values(codes, scales), O.dequantize(a, sf, 130, 96))


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(3)
    h = 1e-6
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            x, dw = rng.standard_normal((3, 9)), rng.standard_normal((3, 4))
            how = dict(score=score, renormalize=renormalize, scale=2.5)
            ids, _ = MO.route(x, 4, **how)
            got, _ = MO.route_backward(x, ids, dw, **how)

            def loss(z):
                s = MO.scores(z, score)
                chosen = np.take_along_axis(s, ids.astype(np.int64), 1)
                return (dw * 2.5 * (chosen / chosen.sum(1, keepdims=True) if renormalize else chosen)).sum()
            for t in range(3):
                for e in range(9):
                    d = np.zeros_like(x)
                    d[t, e] = h
                    assert abs((loss(x + d) - loss(x - d)) / (2 * h) - got[t, e]) < 1e-8
    c, dy, w = rng.standard_normal((6, 8)), rng.standard_normal((2, 8)), rng.standard_normal((2, 3))
    rows = np.array([[4, 0, -1], [1, 5, 2]])
    dc, dwt, _ = MO.combine_backward(dy, c, w, rows)
    f = lambda c, w: (MO.combine(c, w, rows)[0] * dy).sum()  # noqa: E731
    for i, j in np.ndindex(6, 8):
        d = np.zeros_like(c)
        d[i, j] = h
        diff = (f(c + d, w) - f(c - d, w)) / (2 * h)
        assert abs(diff - (0 if np.isnan(dc[i, j]) else dc[i, j])) < 1e-7
    for i, j in np.ndindex(2, 3):
        d = np.zeros_like(w)
        d[i, j] = h
        assert abs((f(c, w + d) - f(c, w - d)) / (2 * h) - dwt[i, j]) < 1e-7
