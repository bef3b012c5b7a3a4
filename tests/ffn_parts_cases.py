"""Sizes of products that reach what those of ffn_cases do not: every tile with parts of k, dense and by experts, shared
with the CPU test that they do."""
from moe_matmul_amd import _ffn_binding as c

# rows, n, k; forward and backward
LINEAR = [(8662, 8248, 136), (275, 7664, 8456)]
# rows, inner, k
GATED = [(5628, 96, 11968), (8226, 160, 5280)]
# tokens, topk, experts, inner, hidden: both projections, a product of inner to hidden, and their gradients
EXPERTS = [
    (1, 1, 16, 96, 2240), (4236, 2, 4, 32, 448), (3798, 2, 2, 288, 64), (2146, 1, 16, 2784, 64), (4067, 1, 16, 32, 2112), (1008, 2, 16, 32, 10400),
    (8399, 1, 8, 288, 416), (547, 2, 4, 4448, 64), (5091, 1, 16, 32, 9408), (4232, 1, 16, 800, 288), (361, 2, 3, 128, 10816),
    (4389, 2, 16, 32, 11264), (137, 1, 4, 2080, 8480), (1136, 1, 16, 4576, 352), (4993, 1, 8, 6976, 160), (259, 2, 4, 5024, 2720),
    (4036, 2, 8, 7104, 160), (987, 2, 8, 1088, 16256), (1081, 1, 4, 6624, 4480), (515, 1, 2, 13920, 9824), (8434, 1, 2, 4224, 160),
]


def _keys(names, rows, n, k, experts):
    """(kernel, by experts, tile's rows, columns, whether in parts of k) of the products with these names."""
    kinds = {"linear": c.NVFP4_FFN_FORWARD, "gated": c.NVFP4_FFN_FORWARD, "codes": c.NVFP4_FFN_FORWARD_CODES, "dx": c.NVFP4_FFN_DX,
             "dw": c.NVFP4_FFN_DW}
    return {(name, bool(experts), tile, cols, splits > 1) for name in names
            for _, tile, cols, splits in c.nvfp4_ffn_product_parts(kinds[name], rows, n, k, experts)}


def linear_kernels(rows, n, k, experts=0):
    return _keys(("linear", "dx", "dw"), rows, n, k, experts)


def gated_kernels(rows, inner, k, experts=0):
    return _keys(("gated", "dx", "dw") + (("codes",) if inner % 32 == 0 else ()), rows, 2 * inner, k, experts)


def experts_kernels(tokens, topk, experts, inner, hidden):
    return gated_kernels(tokens * topk, inner, hidden, experts) | linear_kernels(tokens * topk, hidden, inner, experts)
