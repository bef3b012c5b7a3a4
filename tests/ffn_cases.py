"""Sizes of the products that the GPU tests compute, shared with the CPU test that they reach every kernel."""
from moe_matmul_amd import _ffn_binding as c

PRODUCT_KINDS = (c.NVFP4_FFN_FORWARD, c.NVFP4_FFN_FORWARD_CODES, c.NVFP4_FFN_DX, c.NVFP4_FFN_DW)

# rows, n, k of dense products; each forward and backward
LINEAR = [
    (1, 8, 8), (1, 136, 4096), (3, 24, 40), (8, 264, 72), (9, 8, 200), (16, 128, 64), (17, 136, 72), (64, 264, 200),
    (65, 120, 1000), (40, 512, 4104), (129, 256, 520), (257, 264, 1000), (300, 1032, 8), (2, 4096, 24), (2000, 64, 64),
    (257, 64, 64), (257, 64, 1032), (257, 1024, 64), (257, 4096, 8192), (520, 4096, 1032), (520, 4104, 4096),
    (1024, 64, 64), (2051, 512, 2048), (2051, 64, 2048), (4099, 64, 2048), (4099, 256, 4096), (4099, 1024, 64),
    (4099, 1024, 512), (4099, 2048, 64), (4099, 4096, 128), (600, 4104, 5128), (4100, 2048, 136), (5100, 3136, 64),
    (2051, 264, 4104), (4100, 264, 4104), (330, 8192, 1984), (2051, 1024, 4096), (8200, 2048, 4096), (4800, 2112, 512),
    (2500, 1024, 4096), (8195, 512, 8192),
]
# rows, inner, k of dense gated projections
GATED = [
    (1, 8, 8), (1, 64, 4096), (3, 24, 40), (8, 136, 72), (9, 40, 200), (17, 96, 72), (33, 256, 2048), (64, 96, 264),
    (100, 32, 4096), (129, 160, 520), (300, 520, 64), (257, 32, 64), (257, 32, 1032), (257, 2048, 8192), (4099, 512, 64),
    (4099, 512, 512), (4099, 1024, 64), (4099, 2048, 256), (330, 992, 8192), (4100, 1024, 160), (5100, 1568, 64), (4800, 1056, 512),
]


def parts_of(linear, gated):
    """(kind, parts) of every product that the tests of these sizes compute."""
    for m, n, k in linear:
        yield c.NVFP4_FFN_FORWARD, c.nvfp4_ffn_product_parts(c.NVFP4_FFN_FORWARD, m, n, k, 0)
        yield c.NVFP4_FFN_DX, c.nvfp4_ffn_product_parts(c.NVFP4_FFN_DX, m, n, k, 0)
        yield c.NVFP4_FFN_DW, c.nvfp4_ffn_product_parts(c.NVFP4_FFN_DW, m, n, k, 0)
    for m, i, k in gated:
        yield c.NVFP4_FFN_FORWARD, c.nvfp4_ffn_product_parts(c.NVFP4_FFN_FORWARD, m, 2 * i, k, 0)
        if i % 32 == 0:
            yield c.NVFP4_FFN_FORWARD_CODES, c.nvfp4_ffn_product_parts(c.NVFP4_FFN_FORWARD_CODES, m, 2 * i, k, 0)
        yield c.NVFP4_FFN_DX, c.nvfp4_ffn_product_parts(c.NVFP4_FFN_DX, m, 2 * i, k, 0)
        yield c.NVFP4_FFN_DW, c.nvfp4_ffn_product_parts(c.NVFP4_FFN_DW, m, 2 * i, k, 0)
