"""Few rows of many experts at the sizes where their kernel gives way to tiles, and routings that leave all rows to one
expert, checked as the other few rows are (test_ffn_gpu.py)."""
import pytest

import test_ffn_gpu
from test_ffn_gpu import announce  # noqa: F401

pytestmark = pytest.mark.gpu

# tokens, topk, experts, inner, hidden, share of slots dropped, the only expert
CASES = [(16, 4, 64, 504, 72, 0.1, None), (16, 4, 64, 2056, 136, 0.0, None), (15, 4, 300, 136, 2048, 0.1, None), (8, 8, 256, 64, 512, 0.0, None),
         (64, 1, 64, 512, 136, 0.0, 63), (64, 1, 64, 512, 136, 0.2, 5), (65, 1, 64, 512, 136, 0.0, 63), (13, 5, 64, 264, 200, 0.0, None),
         (16, 4, 16, 96, 5000, 0.0, None), (256, 1, 64, 256, 520, 0.0, 7), (1000, 1, 250, 64, 264, 0.05, 249), (128, 8, 256, 64, 136, 0.0, None)]


@pytest.mark.parametrize("i", range(len(CASES)), ids=lambda i: "-".join(map(str, CASES[i])))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_few_rows_of_many_experts(i, dtype, monkeypatch):
    monkeypatch.setattr(test_ffn_gpu, "FEW", [CASES[i]])
    test_ffn_gpu.test_few_rows_of_many_experts(0, dtype)
