"""Every tile with one part of k and with several, dense and by experts, at the sizes of ffn_parts_cases.py; checked as
the other sizes are (test_ffn_gpu.py)."""
import pytest

import test_ffn_gpu
from ffn_parts_cases import EXPERTS, GATED, LINEAR
from test_ffn_gated_acts_gpu import check_gated
from test_ffn_gpu import announce  # noqa: F401

pytestmark = pytest.mark.gpu

DTYPES = pytest.mark.parametrize("dtype", ["bf16", "fp16"])


def ids(size):
    return "x".join(map(str, size))


@DTYPES
@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu"])
@pytest.mark.parametrize("size", LINEAR, ids=ids)
def test_linear(size, act, dtype, monkeypatch):
    monkeypatch.setattr(test_ffn_gpu, "LINEAR", [size])
    monkeypatch.setattr(test_ffn_gpu, "setting", lambda i: dict(act=act, bias="fp32" if act else "same", residual=act != "relu"))
    test_ffn_gpu.test_linear_and_its_gradients(0, dtype)


@DTYPES
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("size", GATED, ids=ids)
def test_gated(size, act, dtype):
    check_gated(*size, act, dtype)


@DTYPES
@pytest.mark.parametrize("size", EXPERTS, ids=ids)
def test_experts(size, dtype, monkeypatch):
    """What was kept in 16 and in 8 bits, then nothing kept, with its gradient of the weights."""
    monkeypatch.setattr(test_ffn_gpu, "EXPERTS", [(*size, 0.1, None)])
    test_ffn_gpu.test_experts(0, dtype)
    monkeypatch.setattr(test_ffn_gpu, "FEW", [(*size, 0.0, None)])
    test_ffn_gpu.test_few_rows_of_many_experts(0, dtype)
