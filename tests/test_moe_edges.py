"""Edges of the operators around the grouped GEMM that need no GPU: refusals of
entry points, and what the host decides. (Every call here returns before any HIP
call.)"""
import pytest

import moe_matmul_amd as mm
from moe_matmul_amd import _moe_binding as c
from moe_matmul_amd import moe
from test_moe_abi import INVALID, MISALIGNED, P, refused


def test_plan_with_ids_of_its_own_refuses_as_the_plan_does():
    def call(tokens=4, topk=2, experts=8, ids=P, slot_ids=P):
        c.nvfp4_moe_plan_ex(ids, tokens, topk, experts, P, P, P, P, slot_ids, None, 0, 0, 0, 0)
    refused(INVALID, call, -1)
    refused(INVALID, call, 4, 2, 513)
    refused(INVALID, call, 4, 2, 8, 0)
    refused(MISALIGNED, call, 4, 2, 8, P, P + 2)
    refused(mm.NVFP4_ERR_WORKSPACE, call, 4097, 2)


@pytest.mark.parametrize("n,k,codes", [(4096, 7168, True), (16, 16384, True), (7168, 2048, True), (64, 32, True), (1 << 20, 32, False)])
def test_most_rows_of_a_group(n, k, codes):
    """The last number of rows that the grouped GEMM's own check takes; as a rule that of 2^31 bytes of codes."""
    most = moe._most_rows(n, k)
    assert mm.nvfp4_device_group_tiles((most, n, k, 1), (4096,) * 5) > 0
    assert mm.nvfp4_device_group_tiles((most + 1, n, k, 1), (4096,) * 5) == -1
    assert (most == (2 ** 31 - 1) // (k // 2)) == codes
    with pytest.raises(ValueError):
        moe._most_rows(1 << 18, 1 << 14)
