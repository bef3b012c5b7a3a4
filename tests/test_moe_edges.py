"""Edges of the operators around the grouped GEMM that need no GPU: refusals of
entry points, and what the host decides. (Every call here returns before any HIP
call.)"""
import moe_matmul_amd as mm
from moe_matmul_amd import _moe_binding as c
from test_moe_abi import INVALID, MISALIGNED, P, refused


def test_plan_with_ids_of_its_own_refuses_as_the_plan_does():
    def call(tokens=4, topk=2, experts=8, ids=P, slot_ids=P):
        c.nvfp4_moe_plan_ex(ids, tokens, topk, experts, P, P, P, P, slot_ids, None, 0, 0, 0, 0)
    refused(INVALID, call, -1)
    refused(INVALID, call, 4, 2, 513)
    refused(INVALID, call, 4, 2, 8, 0)
    refused(MISALIGNED, call, 4, 2, 8, P, P + 2)
    refused(mm.NVFP4_ERR_WORKSPACE, call, 4097, 2)
