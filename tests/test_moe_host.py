"""What the mixture-of-experts binding refuses by sizes alone, on the CPU."""
import ctypes
import dataclasses

import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
from mxfp4_w4a4_quantized_amd import moe


def stack(experts, n, k):
    return torch.zeros(experts, n, k // 2, dtype=torch.uint8), torch.zeros(experts, n, k // 32, dtype=torch.uint8)


@pytest.mark.parametrize("first,experts", [(-1, 4), (5, 4), (8, 1), (0, 9), (1 << 29, 4)])
def test_ffn_refuses_experts_that_the_logits_do_not_have(first, experts):
    """8 experts routed: this GPU's have to be among them (else they add nothing, silently)."""
    x, logits = torch.zeros(3, 64), torch.zeros(3, 8)
    with pytest.raises(ValueError, match="not among the logits' 8"):
        mx.moe_ffn(x, logits, mx.Router(2), stack(experts, 32, 64), stack(experts, 64, 32), 32, first=first)
    with pytest.raises(ValueError, match="GPU"):                    # (the whole and a part pass this check)
        mx.moe_ffn(x, logits, mx.Router(2), stack(8, 32, 64), stack(8, 64, 32), 32)
    with pytest.raises(ValueError, match="GPU"):
        mx.moe_ffn(x, logits, mx.Router(2), stack(4, 32, 64), stack(4, 64, 32), 32, first=4)


def test_products_refuse_a_plan_whose_words_are_not_of_its_sizes():
    """(the check itself, with the host's number for a device: -1)"""
    need = moe._plan_words(10, 3, 5)
    words = torch.zeros(need, dtype=torch.int32)
    assert moe._plan_ptr(mx.ExpertPlan(words, 10, 3, 5), -1) == words.data_ptr()
    for sizes in ((11, 3, 5), (10, 4, 5), (10, 3, 6), (9, 3, 5), (1000, 8, 64)):
        with pytest.raises(ValueError, match="int32 words"):
            moe._plan_ptr(mx.ExpertPlan(words, *sizes), -1)
    for bad in (words[1:], words.float(), words.long(), torch.zeros(2 * need, dtype=torch.int32)[::2], words.reshape(1, -1)):
        with pytest.raises(ValueError, match="int32 words"):
            moe._plan_ptr(mx.ExpertPlan(bad, 10, 3, 5), -1)
    with pytest.raises(RuntimeError):
        moe._plan_ptr(mx.ExpertPlan(words, 10, 65, 5), -1)
    with pytest.raises(ValueError, match="host"):
        moe._plan_ptr(mx.ExpertPlan(words, 10, 3, 5), 0)
    with pytest.raises(dataclasses.FrozenInstanceError):
        mx.ExpertPlan(words, 10, 3, 5).topk = 30


A = 1 << 20          # an aligned address, never dereferenced
INV, UNS, OK = mx.MXFP4_ERR_INVALID_ARG, mx.MXFP4_ERR_UNSUPPORTED, mx.MXFP4_OK


@pytest.mark.parametrize("of,want", [(0, OK), (8, OK), (9, OK), (1024, OK), (7, INV), (1, INV), (-1, INV), (1025, UNS)])
def test_router_experts_are_at_least_the_plans(of, want):
    """(no columns: nothing is launched)"""
    up = moe.MoeUpDesc(2, 0, A, A, None, None, None, None, of)
    down = moe.MoeDownDesc(A, A, None, 0, of)
    L = mx.lib()
    assert L.mxfp4_moe_up(A, A, A, 4, 2, 8, up, 0, 128, 0, A, 0, 0, None) == want
    assert L.mxfp4_moe_up_requant(A, A, A, 4, 2, 8, up, 0, 128, 0, None, A, A, 0, None) == want
    assert L.mxfp4_moe_down(A, A, A, 4, 2, 8, A, down, 0, 128, 0, None, 0, 0, A, 0, 0, None, 0, None) == want


def test_workspace_of_a_part_of_the_experts():
    """64 tokens x 8 of 128 experts, 16 of them here: a mean of 4 rows, whose products
    are fp32; as if all pairs went to the 16 (32 rows) they would be held in 16 bits."""
    def need(plan, n):
        b = ctypes.c_int64()
        assert mx.lib().mxfp4_moe_down_workspace(plan.tokens, plan.topk, plan.router_experts, n, 2048, 1, mx.MXFP4_BF16,
                                                 ctypes.byref(b)) == OK
        return b.value
    assert need(mx.ExpertPlan(None, 64, 8, 16, 128), 4096) >= 512 * 4096 * 4
    assert need(mx.ExpertPlan(None, 64, 8, 16), 4096) < 512 * 4096 * 4


@pytest.mark.parametrize("tokens,topk,experts,n,k", [(75000, 8, 64, 4096, 14336), (1 << 21, 1, 1, 128, 1 << 13),
                                                     (1 << 12, 1, 1, 1 << 26, 128), (4096, 2, 8, 128, 1 << 26)])
def test_workspace_refuses_what_the_product_refuses(tokens, topk, experts, n, k):
    """Code bytes of A or of one expert past 2^32: known before anything is launched."""
    b = ctypes.c_int64()
    w = moe.MoeDownDesc(A, A, None, 0, 0)
    for layout in (0, 1):
        assert mx.lib().mxfp4_moe_down(A, A, A, tokens, topk, experts, A, w, n, k, layout, None, 0, 0, A, 0, n, A, 1 << 60,
                                       None) == UNS
        assert mx.lib().mxfp4_moe_down_workspace(tokens, topk, experts, n, k, layout, 0, ctypes.byref(b)) == UNS
    with pytest.raises(mx.Mxfp4Error):                                # moe_ffn's sizes of the same block
        moe._ffn_work(tokens, topk, experts, experts, n, k, mx.TILED, mx.MXFP4_F32, -1)
