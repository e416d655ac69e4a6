"""Mixture-of-experts calls of more tokens or columns than one grid's 2^32 threads
hold.  Whole batches are compared on the device, or their rows with those of
short calls on a part of the same logits."""
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F = torch.bfloat16, torch.float32


def announce(*what):
    print("[case]", *what, flush=True)


def test_route_past_one_grid_16_lanes():
    tokens = 2 ** 28 + 70
    gen = torch.Generator(device=DEV).manual_seed(1)
    logits = torch.randn(tokens, 2, generator=gen, device=DEV, dtype=BF)
    announce("moe_route", tokens, 2)
    ids, w = mx.moe_route(logits, mx.Router(1))
    assert torch.equal(ids[:, 0], (logits[:, 1] > logits[:, 0]).int()) and (w == 1).all()


def test_route_past_one_grid_64_lanes():
    tokens, experts, topk = 2 ** 26 + 300, 20, 17
    gen = torch.Generator(device=DEV).manual_seed(2)
    logits = torch.randn(tokens, experts, generator=gen, device=DEV, dtype=BF)
    bias = 0.1 * torch.randn(experts, generator=gen, device=DEV)
    r = mx.Router(topk, "sigmoid", bias, 4, 4, "top2", scale=2.5)
    ids, w = torch.full((tokens, topk), -7, dtype=torch.int32, device=DEV), torch.zeros(tokens, topk, device=DEV)
    announce("moe_route", tokens, experts, topk)
    mx.moe_route(logits, r, ids, w)
    for at in (0, 2 ** 25 - 2000, 2 ** 25 - 4, tokens - 2500):
        part, pw = mx.moe_route(logits[at:at + 2500], r)
        assert torch.equal(ids[at:at + 2500], part) and torch.equal(w[at:at + 2500], pw)
    assert (ids >= 0).all() and ((w.sum(-1) - 2.5).abs() < 1e-5).all()
