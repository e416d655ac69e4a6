"""Mixture-of-experts calls at the largest numbers of choices and experts, and of more
tokens or columns than one grid's 2^32 threads hold.  Whole batches are compared on the device, or their rows with those of
short calls on a part of the same logits."""
import ctypes

import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
import test_gpu_moe as products

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F = torch.bfloat16, torch.float32


def announce(*what):
    print("[case]", *what, flush=True)


def packed(rows, k, seed, *lead):
    """Codes and scales of random MXFP4 rows whose products are exact sums (K 32,
    multiples of 2^-8 below 2^11)."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randint(0, 256, (*lead, rows, k // 2), dtype=torch.uint8, generator=gen, device=DEV),
            torch.randint(124, 128, (*lead, rows, k // 32), dtype=torch.uint8, generator=gen, device=DEV))


def values(codes, scales):
    """fp32 values of [rows, 16] codes and [rows, 1] scales."""
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    lut = torch.cat((lut, -lut))
    v = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).reshape(len(codes), 32)
    return torch.ldexp(v, scales.int() - 127)


def test_down_past_one_grid_of_columns():
    """One pair, 2^27 + 40 columns: the sums are exact in fp32, y = residual + 0.5 z
    one rounding each side."""
    n = 2 ** 27 + 40
    b = ctypes.c_int64()
    assert mx.lib().mxfp4_moe_down_workspace(1, 1, 1, n, 32, mx.ROWMAJOR, mx.MXFP4_F32, ctypes.byref(b)) == 0
    assert b.value >= 4 * n
    h, w = packed(1, 32, 3), packed(n, 32, 4, 1)
    plan = mx.moe_plan(torch.zeros(1, 1, dtype=torch.int32, device=DEV), 1)
    weights = torch.full((1, 1), 0.5, device=DEV)
    y = torch.full((1, n), float("nan"), device=DEV)
    announce("moe_down", 1, n)
    mx.moe_down(*h, plan, weights, w, y=y)
    x = values(*h)
    for at in range(0, n, 2 ** 23):
        rows = slice(at, at + 2 ** 23)
        assert torch.equal(y[0, rows], 0.5 * (values(w[0][0, rows], w[1][0, rows]) * x).sum(-1)), at


def test_down_of_many_tokens():
    """2^26 + 9 tokens of one expert: the weighted sum's grid of three dimensions."""
    tokens, n = 2 ** 26 + 9, 32
    h, w = packed(tokens, 32, 5), packed(n, 32, 6, 1)
    plan = mx.moe_plan(torch.zeros(tokens, 1, dtype=torch.int32, device=DEV), 1)
    weights = torch.full((tokens, 1), 0.25, device=DEV)
    y = torch.full((tokens, n), float("nan"), device=DEV)
    announce("moe_down", tokens, n)
    mx.moe_down(*h, plan, weights, w, y=y)
    wv = values(w[0][0], w[1][0])
    for at in list(range(0, tokens, 2 ** 23 - 5)) + [tokens - 1000]:
        rows = slice(at, at + 100000)
        want = (values(h[0][rows], h[1][rows])[:, None] * wv).sum(-1)
        assert torch.equal(y[rows], 0.25 * want), at


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


@pytest.mark.parametrize("layout", [mx.ROWMAJOR, mx.TILED])
@pytest.mark.parametrize("tokens,topk,experts,k,n", [(2, 64, 100, 128, 96), (5, 64, 100, 128, 96), (40, 17, 1024, 128, 64),
                                                     (300, 12, 20, 128, 288), (90, 64, 64, 256, 40)])
def test_products_of_many_choices_and_experts(tokens, topk, experts, k, n, layout):
    products.test_up(tokens, topk, experts, k, n, True, layout)
    products.test_down(tokens, topk, experts, k, n, layout)
