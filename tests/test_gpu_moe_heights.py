"""Experts' products on both sides of where the row tiles' height changes: 16, 32 and
128 rows of tiled operands, 16 and 128 of row-major ones; and operands past 4 GiB,
whose few rows stay on tiles of 16."""
import ctypes

import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
import test_gpu_moe as products
from test_gpu_moe import DEV, F, R, T, announce

pytestmark = pytest.mark.gpu

# tokens, topk, experts, k, n: mean 10, 11, 18 and 19 rows; K on both ends of 32-row tiles
TILED = [(50, 3, 15, 2048, 96), (55, 2, 10, 2048, 96), (99, 2, 11, 2048, 300), (90, 1, 5, 4096, 128), (57, 3, 9, 2176, 64),
         (33, 3, 9, 1920, 128), (55, 2, 10, 4224, 40), (50, 1, 5, 256, 128), (22, 2, 4, 256, 160)]
ROWS = [(14, 2, 10, 1056, 200), (15, 2, 10, 1056, 200), (8, 2, 8, 2048, 64), (12, 2, 8, 2048, 96), (36, 1, 2, 160, 1000)]


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("tokens,topk,experts,k,n", TILED)
def test_up_tiled(tokens, topk, experts, k, n, gated):
    products.test_up(tokens, topk, experts, k, n, gated, T)


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("tokens,topk,experts,k,n", ROWS)
def test_up_row_major(tokens, topk, experts, k, n, gated):
    products.test_up(tokens, topk, experts, k, n, gated, R)


@pytest.mark.parametrize("layout,tokens,topk,experts,k,n", [(T, *c) for c in TILED] + [(R, *c) for c in ROWS])
def test_down(tokens, topk, experts, k, n, layout):
    products.test_down(tokens, topk, experts, k, n, layout)


@pytest.mark.parametrize("layout", [R, T])
def test_few_rows_of_an_expert_past_4_gib(layout):
    """One expert of 2^16 + 8 rows of K = 2^17, 4.3 GB of codes: 12 rows of ones
    against a row of ones for each column, with a scale of its own (exact: 2^17 2^s)."""
    k, n, tokens = 2 ** 17, 2 ** 16 + 8, 12
    pad = mx.padded_rows(n) if layout == T else n
    codes = torch.full((1, pad, k // 2), 0x22, dtype=torch.uint8, device=DEV)            # every element 1
    power = torch.arange(pad, device=DEV) % 5                                            # of a row
    if layout == T:   # [tile, stage, row, 4 scales]
        scales = (127 + power).to(torch.uint8).view(-1, 1, 256, 1).expand(pad // 256, k // 128, 256, 4)
    else:
        scales = (127 + power).to(torch.uint8)[:, None].expand(pad, k // 32)
    scales = scales.reshape(1, pad, k // 32).contiguous()
    rows = mx.padded_rows(tokens) if layout == T else tokens
    a = torch.full((rows, k // 2), 0x22, dtype=torch.uint8, device=DEV), torch.full((rows, k // 32), 127, dtype=torch.uint8,
                                                                                    device=DEV)
    want = torch.ldexp(torch.full((n,), float(k), device=DEV), power[:n].int())
    plan = mx.moe_plan(torch.zeros(tokens, 1, dtype=torch.int32, device=DEV), 1)
    announce("past 4 GiB", layout)
    y = mx.moe_up(*a, plan, (codes, scales), act="none", out_dtype=F, layout=layout, n=n)
    assert torch.equal(y, want.expand(tokens, n))
    y = mx.moe_down(*a, plan, torch.full((tokens, 1), 0.5, device=DEV), (codes, scales), out_dtype=F, layout=layout, n=n)
    assert torch.equal(y, 0.5 * want.expand(tokens, n))
    # more rows are refused, by the workspace's size too
    b = ctypes.c_int64()
    assert mx.lib().mxfp4_moe_down_workspace(19, 1, 1, n, k, layout, mx.MXFP4_F32, ctypes.byref(b)) == mx.MXFP4_ERR_UNSUPPORTED
    assert mx.lib().mxfp4_moe_down_workspace(18, 1, 1, n, k, layout, mx.MXFP4_F32, ctypes.byref(b)) == mx.MXFP4_OK
    assert b.value >= 18 * n * 4
