"""The router at the token numbers where another number of lanes serves a token, for
expert numbers on both sides of what a lane's registers hold."""
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
from test_gpu_moe_route import BF, DEV, bias_of, check_route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [2999, 3000, 4095, 4096, 4099])
@pytest.mark.parametrize("experts,topk,groups", [(65, 16, 5), (100, 8, 4), (128, 8, 8), (129, 7, 3), (384, 8, 8), (40, 17, 1)])
def test_route_where_lanes_change(tokens, experts, topk, groups):
    gen = torch.Generator().manual_seed(tokens + experts)
    logits = (1.5 * torch.randn(tokens, experts, generator=gen)).to(DEV)
    logits[7, ::2] = -float("inf")
    logits[tokens - 1, 5:] = float("nan")
    check_route(logits, mx.Router(topk, "sigmoid", bias_of(experts), groups, max(1, groups // 2), "top2", scale=2.5), "sigmoid")
    check_route(logits.to(BF), mx.Router(topk), "softmax")
