"""The router at the token numbers where another number of lanes serves a token, for
expert numbers on both sides of what a lane's registers hold."""
import math

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


@pytest.mark.parametrize("tokens,experts,topk,groups,kept", [(20, 64, 10, 8, 1), (4100, 64, 10, 8, 1), (4100, 240, 16, 30, 1),
                                                             (9, 1024, 64, 64, 3), (7, 130, 30, 13, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_where_the_kept_groups_have_fewer_experts_than_choices(tokens, experts, topk, groups, kept, score):
    gen = torch.Generator().manual_seed(tokens)
    logits = torch.randn(tokens, experts, generator=gen).to(DEV)
    for bias in (None, bias_of(experts)):
        ids, w = check_route(logits, mx.Router(topk, score, bias, groups, kept, "max"), "few experts kept")
        left = max(0, topk - experts // groups * kept)
        assert ((ids == -1).sum(1) == left).all() and ((w == 0).sum(1) == left).all()


@pytest.mark.parametrize("base", [-690.0, -703.0, -709.0, -720.0, -738.0])
def test_weights_of_scores_near_binary64s_end(base):
    """Sigmoid scores down to 2^-1074: the chosen ones' ratio is that of e^l, each off
    by half a subnormal step (2^-1075) or by 2^-44 of itself, and a rounding to fp32."""
    logits = torch.tensor([[base, base - 1.0, base - 2.5, base - 6.0], [base - 6.0, base, base, base]])
    for r in (mx.Router(3, "sigmoid"), mx.Router(2, "sigmoid", torch.zeros(4, device=DEV), 2, 1, "top2")):
        ids, w = mx.moe_route(logits.to(DEV), r)
        for row, chosen, got in zip(logits.tolist(), ids.tolist(), w.tolist()):
            e = [math.exp(row[i]) for i in chosen]
            off = max(2.0 ** -1074 / x + 2.0 ** -43 for x in e)
            for x, y in zip(e, got):
                assert abs(y - x / sum(e)) <= (2 * off + 2.0 ** -24) * x / sum(e), (base, chosen, got)
    # a softmax whose largest experts are in another group
    far = torch.tensor([[0.0, 0.0, base, base - 1.0]], device=DEV)
    ids, w = mx.moe_route(far, mx.Router(2, "softmax", torch.tensor([-9.0, -9.0, 0.0, 0.0], device=DEV), 2, 1))
    e = [math.exp(base), math.exp(base - 1.0)]
    assert ids.tolist() == [[2, 3]]
    assert abs(w[0, 1].item() - e[1] / sum(e)) <= (4 * 2.0 ** -1074 / e[1] + 2.0 ** -24 + 2.0 ** -42) * e[1] / sum(e)
