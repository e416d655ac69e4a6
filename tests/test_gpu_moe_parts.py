"""A GPU that holds a part of the experts: its rows are the same sums, bit for bit, as
where all experts are in one stack, since the kernels are chosen by the rows that
an expert can expect of the whole router.  The operands' blocks differ by up to
2^20 in size, so that sums in another order are other bits."""
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
from test_gpu_moe import BF, DEV, F, R, T, announce

pytestmark = pytest.mark.gpu


def block(seed, tokens, experts, d, f, layout):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rough(*shape):
        size = torch.randint(-10, 11, (*shape[:-1], shape[-1] // 32), generator=gen, device=DEV)
        return torch.ldexp(torch.randn(shape, generator=gen, device=DEV), size.repeat_interleave(32, -1))
    up, gate = (mx.quantize_experts(0.05 * rough(experts, f, d), mx.HADAMARD32, layout=layout) for _ in range(2))
    return dict(x=rough(tokens, d).to(BF), logits=torch.randn(tokens, experts, generator=gen, device=DEV), w_up=up, w_gate=gate,
                w_down=mx.quantize_experts(0.05 * rough(experts, d, f), mx.HADAMARD32, layout=layout), rot=mx.HADAMARD32)


def part(w, first, experts):
    return None if w is None else tuple(t[first:first + experts].contiguous() for t in w)


# tokens, router's experts, topk, first, experts, d, hidden: means of 4, 8, 12, 15 and
# 40 rows, which as rows of the part's experts alone are 8 and 4 times as many
@pytest.mark.parametrize("tokens,router,topk,first,experts,d,f,layout", [
    (64, 64, 4, 8, 8, 512, 384, T), (64, 64, 8, 56, 8, 640, 256, T), (96, 32, 4, 0, 8, 256, 640, R), (81, 16, 3, 4, 4, 160, 224, R),
    (80, 16, 8, 12, 4, 512, 512, T)])
def test_parts_have_the_whole_sums(tokens, router, topk, first, experts, d, f, layout):
    b = block(tokens + first, tokens, router, d, f, layout)
    r = mx.Router(topk, "sigmoid")
    residual = torch.randn(tokens, d, device=DEV)
    ids, w = mx.moe_route(b["logits"], r)
    mine = torch.where((ids >= first) & (ids < first + experts), ids, -1)
    announce("moe_ffn, part", tokens, router, topk, first, experts, d, f, layout)
    # the same pairs in the whole stack
    whole = mx.moe_plan(mine, router)
    a = mx.quantize_rotate(b["x"], b["rot"], layout=layout)
    kw = dict(layout=layout, n=f)
    h = mx.moe_up(*a, whole, b["w_up"], b["w_gate"], out_dtype=F, **kw)
    q = mx.moe_up_requant(*a, whole, b["w_up"], b["w_gate"], rot=b["rot"], out_layout=layout, **kw)
    y = mx.moe_down(*q, whole, w, b["w_down"], residual=residual, out_dtype=F, layout=layout, n=d)
    # the part alone
    plan = mx.moe_plan(ids, experts, first, router_experts=router)
    up, gate, down = (part(b[k], first, experts) for k in ("w_up", "w_gate", "w_down"))
    rows = int(plan.offsets[-1])
    assert rows == int(whole.offsets[-1]) and torch.equal(plan.order, whole.order)
    got = mx.moe_up(*a, plan, up, gate, out_dtype=F, **kw)
    assert torch.equal(got[:rows], h[:rows])
    gq = mx.moe_up_requant(*a, plan, up, gate, rot=b["rot"], out_layout=layout, **kw)
    assert torch.equal(mx.moe_down(*gq, plan, w, down, residual=residual, out_dtype=F, layout=layout, n=d), y)
    assert torch.equal(mx.moe_ffn(b["x"], b["logits"], r, up, down, f, gate, rot=b["rot"], residual=residual, first=first,
                                  layout=layout), y)


def test_plan_refuses_parts_that_the_router_does_not_have():
    ids = torch.zeros(6, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="not among 8"):
        mx.moe_plan(ids, 4, 5, router_experts=8)
    plan = mx.moe_plan(ids, 4, 4, router_experts=8)
    assert plan.router_experts == 8 and mx.moe_plan(ids, 4).router_experts == 4
    assert mx.moe_plan(ids, 4, 4, plan) is plan and mx.moe_plan(ids, 4, 0, plan, 8) is plan
    with pytest.raises(ValueError, match="4 of 8 experts"):
        mx.moe_plan(ids, 4, 4, plan, 16)
