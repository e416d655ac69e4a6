"""Refusals of the mixture-of-experts entry points: synchronous status codes from
the library (the pointers are never dereferenced) and ValueErrors from the
binding, all without a GPU."""
import ctypes

import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
from mxfp4_w4a4_quantized_amd import moe

A = 1 << 20          # arbitrary aligned address: never dereferenced
F, BF = mx.MXFP4_F32, mx.MXFP4_BF16
R, T = mx.ROWMAJOR, mx.TILED
INV, UNS, OK = mx.MXFP4_ERR_INVALID_ARG, mx.MXFP4_ERR_UNSUPPORTED, mx.MXFP4_OK


def ref(d):
    return ctypes.byref(d) if d is not None else None


def router(**kw):
    d = dict(score=0, topk=2, groups=1, topk_groups=1, group_score=0, renormalize=1, scale=1.0)
    return moe.RouterDesc(**{**d, **kw})


def route(r, logits=A, dtype=F, tokens=4, experts=8, ld=8, ids=A, weights=A):
    return mx.lib().mxfp4_moe_route(logits, dtype, tokens, experts, ld, ref(r), ids, weights, None)


def test_route_refusals():
    assert route(None) == INV
    for bad in (dict(score=2), dict(score=-1), dict(topk=0), dict(topk=9), dict(groups=0), dict(groups=3), dict(topk_groups=0),
                dict(topk_groups=2), dict(group_score=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(reserved=1)):
        assert route(router(**bad)) == INV, bad
    assert route(router(), dtype=2) == INV
    assert route(router(), tokens=-1) == INV
    assert route(router(), experts=0) == INV
    assert route(router(), ld=7) == INV
    for name in ("logits", "ids", "weights"):
        assert route(router(), **{name: None}) == INV
        assert route(router(), **{name: A + 1}) == UNS
    assert route(router(bias=A + 2)) == UNS
    assert route(router(), experts=1025, ld=1025) == UNS
    assert route(router(topk=65), experts=128, ld=128) == UNS
    assert route(router(groups=128), experts=128, ld=128) == UNS
    assert route(router(), tokens=1 << 30) == UNS
    assert route(router(), tokens=0, logits=None, ids=None, weights=None) == OK


def plan_bytes(tokens, topk, experts):
    b = ctypes.c_int64(-1)
    return mx.lib().mxfp4_moe_plan_bytes(tokens, topk, experts, ctypes.byref(b)), b.value


def plan(ids=A, tokens=4, topk=2, first=0, experts=8, p=A, n=None):
    n = plan_bytes(max(tokens, 0), max(topk, 1), max(1, min(experts, 1024)))[1] if n is None else n
    return mx.lib().mxfp4_moe_plan(ids, tokens, topk, first, experts, p, n, None)


def test_plan_refusals():
    assert mx.lib().mxfp4_moe_plan_bytes(1, 1, 1, None) == INV
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0)):
        assert plan_bytes(*bad)[0] == INV
        assert plan(tokens=bad[0], topk=bad[1], experts=bad[2]) == INV
    for bad in ((1, 65, 1), (1, 1, 1025), (1 << 28, 1, 1), (1 << 25, 8, 1), (1 << 62, 64, 1)):
        assert plan_bytes(*bad)[0] == UNS
        assert plan(tokens=bad[0], topk=bad[1], experts=bad[2], n=1 << 50) == UNS
    st, n = plan_bytes(100, 3, 7)
    assert st == OK and n >= 4 * (8 + 3 * 300)
    assert plan(tokens=100, topk=3, experts=7, n=n - 4) == INV
    assert plan(first=-1) == INV
    assert plan(first=1 << 30) == UNS
    assert plan(ids=None) == INV
    assert plan(p=None) == INV
    assert plan(p=A + 4) == UNS
    assert plan(ids=A + 1) == UNS


def test_plan_bytes_cover_every_table():
    """Rows, slots, tokens, tiles of four heights and, past one chunk, its counts."""
    for tokens, topk, experts in ((0, 1, 1), (1, 1, 1), (5, 3, 40), (4096, 1, 9), (4097, 1, 9), (100000, 7, 300)):
        p = tokens * topk
        tiles = sum(p // h + min(p, experts) for h in (16, 32, 128, 256))
        st, n = plan_bytes(tokens, topk, experts)
        assert st == OK and n >= 4 * (experts + 1 + 3 * p + 4 + 4 * tiles)


def up_weights(**kw):
    d = dict(act=2, vec_dtype=BF, u_codes=A, u_scales=A, g_codes=A, g_scales=A)
    return moe.MoeUpDesc(**{**d, **kw})


def up(w, ac=A, as_=A, p=A, tokens=4, topk=2, experts=8, n=64, k=128, layout=R, y=A, y_dtype=BF, ld_y=64):
    return mx.lib().mxfp4_moe_up(ac, as_, p, tokens, topk, experts, ref(w), n, k, layout, y, y_dtype, ld_y, None)


def upq(w, rot=None, n=64, k=128, layout=R, yc=A, ys=A, y_layout=R, p=A, tokens=4, topk=2):
    return mx.lib().mxfp4_moe_up_requant(A, A, p, tokens, topk, 8, ref(w), n, k, layout, ref(rot), yc, ys, y_layout, None)


def test_up_refusals():
    assert up(None) == INV
    for bad in (dict(act=5), dict(act=-1), dict(vec_dtype=2), dict(reserved=1), dict(u_codes=None), dict(u_scales=None),
                dict(g_scales=None), dict(g_codes=None), dict(g_codes=None, g_scales=None, bias_g=A)):
        assert up(up_weights(**bad)) == INV, bad
        assert upq(up_weights(**bad)) == INV, bad
    w = up_weights()
    for bad in (dict(ac=None), dict(as_=None), dict(p=None), dict(y=None), dict(tokens=-1), dict(topk=0), dict(experts=0),
                dict(n=-1), dict(k=0), dict(k=100), dict(layout=2), dict(layout=T, k=96), dict(y_dtype=2), dict(ld_y=63)):
        assert up(w, **bad) == INV, bad
    for bad in (dict(ac=A + 8), dict(as_=A + 2), dict(p=A + 8), dict(y=A + 1), dict(topk=65), dict(experts=1025),
                dict(tokens=1 << 28), dict(n=1 << 30, ld_y=1 << 30), dict(k=1 << 30),
                dict(tokens=1 << 21, topk=1, k=1 << 13, experts=1), dict(tokens=1 << 12, topk=1, k=128, n=1 << 26, ld_y=1 << 26, experts=1)):
        assert up(w, **bad) == UNS, bad
    for bad in (dict(u_codes=A + 8), dict(g_codes=A + 8), dict(u_scales=A + 1), dict(g_scales=A + 2), dict(bias_u=A + 1),
                dict(bias_g=A + 1)):
        assert up(up_weights(**bad)) == UNS, bad
    assert up(w, tokens=0, ac=None, p=None, y=None) == OK
    assert up(w, n=0) == OK
    assert upq(w, yc=None) == INV and upq(w, ys=None) == INV and upq(w, y_layout=2) == INV and upq(w, p=None) == INV
    assert upq(w, n=40) == UNS and upq(w, y_layout=T) == UNS and upq(w, yc=A + 8) == UNS and upq(w, ys=A + 2) == UNS
    kron = mx.RotationDesc(mx.ROT_KRON, 4, 8, 0, A, A)
    assert upq(w, rot=kron) == UNS
    assert upq(w, rot=mx.RotationDesc(9, 0, 0, 0, None, None)) == INV
    assert upq(w, tokens=0) == OK


def down_bytes(tokens=40, topk=4, experts=64, n=64, k=128, layout=R, y_dtype=BF):
    b = ctypes.c_int64(-1)
    return mx.lib().mxfp4_moe_down_workspace(tokens, topk, experts, n, k, layout, y_dtype, ctypes.byref(b)), b.value


def down(w, hc=A, hs=A, p=A, tokens=40, topk=4, experts=64, weights=A, n=64, k=128, layout=R, res=None, rt=BF, ld_r=64, y=A,
         y_dtype=BF, ld_y=64, ws=A, size=1 << 40):
    return mx.lib().mxfp4_moe_down(hc, hs, p, tokens, topk, experts, weights, ref(w), n, k, layout, res, rt, ld_r, y, y_dtype,
                                   ld_y, ws, size, None)


def test_down_refusals():
    ok = dict(codes=A, scales=A, vec_dtype=BF)
    assert down(None) == INV
    for bad in (dict(codes=None), dict(scales=None), dict(vec_dtype=3), dict(reserved=1)):
        assert down(moe.MoeDownDesc(**{**ok, **bad})) == INV, bad
    for bad in (dict(codes=A + 8), dict(scales=A + 1), dict(bias=A + 1)):
        assert down(moe.MoeDownDesc(**{**ok, **bad})) == UNS, bad
    w = moe.MoeDownDesc(**ok)
    for bad in (dict(hc=None), dict(hs=None), dict(p=None), dict(weights=None), dict(y=None), dict(ws=None), dict(tokens=-1),
                dict(topk=0), dict(experts=0), dict(n=-1), dict(k=0), dict(k=100), dict(layout=2), dict(layout=T, k=96), dict(rt=2),
                dict(y_dtype=2), dict(ld_y=63), dict(res=A, ld_r=63), dict(size=0), dict(size=down_bytes()[1] - 1)):
        assert down(w, **bad) == INV, bad
    for bad in (dict(hc=A + 8), dict(hs=A + 2), dict(p=A + 8), dict(weights=A + 2), dict(y=A + 1), dict(ws=A + 128),
                dict(res=A + 1), dict(topk=65), dict(experts=1025), dict(tokens=1 << 28), dict(n=1 << 30, ld_y=1 << 30),
                dict(k=1 << 30)):
        assert down(w, **bad) == UNS, bad
    assert down(w, tokens=0, p=None, ws=None) == OK
    assert down(w, n=0) == OK


def test_down_workspace():
    assert mx.lib().mxfp4_moe_down_workspace(1, 1, 1, 32, 32, R, BF, None) == INV
    for bad in (dict(tokens=-1), dict(topk=0), dict(experts=0), dict(n=-1), dict(k=0), dict(k=33), dict(layout=5), dict(y_dtype=4)):
        assert down_bytes(**bad)[0] == INV, bad
    for bad in (dict(topk=65), dict(experts=1025), dict(tokens=1 << 28), dict(n=1 << 30), dict(k=1 << 30)):
        assert down_bytes(**bad)[0] == UNS, bad
    assert down_bytes(tokens=0) == (OK, 0) and down_bytes(n=0) == (OK, 0)
    # fp32 products for few rows or an fp32 result, else 16 bits and a byte for 32 columns
    assert down_bytes()[1] >= 160 * 64 * 4
    assert down_bytes(tokens=4) == (OK, 0)             # few pairs: products and sum in one launch
    big = dict(tokens=4096, topk=2, experts=8, n=256)
    assert down_bytes(**big, y_dtype=F)[1] >= 8192 * 256 * 4
    assert 8192 * (512 + 8) <= down_bytes(**big)[1] < 8192 * 256 * 4
    assert down_bytes(**{**big, "n": 250})[1] >= 8192 * 250 * 4


def test_structs_match_the_header():
    """Field offsets as the C compiler lays them out (4-byte integers, then 8-byte pointers)."""
    assert ctypes.sizeof(moe.RouterDesc) == 40 and moe.RouterDesc.bias.offset == 32 and moe.RouterDesc.scale.offset == 24
    assert ctypes.sizeof(moe.MoeUpDesc) == 64 and moe.MoeUpDesc.u_codes.offset == 8 and moe.MoeUpDesc.reserved.offset == 56
    assert ctypes.sizeof(moe.MoeDownDesc) == 32 and moe.MoeDownDesc.vec_dtype.offset == 24


def test_binding_refuses_before_the_library():
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        mx.moe_route(cpu, mx.Router(2))
    with pytest.raises(ValueError, match="2-D"):
        mx.moe_route(cpu[0], mx.Router(2))
    with pytest.raises(ValueError, match="GPU"):
        mx.moe_plan(torch.zeros(4, 2, dtype=torch.int32), 8)
    with pytest.raises(ValueError, match="topk"):
        mx.moe_plan(torch.zeros(4, dtype=torch.int32), 8)
    with pytest.raises(ValueError, match="2-D"):
        mx.moe_ffn(cpu[0], cpu, mx.Router(2), None, None, 32)
    with pytest.raises(ValueError, match="rot"):
        mx.moe_ffn(cpu, cpu, mx.Router(2), None, None, 32, rot="h64")
    with pytest.raises(ValueError, match="logits"):
        mx.moe_ffn(cpu, cpu[:2], mx.Router(2), None, None, 32)
    with pytest.raises(ValueError, match="experts, n, k"):
        mx.quantize_experts(cpu)
