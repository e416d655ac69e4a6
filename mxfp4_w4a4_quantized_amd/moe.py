"""Mixture-of-experts operators over the same library:

  moe_route(logits, router)            experts and weights of each token
  moe_plan(ids, experts)               the (token, choice) pairs in expert order
  moe_up(a, plan, w_up, w_gate)        act(A G_e^T + bg) * (A U_e^T + bu) of every
                                       pair, or act(A U_e^T + bu) without a gate
  moe_up_requant(..., rot)             the same, requantized to MXFP4
  moe_down(h, plan, weights, w_down)   residual + sum over a token's choices of
                                       weight * (h D_e^T + b)
  moe_ffn(x, logits, router, w_up, w_down)
                                       quantize, route, plan, up projection to
                                       MXFP4, down projection and sum

Formulas, types and limits are those of include/mxfp4.h.  Experts' weights are
stacked tensors: codes [experts, rows, k/2], scales [experts, rows, k/32] with
rows = n (ROWMAJOR) or padded_rows(n) (TILED); quantize_experts makes them.
Inference only: results carry no gradient.
"""
import ctypes
import functools
from dataclasses import dataclass
from typing import Optional

import torch

from . import (HADAMARD32, ROWMAJOR, TILED, RotationDesc, _check, _out_shapes, lib, padded_rows, quantize_weight)
from .feedforward import (_H32, _act_code, _bad, _code, _dense_output, _gpu, _matrix, _packed, _packed_outputs,
                          _rotation, _stream)

SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}


class RouterDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("score", "topk", "groups", "topk_groups", "group_score", "renormalize")] +
                [("scale", ctypes.c_float), ("reserved", ctypes.c_int32), ("bias", ctypes.c_void_p)])


class MoeUpDesc(ctypes.Structure):
    _fields_ = ([("act", ctypes.c_int32), ("vec_dtype", ctypes.c_int32)] +
                [(n, ctypes.c_void_p) for n in ("u_codes", "u_scales", "g_codes", "g_scales", "bias_u", "bias_g")] +
                [("router_experts", ctypes.c_int32)])


class MoeDownDesc(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("vec_dtype", ctypes.c_int32), ("router_experts", ctypes.c_int32)]


for _desc in (MoeUpDesc, MoeDownDesc):
    _desc.reserved = _desc.router_experts   # the field's name while it had to be 0


def declare(L):
    """Argument types of the mixture-of-experts entry points."""
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    L.mxfp4_moe_route.argtypes = [vp, i32, i64, i64, i64, ctypes.POINTER(RouterDesc), vp, vp, vp]
    L.mxfp4_moe_plan_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(i64)]
    L.mxfp4_moe_plan.argtypes = [vp, i64, i64, i64, i64, vp, i64, vp]
    up = [vp, vp, vp, i64, i64, i64, ctypes.POINTER(MoeUpDesc), i64, i64, i32]
    L.mxfp4_moe_up.argtypes = up + [vp, i32, i64, vp]
    L.mxfp4_moe_up_requant.argtypes = up + [ctypes.POINTER(RotationDesc), vp, vp, i32, vp]
    L.mxfp4_moe_down_workspace.argtypes = [i64, i64, i64, i64, i64, i32, i32, ctypes.POINTER(i64)]
    L.mxfp4_moe_down.argtypes = [vp, vp, vp, i64, i64, i64, vp, ctypes.POINTER(MoeDownDesc), i64, i64, i32, vp, i32,
                                 i64, vp, i32, i64, vp, i64, vp]
    for f in (L.mxfp4_moe_route, L.mxfp4_moe_plan_bytes, L.mxfp4_moe_plan, L.mxfp4_moe_up, L.mxfp4_moe_up_requant,
              L.mxfp4_moe_down_workspace, L.mxfp4_moe_down):
        f.restype = i32


@dataclass
class Router:
    """How a token's experts are chosen from its logits: scores softmax or
    sigmoid; keys the logits, or scores + bias ([experts] fp32, for the choice
    only); with groups > 1 only the topk_groups best groups of consecutive experts
    ("max": by their largest key, "top2": by the sum of their two largest).
    Weights are the scores of the chosen, divided by their sum if renormalize,
    times scale."""
    topk: int
    score: str = "softmax"
    bias: Optional[torch.Tensor] = None
    groups: int = 1
    topk_groups: int = 1
    group_score: str = "max"
    renormalize: bool = True
    scale: float = 1.0


@dataclass(frozen=True, init=False)
class ExpertPlan:
    """The pairs (token * topk + choice) in expert order.  offsets [experts + 1]:
    first row of each expert, then the number of rows; order [tokens * topk]: pair
    of each row, -1 behind the last; slot [tokens * topk]: row of each pair, -1
    where its expert is not among these.  All int32, views of `words`.
    router_experts: those that the pairs are spread over, more than experts where
    other GPUs hold the rest.  Plans come from moe_plan; their sizes do not change."""
    words: torch.Tensor
    tokens: int
    topk: int
    experts: int
    router_experts: int

    def __init__(self, words, tokens, topk, experts, router_experts=None):
        # (a frozen dataclass's own constructor takes 0.4 us more, of a call of 7)
        self.__dict__.update(words=words, tokens=tokens, topk=topk, experts=experts,
                             router_experts=experts if router_experts is None else router_experts)

    @property
    def offsets(self):
        return self.words[:self.experts + 1]

    @property
    def order(self):
        return self.words[self.experts + 1:self.experts + 1 + self.tokens * self.topk]

    @property
    def slot(self):
        at = self.experts + 1 + self.tokens * self.topk
        return self.words[at:at + self.tokens * self.topk]


def _router_desc(r, experts, dev):
    if r.score not in SCORES:
        raise ValueError(f"unknown score {r.score!r} (one of {', '.join(SCORES)})")
    if r.group_score not in GROUP_SCORES:
        raise ValueError(f"unknown group score {r.group_score!r} (one of {', '.join(GROUP_SCORES)})")
    bias = None
    if r.bias is not None:
        if r.bias.get_device() != dev or r.bias.shape != (experts,) or not r.bias.is_contiguous():
            raise _bad("bias", r.bias, (experts,), dev)
        if r.bias.dtype != torch.float32:
            raise ValueError(f"bias is {r.bias.dtype}, expected torch.float32")
        bias = r.bias.data_ptr()
    return RouterDesc(SCORES[r.score], r.topk, r.groups, r.topk_groups, GROUP_SCORES[r.group_score],
                      1 if r.renormalize else 0, r.scale, 0, bias)


def _pairs(name, t, shape, dtype, dev):
    """Checks a dense [tokens, topk] tensor and gives its pointer."""
    if t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise _bad(name, t, shape, dev) if t.get_device() != dev or t.shape != shape else \
            ValueError(f"{name} must be contiguous")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    return t.data_ptr()


def moe_route(logits, r: Router, ids=None, weights=None):
    """(ids int32, weights fp32), both [tokens, topk]: the experts of each token,
    best first, -1 where no more can be chosen."""
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D with unit column stride")
    dev = _gpu(logits)
    tokens, experts = logits.shape
    ptr, ld = _matrix("logits", logits, logits.shape, dev)
    desc = _router_desc(r, experts, dev)
    if r.topk < 1:
        raise ValueError(f"topk must be at least 1, got {r.topk}")
    # (empty_strided and empty_like: 0.5 us less each than empty, of a call of 8)
    shape = (tokens, r.topk)
    if ids is None:
        ids = torch.empty_strided(shape, (r.topk, 1), dtype=torch.int32, device=logits.device)
        ip = ids.data_ptr()
    else:
        ip = _pairs("ids", ids, shape, torch.int32, dev)
    if weights is None:
        weights = torch.empty_like(ids, dtype=torch.float32)
        wp = weights.data_ptr()
    else:
        wp = _pairs("weights", weights, shape, torch.float32, dev)
    _check(lib().mxfp4_moe_route(ptr, _code(logits.dtype), tokens, experts, ld, desc, ip, wp, _stream(dev)),
           "mxfp4_moe_route")
    return ids, weights


@functools.lru_cache(maxsize=4096)
def _plan_words(tokens, topk, experts):
    """int32 words of a plan (a number of the sizes alone)."""
    n = ctypes.c_int64()
    _check(lib().mxfp4_moe_plan_bytes(tokens, topk, experts, ctypes.byref(n)), "mxfp4_moe_plan_bytes")
    return n.value // 4


def _plan_ptr(plan, dev):
    """Checks that a plan's words are as many as its sizes ask for: the products
    read tile tables, tokens and slots from them."""
    words = plan.words
    if words.get_device() != dev:
        raise _bad("the plan", words, words.shape, dev)
    need = _plan_words(plan.tokens, plan.topk, plan.experts)
    if words.numel() != need or words.dtype != torch.int32 or words.dim() != 1 or not words.is_contiguous():
        raise ValueError(f"a plan of {plan.tokens} tokens, {plan.topk} choices and {plan.experts} experts has {need} "
                         f"contiguous int32 words, got {words.dtype} {tuple(words.shape)}")
    return words.data_ptr()


def moe_plan(ids, experts: int, first: int = 0, plan: ExpertPlan = None, router_experts: int = None):
    """The plan for ids [tokens, topk] (int32) over the experts first .. first +
    experts - 1; other ids, -1 among them, have no row.  router_experts: how many
    the ids are from, where these are a part of them (the products then choose
    their kernels by the rows to expect).  `plan`: one of the same sizes, written
    again."""
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, topk]")
    dev = _gpu(ids)
    tokens, topk = ids.shape
    ip = _pairs("ids", ids, (tokens, topk), torch.int32, dev)
    if router_experts is not None and first + experts > router_experts:
        raise ValueError(f"experts {first} .. {first + experts - 1} are not among {router_experts}")
    if plan is None:
        words = torch.empty_strided((_plan_words(tokens, topk, experts),), (1,), dtype=torch.int32, device=ids.device)
        plan = ExpertPlan(words, tokens, topk, experts, router_experts)
        ptr = words.data_ptr()
    elif (plan.tokens, plan.topk, plan.experts) != (tokens, topk, experts) or plan.words.get_device() != dev or (
            router_experts is not None and router_experts != plan.router_experts):
        raise ValueError(f"the plan is for {plan.tokens} tokens, {plan.topk} choices and {plan.experts} of "
                         f"{plan.router_experts} experts on {plan.words.device}")
    else:
        ptr = _plan_ptr(plan, dev)
    _check(lib().mxfp4_moe_plan(ip, tokens, topk, first, experts, ptr, plan.words.numel() * 4, _stream(dev)),
           "mxfp4_moe_plan")
    return plan


def quantize_experts(w, rot=None, layout: int = ROWMAJOR, fit: bool = False):
    """(codes, scales) stacks of experts' weights w [experts, n, k], each as
    quantize_weight makes it."""
    if w.dim() != 3:
        raise ValueError("w must be [experts, n, k]")
    each = [quantize_weight(m, rot, layout=layout, fit=fit) for m in w]
    return torch.stack([c for c, _ in each]), torch.stack([s for _, s in each])


# What depends on the sizes of a call alone is worked out once for each of them: a
# small block's kernels take no longer than its Python.


@functools.lru_cache(maxsize=4096)
def _stack_shapes(experts, n, k, layout):
    cshape, sshape = _out_shapes(n, k, layout)
    return (experts, *cshape), (experts, *sshape)


def _stack(name, codes, scales, experts, n, k, layout, dev):
    """Checks stacked weights: (pointers)"""
    cshape, sshape = _stack_shapes(experts, n, k, layout)
    if (codes.shape != cshape or scales.shape != sshape or codes.get_device() != dev or scales.get_device() != dev or
            codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not codes.is_contiguous() or
            not scales.is_contiguous()):
        for t in (codes, scales):
            if t.get_device() != dev:
                raise _bad(f"{name} codes/scales", t, t.shape, dev)
        if codes.shape != cshape or scales.shape != sshape:
            raise ValueError(f"{name}: codes/scales must be {cshape} / {sshape}, got {tuple(codes.shape)} / "
                             f"{tuple(scales.shape)}")
        raise ValueError(f"{name}: codes and scales must be contiguous uint8 tensors")
    return codes.data_ptr(), scales.data_ptr()


def _expert_bias(name, t, experts, n, dtype, dev):
    """Checks [experts, n] biases and gives (pointer, dtype of the call's)."""
    if t.get_device() != dev or t.shape != (experts, n):
        raise _bad(name, t, (experts, n), dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype} (the vectors of a call share a dtype)")
    return t.data_ptr(), t.dtype


def _up_desc(act, w_up, w_gate, bias_up, bias_gate, experts, router_experts, n, k, layout, dev):
    uc, us = _stack("w_up", *w_up, experts, n, k, layout, dev)
    gc, gs = (None, None) if w_gate is None else _stack("w_gate", *w_gate, experts, n, k, layout, dev)
    bu, bg, dtype = None, None, None
    if bias_up is not None:
        bu, dtype = _expert_bias("bias_up", bias_up, experts, n, dtype, dev)
    if bias_gate is not None:
        if w_gate is None:
            raise ValueError("bias_gate needs w_gate")
        bg, dtype = _expert_bias("bias_gate", bias_gate, experts, n, dtype, dev)
    return MoeUpDesc(_act_code(act), 0 if dtype is None else _code(dtype), uc, us, gc, gs, bu, bg, router_experts)


def _width(codes, n):
    """Rows of one expert's weight: n, or all that the stack holds (TILED: the
    padding too)."""
    return codes.shape[1] if n is None else n


def moe_up(a_codes, a_scales, plan: ExpertPlan, w_up, w_gate=None, act="silu", bias_up=None, bias_gate=None,
           out_dtype=torch.bfloat16, y=None, layout: int = ROWMAJOR, n: int = None):
    """H [tokens * topk, n], row p for row p of the plan (rows behind its last are
    not written).  a: the tokens' packed activations; w_up, w_gate: (codes, scales)
    stacks; bias_up, bias_gate: [experts, n].  n: rows of one expert's weight, by
    default all that its stack holds (for TILED weights the padding too: give n
    where it is no multiple of 256)."""
    dev = _gpu(a_codes)
    n, k = _width(w_up[0], n), a_codes.shape[1] * 2
    ac, as_ = _packed("activations", a_codes, a_scales, plan.tokens, k, layout, dev)
    desc = _up_desc(act, w_up, w_gate, bias_up, bias_gate, plan.experts, plan.router_experts, n, k, layout, dev)
    y, ptr, ld, yt = _dense_output(y, plan.tokens * plan.topk, n, out_dtype, a_codes)
    _check(lib().mxfp4_moe_up(ac, as_, _plan_ptr(plan, dev), plan.tokens, plan.topk, plan.experts, desc, n, k, layout, ptr,
                              yt, ld, _stream(dev)), "mxfp4_moe_up")
    return y


def moe_up_requant(a_codes, a_scales, plan: ExpertPlan, w_up, w_gate=None, act="silu", bias_up=None, bias_gate=None,
                   rot=None, layout: int = ROWMAJOR, out_layout: int = ROWMAJOR, n: int = None, y_codes=None,
                   y_scales=None):
    """(codes, scales) of rot(H), H as moe_up gives it in fp32 (n as there); rot None
    or "h32"."""
    dev = _gpu(a_codes)
    n, k = _width(w_up[0], n), a_codes.shape[1] * 2
    ac, as_ = _packed("activations", a_codes, a_scales, plan.tokens, k, layout, dev)
    desc = _up_desc(act, w_up, w_gate, bias_up, bias_gate, plan.experts, plan.router_experts, n, k, layout, dev)
    rdesc, _keep = _rotation(rot, a_codes, n)
    y_codes, y_scales, yc, ys = _packed_outputs(plan.tokens * plan.topk, n, out_layout, y_codes, y_scales, a_codes)
    _check(lib().mxfp4_moe_up_requant(ac, as_, _plan_ptr(plan, dev), plan.tokens, plan.topk, plan.experts, desc, n, k,
                                      layout, rdesc, yc, ys, out_layout, _stream(dev)), "mxfp4_moe_up_requant")
    return y_codes, y_scales


@functools.lru_cache(maxsize=4096)
def _down_workspace(tokens, topk, router_experts, n, k, layout, yt, dev):
    """Bytes of the workspace on GPU dev (the current one)."""
    b = ctypes.c_int64()
    _check(lib().mxfp4_moe_down_workspace(tokens, topk, router_experts, n, k, layout, yt, ctypes.byref(b)),
           "mxfp4_moe_down_workspace")
    return b.value


def _residual(residual, shape, dev):
    """(pointer, dtype code, row stride) of a residual, or of none."""
    if residual is None:
        return None, 0, 0
    ptr, ld = _matrix("residual", residual, shape, dev)
    return ptr, _code(residual.dtype), ld


def moe_down(h_codes, h_scales, plan: ExpertPlan, weights, w_down, bias=None, residual=None, out_dtype=torch.bfloat16,
             y=None, layout: int = ROWMAJOR, n: int = None, workspace=None):
    """y [tokens, n] = residual + sum over a token's choices of weight * (h D_e^T +
    bias).  h: packed activations of tokens * topk rows, in the plan's order;
    weights: [tokens, topk] fp32; bias: [experts, n]; residual may be y itself; n as
    in moe_up; workspace: uint8, of moe_down_workspace bytes (a new one if not given).
    A bf16 y may come from products held in 11 bits each; an fp32 one never does."""
    dev = _gpu(h_codes)
    n, k = _width(w_down[0], n), h_codes.shape[1] * 2
    rows = plan.tokens * plan.topk
    hc, hs = _packed("hidden activations", h_codes, h_scales, rows, k, layout, dev)
    wp = _pairs("weights", weights, (plan.tokens, plan.topk), torch.float32, dev)
    dc, ds = _stack("w_down", *w_down, plan.experts, n, k, layout, dev)
    bp, bt = (None, None) if bias is None else _expert_bias("bias", bias, plan.experts, n, None, dev)
    desc = MoeDownDesc(dc, ds, bp, 0 if bt is None else _code(bt), plan.router_experts)
    res, rt, ld_r = _residual(residual, (plan.tokens, n), dev)
    y, ptr, ld, yt = _dense_output(y, plan.tokens, n, out_dtype, h_codes)
    need = _down_workspace(plan.tokens, plan.topk, plan.router_experts, n, k, layout, yt, dev)
    wsp, size = None, 0
    if workspace is None:
        if need > 0:
            workspace = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=h_codes.device)
            wsp, size = workspace.data_ptr(), need
    elif workspace.get_device() != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the operands' GPU")
    else:
        wsp, size = workspace.data_ptr(), workspace.numel()
    _check(lib().mxfp4_moe_down(hc, hs, _plan_ptr(plan, dev), plan.tokens, plan.topk, plan.experts, wp, desc, n, k, layout,
                                res, rt, ld_r, ptr, yt, ld, wsp, size, _stream(dev)),
           "mxfp4_moe_down")
    return y


def moe_down_workspace(plan: ExpertPlan, n: int, k: int, out_dtype=torch.bfloat16, layout: int = ROWMAJOR):
    """Bytes of moe_down's workspace for hidden activations of width k."""
    return _down_workspace(plan.tokens, plan.topk, plan.router_experts, n, k, layout, _code(out_dtype), _gpu(plan.words))


@functools.lru_cache(maxsize=4096)
def _ffn_work(tokens, topk, experts, router_experts, d, hidden, layout, yt, dev):
    """Offsets of what lies between moe_ffn's calls in its allocation (ids, weights,
    plan, codes and scales of x and of the hidden activations, workspace), the
    allocation's size, and the plan's and the workspace's."""
    rows = tokens * topk
    tp, rp = (padded_rows(tokens), padded_rows(rows)) if layout == TILED else (tokens, rows)
    plan = 4 * _plan_words(tokens, topk, experts)
    work = _down_workspace(tokens, topk, router_experts, d, hidden, layout, yt, dev)
    starts, total = [], 0
    for size in (rows * 4, rows * 4, plan, tp * d // 2, tp * d // 32, rp * hidden // 2, rp * hidden // 32, work):
        starts.append(total)
        total += (size + 255) // 256 * 256
    return tuple(starts), total, plan, work


def moe_ffn(x, logits, r: Router, w_up, w_down, hidden: int, w_gate=None, act="silu", rot=None, bias_up=None,
            bias_gate=None, bias_down=None, residual=None, first: int = 0, layout: int = ROWMAJOR, out_dtype=None, y=None):
    """A mixture-of-experts feed-forward block:
         ids, weights = moe_route(logits, r)
         a = MXFP4(rot(x))
         h = MXFP4(rot(act(a G_e^T + bg) * (a U_e^T + bu)))  for each pair (gated)
         y = residual + sum over a token's choices of weight * (h D_e^T + bd)
    x: [tokens, d] dense (the block's norm is done: the router's logits need it
    too); logits: [tokens, all experts]; w_up, w_gate ([hidden, d] each) and w_down
    ([d, hidden]): stacks over this GPU's experts, first .. first + experts - 1 of
    the logits' (the others add nothing here), quantized with the weight side of
    `rot` (None or "h32").  y: residual's type, or x's."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D with unit column stride")
    if rot is not None and rot != HADAMARD32:
        raise ValueError("rot must be None or \"h32\" (the transform is also that of the hidden activations)")
    if logits.dim() != 2 or logits.shape[0] != x.shape[0]:
        raise ValueError("logits must be [tokens, experts], with x's tokens")
    if r.topk < 1:
        raise ValueError(f"topk must be at least 1, got {r.topk}")
    experts = w_up[0].shape[0]
    if first < 0 or first + experts > logits.shape[1]:
        raise ValueError(f"experts {first} .. {first + experts - 1} of weights are not among the logits' {logits.shape[1]}")
    dev = _gpu(x)
    (tokens, d), topk = x.shape, r.topk
    # the calls of quantize_rotate, moe_route, moe_plan, moe_up_requant and
    # moe_down, with everything between them in one allocation and not checked again
    xp, ld_x = _matrix("x", x, x.shape, dev)
    lp, ld_l = _matrix("logits", logits, logits.shape, dev)
    router = _router_desc(r, logits.shape[1], dev)
    rdesc = None if rot is None else _H32
    up = _up_desc(act, w_up, w_gate, bias_up, bias_gate, experts, logits.shape[1], hidden, d, layout, dev)
    dc, ds = _stack("w_down", *w_down, experts, d, hidden, layout, dev)
    bp, bt = (None, None) if bias_down is None else _expert_bias("bias_down", bias_down, experts, d, None, dev)
    down = MoeDownDesc(dc, ds, bp, 0 if bt is None else _code(bt), logits.shape[1])
    res, rt, ld_r = _residual(residual, x.shape, dev)
    if out_dtype is None:
        out_dtype = x.dtype if residual is None else residual.dtype
    y, yp, ld_y, yt = _dense_output(y, tokens, d, out_dtype, x)
    if tokens == 0:
        return y
    starts, total, plan_size, work_size = _ffn_work(tokens, topk, experts, logits.shape[1], d, hidden, layout, yt, dev)
    work = torch.empty_strided((total,), (1,), dtype=torch.uint8, device=x.device)
    base = work.data_ptr()
    ids, weights, plan, ac, as_, hc, hs, ws = [base + at for at in starts]
    L, stream = lib(), _stream(dev)
    _check(L.mxfp4_moe_route(lp, _code(logits.dtype), tokens, logits.shape[1], ld_l, router, ids, weights, stream),
           "mxfp4_moe_route")
    _check(L.mxfp4_moe_plan(ids, tokens, topk, first, experts, plan, plan_size, stream), "mxfp4_moe_plan")
    _check(L.mxfp4_quantize_rotate(xp, _code(x.dtype), tokens, d, ld_x, rdesc, layout, ac, as_, stream),
           "mxfp4_quantize_rotate")
    _check(L.mxfp4_moe_up_requant(ac, as_, plan, tokens, topk, experts, up, hidden, d, layout, rdesc, hc, hs, layout,
                                  stream), "mxfp4_moe_up_requant")
    _check(L.mxfp4_moe_down(hc, hs, plan, tokens, topk, experts, weights, down, d, hidden, layout, res, rt, ld_r, yp, yt,
                            ld_y, ws, work_size, stream), "mxfp4_moe_down")
    return y
