"""Feed-forward operators around the MXFP4 GEMMs, over the same library:

  norm(x, p, residual)                 RMS / layer norm with the residual add,
                                       post-norm, gate and modulation around it
  norm_quantize(x, p, residual, rot)   the same, quantized to MXFP4
  gemm_epilogue(a, b, e)               Y = residual + gate * act(A B^T + bias)
  gemm_epilogue_requant(a, b, e, rot)  act(A B^T + bias) requantized to MXFP4
  gemm_glu(a, g, u, act)               H = act(A G^T + bg) * (A U^T + bu)
  gemm_glu_requant(a, g, u, act, rot)  the same, requantized to MXFP4
  ffn(x, p, residual, w_up, w_down)    norm -> (gated) up projection -> down
                                       projection + residual in three launches,
                                       MXFP4 activations in between

Formulas, types and limits are those of include/mxfp4.h.  Vectors (weight,
bias, gate, scale, shift) of one call share a dtype, fp32 or bf16.  Inference
only: results carry no gradient.
"""
import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import (ROWMAJOR, RotationDesc, _check, _dtype_code, _on_device, _out_shapes, _rot_desc, _stream, lib)

ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
NORM_KINDS = {"rms": 0, "layer": 1}


class NormDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("kind", "x_dtype", "r_dtype", "vec_dtype")] +
                [(n, ctypes.c_int64) for n in ("rows", "d")] +
                [("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("residual", ctypes.c_void_p),
                 ("ld_r", ctypes.c_int64), ("residual_out", ctypes.c_void_p), ("ld_ro", ctypes.c_int64)] +
                [(n, ctypes.c_void_p) for n in ("post_weight", "weight", "bias", "gate", "scale", "shift")] +
                [("ld_vec", ctypes.c_int64), ("group_rows", ctypes.c_int64), ("residual_scale", ctypes.c_float),
                 ("eps", ctypes.c_float), ("post_norm", ctypes.c_int32), ("reserved", ctypes.c_int32)])


class EpilogueDesc(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("vec_dtype", ctypes.c_int32), ("bias", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("ld_gate", ctypes.c_int64), ("group_rows", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("ld_res", ctypes.c_int64), ("res_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class GluDesc(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("vec_dtype", ctypes.c_int32), ("g_codes", ctypes.c_void_p),
                ("g_scales", ctypes.c_void_p), ("u_codes", ctypes.c_void_p), ("u_scales", ctypes.c_void_p),
                ("bias_g", ctypes.c_void_p), ("bias_u", ctypes.c_void_p), ("reserved", ctypes.c_int32)]


def declare(L):
    """Argument types of the feed-forward entry points."""
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    rot = ctypes.POINTER(RotationDesc)
    L.mxfp4_norm.argtypes = [ctypes.POINTER(NormDesc), vp, i32, i64, vp]
    L.mxfp4_norm_quantize.argtypes = [ctypes.POINTER(NormDesc), rot, i32, vp, vp, vp]
    operands = [vp, vp, i64, vp, vp, i64, i64, i32, ctypes.POINTER(EpilogueDesc)]
    L.mxfp4_gemm_epilogue.argtypes = operands + [vp, i32, i64, vp]
    L.mxfp4_gemm_epilogue_requant.argtypes = operands + [rot, vp, vp, i32, vp]
    operands = [vp, vp, i64, ctypes.POINTER(GluDesc), i64, i64, i32]
    L.mxfp4_gemm_glu.argtypes = operands + [vp, i32, i64, vp]
    L.mxfp4_gemm_glu_requant.argtypes = operands + [rot, vp, vp, i32, vp]
    for f in (L.mxfp4_norm, L.mxfp4_norm_quantize, L.mxfp4_gemm_epilogue, L.mxfp4_gemm_epilogue_requant,
              L.mxfp4_gemm_glu, L.mxfp4_gemm_glu_requant):
        f.restype = i32


@dataclass
class Norm:
    """A norm and what surrounds it: r = residual_scale * residual + gate[g] *
    ([norm](x) * post_weight); y = (norm(r) * weight + bias) * (1 + scale[g])
    + shift[g], with g = row // group_rows.  weight, bias, post_weight: [d];
    gate, scale, shift: [groups, d] with one common row stride."""
    kind: str = "rms"
    eps: float = 1e-6
    weight: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None
    scale: Optional[torch.Tensor] = None
    shift: Optional[torch.Tensor] = None
    gate: Optional[torch.Tensor] = None
    post_norm: bool = False
    post_weight: Optional[torch.Tensor] = None
    residual_scale: float = 1.0
    group_rows: int = 0


@dataclass
class Epilogue:
    """Y = residual + gate[g] * act(A B^T + bias), g = row // group_rows.
    bias: [n]; gate: [groups, n]; residual: [m, n], may be the output itself."""
    act: str = "none"
    bias: Optional[torch.Tensor] = None
    gate: Optional[torch.Tensor] = None
    group_rows: int = 0
    residual: Optional[torch.Tensor] = None


def _vec(name, t, shape, dtype, device):
    """Checks a vector (or [groups, d] tensor) and gives (pointer, dtype of the call's vectors)."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device} (all operands on one GPU)")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name} must have unit column stride")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype} (the vectors of a call share a dtype)")
    return t.data_ptr(), t.dtype


def _matrix(name, t, shape, device):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device} (all operands on one GPU)")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(1) != 1 and t.shape[1] != 1:
        raise ValueError(f"{name} must have unit column stride")


def _ld(t):
    """Row stride of a matrix (its width where it has one row)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _act_code(act):
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r} (one of {', '.join(ACTS)})")
    return ACTS[act]


def _groups(rows, group_rows, what):
    if group_rows < 1:
        raise ValueError(f"{what} needs group_rows >= 1, got {group_rows}")
    return -(-rows // group_rows)


def _norm_desc(x, p, residual, residual_out):
    if x.dim() != 2 or (x.stride(1) != 1 and x.shape[1] != 1):
        raise ValueError("x must be 2-D with unit column stride")
    if p.kind not in NORM_KINDS:
        raise ValueError(f"unknown norm {p.kind!r} (one of {', '.join(NORM_KINDS)})")
    if p.post_weight is not None and not p.post_norm:
        raise ValueError("post_weight needs post_norm")
    device = x.device
    _on_device(device)
    rows, d = x.shape
    d_ = NormDesc()
    d_.kind, d_.x_dtype, d_.rows, d_.d = NORM_KINDS[p.kind], _dtype_code(x.dtype), rows, d
    d_.x, d_.ld_x = x.data_ptr(), _ld(x)
    changed = residual is not None or p.gate is not None or p.post_norm or residual_out is not None
    if residual is not None:
        _matrix("residual", residual, x.shape, device)
        d_.residual, d_.ld_r = residual.data_ptr(), _ld(residual)
    if changed:
        if residual_out is None:
            residual_out = torch.empty_like(x if residual is None else residual, memory_format=torch.contiguous_format)
        else:
            _matrix("residual_out", residual_out, x.shape, device)
            if residual is not None and residual_out.dtype != residual.dtype:
                raise ValueError(f"residual_out is {residual_out.dtype}, residual {residual.dtype}")
        d_.residual_out, d_.ld_ro = residual_out.data_ptr(), _ld(residual_out)
        d_.r_dtype = _dtype_code(residual_out.dtype)
    dtype = None
    for name in ("post_weight", "weight", "bias"):
        t = getattr(p, name)
        if t is not None:
            ptr, dtype = _vec(name, t, (d,), dtype, device)
            setattr(d_, name, ptr)
    ld_vec = None
    for name in ("gate", "scale", "shift"):
        t = getattr(p, name)
        if t is not None:
            ptr, dtype = _vec(name, t, (_groups(rows, p.group_rows, name), d), dtype, device)
            setattr(d_, name, ptr)
            if ld_vec is not None and _ld(t) != ld_vec and t.shape[0] > 1:
                raise ValueError("gate, scale and shift must have the same row stride")
            ld_vec = _ld(t)
    if ld_vec is not None:
        d_.ld_vec, d_.group_rows = ld_vec, p.group_rows
    if dtype is not None:
        d_.vec_dtype = _dtype_code(dtype)
    d_.residual_scale, d_.eps, d_.post_norm = p.residual_scale, p.eps, int(p.post_norm)
    return d_, residual_out if changed else None


def norm(x, p: Norm, residual=None, out_dtype=None, y=None, residual_out=None):
    """Returns (y, r): the norm of r (dense, x's dtype by default) and the new
    residual stream r (residual's dtype; None where r is x itself).
    residual_out may be `residual`, which then holds r."""
    desc, r = _norm_desc(x, p, residual, residual_out)
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    else:
        _matrix("y", y, x.shape, x.device)
    _check(lib().mxfp4_norm(ctypes.byref(desc), y.data_ptr(), _dtype_code(y.dtype), _ld(y), _stream(x.device)),
           "mxfp4_norm")
    return y, r


def _packed_outputs(rows, k, layout, codes, scales, device):
    cshape, sshape = _out_shapes(rows, k, layout)
    if codes is None:
        codes = torch.empty(cshape, dtype=torch.uint8, device=device)
    if scales is None:
        scales = torch.empty(sshape, dtype=torch.uint8, device=device)
    _packed("output", codes, scales, cshape, sshape, device)
    return codes, scales


def _packed(name, codes, scales, cshape, sshape, device):
    for t, shape in ((codes, cshape), (scales, sshape)):
        if t.device != device:
            raise ValueError(f"{name} codes/scales are on {t.device}, expected {device} (all operands on one GPU)")
        if t.shape != shape:
            raise ValueError(f"{name} codes/scales must be {cshape} / {sshape}")
        if t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError(f"{name} codes and scales must be contiguous uint8 tensors")


def norm_quantize(x, p: Norm, residual=None, rot=None, layout: int = ROWMAJOR, codes=None, scales=None,
                  residual_out=None):
    """Returns (codes, scales, r): the norm quantized to MXFP4 in `layout`
    after the block transform `rot` (the bytes that quantize_rotate gives for
    the fp32 y of norm()), and r as norm() returns it."""
    desc, r = _norm_desc(x, p, residual, residual_out)
    rows, d = x.shape
    codes, scales = _packed_outputs(rows, d, layout, codes, scales, x.device)
    rdesc, _keep = _rot_desc(rot, x.device, d)
    _check(lib().mxfp4_norm_quantize(ctypes.byref(desc), ctypes.byref(rdesc) if rdesc is not None else None, layout,
                                     codes.data_ptr(), scales.data_ptr(), _stream(x.device)), "mxfp4_norm_quantize")
    return codes, scales, r


def _operand_sizes(a_codes, a_scales, weights, layout, m, n):
    """Checks the packed operands; gives (m, n, k).  For TILED operands pass
    the real row counts."""
    device = a_codes.device
    _on_device(device)
    k = a_codes.shape[1] * 2
    m = a_codes.shape[0] if m is None else m
    n = weights[0][0].shape[0] if n is None else n
    _packed("operand A:", a_codes, a_scales, *_out_shapes(m, k, layout), device)
    shapes = _out_shapes(n, k, layout)
    for c, s in weights:
        _packed("weight:", c, s, *shapes, device)
    return m, n, k


def _dense_output(y, m, n, out_dtype, device):
    if y is None:
        return torch.empty((m, n), dtype=out_dtype, device=device)
    _matrix("y", y, (m, n), device)
    return y


def _epilogue_desc(e, m, n, device):
    d = EpilogueDesc()
    if e is None:
        return d
    d.act = _act_code(e.act)
    dtype = None
    if e.bias is not None:
        d.bias, dtype = _vec("bias", e.bias, (n,), dtype, device)
    if e.gate is not None:
        d.gate, dtype = _vec("gate", e.gate, (_groups(m, e.group_rows, "gate"), n), dtype, device)
        d.ld_gate, d.group_rows = _ld(e.gate), e.group_rows
    if dtype is not None:
        d.vec_dtype = _dtype_code(dtype)
    if e.residual is not None:
        _matrix("residual", e.residual, (m, n), device)
        d.residual, d.ld_res, d.res_dtype = e.residual.data_ptr(), _ld(e.residual), _dtype_code(e.residual.dtype)
    return d


def gemm_epilogue(a_codes, a_scales, b_codes, b_scales, e: Epilogue = None, out_dtype=torch.bfloat16, y=None,
                  layout: int = ROWMAJOR, m: int = None, n: int = None):
    """Y = residual + gate * act(A B^T + bias) on packed MXFP4 operands, fp32
    throughout, rounded once to fp32 or bf16 Y [m, n]."""
    m, n, k = _operand_sizes(a_codes, a_scales, ((b_codes, b_scales),), layout, m, n)
    device = a_codes.device
    desc = _epilogue_desc(e, m, n, device)
    y = _dense_output(y, m, n, out_dtype, device)
    _check(lib().mxfp4_gemm_epilogue(a_codes.data_ptr(), a_scales.data_ptr(), m, b_codes.data_ptr(),
                                     b_scales.data_ptr(), n, k, layout, ctypes.byref(desc), y.data_ptr(),
                                     _dtype_code(y.dtype), _ld(y), _stream(device)), "mxfp4_gemm_epilogue")
    return y


def gemm_epilogue_requant(a_codes, a_scales, b_codes, b_scales, e: Epilogue = None, rot=None, layout: int = ROWMAJOR,
                          out_layout: int = ROWMAJOR, m: int = None, n: int = None, y_codes=None, y_scales=None):
    """(codes, scales) of rot(act(A B^T + bias)) in `out_layout`; rot None or "h32"."""
    m, n, k = _operand_sizes(a_codes, a_scales, ((b_codes, b_scales),), layout, m, n)
    device = a_codes.device
    desc = _epilogue_desc(e, m, n, device)
    rdesc, _keep = _rot_desc(rot, device, n)
    y_codes, y_scales = _packed_outputs(m, n, out_layout, y_codes, y_scales, device)
    _check(lib().mxfp4_gemm_epilogue_requant(
        a_codes.data_ptr(), a_scales.data_ptr(), m, b_codes.data_ptr(), b_scales.data_ptr(), n, k, layout,
        ctypes.byref(desc), ctypes.byref(rdesc) if rdesc is not None else None, y_codes.data_ptr(),
        y_scales.data_ptr(), out_layout, _stream(device)), "mxfp4_gemm_epilogue_requant")
    return y_codes, y_scales


def _glu_desc(act, g, u, bias_g, bias_u, n, device):
    d = GluDesc(act=_act_code(act), g_codes=g[0].data_ptr(), g_scales=g[1].data_ptr(), u_codes=u[0].data_ptr(),
                u_scales=u[1].data_ptr())
    dtype = None
    if bias_g is not None:
        d.bias_g, dtype = _vec("bias_g", bias_g, (n,), dtype, device)
    if bias_u is not None:
        d.bias_u, dtype = _vec("bias_u", bias_u, (n,), dtype, device)
    if dtype is not None:
        d.vec_dtype = _dtype_code(dtype)
    return d


def gemm_glu(a_codes, a_scales, g_codes, g_scales, u_codes, u_scales, act="silu", bias_g=None, bias_u=None,
             out_dtype=torch.bfloat16, y=None, layout: int = ROWMAJOR, m: int = None, n: int = None):
    """H = act(A G^T + bias_g) * (A U^T + bias_u) in one kernel: G and U the
    gate and up projections' packed weights, n rows each."""
    m, n, k = _operand_sizes(a_codes, a_scales, ((g_codes, g_scales), (u_codes, u_scales)), layout, m, n)
    device = a_codes.device
    desc = _glu_desc(act, (g_codes, g_scales), (u_codes, u_scales), bias_g, bias_u, n, device)
    y = _dense_output(y, m, n, out_dtype, device)
    _check(lib().mxfp4_gemm_glu(a_codes.data_ptr(), a_scales.data_ptr(), m, ctypes.byref(desc), n, k, layout,
                                y.data_ptr(), _dtype_code(y.dtype), _ld(y), _stream(device)), "mxfp4_gemm_glu")
    return y


def gemm_glu_requant(a_codes, a_scales, g_codes, g_scales, u_codes, u_scales, act="silu", bias_g=None, bias_u=None,
                     rot=None, layout: int = ROWMAJOR, out_layout: int = ROWMAJOR, m: int = None, n: int = None,
                     y_codes=None, y_scales=None):
    """(codes, scales) of rot(act(A G^T + bias_g) * (A U^T + bias_u)); rot None or "h32"."""
    m, n, k = _operand_sizes(a_codes, a_scales, ((g_codes, g_scales), (u_codes, u_scales)), layout, m, n)
    device = a_codes.device
    desc = _glu_desc(act, (g_codes, g_scales), (u_codes, u_scales), bias_g, bias_u, n, device)
    rdesc, _keep = _rot_desc(rot, device, n)
    y_codes, y_scales = _packed_outputs(m, n, out_layout, y_codes, y_scales, device)
    _check(lib().mxfp4_gemm_glu_requant(
        a_codes.data_ptr(), a_scales.data_ptr(), m, ctypes.byref(desc), n, k, layout,
        ctypes.byref(rdesc) if rdesc is not None else None, y_codes.data_ptr(), y_scales.data_ptr(), out_layout,
        _stream(device)), "mxfp4_gemm_glu_requant")
    return y_codes, y_scales


def ffn(x, p: Norm, residual, w_up, w_down, hidden: int, w_gate=None, act="silu", rot=None, gate=None, bias_up=None,
        bias_gate=None, bias_down=None, layout: int = ROWMAJOR, y=None):
    """A feed-forward block on the residual stream, three launches:
         codes, r = norm_quantize(x, p, residual, rot)
         h        = MXFP4(rot(act(codes W_gate^T) * (codes W_up^T)))   (gated)
                    MXFP4(rot(act(codes W_up^T)))                      (w_gate None)
         y        = r + gate[g] * (h W_down^T + bias_down)
    x, residual: [rows, d]; w_up, w_gate ([hidden, d]) and w_down ([d,
    hidden]): (codes, scales) in `layout`, quantized with the weight side of
    `rot` (None or "h32"); gate: [groups, d], by p.group_rows.  Returns (y, r),
    r the residual stream between the norm and the block (x where there is no
    residual add)."""
    rows, d = x.shape
    codes, scales, r = norm_quantize(x, p, residual, rot, layout)
    if w_gate is not None:
        h = gemm_glu_requant(codes, scales, *w_gate, *w_up, act=act, bias_g=bias_gate, bias_u=bias_up, rot=rot,
                             layout=layout, out_layout=layout, m=rows, n=hidden)
    else:
        h = gemm_epilogue_requant(codes, scales, *w_up, Epilogue(act=act, bias=bias_up), rot=rot, layout=layout,
                                  out_layout=layout, m=rows, n=hidden)
    r = x if r is None else r
    e = Epilogue(bias=bias_down, gate=gate, group_rows=p.group_rows, residual=r)
    return gemm_epilogue(*h, *w_down, e, out_dtype=r.dtype, y=y, layout=layout, m=rows, n=d), r
