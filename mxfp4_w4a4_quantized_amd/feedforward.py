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

from . import (HADAMARD32, MXFP4_BF16, MXFP4_F32, ROT_HADAMARD32, ROWMAJOR, TILED, RotationDesc, _check,
               _out_shapes, _rot_desc, lib, padded_rows)

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


# The hipStream_t of a GPU's current stream.  torch.cuda.current_stream(dev)
# .cuda_stream gives the same through a Stream object, which costs 1.7 us more
# on each call.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _stream(dev):
    """The current stream of GPU dev.  The handle of a default stream is 0 for
    every GPU, and a launch on it goes to the current one."""
    stream = _raw_stream(dev)
    if stream == 0 and _current_device() != dev:
        raise ValueError(f"the operands are on GPU {dev}, whose default stream needs it as the current device "
                         f"(torch.cuda.device({dev}))")
    return stream


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


# The checks below run on every call of a decode step, whose kernels take a few
# microseconds: they use the cheap tensor accessors (get_device, stride) and
# fill each descriptor with one constructor call.


def _bad(name, t, shape, dev):
    """Why tensor t was refused."""
    if t.get_device() != dev:
        where = "the host" if t.get_device() < 0 else f"GPU {t.get_device()}"
        return ValueError(f"{name} is on {where}, expected GPU {dev} (all operands on one GPU)")
    if t.shape != shape:
        return ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return ValueError(f"{name} must have unit column stride")


def _vec(name, t, shape, dtype, dev):
    """Checks a vector and gives (pointer, dtype of the call's vectors)."""
    if t.get_device() != dev or t.shape != shape or (t.stride() != (1,) and shape[0] != 1):
        raise _bad(name, t, shape, dev)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype} (the vectors of a call share a dtype)")
    return t.data_ptr(), t.dtype


def _matrix(name, t, shape, dev):
    """Checks a dense matrix and gives (pointer, row stride: its width where
    it has one row)."""
    if t.get_device() != dev or t.shape != shape:
        raise _bad(name, t, shape, dev)
    ld, col = t.stride()
    rows, cols = shape
    if col != 1 and cols != 1:
        raise _bad(name, t, shape, dev)
    return t.data_ptr(), ld if rows > 1 else cols


def _grouped(name, t, shape, dtype, dev):
    """Checks a [groups, d] tensor of vectors: (pointer, dtype, row stride)."""
    ptr, ld = _matrix(name, t, shape, dev)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype} (the vectors of a call share a dtype)")
    return ptr, t.dtype, ld


# Layout of a result like x: by itself empty_like takes over the row stride of a
# view of one row.
_ROWS = torch.contiguous_format
_CODES = {torch.float32: MXFP4_F32, torch.bfloat16: MXFP4_BF16}


def _code(dtype):
    if dtype not in _CODES:
        raise ValueError(f"unsupported dtype {dtype}")
    return _CODES[dtype]


def _gpu(t):
    """The GPU that a call's first operand is on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"tensors must be on a GPU, got {t.device}")
    return dev


def _act_code(act):
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r} (one of {', '.join(ACTS)})")
    return ACTS[act]


def _groups(rows, group_rows, what):
    if group_rows < 1:
        raise ValueError(f"{what} needs group_rows >= 1, got {group_rows}")
    return -(-rows // group_rows)


def _norm_desc(x, p, residual, residual_out):
    """(descriptor, residual_out or the new tensor for it, GPU)"""
    if x.dim() != 2:
        raise ValueError("x must be 2-D with unit column stride")
    if p.kind not in NORM_KINDS:
        raise ValueError(f"unknown norm {p.kind!r} (one of {', '.join(NORM_KINDS)})")
    if p.post_weight is not None and not p.post_norm:
        raise ValueError("post_weight needs post_norm")
    dev = _gpu(x)
    shape = x.shape
    rows, d = shape
    xp, ld_x = _matrix("x", x, shape, dev)
    res, ld_r, out, ld_ro, rt = None, 0, None, 0, 0
    if residual is not None:
        res, ld_r = _matrix("residual", residual, shape, dev)
    if residual is not None or residual_out is not None or p.gate is not None or p.post_norm:
        like = x if residual is None else residual
        if residual_out is None:
            residual_out = torch.empty_like(like, memory_format=_ROWS)
        elif residual is not None and residual_out.dtype != residual.dtype:
            raise ValueError(f"residual_out is {residual_out.dtype}, residual {residual.dtype}")
        out, ld_ro = _matrix("residual_out", residual_out, shape, dev)
        rt = _code(residual_out.dtype)
    dtype, post, weight, bias, gate, scale, shift, ld_vec = None, None, None, None, None, None, None, 0
    if p.post_weight is not None:
        post, dtype = _vec("post_weight", p.post_weight, (d,), dtype, dev)
    if p.weight is not None:
        weight, dtype = _vec("weight", p.weight, (d,), dtype, dev)
    if p.bias is not None:
        bias, dtype = _vec("bias", p.bias, (d,), dtype, dev)
    if p.gate is not None or p.scale is not None or p.shift is not None:
        vshape = (_groups(rows, p.group_rows, "a grouped vector"), d)
        lds = set()
        if p.gate is not None:
            gate, dtype, ld = _grouped("gate", p.gate, vshape, dtype, dev)
            lds.add(ld)
        if p.scale is not None:
            scale, dtype, ld = _grouped("scale", p.scale, vshape, dtype, dev)
            lds.add(ld)
        if p.shift is not None:
            shift, dtype, ld = _grouped("shift", p.shift, vshape, dtype, dev)
            lds.add(ld)
        if len(lds) > 1 and vshape[0] > 1:
            raise ValueError("gate, scale and shift must have the same row stride")
        ld_vec = max(lds)
    desc = NormDesc(NORM_KINDS[p.kind], _code(x.dtype), rt, 0 if dtype is None else _code(dtype), rows, d, xp, ld_x,
                    res, ld_r, out, ld_ro, post, weight, bias, gate, scale, shift, ld_vec, p.group_rows,
                    p.residual_scale, p.eps, 1 if p.post_norm else 0, 0)
    return desc, residual_out, dev


def norm(x, p: Norm, residual=None, out_dtype=None, y=None, residual_out=None):
    """Returns (y, r): the norm of r (dense, x's dtype by default) and the new
    residual stream r (residual's dtype; None where r is x itself).
    residual_out may be `residual`, which then holds r."""
    desc, r, dev = _norm_desc(x, p, residual, residual_out)
    if y is None:
        y = torch.empty_like(x, dtype=out_dtype, memory_format=_ROWS)
    ptr, ld = _matrix("y", y, x.shape, dev)
    _check(lib().mxfp4_norm(desc, ptr, _code(y.dtype), ld, _stream(dev)), "mxfp4_norm")
    return y, r


def _packed(name, codes, scales, rows, k, layout, dev):
    """Checks packed codes and scales of [rows, k] in `layout`: (pointers)"""
    cshape, sshape = _out_shapes(rows, k, layout)
    if (codes.shape != cshape or scales.shape != sshape or codes.get_device() != dev or scales.get_device() != dev or
            codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not codes.is_contiguous() or
            not scales.is_contiguous()):
        for t in (codes, scales):
            if t.get_device() != dev:
                raise _bad(f"{name} codes/scales", t, t.shape, dev)
        if codes.shape != cshape or scales.shape != sshape:
            raise ValueError(f"{name}: codes/scales must be {cshape} / {sshape}")
        raise ValueError(f"{name}: codes and scales must be contiguous uint8 tensors")
    return codes.data_ptr(), scales.data_ptr()


def _packed_outputs(rows, k, layout, codes, scales, like):
    """Codes and scales for a packed result (new ones beside tensor `like`
    where not given) and their pointers."""
    if codes is None or scales is None:
        cshape, sshape = _out_shapes(rows, k, layout)
        new = codes is None and scales is None
        if codes is None:
            codes = torch.empty(cshape, dtype=torch.uint8, device=like.device)
        if scales is None:
            scales = torch.empty(sshape, dtype=torch.uint8, device=like.device)
        if new:
            return codes, scales, codes.data_ptr(), scales.data_ptr()
    return codes, scales, *_packed("output", codes, scales, rows, k, layout, like.get_device())


def norm_quantize(x, p: Norm, residual=None, rot=None, layout: int = ROWMAJOR, codes=None, scales=None,
                  residual_out=None):
    """Returns (codes, scales, r): the norm quantized to MXFP4 in `layout`
    after the block transform `rot` (the bytes that quantize_rotate gives for
    the fp32 y of norm()), and r as norm() returns it."""
    desc, r, dev = _norm_desc(x, p, residual, residual_out)
    rows, d = x.shape
    codes, scales, cp, sp = _packed_outputs(rows, d, layout, codes, scales, x)
    rdesc, _keep = _rotation(rot, x, d)
    _check(lib().mxfp4_norm_quantize(desc, rdesc, layout, cp, sp, _stream(dev)), "mxfp4_norm_quantize")
    return codes, scales, r


_H32 = RotationDesc(ROT_HADAMARD32, 0, 0, 0, None, None)


def _rotation(rot, like, k):
    """Rotation descriptor and the factor tensors it points to."""
    if rot is None:
        return None, ()
    return (_H32, ()) if rot == HADAMARD32 else _rot_desc(rot, like.device, k)


def _sizes(a_codes, b_codes, m, n):
    """(m, n, k): for TILED operands the caller passes the real row counts."""
    return (a_codes.shape[0] if m is None else m, b_codes.shape[0] if n is None else n, a_codes.shape[1] * 2)


def _dense_output(y, m, n, out_dtype, like):
    """(y, its pointer, its row stride, its dtype code)"""
    if y is None:
        y = torch.empty((m, n), dtype=out_dtype, device=like.device)
        return y, y.data_ptr(), n, _code(out_dtype)
    ptr, ld = _matrix("y", y, (m, n), like.get_device())
    return y, ptr, ld, _code(y.dtype)


def _epilogue_desc(e, m, n, dev):
    if e is None:
        return None
    bias, gate, ld_gate, res, ld_res, rt, dtype = None, None, 0, None, 0, 0, None
    if e.bias is not None:
        bias, dtype = _vec("bias", e.bias, (n,), dtype, dev)
    if e.gate is not None:
        gate, dtype, ld_gate = _grouped("gate", e.gate, (_groups(m, e.group_rows, "gate"), n), dtype, dev)
    if e.residual is not None:
        res, ld_res = _matrix("residual", e.residual, (m, n), dev)
        rt = _code(e.residual.dtype)
    return EpilogueDesc(_act_code(e.act), 0 if dtype is None else _code(dtype), bias, gate, ld_gate,
                        e.group_rows, res, ld_res, rt, 0)


def gemm_epilogue(a_codes, a_scales, b_codes, b_scales, e: Epilogue = None, out_dtype=torch.bfloat16, y=None,
                  layout: int = ROWMAJOR, m: int = None, n: int = None):
    """Y = residual + gate * act(A B^T + bias) on packed MXFP4 operands, fp32
    throughout, rounded once to fp32 or bf16 Y [m, n]."""
    dev = _gpu(a_codes)
    m, n, k = _sizes(a_codes, b_codes, m, n)
    ac, as_ = _packed("operand A", a_codes, a_scales, m, k, layout, dev)
    bc, bs = _packed("operand B", b_codes, b_scales, n, k, layout, dev)
    desc = _epilogue_desc(e, m, n, dev)
    y, ptr, ld, yt = _dense_output(y, m, n, out_dtype, a_codes)
    _check(lib().mxfp4_gemm_epilogue(ac, as_, m, bc, bs, n, k, layout, desc, ptr, yt, ld, _stream(dev)),
           "mxfp4_gemm_epilogue")
    return y


def gemm_epilogue_requant(a_codes, a_scales, b_codes, b_scales, e: Epilogue = None, rot=None, layout: int = ROWMAJOR,
                          out_layout: int = ROWMAJOR, m: int = None, n: int = None, y_codes=None, y_scales=None):
    """(codes, scales) of rot(act(A B^T + bias)) in `out_layout`; rot None or "h32"."""
    dev = _gpu(a_codes)
    m, n, k = _sizes(a_codes, b_codes, m, n)
    ac, as_ = _packed("operand A", a_codes, a_scales, m, k, layout, dev)
    bc, bs = _packed("operand B", b_codes, b_scales, n, k, layout, dev)
    desc = _epilogue_desc(e, m, n, dev)
    rdesc, _keep = _rotation(rot, a_codes, n)
    y_codes, y_scales, yc, ys = _packed_outputs(m, n, out_layout, y_codes, y_scales, a_codes)
    _check(lib().mxfp4_gemm_epilogue_requant(ac, as_, m, bc, bs, n, k, layout, desc, rdesc, yc, ys, out_layout,
                                             _stream(dev)), "mxfp4_gemm_epilogue_requant")
    return y_codes, y_scales


def _glu_desc(act, g_codes, g_scales, u_codes, u_scales, bias_g, bias_u, n, k, layout, dev):
    gc, gs = _packed("weight G", g_codes, g_scales, n, k, layout, dev)
    uc, us = _packed("weight U", u_codes, u_scales, n, k, layout, dev)
    bg, bu, dtype = None, None, None
    if bias_g is not None:
        bg, dtype = _vec("bias_g", bias_g, (n,), dtype, dev)
    if bias_u is not None:
        bu, dtype = _vec("bias_u", bias_u, (n,), dtype, dev)
    return GluDesc(_act_code(act), 0 if dtype is None else _code(dtype), gc, gs, uc, us, bg, bu, 0)


def gemm_glu(a_codes, a_scales, g_codes, g_scales, u_codes, u_scales, act="silu", bias_g=None, bias_u=None,
             out_dtype=torch.bfloat16, y=None, layout: int = ROWMAJOR, m: int = None, n: int = None):
    """H = act(A G^T + bias_g) * (A U^T + bias_u) in one kernel: G and U the
    gate and up projections' packed weights, n rows each."""
    dev = _gpu(a_codes)
    m, n, k = _sizes(a_codes, g_codes, m, n)
    ac, as_ = _packed("operand A", a_codes, a_scales, m, k, layout, dev)
    desc = _glu_desc(act, g_codes, g_scales, u_codes, u_scales, bias_g, bias_u, n, k, layout, dev)
    y, ptr, ld, yt = _dense_output(y, m, n, out_dtype, a_codes)
    _check(lib().mxfp4_gemm_glu(ac, as_, m, desc, n, k, layout, ptr, yt, ld, _stream(dev)), "mxfp4_gemm_glu")
    return y


def gemm_glu_requant(a_codes, a_scales, g_codes, g_scales, u_codes, u_scales, act="silu", bias_g=None, bias_u=None,
                     rot=None, layout: int = ROWMAJOR, out_layout: int = ROWMAJOR, m: int = None, n: int = None,
                     y_codes=None, y_scales=None):
    """(codes, scales) of rot(act(A G^T + bias_g) * (A U^T + bias_u)); rot None or "h32"."""
    dev = _gpu(a_codes)
    m, n, k = _sizes(a_codes, g_codes, m, n)
    ac, as_ = _packed("operand A", a_codes, a_scales, m, k, layout, dev)
    desc = _glu_desc(act, g_codes, g_scales, u_codes, u_scales, bias_g, bias_u, n, k, layout, dev)
    rdesc, _keep = _rotation(rot, a_codes, n)
    y_codes, y_scales, yc, ys = _packed_outputs(m, n, out_layout, y_codes, y_scales, a_codes)
    _check(lib().mxfp4_gemm_glu_requant(ac, as_, m, desc, n, k, layout, rdesc, yc, ys, out_layout, _stream(dev)),
           "mxfp4_gemm_glu_requant")
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
    # the calls of norm_quantize, gemm_glu_requant / gemm_epilogue_requant and
    # gemm_epilogue, with the intermediates in one allocation and not checked
    # again: a decode step's kernels take 30 us, as long as the three bindings
    desc, r, dev = _norm_desc(x, p, residual, None)
    rows, d = x.shape
    r = x if r is None else r
    if rot is not None and rot != HADAMARD32:
        raise ValueError("rot must be None or \"h32\" (the transform is also that of the hidden activations)")
    rdesc = None if rot is None else _H32
    down = _packed("w_down", *w_down, d, hidden, layout, dev)
    if w_gate is not None:
        glu = _glu_desc(act, *w_gate, *w_up, bias_gate, bias_up, hidden, d, layout, dev)
    else:
        if bias_gate is not None:
            raise ValueError("bias_gate needs w_gate")
        up = _packed("w_up", *w_up, hidden, d, layout, dev)
        e_up = _epilogue_desc(Epilogue(act=act, bias=bias_up), rows, hidden, dev)
    e_down = _epilogue_desc(Epilogue(bias=bias_down, gate=gate, group_rows=p.group_rows, residual=r), rows, d, dev)
    y, yp, ld, yt = _dense_output(y, rows, d, r.dtype, x)
    if rows == 0:
        return y, r
    rp = padded_rows(rows) if layout == TILED else rows
    sizes = [rp * d // 2, rp * d // 32, rp * hidden // 2, rp * hidden // 32]
    starts, total = [], 0
    for size in sizes:
        starts.append(total)
        total += (size + 255) // 256 * 256
    work = torch.empty(total, dtype=torch.uint8, device=x.device)
    base = work.data_ptr()
    xc, xs, hc, hs = (base + at for at in starts)
    L, stream = lib(), _stream(dev)
    _check(L.mxfp4_norm_quantize(desc, rdesc, layout, xc, xs, stream), "mxfp4_norm_quantize")
    if w_gate is not None:
        _check(L.mxfp4_gemm_glu_requant(xc, xs, rows, glu, hidden, d, layout, rdesc, hc, hs, layout, stream),
               "mxfp4_gemm_glu_requant")
    else:
        _check(L.mxfp4_gemm_epilogue_requant(xc, xs, rows, *up, hidden, d, layout, e_up, rdesc, hc, hs, layout, stream),
               "mxfp4_gemm_epilogue_requant")
    _check(L.mxfp4_gemm_epilogue(hc, hs, rows, *down, d, hidden, layout, e_down, yp, yt, ld, stream),
           "mxfp4_gemm_epilogue")
    return y, r
