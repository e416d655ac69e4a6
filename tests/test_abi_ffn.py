"""Refusals of the feed-forward entry points: synchronous status codes from the
library (the pointers are never dereferenced) and ValueErrors from the binding,
all without a GPU."""
import ctypes

import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
from mxfp4_w4a4_quantized_amd import feedforward as ff

A = 1 << 20          # arbitrary aligned address: never dereferenced
F, BF = mx.MXFP4_F32, mx.MXFP4_BF16
R, T = mx.ROWMAJOR, mx.TILED
INV, UNS, OK = mx.MXFP4_ERR_INVALID_ARG, mx.MXFP4_ERR_UNSUPPORTED, mx.MXFP4_OK


def ref(d):
    return ctypes.byref(d) if d is not None else None


def norm_args(**kw):
    d = dict(kind=0, x_dtype=BF, r_dtype=BF, vec_dtype=BF, rows=4, d=64, x=A, ld_x=64, residual_scale=1.0, eps=1e-6)
    d.update(kw)
    return ff.NormDesc(**d)


def norm(d, y=A, y_dtype=BF, ld_y=64):
    return mx.lib().mxfp4_norm(ref(d), y, y_dtype, ld_y, None)


def normq(d, rot=None, layout=R, codes=A, scales=A):
    return mx.lib().mxfp4_norm_quantize(ref(d), ref(rot), layout, codes, scales, None)


def test_norm_refusals():
    assert norm(None) == INV
    assert norm(norm_args(kind=2)) == INV
    for f in ("x_dtype", "r_dtype", "vec_dtype"):
        assert norm(norm_args(**{f: 7})) == INV
    assert norm(norm_args(), y_dtype=9) == INV
    assert norm(norm_args(rows=-1)) == INV
    assert norm(norm_args(d=0)) == INV
    assert norm(norm_args(ld_x=63)) == INV
    assert norm(norm_args(), ld_y=63) == INV
    assert norm(norm_args(x=None)) == INV
    assert norm(norm_args(residual=A, ld_r=32)) == INV
    assert norm(norm_args(residual_out=A, ld_ro=32)) == INV
    assert norm(norm_args(post_weight=A)) == INV                            # without post_norm
    assert norm(norm_args(gate=A, ld_vec=64, group_rows=0)) == INV
    assert norm(norm_args(scale=A, ld_vec=32, group_rows=1)) == INV
    assert norm(norm_args(eps=-1.0)) == INV
    assert norm(norm_args(eps=float("nan"))) == INV
    assert norm(norm_args(eps=float("inf"))) == INV
    assert norm(norm_args(reserved=1)) == INV
    assert norm(norm_args(), y=None) == INV                                 # no output at all
    assert norm(norm_args(x=A + 1)) == UNS
    assert norm(norm_args(weight=A + 1)) == UNS
    assert norm(norm_args(residual_out=A + 1, ld_ro=64)) == UNS
    assert norm(norm_args(), y=A + 1) == UNS
    assert norm(norm_args(d=65537, ld_x=65537), ld_y=65537) == UNS
    assert norm(norm_args(rows=1 << 30)) == UNS
    assert norm(norm_args(rows=0, x=None), y=None) == OK                     # nothing to do


def test_norm_quantize_refusals():
    assert normq(None) == INV
    assert normq(norm_args(), layout=2) == INV
    assert normq(norm_args(d=48, ld_x=64)) == INV                           # d % 32
    assert normq(norm_args(), layout=T) == INV                              # d % 128
    assert normq(norm_args(), codes=None) == INV
    assert normq(norm_args(), scales=None) == INV
    assert normq(norm_args(), codes=A + 8) == UNS
    assert normq(norm_args(d=128, ld_x=128), layout=T, scales=A + 2) == UNS
    assert normq(norm_args(x=A + 8)) == UNS                                 # the vector path only
    assert normq(norm_args(ld_x=68)) == UNS
    assert normq(norm_args(weight=A + 2)) == UNS
    bad = mx.RotationDesc(mx.ROT_KRON, 4, 4, 0, A, A)
    assert normq(norm_args(), rot=bad) == INV
    kr = mx.RotationDesc(mx.ROT_KRON, 4, 8, 0, A, A)
    assert normq(norm_args(d=16416, ld_x=16416), rot=kr) == UNS
    assert normq(norm_args(rows=1 << 29, d=128, ld_x=128)) == UNS           # 2^31 blocks
    assert normq(norm_args(rows=0, x=None), codes=None, scales=None) == OK


def gemm(m=4, n=8, k=64, layout=R, e=None, y=A, dt=F, ld=None, a=A, sa=A, b=A, sb=A):
    return mx.lib().mxfp4_gemm_epilogue(a, sa, m, b, sb, n, k, layout, ref(e), y, dt, n if ld is None else ld, None)


def gemmq(m=4, n=32, k=64, layout=R, e=None, rot=None, yc=A, ys=A, yl=R, a=A, sa=A, b=A, sb=A):
    return mx.lib().mxfp4_gemm_epilogue_requant(a, sa, m, b, sb, n, k, layout, ref(e), ref(rot), yc, ys, yl, None)


def glu(w, m=4, n=8, k=64, layout=R, y=A, dt=F, ld=None, a=A, sa=A):
    return mx.lib().mxfp4_gemm_glu(a, sa, m, ref(w), n, k, layout, y, dt, n if ld is None else ld, None)


def gluq(w, m=4, n=32, k=64, layout=R, rot=None, yc=A, ys=A, yl=R, a=A, sa=A):
    return mx.lib().mxfp4_gemm_glu_requant(a, sa, m, ref(w), n, k, layout, ref(rot), yc, ys, yl, None)


def weights(**kw):
    d = dict(g_codes=A, g_scales=A, u_codes=A, u_scales=A)
    d.update(kw)
    return ff.GluDesc(**d)


def test_gemm_epilogue_refusals():
    E = ff.EpilogueDesc
    assert gemm(dt=5) == INV and gemm(layout=3) == INV and gemm(k=48) == INV and gemm(k=0) == INV
    assert gemm(m=-1) == INV and gemm(n=-1, ld=8) == INV and gemm(ld=4) == INV and gemm(k=64, layout=T) == INV
    for p in ("a", "sa", "b", "sb", "y"):
        assert gemm(**{p: None}) == INV, p
    assert gemm(e=E(act=5)) == INV and gemm(e=E(act=-1)) == INV
    assert gemm(e=E(vec_dtype=2)) == INV and gemm(e=E(res_dtype=2)) == INV and gemm(e=E(reserved=1)) == INV
    assert gemm(e=E(gate=A, ld_gate=4, group_rows=1)) == INV
    assert gemm(e=E(gate=A, ld_gate=8, group_rows=0)) == INV
    assert gemm(e=E(residual=A, ld_res=4)) == INV
    assert gemm(e=E(bias=A + 2)) == UNS and gemm(e=E(vec_dtype=BF, bias=A + 1)) == UNS
    assert gemm(e=E(residual=A + 2, ld_res=8)) == UNS
    assert gemm(e=E(gate=A + 2, ld_gate=8, group_rows=1)) == UNS
    assert gemm(a=A + 4) == UNS and gemm(b=A + 8) == UNS and gemm(y=A + 2) == UNS
    assert gemm(k=128, layout=T, sb=A + 1) == UNS
    assert gemm(m=1 << 30) == UNS
    assert gemm(m=64 * 65536, k=96) == UNS                                  # past the grid
    assert gemm(m=0, a=None, y=None) == OK and gemm(n=0, ld=0, b=None, y=None) == OK


def test_gemm_epilogue_requant_refusals():
    E = ff.EpilogueDesc
    H = mx.RotationDesc(mx.ROT_HADAMARD32, 0, 0, 0, None, None)
    assert gemmq(yl=2) == INV and gemmq(layout=2) == INV and gemmq(k=48) == INV
    assert gemmq(yc=None) == INV and gemmq(ys=None, rot=H) == INV
    assert gemmq(e=E(act=9)) == INV
    assert gemmq(n=48) == UNS and gemmq(n=96, yl=T) == UNS
    assert gemmq(yc=A + 8) == UNS and gemmq(ys=A + 2) == UNS
    assert gemmq(e=E(gate=A, ld_gate=32, group_rows=1)) == UNS
    assert gemmq(e=E(residual=A, ld_res=32)) == UNS
    assert gemmq(rot=mx.RotationDesc(mx.ROT_SMOOTH, 0, 0, 0, A, None)) == UNS
    assert gemmq(rot=mx.RotationDesc(mx.ROT_KRON, 4, 8, 0, A, A)) == UNS
    assert gemmq(rot=mx.RotationDesc(9, 0, 0, 0, None, None)) == INV
    assert gemmq(m=0, yc=None) == OK


def test_gemm_glu_refusals():
    w = weights
    assert glu(None) == INV and gluq(None) == INV
    for f in ("g_codes", "g_scales", "u_codes", "u_scales"):
        assert glu(w(**{f: None})) == INV, f
        assert gluq(w(**{f: None})) == INV, f
    assert glu(w(act=7)) == INV and glu(w(vec_dtype=3)) == INV and glu(w(reserved=2)) == INV
    assert glu(w(), dt=4) == INV and glu(w(), k=48) == INV and glu(w(), ld=4) == INV and glu(w(), y=None) == INV
    assert glu(w(u_codes=A + 8)) == UNS and glu(w(bias_g=A + 2)) == UNS and glu(w(vec_dtype=BF, bias_u=A + 1)) == UNS
    assert glu(w(u_scales=A + 1), k=128, layout=T) == UNS
    assert gluq(w(), n=48) == UNS and gluq(w(), yl=T, n=32) == UNS and gluq(w(), ys=A + 1) == UNS
    assert gluq(w(), rot=mx.RotationDesc(mx.ROT_KRON, 4, 8, 0, A, A)) == UNS
    assert glu(w(), m=0, y=None) == OK and gluq(w(), n=0, yc=None) == OK


def test_descriptor_layouts_match_the_header():
    """ctypes mirrors of the C structs: the sizes a C compiler gives them."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [("mxfp4_norm_args", ff.NormDesc), ("mxfp4_epilogue", ff.EpilogueDesc), ("mxfp4_glu", ff.GluDesc)]
    code = '#include <stdio.h>\n#include <stddef.h>\n#include "mxfp4.h"\nint main(void) {\n'
    for name, d in fields:
        code += f'  printf("%zu", sizeof({name}));\n'
        for f, _ in d._fields_:
            code += f'  printf(" %zu", offsetof({name}, {f}));\n'
        code += '  printf("\\n");\n'
    code += "  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as t:
        src, exe = os.path.join(t, "s.c"), os.path.join(t, "s")
        open(src, "w").write(code)
        subprocess.run(["gcc", "-I" + os.path.join(root, "include"), src, "-o", exe], check=True)
        out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines()
    for line, (name, d) in zip(out, fields):
        want = [ctypes.sizeof(d)] + [getattr(d, f).offset for f, _ in d._fields_]
        assert [int(v) for v in line.split()] == want, name


def test_binding_refuses_host_tensors_and_bad_names():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mx.norm(x, mx.Norm())
    with pytest.raises(ValueError):
        mx.norm_quantize(x, mx.Norm())
    with pytest.raises(ValueError):
        mx.norm(x, mx.Norm(kind="batch"))
    with pytest.raises(ValueError):
        mx.norm(x, mx.Norm(post_weight=x[0]))
    with pytest.raises(ValueError):
        mx.norm(x[0], mx.Norm())
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mx.gemm_epilogue(c, s, c, s)
    with pytest.raises(ValueError):
        mx.gemm_glu(c, s, c, s, c, s)
    with pytest.raises(ValueError):
        ff._act_code("swish")
