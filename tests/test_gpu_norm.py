"""The fused norm against its formula in 64 bits, and its MXFP4 result against
the oracle's quantizer.

Tolerance of an fp32 result (u = 2^-24): every elementary fp32 operation is off
by at most u of its result (v_rsq_f32: 2u).  The residual sum r has at most 3
roundings of its two terms.  The mean square is a sum of non-negative terms
over chains of at most 64 + 20 additions, so its relative error is below 90u
and that of its inverse root below 47u; the mean (layer norm) is off by at most
90u * mean|r|.  A post-norm adds its own such error to p.  The modulation has
at most 4 more roundings of terms bounded by |y| + |bias (1 + scale)| + |shift|.
bf16 results: half a step more, 2^-8 of the value.
The MXFP4 result must equal the oracle's quantizer applied to the fp32 y, bit
for bit."""
import numpy as np
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32


def announce(*what):
    print("[case]", *what, flush=True)


def rand(gen, *shape, dtype=F, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=gen) * std + mean).to(dtype)


def reference(x, p, residual):
    """(y, r, bound of y, bound of r) in 64 bits, before the outputs' rounding."""
    f = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    x, residual = f(x), f(residual)
    rows, d = x.shape

    def stats(v, dv):
        """norm(v) and the bound of its error for v off by dv."""
        mu = v.mean(-1, keepdim=True) if p.kind == "layer" else torch.zeros(rows, 1, dtype=torch.float64)
        dmu = 90 * U * v.abs().mean(-1, keepdim=True) + dv.mean(-1, keepdim=True) if p.kind == "layer" else 0.0
        c = v - mu
        inv = torch.rsqrt((c * c).mean(-1, keepdim=True) + p.eps)
        z = c * inv
        dc = dv + dmu + U * c.abs()
        # the inverse root follows the centred values' relative change in norm
        rel = 47 * U + (dc.norm(dim=-1, keepdim=True) / c.norm(dim=-1, keepdim=True).clamp(min=1e-300))
        rel = torch.where(c.norm(dim=-1, keepdim=True) == 0, torch.full_like(rel, 47 * U), rel)
        return z, dc * inv + rel * z.abs() + U * z.abs()

    v, dv = x, torch.zeros_like(x)
    if p.post_norm:
        v, dv = stats(v, dv)
        if p.post_weight is not None:
            w = f(p.post_weight)
            v, dv = v * w, dv * w.abs() + U * (v * w).abs()
    grp = torch.arange(rows) // max(1, p.group_rows)
    if p.gate is not None:
        g = f(p.gate)[grp]
        v, dv = v * g, dv * g.abs() + U * (v * g).abs()
    if residual is not None:
        s = p.residual_scale * residual
        dv = dv + 3 * U * (v.abs() + s.abs())
        v = v + s
    r, dr = v, dv
    y, dy = stats(r, dr)
    mag = torch.zeros_like(y)
    if p.weight is not None:
        w = f(p.weight)
        y, dy = y * w, dy * w.abs()
    mag = mag + y.abs()
    if p.bias is not None:
        y = y + f(p.bias)
        mag = mag + f(p.bias).abs()
    if p.scale is not None:
        m = 1 + f(p.scale)[grp]
        y, dy, mag = y * m, dy * m.abs(), mag * (m.abs() + 2 * U)
    if p.shift is not None:
        y = y + f(p.shift)[grp]
        mag = mag + f(p.shift)[grp].abs()
    return y, r, dy + 4 * U * mag + 1e-37, dr + 1e-37


def check(got, want, bound, what):
    got = got.detach().cpu()
    step = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    err = (got.double() - want).abs()
    lim = bound + step * (want.abs() + bound)
    bad = ~(err <= lim)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / lim).max()):.3g} of the bound"


def build(gen, rows, d, kind, form, vdt):
    """A norm of one of the forms, its vectors on the device."""
    p = mx.Norm(kind=kind, eps=1e-5)
    vec = lambda mean: rand(gen, d, dtype=vdt, std=0.2, mean=mean).to(DEV)  # noqa: E731
    if form != "bare":
        p.weight = vec(1.0)
        if kind == "layer":
            p.bias = vec(0.0)
    if form in ("mod", "all"):
        p.group_rows = max(1, rows // 3)
        groups = -(-rows // p.group_rows)
        m = rand(gen, groups, 3 * d, dtype=vdt, std=0.3).to(DEV)    # slices of one tensor
        p.scale, p.shift, p.gate = m[:, :d], m[:, d:2 * d], m[:, 2 * d:]
    if form in ("post", "all"):
        p.post_norm, p.post_weight, p.residual_scale = True, vec(1.0), 0.75
    return p


SHAPES = [(1, 32), (1, 4096), (3, 96), (5, 8), (7, 1), (2, 37), (4, 1000), (13, 2048), (3, 2056), (2, 5120), (3, 8200),
          (2, 16384), (2, 16392), (1, 65536), (300, 160)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("form", ["bare", "weight", "mod", "post", "all"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_norm(rows, d, form, kind):
    i = SHAPES.index((rows, d))
    gen = torch.Generator().manual_seed(1000 * i + len(form) + (kind == "rms"))
    xdt, rdt, vdt = (BF, F)[i % 2], (F, BF)[i // 2 % 2], (BF, F)[i // 3 % 2]
    p = build(gen, rows, d, kind, form, vdt)
    x = rand(gen, rows, d, dtype=xdt, std=2.0, mean=0.5).to(DEV)
    residual = None if form == "bare" else rand(gen, rows, d, dtype=rdt, std=3.0).to(DEV)
    announce("norm", rows, d, kind, form, xdt, rdt, vdt)
    y, r = mx.norm(x, p, residual, out_dtype=F)
    yb, _ = mx.norm(x, p, residual, out_dtype=BF)
    torch.cuda.synchronize()
    want, wr, by, br = reference(x, p, residual)
    check(y, want, by, "y")
    check(yb, want, by, "y bf16")
    assert torch.equal(yb, y.to(BF))
    if form == "bare":
        assert r is None
    else:
        assert r.dtype == rdt
        check(r, wr, br, "r")


def rotations(d, gen):
    kr = lambda q: np.eye(q, dtype=np.float32) + 0.1 * torch.randn(q, q, generator=gen).numpy()  # noqa: E731
    out = [None, "h32", ("smooth", (0.5 + torch.rand(d, generator=gen)).numpy())]
    return out + [("kron", kr(q), kr(32 // q)) for q in (1, 2, 4, 8, 16, 32)]


def device_rot(rot):
    if rot is None or rot == "h32":
        return rot
    if rot[0] == "smooth":
        return mx.Smooth.from_host(rot[1], DEV)
    return mx.Kron.from_host(rot[1], rot[2], DEV)


@pytest.mark.parametrize("layout", [mx.ROWMAJOR, mx.TILED])
@pytest.mark.parametrize("rows,d", [(1, 128), (5, 384), (3, 96), (17, 2048), (260, 640), (2, 4224), (2, 16384),
                                    (1, 20480)])
def test_norm_quantize(rows, d, layout):
    if layout == mx.TILED and d % 128:
        pytest.skip("tiled needs d % 128 == 0")
    gen = torch.Generator().manual_seed(rows * 31 + d)
    x = rand(gen, rows, d, dtype=BF, std=2.0).to(DEV)
    residual = rand(gen, rows, d, dtype=BF, std=3.0).to(DEV)
    if rows > 2:
        x[1] = 0                                                    # a row that is zero throughout
        residual[1] = 0
    for rot in rotations(d, gen):
        if rot is not None and rot[0] == "kron" and d > 16384:
            continue
        for form, kind in (("weight", "rms"), ("mod", "layer")):
            p = build(gen, rows, d, kind, form, BF)
            announce("norm_quantize", rows, d, layout, rot if isinstance(rot, str) else rot and rot[0], form)
            y, r0 = mx.norm(x, p, residual, out_dtype=F)
            codes, scales, r = mx.norm_quantize(x, p, residual, device_rot(rot), layout)
            torch.cuda.synchronize()
            assert torch.equal(r, r0)
            got = (codes.cpu().numpy(), scales.cpu().numpy())
            if layout == mx.TILED:
                got = mx.untile_host(*got, rows)
            want = oracle.quantize(y.cpu().numpy(), rot=rot)
            assert np.array_equal(got[1], want[1]), "scales"
            assert np.array_equal(got[0], want[0]), "codes"


def test_strides_in_place_and_guard_columns():
    """Strided x, residual and outputs; residual_out the residual itself; the
    columns past d stay as they were."""
    gen = torch.Generator().manual_seed(5)
    for d, ld in ((200, 208), (201, 211), (96, 104)):
        rows = 9
        p = mx.Norm(kind="rms", weight=rand(gen, d, dtype=BF).to(DEV))
        xs = rand(gen, rows, ld, dtype=BF).to(DEV)
        rs = rand(gen, rows, ld, dtype=BF).to(DEV)
        ys = torch.full((rows, ld), 7.0, dtype=F, device=DEV)
        x, res, y = xs[:, :d], rs[:, :d], ys[:, :d]
        want, wr, by, br = reference(x, p, res)
        keep = rs[:, d:].clone()
        announce("strided norm", rows, d, ld)
        _, r = mx.norm(x, p, res, y=y, residual_out=res)
        torch.cuda.synchronize()
        assert r.data_ptr() == rs.data_ptr()
        check(y, want, by, "y")
        check(r, wr, br, "r")
        assert torch.equal(rs[:, d:], keep) and bool((ys[:, d:] == 7.0).all())


def test_empty_nan_and_extreme_rows():
    p = mx.Norm()
    x = torch.zeros(0, 64, dtype=BF, device=DEV)
    y, r = mx.norm(x, p)
    assert y.shape == (0, 64) and r is None
    x = torch.ones(5, 64, dtype=F, device=DEV)
    x[1, 3] = float("nan")
    x[2, 4] = float("inf")
    x[3] = 0
    x[4] = 1e-30
    announce("norm with NaN, infinity and zero rows")
    y, _ = mx.norm(x, p)
    torch.cuda.synchronize()
    assert torch.isfinite(y[[0, 3, 4]]).all()
    assert torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 4]) and bool((y[2, :4] == 0).all())       # 1 / infinity elsewhere
    assert bool((y[3] == 0).all())
    assert float((y[0] - 1).abs().max()) <= 1e-6


def test_more_rows_than_one_grid_holds():
    """64 threads a row: 2^26 rows pass the 2^32 threads of a launch."""
    rows, d, tail = (1 << 26) + 300, 32, 600
    x = torch.zeros(rows, d, dtype=BF, device=DEV)
    last = rand(torch.Generator().manual_seed(8), tail, d, dtype=BF, std=2.0)
    x[-tail:] = last.to(DEV)
    p = mx.Norm(kind="rms")
    announce("norm of 2^26 + 300 rows")
    y = torch.full((rows, d), 3.0, dtype=BF, device=DEV)
    mx.norm(x, p, y=y)
    codes, scales, _ = mx.norm_quantize(x, p, None, "h32")
    torch.cuda.synchronize()
    want, _, by, _ = reference(x[-tail:], p, None)
    check(y[-tail:], want, by, "y")
    assert float(y[:-tail].abs().amax()) == 0.0
    y32, _ = mx.norm(x[-tail:].contiguous(), p, out_dtype=F)
    wc, ws = mx.quantize_rotate(y32, "h32")
    assert torch.equal(codes[-tail:], wc) and torch.equal(scales[-tail:], ws)
