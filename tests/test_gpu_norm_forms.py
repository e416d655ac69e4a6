"""Forms of the fused norm beside those of test_gpu_norm.py, with its
references and bounds."""
import dataclasses

import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
from mxfp4_w4a4_quantized_amd import feedforward
from test_gpu_norm import BF, DEV, F, announce, build, check, rand, reference

pytestmark = pytest.mark.gpu


def test_one_row_views_of_any_stride():
    """Views of a single row (x, residual, outputs) and of a single group of
    vectors: their row stride leads nowhere, so an unaligned one is no reason to
    refuse them."""
    gen = torch.Generator().manual_seed(11)
    d = 96
    view = lambda dt: rand(gen, 1, 211, dtype=dt).to(DEV)[:, :d]  # noqa: E731
    x, residual, out = view(BF), view(BF), view(BF)
    vec = rand(gen, 1, 3 * d + 5, dtype=BF, std=0.3).to(DEV)
    p = mx.Norm(group_rows=1, scale=vec[:, :d], shift=vec[:, d:2 * d], gate=vec[:, 2 * d:3 * d])
    announce("norm of one-row views")
    y, r = mx.norm(x, p, residual, out_dtype=F, residual_out=out)
    codes, scales, r2 = mx.norm_quantize(x, p, residual)
    wc, ws = mx.quantize_rotate(y)
    torch.cuda.synchronize()
    want, wr, by, br = reference(x, p, residual)
    check(y, want, by, "y")
    check(r, wr, br, "r")
    assert torch.equal(r, r2) and torch.equal(codes, wc) and torch.equal(scales, ws)
    rows = rand(gen, 5, d, dtype=BF).to(DEV)
    p.group_rows = 5
    announce("norm of five rows with a one-group view")
    y, _ = mx.norm(rows, p, None, out_dtype=F)
    codes, scales, _ = mx.norm_quantize(rows, p, None)
    wc, ws = mx.quantize_rotate(y)
    torch.cuda.synchronize()
    check(y, *(reference(rows, p, None)[i] for i in (0, 2)), "y")
    assert torch.equal(codes, wc) and torch.equal(scales, ws)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("form", ["weight", "mod", "post", "all"])
@pytest.mark.parametrize("rows,d", [(600, 3072), (1100, 1000), (700, 5120), (3, 9000)])
def test_two_chunks_per_lane_with_bf16_vectors(rows, d, form, kind):
    """More than two rows a CU, or more than 8192 columns: 1024 columns a wave, the
    last step's bf16 vectors read ahead of the statistics."""
    gen = torch.Generator().manual_seed(rows + d + len(form))
    p = build(gen, rows, d, kind, form, BF)
    for xdt, rdt in ((BF, BF), (F, BF), (BF, F)):
        x = rand(gen, rows, d, dtype=xdt, std=2.0, mean=0.5).to(DEV)
        residual = rand(gen, rows, d, dtype=rdt, std=3.0).to(DEV)
        announce("norm", rows, d, kind, form, xdt, rdt)
        y, r = mx.norm(x, p, residual, out_dtype=F)
        yb, _ = mx.norm(x, p, residual, out_dtype=BF)
        torch.cuda.synchronize()
        want, wr, by, br = reference(x, p, residual)
        check(y, want, by, "y")
        check(r, wr, br, "r")
        assert torch.equal(yb, y.to(BF))


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_inputs_past_the_last_level_cache(kind):
    """Over 256 MiB of input: non-temporal loads and stores, with every operand,
    in place; sampled rows, the groups' first and last ones among them."""
    rows, d, group = 17001, 4096, 4000
    gen = torch.Generator(device=DEV).manual_seed(6)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=gen, device=DEV) * std).to(BF)  # noqa: E731
    x, before = rnd(rows, d, std=2.0), rnd(rows, d, std=3.0)
    vec = rnd(-(-rows // group), 3 * d, std=0.3)
    p = mx.Norm(kind=kind, eps=1e-5, weight=rnd(d), bias=rnd(d) if kind == "layer" else None, group_rows=group,
                scale=vec[:, :d], shift=vec[:, d:2 * d], gate=vec[:, 2 * d:], post_norm=True, post_weight=rnd(d),
                residual_scale=0.75)
    residual = before.clone()
    announce("norm past 256 MiB, in place", kind)
    y, r = mx.norm(x, p, residual, out_dtype=F, residual_out=residual)
    assert r.data_ptr() == residual.data_ptr()
    codes, scales, r2 = mx.norm_quantize(x, p, before, "h32", mx.TILED)
    wc, ws = mx.quantize_rotate(y, "h32", layout=mx.TILED)
    torch.cuda.synchronize()
    assert torch.equal(r, r2)
    # (the padding rows of the last tile are not written)
    got, want = (mx.untile_host(a.cpu().numpy(), b.cpu().numpy(), rows) for a, b in ((codes, scales), (wc, ws)))
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()
    edges = [i for g in range(0, rows, group) for i in (g, min(g + group, rows) - 1)]
    at = torch.tensor(sorted(set(edges + list(range(5, rows, 571)))))
    sub = dataclasses.replace(p, group_rows=1, scale=p.scale[at // group], shift=p.shift[at // group],
                              gate=p.gate[at // group])
    want, wr, by, br = reference(x[at.to(DEV)], sub, before[at.to(DEV)])
    check(y[at.to(DEV)], want, by, "y")
    check(r[at.to(DEV)], wr, br, "r")


@pytest.mark.parametrize("rows,d", [(5, 256), (9, 201), (700, 1024)])
def test_residual_out_is_x_itself(rows, d):
    gen = torch.Generator().manual_seed(d)
    for dt in (BF, F):
        p = build(gen, rows, d, "rms", "all", BF)
        first = rand(gen, rows, d, dtype=dt, std=2.0).to(DEV)
        residual = rand(gen, rows, d, dtype=dt, std=3.0).to(DEV)
        for res in (residual, None):
            x = first.clone()
            announce("norm with residual_out x itself", rows, d, dt, res is not None)
            y, r = mx.norm(x, p, res, out_dtype=F, residual_out=x)
            torch.cuda.synchronize()
            want, wr, by, br = reference(first, p, res)
            assert r.data_ptr() == x.data_ptr()
            check(y, want, by, "y")
            check(x, wr, br, "r")


@pytest.mark.parametrize("rows,d", [(1, 96), (9, 201), (700, 1024)])
def test_residual_alone(rows, d):
    """mxfp4_norm without y: the residual stream only."""
    gen = torch.Generator().manual_seed(d)
    p = build(gen, rows, d, "layer", "all", BF)
    x = rand(gen, rows, d, dtype=BF, std=2.0).to(DEV)
    residual = rand(gen, rows, d, dtype=F, std=3.0).to(DEV)
    desc, r, _ = feedforward._norm_desc(x, p, residual, None)
    announce("norm without y", rows, d)
    assert mx.lib().mxfp4_norm(desc, None, mx.MXFP4_F32, 0, torch.cuda.current_stream().cuda_stream) == mx.MXFP4_OK
    _, want = mx.norm(x, p, residual)
    torch.cuda.synchronize()
    _, wr, _, br = reference(x, p, residual)
    check(r, wr, br, "r")
    assert torch.equal(r, want)
