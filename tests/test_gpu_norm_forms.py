"""Forms of the fused norm beside those of test_gpu_norm.py, with its
references and bounds."""
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
from test_gpu_norm import BF, DEV, F, announce, check, rand, reference

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
