"""The fused norm at the ends of the fp32 range: rows whose mean square
underflows, is subnormal or overflows, with eps = 0 or a subnormal eps.  The
formula does not depend on a row's magnitude there, so neither does the bound:
it is that of test_gpu_norm.py."""
import dataclasses

import numpy as np
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
import oracle
from test_gpu_norm import BF, DEV, F, announce, check, rand, reference

pytestmark = pytest.mark.gpu

# row magnitudes: mean squares that are subnormal, 0, ordinary and infinite in fp32
MAGS = [1e-20, 1.0, 1e-23, 2.0 ** -126, 2.0 ** -140, 1e-15, 3e19, 1e25]


def against_formula(y, x, p, what):
    """y against the formula: NaN where it is 0 / 0 (a row that rounds to zeros,
    eps = 0), the bound elsewhere.  eps is fp32 in the interface."""
    want, _, bound, _ = reference(x, dataclasses.replace(p, eps=float(np.float32(p.eps))), None)
    undefined = torch.isnan(want)
    assert torch.equal(torch.isnan(y.cpu()), undefined), what
    check(torch.where(undefined, 0.0, y.cpu()), torch.where(undefined, 0.0, want), torch.where(undefined, 0.0, bound), what)


def rows_of(gen, d, dtype):
    x = rand(gen, len(MAGS), d, std=1.0, mean=0.5) * torch.tensor(MAGS, dtype=torch.float64)[:, None]
    return x.to(dtype).to(DEV)


@pytest.mark.parametrize("eps", [0.0, 1e-42])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("d", [64, 1000, 1001, 4096, 8200, 20000])
def test_rows_of_any_magnitude(d, dtype, kind, eps):
    gen = torch.Generator().manual_seed(d)
    x = rows_of(gen, d, dtype)
    for post in (False, True):
        p = mx.Norm(kind=kind, eps=eps, post_norm=post)
        announce("norm, rows of any magnitude", d, dtype, kind, eps, post)
        y, _ = mx.norm(x, p, out_dtype=F)
        torch.cuda.synchronize()
        against_formula(y, x, p, f"{kind} post={post}")


def test_many_rows_take_two_chunks_per_lane():
    gen = torch.Generator().manual_seed(3)
    d, rows = 1024, 1100
    x = rand(gen, rows, d) * torch.tensor(MAGS, dtype=torch.float64).repeat(rows)[:rows, None]
    x = x.float().to(DEV)
    p = mx.Norm(kind="layer", eps=0.0, weight=torch.ones(d, dtype=BF, device=DEV))
    announce("norm, 1100 rows of any magnitude")
    y, _ = mx.norm(x, p, out_dtype=F)
    torch.cuda.synchronize()
    against_formula(y, x, p, "y")


@pytest.mark.parametrize("layout", [mx.ROWMAJOR, mx.TILED])
def test_quantized_rows_of_any_magnitude(layout):
    gen = torch.Generator().manual_seed(4)
    d = 640
    x = rows_of(gen, d, F)
    p = mx.Norm(eps=0.0, weight=rand(gen, d, dtype=BF, mean=1.0, std=0.1).to(DEV))
    for rot in (None, "h32"):
        announce("norm_quantize, rows of any magnitude", layout, rot)
        y, _ = mx.norm(x, p, out_dtype=F)
        codes, scales, _ = mx.norm_quantize(x, p, None, rot, layout)
        torch.cuda.synchronize()
        assert torch.isfinite(y).all()
        got = (codes.cpu().numpy(), scales.cpu().numpy())
        if layout == mx.TILED:
            got = mx.untile_host(*got, len(MAGS))
        want = oracle.quantize(y.cpu().numpy(), rot=rot)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


def test_zero_row_without_eps_is_undefined_as_in_the_formula():
    x = torch.ones(3, 96, device=DEV)
    x[1] = 0
    announce("norm, a zero row and eps = 0")
    y, _ = mx.norm(x, mx.Norm(eps=0.0))
    torch.cuda.synchronize()
    assert torch.isnan(y[1]).all()
    assert float((y[[0, 2]] - 1).abs().max()) <= 100 * 2.0 ** -24
