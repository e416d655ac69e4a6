"""What the GEMM epilogues round, on sums that are themselves exact.

Operands as in test_gpu_gemm_fused.py: every partial sum is a multiple of 2^-9
below 2^15, so the accumulators equal the oracle's binary64 product."""
import numpy as np
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
import oracle
from test_gpu_gemm_fused import DEV, F, R, T, U, announce, operand

pytestmark = pytest.mark.gpu

# the small-M, 128 x 128 and 256 x 256 tile kernels; long and short K; edges
SHAPES = [(16, 300, 512), (64, 128, 4096), (520, 8200, 256), (200, 4100, 4096), (130, 9001, 512), (770, 12850, 1280)]


def within(got, want, bound, what):
    err = np.abs(got.cpu().double().numpy() - want)
    bad = ~(err <= bound)
    worst = float((err / np.maximum(bound, 1e-300)).max())
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {worst:.3g} of the bound"


@pytest.mark.parametrize("layout", [R, T])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_bias_is_added_to_the_finished_sum(m, n, k, layout):
    """A bias far above the products: the sum rounds once (u of the result),
    the gated product once more for each factor and for itself (3 u and the
    products of those)."""
    rng = np.random.default_rng(m + n + k)
    gen = torch.Generator().manual_seed(k)
    ac, as_, dac, das = operand(rng, m, k, -6, -4, layout)
    bc, bs, dbc, dbs = operand(rng, n, k, -1, 1, layout)
    acc = oracle.gemm(ac, as_, bc, bs)
    big = [(torch.randn(n, generator=gen) * 2.0 ** 17) for _ in range(2)]
    kw = dict(layout=layout, m=m, n=n)
    x = [acc + b.double().numpy()[None, :] for b in big]
    announce("bias above the products", m, n, k, layout)
    y = mx.gemm_epilogue(dac, das, dbc, dbs, mx.Epilogue(bias=big[0].to(DEV)), F, **kw)
    h = mx.gemm_glu(dac, das, dbc, dbs, dbc, dbs, "none", big[0].to(DEV), big[1].to(DEV), F, **kw)
    one = mx.gemm_glu(dac, das, dbc, dbs, dbc, dbs, "none", None, big[1].to(DEV), F, **kw)
    torch.cuda.synchronize()
    within(y, x[0], U * np.abs(x[0]), "bias")
    want = x[0] * x[1]
    within(h, want, 3.01 * U * np.abs(want), "gated, both biases")
    want = acc * x[1]
    within(one, want, 2.01 * U * np.abs(want), "gated, up bias")
