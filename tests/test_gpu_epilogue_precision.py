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


def activation(act, x, m, glu=False):
    """act of the values x [n] through the epilogue of an m-row GEMM: zero
    products, x as the bias (fp32 result, every row alike).  glu: through the
    gated form, times an up projection of 1."""
    n, k = x.numel(), 256
    a = torch.zeros(m, k // 2, dtype=torch.uint8, device=DEV), torch.full((m, k // 32), 127, dtype=torch.uint8, device=DEV)
    b = torch.zeros(n, k // 2, dtype=torch.uint8, device=DEV), torch.full((n, k // 32), 127, dtype=torch.uint8, device=DEV)
    x = x.to(DEV)
    if glu:
        y = mx.gemm_glu(*a, *b, *b, act, x, torch.ones(n, device=DEV), F)
    else:
        y = mx.gemm_epilogue(*a, *b, mx.Epilogue(act=act, bias=x), F)
    torch.cuda.synchronize()
    same = (y == y[:1]) | (torch.isnan(y) & torch.isnan(y[:1]))
    assert bool(same.all())
    return y[0].cpu()


# rows and columns that take the small-M, the 128 x 128 and the 256 x 256 tile kernels
ROUTES = [(3, 1000), (130, 9000), (770, 12800)]


def test_gelu_keeps_the_tail():
    """gelu(x) = x Phi(x) relative to the result, through the negative tail.
    x Phi(-|x|) is x t poly(t) 2^(c x^2), t = 1 / (1 + p |x|), p = 0.285:
      fit 3 u, coefficients 1 u; t 3 u, times |d ln Phi(-a) e^(a^2/2) / d ln t|
      <= 0.8 / p: 9 u; Horner's 8 steps, 2 u each of sums of positive and
      negative terms at most 1.4 times the value: 23 u; the products t poly, x q,
      q E 3 u; the exponent 2.5 u of x^2 / 2 (its square, its product, its
      constant) and v_exp_f32 2 u: 41 u + 1.25 x^2 u.
    For x > 0, x - that: at most as much and 2 u.  Bound (45 + 1.5 x^2) u.  The
    exponential flushes below 2^-126, where the result is below 0.4 2^-126."""
    for m, n in ROUTES:
        x = torch.cat([torch.linspace(-13.3, 8, n - 6), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 40.0, 1e30])])
        v = x.double()
        want = (v * 0.5 * torch.special.erfc(-v / np.sqrt(2.0))).numpy()
        bound = (45 + 1.5 * v.numpy() ** 2) * U * np.abs(want) + 2.0 ** -127
        bound[-1] = U * 1e30
        for glu in (False, True):
            announce("gelu", m, n, glu)
            within(activation("gelu", x, m, glu), want, bound, f"gelu {m} {glu}")


def quotient64(act, x):
    """x / (1 + 2^t) in 64 bits, and |t|."""
    p = x if act == "silu" else 2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
    q = np.exp(-np.abs(p))
    return x * np.where(p >= 0, 1 / (1 + q), q / (1 + q)), np.abs(p) * 1.4426950408889634


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_silu_and_tanh_gelu_over_the_range_of_fp32(act):
    """Relative to the result wherever that is normal: t carries 4 roundings,
    times ln 2 in the exponential, v_exp_f32 and v_rcp_f32 2 u each, the sum and
    the products 6 u: (4 |t| + 10) u, as test_gpu_gemm_fused.py has it, here
    with no absolute part but the spacing of subnormal results, 2^-149."""
    for m, n in ROUTES:
        lo = -92.0 if act == "silu" else -10.2
        tiny = torch.tensor([s * f * 2.0 ** e for e in range(-126, -90, 3) for s in (1, -1) for f in (1.0, 1.4, 1.9)])
        ends = torch.tensor([lo + 3.2, lo + 0.5, lo, -88.8 if act == "silu" else -9.95, 2.0 ** 100, 3e38, -3e38, 0.0])
        x = torch.cat([tiny, ends, torch.linspace(lo, 9, n - tiny.numel() - ends.numel())])
        want, t = quotient64(act, x.double().numpy())
        bound = (4 * np.minimum(t, 200) + 10) * U * np.abs(want) + 2.0 ** -149
        for glu in (False, True):
            announce(act, m, n, glu)
            within(activation(act, x, m, glu), want, bound, f"{act} {m} {glu}")
