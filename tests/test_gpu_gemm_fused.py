"""GEMMs with a feed-forward epilogue and the gated GEMM against their formulas
in 64 bits.

Operands: block exponents in [-6, -4] (A) and [-1, 1] (weights) with K <= 4096
make every partial sum a multiple of 2^-9 below 2^15, exact in fp32 whatever
the order, so the accumulators equal the oracle's binary64 product.  Then only
the epilogue rounds (u = 2^-24):
  the bias sum: a kernel may start the accumulation from the bias, which is on
    no grid, so each of the K / 64 + 2 accumulations may be off by an ulp (2 u)
    of a running sum below |A| |B|^T + |bias|;
  act: its slope is at most 1.13; silu and gelu_tanh are x * rcp(1 + exp2(t)),
    off by at most (4 |t| + 10) u of the result (t 4 roundings, times ln 2 in
    the exponential, v_exp_f32 and v_rcp_f32 one ulp each); gelu has the
    rational approximation's 0.75e-7 and 12 u, times |x|;
  gate, product and residual: one rounding each.
bf16 results: half a step more, 2^-8 of the value.  MXFP4 results must equal
the oracle's quantizer on the fp32 result, bit for bit."""
import numpy as np
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
import oracle
import workloads

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32
R, T = mx.ROWMAJOR, mx.TILED
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def announce(*what):
    print("[case]", *what, flush=True)


def to_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def operand(rng, rows, k, e_lo, e_hi, layout):
    """(host codes, host scales, device codes, device scales); the tiled
    padding rows hold NaN scale bytes."""
    c, s = workloads.random_mxfp4(rng, rows, k, e_lo, e_hi)
    if layout == T:
        dc, ds = mx.tile_host(np.vstack([c, np.full((mx.padded_rows(rows) - rows, k // 2), 0x77, np.uint8)]),
                              np.vstack([s, np.full((mx.padded_rows(rows) - rows, k // 32), 0xFF, np.uint8)]))
    else:
        dc, ds = c, s
    return c, s, to_dev(dc), to_dev(ds)


def act64(name, x):
    """act(x) in binary64 and the bound of the kernel's own error in it."""
    if name == "none":
        return x, 0.0 * x
    if name == "relu":
        return np.maximum(x, 0.0), 0.0 * x
    if name == "gelu":
        return x * 0.5 * torch.special.erfc(torch.from_numpy(-x / np.sqrt(2.0))).numpy(), np.abs(x) * (0.75e-7 + 12 * U)
    p = x if name == "silu" else 2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
    y = x * np.where(p >= 0, 1 / (1 + np.exp(-np.abs(p))), np.exp(-np.abs(p)) / (1 + np.exp(-np.abs(p))))
    return y, (4 * 1.4427 * np.abs(p) + 10) * U * np.abs(y) + 1e-36


def check(got, want, bound, what):
    got = got.detach().cpu()
    step = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    err = np.abs(got.double().numpy() - want)
    lim = bound + step * (np.abs(want) + bound)
    bad = ~(err <= lim)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {float((err / lim).max()):.3g} of the bound"


def preact(acc, absacc, bias, k):
    if bias is None:
        return acc, 0.0 * acc
    b = bias.double().cpu().numpy()[None, :]
    return acc + b, 2 * (k / 64 + 2) * U * (absacc + np.abs(b))


def absdot(ac, as_, bc, bs):
    """|A| |B|^T"""
    return np.abs(oracle.dequantize(ac, as_)) @ np.abs(oracle.dequantize(bc, bs)).T


# (m, n, k): one token, M groups of the decode kernels, more rows, edges of
# 16, 32, 64, 128 and 256, odd widths, K tails
SHAPES = [(1, 1, 32), (1, 256, 4096), (5, 40, 96), (16, 300, 512), (17, 96, 128), (33, 31, 160), (48, 64, 1024),
          (64, 128, 384), (65, 33, 96), (130, 520, 256), (300, 1000, 1184), (257, 259, 128), (520, 1030, 1152),
          (1100, 640, 256)]
# shapes that the 128 x 128 and (the last) the 256 x 256 tile kernels take
TILES = [(520, 8200, 256), (130, 9001, 512), (200, 4100, 4096), (770, 12850, 1280), (770, 12848, 1280)]
GLU_TILES = [(520, 4100, 256), (130, 9001, 512), (770, 6425, 1280)]


def vectors(gen, m, n, dtype):
    group = max(1, m // 3)
    bias = torch.randn(n, generator=gen).to(dtype).to(DEV)
    gate = torch.randn(-(-m // group), n + 3, generator=gen).to(dtype).to(DEV)[:, :n]
    return group, bias, gate


@pytest.mark.parametrize("layout", [R, T])
@pytest.mark.parametrize("m,n,k", SHAPES + TILES)
def test_epilogue(m, n, k, layout):
    if layout == T and k % 128:
        pytest.skip("tiled needs k % 128 == 0")
    rng = np.random.default_rng(m + 7 * n + k)
    gen = torch.Generator().manual_seed(m + n + k)
    ac, as_, dac, das = operand(rng, m, k, -6, -4, layout)
    bc, bs, dbc, dbs = operand(rng, n, k, -1, 1, layout)
    acc, absacc = oracle.gemm(ac, as_, bc, bs), absdot(ac, as_, bc, bs)
    for i, act in enumerate(ACTS):
        vdt, rdt = (BF, F)[i % 2], (F, BF)[i % 3 % 2]
        group, bias, gate = vectors(gen, m, n, vdt)
        residual = torch.randn(m, n, generator=gen).to(rdt).to(DEV)
        for form in ("bias", "plain", "gate", "residual", "all"):
            if i != (0, 3, 2, 1, 4)[("bias", "plain", "gate", "residual", "all").index(form)] and form != "all":
                continue
            e = mx.Epilogue(act=act, group_rows=group)
            if form in ("bias", "all"):
                e.bias = bias
            if form in ("gate", "all"):
                e.gate = gate
            if form in ("residual", "all"):
                e.residual = residual
            x, dx = preact(acc, absacc, e.bias, k)
            want, own = act64(act, x)
            bound = 1.13 * dx + own
            if e.gate is not None:
                g = gate.double().cpu().numpy()[np.arange(m) // group]
                want, bound = want * g, bound * np.abs(g) + U * np.abs(want * g)
            if e.residual is not None:
                r = residual.double().cpu().numpy()
                want, bound = want + r, bound + U * (np.abs(want) + np.abs(r))
            announce("gemm_epilogue", m, n, k, layout, act, form)
            y = mx.gemm_epilogue(dac, das, dbc, dbs, e, F, layout=layout, m=m, n=n)
            yb = mx.gemm_epilogue(dac, das, dbc, dbs, e, BF, layout=layout, m=m, n=n)
            torch.cuda.synchronize()
            check(y, want, bound, f"{act} {form}")
            check(yb, want, bound, f"{act} {form} bf16")
            if form == "plain":
                assert torch.equal(yb, y.to(BF))


@pytest.mark.parametrize("layout", [R, T])
@pytest.mark.parametrize("m,n,k", SHAPES + GLU_TILES)
def test_glu(m, n, k, layout):
    if layout == T and k % 128:
        pytest.skip("tiled needs k % 128 == 0")
    rng = np.random.default_rng(3 * m + 5 * n + k)
    gen = torch.Generator().manual_seed(m + n + k)
    ac, as_, dac, das = operand(rng, m, k, -6, -4, layout)
    gc, gs, dgc, dgs = operand(rng, n, k, -1, 1, layout)
    uc, us, duc, dus = operand(rng, n, k, -1, 1, layout)
    acc_g, acc_u = oracle.gemm(ac, as_, gc, gs), oracle.gemm(ac, as_, uc, us)
    abs_g, abs_u = absdot(ac, as_, gc, gs), absdot(ac, as_, uc, us)
    for i, act in enumerate(ACTS):
        bg = torch.randn(n, generator=gen).to((BF, F)[i % 2]).to(DEV) if i in (0, 2, 4) else None
        bu = torch.randn(n, generator=gen).to((BF, F)[i % 2]).to(DEV) if i in (2, 3) else None
        xg, dg = preact(acc_g, abs_g, bg, k)
        xu, du = preact(acc_u, abs_u, bu, k)
        a, own = act64(act, xg)
        want = a * xu
        bound = (1.13 * dg + own) * (np.abs(xu) + du) + np.abs(a) * du + 2 * U * np.abs(want)
        announce("gemm_glu", m, n, k, layout, act)
        y = mx.gemm_glu(dac, das, dgc, dgs, duc, dus, act, bg, bu, F, layout=layout, m=m, n=n)
        yb = mx.gemm_glu(dac, das, dgc, dgs, duc, dus, act, bg, bu, BF, layout=layout, m=m, n=n)
        torch.cuda.synchronize()
        check(y, want, bound, act)
        check(yb, want, bound, act + " bf16")


QSHAPES = [(1, 32, 96), (16, 128, 4096), (20, 256, 256), (40, 384, 128), (64, 128, 640), (130, 96, 384),
           (300, 640, 256), (1030, 768, 384), (1100, 640, 1184), (520, 8192, 256), (520, 4096, 256),
           (770, 12800, 1280), (770, 6400, 1280)]


@pytest.mark.parametrize("out_layout", [R, T])
@pytest.mark.parametrize("layout", [R, T])
@pytest.mark.parametrize("m,n,k", QSHAPES)
def test_requant(m, n, k, layout, out_layout):
    if (layout == T and k % 128) or (out_layout == T and n % 128):
        pytest.skip("tiled needs multiples of 128")
    rng = np.random.default_rng(m + n + k)
    gen = torch.Generator().manual_seed(m + n)
    # wide exponents too: rounded sums must requantize to the same bytes
    e = (-9, 2) if m % 2 == 0 else (-6, -4)
    _, _, dac, das = operand(rng, m, k, *e, layout)
    _, _, dgc, dgs = operand(rng, n, k, -1, 1, layout)
    _, _, duc, dus = operand(rng, n, k, -1, 1, layout)
    kw = dict(layout=layout, m=m, n=n)
    for i, act in enumerate(ACTS):
        rot = (None, "h32")[i % 2] if i < 4 else "h32"
        bias = torch.randn(n, generator=gen).to(BF).to(DEV) if i != 1 else None
        for glu in (False, True):
            announce("requant", m, n, k, layout, out_layout, act, rot, glu)
            if glu:
                y = mx.gemm_glu(dac, das, dgc, dgs, duc, dus, act, bias, None, F, **kw)
                q = mx.gemm_glu_requant(dac, das, dgc, dgs, duc, dus, act, bias, None, rot, out_layout=out_layout, **kw)
            else:
                ep = mx.Epilogue(act=act, bias=bias)
                y = mx.gemm_epilogue(dac, das, dgc, dgs, ep, F, **kw)
                q = mx.gemm_epilogue_requant(dac, das, dgc, dgs, ep, rot, out_layout=out_layout, **kw)
            torch.cuda.synchronize()
            got = tuple(t.cpu().numpy() for t in q)
            if out_layout == T:
                got = mx.untile_host(*got, m)
            want = oracle.quantize(y.cpu().numpy(), rot=rot)
            assert np.array_equal(got[1], want[1]), f"{act} {rot} {glu}: {np.count_nonzero(got[1] != want[1])} scales"
            assert np.array_equal(got[0], want[0]), f"{act} {rot} {glu}: {np.count_nonzero(got[0] != want[0])} codes"


@pytest.mark.parametrize("m,n,k", [(3, 50, 256), (300, 522, 256), (600, 1024, 128), (1030, 768, 256), (520, 8200, 256),
                                   (770, 12852, 1280)])
def test_strided_output_in_place_residual_and_guards(m, n, k):
    """Y and the residual are one strided buffer; what lies past column n stays."""
    for ld in (n + 6, n + 8, n + 1):
        for dt in (F, BF):
            rng = np.random.default_rng(m)
            gen = torch.Generator().manual_seed(ld)
            _, _, dac, das = operand(rng, m, k, -6, -4, R)
            _, _, dbc, dbs = operand(rng, n, k, -1, 1, R)
            buf = torch.randn(m, ld, generator=gen).to(dt).to(DEV)
            before = buf.clone()
            y = buf[:, :n]
            announce("strided in-place epilogue", m, n, k, ld, dt)
            want = mx.gemm_epilogue(dac, das, dbc, dbs, mx.Epilogue(act="relu", residual=before[:, :n].contiguous()), dt)
            mx.gemm_epilogue(dac, das, dbc, dbs, mx.Epilogue(act="relu", residual=y), y=y)
            torch.cuda.synchronize()
            assert torch.equal(buf[:, n:], before[:, n:])
            assert torch.equal(buf[:, :n], want)


def test_empty_and_not_finite():
    rng = np.random.default_rng(0)
    ac, as_, dac, das = operand(rng, 300, 128, -6, -4, R)
    _, _, dbc, dbs = operand(rng, 520, 128, -1, 1, R)
    announce("epilogue: no rows, no columns")
    assert mx.gemm_epilogue(dac[:0], das[:0], dbc, dbs).shape == (0, 520)
    assert mx.gemm_epilogue(dac, das, dbc[:0], dbs[:0]).shape == (300, 0)
    assert mx.gemm_glu(dac[:0], das[:0], dbc, dbs, dbc, dbs).shape == (0, 520)
    for m in (7, 300):
        res = torch.zeros(m, 520, device=DEV)
        res[2, 3], res[5, 519] = float("nan"), float("inf")
        bias = torch.zeros(520, device=DEV)
        bias[100], bias[200], bias[300] = float("nan"), float("inf"), -float("inf")
        announce("epilogue: NaN and infinities", m)
        for act in ACTS:
            y = mx.gemm_epilogue(dac[:m], das[:m], dbc, dbs, mx.Epilogue(act=act, bias=bias, residual=res), F)
            torch.cuda.synchronize()
            fin = torch.isfinite(y)
            want = torch.ones_like(fin)
            want[2, 3] = want[5, 519] = False
            want[:, 100] = want[:, 200] = False
            if act != "relu":
                want[:, 300] = False
            assert torch.equal(fin, want), act
            assert torch.isnan(y[:, 100]).all() and bool((y[:, 200] == float("inf")).all()), act


def test_side_stream_and_graph_replays():
    """The whole path on a stream of its own, then captured and replayed with
    new inputs between replays: every replay equals the eager result."""
    m, d, f = 37, 256, 640
    gen = torch.Generator().manual_seed(1)
    w = [mx.quantize_weight((torch.randn(*s, generator=gen) * 0.05).to(DEV), "h32", layout=T)
         for s in ((f, d), (f, d), (d, f))]
    p = mx.Norm(weight=torch.ones(d, dtype=BF, device=DEV))
    x, res = (torch.randn(m, d, generator=gen).to(BF).to(DEV) for _ in range(2))

    def path():
        return mx.ffn(x, p, res, w[0], w[2], f, w_gate=w[1], rot="h32", layout=T)

    announce("ffn on a side stream and in a graph")
    eager = [t.clone() for t in path()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = path()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = path()
    for i in range(4):
        x.copy_(torch.randn(m, d, generator=gen).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = path()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_ffn_row_major_without_residual_and_empty():
    d, f, m = 96, 160, 9
    gen = torch.Generator().manual_seed(3)
    w = [mx.quantize_weight((torch.randn(*s, generator=gen) * 0.05).to(DEV)) for s in ((f, d), (f, d), (d, f))]
    x = torch.randn(m, d, generator=gen).to(BF).to(DEV)
    bias = [torch.randn(n, generator=gen).to(BF).to(DEV) for n in (f, f, d)]
    p = mx.Norm(kind="layer")
    announce("ffn row-major, no residual add before the norm")
    for gated in (False, True):
        kw = dict(w_gate=w[1], bias_gate=bias[1]) if gated else {}
        y, r = mx.ffn(x, p, None, w[0], w[2], f, act="silu", bias_up=bias[0], bias_down=bias[2], **kw)
        c, s, r2 = mx.norm_quantize(x, p)
        assert r2 is None
        if gated:
            h = mx.gemm_glu_requant(c, s, *w[1], *w[0], act="silu", bias_g=bias[1], bias_u=bias[0])
        else:
            h = mx.gemm_epilogue_requant(c, s, *w[0], mx.Epilogue(act="silu", bias=bias[0]))
        want = mx.gemm_epilogue(*h, *w[2], mx.Epilogue(bias=bias[2], residual=x))
        torch.cuda.synchronize()
        assert torch.equal(r, x) and torch.equal(y, want)
    y, r = mx.ffn(x[:0], p, None, w[0], w[2], f)
    assert y.shape == (0, d) and r.shape == (0, d)
    with pytest.raises(ValueError):
        mx.ffn(x, p, None, w[0], w[2], f, bias_gate=bias[1])
    with pytest.raises(ValueError):
        mx.ffn(x, p, None, w[2], w[2], f)
    with pytest.raises(ValueError):
        mx.ffn(x, p, None, w[0], w[2], f, rot=mx.Smooth(torch.ones(d, device=DEV)))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m", [1, 16, 70, 1100])
def test_ffn_equals_its_parts(m, gated):
    """ffn() is its three calls; and near the unquantized block in 64 bits (the
    4-bit formats' own error, about 12% per product: a wiring error is off by
    100%)."""
    d, f = 512, 1408
    gen = torch.Generator().manual_seed(m)
    host = [torch.randn(*s, generator=gen) * 0.05 for s in ((f, d), (f, d), (d, f))]
    w = [mx.quantize_weight(t.to(DEV), "h32", layout=T) for t in host]
    x, res = (torch.randn(m, d, generator=gen).to(BF).to(DEV) for _ in range(2))
    g = torch.randn(1, d, generator=gen).to(BF).to(DEV)
    p = mx.Norm(weight=torch.ones(d, dtype=BF, device=DEV), group_rows=m)
    act = "silu" if gated else "gelu_tanh"
    announce("ffn", m, gated)
    y, r = mx.ffn(x, p, res, w[0], w[2], f, w_gate=w[1] if gated else None, act=act, rot="h32", gate=g, layout=T)
    c, s, r2 = mx.norm_quantize(x, p, res, "h32", T)
    if gated:
        h = mx.gemm_glu_requant(c, s, *w[1], *w[0], act=act, rot="h32", layout=T, out_layout=T, m=m, n=f)
    else:
        h = mx.gemm_epilogue_requant(c, s, *w[0], mx.Epilogue(act=act), "h32", T, T, m=m, n=f)
    y2 = mx.gemm_epilogue(*h, *w[2], mx.Epilogue(gate=g, group_rows=m, residual=r2), layout=T, m=m, n=d)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(r, r2)
    v = x.cpu().double() + res.cpu().double()
    z = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + p.eps)
    up = z @ host[0].double().T
    hid = torch.from_numpy(act64(act, (z @ host[1].double().T if gated else up).numpy())[0])
    hid = hid * up if gated else hid
    want = hid @ host[2].double().T * g.cpu().double()
    got = y.cpu().double() - r.cpu().double()
    assert float((got - want).norm() / want.norm()) < 0.5
