"""The tile kernels of the GEMM epilogues where a workgroup takes several tiles:
bias, gate, residual and the accumulators' clearing of the second tile, and ring
loads that run across it.  Sums are exact (operands as in test_gpu_gemm_fused.py),
and a bias is added once, so x = A B^T + bias is off by at most u of itself; the
rest as there.  Sampled rows, every tile's among them; all columns."""
import numpy as np
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
import oracle
from test_gpu_gemm_fused import ACTS, BF, DEV, F, R, T, U, act64, announce, check, operand, vectors

pytestmark = pytest.mark.gpu

# (m, k, columns in all of the weights, tile): of 256 x 256 and of 128 x 128,
# with workgroups of one tile and of two, edges in both directions; 7500 and 5980
# columns are whole pieces of 4, 7501 are not
CASES = [(4100, 640, 7500, 256), (4100, 640, 7501, 256), (1900, 256, 5980, 128), (1900, 256, 5989, 128)]


def expect_tiles(m, k, wide, tile):
    """The choice of a kernel by expected time, as the library makes it, has to
    give this tile, and more tiles than there are workgroups."""
    cus, nk = torch.cuda.get_device_properties(0).multi_processor_count, k // 128
    tiles = {t: -(-m // t) * -(-wide // t) for t in (128, 256)}
    rest = tiles[128] % (2 * cus)
    last = 0 if rest == 0 else (3 * nk if rest <= cus else 5 * nk) + 50
    cost = {256: -(-tiles[256] // cus) * (5 * nk + 120), 128: tiles[128] // (2 * cus) * (5 * nk + 50) + last,
            "small": 40 + -(-m // 64) * (wide * (k // 32) * 17 // 260000)}
    assert cost["small"] >= min(cost[128], cost[256])
    assert (128 if cost[128] < cost[256] else 256) == tile
    assert tiles[tile] > (cus if tile == 256 else 2 * cus)


def sample(m, tile):
    """Rows of every row of tiles: its first, its last and some between."""
    at = [i for t in range(0, m, tile) for i in (t, t + 33, t + 95, t + tile - 1)]
    return np.array(sorted(i for i in set(at + [m - 1]) if i < m))


@pytest.mark.parametrize("layout", [R, T])
@pytest.mark.parametrize("m,k,n,tile", CASES)
def test_epilogue_over_several_tiles(m, k, n, tile, layout):
    expect_tiles(m, k, n, tile)
    rng = np.random.default_rng(m + n)
    gen = torch.Generator().manual_seed(n)
    ac, as_, dac, das = operand(rng, m, k, -6, -4, layout)
    bc, bs, dbc, dbs = operand(rng, n, k, -1, 1, layout)
    at = sample(m, tile)
    acc = oracle.gemm(ac[at], as_[at], bc, bs)
    kw = dict(layout=layout, m=m, n=n)
    for i, act in enumerate(ACTS):
        vdt, rdt = (BF, F)[i % 2], (F, BF)[i // 2 % 2]
        group, bias, gate = vectors(gen, m, n, vdt)
        residual = torch.randn(m, n, generator=gen).to(rdt).to(DEV)
        for form in ("bias", "plain", "gate", "residual", "all"):
            if i == 2 and form == "all":   # groups of fewer rows than a wave's
                group = 5
                gate = torch.randn(-(-m // group), n, generator=gen).to(vdt).to(DEV)
            e = mx.Epilogue(act=act, group_rows=group, bias=bias if form in ("bias", "all") else None,
                            gate=gate if form in ("gate", "all") else None,
                            residual=residual if form in ("residual", "all") else None)
            x = acc if e.bias is None else acc + bias.double().cpu().numpy()[None, :]
            want, own = act64(act, x)
            bound = own + (0.0 if e.bias is None else 1.13 * U * np.abs(x))
            if e.gate is not None:
                g = gate.double().cpu().numpy()[at // group]
                want, bound = want * g, bound * np.abs(g) + U * np.abs(want * g)
            if e.residual is not None:
                r = residual[torch.from_numpy(at).to(DEV)].double().cpu().numpy()
                want, bound = want + r, bound + U * (np.abs(want) + np.abs(r))
            announce("several tiles", m, k, n, tile, layout, act, form, rdt)
            for dt in (F, BF):
                y = mx.gemm_epilogue(dac, das, dbc, dbs, e, dt, **kw)
                torch.cuda.synchronize()
                check(y[torch.from_numpy(at).to(DEV)], want, bound, f"{act} {form} {dt}")


@pytest.mark.parametrize("layout", [R, T])
@pytest.mark.parametrize("m,k,wide,tile", [(4100, 640, 7500, 256), (1900, 256, 5980, 128)])
def test_glu_over_several_tiles(m, k, wide, tile, layout):
    expect_tiles(m, k, wide, tile)
    n = wide // 2
    rng = np.random.default_rng(m)
    gen = torch.Generator().manual_seed(n)
    ac, as_, dac, das = operand(rng, m, k, -6, -4, layout)
    gc, gs, dgc, dgs = operand(rng, n, k, -1, 1, layout)
    uc, us, duc, dus = operand(rng, n, k, -1, 1, layout)
    at = sample(m, tile)
    acc_g, acc_u = oracle.gemm(ac[at], as_[at], gc, gs), oracle.gemm(ac[at], as_[at], uc, us)
    for i, act in enumerate(ACTS):
        bg = torch.randn(n, generator=gen).to((BF, F)[i % 2]).to(DEV) if i in (0, 2, 4) else None
        bu = torch.randn(n, generator=gen).to((BF, F)[i % 2]).to(DEV) if i in (2, 3) else None
        xg, xu = (x if b is None else x + b.double().cpu().numpy()[None, :] for x, b in ((acc_g, bg), (acc_u, bu)))
        a, own = act64(act, xg)
        du = 0.0 if bu is None else U * np.abs(xu)
        want = a * xu
        bound = (own + (0.0 if bg is None else 1.13 * U * np.abs(xg))) * (np.abs(xu) + du) + np.abs(a) * du + 2 * U * np.abs(want)
        announce("several gated tiles", m, k, n, tile, layout, act)
        for dt in (F, BF):
            y = mx.gemm_glu(dac, das, dgc, dgs, duc, dus, act, bg, bu, dt, layout=layout, m=m, n=n)
            torch.cuda.synchronize()
            check(y[torch.from_numpy(at).to(DEV)], want, bound, f"{act} {dt}")


@pytest.mark.parametrize("m,k,wide,tile", [(4100, 640, 7424, 256), (1900, 256, 5888, 128)])
def test_requant_over_several_tiles(m, k, wide, tile):
    """MXFP4 outputs are the oracle's quantizer on the fp32 ones (which the tests
    above hold to the formula)."""
    expect_tiles(m, k, wide, tile)
    rng = np.random.default_rng(k)
    gen = torch.Generator().manual_seed(m)
    at = sample(m, tile)
    pick = torch.from_numpy(at).to(DEV)
    _, _, dac, das = operand(rng, m, k, -9, 2, T)
    for glu in (False, True):
        n = wide // 2 if glu else wide
        w = [operand(rng, n, k, -1, 1, T)[2:] for _ in range(2 if glu else 1)]
        bias = torch.randn(n, generator=gen).to(BF).to(DEV)
        for act, rot, out in (("gelu_tanh", "h32", T), ("silu", None, R), ("gelu", "h32", R), ("none", None, T)):
            kw = dict(layout=T, m=m, n=n)
            announce("several requantized tiles", m, k, n, tile, act, rot, out, glu)
            if glu:
                y = mx.gemm_glu(dac, das, *w[0], *w[1], act, bias, None, F, **kw)
                q = mx.gemm_glu_requant(dac, das, *w[0], *w[1], act, bias, None, rot, out_layout=out, **kw)
            else:
                e = mx.Epilogue(act=act, bias=bias)
                y = mx.gemm_epilogue(dac, das, *w[0], e, F, **kw)
                q = mx.gemm_epilogue_requant(dac, das, *w[0], e, rot, out_layout=out, **kw)
            torch.cuda.synchronize()
            got = tuple(t.cpu().numpy() for t in q)
            got = mx.untile_host(*got, m) if out == T else got
            want = oracle.quantize(y[pick].cpu().numpy(), rot=rot)
            assert np.array_equal(got[1][at], want[1]) and np.array_equal(got[0][at], want[0]), (act, rot, glu)


def test_image_block_repeats_and_is_each_stage_of_the_formula():
    """The feed-forward block of 3584 image tokens (3072 -> 12288, modulation, gate,
    Hadamard): the same bits again and again, with a block on other inputs between
    the calls, and each stage near its own 64-bit value: the products' fp32 sums of
    K terms are off by at most 2 (K / 64 + 2) u of |A| |B|^T, the codes are the
    quantizer's."""
    m, d, f = 3584, 3072, 12288
    gen = torch.Generator(device=DEV).manual_seed(12)
    rnd = lambda *s, std=1.0: torch.randn(s, generator=gen, device=DEV) * std  # noqa: E731
    up, down = (mx.quantize_weight(rnd(*s, std=0.02), "h32", layout=T) for s in ((f, d), (d, f)))

    def state():
        vec = rnd(1, 3 * d, std=0.2).to(BF)
        p = mx.Norm(kind="layer", scale=vec[:, :d], shift=vec[:, d:2 * d], group_rows=m)
        return rnd(m, d).to(BF), p, rnd(m, d).to(BF), vec[:, 2 * d:]

    def block(x, p, residual, gate):
        return mx.ffn(x, p, residual, up, down, f, act="gelu_tanh", rot="h32", gate=gate, layout=T)

    one, other = state(), state()
    x, p, residual, gate = one
    announce("image block, repeated")
    first = [t.clone() for t in block(*one)]
    for _ in range(20):
        block(*other)
        again = block(*one)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    y, r = first
    at = np.arange(0, m, 61)
    pick = torch.from_numpy(at).to(DEV)
    announce("image block, stage by stage")
    n32, _ = mx.norm(x, p, residual, out_dtype=F)
    c, s, r2 = mx.norm_quantize(x, p, residual, "h32", T)
    h32 = mx.gemm_epilogue(c, s, *up, mx.Epilogue(act="gelu_tanh"), F, layout=T, m=m, n=f)
    hc, hs = mx.gemm_epilogue_requant(c, s, *up, mx.Epilogue(act="gelu_tanh"), "h32", T, T, m=m, n=f)
    y2 = mx.gemm_epilogue(hc, hs, *down, mx.Epilogue(gate=gate, group_rows=m, residual=r2), layout=T, m=m, n=d)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(r, r2)
    host = lambda q, rows: mx.untile_host(q[0].cpu().numpy(), q[1].cpu().numpy(), rows)  # noqa: E731
    for dense, q in ((n32, (c, s)), (h32, (hc, hs))):
        want = oracle.quantize(dense[pick].cpu().numpy(), rot="h32")
        got = host(q, m)
        assert np.array_equal(got[0][at], want[0]) and np.array_equal(got[1][at], want[1])

    def product(q, w, rows, k):
        a, b = host(q, m), host(w, rows)
        a = a[0][at], a[1][at]
        da, db = (torch.from_numpy(oracle.dequantize(*v)) for v in (a, b))
        return (da @ db.T).numpy(), 2 * (k / 64 + 2) * U * (da.abs() @ db.abs().T).numpy()

    acc, bound = product((c, s), up, f, d)
    want, own = act64("gelu_tanh", acc)
    check(h32[pick], want, 1.13 * bound + own, "hidden")
    acc, bound = product((hc, hs), down, d, f)
    g, res = gate.double().cpu().numpy(), r[pick].double().cpu().numpy()
    want = acc * g + res
    check(y[pick], want, bound * np.abs(g) + 2 * U * (np.abs(acc * g) + np.abs(res)), "y")
