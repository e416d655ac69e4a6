"""The experts' products and the mixture-of-experts block against their formulas
in 64 bits.

Operands: block exponents in [-6, -4] (A) and [-1, 1] (weights) with K <= 4096
make every partial sum a multiple of 2^-9 below 2^15, exact in fp32 whatever the
order, so the products equal the binary64 ones and only what follows rounds
(u = 2^-24): the bias one rounding; act as (4 |t| + 10) u of the result for silu
and tanh GELU, t its exponent, and (45 + 1.5 x^2) u for GELU, its slope at most
1.13; the gated product one rounding; a result in bf16 2^-8 of the value.
MXFP4 results have to equal the quantizer's bytes for the fp32 result.
The weighted sum: one rounding for each choice, of a running sum below
S = |residual| + sum |w| (|z| + |b|); in the 16-bit form each product is off by
2^-11 of itself or by 2^-25 of 2^15 2^-14 times its block's largest, at most
2^-24 of it."""
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
    """(values, device codes, device scales); tiled padding rows hold NaN scales."""
    c, s = workloads.random_mxfp4(rng, rows, k, e_lo, e_hi)
    v = oracle.dequantize(c, s)
    if layout == T:
        c, s = mx.tile_host(np.vstack([c, np.full((mx.padded_rows(rows) - rows, k // 2), 0x77, np.uint8)]),
                            np.vstack([s, np.full((mx.padded_rows(rows) - rows, k // 32), 0xFF, np.uint8)]))
    return v, to_dev(c), to_dev(s)


def experts_weights(rng, experts, n, k, layout):
    each = [operand(rng, n, k, -1, 1, layout) for _ in range(experts)]
    return [e[0] for e in each], (torch.stack([e[1] for e in each]), torch.stack([e[2] for e in each]))


def act64(name, x):
    if name == "none":
        return x, 0.0 * x
    if name == "relu":
        return np.maximum(x, 0.0), 0.0 * x
    if name == "gelu":
        y = x * 0.5 * torch.special.erfc(torch.from_numpy(-x / np.sqrt(2.0))).numpy()
        return y, (45 + 1.5 * x * x) * U * np.abs(y) + 1e-36
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


def choose(rng, tokens, topk, experts, how):
    """ids: "even"; "skewed" (half of all pairs at expert 1, some experts empty);
    "part" (a third of the ids belong to no expert here, a token's all)"""
    ids = np.stack([rng.permutation(max(experts, topk))[:topk] for _ in range(tokens)]) % experts
    if how == "skewed":
        ids[rng.random(ids.shape) < 0.5] = min(1, experts - 1)
        ids[ids == experts - 1] = 0
    elif how == "part":
        ids[rng.random(ids.shape) < 0.3] = -1
        ids[tokens // 2] = experts + 3
    return ids


def rows_of(plan):
    order = plan.order.cpu().numpy()
    offsets = plan.offsets.cpu().numpy()
    expert = np.repeat(np.arange(plan.experts), np.diff(offsets))
    return order[:offsets[-1]], expert


def up64(a, wu, wg, bu, bg, act, tokens, experts):
    """H, its bound, for rows (tokens, experts)."""
    h, b = np.empty((len(tokens), wu[0].shape[0])), np.empty((len(tokens), wu[0].shape[0]))
    for e in np.unique(experts):
        at = np.flatnonzero(experts == e)
        rows = a[tokens[at]]
        u = rows @ wu[e].T
        du = 0 * u
        if bu is not None:
            u = u + bu[e]
            du = U * np.abs(u)
        if wg is None:
            y, own = act64(act, u)
            h[at], b[at] = y, 1.13 * du + own
            continue
        g = rows @ wg[e].T
        dg = 0 * g
        if bg is not None:
            g = g + bg[e]
            dg = U * np.abs(g)
        y, own = act64(act, g)
        dy = 1.13 * dg + own
        h[at] = y * u
        b[at] = dy * np.abs(u) + np.abs(y) * du + dy * du + U * np.abs(y * u)
    return h, b


# (tokens, topk, experts, d, n): one pair; row tiles of 16 and 32 rows (up to 7 and 18
# pairs an expert) and of 128; K tails; odd widths
UP = [(1, 1, 1, 128, 128), (1, 2, 8, 4096, 96), (5, 2, 3, 96, 40), (40, 3, 10, 160, 1000), (64, 4, 16, 512, 64),
      (61, 4, 12, 384, 300), (100, 3, 8, 1152, 33), (130, 2, 6, 96, 200), (300, 2, 5, 256, 300), (300, 2, 5, 128, 259),
      (700, 3, 4, 640, 520), (1300, 1, 2, 256, 130), (1100, 2, 3, 1280, 515), (2600, 2, 3, 128, 258), (150, 2, 4, 32, 200), (400, 2, 3, 1184, 200), (1500, 2, 4, 416, 160)]


@pytest.mark.parametrize("layout", [R, T])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("tokens,topk,experts,d,n", UP)
def test_up(tokens, topk, experts, d, n, gated, layout):
    if layout == T and d % 128:
        pytest.skip("tiled needs k % 128 == 0")
    rng = np.random.default_rng(tokens + n)
    a, ac, as_ = operand(rng, tokens, d, -6, -4, layout)
    wu, wud = experts_weights(rng, experts, n, d, layout)
    wg, wgd = experts_weights(rng, experts, n, d, layout) if gated else (None, None)
    for i, how in enumerate(("even", "skewed", "part")):
        act, dtype = ACTS[(i + tokens) % 5] if not gated else ACTS[2 + (i + tokens) % 3], (BF, F)[i % 2]
        ids = choose(rng, tokens, topk, experts, how)
        plan = mx.moe_plan(to_dev(ids.astype(np.int32)), experts)
        bu = to_dev(rng.standard_normal((experts, n)).astype(np.float32)).to(dtype) if i else None
        bg = to_dev(rng.standard_normal((experts, n)).astype(np.float32)).to(dtype) if gated and i == 1 else None
        pairs, ex = rows_of(plan)
        f64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        want, bound = up64(a, wu, wg, f64(bu), f64(bg), act, pairs // topk, ex)
        kw = dict(w_gate=wgd, act=act, bias_up=bu, bias_gate=bg, layout=layout, n=n)
        for out in (F, BF):
            announce("moe_up", tokens, topk, experts, d, n, gated, layout, how, act, out)
            # a strided result with a border: nothing behind the last row or column is written
            y = torch.full((tokens * topk + 2, n + 5), 77.0, dtype=out, device=DEV)
            mx.moe_up(ac, as_, plan, wud, y=y[:tokens * topk, :n], **kw)
            check(y[:len(pairs), :n], want, bound, f"{how} {act} {out}")
            assert (y[len(pairs):] == 77).all() and (y[:, n:] == 77).all()
            z = mx.moe_up(ac, as_, plan, wud, out_dtype=out, **kw)
            assert torch.equal(z[:len(pairs)], y[:len(pairs), :n])
            if out == F:
                exact = z[:len(pairs)].clone()
        for out_layout in (R, T):
            if n % (128 if out_layout == T else 32):
                continue
            for rot in (None, "h32"):
                announce("moe_up_requant", how, out_layout, rot)
                yc, ys = mx.moe_up_requant(ac, as_, plan, wud, rot=rot, out_layout=out_layout, **kw)
                if len(pairs) == 0:
                    continue
                qc, qs = mx.quantize_rotate(exact, rot)
                if out_layout == T:
                    hc, hs = mx.untile_host(yc.cpu().numpy(), ys.cpu().numpy(), len(pairs))
                else:
                    hc, hs = yc[:len(pairs)].cpu().numpy(), ys[:len(pairs)].cpu().numpy()
                assert np.array_equal(hc, qc.cpu().numpy()) and np.array_equal(hs, qs.cpu().numpy())


# Several tiles a workgroup: of 128 rows, with K of one stage (the ring is then three
# tiles ahead), two and three; of 256 rows.
LARGE = [(3000, 2, 4, 128, 8200), (1500, 3, 3, 256, 8200), (1000, 3, 3, 384, 8200), (3000, 2, 2, 768, 12900),
         (1500, 3, 3, 1024, 9000), (2100, 2, 5, 1280, 12900)]


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("tokens,topk,experts,d,n", LARGE)
def test_large_tiles(tokens, topk, experts, d, n, gated):
    """A sample of rows, the last and first ones of the experts among them; each of
    all columns.  moe_up in fp32, bf16 and MXFP4, moe_down (not gated) in both."""
    rng = np.random.default_rng(tokens)
    n //= 2 if gated else 1
    n8 = n // 128 * 128
    a, ac, as_ = operand(rng, tokens, d, -6, -4, T)
    wu, wud = experts_weights(rng, experts, n8, d, T)
    wg, wgd = experts_weights(rng, experts, n8, d, T) if gated else (None, None)
    ids = choose(rng, tokens, topk, experts, "part")
    plan = mx.moe_plan(to_dev(ids.astype(np.int32)), experts)
    pairs, ex = rows_of(plan)
    edges = plan.offsets.cpu().numpy()
    some = np.unique(np.clip(np.concatenate((edges, edges - 1, edges + 255, edges + 256, rng.integers(0, len(pairs), 200))), 0,
                             len(pairs) - 1))
    bu = to_dev(rng.standard_normal((experts, n8)).astype(np.float32))
    want, bound = up64(a, wu, wg, bu.double().cpu().numpy(), None, "silu", pairs[some] // topk, ex[some])
    at = torch.from_numpy(some).to(DEV)
    kw = dict(w_gate=wgd, act="silu", bias_up=bu, layout=T, n=n8)
    for out in (F, BF):
        announce("moe_up, large tiles", tokens, topk, experts, d, n8, gated, out)
        y = mx.moe_up(ac, as_, plan, wud, out_dtype=out, **kw)
        check(y[at], want, bound, str(out))
        if out == F:
            exact = y[:len(pairs)].clone()
    yc, ys = mx.moe_up_requant(ac, as_, plan, wud, rot="h32", out_layout=T, **kw)
    qc, qs = mx.quantize_rotate(exact, "h32", layout=T)
    # whole 256-row tiles of the layout
    rows = len(pairs) // 256 * 256
    assert torch.equal(yc[:rows], qc[:rows]) and torch.equal(ys[:rows], qs[:rows])
    if gated:
        return
    h, hc, hs = operand(rng, tokens * topk, d, -6, -4, T)
    weights = torch.rand(tokens, topk, device=DEV)
    residual = torch.randn(tokens, n8, device=DEV)
    slot = plan.slot.cpu().numpy().reshape(tokens, topk)
    some = np.unique(np.concatenate(([0, tokens - 1, tokens // 2], rng.integers(0, tokens, 100))))
    want = residual[torch.from_numpy(some).to(DEV)].double().cpu().numpy()
    S, Z = np.abs(want), 0 * want
    for i, t in enumerate(some):
        for j in range(topk):
            if slot[t, j] >= 0:
                q, z = float(weights[t, j]), wu[ids[t, j]] @ h[slot[t, j]] + bu[ids[t, j]].double().cpu().numpy()
                want[i] += q * z
                S[i] += np.abs(q * z)
                Z[i] += q * np.abs(z).reshape(-1, 32).max(1).repeat(32)
    for out in (F, BF):
        announce("moe_down, large tiles", out)
        y = mx.moe_down(hc, hs, plan, weights, wud, bias=bu, residual=residual, out_dtype=out, layout=T, n=n8)
        check(y[torch.from_numpy(some).to(DEV)], want, (topk + 2) * U * S + (2.0 ** -11 * S + 2.0 ** -24 * Z if out == BF else 0), str(out))


def test_up_requant_leaves_rows_behind_the_last():
    rng = np.random.default_rng(3)
    for tokens, topk, experts in ((20, 4, 6), (200, 4, 3), (900, 4, 2)):
        a, ac, as_ = operand(rng, tokens, 256, -6, -4, T)
        _, wud = experts_weights(rng, experts, 256, 256, T)
        ids = choose(rng, tokens, topk, experts, "part")
        plan = mx.moe_plan(to_dev(ids.astype(np.int32)), experts)
        rows = int(plan.offsets[-1])
        yc = torch.full((tokens * topk, 128), 0xA5, dtype=torch.uint8, device=DEV)
        ys = torch.full((tokens * topk, 8), 0x5A, dtype=torch.uint8, device=DEV)
        announce("moe_up_requant border", tokens)
        mx.moe_up_requant(ac, as_, plan, wud, layout=T, n=256, y_codes=yc, y_scales=ys)
        assert 0 < rows < tokens * topk and (yc[rows:] == 0xA5).all() and (ys[rows:] == 0x5A).all()


def down64(h, wd, bias, weights, plan, residual):
    """y and S, the sum of the absolute terms, by token."""
    pairs, ex = rows_of(plan)
    tokens, topk = weights.shape
    n = wd[0].shape[0]
    y = np.zeros((tokens, n)) if residual is None else residual.copy()
    S, Z = np.abs(y), np.zeros((tokens, n))
    for e in np.unique(ex):
        at = np.flatnonzero(ex == e)
        z = h[at] @ wd[e].T
        if bias is not None:
            z = z + bias[e]
        w = weights.reshape(-1)[pairs[at], None]
        np.add.at(y, pairs[at] // topk, w * z)
        np.add.at(S, pairs[at] // topk, np.abs(w * z))
        # the largest of each block of 32 columns
        top = np.abs(z)
        pad = np.pad(top, ((0, 0), (0, -n % 32))).reshape(len(at), -1, 32).max(-1).repeat(32, 1)[:, :n]
        np.add.at(Z, pairs[at] // topk, np.abs(w) * pad)
    return y, S, Z


DOWN = [(1, 1, 1, 128, 128), (1, 2, 8, 1024, 96), (5, 3, 3, 96, 40), (40, 3, 10, 160, 1000), (64, 4, 16, 512, 64),
        (61, 4, 12, 384, 300), (100, 3, 8, 1152, 33), (300, 2, 5, 256, 300), (300, 2, 5, 128, 288), (700, 3, 4, 640, 520),
        (700, 3, 4, 640, 544), (1100, 2, 3, 1280, 515), (2600, 2, 3, 128, 320),
        (150, 2, 4, 64, 200), (400, 2, 3, 1184, 224), (1500, 2, 4, 416, 160),
        (60, 4, 48, 256, 200), (60, 4, 48, 96, 33),
        # few pairs and a wide result: products and sum in one launch, with K in parts and whole
        (1, 1, 1, 128, 4096), (1, 2, 8, 2048, 4096), (5, 3, 4, 160, 4100), (16, 8, 128, 384, 3200), (128, 1, 16, 128, 7300)]


@pytest.mark.parametrize("layout", [R, T])
@pytest.mark.parametrize("tokens,topk,experts,k,n", DOWN)
def test_down(tokens, topk, experts, k, n, layout):
    if layout == T and k % 128:
        pytest.skip("tiled needs k % 128 == 0")
    rng = np.random.default_rng(tokens + n)
    h, hc, hs = operand(rng, tokens * topk, k, -6, -4, layout)
    wd, wdd = experts_weights(rng, experts, n, k, layout)
    for i, how in enumerate(("even", "skewed", "part")):
        ids = choose(rng, tokens, topk, experts, how)
        plan = mx.moe_plan(to_dev(ids.astype(np.int32)), experts)
        weights = to_dev(rng.standard_normal((tokens, topk)).astype(np.float32))
        if how == "part":
            weights[to_dev(ids) < 0] = float("nan")                 # not read
        bias = to_dev(rng.standard_normal((experts, n)).astype(np.float32)).to((F, BF)[i % 2]) if i else None
        for res_dtype, out in ((None, F), (BF, BF), (F, BF), (BF, F)):
            residual = None if res_dtype is None else \
                to_dev(rng.standard_normal((tokens, n + 3)).astype(np.float32)).to(res_dtype)[:, :n]
            want, S, Z = down64(h, wd, None if bias is None else bias.double().cpu().numpy(),
                                np.nan_to_num(weights.double().cpu().numpy()), plan,
                                None if residual is None else residual.double().cpu().numpy())
            bound = (topk + 2) * U * S + (2.0 ** -11 * S + 2.0 ** -24 * Z if out == BF else 0)
            announce("moe_down", tokens, topk, experts, k, n, layout, how, res_dtype, out)
            y = torch.full((tokens + 1, n + 5), 77.0, dtype=out, device=DEV)
            mx.moe_down(hc, hs, plan, weights, wdd, bias=bias, residual=residual, y=y[:tokens, :n], layout=layout, n=n)
            check(y[:tokens, :n], want, bound, f"{how} {res_dtype} {out}")
            assert (y[tokens:] == 77).all() and (y[:, n:] == 77).all()
            z = mx.moe_down(hc, hs, plan, weights, wdd, bias=bias, residual=residual, out_dtype=out, layout=layout, n=n)
            assert torch.equal(z, y[:tokens, :n])
            if residual is not None and res_dtype == out:              # in place
                r = residual.clone()
                mx.moe_down(hc, hs, plan, weights, wdd, bias=bias, residual=r, y=r, layout=layout, n=n)
                assert torch.equal(r, z)


def test_down_of_a_token_without_experts_is_its_residual():
    rng = np.random.default_rng(9)
    for tokens, experts in ((6, 4), (600, 3)):
        _, hc, hs = operand(rng, tokens * 2, 128, -6, -4, T)
        _, wdd = experts_weights(rng, experts, 256, 128, T)
        ids = rng.integers(0, experts, (tokens, 2)).astype(np.int32)
        ids[3] = -1
        plan = mx.moe_plan(to_dev(ids), experts)
        residual = torch.randn(tokens, 256, device=DEV).to(BF)
        weights = torch.rand(tokens, 2, device=DEV)
        announce("moe_down, empty rows", tokens)
        y = mx.moe_down(hc, hs, plan, weights, wdd, residual=residual, layout=T)
        assert torch.equal(y[3], residual[3]) and not torch.equal(y[2], residual[2])
        y = mx.moe_down(hc, hs, plan, weights, wdd, layout=T)
        assert (y[3] == 0).all()
        nobody = mx.moe_plan(to_dev(np.full((tokens, 2), -1, np.int32)), experts)
        assert torch.equal(mx.moe_down(hc, hs, nobody, weights, wdd, residual=residual, layout=T), residual)


@pytest.mark.parametrize("e", [-110, 100])
def test_down_far_scales(e):
    """Products near both ends of fp32's range keep their precision in the 16-bit
    form, and a NaN scale of a weight reaches its own column only.  The weights'
    blocks differ by up to 2^21, so the fp32 sums over K round too: K / 64 + 4
    times an ulp of the absolute terms at most."""
    rng = np.random.default_rng(10)
    tokens, topk, experts, k, n = 300, 2, 3, 128, 256
    c, s = workloads.random_mxfp4(rng, tokens * topk, k, e, e)
    h = oracle.dequantize(c, s)
    c, s = (to_dev(t) for t in mx.tile_host(c, s))
    w = [workloads.random_mxfp4(rng, n, k, -20, 1) for _ in range(experts)]
    wd = [oracle.dequantize(*x) for x in w]
    tw = [mx.tile_host(*x) for x in w]
    wdd = (to_dev(np.stack([x[0] for x in tw])), to_dev(np.stack([x[1] for x in tw])))
    plan = mx.moe_plan(to_dev(rng.integers(0, experts, (tokens, topk)).astype(np.int32)), experts)
    weights = torch.rand(tokens, topk, device=DEV)
    w64 = weights.double().cpu().numpy()
    want, S, Z = down64(h, wd, None, w64, plan, None)
    pairs, ex = rows_of(plan)
    mag = np.zeros_like(S)
    for x in range(experts):
        at = np.flatnonzero(ex == x)
        np.add.at(mag, pairs[at] // topk, w64.reshape(-1)[pairs[at], None] * (np.abs(h[at]) @ np.abs(wd[x]).T))
    bound = (topk + 2) * U * S + 2.0 ** -11 * S + 2.0 ** -24 * Z + 2 * (k / 64 + 4) * U * mag
    announce("moe_down, exponent", e)
    check(mx.moe_down(c, s, plan, weights, wdd, layout=T), want, bound, f"2^{e}")
    sc = wdd[1].clone()
    sc[0, 5, 2] = 0xFF                                                 # expert 0, row 5 (one tile, one stage)
    y = mx.moe_down(c, s, plan, weights, (wdd[0], sc), layout=T)
    keep = np.arange(n) != 5
    assert torch.isnan(y[:, 5]).any()
    check(y[:, torch.from_numpy(keep)], want[:, keep], bound[:, keep], "beside NaN")


def test_down_infinite_products():
    """A product that leaves fp32's range reaches its own element only, in the
    16-bit form too."""
    rng = np.random.default_rng(11)
    tokens, topk, experts, k, n = 300, 2, 2, 128, 256
    c, s = workloads.random_mxfp4(rng, tokens * topk, k, -6, -4)
    h = oracle.dequantize(c, s)
    w = [workloads.random_mxfp4(rng, n, k, -1, 1) for _ in range(experts)]
    wd = [oracle.dequantize(*x) for x in w]
    for x in w:                                       # column 70: products of some 2^127 and more
        x[1][70] = 254
    col = [oracle.dequantize(*x)[70] for x in w]
    tw = [mx.tile_host(*x) for x in w]
    wdd = (to_dev(np.stack([x[0] for x in tw])), to_dev(np.stack([x[1] for x in tw])))
    c, s = (to_dev(t) for t in mx.tile_host(c, s))
    plan = mx.moe_plan(to_dev(rng.integers(0, experts, (tokens, topk)).astype(np.int32)), experts)
    weights = torch.ones(tokens, topk, device=DEV)
    want, S, Z = down64(h, wd, None, weights.double().cpu().numpy(), plan, None)
    announce("moe_down, infinities")
    y = mx.moe_down(c, s, plan, weights, wdd, layout=T)
    keep = np.arange(n) != 70
    other = (torch.arange(n) // 32 == 70 // 32).numpy()
    assert torch.isinf(y[:, 70].float()).any()
    near = keep & other                                # the block's other columns: held beside numbers of 2^127
    far = keep & ~other
    check(y[:, torch.from_numpy(far)], want[:, far], ((topk + 2) * U * S + 2.0 ** -11 * S + 2.0 ** -24 * Z)[:, far], "other blocks")
    both = np.ones(tokens, bool)                       # tokens whose every product in column 70 is infinite
    order, ex = rows_of(plan)
    z = np.array([h[p] @ col[e] for p, e in enumerate(ex)])
    np.logical_and.at(both, order // topk, np.abs(z) > 3.5e38)
    assert both.any()
    sel = np.ix_(both, near)
    check(y[torch.from_numpy(both)][:, torch.from_numpy(near)], want[sel], ((topk + 2) * U * S + 2.0 ** -11 * S + 2.0 ** -24 * Z)[sel],
          "beside infinities")


def test_rows_past_4_gib():
    """Results and products whose byte offsets pass 32 bits, on a sample of rows."""
    rng = np.random.default_rng(12)
    tokens, topk, experts, k, n = 36000, 8, 24, 128, 4096
    a, ac, as_ = operand(rng, tokens, k, -6, -4, T)
    w, wd = experts_weights(rng, experts, n, k, T)
    ids = np.stack([rng.permutation(experts)[:topk] for _ in range(tokens)]).astype(np.int32)
    plan = mx.moe_plan(to_dev(ids), experts)
    pairs, ex = rows_of(plan)
    some = np.unique(np.concatenate(([0, 1, len(pairs) - 1, len(pairs) - 2], rng.integers(0, len(pairs), 60),
                                     rng.integers(2 ** 32 // (4 * n), len(pairs), 60))))
    want = np.stack([w[ex[p]] @ a[pairs[p] // topk] for p in some])
    for out in (F, BF):
        announce("moe_up past 4 GiB", out)
        y = mx.moe_up(ac, as_, plan, wd, act="none", out_dtype=out, layout=T, n=n)
        assert y.numel() * y.element_size() > (2 ** 32 if out == F else 2 ** 31)
        check(y[torch.from_numpy(some).to(DEV)], want, 0 * want, str(out))
        del y
    hc, hs = workloads.random_mxfp4(rng, tokens * topk, k, -6, -4)
    slot = plan.slot.cpu().numpy().reshape(tokens, topk)
    some = np.unique(np.concatenate(([0, tokens - 1], rng.integers(0, tokens, 40))))
    weights = torch.rand(tokens, topk, device=DEV)
    want, S, Z = np.zeros((len(some), n)), np.zeros((len(some), n)), np.zeros((len(some), n))
    for i, t in enumerate(some):
        for j in range(topk):
            z = w[ids[t, j]] @ oracle.dequantize(hc[slot[t, j]][None], hs[slot[t, j]][None])[0]
            q = float(weights[t, j])
            want[i] += q * z
            S[i] += np.abs(q * z)
            Z[i] += q * np.abs(z).reshape(-1, 32).max(1).repeat(32)
    tc, ts = (to_dev(x) for x in mx.tile_host(hc, hs))
    for out in (F, BF):
        announce("moe_down past 4 GiB", out)
        y = mx.moe_down(tc, ts, plan, weights, wd, out_dtype=out, layout=T, n=n)
        check(y[torch.from_numpy(some).to(DEV)], want, (topk + 2) * U * S + (2.0 ** -11 * S + 2.0 ** -24 * Z if out == BF else 0), str(out))


# ---------------------------------------------------------------------------
# the block


def block(rng, tokens, experts, topk, d, f, layout, gated=True, h32=True):
    rot = mx.HADAMARD32 if h32 else None
    dev = lambda *s: to_dev(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    x = dev(tokens, d).to(BF)
    logits = dev(tokens, experts)
    up, gate = (mx.quantize_experts(dev(experts, f, d) * 0.05, rot, layout=layout) for _ in range(2))
    down = mx.quantize_experts(dev(experts, d, f) * 0.05, rot, layout=layout)
    return dict(x=x, logits=logits, w_up=up, w_down=down, hidden=f, w_gate=gate if gated else None, rot=rot, layout=layout)


def chain(b, r, act, residual, first=0, experts=None, biases=(None, None, None), out_dtype=None):
    """The block by its parts."""
    ids, w = mx.moe_route(b["logits"], r)
    experts = b["w_up"][0].shape[0]
    plan = mx.moe_plan(ids, experts, first)
    ac, as_ = mx.quantize_rotate(b["x"], b["rot"], layout=b["layout"])
    hc, hs = mx.moe_up_requant(ac, as_, plan, b["w_up"], b["w_gate"], act, biases[0], biases[1], b["rot"], b["layout"],
                               b["layout"], n=b["hidden"])
    return mx.moe_down(hc, hs, plan, w, b["w_down"], biases[2], residual, out_dtype or BF, layout=b["layout"],
                       n=b["x"].shape[1]), (ids, w, plan, ac, as_, hc, hs)


@pytest.mark.parametrize("tokens,experts,topk,d,f,layout", [
    (1, 8, 2, 512, 256, T), (4, 16, 4, 256, 384, T), (33, 6, 3, 160, 96, R), (64, 32, 8, 256, 128, T), (300, 5, 2, 384, 256, T),
    (1200, 4, 2, 256, 384, T), (1200, 4, 2, 256, 384, R)])
def test_ffn_equals_its_parts(tokens, experts, topk, d, f, layout):
    rng = np.random.default_rng(tokens)
    b = block(rng, tokens, experts, topk, d, f, layout, gated=tokens != 33, h32=tokens != 4)
    r = mx.Router(topk, "sigmoid", bias_of(experts), renormalize=tokens != 64)
    residual = torch.randn(tokens, d, device=DEV).to(BF)
    vec = lambda *s: to_dev(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    biases = (None, None, None) if tokens < 64 else (vec(experts, f), vec(experts, f), vec(experts, d))
    announce("moe_ffn", tokens, experts, topk, d, f, layout)
    want, parts = chain(b, r, "silu", residual, biases=biases)
    y = mx.moe_ffn(**{k: b[k] for k in b if k not in ("x", "logits")}, x=b["x"], logits=b["logits"], r=r,
                   residual=residual, bias_up=biases[0], bias_gate=biases[1], bias_down=biases[2])
    assert y.dtype == BF and torch.equal(y, want)
    # without a residual, in fp32
    want, _ = chain(b, r, "silu", None, biases=biases, out_dtype=F)
    y = mx.moe_ffn(**{k: b[k] for k in b if k not in ("x", "logits")}, x=b["x"], logits=b["logits"], r=r, out_dtype=F,
                   bias_up=biases[0], bias_gate=biases[1], bias_down=biases[2])
    assert torch.equal(y, want)


def bias_of(E, seed=0):
    return (0.3 * torch.randn(E, generator=torch.Generator().manual_seed(seed))).to(DEV)


def test_ffn_over_parts_of_the_experts_adds_up():
    """Two halves of the experts, as two GPUs hold them: the second one's residual
    is the first one's result (fp32: one more rounding)."""
    rng = np.random.default_rng(2)
    for tokens in (5, 400):
        b = block(rng, tokens, 8, 3, 256, 256, T)
        r = mx.Router(3)
        kw = dict(x=b["x"], logits=b["logits"], r=r, hidden=256, rot=b["rot"], layout=T, out_dtype=F)
        whole = mx.moe_ffn(w_up=b["w_up"], w_gate=b["w_gate"], w_down=b["w_down"], **kw)
        half = lambda w, i: tuple(t[4 * i:4 * i + 4].contiguous() for t in w)  # noqa: E731
        y = None
        for i in range(2):
            y = mx.moe_ffn(w_up=half(b["w_up"], i), w_gate=half(b["w_gate"], i), w_down=half(b["w_down"], i), first=4 * i,
                           residual=y, **kw)
        top = whole.abs().amax()
        assert (y - whole).abs().amax() <= 8 * 4 * U * top              # 4 roundings of partial sums a few times the result


def test_ffn_against_64_bits():
    """Routing, both products and the sum from the definition, on the hidden
    codes that the device wrote."""
    rng = np.random.default_rng(4)
    for tokens, experts, topk in ((7, 6, 2), (500, 6, 2)):
        b = block(rng, tokens, experts, topk, 256, 384, R)
        r = mx.Router(topk, "softmax")
        residual = torch.randn(tokens, 256, device=DEV).to(BF)
        y, (ids, w, plan, ac, as_, hc, hs) = chain(b, r, "silu", residual)
        pairs, ex = rows_of(plan)
        val = lambda t: [oracle.dequantize(t[0][e].cpu().numpy(), t[1][e].cpu().numpy()) for e in range(experts)]  # noqa: E731
        a = oracle.dequantize(ac.cpu().numpy(), as_.cpu().numpy())
        h = oracle.dequantize(hc.cpu().numpy(), hs.cpu().numpy())
        p = torch.softmax(b["logits"].double(), -1).cpu().numpy()
        assert np.array_equal(ids.cpu().numpy(), np.argsort(-p, axis=1, kind="stable")[:, :topk])
        pw = np.take_along_axis(p, ids.cpu().numpy().astype(np.int64), 1)
        pw /= pw.sum(1, keepdims=True)
        want, S, Z = down64(h, val(b["w_down"]), None, pw, plan, residual.double().cpu().numpy())
        mag = np.abs(h) @ np.abs(np.stack(val(b["w_down"]))).max(0).T     # no row's absolute sums are larger
        big = np.zeros_like(S)
        np.add.at(big, pairs // topk, mag)
        check(y, want, (topk + 2) * U * S + 2.0 ** -11 * S + 2.0 ** -24 * Z + 2 * (384 / 64 + 4) * U * big, "ffn")
        # the hidden activations: within half an E2M1 step (a quarter of the block's power of two ..) of the formula
        want, bound = up64(a, val(b["w_up"]), val(b["w_gate"]), None, None, "silu", pairs // topk, ex)
        i = np.arange(32)
        sign = 1 - 2 * (np.array([[bin(x & y).count("1") for y in i] for x in i]) & 1)
        rotated = (want.reshape(-1, 32) @ sign / np.sqrt(32.0)).reshape(want.shape)
        blocks = np.abs(rotated).reshape(len(rotated), -1, 32).max(-1)
        step = 2.0 ** np.floor(np.log2(blocks)) / 4                        # the block's scale; E2M1 steps up to 2 of it, 6 at most
        assert (np.abs(h - rotated) <= 2.05 * np.repeat(step, 32, 1)).all()


def test_ffn_captured_and_replayed():
    rng = np.random.default_rng(5)
    for tokens in (4, 700):
        b = block(rng, tokens, 8, 2, 256, 256, T)
        r = mx.Router(2, "sigmoid", bias_of(8), 4, 2, "top2")
        x, logits = b["x"].clone(), b["logits"].clone()
        residual = torch.randn(tokens, 256, device=DEV).to(BF)
        y = torch.empty_like(residual)
        call = lambda: mx.moe_ffn(x, logits, r, b["w_up"], b["w_down"], 256, b["w_gate"], rot="h32", residual=residual,  # noqa: E731
                                  layout=T, y=y)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        for rep in range(4):
            x.copy_(torch.from_numpy(rng.standard_normal((tokens, 256)).astype(np.float32)))
            logits.copy_(torch.from_numpy(rng.standard_normal((tokens, 8)).astype(np.float32)))
            if rep == 2:
                logits[:, 1:] = -float("inf")                            # one expert takes all
            want, _ = chain({**b, "x": x, "logits": logits}, r, "silu", residual)
            y.fill_(float("nan"))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want), f"replay {rep} of {tokens} tokens"


def test_two_streams_at_once():
    """Blocks of different inputs on two streams, each with its own plan and workspace."""
    rng = np.random.default_rng(6)
    b = [block(rng, n, 8, 2, 256, 256, T) for n in (300, 40)]
    r = mx.Router(2)
    want = [chain(x, r, "silu", None)[0] for x in b]
    streams = [torch.cuda.Stream() for _ in b]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mx.moe_ffn(b[i]["x"], b[i]["logits"], r, b[i]["w_up"], b[i]["w_down"], 256, b[i]["w_gate"],
                                         rot="h32", layout=T))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_empty_batch():
    rng = np.random.default_rng(7)
    b = block(rng, 3, 4, 2, 256, 256, T)
    r = mx.Router(2)
    y = mx.moe_ffn(b["x"][:0], b["logits"][:0], r, b["w_up"], b["w_down"], 256, b["w_gate"], rot="h32", layout=T)
    assert y.shape == (0, 256)
    plan = mx.moe_plan(torch.zeros(0, 2, dtype=torch.int32, device=DEV), 4)
    none = torch.zeros(0, 128, dtype=torch.uint8, device=DEV), torch.zeros(0, 8, dtype=torch.uint8, device=DEV)
    assert mx.moe_up(*none, plan, b["w_up"], b["w_gate"], layout=T).shape == (0, 256)
    assert mx.moe_down(*none, plan, torch.zeros(0, 2, device=DEV), b["w_down"], layout=T).shape == (0, 256)
