"""Experts' products of row-major operands with several tiles a workgroup: the tile
kernel for K a multiple of 32 (its ring runs from one tile into the next, of
another expert), and both heights of the others.  Exact sums, as test_gpu_moe.py
derives them; a sample of rows, the first and last of each expert and of row tiles
among them, with all columns."""
import numpy as np
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx
from test_gpu_moe import BF, DEV, F, R, U, announce, check, choose, experts_weights, operand, rows_of, to_dev, up64

pytestmark = pytest.mark.gpu

# K of one stage and of two (rows asked for as the ring reaches them), of three and
# four (two tiles ahead), each a tail; then whole stages.  Tiles of 128 x 128: 27 x 80
# and more on 512 workgroups; gated, half the columns each.  The last two: 256 x 256.
CASES = [(1500, 2, 3, 32, 10240), (1500, 2, 3, 96, 10240), (1500, 2, 3, 160, 10240), (1500, 2, 3, 352, 10240),
         (1200, 3, 4, 416, 8000), (1500, 2, 3, 128, 10240), (1000, 3, 3, 384, 8224), (3000, 2, 2, 768, 12900),
         (2100, 2, 5, 1280, 12900)]


def sample(rng, plan, rows):
    edges = plan.offsets.cpu().numpy()
    near = [edges + d for d in (-129, -128, -1, 0, 1, 127, 128, 255, 256)]
    return np.unique(np.clip(np.concatenate(near + [rng.integers(0, rows, 150)]), 0, rows - 1))


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("tokens,topk,experts,d,n", CASES)
def test_up_row_major_tiles(tokens, topk, experts, d, n, gated):
    rng = np.random.default_rng(tokens + d)
    n = n // 2 // 32 * 32 if gated else n // 32 * 32
    a, ac, as_ = operand(rng, tokens, d, -6, -4, R)
    wu, wud = experts_weights(rng, experts, n, d, R)
    wg, wgd = experts_weights(rng, experts, n, d, R) if gated else (None, None)
    for how in ("part", "skewed"):
        plan = mx.moe_plan(to_dev(choose(rng, tokens, topk, experts, how).astype(np.int32)), experts)
        pairs, ex = rows_of(plan)
        some = sample(rng, plan, len(pairs))
        bu = to_dev(rng.standard_normal((experts, n)).astype(np.float32))
        want, bound = up64(a, wu, wg, bu.double().cpu().numpy(), None, "silu", pairs[some] // topk, ex[some])
        at = torch.from_numpy(some).to(DEV)
        kw = dict(w_gate=wgd, act="silu", bias_up=bu, n=n)
        for out in (F, BF):
            announce("moe_up, row-major tiles", tokens, topk, experts, d, n, gated, how, out)
            y = mx.moe_up(ac, as_, plan, wud, out_dtype=out, **kw)
            check(y[at], want, bound, f"{how} {out}")
            if out == F:
                exact = y[:len(pairs)].clone()
        yc, ys = mx.moe_up_requant(ac, as_, plan, wud, rot="h32", **kw)
        qc, qs = mx.quantize_rotate(exact, "h32")
        assert torch.equal(yc[:len(pairs)], qc) and torch.equal(ys[:len(pairs)], qs)


@pytest.mark.parametrize("tokens,topk,experts,k,n", CASES)
def test_down_row_major_tiles(tokens, topk, experts, k, n):
    rng = np.random.default_rng(tokens + k + 1)
    h, hc, hs = operand(rng, tokens * topk, k, -6, -4, R)
    wd, wdd = experts_weights(rng, experts, n, k, R)
    ids = choose(rng, tokens, topk, experts, "part")
    plan = mx.moe_plan(to_dev(ids.astype(np.int32)), experts)
    weights, residual = torch.rand(tokens, topk, device=DEV), torch.randn(tokens, n, device=DEV)
    slot = plan.slot.cpu().numpy().reshape(tokens, topk)
    some = np.unique(np.concatenate(([0, tokens - 1, tokens // 2], rng.integers(0, tokens, 120))))
    want = residual[torch.from_numpy(some).to(DEV)].double().cpu().numpy()
    S, Z = np.abs(want), 0 * want
    for i, t in enumerate(some):
        for j in range(topk):
            if slot[t, j] >= 0:
                q, z = float(weights[t, j]), wd[ids[t, j]] @ h[slot[t, j]]
                want[i] += q * z
                S[i] += np.abs(q * z)
                Z[i] += q * np.pad(np.abs(z), (0, -n % 32)).reshape(-1, 32).max(1).repeat(32)[:n]
    for out in (F, BF):
        announce("moe_down, row-major tiles", tokens, topk, experts, k, n, out)
        y = mx.moe_down(hc, hs, plan, weights, wdd, residual=residual, out_dtype=out)
        check(y[torch.from_numpy(some).to(DEV)], want,
              (topk + 2) * U * S + (2.0 ** -11 * S + 2.0 ** -24 * Z if out == BF else 0), str(out))
