"""Router and expert plan against plain implementations in 64 bits.

Router: scores, keys with a bias and group sums are formed in binary64 by both
sides, so ids have to be equal (inputs are random: no two different keys are
within some 1e-15 of each other); weights are rounded once to fp32, half a step
is 2^-24 of the value.  Plan: whole numbers, all equal."""
import numpy as np
import pytest
import torch

import mxfp4_w4a4_quantized_amd as mx

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F = torch.bfloat16, torch.float32


def announce(*what):
    print("[case]", *what, flush=True)


def route64(logits, r):
    """ids, weights [tokens, topk], one token after the other."""
    x = logits.double().cpu().numpy()
    bias = None if r.bias is None else r.bias.double().cpu().numpy()
    T, E = x.shape
    ids, ws = np.full((T, r.topk), -1), np.zeros((T, r.topk))
    for t in range(T):
        ok = x[t] > -np.inf                                  # NaN: not
        if not ok.any():
            continue
        l = np.where(ok, x[t], 0.0)
        if r.score == "softmax":
            e = np.where(ok, np.exp(np.minimum(l - l[ok].max(), 0.0)), 0.0)
            s = e / e.sum()
        else:
            s = np.where(ok, 1 / (1 + np.exp(-l)), 0.0)
        key = np.where(ok, x[t] if bias is None else s + bias, -np.inf)
        if r.groups > 1:
            by = np.where(key > -np.inf, s if bias is None else key, -np.inf).reshape(r.groups, -1)
            top = -np.sort(-by, axis=1)
            score = top[:, 0].copy()
            if r.group_score == "top2" and top.shape[1] > 1:
                score += np.where(top[:, 1] > -np.inf, top[:, 1], 0.0)
            kept = np.argsort(-score, kind="stable")[:r.topk_groups]
            keep = np.zeros(r.groups, bool)
            keep[kept] = True
            key = np.where(np.repeat(keep, E // r.groups), key, -np.inf)
        best = np.argsort(-key, kind="stable")[:r.topk]
        best = best[key[best] > -np.inf]
        w = s[best]
        if r.renormalize:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        ids[t, :len(best)], ws[t, :len(best)] = best, w * r.scale
    return ids, ws


def check_route(logits, r, what):
    announce("moe_route", what, tuple(logits.shape), logits.dtype)
    ids, w = mx.moe_route(logits, r)
    want, ww = route64(logits, r)
    assert ids.dtype == torch.int32 and w.dtype == F and ids.shape == w.shape == (logits.shape[0], r.topk)
    assert np.array_equal(ids.cpu().numpy(), want), what
    err = np.abs(w.double().cpu().numpy() - ww)
    assert (err <= (2.0 ** -24 + 1e-12) * np.abs(ww) + 1e-45).all(), what
    return ids, w


def bias_of(E, seed=0):
    return (0.3 * torch.randn(E, generator=torch.Generator().manual_seed(seed))).to(DEV)


CASES = [
    # tokens, experts, topk, score, bias, groups, kept, group score, renormalize, scale
    (1, 1, 1, "softmax", False, 1, 1, "max", True, 1.0),
    (5, 8, 2, "softmax", False, 1, 1, "max", True, 1.0),
    (7, 8, 8, "sigmoid", True, 1, 1, "max", False, 2.5),
    (33, 60, 4, "softmax", True, 1, 1, "max", False, 1.0),
    (64, 64, 6, "sigmoid", False, 8, 3, "top2", True, 1.0),
    (65, 65, 7, "softmax", False, 5, 2, "max", True, 0.5),
    (16, 128, 8, "softmax", False, 1, 1, "max", True, 1.0),
    (129, 160, 6, "sigmoid", True, 8, 3, "top2", True, 16.0),
    (40, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5),
    (40, 256, 8, "softmax", False, 8, 4, "max", False, 2.5),
    (11, 300, 10, "softmax", True, 3, 2, "top2", True, 1.0),
    (9, 512, 64, "sigmoid", False, 64, 32, "max", True, 1.0),
    (6, 1024, 33, "softmax", True, 1, 1, "max", True, 1.0),
    (3, 64, 3, "sigmoid", True, 64, 5, "top2", True, 1.0),      # groups of one
    (3050, 48, 4, "softmax", False, 1, 1, "max", True, 1.0),       # 16 and 32 lanes a token
    (3001, 64, 6, "sigmoid", True, 16, 5, "top2", True, 1.0),
    (3003, 100, 16, "softmax", True, 4, 3, "max", False, 1.0),
    (3002, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5),
    (3005, 200, 16, "softmax", False, 40, 11, "max", False, 1.0),
]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("case", CASES)
def test_route(case, dtype):
    T, E, k, score, bias, groups, kept, gs, renorm, scale = case
    gen = torch.Generator().manual_seed(T + E)
    logits = (1.5 * torch.randn(T, E, generator=gen)).to(dtype).to(DEV)
    r = mx.Router(k, score, bias_of(E) if bias else None, groups, kept, gs, renorm, scale)
    check_route(logits, r, str(case))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("bias", [False, True])
def test_route_ties_go_to_the_lowest_index(score, groups, bias):
    gen = torch.Generator().manual_seed(5)
    few = torch.tensor([-1.0, 0.0, 0.5, 2.0])
    logits = few[torch.randint(0, 4, (70, 96), generator=gen)].to(DEV)
    logits[0] = 0.25                                            # every expert alike
    b = few[torch.randint(0, 2, (96,), generator=gen)].to(DEV) if bias else None
    check_route(logits, mx.Router(9, score, b, groups, max(1, groups // 2), "top2"), "ties")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 6])
@pytest.mark.parametrize("bias", [False, True])
def test_route_masked_logits(score, groups, bias):
    """-inf and NaN logits: no candidates; rows with fewer than topk, with one
    and with none; the lowest value of the type is still a candidate."""
    gen = torch.Generator().manual_seed(6)
    for dtype in (BF, F):
        logits = torch.randn(40, 30, generator=gen)
        mask = torch.rand(40, 30, generator=gen) < 0.7
        logits[mask] = -float("inf")
        logits[1] = -float("inf")
        logits[2] = float("nan")
        logits[3] = -float("inf")
        logits[3, 17] = torch.finfo(dtype).min
        logits[4, ::3] = float("nan")
        logits[5] = torch.finfo(dtype).min
        logits[6] = torch.finfo(dtype).max
        b = bias_of(30, 2) if bias else None
        if bias:
            b[4] = -float("inf")
        ids, w = check_route(logits.to(dtype).to(DEV), mx.Router(5, score, b, groups, max(1, groups // 2), "top2"), "masked")
        assert (ids[1] == -1).all() and (w[1] == 0).all() and (ids[2] == -1).all()


def test_route_far_scores():
    """Scores that leave fp32's range, and sums of weights that vanish."""
    logits = torch.tensor([[-120.0, -130.0, -100.0, -400.0], [-900.0, -901.0, -950.0, -1000.0], [90.0, 100.0, -90.0, 0.0],
                           [1e30, -1e30, 0.0, 3.0]], device=DEV)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            check_route(logits, mx.Router(3, score, renormalize=renorm), f"far {score} {renorm}")


def test_route_views_and_streams():
    gen = torch.Generator().manual_seed(7)
    wide = torch.randn(50, 90, generator=gen).to(DEV)
    r = mx.Router(4, "sigmoid", bias_of(64), 8, 4, "top2")
    check_route(wide[:, 7:71], r, "row stride 90")
    check_route(wide[:1, 7:71], r, "one row of a view")
    ids, w = mx.moe_route(wide[:, 7:71], r)
    side = torch.cuda.Stream()
    out, ow = torch.full((50, 4), -7, dtype=torch.int32, device=DEV), torch.zeros(50, 4, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        mx.moe_route(wide[:, 7:71], r, out, ow)
    side.synchronize()
    assert torch.equal(out, ids) and torch.equal(ow, w)
    empty, ew = mx.moe_route(wide[:0, 7:71], r)
    assert empty.shape == ew.shape == (0, 4)


# ---------------------------------------------------------------------------


def plan_ref(ids, experts, first):
    e = ids.astype(np.int64).reshape(-1) - first
    ok = (e >= 0) & (e < experts)
    e = np.where(ok, e, experts)
    order = np.argsort(e, kind="stable")
    n = int(ok.sum())
    offsets = np.concatenate(([0], np.cumsum(np.bincount(e, minlength=experts + 1)[:experts])))
    slot = np.full(e.size, -1)
    slot[order[:n]] = np.arange(n)
    return offsets, np.where(np.arange(e.size) < n, order, -1), slot


def check_plan(ids, experts, first=0, plan=None):
    announce("moe_plan", ids.shape, experts, first)
    plan = mx.moe_plan(torch.from_numpy(ids.astype(np.int32)).to(DEV), experts, first, plan)
    offsets, order, slot = plan_ref(ids, experts, first)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.order.cpu().numpy(), order)
    assert np.array_equal(plan.slot.cpu().numpy(), slot)
    # the part that the products read: tokens of the rows, row tiles of each height
    pairs, topk = ids.size, ids.shape[1]
    words = plan.words.cpu().numpy()
    at = experts + 1 + 2 * pairs
    assert np.array_equal(words[at:at + pairs], np.where(order >= 0, order // topk, 0))
    at = (at + pairs + 3) // 4 * 4
    ntiles, at = words[at:at + 4], at + 8
    for i, h in enumerate((16, 32, 128, 256)):
        counts = np.diff(offsets)
        tiles = -(-counts // h)
        want = [(e, offsets[e], offsets[e + 1], tiles[:e].sum()) for e in range(experts) for _ in range(tiles[e])]
        assert ntiles[i] == len(want) <= pairs // h + min(experts, pairs)
        got = words[at:at + 4 * len(want)].reshape(-1, 4)
        assert np.array_equal(got, np.array(want).reshape(-1, 4))
        at += 4 * (pairs // h + min(experts, pairs))
    return plan


@pytest.mark.parametrize("tokens,topk,experts", [
    (1, 1, 1), (1, 2, 8), (3, 5, 7), (8, 8, 64), (63, 1, 3), (64, 1, 1024), (65, 1, 65), (64, 8, 128), (100, 41, 33),
    (4095, 1, 16), (4096, 1, 200), (4097, 1, 16), (2049, 2, 1024), (3000, 3, 5), (8192, 8, 64), (40000, 5, 256)])
def test_plan(tokens, topk, experts):
    rng = np.random.default_rng(tokens + experts)
    check_plan(rng.integers(0, experts, (tokens, topk)), experts)


@pytest.mark.parametrize("tokens,topk", [(40, 3), (3000, 4), (70000, 2)])
def test_plan_of_a_part_of_the_experts(tokens, topk):
    rng = np.random.default_rng(tokens)
    ids = rng.integers(0, 96, (tokens, topk))
    ids[rng.random(ids.shape) < 0.1] = -1
    ids[0, 0], ids[-1, -1] = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    for first, experts in ((0, 96), (0, 31), (31, 40), (95, 1), (96, 5), (2 ** 30 - 1, 1024)):
        check_plan(ids, experts, first)
    check_plan(np.full((tokens, topk), -1), 4)                      # nobody
    check_plan(np.full((tokens, topk), 2), 5)                       # one expert takes all, twice and more per token


def test_plan_written_again():
    rng = np.random.default_rng(1)
    plan = check_plan(rng.integers(0, 64, (2000, 4)), 64)
    for seed in range(3):
        ids = np.random.default_rng(seed).integers(-5, 64, (2000, 4))
        check_plan(ids, 64, plan=plan)
    with pytest.raises(ValueError, match="plan"):
        mx.moe_plan(torch.zeros(1999, 4, dtype=torch.int32, device=DEV), 64, plan=plan)


def test_plan_without_tokens():
    plan = mx.moe_plan(torch.zeros(0, 4, dtype=torch.int32, device=DEV), 6)
    assert plan.offsets.tolist() == [0] * 7 and plan.order.numel() == plan.slot.numel() == 0
