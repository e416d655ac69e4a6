"""Cases that measure the mixture-of-experts operators of the MXFP4 library: the
router, the plan that sorts (token, choice) pairs by expert, the experts' gated
up projection, their down projection with the weighted sum over a token's
choices, and the feed-forward path that chains them.

A case is a dict of plain values.  "op" names the operator:
  route  ids, weights = the topk experts of each token, from router logits
  plan   offsets, order, slot: the pairs in expert order (stable), and back
  up     H = act(A G_e^T + bg_e) * (A U_e^T + bu_e) for each pair, in expert
         order, from the tokens' packed activations (and the plan for its ids)
  down   y = residual + sum over a token's choices of weight * (h D_e^T), from
         packed hidden activations in expert order (and the plan)
  ffn    dense activations -> MXFP4, route, plan, up (MXFP4), down
Packed operands are E2M1 codes (two per byte) and one E8M0 byte per 32 elements
along K.  Expert weights are kept row-major and, where K allows it, in the
library's 256-row tiled layout, as a serving program lays its weights out once.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BF16, F32 = torch.bfloat16, torch.float32

ROUTER = dict(tokens=1, experts=8, topk=2, score="softmax", bias=False, groups=1, topk_groups=1, group_score="max",
              renorm=True, scale=1.0, bf16=True)


def _case(op, name, **kw):
    base = {"route": {}, "plan": dict(first=0, local=0), "up": dict(d=128, f=128, act="silu", biases=False, out_f32=False),
            "down": dict(d=128, f=128, biases=False, residual=True, out_f32=False),
            "ffn": dict(d=128, f=128, act="silu", h32=True, residual=True)}[op]
    return {"name": name, "op": op, **ROUTER, **base, **kw}


GROUPED = dict(score="sigmoid", bias=True, groups=8, topk_groups=4, group_score="top2", scale=2.5, bf16=False)


def listed():
    return [
        # --- route
        # a decode batch: launch latency
        _case("route", "route_decode_16x128", tokens=16, experts=128, topk=8),
        # a long prompt through a router with a balance bias and expert groups
        _case("route", "route_prompt_8192x256", tokens=8192, experts=256, topk=8, **GROUPED),
        # --- plan
        # a decode batch
        _case("plan", "plan_decode_64x8_128", tokens=64, experts=128, topk=8),
        # several long prompts on one of four GPUs that share the experts
        _case("plan", "plan_prompt_32768x8_256", tokens=32768, experts=256, topk=8, first=64, local=64),
        # --- the experts' gated up projection
        # a decode batch that reaches most experts: their weights streamed once
        _case("up", "up_decode_16x4096_2048_e128", tokens=16, experts=128, topk=8, d=4096, f=2048),
        # ragged prompt, odd widths (K not of 128), biases, 32-bit output
        _case("up", "up_odd_301x1184_1000_e10", tokens=301, experts=10, topk=3, d=1184, f=1000, act="gelu_tanh",
              biases=True, out_f32=True),
        # a long prompt
        _case("up", "up_prompt_8192x4096_2048_e64", tokens=8192, experts=64, topk=8, d=4096, f=2048),
        # --- the experts' down projection and the sum over a token's choices
        # one token through two wide experts
        _case("down", "down_token_1x14336_4096_e8", tokens=1, experts=8, topk=2, d=4096, f=14336),
        # a long prompt
        _case("down", "down_prompt_8192x2048_4096_e64", tokens=8192, experts=64, topk=8, d=4096, f=2048),
        # --- the path
        # one decode step of 4 sequences, wide experts
        _case("ffn", "ffn_decode_4x4096_14336_e8", tokens=4, experts=8, topk=2, d=4096, f=14336),
        # one decode step of 64 sequences, many narrow experts
        _case("ffn", "ffn_decode_64x4096_2048_e128", tokens=64, experts=128, topk=8, d=4096, f=2048),
        # a prompt through grouped routing
        _case("ffn", "ffn_prompt_4096x2048_1408_e64", tokens=4096, experts=64, topk=6, d=2048, f=1408, **GROUPED),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "plan", "up", "down", "ffn"))
    yes = lambda p=0.5: rng.random() < p  # noqa: E731
    groups = rng.choice((1, 1, 2, 4, 8))
    per = _log_int(rng, max(2, 8 // groups), max(3, (384 if op in ("route", "plan") else 128) // groups))
    experts = groups * per
    kept = rng.randint((groups + 1) // 2, groups)
    topk = rng.randint(1, min(8, kept * per))
    r = dict(experts=experts, topk=topk, groups=groups, topk_groups=kept, score=rng.choice(("softmax", "sigmoid")),
             bias=yes(), group_score=rng.choice(("max", "top2")), renorm=yes(0.8), scale=rng.choice((1.0, 2.5)),
             bf16=yes())
    if op in ("route", "plan"):
        r["tokens"] = _log_int(rng, 1, 32768 if op == "plan" else max(16, min(32768, 8192 * 256 // experts)))
        if op == "plan" and yes():
            r["local"] = rng.randint(1, experts)
            r["first"] = rng.randint(0, experts - r["local"])
        c = _case(op, "", **r)
    else:
        unit = 128 if op == "ffn" or yes(0.8) else 32
        d, f = unit * _log_int(rng, 512 // unit, 4096 // unit), unit * _log_int(rng, 512 // unit, 4096 // unit)
        # weights no larger than the largest listed case's, rows no more than the long prompt's
        experts = max(groups * 2, min(experts, 3 * 128 * 2048 * 4096 // (3 * d * f)) // groups * groups)
        rows = min(65536, 65536 * 2048 * 4096 // (d * f))
        r.update(experts=experts, topk=min(topk, kept * (experts // groups)))
        r["tokens"] = _log_int(rng, 1, max(2, min(8192, rows // r["topk"] // (2 if op == "ffn" else 1))))
        kw = {"up": dict(act=rng.choice(("silu", "gelu", "gelu_tanh", "relu")), biases=yes(0.3), out_f32=yes(0.3)),
              "down": dict(biases=yes(0.3), residual=yes(), out_f32=yes(0.3)),
              "ffn": dict(act=rng.choice(("silu", "gelu_tanh")), h32=yes(), residual=yes())}[op]
        c = _case(op, "", d=d, f=f, **r, **kw)
    return {k: v for k, v in c.items() if k != "name"}


# ---------------------------------------------------------------------------
# packed operands


def _encode(y):
    """E2M1 codes (0..15, one per byte) and E8M0 bytes of y [rows, k]."""
    rows, k = y.shape
    b = y.reshape(rows, k // 32, 32)
    _, ex = torch.frexp(b.abs().amax(-1))          # amax = f * 2^ex, f in [0.5, 1): floor(log2) = ex - 1
    e = (ex - 3).clamp(min=-126)
    t = torch.ldexp(b.abs(), -e[..., None])
    i = (t > 0.25).to(torch.uint8) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5)
    return (i | (torch.signbit(b).to(torch.uint8) << 3)).reshape(rows, k), (e + 127).to(torch.uint8)


def _tile(codes, scales):
    """The library's tiled layout: 256-row tiles x 128-element stages, the
    16-byte blocks of a row's stage XOR-permuted by its row number."""
    rows, half = codes.shape
    t, s = (rows + 255) // 256, half // 64
    c = torch.zeros((t * 256, half), dtype=torch.uint8, device=codes.device)
    sc = torch.zeros((t * 256, half // 16), dtype=torch.uint8, device=codes.device)
    c[:rows], sc[:rows] = codes, scales
    r = torch.arange(256, device=codes.device)
    at = torch.arange(4, device=codes.device)[None, :] ^ (((r >> 1) ^ (r >> 2)) & 3)[:, None]
    c = c.view(t, 256, s, 4, 16).permute(0, 2, 1, 3, 4)
    c = torch.take_along_dim(c, at.view(1, 1, 256, 4, 1).expand(t, s, 256, 4, 16), 3)
    sc = sc.view(t, 256, s, 4).permute(0, 2, 1, 3)
    return c.reshape(t * 256, half).contiguous(), sc.reshape(t * 256, half // 16).contiguous()


def _pack(y):
    """Row-major (codes, scales) of y, and the tiled pair where K allows it."""
    code, scales = _encode(y.float())
    row = ((code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), scales.contiguous())
    return {"row": row, "tiled": _tile(*row) if y.shape[1] % 128 == 0 else None}


def _h32(dtype):
    i = torch.arange(32, device=DEV)
    bits = i[:, None] & i[None, :]
    parity = sum((bits >> s) & 1 for s in range(5)) & 1
    return (1 - 2 * parity).to(dtype) / math.sqrt(32.0)


def _rotate(y, h32):
    return (y.reshape(-1, 32) @ _h32(y.dtype)).reshape(y.shape) if h32 else y


def _expert_weights(rnd, experts, n, k, h32):
    """Packed weights of every expert, stacked: [experts, rows, ...]."""
    each = [_pack(_rotate(rnd(n, k) * 0.02, h32)) for _ in range(experts)]
    return {key: None if each[0][key] is None else tuple(torch.stack([w[key][i] for w in each]) for i in range(2))
            for key in ("row", "tiled")}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1_000_003 * (seed + 1))
    rnd = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    c = dict(case)
    t, e, k = c["tokens"], c["experts"], c["topk"]
    # router logits, some experts more liked than others
    s = {"case": c, "logits": (rnd(t, e) + 0.3 * rnd(e)).to(BF16 if c["bf16"] else F32),
         "bias": 0.1 * rnd(e) if c["bias"] else None}
    if c["op"] == "route":
        return s
    if c["op"] in ("plan", "up", "down"):
        s["ids"], s["weights"] = _route(c, s["logits"], s["bias"])
    if c["op"] == "plan":
        return s
    d, f = c["d"], c["f"]
    h32 = c.get("h32", False)
    if c["op"] in ("up", "ffn"):
        s["up"], s["gate"] = (_expert_weights(rnd, e, f, d, h32) for _ in range(2))
    if c["op"] in ("down", "ffn"):
        s["down"] = _expert_weights(rnd, e, d, f, h32)
        s["residual"] = rnd(t, d).to(BF16) if c["residual"] else None
    if c["op"] == "up":
        s["a"] = _pack(rnd(t, d))
        s["bias_up"], s["bias_gate"] = ((0.2 * rnd(e, f)).to(BF16) if c["biases"] else None for _ in range(2))
    elif c["op"] == "down":
        # hidden activations of the pairs in expert order
        s["h"] = _pack(rnd(t * k, f))
        s["bias_down"] = (0.2 * rnd(e, d)).to(BF16) if c["biases"] else None
    else:
        s["x"] = rnd(t, d).to(BF16)
    return s


# ---------------------------------------------------------------------------
# plain forms: 32 bits, one rounding at the end (the choice of experts, where a
# border between two of them decides, and the weights in 64)


def _route(c, logits, bias):
    x = logits.double()
    if c["score"] == "softmax":
        s = torch.exp(x - x.amax(-1, keepdim=True))
        s = s / s.sum(-1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-x))
    # without a bias the choice goes by the logits: the scores' order, before any rounding
    by = x if bias is None else s + bias.double()
    if c["groups"] > 1:
        g = (s if bias is None else by).reshape(x.shape[0], c["groups"], -1).sort(dim=-1, descending=True).values
        g = g[..., 0] if c["group_score"] == "max" else g[..., :2].sum(-1)
        best = g.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros_like(g, dtype=torch.bool).scatter_(1, best, True)
        by = torch.where(keep.repeat_interleave(x.shape[1] // c["groups"], 1), by, -math.inf)
    ids = by.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk"]]
    w = torch.gather(s, 1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.int(), (w * c["scale"]).float()


def _plan(ids, first, experts):
    """offsets, order (pairs in expert order, -1 behind the last) and slot (its
    inverse, -1 for pairs of other experts)."""
    e = ids.flatten().long() - first
    e = torch.where((e >= 0) & (e < experts), e, experts)
    counts = e.new_zeros(experts + 1).index_add_(0, e, torch.ones_like(e))
    offsets = torch.cat((e.new_zeros(1), counts[:experts].cumsum(0)))
    by = torch.sort(e, stable=True).indices
    place = torch.arange(e.numel(), device=DEV)
    slot = torch.empty_like(by).scatter_(0, by, place)
    here = offsets[-1]
    return offsets.int(), torch.where(place < here, by, -1).int(), torch.where(slot < here, slot, -1).int()


def _values(codes, scales):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack((lut[byte & 15], lut[byte >> 4]), -1)
    v = pair[codes.int()].reshape(scales.shape[0], scales.shape[1], 32)
    return (v * torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)[..., None]).reshape(
        codes.shape[0], -1)


def _quantized(y):
    """The values that MXFP4 keeps of y."""
    rows, k = y.shape
    b = y.reshape(rows, k // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    _, ex = torch.frexp(amax)
    e = torch.where(amax > 0, (ex - 3).clamp(min=-127), torch.full_like(ex, -127))
    t = torch.ldexp(b.abs(), -e)
    i = ((t > 0.25).int() + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5))
    v = torch.tensor(E2M1, device=y.device, dtype=y.dtype)[i]
    return torch.ldexp(torch.where(torch.signbit(b), -v, v), e).reshape(rows, k)


def _act(name, x):
    if name == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _by_expert(rows, weights, offsets, biases):
    """rows[p] W_e^T + b_e for the rows of each expert, in expert order."""
    out = torch.empty((rows.shape[0], weights[0].shape[1]), device=DEV)
    at = offsets.tolist()
    for e, (i, j) in enumerate(zip(at, at[1:])):
        if j > i:
            out[i:j] = rows[i:j] @ _values(weights[0][e], weights[1][e]).T
            if biases is not None:
                out[i:j] += biases[e].float()
    return out


def _summed(z, slot, weights, residual):
    """residual + sum over a token's choices of weight * z[slot]"""
    t, k = weights.shape
    y = (z[slot.long()].reshape(t, k, -1) * weights[..., None]).sum(1)
    return y if residual is None else y + residual.float()


def _plain(s):
    c = s["case"]
    if c["op"] in ("route", "ffn"):
        ids, weights = _route(c, s["logits"], s["bias"])
        if c["op"] == "route":
            return {"ids": ids, "weights": weights}
    else:
        ids, weights = s["ids"], s["weights"]
    experts = c.get("local", 0) or c["experts"]
    offsets, order, slot = _plan(ids, c.get("first", 0), experts)
    if c["op"] == "plan":
        return {"offsets": offsets, "order": order, "slot": slot}
    token = order.long() // c["topk"]
    if c["op"] in ("up", "ffn"):
        a = _values(*s["a"]["row"]) if c["op"] == "up" else _quantized(_rotate(s["x"].float(), c["h32"]))
        a = a[token]
        h = _act(c["act"], _by_expert(a, s["gate"]["row"], offsets, s.get("bias_gate")))
        h = h * _by_expert(a, s["up"]["row"], offsets, s.get("bias_up"))
        if c["op"] == "up":
            return h.to(F32 if c["out_f32"] else BF16)
        h = _quantized(_rotate(h, c["h32"]))
    else:
        h = _values(*s["h"]["row"])
    y = _summed(_by_expert(h, s["down"]["row"], offsets, s.get("bias_down")), slot, weights, s["residual"])
    return y.to(F32 if c.get("out_f32") else BF16)


# ---------------------------------------------------------------------------
# the library's calls


def _own(s):
    import mxfp4_w4a4_quantized_amd as mx
    c = s["case"]
    if c["op"] in ("route", "ffn"):
        router = mx.Router(topk=c["topk"], score=c["score"], bias=s["bias"], groups=c["groups"],
                           topk_groups=c["topk_groups"], group_score=c["group_score"], renormalize=c["renorm"],
                           scale=c["scale"])
    if c["op"] == "route":
        ids, weights = mx.moe_route(s["logits"], router)
        return {"ids": ids, "weights": weights}
    if c["op"] == "plan":
        plan = mx.moe_plan(s["ids"], c["local"] or c["experts"], first=c["first"])
        return {"offsets": plan.offsets, "order": plan.order, "slot": plan.slot}
    tiled = c["d"] % 128 == 0 and c["f"] % 128 == 0
    layout, key = (mx.TILED, "tiled") if tiled else (mx.ROWMAJOR, "row")
    out = F32 if c.get("out_f32") else BF16
    if c["op"] == "ffn":
        return mx.moe_ffn(s["x"], s["logits"], router, s["up"][key], s["down"][key], c["f"], w_gate=s["gate"][key],
                          act=c["act"], rot=mx.HADAMARD32 if c["h32"] else None, residual=s["residual"],
                          layout=layout)
    plan = mx.moe_plan(s["ids"], c["experts"])
    if c["op"] == "up":
        return mx.moe_up(*s["a"][key], plan, s["up"][key], w_gate=s["gate"][key], act=c["act"],
                         bias_up=s["bias_up"], bias_gate=s["bias_gate"], out_dtype=out, layout=layout, n=c["f"])
    return mx.moe_down(*s["h"][key], plan, s["weights"], s["down"][key], bias=s["bias_down"], residual=s["residual"],
                       out_dtype=out, layout=layout, n=c["d"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """What a pass cannot do without: inputs read once, outputs written once,
    the weights of the experts that a uniform choice reaches."""
    c = case
    t, e, k = c["tokens"], c["experts"], c["topk"]
    p = t * k
    if c["op"] == "route":
        return {"bytes": t * e * (2 if c["bf16"] else 4) + 4 * e * c["bias"] + 8 * p, "flops": 40 * t * e}
    if c["op"] == "plan":
        return {"bytes": 12 * p + 4 * ((c["local"] or e) + 1), "flops": p}
    d, f = c["d"], c["f"]
    packed = 0.5 + 1 / 32
    w = e * (1 - (1 - k / e) ** t) * d * f * packed
    if c["op"] == "up":
        return {"bytes": 2 * w + t * d * packed + p * f * (4 if c["out_f32"] else 2) + 4 * p, "flops": 4 * p * d * f}
    out = t * d * ((4 if c.get("out_f32") else 2) + 2 * c["residual"])
    if c["op"] == "down":
        return {"bytes": w + p * f * packed + out + 8 * p, "flops": 2 * p * d * f}
    return {"bytes": 3 * w + 2 * t * d + t * e * (2 if c["bf16"] else 4) + out, "flops": 6 * p * d * f}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _values64(codes, scales):
    nib = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    ex, man, sign = (nib >> 1) & 3, (nib & 1).double(), 1.0 - 2.0 * (nib >> 3).double()
    mag = torch.where(ex == 0, 0.5 * man, torch.exp2(ex.double() - 1) * (1 + 0.5 * man))
    return sign * mag * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def _mx64(y):
    b = y.reshape(y.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2
    e = torch.where(torch.exp2(e + 2) > top, e - 1, e).clamp(min=-127)
    t = b.abs() / torch.exp2(e)
    step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0))
    return (torch.sign(b) * (torch.round(t / step) * step).clamp(max=6) * torch.exp2(e)).reshape(y.shape)


def _act64(name, x):
    if name == "relu":
        return x.clamp(min=0)
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return x * 0.5 * torch.erfc(-x / math.sqrt(2))
    return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))


def _choice64(c, logits, bias):
    """ids and weights, one choice after the other."""
    x = logits.double()
    s = torch.softmax(x, -1) if c["score"] == "softmax" else torch.sigmoid(x)
    by = x.clone() if bias is None else s + bias.double()
    first = torch.arange(x.shape[1], device=DEV)

    def largest(v):   # the lowest index of the largest value
        top = v.amax(-1, keepdim=True)
        return torch.where(v == top, first[:v.shape[1]], v.shape[1]).amin(-1, keepdim=True)
    if c["groups"] > 1:
        size = x.shape[1] // c["groups"]
        top = torch.topk((s if bias is None else by).reshape(-1, c["groups"], size), min(2, size), -1).values
        score = top[..., 0] if c["group_score"] == "max" else top.sum(-1)
        out = torch.ones_like(score, dtype=torch.bool)
        for _ in range(c["topk_groups"]):
            g = largest(score)
            out.scatter_(1, g, False)
            score = score.scatter(1, g, -math.inf)
        by[out.repeat_interleave(size, 1)] = -math.inf
    ids = []
    for _ in range(c["topk"]):
        ids.append(largest(by))
        by = by.scatter(1, ids[-1], -math.inf)
    ids = torch.cat(ids, 1)
    w = s.gather(1, ids)
    return ids, c["scale"] * (w / w.sum(-1, keepdim=True) if c["renorm"] else w)


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "plan":
        return None   # whole numbers
    if c["op"] in ("route", "ffn"):
        ids, weights = _choice64(c, s["logits"], s["bias"])
        if c["op"] == "route":
            return {"ids": None, "weights": weights}
    else:
        ids, weights = s["ids"].long(), s["weights"].double()
    t, k = ids.shape
    flat = ids.flatten()
    by = torch.argsort(flat, stable=True)

    def product(rows, packed, bias, e):
        z = rows @ _values64(packed[0][e], packed[1][e]).T
        return z if bias is None else z + bias[e].double()
    if c["op"] != "down":
        a = _values64(*s["a"]["row"]) if c["op"] == "up" else _mx64(_rotate(s["x"].double(), c["h32"]))
        h = torch.empty((t * k, c["f"]), dtype=torch.float64, device=DEV)   # by pair
        for e in range(c["experts"]):
            at = torch.nonzero(flat == e).flatten()
            if at.numel():
                rows = a[at // k]
                h[at] = _act64(c["act"], product(rows, s["gate"]["row"], s.get("bias_gate"), e)) * \
                    product(rows, s["up"]["row"], s.get("bias_up"), e)
        if c["op"] == "up":
            return h[by]
        h = _mx64(_rotate(h, c["h32"]))
    else:
        h = torch.empty((t * k, c["f"]), dtype=torch.float64, device=DEV)
        h[by] = _values64(*s["h"]["row"])
    y = torch.zeros((t, c["d"]), dtype=torch.float64, device=DEV) if s["residual"] is None else s["residual"].double()
    for e in range(c["experts"]):
        at = torch.nonzero(flat == e).flatten()
        if at.numel():
            y.index_add_(0, at // k, weights.flatten()[at, None] *
                         product(h[at], s["down"]["row"], s.get("bias_down"), e))
    return y
