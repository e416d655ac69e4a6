"""Cases that measure the feed-forward operators of the MXFP4 library: the
fused norm (residual add, gate, post-norm, modulation), the GEMM with a bias /
activation / gate / residual epilogue, the gated (GLU) GEMM, and the
feed-forward path that chains them through MXFP4 activations.

A case is a dict of plain values.  "op" names the operator:
  norm   y, r = norm(residual_scale * residual + gate * [postnorm](x)) ...
  epi    Y = residual + gate * act(A B^T + bias) on packed MXFP4 operands
  glu    H = act(A G^T + bg) * (A U^T + bu) on packed MXFP4 operands
  ffn    norm -> MXFP4 -> (gated) up projection -> MXFP4 -> down projection
         + residual, three launches with MXFP4 activations in between
Packed operands are E2M1 codes (two per byte) and one E8M0 byte per 32 elements
along K; they are kept row-major and, where K allows it, in the library's
256-row tiled layout, as a serving program lays its weights out once.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def _case(op, name, **kw):
    base = {"norm": dict(rows=1, d=32, kind="rms", residual=True, post=False, mod=False, gate=False, rscale=1.0,
                         group_rows=0, x_f32=False, r_f32=False),
            "epi": dict(m=1, k=128, n=32, act="none", bias=False, gate=False, residual=False, group_rows=0,
                        out_f32=False),
            "glu": dict(m=1, k=128, n=32, act="silu", bias=False, out_f32=False),
            "ffn": dict(m=1, d=128, f=128, kind="rms", act="silu", gated=True, h32=True, mod=False,
                        group_rows=0)}[op]
    return {"name": name, "op": op, **base, **kw}


def listed():
    return [
        # --- norm
        # the residual add and pre-norm of a decode batch: launch latency
        _case("norm", "norm_decode_16x4096", rows=16, d=4096),
        # an odd token count through a sandwich norm (post-norm, gate, scaled
        # residual) with a 32-bit residual stream
        _case("norm", "norm_sandwich_777x5120", rows=777, d=5120, post=True, gate=True, rscale=0.5, group_rows=111,
              r_f32=True),
        # diffusion transformer, batch 16 x 3584 tokens: layer norm with
        # per-image scale, shift and gate
        _case("norm", "norm_adaln_57344x3072", rows=57344, d=3072, kind="layer", mod=True, gate=True,
              group_rows=3584),
        # --- GEMM with an epilogue
        # one token through a down projection onto the residual stream
        _case("epi", "epi_token_1x14336_4096", m=1, k=14336, n=4096, residual=True),
        # ragged sizes (no multiple of the tiles, K not of 128), erf GELU, 32-bit output
        _case("epi", "epi_odd_301x1184_1000", m=301, k=1184, n=1000, act="gelu", bias=True, out_f32=True),
        # diffusion transformer's down projection: bias, per-image gate, residual
        _case("epi", "epi_down_3584x12288_3072", m=3584, k=12288, n=3072, bias=True, gate=True, residual=True,
              group_rows=1792),
        # its up projection at batch 16: bias and tanh GELU, the largest
        _case("epi", "epi_up_57344x3072_12288", m=57344, k=3072, n=12288, act="gelu_tanh", bias=True),
        # --- gated GEMM
        # decode batch: two weight matrices streamed once
        _case("glu", "glu_decode_16x4096_14336", m=16, k=4096, n=14336),
        # ragged prompt, odd width, biases, 32-bit output
        _case("glu", "glu_odd_523x1408_3001", m=523, k=1408, n=3001, act="gelu_tanh", bias=True, out_f32=True),
        # a long prompt
        _case("glu", "glu_prompt_8192x4096_14336", m=8192, k=4096, n=14336),
        # --- the feed-forward path
        # one decode step of 4 sequences
        _case("ffn", "ffn_decode_4x4096_14336", m=4, d=4096, f=14336),
        # one image (3584 tokens) through a diffusion transformer's MLP
        _case("ffn", "ffn_image_3584x3072_12288", m=3584, d=3072, f=12288, kind="layer", act="gelu_tanh",
              gated=False, mod=True, group_rows=3584),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "epi", "glu", "ffn"))
    yes = lambda p=0.5: rng.random() < p  # noqa: E731
    if op == "norm":
        d = 32 * _log_int(rng, 32, 256)
        rows = _log_int(rng, 1, max(2, min(57344, 57344 * 3072 // d)))
        grouped = yes()
        return {k: v for k, v in _case("norm", "", rows=rows, d=d, kind=rng.choice(("rms", "layer")), residual=True,
                                       post=yes(0.4), mod=grouped, gate=grouped and yes(),
                                       rscale=rng.choice((1.0, 0.5)), group_rows=_log_int(rng, 1, rows),
                                       x_f32=yes(0.2), r_f32=yes(0.3)).items() if k != "name"}
    if op in ("epi", "glu"):
        m = _log_int(rng, 1, 16384)
        n = _log_int(rng, 256, 14336)
        k = (128 if yes(0.8) else 32) * _log_int(rng, 8, 96)
        if op == "epi":
            c = _case("epi", "", m=m, k=k, n=n, act=rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")),
                      bias=yes(), gate=yes(0.4), residual=yes(), group_rows=_log_int(rng, 1, m), out_f32=yes(0.3))
        else:
            c = _case("glu", "", m=m, k=k, n=n, act=rng.choice(("silu", "gelu", "gelu_tanh", "relu")), bias=yes(0.3),
                      out_f32=yes(0.3))
        return {k: v for k, v in c.items() if k != "name"}
    m, gated = _log_int(rng, 1, 4096), yes()
    c = _case("ffn", "", m=m, d=128 * _log_int(rng, 8, 32), f=128 * _log_int(rng, 16, 112), gated=gated,
              kind=rng.choice(("rms", "layer")), act=rng.choice(("silu", "gelu_tanh")), h32=yes(), mod=yes(0.4),
              group_rows=_log_int(rng, 1, m))
    return {k: v for k, v in c.items() if k != "name"}


# ---------------------------------------------------------------------------
# packed operands


def _encode(y):
    """E2M1 codes (0..15, one per byte) and E8M0 bytes of y [rows, k]."""
    rows, k = y.shape
    b = y.float().reshape(rows, k // 32, 32)
    amax = b.abs().amax(-1)
    _, ex = torch.frexp(amax)                      # amax = f * 2^ex, f in [0.5, 1): floor(log2) = ex - 1
    e = torch.where(amax > 0, (ex - 3).clamp(min=-127), torch.full_like(ex, -127))
    t = torch.ldexp(b.abs().double(), -e[..., None].double())
    i = ((t > 0.25).to(torch.uint8) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5))
    code = i.to(torch.uint8) | (torch.signbit(b).to(torch.uint8) << 3)
    return code.reshape(rows, k), (e + 127).to(torch.uint8)


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
    code, scales = _encode(y)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    row = (codes, scales.contiguous())
    return {"row": row, "tiled": _tile(*row) if y.shape[1] % 128 == 0 else None, "rows": y.shape[0]}


def _h32(dtype, device):
    i = torch.arange(32, device=device)
    bits = i[:, None] & i[None, :]
    parity = sum((bits >> s) & 1 for s in range(5)) & 1
    return (1 - 2 * parity).to(dtype) / math.sqrt(32.0)


def _rotate(y, h32):
    rows, k = y.shape
    return (y.reshape(-1, 32) @ _h32(y.dtype, y.device)).reshape(rows, k) if h32 else y


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1_000_003 * (seed + 1))
    rnd = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    c = dict(case)
    s = {"case": c}
    groups = lambda rows: -(-rows // max(1, c["group_rows"]))  # noqa: E731
    if c["op"] == "norm":
        rows, d = c["rows"], c["d"]
        # a residual stream with a few channels far above the others
        lift = torch.where(torch.rand(d, generator=gen, device=DEV) < 0.01, 10.0, 1.0)
        s["x"] = rnd(rows, d).to(F32 if c["x_f32"] else BF16)
        s["residual"] = (rnd(rows, d) * lift).to(F32 if c["r_f32"] else BF16) if c["residual"] else None
        s["weight"] = None if c["mod"] else (1 + 0.1 * rnd(d)).to(BF16)
        s["bias"] = (0.1 * rnd(d)).to(BF16) if c["kind"] == "layer" and not c["mod"] else None
        s["post_weight"] = (1 + 0.1 * rnd(d)).to(BF16) if c["post"] else None
        if c["mod"] or c["gate"]:
            # one tensor of modulation vectors per group, used by slices
            vec = (0.2 * rnd(groups(rows), 3 * d)).to(BF16)
            s["scale"], s["shift"], s["gate"] = (vec[:, i * d:(i + 1) * d] for i in range(3))
        if not c["mod"]:
            s["scale"] = s["shift"] = None
        if not c["gate"]:
            s["gate"] = None
        return s
    if c["op"] in ("epi", "glu"):
        m, n, k = c["m"], c["n"], c["k"]
        s["a"] = _pack(rnd(m, k))
        for name in ("b",) if c["op"] == "epi" else ("g", "u"):
            s[name] = _pack(rnd(n, k) * 0.02)
            s["bias_" + name] = (0.2 * rnd(n)).to(BF16) if c["bias"] else None
        if c["op"] == "epi":
            s["gate"] = rnd(groups(m), n).to(BF16) if c["gate"] else None
            s["residual"] = rnd(m, n).to(BF16) if c["residual"] else None
        return s
    m, d, f = c["m"], c["d"], c["f"]
    s["x"] = rnd(m, d).to(BF16)
    s["residual"] = rnd(m, d).to(BF16)
    s["weight"] = None if c["mod"] else (1 + 0.1 * rnd(d)).to(BF16)
    vec = (0.2 * rnd(groups(m), 3 * d)).to(BF16) if c["mod"] else None
    s["scale"], s["shift"], s["gate"] = (vec[:, i * d:(i + 1) * d] if c["mod"] else None for i in range(3))
    s["up"] = _pack(_rotate(rnd(f, d) * 0.02, c["h32"]))
    s["gated"] = _pack(_rotate(rnd(f, d) * 0.02, c["h32"])) if c["gated"] else None
    s["down"] = _pack(_rotate(rnd(d, f) * 0.02, c["h32"]))
    return s


# ---------------------------------------------------------------------------
# plain forms: 32 bits, one rounding at the end


def _values(p):
    codes, scales = p["row"]
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
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _by_row(vec, rows, group_rows):
    """Row i of the result is vec's row i // group_rows."""
    return vec.float().repeat_interleave(group_rows, 0)[:rows]


def _normed(kind, v):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _norm_plain(c, s, rows):
    p = s["x"].float()
    if s.get("post_weight") is not None:
        p = _normed(c["kind"], p) * s["post_weight"].float()
    if c["op"] == "norm" and s["gate"] is not None:
        p = p * _by_row(s["gate"], rows, c["group_rows"])
    r = p + c.get("rscale", 1.0) * s["residual"].float() if s["residual"] is not None else p
    y = _normed(c["kind"], r)
    if s["weight"] is not None:
        y = y * s["weight"].float()
    if s.get("bias") is not None:
        y = y + s["bias"].float()
    if s["scale"] is not None:
        y = y * (1 + _by_row(s["scale"], rows, c["group_rows"])) + _by_row(s["shift"], rows, c["group_rows"])
    return y, r


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        y, r = _norm_plain(c, s, c["rows"])
        return {"y": y.to(BF16), "r": r.to(F32 if c["r_f32"] else BF16)}
    if c["op"] == "ffn":
        y, r = _norm_plain(c, s, c["m"])
        x = _quantized(_rotate(y, c["h32"]))
        h = x @ _values(s["up"]).T
        h = _act(c["act"], x @ _values(s["gated"]).T) * h if c["gated"] else _act(c["act"], h)
        out = _quantized(_rotate(h, c["h32"])) @ _values(s["down"]).T
        if s["gate"] is not None:
            out = out * _by_row(s["gate"], c["m"], c["group_rows"])
        return {"y": (out + r.to(BF16).float()).to(BF16), "r": r.to(BF16)}
    out = F32 if c["out_f32"] else BF16
    a = _values(s["a"])
    if c["op"] == "glu":
        g, u = a @ _values(s["g"]).T, a @ _values(s["u"]).T
        if c["bias"]:
            g, u = g + s["bias_g"].float(), u + s["bias_u"].float()
        return (_act(c["act"], g) * u).to(out)
    y = a @ _values(s["b"]).T
    if c["bias"]:
        y = y + s["bias_b"].float()
    y = _act(c["act"], y)
    if c["gate"]:
        y = y * _by_row(s["gate"], c["m"], c["group_rows"])
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(out)


# ---------------------------------------------------------------------------
# the library's calls


def _own(s):
    import mxfp4_w4a4_quantized_amd as mx
    c = s["case"]
    if c["op"] in ("norm", "ffn"):
        norm = mx.Norm(kind=c["kind"], eps=EPS, weight=s["weight"], bias=s.get("bias"), scale=s["scale"],
                       shift=s["shift"], gate=s["gate"] if c["op"] == "norm" else None,
                       post_norm=s.get("post_weight") is not None, post_weight=s.get("post_weight"),
                       residual_scale=c.get("rscale", 1.0), group_rows=c["group_rows"])
    if c["op"] == "norm":
        y, r = mx.norm(s["x"], norm, s["residual"], out_dtype=BF16)
        return {"y": y, "r": r}
    if c["op"] == "ffn":
        rot = mx.HADAMARD32 if c["h32"] else None
        y, r = mx.ffn(s["x"], norm, s["residual"], s["up"]["tiled"], s["down"]["tiled"], c["f"],
                      w_gate=s["gated"]["tiled"] if c["gated"] else None, act=c["act"], rot=rot, gate=s["gate"],
                      layout=mx.TILED)
        return {"y": y, "r": r}
    layout, key = (mx.TILED, "tiled") if s["a"]["tiled"] is not None else (mx.ROWMAJOR, "row")
    kw = dict(out_dtype=F32 if c["out_f32"] else BF16, layout=layout, m=c["m"], n=c["n"])
    if c["op"] == "glu":
        return mx.gemm_glu(*s["a"][key], *s["g"][key], *s["u"][key], act=c["act"], bias_g=s["bias_g"],
                           bias_u=s["bias_u"], **kw)
    epi = mx.Epilogue(act=c["act"], bias=s["bias_b"], gate=s["gate"], group_rows=c["group_rows"],
                      residual=s["residual"])
    return mx.gemm_epilogue(*s["a"][key], *s["b"][key], epi, **kw)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """What a pass cannot do without: inputs read once, outputs written once."""
    c = case
    packed = lambda rows, k: rows * k * (0.5 + 1 / 32)  # noqa: E731
    if c["op"] == "norm":
        e = c["rows"] * c["d"]
        r = 4 if c["r_f32"] else 2
        groups = -(-c["rows"] // max(1, c["group_rows"])) if c["mod"] or c["gate"] else 0
        vec = 2 * c["d"] * (2 + groups * (2 * c["mod"] + c["gate"]))
        return {"bytes": e * ((4 if c["x_f32"] else 2) + 2 * r + 2) + vec, "flops": 12 * e}
    if c["op"] == "ffn":
        w = (3 if c["gated"] else 2) * packed(c["d"], c["f"])
        return {"bytes": w + 4 * 2 * c["m"] * c["d"], "flops": (6 if c["gated"] else 4) * c["m"] * c["d"] * c["f"]}
    y = c["m"] * c["n"]
    mats = 2 if c["op"] == "glu" else 1
    b = packed(c["m"], c["k"]) + mats * packed(c["n"], c["k"]) + y * (4 if c["out_f32"] else 2)
    if c["op"] == "epi":
        b += 2 * y * c["residual"] + 2 * c["n"] * c["gate"] * -(-c["m"] // max(1, c["group_rows"]))
    return {"bytes": b, "flops": 2 * mats * y * c["k"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _values64(p):
    codes, scales = p["row"]
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
    if name == "gelu_tanh":
        return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    return x


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    rows = c["rows"] if c["op"] == "norm" else c["m"]
    grp = torch.arange(rows, device=DEV) // max(1, c.get("group_rows", 0))
    if c["op"] in ("norm", "ffn"):
        def stat(v):
            mu = v.mean(-1, keepdim=True) if c["kind"] == "layer" else 0.0
            return (v - mu) / torch.sqrt(((v - mu) ** 2).mean(-1, keepdim=True) + EPS)
        p = f64(s["x"])
        if s.get("post_weight") is not None:
            p = stat(p) * f64(s["post_weight"])
        if c["op"] == "norm" and s["gate"] is not None:
            p = p * f64(s["gate"])[grp]
        r = p if s["residual"] is None else p + c.get("rscale", 1.0) * f64(s["residual"])
        y = stat(r)
        y = y if s["weight"] is None else y * f64(s["weight"])
        y = y if s.get("bias") is None else y + f64(s["bias"])
        if s["scale"] is not None:
            y = y * (1 + f64(s["scale"])[grp]) + f64(s["shift"])[grp]
        if c["op"] == "norm":
            return {"y": y, "r": r}
        x = _mx64(_rotate(y, c["h32"]))
        h = x @ _values64(s["up"]).T
        h = _act64(c["act"], x @ _values64(s["gated"]).T) * h if c["gated"] else _act64(c["act"], h)
        out = _mx64(_rotate(h, c["h32"])) @ _values64(s["down"]).T
        out = out if s["gate"] is None else out * f64(s["gate"])[grp]
        return {"y": out + r.to(BF16).double(), "r": r}
    a = _values64(s["a"])
    mats = [a @ _values64(s[w]).T for w in (("b",) if c["op"] == "epi" else ("g", "u"))]
    if c["bias"]:
        mats = [v + f64(s["bias_" + w]) for v, w in zip(mats, ("b",) if c["op"] == "epi" else ("g", "u"))]
    y = _act64(c["act"], mats[0])
    if c["op"] == "glu":
        return y * mats[1]
    if c["gate"]:
        y = y * f64(s["gate"])[grp]
    return y if not c["residual"] else y + f64(s["residual"])
