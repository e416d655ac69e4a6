"""A mixture-of-experts feed-forward block on MXFP4 weights: norm with the
residual add, the router's product, and the block itself (moe_ffn), as a decode
step, over a prompt, and over a prompt with a balance bias and groups of experts.
Random weights, synthetic inputs; prints each block's time and its distance from
the same block in fp32 without quantization (the 4-bit formats' own error).

    python examples/mixture_of_experts.py [--d 2048] [--hidden 1408] [--experts 64] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_w4a4_quantized_amd as mx  # noqa: E402

BF = torch.bfloat16


def plain(n, residual, ids, weights, dense):
    """The block in fp32 from the unquantized weights, on the same choices."""
    up, gate, down = dense
    y = residual.float().clone()
    for e in range(up.shape[0]):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if len(token):
            x = n[token].float()
            h = torch.nn.functional.silu(x @ gate[e].T) * (x @ up[e].T)
            y.index_add_(0, token, (h @ down[e].T) * weights[token, slot, None])
    return y


def block(name, rows, d, hidden, experts, router, steps):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    dense = [rnd(experts, hidden, d) * d ** -0.5, rnd(experts, hidden, d) * d ** -0.5, rnd(experts, d, hidden) * hidden ** -0.5]
    up, gate, down = (mx.quantize_experts(w, mx.HADAMARD32, layout=mx.TILED) for w in dense)
    w_router = (rnd(experts, d) * d ** -0.5).to(BF)
    norm = mx.Norm("rms", weight=(1 + 0.1 * rnd(d)).to(BF))
    x, stream = rnd(rows, d).to(BF), rnd(rows, d).to(BF)

    def run():
        n, r = mx.norm(x, norm, stream)
        logits = n @ w_router.T
        return n, r, logits, mx.moe_ffn(n, logits, router, up, down, hidden, w_gate=gate, rot=mx.HADAMARD32, residual=r,
                                        layout=mx.TILED)

    n, r, logits, y = run()
    ids, weights = mx.moe_route(logits, router)
    want = plain(n, r, ids, weights, dense)
    err = ((y.float() - want).norm() / (want - r.float()).norm()).item()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        run()
    end.record()
    end.synchronize()
    print(f"{name}: {rows} tokens, {start.elapsed_time(end) / steps * 1e3:.1f} us, error {err:.3f} of the block's result")
    return err


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--d", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1408)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    bias = torch.randn(a.experts, device="cuda") * 0.05
    grouped = mx.Router(6, "sigmoid", bias, groups=8, topk_groups=4, group_score="top2", scale=2.5)
    return [block("decode", 4, a.d, a.hidden, a.experts, mx.Router(6), a.steps),
            block("prompt", a.prompt, a.d, a.hidden, a.experts, mx.Router(6), a.steps),
            block("prompt, grouped experts", a.prompt, a.d, a.hidden, a.experts, grouped, a.steps)]


if __name__ == "__main__":
    main()
