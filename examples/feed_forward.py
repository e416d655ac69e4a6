"""Feed-forward blocks on MXFP4 weights: a gated one (SwiGLU) as a decode step
and over a prompt, and a modulated one (layer norm, tanh GELU, gate) over image
tokens.  Random weights, synthetic inputs; prints each block's time and its
distance from the same block in fp32 without quantization (the 4-bit formats'
own error).

    python examples/feed_forward.py [--d 4096] [--hidden 14336] [--steps 50]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_w4a4_quantized_amd as mx  # noqa: E402

BF = torch.bfloat16


def weights(gen, d, hidden, gated):
    shapes = [(hidden, d), (d, hidden)] + ([(hidden, d)] if gated else [])
    dense = [torch.randn(*s, generator=gen, device="cuda") * s[1] ** -0.5 for s in shapes]
    return dense, [mx.quantize_weight(w, mx.HADAMARD32, layout=mx.TILED) for w in dense]


def plain(x, p, residual, dense, act, gate):
    """The block in fp32 from the unquantized weights."""
    r = x.float() + residual.float()
    d = r.shape[1]
    if p.kind == "rms":
        z = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + p.eps) * p.weight.float()
    else:
        z = torch.nn.functional.layer_norm(r, (d,), eps=p.eps) * (1 + p.scale.float()) + p.shift.float()
    up = z @ dense[0].T
    if act == "silu":
        h = torch.nn.functional.silu(z @ dense[2].T) * up
    else:
        h = torch.nn.functional.gelu(up, approximate="tanh")
    y = h @ dense[1].T
    return r, y if gate is None else y * gate.float()


def block(name, rows, d, hidden, gated, steps):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    dense, q = weights(gen, d, hidden, gated)
    x, residual = (torch.randn(rows, d, generator=gen, device="cuda").to(BF) for _ in range(2))
    vec = lambda: (torch.randn(1, d, generator=gen, device="cuda") * 0.1).to(BF)  # noqa: E731
    if gated:
        p, gate, act = mx.Norm("rms", weight=1 + vec()[0]), None, "silu"
    else:
        p, gate, act = mx.Norm("layer", scale=vec(), shift=vec(), group_rows=rows), vec(), "gelu_tanh"

    def step():
        return mx.ffn(x, p, residual, q[0], q[1], hidden, w_gate=q[2] if gated else None, act=act,
                      rot=mx.HADAMARD32, gate=gate, layout=mx.TILED)

    y, r = step()
    want_r, want = plain(x, p, residual, dense, act, gate)
    err = float((y.float() - r.float() - want).norm() / want.norm())
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(steps):
        step()
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) * 1e3 / steps
    flops = 2 * rows * d * hidden * (3 if gated else 2)
    print(f"{name:12s} {rows:6d} x {d} -> {hidden}: {us:8.1f} us, {flops / us * 1e-6:7.1f} TFLOP/s, "
          f"relative distance from fp32 {err:.3f}", flush=True)
    return err


def main(argv=None):
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--d", type=int, default=4096)
    a.add_argument("--hidden", type=int, default=14336)
    a.add_argument("--prompt", type=int, default=2048)
    a.add_argument("--steps", type=int, default=50)
    a = a.parse_args(argv)
    return [block("decode", 4, a.d, a.hidden, True, a.steps),
            block("prompt", a.prompt, a.d, a.hidden, True, a.steps),
            block("modulated", a.prompt, a.d, a.hidden, False, a.steps)]


if __name__ == "__main__":
    main()
