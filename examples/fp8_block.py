"""A modulated transformer block on 8-bit floating-point linears.

    python examples/fp8_block.py [--rows 4608] [--width 3072] [--heads 24] [--samples 2]

The block norms and the fp8 linears as a diffusion transformer would call
them: each norm leaves codes that the next linears read, the gate and residual
of a branch share a pass with the norm of the next, and q, k and v are one
launch on one packed activation. Attention and the activation between them are
plain torch. Prints the error against the same block in float32 and the time
of one pass.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from int8_hadamard_rotated_gb300 import ops  # noqa: E402

EPS = 1e-6


class Block:
    """Weights of one block: float32, and packed for the fp8 linears."""

    def __init__(self, width: int, heads: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.width, self.heads = width, heads
        shapes = dict(q=(width, width), k=(width, width), v=(width, width), out=(width, width),
                      up=(4 * width, width), down=(width, 4 * width))
        self.W = {n: r(*s) * s[1] ** -0.5 for n, s in shapes.items()}
        self.b = {n: 0.1 * r(s[0]) for n, s in shapes.items()}
        self.codes = {n: ops.fp8_prepare_weight(w) for n, w in self.W.items()}

    def _linears(self, names):
        return [self.codes[n][0] for n in names], [self.codes[n][1] for n in names], [self.b[n] for n in names]

    def _attend(self, q, k, v, samples):
        split = lambda t: t.view(samples, -1, self.heads, self.width // self.heads).transpose(1, 2)  # noqa: E731
        o = torch.nn.functional.scaled_dot_product_attention(split(q), split(k), split(v))
        return o.transpose(1, 2).reshape(q.shape)

    def forward(self, h, mod, samples):
        """h [rows, width] (rows of a sample together), mod [samples, 6 width]:
        shift, scale and gate of the attention, then of the MLP."""
        shift1, scale1, gate1, shift2, scale2, gate2 = mod.split(self.width, dim=1)
        per = h.shape[0] // samples
        norm = dict(pre_norm=ops.NORM_LAYER, pre_eps=EPS, rows_per_sample=per)
        _, q8, s = ops.convrot_block_norm_fp8(h, want_h=False, scale=scale1, shift=shift1, **norm)
        q, k, v = ops.fp8_linear_packed(q8, s, *self._linears(("q", "k", "v")))
        a = self._attend(q, k, v, samples)
        (a,) = ops.fp8_linear(a, *self._linears(("out",)))
        h, q8, s = ops.convrot_block_norm_fp8(h, a, gate=gate1, scale=scale2, shift=shift2, **norm)
        (u,) = ops.fp8_linear_packed(q8, s, *self._linears(("up",)))
        (d,) = ops.fp8_linear(torch.nn.functional.gelu(u), *self._linears(("down",)))
        return ops.convrot_block_norm(h, d, gate=gate2, pre_norm=ops.NORM_NONE, rows_per_sample=per, want_u=False)[0]

    def forward_float(self, h, mod, samples):
        """The same in float32."""
        rows = torch.arange(h.shape[0], device=h.device) // (h.shape[0] // samples)
        shift1, scale1, gate1, shift2, scale2, gate2 = mod[rows].split(self.width, dim=1)
        norm = lambda x, sc, sh: torch.nn.functional.layer_norm(x, (self.width,), eps=EPS) * (1 + sc) + sh  # noqa: E731
        lin = lambda x, n: x @ self.W[n].t() + self.b[n]  # noqa: E731
        h = h.float()
        u = norm(h, scale1, shift1)
        h = h + gate1 * lin(self._attend(lin(u, "q"), lin(u, "k"), lin(u, "v"), samples), "out")
        u = torch.nn.functional.gelu(lin(norm(h, scale2, shift2), "up"))
        return h + gate2 * lin(u, "down")


def inputs(rows: int, width: int, samples: int, seed: int = 1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(rows, width, generator=gen, device="cuda").to(torch.bfloat16)
    return h, 0.3 * torch.randn(samples, 6 * width, generator=gen, device="cuda")


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=4608)
    ap.add_argument("--width", type=int, default=3072)
    ap.add_argument("--heads", type=int, default=24)
    ap.add_argument("--samples", type=int, default=2)
    a = ap.parse_args(argv)
    block = Block(a.width, a.heads)
    h, mod = inputs(a.rows, a.width, a.samples)
    y, ref = block.forward(h, mod, a.samples).float(), block.forward_float(h, mod, a.samples)
    print(f"relative error against float32: {float((y - ref).norm() / ref.norm()):.4f}")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        block.forward(h, mod, a.samples)
    start.record()
    for _ in range(10):
        block.forward(h, mod, a.samples)
    end.record()
    end.synchronize()
    print(f"one pass of {a.rows} x {a.width}: {start.elapsed_time(end) / 10:.3f} ms")
    status = ops.convrot_device_status()
    if status != ops.OK:
        raise SystemExit(f"device status {status}")


if __name__ == "__main__":
    main()
