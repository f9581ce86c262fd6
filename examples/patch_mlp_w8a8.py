"""A patch embedding followed by gated 8-bit MLP blocks, on random weights.

Images are embedded by ``conv_fwd`` (stride == filter: one GEMM row per patch);
each block then runs

    a, sa, stream = rms_norm_quant(y, gain, residual=stream)   # 8 bits per token
    h = linear_w8a8(a, up, sa, s_up)                            # gate and value halves
    b, sb = act_quant(h, "silu", gated=True)                    # 8 bits per token
    y = linear_w8a8(b, down, sb, s_down)

with the residual stream updated in place.  The blocks are captured once in a
CUDA graph and replayed on new images; the result is compared with the same
blocks on unquantised weights and activations.

    python examples/patch_mlp_w8a8.py [--images 8] [--blocks 4] [--dtype int8]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import implicit_gemm_convolution_conv3d_gb300 as c3d   # noqa: E402

CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


class GatedBlock:
    """One block: the weights' codes with a scale per output channel, and the
    buffers its calls write."""

    def __init__(self, width, inner, tokens, qdtype, gen):
        draw = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
        self.w_up, self.w_down = draw(2 * inner, width) / math.sqrt(width), draw(width, inner) / math.sqrt(inner)
        self.up, self.s_up = c3d.act_quant(self.w_up, qdtype=qdtype)
        self.down, self.s_down = c3d.act_quant(self.w_down, qdtype=qdtype)
        self.gain = (1.0 + 0.1 * draw(width)).bfloat16()
        new = lambda n, t: torch.empty(tokens, n, dtype=t, device="cuda")   # noqa: E731
        self.a, self.b = new(width, qdtype), new(inner, qdtype)
        self.sa, self.sb = (torch.empty(tokens, device="cuda") for _ in range(2))
        self.h, self.y = new(2 * inner, torch.bfloat16), new(width, torch.bfloat16)

    def __call__(self, y, stream):
        c3d.rms_norm_quant(y, self.gain, residual=stream, out=self.a, scale_out=self.sa,
                           residual_out=stream)
        c3d.linear_w8a8(self.a, self.up, self.sa, self.s_up, out=self.h)
        c3d.act_quant(self.h, "silu", gated=True, out=self.b, scale_out=self.sb)
        return c3d.linear_w8a8(self.b, self.down, self.sb, self.s_down, out=self.y)

    def unquantised(self, y, stream):
        """The same block in fp32 torch operations."""
        stream = stream + y
        v = stream * torch.rsqrt((stream * stream).mean(-1, keepdim=True) + 1e-6) * self.gain.float()
        gate, value = (v @ self.w_up.t()).chunk(2, dim=-1)
        return (gate / (1.0 + torch.exp(-gate)) * value) @ self.w_down.t(), stream


def run(images=8, blocks=4, dtype="int8", width=1024, inner=4096, patch=14, seed=0):
    """(relative error of the output tokens, milliseconds per replay)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    side = 224 // patch
    tokens = images * side * side
    w_patch = (torch.randn(width, 1, patch, patch, 3, generator=gen, device="cuda")
               / math.sqrt(3 * patch * patch)).bfloat16()
    layers = [GatedBlock(width, inner, tokens, CODES[dtype], gen) for _ in range(blocks)]
    pixels = torch.empty(images, 1, 224, 224, 3, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(tokens, width, dtype=torch.bfloat16, device="cuda")

    def forward():
        stream = c3d.conv_fwd(pixels, w_patch, (1, patch, patch), 0, 1).view(tokens, width)
        y = zero
        for layer in layers:
            y = layer(y, stream)
        return y, stream

    pixels.normal_(generator=gen)
    forward()                                       # loads the kernels before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, stream = forward()
    pixels.normal_(generator=gen)                   # new images into the captured buffer
    graph.replay()
    got = y.float() + stream.float()

    s = c3d.conv_fwd(pixels, w_patch, (1, patch, patch), 0, 1).view(tokens, width).float()
    r = torch.zeros_like(s)
    for layer in layers:
        r, s = layer.unquantised(r, s)
    want = r + s
    error = float((got - want).norm() / want.norm())

    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if c3d.conv_get_device_status() != 0:
        raise RuntimeError("a kernel gave up on a bounded wait")
    return error, start.elapsed_time(end) / 20


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--images", type=int, default=8)
    ap.add_argument("--blocks", type=int, default=4)
    ap.add_argument("--dtype", choices=sorted(CODES), default="int8")
    a = ap.parse_args()
    error, ms = run(a.images, a.blocks, a.dtype)
    print(f"{a.images} images, {a.blocks} blocks, {a.dtype}: {ms:.3f} ms per replay, "
          f"{100 * error:.2f}% from the unquantised blocks")
