"""A layer of experts over 4-bit microscaled weights: a prompt, then decode steps in a CUDA graph.

    python examples/experts.py [--hidden 2048] [--inner 1408] [--experts 64] [--top-k 8] [--prompt 500] [--steps 100]

Each step adds the residual and takes the norm into e4m3 blocks (one kernel), scores the experts (an F16
product), chooses top_k of them with the rows sorted by expert, computes the chosen experts' gated unit
and down products on the tensor cores, and sums each token's experts onto the residual.  The batch of the
decode steps has room for 8 sequences; the tokens in use are a number on the device, so that one captured
graph serves any of them.

At the end the last step is computed again in 64 bits, from the weights and blocks read back.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_skinny_matmul_gb300 as gq  # noqa: E402


class Layer:
    """x + experts(norm(x))."""

    def __init__(self, hidden, inner, experts, top_k, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.norm = torch.ones(hidden, device="cuda")
        self.gate = (torch.randn((experts, hidden), generator=gen, device="cuda") / math.sqrt(hidden)).half()
        self.router = gq.Router(experts, top_k)

        def weights(count, n, k):
            q = gq.quantize_mx(torch.randn((count * n, k), generator=gen, device="cuda") / math.sqrt(k), gq.GQ_MX_E2M1)
            return gq.repack_mxfp4(q.codes, q.scales, n, k), q

        self.up, self.up_blocks = weights(2 * experts, inner, hidden)     # gate, up of expert 0, of expert 1, ..
        self.down, self.down_blocks = weights(experts, hidden, inner)

    def forward(self, x, residual, used=None):
        """(the layer's output, what led to it); rows from `used` on are padding."""
        h, blocks, y = gq.rms_norm_mx(x, self.norm, 1e-6, residual=residual, y_dtype=torch.float32)
        ids, weights, plan = gq.route(gq.mul_mat_f16_f32(self.gate, y), self.router, used)
        act = gq.swiglu_mxfp4(self.up, blocks, plan, gather=True)
        out = gq.experts_combine(gq.mul_mat_mxfp4(self.down, act, plan), plan, weights, residual=h)
        return out, (h, blocks, ids, weights, plan, act)


def check(layer, out, parts, tokens):
    """How far the first `tokens` rows are off their 64-bit values, from the blocks as they are (NaN if anything is)."""
    h, blocks, ids, weights, plan, act = parts
    A, pos = gq.dequantize_mx(act).double(), plan.pos.tolist()
    N, K = layer.down.N, layer.down.K
    worst = []
    W = gq.dequantize_mx(layer.down_blocks).view(-1, N, K)
    for t in range(tokens):
        want = h[t].double()
        for j, e in enumerate(ids[t].tolist()):
            want = want + weights[t, j].double() * (W[e].double() @ A[pos[t][j]])
        worst.append((out[t].double() - want).abs().max() / want.abs().max())
    # the gated units in e4m3: half a step is 2^-4 of a value, or of its block's smallest normal one; what is
    # beyond that, of the block's largest value
    X, U = gq.dequantize_mx(blocks), gq.dequantize_mx(layer.up_blocks).view(-1, 2, layer.up.N, layer.up.K)
    unit = []
    for t in range(tokens):
        for j, e in enumerate(ids[t].tolist()):
            g, u = (U[e].double() @ X[t].double())
            v = torch.nn.functional.silu(g) * u
            top = v.view(-1, 32).abs().amax(-1, keepdim=True).expand(-1, 32).reshape(-1)
            off = (A[pos[t][j]] - v).abs() - torch.maximum(v.abs(), top * 2.0 ** -13) / 16
            unit.append((off / top.clamp(min=1e-30)).max().clamp(min=0.0))
    return tuple(float(torch.stack(x).max()) if x else 0.0 for x in (worst, unit))


def run(hidden=2048, inner=1408, experts=64, top_k=8, prompt=500, steps=100, room=8):
    """(microseconds per step, relative error of the output, of the gated unit beyond its rounding) after a prompt and `steps` steps."""
    layer = Layer(hidden, inner, experts, top_k)
    gen = torch.Generator("cuda").manual_seed(1)
    layer.forward(torch.randn((prompt, hidden), generator=gen, device="cuda"), torch.zeros((prompt, hidden), device="cuda"))
    x, residual = (torch.randn((room, hidden), generator=gen, device="cuda") for _ in range(2))
    used = torch.tensor([room], dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.forward(x, residual, used)                                  # (workspaces grow before the capture)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out, parts = layer.forward(x, residual, used)
            x.copy_(out).mul_(0.5)
        graph.replay()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for step in range(steps):
            used.fill_(room - step % 3)                                   # sequences come and go
            graph.replay()
        end.record()
    stream.synchronize()
    us = begin.elapsed_time(end) * 1e3 / steps
    return (us,) + check(layer, out, parts, int(used))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1408)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    us, err, unit = run(a.hidden, a.inner, a.experts, a.top_k, a.prompt, a.steps)
    print(f"{us:.1f} us per step; output off by {err:.2e}, gated unit by {unit:.2e} beyond its rounding")


if __name__ == "__main__":
    main()
