"""Decoding within a fixed budget of cache pages: one attention layer, end to end.

    python examples/paged_decode.py [--batch 4] [--prompt 700] [--steps 300] [--budget 24]

The layer has joined Q | K | V weights and an output projection in Q4_0, and keeps its keys and
values in 8-bit pages with one scale per page.  A ragged batch of prompts goes through it at once;
then tokens are decoded one by one, the step captured once into a CUDA graph.  Every step writes the
new token into the pages, attends over what is held (with a bias by distance, so positions matter),
gathers the attention weight of every page and drops the lightest pages beyond the budget.

At the end the last step's attention is computed again in 64 bits from the values read back.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_skinny_matmul_gb300 as gq  # noqa: E402


class Layer:
    """x + O(attention(norm(x))) over a paged cache, for a batch of sequences."""

    def __init__(self, batch, tokens, hidden, heads, kv_heads, D, page, budget, kind, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.D, self.hidden, self.budget = heads, kv_heads, D, hidden, budget

        def weights(n, k):
            w = torch.randn((n, k), generator=gen, device="cuda") * (1.5 / math.sqrt(k))
            return gq.repack_q4_0(gq.quantize_q4_0(w), n, k)

        self.rows = (heads + 2 * kv_heads) * D
        self.qkv, self.o = weights(self.rows, hidden), weights(hidden, heads * D)
        self.cache = gq.KVPages.empty(batch, kv_heads, D, tokens, page, kind)
        self.gathered = torch.zeros((batch, kv_heads, self.cache.NB), device="cuda")
        self.slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], device="cuda")
        self.scores = gq.AttnScores(1.0 / math.sqrt(D), slopes=self.slopes)

    def forward(self, x, cu, new, max_n):
        """x: packed rows [T, hidden]; cu: offsets; new: int32 [batch], the rows of each sequence."""
        c, nq, nk = self.cache, self.heads * self.D, self.kv_heads * self.D
        normed = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        y = gq.mul_mat_q4_0_f32(self.qkv, normed, self.rows)
        self.q = y[:, :nq]                                       # rows may be strided
        gq.kv_pages_append(c, y[:, nq:nq + nk], y[:, nq + nk:], cu, max_n)
        a, w = gq.attn_pages(c, self.q, cu, max_n, self.scores, weights=self.gathered, decay=0.98)
        self.attended = a
        c.held += new
        c.seen += new
        # (in place: every row of the table is read before it is written)
        gq.gq_kv_pages_evict(c, w, self.budget, 1, 2, c.table, c.base, self.gathered, c.held)
        return x + gq.mul_mat_q4_0_f32(self.o, a.reshape(x.shape[0], nq), self.hidden)


def check(layer, q, out, before):
    """The attention of one decode step in 64 bits, from the cache as it was before eviction."""
    c = layer.cache
    table, base, held, seen = before
    cache = gq.KVPages(c.kind, c.k, c.v, c.ks, c.vs, table, base, held, seen)
    n = held.tolist()
    cu = torch.tensor([0] + n, device="cuda").cumsum(0).to(torch.int32)
    k, v = gq.kv_pages_read(cache, torch.zeros_like(held), cu, int(cu[-1]), max(n))
    worst, G = 0.0, layer.heads // layer.kv_heads
    for b in range(c.B):
        kb, vb = (t[int(cu[b]):int(cu[b + 1])].double() for t in (k, v))
        slot = torch.arange(n[b], device="cuda")
        pos = base[b][:, slot // c.P].long() + slot % c.P        # [kv_heads, n]
        for h in range(layer.heads):
            z = kb[:, h // G] @ q[b].view(layer.heads, layer.D)[h].double() / math.sqrt(layer.D)
            z = z - layer.slopes[h].double() * (int(seen[b]) - 1 - pos[h // G]).abs()
            want = torch.softmax(z, 0) @ vb[:, h // G]
            worst = max(worst, float((out[b, h].double() - want).abs().max() / want.abs().max()))
    return worst


def run(batch=4, prompt=700, steps=300, budget=24, hidden=4096, heads=32, kv_heads=8, D=128, page=32, kind=gq.GQ_KV_I8):
    """Returns (microseconds per step, pages held per sequence and head, worst relative error of the last step)."""
    lengths = [max(1, prompt - 37 * b) for b in range(batch)]
    layer = Layer(batch, max(lengths) + page * (budget + 2), hidden, heads, kv_heads, D, page, budget, kind)
    c, gen = layer.cache, torch.Generator("cuda").manual_seed(1)

    cu = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    new = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    x = torch.randn((sum(lengths), hidden), generator=gen, device="cuda")
    y = layer.forward(x, cu, new, max(lengths))
    token = y[cu[1:].long() - 1].clone()                         # the last row of each prompt

    one = torch.ones(batch, dtype=torch.int32, device="cuda")
    cu1 = torch.arange(batch + 1, dtype=torch.int32, device="cuda")

    def step():
        y = layer.forward(token, cu1, one, 1)
        token.copy_(y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                                   # workspaces are there before the capture
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)

    times = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    times[0].record()
    for _ in range(steps - 1):
        graph.replay()
    times[1].record()
    torch.cuda.synchronize()
    us = times[0].elapsed_time(times[1]) * 1e3 / max(1, steps - 1)

    # one more step, not captured; the pages are written in place, so the state before eviction is
    # the table and the positions from before the step, with one token more
    before = (c.table.clone(), c.base.clone(), c.held + 1, c.seen + 1)
    pages = c.held.div(page, rounding_mode="floor")
    first = (c.held % page == 0).nonzero().flatten().tolist()    # sequences that begin a page in this step
    for b in first:
        before[1][b, :, int(pages[b])] = c.seen[b]
    layer.forward(token, cu1, one, 1)
    status = gq.gq_last_error()
    if status != gq.GQ_OK:
        raise RuntimeError(f"the library reports status {status}")
    return us, (-(-c.held // page)).tolist(), check(layer, layer.q, layer.attended, before)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("batch", 4), ("prompt", 700), ("steps", 300), ("budget", 24)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    us, pages, err = run(a.batch, a.prompt, a.steps, a.budget)
    print(f"{us:.1f} us per step of {a.batch} tokens, {pages} pages held, last step within {err:.1e} of 64 bits")
    if not err < 1e-4:
        raise SystemExit("the last step is off")


if __name__ == "__main__":
    main()
