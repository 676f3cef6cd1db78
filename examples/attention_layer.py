"""A decoder's attention layer between two scaled GEMMs, prompt and then token by token.

    x -> quantise -> QKV GEMM (ptpc) -> append (rotary positions, paged e4m3 cache)
      -> attention (prompt: over the prompt itself; decode: over the cache)
      -> quantise -> output GEMM (ptpc)

    python examples/attention_layer.py          # needs a GB300

``AttentionLayer`` keeps the plans, the quantised weights and the cache; ``prompt`` and
``decode`` are what a server calls.  The decode step is captured in a CUDA graph,
with the lengths and the block table in fixed buffers.

``step`` is a layer of a server that mixes them: the residual's addition, norm and quantisation in
one, and attention over the cache for as many new tokens as each sequence has, whose pages a ``PagePool`` hands out
(``--answers N`` forks the first prompt N times and lets each fork go on by itself).
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from fp8_scaled_gemm_sm_gb300 import PagedAttention, PagePool, ScaledGemm, binding, norm_quantize, rotary_table


class AttentionLayer:
    def __init__(self, hidden, q_heads, kv_heads, dim, w_qkv, w_out, max_rows, num_pages, page=64, max_pos=4096):
        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        self.plan = PagedAttention(q_heads, kv_heads, dim, page, rotary=rotary_table(max_pos, dim))
        self.cache = self.plan.new_cache(num_pages)
        width = (q_heads + 2 * kv_heads) * dim
        # per-channel scales of the weights: quantised once
        self.qkv, self.out = ScaledGemm("ptpc", width, hidden, max_rows), ScaledGemm("ptpc", hidden, q_heads * dim, max_rows)
        self.w_qkv, self.w_out = binding.quantize("ptpc", w_qkv), binding.quantize("ptpc", w_out)

    def _project(self, x):
        return self._heads(*binding.quantize("ptpc", x), x)

    def _heads(self, codes, scale, x):
        rows = self.qkv(codes, self.w_qkv[0], scale, self.w_qkv[1]).view(x.shape[0], -1, self.dim)
        q, k = self.q_heads, self.kv_heads
        return rows[:, :q], rows[:, q:q + k], rows[:, q + k:]

    def _output(self, o):
        codes, scale = binding.quantize("ptpc", o.view(o.shape[0], -1))
        return self.out(codes, self.w_out[0], scale, self.w_out[1])

    def prompt(self, x, block_table, cu_seqlens):
        """x [tokens, hidden]: whole prompts packed by cu_seqlens, from empty caches."""
        q, k, v = self._project(x)
        q, k = self.plan.append(q, k, v, self.cache, block_table, torch.zeros_like(cu_seqlens[1:]), cu_seqlens, k_out=True)
        o, _ = self.plan.prompt(q, k, v, cu_seqlens)
        return self._output(o)

    def decode(self, x, block_table, ctx_lens, cu_seqlens):
        """x [sequences, hidden]: one new token of each; ctx_lens tokens before it are in the cache."""
        q, k, v = self._project(x)
        q, _ = self.plan.append(q, k, v, self.cache, block_table, ctx_lens, cu_seqlens)
        o, _ = self.plan.decode(q, self.cache, block_table, ctx_lens + 1)
        return self._output(o)

    def step(self, x, residual, weight, pool, rows, tokens, cu_seqlens):
        """x and residual [tokens, hidden], packed by cu_seqlens: `tokens` new ones of each of the pool's `rows`, whose pages it
        hands out here.  Returns the output, the residual stream, and whether each row got its pages; a row that did not is left as
        it was, and its tokens attend to nothing."""
        codes, scale, residual = norm_quantize("ptpc", x, weight, residual=residual)
        q, k, v = self._heads(codes, scale, x)
        at = rows.long()
        before = pool.lens[at]
        ok = pool.grow(rows, tokens)
        # without pages for its new tokens a row has none in this step: behind its last token they would go into a page that it holds
        table = torch.where(ok[:, None] > 0, pool.table[at], -1)
        q, _ = self.plan.append(q, k, v, self.cache, table, before, cu_seqlens)
        o, _ = self.plan.chunk(q, self.cache, table, pool.lens[at], cu_seqlens)
        return self._output(o), residual, ok


def answers(layer, count, tokens, prompt, weight, page):
    """`count` answers to one prompt [tokens, hidden]: a row holds the prompt, forks share its pages."""
    dev, n = prompt.device, prompt.shape[0]
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    pool = PagePool.new(layer.plan, layer.cache, count + 1, -(-(n + tokens) // page) + 1)
    y, r, ok = layer.step(prompt, torch.zeros_like(prompt), weight, pool, ints(0), ints(n), ints(0, n))
    forks = torch.arange(1, count + 1, dtype=torch.int32, device=dev)
    forked = pool.fork(torch.zeros_like(forks), forks)
    x, res = y[-1:].repeat(count, 1), r[-1:].repeat(count, 1)
    each, one = torch.arange(count + 1, dtype=torch.int32, device=dev), torch.ones_like(forks)
    for _ in range(tokens):
        x, res, grown = layer.step(x, res, weight, pool, forks, one, each)
        ok = torch.cat([ok, grown])
    used = int((pool.refs > 0).sum())
    if not bool(ok.all()) or not bool(forked.all()):
        raise SystemExit("no pages left")
    print("answers: %d forks of %d tokens, %d more each, on %d pages" % (count, n, tokens, used))
    pool.release(forks)
    pool.compact()
    return x


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--heads", type=int, nargs=2, default=[16, 4], metavar=("QUERY", "KV"))
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 33, 1])
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--answers", type=int, default=0, metavar="N", help="forks of the first prompt, each answered by itself")
    a = ap.parse_args(argv)
    dev, page = "cuda", 64
    g = torch.Generator(dev).manual_seed(0)
    (hq, hk), n = a.heads, len(a.prompts)
    need = [-(-(p + a.steps) // page) for p in a.prompts]
    width = (hq + 2 * hk) * a.dim
    w_qkv = (torch.randn(width, a.hidden, generator=g, device=dev) * a.hidden ** -0.5).bfloat16()
    w_out = (torch.randn(a.hidden, hq * a.dim, generator=g, device=dev) * (hq * a.dim) ** -0.5).bfloat16()
    spare = need[0] + 2 * a.answers if a.answers else 0
    layer = AttentionLayer(a.hidden, hq, hk, a.dim, w_qkv, w_out, max(sum(a.prompts), n, a.answers), sum(need) + spare, page)
    if a.answers:
        x = torch.randn(a.prompts[0], a.hidden, generator=torch.Generator(dev).manual_seed(1), device=dev).bfloat16()
        answers(layer, a.answers, a.steps, x, torch.ones(a.hidden, dtype=torch.bfloat16, device=dev), page)
    table = torch.full((n, max(need)), -1, dtype=torch.int32, device=dev)
    ids = iter(torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)).tolist())
    for b, pages in enumerate(need):
        table[b, :pages] = torch.tensor([next(ids) for _ in range(pages)], dtype=torch.int32)

    cu = torch.tensor([sum(a.prompts[:i]) for i in range(n + 1)], dtype=torch.int32, device=dev)
    y = layer.prompt(torch.randn(sum(a.prompts), a.hidden, generator=g, device=dev).bfloat16(), table, cu)
    print("prompt: %d tokens of %d sequences -> %s" % (sum(a.prompts), n, tuple(y.shape)))

    # one decode step, captured once and replayed with the lengths advancing in place
    x, ctx = y[(cu[1:] - 1).long()].clone(), (cu[1:] - cu[:-1]).clone()
    each = torch.arange(n + 1, dtype=torch.int32, device=dev)
    layer.decode(x, table, ctx, each)  # warm-up, outside the capture; the replay writes the same tokens again
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step = layer.decode(x, table, ctx, each)
    t0, t1 = torch.cuda.Event(True), torch.cuda.Event(True)
    t0.record()
    for _ in range(a.steps):
        graph.replay()
        x.copy_(step)
        ctx.add_(1)
    t1.record()
    torch.cuda.synchronize()
    print("decode: %d steps of %d sequences, %.1f us a step" % (a.steps, n, 1e3 * t0.elapsed_time(t1) / a.steps))
    if not bool(torch.isfinite(step.float()).all()):
        raise SystemExit("non-finite output")
    return step


if __name__ == "__main__":
    main()
