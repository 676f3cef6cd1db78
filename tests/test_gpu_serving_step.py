"""Norm, GEMM, page pool, append and chunk together, as a server's layer runs them (examples/attention_layer.py)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")
    import gpu_util

    gpu_util.lib_ready()
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _layer(example, hidden=512, hq=8, hk=2, d=64, page=32, pages=40):
    g = torch.Generator("cuda").manual_seed(5)
    w_qkv = (torch.randn((hq + 2 * hk) * d, hidden, generator=g, device="cuda") * hidden ** -0.5).bfloat16()
    w_out = (torch.randn(hidden, hq * d, generator=g, device="cuda") * (hq * d) ** -0.5).bfloat16()
    weight = (1 + 0.2 * torch.randn(hidden, generator=g, device="cuda")).bfloat16()
    return example.AttentionLayer(hidden, hq, hk, d, w_qkv, w_out, 512, pages, page), weight, g


def test_forks_continue_as_sequences_of_their_own(example):
    """A prompt, forked three times, each fork with a chunk of its own length, against sequences that share nothing.  The kernel
    deals the work of the two batches out differently: sums in another order, weights of other references, so outputs may
    lie a bf16 step apart, and what follows rounds them again."""
    layer, weight, g = _layer(example)
    n, more = 70, [5, 1, 40]
    prompt = torch.randn(n, 512, generator=g, device="cuda").bfloat16()
    rest = [torch.randn(m, 512, generator=g, device="cuda").bfloat16() for m in more]
    pool = example.PagePool.new(layer.plan, layer.cache, 4, 4)
    zero = torch.zeros_like(prompt)
    layer.step(prompt, zero, weight, pool, ints(0), ints(n), ints(0, n))
    assert pool.fork(ints(0, 0, 0), ints(1, 2, 3)).tolist() == [1, 1, 1]
    cu = ints(0, 5, 6, 46)
    x = torch.cat(rest)
    y, r, ok = layer.step(x, torch.zeros_like(x), weight, pool, ints(1, 2, 3), ints(*more), cu)
    assert ok.tolist() == [1, 1, 1] and torch.equal(r, x)
    # 70 tokens are two full pages, shared, and a third that each has for itself; the longest fork has a fourth
    assert int((pool.refs > 0).sum()) == 2 + 4 + 1 and pool.lens.tolist() == [70, 75, 71, 110]
    lone, _, _ = _layer(example)
    own = example.PagePool.new(lone.plan, lone.cache, 3, 4)
    t0 = 0
    for i, m in enumerate(more):
        lone.step(prompt, zero, weight, own, ints(i), ints(n), ints(0, n))
        want, _, _ = lone.step(rest[i], torch.zeros_like(rest[i]), weight, own, ints(i), ints(m), ints(0, m))
        got = y[t0:t0 + m].float()
        assert float((got - want.float()).norm() / want.float().norm()) < 2.0 ** -5
        t0 += m


def test_chunk_of_a_step_against_its_cache(example):
    """What the step's chunk attends over is what the cache holds."""
    layer, weight, g = _layer(example)
    pool = example.PagePool.new(layer.plan, layer.cache, 2, 6)
    x = torch.randn(150, 512, generator=g, device="cuda").bfloat16()
    layer.step(x[:100], torch.zeros_like(x[:100]), weight, pool, ints(0), ints(100), ints(0, 100))
    codes, scale, _ = example.norm_quantize("ptpc", x[100:], weight)
    q, k, v = layer._heads(codes, scale, x[100:])
    before = pool.lens[:1].clone()
    assert pool.grow(ints(0), ints(50)).tolist() == [1]
    q, _ = layer.plan.append(q, k, v, layer.cache, pool.table[:1], before, ints(0, 50))
    out, lse = layer.plan.chunk(q, layer.cache, pool.table[:1], pool.lens[:1], ints(0, 50))
    host = [t.cpu().numpy() for t in (layer.cache.k, layer.cache.k_scale, layer.cache.v, layer.cache.v_scale)]
    table = pool.table[0].cpu().numpy()
    kk, _ = ref.cached(host[0], host[1], table, 2, 32, 150)
    vv, _ = ref.cached(host[2], host[3], table, 2, 32, 150)
    o, ls, mag, big = ref.attend(q.float().cpu().numpy().astype(np.float64), kk, vv, 101 + np.arange(50), 64 ** -0.5)
    assert (np.abs(out.float().cpu().numpy() - o) <= ref.out_tolerance(o, mag, 11)).all()
    assert (np.abs(lse.cpu().numpy() - ls) <= ref.lse_tolerance(ls, big)).all()
    # the same sequence where its pages went: the same bits
    pool.compact()
    again, _ = layer.plan.chunk(q, layer.cache, pool.table[:1], pool.lens[:1], ints(0, 50))
    assert torch.equal(again, out)


def test_a_captured_step(example):
    """A step of single tokens as a graph: the pool grows inside it, replay after replay."""
    layer, weight, g = _layer(example)
    pool = example.PagePool.new(layer.plan, layer.cache, 2, 6)
    x = torch.randn(40, 512, generator=g, device="cuda").bfloat16()
    layer.step(x, torch.zeros_like(x), weight, pool, ints(0, 1), ints(30, 10), ints(0, 30, 40))
    token, res, rows, one, each = x[:2].clone(), torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda"), ints(0, 1), ints(1, 1), ints(0, 1, 2)
    state = [t.clone() for t in (pool.table, pool.lens, pool.refs, layer.cache.k, layer.cache.v, layer.cache.k_scale, layer.cache.v_scale)]
    plain = [layer.step(token, res, weight, pool, rows, one, each)[0].clone() for _ in range(4)]
    for t, s in zip((pool.table, pool.lens, pool.refs, layer.cache.k, layer.cache.v, layer.cache.k_scale, layer.cache.v_scale), state):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _, ok = layer.step(token, res, weight, pool, rows, one, each)
    for want in plain:
        graph.replay()
        assert ok.tolist() == [1, 1] and torch.equal(y, want)
    assert pool.lens.tolist() == [34, 14]


def test_command(example, capsys):
    example.main(["--hidden", "512", "--heads", "8", "2", "--dim", "64", "--prompts", "130", "7", "--steps", "3", "--answers", "5"])
    assert "answers: 5 forks of 130 tokens, 3 more each" in capsys.readouterr().out


def test_a_row_that_gets_no_pages_is_left_alone(example):
    """Its cache and length stay as they were, its tokens see nothing, and the other rows are as in a step without it."""
    layer, weight, g = _layer(example, pages=4)
    pool = example.PagePool.new(layer.plan, layer.cache, 2, 4)
    x = torch.randn(90, 512, generator=g, device="cuda").bfloat16()
    layer.step(x[:60], torch.zeros_like(x[:60]), weight, pool, ints(0, 1), ints(40, 20), ints(0, 40, 60))  # 2 pages and 1
    cache = (layer.cache.k, layer.cache.v, layer.cache.k_scale, layer.cache.v_scale)
    before = [t.clone() for t in cache + (pool.table, pool.lens, pool.refs)]
    # row 0 gets the last page for its 70 tokens, and there is none for row 1, which has room for 12 of its 15 in the page that it holds
    lone, _, _ = layer.step(x[60:], torch.zeros_like(x[60:]), weight, pool, ints(0), ints(30), ints(0, 30))
    for t, b in zip(cache + (pool.table, pool.lens, pool.refs), before):
        t.copy_(b)
    both = torch.cat([x[60:], x[60:75]])
    y, r, ok = layer.step(both, torch.zeros_like(both), weight, pool, ints(0, 1), ints(30, 15), ints(0, 30, 45))
    assert ok.tolist() == [1, 0] and pool.lens.tolist() == [70, 20]
    page = int(before[4][1, 0])
    for t, b in zip(cache, before):
        assert torch.equal(t[page], b[page])
    assert torch.equal(pool.table[1], before[4][1]) and torch.equal(r, both)
    assert bool((y[30:] == 0).all())
    got, want = y[:30].float(), lone.float()
    assert float((got - want).norm() / want.norm()) < 2.0 ** -5
