"""Attention of chunks over the paged cache (scaled_attn_chunk) against 64-bit arithmetic (attn_ref).

Tolerances.  The output: half a bf16 step, fp16 weights (2^-11 of each, and 2^-31 of the row's largest for light ones), fp32
scores, exponentials and sums (attn_ref.out_tolerance).  Scores: products and sums in fp32, as
attn_ref.lse_tolerance has them, and a query's elements below 2^-13 of its row's largest, which are off by
up to 2^-21 of that (tests/test_chunk_terms.py): a score moves by at most 2^-21 max|q| sum|k|, and so does the logarithm of the sum; a weight
moves by that share of itself, and the output by twice that share of sum w |v| (weights and their sum)."""
import ctypes

import numpy as np
import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")
    import gpu_util

    gpu_util.lib_ready()


def _pkg():
    import fp8_scaled_gemm_sm_gb300 as pkg

    return pkg


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _cum(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _ints(x):
    return _dev(np.array(x, np.int32))


def _cache(lens, hk, page, d, seed, scale=(114, 124)):
    """Tables over shuffled pages; what no token has been written to holds NaN codes and any scale."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    ids = iter(rng.permutation(pages))
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    codes = [np.full((pages, hk, page, d), 0x7F, np.uint8) for _ in range(2)]
    scales = [np.full((pages, hk, page // 16), 255, np.uint8) for _ in range(2)]
    for b, n in enumerate(lens):
        for i in range(need[b]):
            pg = table[b, i] = next(ids)
            m = min(n - i * page, page)
            for c, s in zip(codes, scales):
                c[pg, :, :m] = ref.e4m3_round(rng.normal(size=(hk, m, d)) * 100)
                s[pg, :, :-(-m // 16)] = rng.integers(scale[0], scale[1], (hk, -(-m // 16)))
    return table, codes, scales


class Case:
    def __init__(self, hq, hk, d, page, new, ctx, seed, edit=None, q_scale=2.0, scale=None, **kw):
        self.hq, self.hk, self.d, self.page, self.new = hq, hk, d, page, new
        self.lens = [a + b for a, b in zip(new, ctx)]
        self.host = _cache(self.lens, hk, page, d, seed, **kw)
        if edit:
            edit(*self.host)
        pkg = _pkg()
        self.plan = pkg.PagedAttention(hq, hk, d, page)
        self.cache = pkg.KVCache(*[_dev(c) for c in self.host[1]], *[_dev(s) for s in self.host[2]])
        g = torch.Generator("cpu").manual_seed(seed)
        # a view of rows that are longer
        self.q = (torch.randn(sum(new), hq + 1, d, generator=g) * q_scale).bfloat16().cuda()[:, :hq]
        self.scale = d ** -0.5 if scale is None else scale
        self.args = [_dev(self.host[0]), _ints(self.lens), _ints(_cum(new))]

    def run(self, **kw):
        out, lse = self.plan.chunk(self.q, self.cache, *self.args, scale=self.scale, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, q=None, lens=None, rows=None):
        """rows: of each sequence, those that are looked at (all)."""
        table, codes, scales = self.host
        go, gl, qh = _f64(out), _f64(lse), _f64(self.q if q is None else q)
        t0 = 0
        for b, n in enumerate(self.new):
            m = self.lens[b] if lens is None else lens[b]
            m = min(max(m, 0), table.shape[1] * self.page)
            if n == 0:
                continue
            k, has = ref.cached(codes[0], scales[0], table[b], self.hk, self.page, m)
            v, _ = ref.cached(codes[1], scales[1], table[b], self.hk, self.page, m)
            i = np.arange(n) if rows is None else np.array(sorted({x % n for x in rows}))
            see = np.maximum(m - (n - 1 - i), 0)
            vis = (np.arange(m)[None, :] < see[:, None]) & has[None, :]
            o, ls, mag, big = ref.attend(qh[t0 + i], k, v, vis, self.scale)
            # what light weights and a row's smallest elements may add
            kk = np.abs(np.nan_to_num(k)).sum(2).max(0, initial=0).repeat(self.hq // self.hk)
            vv = np.abs(np.nan_to_num(v)).max((0, 2), initial=0).repeat(self.hq // self.hk)
            small = 2.0 ** -21 * np.abs(np.nan_to_num(qh[t0 + i])).max(2) * kk[None] * self.scale
            tol = ref.out_tolerance(o, mag, 11) + 2 * small[..., None] * mag + (m * 2.0 ** -31 * vv)[None, :, None]
            err = np.abs(go[t0 + i] - o)
            assert (err <= tol).all(), (b, n, m, np.argwhere(~(err <= tol))[:4].tolist(), float(np.nanmax(err / tol)))
            assert np.array_equal(np.isinf(gl[t0 + i]), np.isinf(ls)), (b, n, m)
            fin = np.isfinite(ls)
            assert (np.abs(gl[t0 + i][fin] - ls[fin]) <= (ref.lse_tolerance(ls, big) + small)[fin]).all(), (b, n, m)
            t0 += n


CASES = [
    # hq, hk, d, page, new tokens, tokens before
    (8, 2, 128, 64, [5], [40]),
    (4, 4, 64, 16, [1, 0, 17, 130], [0, 9, 300, 64]),
    (10, 2, 96, 32, [33, 64, 1], [500, 0, 127]),
    (5, 1, 80, 128, [26, 25, 51, 200], [100, 3, 0, 513]),
    (2, 2, 16, 16, [7, 40], [20, 0]),
    (3, 1, 112, 16, [43, 86, 128], [128, 42, 600]),
    (128, 1, 128, 32, [3, 1], [200, 0]),
    (256, 1, 64, 64, [2, 3], [100, 129]),
    (1, 1, 128, 128, [128, 129, 256, 257, 255], [0, 0, 128, 127, 1]),
    (8, 2, 128, 64, [300], [2000]),
    (4, 1, 128, 64, [64, 65, 96, 32, 31, 33], [64, 63, 160, 96, 97, 95]),
    (16, 16, 32, 16, [20, 3], [50, 700]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_chunk(case):
    c = Case(*CASES[case], seed=300 + case)
    out, lse = c.run()
    c.check(out, lse)
    for _ in range(3):
        again = c.run()  # the same bits
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    from fp8_scaled_gemm_sm_gb300 import binding

    assert binding.scaled_attn_debug_status(c.plan.handle)[0] == 0


@pytest.mark.parametrize("B,hq,hk,d,long", [(30, 4, 2, 64, 900), (500, 2, 1, 128, 700), (1300, 1, 1, 64, 300)])
def test_many_sequences(B, hq, hk, d, long):
    rng = np.random.default_rng(B)
    new = [int(x) for x in rng.integers(0, 4, B)]
    ctx = [int(x) for x in rng.integers(0, 60, B)]
    for b in (0, B // 2, B - 1):
        new[b], ctx[b] = 40 + b % 7, long
    ctx[1], new[1] = 0, 1
    c = Case(hq, hk, d, 16, new, ctx, seed=B)
    c.check(*c.run())


@pytest.mark.parametrize("hq,hk,d,new,ctx", [
    (2, 1, 128, [3], [20011]),              # one unit over every CTA
    (8, 2, 64, [2, 40], [9000, 5000]),
    (4, 1, 128, [80], [12000]),             # two row tiles, cut
    (4, 4, 128, [1, 1, 1], [6000, 1, 3000]),
])
def test_cut_units(hq, hk, d, new, ctx):
    c = Case(hq, hk, d, 64, new, ctx, seed=sum(ctx))
    c.check(*c.run(), rows=[0, 1, 31, -1])


def test_more_tokens_than_keys():
    """The first rows of a chunk that is longer than its sequence see nothing."""
    c = Case(4, 2, 64, 16, [50, 3, 200], [0, 0, 0], seed=5)
    lens = [20, 0, 61]
    c.args[1] = _ints(lens)
    out, lse = c.run()
    c.check(out, lse, lens=lens)
    assert bool((out[:30] == 0).all()) and bool(torch.isinf(lse[:30]).all()) and bool((out[50:53] == 0).all())


def test_missing_pages_are_not_seen():
    def edit(table, codes, scales):
        table[0, 1] = -1
        table[1, 0] = codes[0].shape[0]
        table[1, 3] = -7
        table[2, :] = -1

    c = Case(4, 2, 64, 16, [10, 30, 5], [100, 130, 48], seed=6, edit=edit)
    out, lse = c.run()
    c.check(out, lse)
    assert bool((out[40:] == 0).all()) and bool(torch.isinf(lse[40:]).all())


def test_lengths_outside_the_table():
    c = Case(4, 2, 64, 32, [6, 3], [58, 37], seed=7)
    c.args[1] = _ints([5000, -3])
    c.check(*c.run(), lens=[5000, -3])


@pytest.mark.parametrize("kind", ["value scales far apart", "zero blocks", "large scores", "equal scores", "huge scores", "light values"])
@pytest.mark.parametrize("new,ctx", [([12, 3, 90], [150, 33, 16])])
def test_extreme_scales(kind, new, ctx):
    def edit(table, codes, scales):
        if kind == "value scales far apart":
            scales[1][scales[1] < 255] = np.random.default_rng(1).integers(60, 190, (scales[1] < 255).sum())
        elif kind == "zero blocks":
            for n in (0, 1):
                codes[n][table[0, 1]] = 0
                scales[n][table[0, 1]] = 0
            codes[1][table[1, 0]] = 0
            scales[1][table[1, 0]] = 0
        elif kind == "large scores":
            scales[0][scales[0] < 255] = 126
        elif kind == "huge scores":
            scales[0][scales[0] < 255] = 145
        elif kind == "light values":  # all values near bf16's least normal ones
            scales[1][scales[1] < 255] = 12
        else:
            codes[0][(codes[0] & 127) != 127] = 0

    c = Case(4, 2, 64, 16, new, ctx, seed=8, edit=edit, q_scale=0.5 if kind == "large scores" else 2.0)
    c.check(*c.run())


def test_rows_of_very_different_size():
    c = Case(6, 1, 128, 32, [5, 70], [90, 200], seed=9)
    size = torch.tensor([1e-30, 1e-6, 1.0, 30.0, 0.0, 1e-2], device="cuda")[None, :, None]
    c.q = (c.q.float() * size).bfloat16()
    c.check(*c.run())


def test_queries_with_outliers():
    """One dimension far above the others, whose keys are zero there: what is left of the small ones decides."""
    def edit(table, codes, scales):
        codes[0][..., 5][(codes[0][..., 5] & 127) != 127] = 0

    c = Case(4, 2, 128, 32, [9, 40], [300, 77], seed=10, edit=edit)
    for k in (6, 12, 16):
        q = c.q.clone()
        q[:, :, 5] = 2.0 ** k
        c.q = q
        c.check(*c.run())


def test_rows_that_are_not_finite_stay_alone():
    c = Case(6, 2, 64, 16, [40, 7], [70, 33], seed=11)
    clean = c.run()
    c.q = c.q.clone()
    c.q[3, 1, 3] = float("nan")
    c.q[44, 5, 0] = float("inf")
    out, lse = c.run()
    for r, h in ((3, 1), (44, 5)):
        assert bool(torch.isnan(out[r, h].float()).all()) and bool(torch.isnan(lse[r, h]))
        out[r, h], lse[r, h] = clean[0][r, h], clean[1][r, h]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 1, 128)])
def test_keys_and_values_that_are_not_finite(hq, hk, d):
    """A NaN reaches the rows that see it and, of a value, rows of its row tile before it in that dimension (zero times NaN)."""
    c = Case(hq, hk, d, 16, [30, 25], [100, 60], seed=12)
    clean = c.run()
    for what in ("key code", "value code", "key scale", "value scale"):
        codes, scales = [c.cache.k.clone(), c.cache.v.clone()], [c.cache.k_scale.clone(), c.cache.v_scale.clone()]
        which, key = what.startswith("value"), 110  # the context's 100 keys, and row 10 of the new ones
        pg, slot = int(c.host[0][0, key // 16]), key % 16
        if what.endswith("code"):
            codes[which][pg, 0, slot, 3] = 0x7F
            first, dims = key - 100, slice(3, 4)
        else:
            scales[which][pg, 0, slot // 16] = 255
            first, dims = 0, slice(0, d)  # the block's first keys, 96 to 99, are before the new tokens: every row sees them
        cache = _pkg().KVCache(*codes, *scales)
        out, lse = c.plan.chunk(c.q, cache, *c.args)
        torch.cuda.synchronize()
        sees = slice(first, 30)
        heads = slice(0, hq // hk)
        if which:
            assert bool(torch.isnan(out[sees, heads, dims].float()).all())
            # the weights know nothing of values
            assert torch.allclose(lse, clean[1], rtol=0, atol=1e-4)
            out[:30, heads, dims] = clean[0][:30, heads, dims]
            tol = 2.0 ** -7 * clean[0].float().abs() + 2.0 ** -9 * 2000
        else:
            assert bool(torch.isnan(out[sees, heads].float()).all()) and bool(torch.isnan(lse[sees, heads]).all())
            out[sees, heads], lse[sees, heads] = clean[0][sees, heads], clean[1][sees, heads]
            assert torch.allclose(lse, clean[1], rtol=0, atol=1e-4)
            tol = 2.0 ** -7 * clean[0].float().abs() + 2.0 ** -9 * 2000
        assert bool(((out.float() - clean[0].float()).abs() <= tol).all()), what


def test_agrees_with_decode():
    """Chunks of equal length are what decode takes."""
    c = Case(8, 2, 128, 64, [4] * 20, list(range(0, 4000, 200)), seed=13)
    out, lse = c.run()
    want = c.plan.decode(c.q, c.cache, c.args[0], c.args[1], q_tokens=4)
    torch.cuda.synchronize()
    c.check(out, lse)
    c.check(*want)


def test_rows_behind_the_last_sequence_are_not_written():
    c = Case(4, 2, 64, 16, [5, 9, 20], [30, 0, 11], seed=14)
    out = torch.full((34, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((34, 4), 7.0, device="cuda")
    c.args[2] = _ints([0, 5, 14, 14])
    c.run(out=out, lse=lse)
    assert bool((out[14:] == 7).all()) and bool((lse[14:] == 7).all())
    c.new = [5, 9, 0]
    c.check(out, lse)


def test_offsets_past_32_bits():
    """Pages far apart: the last ones start beyond 4 GiB of codes."""
    pkg = _pkg()
    hk, page, d, pages = 1, 128, 128, 70
    step = 80 << 20
    c = Case(2, hk, d, page, [40, 3], [260, 254], seed=15)
    big = [torch.empty(pages * step, dtype=torch.uint8, device="cuda") for _ in range(2)]
    views = [b.as_strided((pages, hk, page, d), (step, page * d, d, 1)) for b in big]
    where = {int(p): 69 - i for i, p in enumerate(c.host[0][c.host[0] >= 0])}
    scales = [torch.zeros(pages, hk, page // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for a, b in where.items():
        for n in (0, 1):
            views[n][b] = (c.cache.k, c.cache.v)[n][a]
            scales[n][b] = (c.cache.k_scale, c.cache.v_scale)[n][a]
    c.args[0] = _dev(np.vectorize(lambda p: where.get(int(p), -1))(c.host[0]).astype(np.int32))
    c.cache = pkg.KVCache(views[0], views[1], *scales)
    c.check(*c.run())


def test_lengths_up_to_31_bits():
    """A table whose pages are nearly all missing: the numbers of keys and of work pass 2^31."""
    pkg = _pkg()
    plan = pkg.PagedAttention(2, 1, 64, 128)
    width = (1 << 31) // 128 - 1
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(3)
    codes = [ref.e4m3_round(rng.normal(size=(3, 1, 128, 64)) * 100) for _ in range(2)]
    scales = [rng.integers(114, 122, (3, 1, 8)).astype(np.uint8) for _ in range(2)]
    table[0, 0], table[0, -1], table[1, 5] = 1, 2, 0
    n = [300, 2]
    lens = [width * 128 - 40, 700]
    q = torch.randn(302, 2, 64, generator=torch.Generator("cpu").manual_seed(1)).bfloat16().cuda()
    out, lse = plan.chunk(q, pkg.KVCache(*[_dev(x) for x in codes], *[_dev(x) for x in scales]), table, _ints(lens), _ints(_cum(n)))
    torch.cuda.synchronize()
    val = [ref.E4M3[x[:, 0].reshape(3, 128, 64)] * ref.pow2(s[:, 0]).repeat(16, 1)[..., None] for x, s in zip(codes, scales)]
    # sequence 0: the first page, and what rows see of the last
    k, v = (np.concatenate([x[1], x[2]])[:, None] for x in val)
    last = (width - 1) * 128
    see = np.array([128 + min(max(lens[0] - 299 + i - last, 0), 128) for i in range(300)])
    o, ls, mag, big = ref.attend(_f64(q[:300]), k, v, see, 64 ** -0.5)
    assert (np.abs(_f64(out[:300]) - o) <= ref.out_tolerance(o, mag, 11)).all()
    assert (np.abs(_f64(lse[:300]) - ls) <= ref.lse_tolerance(ls, big)).all()
    vis = np.arange(128)[None, :] + 5 * 128 < (np.array([699, 700])[:, None])
    o, ls, mag, big = ref.attend(_f64(q[300:]), val[0][0][:, None], val[1][0][:, None], vis, 64 ** -0.5)
    assert (np.abs(_f64(out[300:]) - o) <= ref.out_tolerance(o, mag, 11)).all()


def test_captured_and_replayed_with_other_lengths():
    c = Case(8, 2, 128, 64, [40, 3, 100], [0, 700, 5], seed=16)
    out, lse = torch.empty(143, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(143, 8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.plan.chunk(c.q, c.cache, *c.args, out=out, lse=lse)
    graph.replay()
    c.check(out, lse)
    for new, lens in (([1, 70, 72], [30, 703, 105]), ([143, 0, 0], [143, 5, 9]), ([40, 3, 100], c.lens)):
        # within the pages that each sequence has
        lens = [min(x, y) for x, y in zip(lens, c.lens)]
        c.args[1].copy_(_ints(lens))
        c.args[2].copy_(_ints(_cum(new)))
        graph.replay()
        c.new = new
        c.check(out, lse, lens=lens)


def test_two_plans_on_two_streams():
    a, b = Case(8, 2, 128, 64, [200, 30], [3000, 500], seed=17), Case(4, 4, 64, 16, [60, 61], [900, 20], seed=18)
    want = [x.run() for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for x, s in zip((a, b), streams):
            s.wait_stream(torch.cuda.current_stream())
            got.append(x.plan.chunk(x.q, x.cache, *x.args, scale=x.scale, stream=s.cuda_stream))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], want[i % 2][0]) and torch.equal(g[1], want[i % 2][1])


def test_between_decodes_on_one_plan():
    """The workspace that both use: in a row on one stream."""
    c = Case(8, 2, 128, 64, [2, 2, 2], [9000, 40, 700], seed=19)
    out, lse = c.run()
    dec = c.plan.decode(c.q, c.cache, c.args[0], c.args[1], q_tokens=2)
    for _ in range(10):
        o1 = c.plan.chunk(c.q, c.cache, *c.args, scale=c.scale)
        d1 = c.plan.decode(c.q, c.cache, c.args[0], c.args[1], q_tokens=2)
    torch.cuda.synchronize()
    assert torch.equal(o1[0], out) and torch.equal(d1[0], dec[0])


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (6, 6, 64)])
def test_other_batches_in_a_row_on_one_plan(hq, hk, d):
    """Parts and cut units of one call are not those of the next: the whole batch, its first sequence, the others, in turn."""
    c = Case(hq, hk, d, 32, [70, 300, 3, 129], [6000, 40, 9000, 1300], seed=21)
    table, lens, cu = c.args
    parts = []
    for first, last in ((0, 4), (0, 1), (1, 4), (2, 3)):
        lo, hi = (int(cu[i]) for i in (first, last))
        parts.append((c.q[lo:hi], table[first:last], lens[first:last], cu[first:last + 1] - cu[first]))
    call = lambda q, *rest: c.plan.chunk(q, c.cache, *rest, scale=c.scale)  # noqa: E731
    want = []
    for x in parts:
        want.append(call(*x))
        torch.cuda.synchronize()
    c.check(*want[0])
    got = [call(*x) for _ in range(4) for x in parts]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], want[i % 4][0]) and torch.equal(g[1], want[i % 4][1])


@pytest.mark.parametrize("hq,hk,d,new,ctx,tile", [(8, 2, 128, [30, 100], [500, 900], 0), (4, 4, 64, [5, 9], [3000, 100], 3), (4, 1, 128, [2], [9000], 40)])
def test_gives_up(hq, hk, d, new, ctx, tile):
    """A load that never comes: the call ends, says so, and the next one is right."""
    from fp8_scaled_gemm_sm_gb300 import binding

    c = Case(hq, hk, d, 64, new, ctx, seed=20)
    want = c.run()
    binding.scaled_attn_set_debug(c.plan.handle, 20_000_000, tile)
    c.run()
    code, where = binding.scaled_attn_debug_status(c.plan.handle)
    assert code == 6 and where != 0
    binding.scaled_attn_set_debug(c.plan.handle, 0, -1)
    got = c.run()
    assert binding.scaled_attn_debug_status(c.plan.handle)[0] == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_without_pages_or_tokens():
    pkg = _pkg()
    c = Case(4, 2, 64, 16, [5, 9], [30, 0], seed=21)
    out, lse = c.plan.chunk(c.q, c.plan.new_cache(0), *c.args)
    assert bool((out == 0).all()) and bool(torch.isinf(lse).all())
    out, lse = c.plan.chunk(c.q[:0], c.cache, *c.args)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    kept = torch.full_like(c.q, 3.0)
    c.plan.chunk(c.q, c.cache, c.args[0][:0], none, _ints([0]), out=kept)
    torch.cuda.synchronize()
    assert bool((kept == 3).all())
    assert pkg is not None


def test_refusals():
    from fp8_scaled_gemm_sm_gb300 import ScaledGemmError, binding

    c = Case(4, 2, 64, 16, [5, 9], [30, 0], seed=22)
    t, n, cu = c.args
    for bad in ((c.q.float(), c.cache, t, n, cu), (c.q[:, :2], c.cache, t, n, cu), (c.q, c.cache, t.long(), n, cu), (c.q, c.cache, t[:1], n, cu),
                (c.q, c.cache, t, n, cu[:2]), (c.q, c.cache, t, n.cpu(), cu), (c.q, c.plan.new_cache(3), t, n, None)):
        with pytest.raises((ValueError, TypeError)):
            c.plan.chunk(*bad)
    with pytest.raises(ValueError):
        c.plan.chunk(c.q, _pkg().KVCache.new(4, 2, 32, 64), t, n, cu)
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(ScaledGemmError):
            c.plan.chunk(c.q, c.cache, t, n, cu, scale=scale)
    q = c.q.contiguous()
    with pytest.raises(ScaledGemmError):
        c.plan.chunk(q, c.cache, t, n, cu, out=q)
    L, h = binding.lib(), c.plan.handle
    args = binding.KvCacheArgs(*(x.data_ptr() for x in (c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale)), c.cache.k.shape[0],
                               c.cache.k.stride(0), c.cache.v.stride(0))
    out = torch.empty_like(q)
    good = [h, ctypes.byref(args), q.data_ptr(), 256, t.data_ptr(), t.shape[1], n.data_ptr(), cu.data_ptr(), 14, 2, 0.1, out.data_ptr(), None, None]
    for i, v, status in ((0, None, 1), (1, None, 1), (2, None, 1), (2, q.data_ptr() + 2, 3), (3, 248, 1), (3, 257, 3), (4, None, 1), (5, -1, 1), (5, 1 << 30, 2), (6, None, 1), (7, None, 1),
                         (7, cu.data_ptr() + 2, 3), (8, -1, 1), (8, 1 << 31, 2), (9, -1, 1), (9, 1 << 25, 2), (11, None, 1), (11, out.data_ptr() + 8, 3), (12, out.data_ptr() + 2, 3)):
        a = list(good)
        a[i] = v
        assert L.scaled_attn_chunk(*a) == status, (i, v)
    assert L.scaled_attn_chunk(*good) == 0
    torch.cuda.synchronize()


def test_infinite_queries_that_see_no_key():
    """Zero and -infinity as for any row that sees nothing, where the rows of its tile after it do: ahead of the sequence's first token, and
    over pages that are not there."""
    def edit(table, codes, scales):
        table[1, :2] = -1

    c = Case(4, 2, 64, 16, [50, 20], [0, 20], seed=23, edit=edit)
    lens = [20, 40]
    c.args[1] = _ints(lens)
    clean = c.run()
    c.check(*clean, lens=lens)
    assert bool((clean[0][:30] == 0).all()) and bool((clean[0][50:62] == 0).all())  # 12 rows see up to 32 keys, none of which is there
    c.q = c.q.clone()
    for r, value in ((7, float("inf")), (29, -float("inf")), (51, float("inf")), (61, float("nan"))):
        c.q[r, 1, 3] = value
    out, lse = c.run()
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    c.q[30, 1, 3] = c.q[62, 1, 3] = float("inf")  # the first rows that see a key
    out, lse = c.run()
    for r in (30, 62):
        assert bool(torch.isnan(out[r, 1].float()).all()) and bool(torch.isnan(lse[r, 1]))
        out[r, 1], lse[r, 1] = clean[0][r, 1], clean[1][r, 1]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("k_code,v_code", [(127, 127), (127, 20), (127, 230), (57, 127)])
def test_sum_of_many_equal_weights(k_code, v_code):
    """Sums of up to 130000 weights of 2^-0.95, with scales that take the slower way too.  A CTA adds up to every second block of a row:
    the sum of a block is off by at most (15 + 7) 2^-24, each of 508 additions by 2^-24 of what they give, the exponential by 2^-22; the
    logarithm's two roundings and the last product's are of numbers below 32, 2^-20 each."""
    pkg = _pkg()
    plan = pkg.PagedAttention(1, 1, 64, 128)
    codes = [torch.zeros(1, 1, 128, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    codes[0][..., 0] = 0x38  # 1
    codes[1][:] = 0x38
    scales = [torch.full((1, 1, 8), x, dtype=torch.uint8, device="cuda") for x in (k_code, v_code)]
    B, most = 160, 130000  # more sequences than CTAs: a range of the work is nearly a sequence
    table = torch.zeros(B, 1016, dtype=torch.int32, device="cuda")
    lens = np.array([most - 37 * b for b in range(B)])
    q = torch.zeros(B, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = 2.0 ** (127 - k_code)
    out, lse = plan.chunk(q, pkg.KVCache(*codes, *scales), table, _ints(lens), _ints(list(range(B + 1))), scale=0.05 * np.log(2))
    torch.cuda.synchronize()
    want = 0.05 * np.log(2) + np.log(lens)
    assert float(np.abs(_f64(lse)[:, 0] - want).max()) <= (15 + 7 + 508) * 2.0 ** -24 + 2.0 ** -22 + 3 * 2.0 ** -20
    value = 2.0 ** (v_code - 127)
    assert bool(((out.double() - value).abs() <= value * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13)).all())


def test_outputs_that_overlap_are_refused():
    """lse over the queries or the output, in each of the attention calls."""
    from fp8_scaled_gemm_sm_gb300 import ScaledGemmError

    c = Case(4, 2, 64, 16, [1, 1, 1], [5, 30, 0], seed=24)
    q = c.q.contiguous()
    n = q.shape[0]
    room = torch.empty(n * 4 * 64, dtype=torch.bfloat16, device="cuda")
    whole = room.view(n, 4, 64)
    kv = torch.randn(n, 2, 64, generator=torch.Generator("cpu").manual_seed(1)).bfloat16().cuda()
    calls = {"chunk": lambda **kw: c.plan.chunk(q, c.cache, *c.args, **kw), "decode": lambda **kw: c.plan.decode(q, c.cache, *c.args[:2], **kw),
             "prompt": lambda **kw: c.plan.prompt(q, kv, kv, c.args[2], **kw)}
    over = lambda t: t.view(-1)[-2 * n * 4:].view(torch.float32).view(n, 4)  # noqa: E731
    for name, call in calls.items():
        for kw in (dict(out=whole, lse=over(room)), dict(lse=over(q)), dict(out=q)) + ((dict(lse=over(kv)),) if name == "prompt" else ()):
            with pytest.raises(ScaledGemmError):
                call(**kw)
        both = torch.empty(n * 4 * 66, dtype=torch.bfloat16, device="cuda")  # side by side
        out, lse = call(out=both[:n * 4 * 64].view(n, 4, 64), lse=both[n * 4 * 64:].view(torch.float32).view(n, 4))
        want = call()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("hq,hk,d,ctx", [(4, 2, 64, 100), (8, 1, 128, 100), (4, 2, 128, 700), (2, 2, 96, 260)])
@pytest.mark.parametrize("what", ["key code", "value code", "key scale", "value scale"])
@pytest.mark.parametrize("row", [0, 12, 29])
def test_what_is_not_finite_leaves_the_rest_right(hq, hk, d, ctx, what, row):
    """One key or value, or one scale, of the new token `row` and head 0 is NaN.  Rows that see it give NaN (a value's code: in its dimension); rows before it may
    where it is a value's; all else of the head is the formula's, and of other heads and sequences the same bits."""
    new, seq = 30, ctx + 30
    c = Case(hq, hk, d, 16, [new, 25], [ctx, 60], seed=25)
    out0, lse0 = c.run()
    table, codes, scales = c.host
    group, which, key, dim = hq // hk, what.startswith("value"), ctx + row, 3
    pg, slot = int(table[0, key // 16]), key % 16
    tensors = [[t.clone() for t in (c.cache.k, c.cache.v)], [t.clone() for t in (c.cache.k_scale, c.cache.v_scale)]]
    if what.endswith("code"):
        tensors[0][which][pg, 0, slot, dim] = 0x7F
        first = key
    else:
        tensors[1][which][pg, 0, slot // 16] = 255
        first = key // 16 * 16
    out, lse = c.plan.chunk(c.q, _pkg().KVCache(*tensors[0], *tensors[1]), *c.args, scale=c.scale)
    torch.cuda.synchronize()
    assert torch.equal(out[new:], out0[new:]) and torch.equal(lse[new:], lse0[new:])
    assert torch.equal(out[:new, group:], out0[:new, group:]) and torch.equal(lse[:new, group:], lse0[:new, group:])
    # head 0's queries, over what was there before
    k, _ = ref.cached(codes[0], scales[0], table[0], hk, 16, seq)
    v, _ = ref.cached(codes[1], scales[1], table[0], hk, 16, seq)
    q = _f64(c.q[:new, :group])
    see = ctx + 1 + np.arange(new)
    o, ls, mag, big = ref.attend(q, k[:, :1], v[:, :1], see, c.scale)
    small = 2.0 ** -21 * np.abs(q).max(2) * np.abs(k[:, 0]).sum(1).max() * c.scale
    tol = ref.out_tolerance(o, mag, 11) + 2 * small[..., None] * mag + seq * 2.0 ** -31 * np.abs(v[:, 0]).max()
    sees = np.broadcast_to((see > first)[:, None, None], o.shape)
    dims = np.zeros(d, bool)
    dims[dim if what == "value code" else slice(None)] = True
    hit = np.broadcast_to(dims, o.shape)
    go, gl = _f64(out[:new, :group]), _f64(lse[:new, :group])
    assert np.isnan(go[sees & hit]).all() and (sees & hit).any()
    right = np.abs(go - o) <= tol
    may = ~sees & hit & np.isnan(go) if which else np.zeros_like(sees)
    assert (right | (sees & hit) | may).all(), (float(np.nanmax(np.abs(go - o) / tol)), np.argwhere(~(right | (sees & hit) | may))[:4].tolist())
    if which:
        assert (np.abs(gl - ls) <= ref.lse_tolerance(ls, big) + small).all()
    else:
        assert np.isnan(gl[sees[..., 0]]).all()
        assert (np.abs(gl - ls) <= ref.lse_tolerance(ls, big) + small)[~sees[..., 0]].all()


def test_terms_of_every_query_value():
    """The kernel's own two terms of each finite bf16 value below 2^8, beside one of 255 in its row: a sequence of one key, which is 1 in the value's dimension and
    zero in the other's, so that lse is the value.  Rounding: of the score by 2^-24 of itself, of the reference and its logarithm added up by as much, of the exponential, the
    sum and the logarithm by 2^-22 each; below 2^-6 the terms leave up to 2^-14."""
    pkg = _pkg()
    bits = np.arange(1 << 16, dtype=np.uint32) << 16
    x = bits.view(np.float32)
    x = x[np.isfinite(x) & (np.abs(x) < 256)]
    heads = 64
    x = np.resize(x, -(-len(x) // heads) * heads).reshape(-1, heads)
    n = len(x)
    plan = pkg.PagedAttention(heads, 1, 64, 16)
    codes = [torch.zeros(1, 1, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    codes[0][..., 1] = 0x38  # 1
    scales = [torch.full((1, 1, 1), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    q = torch.zeros(n, heads, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 255
    q[..., 1] = torch.from_numpy(x).bfloat16().cuda()
    ones = torch.ones(n, dtype=torch.int32, device="cuda")
    _, lse = plan.chunk(q, pkg.KVCache(*codes, *scales), torch.zeros(n, 1, dtype=torch.int32, device="cuda"), ones, _ints(list(range(n + 1))), scale=1.0)
    v = x.astype(np.float64)
    off = np.abs(_f64(lse) - v)
    tol = np.abs(v) * 2.0 ** -21 + 2.0 ** -20 + np.where(np.abs(v) < 2.0 ** -6, 2.0 ** -14, 0)
    assert (off <= tol).all(), (float((off / tol).max()), v.flat[np.argmax(off / tol)])


@pytest.mark.parametrize("B", [1 << 24, (1 << 24) - 33, 40, 33])
def test_idle_sequences_between(B):
    """Up to as many sequences as a call may have, all but the first, one in the middle and the last idle, most of those with keys."""
    from fp8_scaled_gemm_sm_gb300 import binding

    c = Case(4, 2, 64, 16, [3, 1, 40], [60, 20, 11], seed=26)
    want = c.run()
    c.check(*want)
    at = torch.tensor([0, B // 2 + 1, B - 1], device="cuda")
    table = torch.zeros(B, c.args[0].shape[1], dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 30, dtype=torch.int32, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    table[at], lens[at], new[at] = c.args[0], c.args[1], _ints(c.new)
    cu = torch.cat([_ints([0]), new.cumsum(0, dtype=torch.int32)])
    out, lse = c.plan.chunk(c.q, c.cache, table, lens, cu, scale=c.scale)
    torch.cuda.synchronize()
    assert binding.scaled_attn_debug_status(c.plan.handle)[0] == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
