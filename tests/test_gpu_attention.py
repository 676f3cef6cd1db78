"""GPU tests of the attention operators (include/scaled_attention.h) against plain
64-bit implementations (attn_ref), at the sizes, masks, layouts and values where they can go wrong."""
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


def _gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _cum(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _table(lens, page, seed, width=None):
    need = [-(-n // page) for n in lens]
    width = max(max(need), 1) if width is None else width
    rng = np.random.default_rng(seed)
    total = sum(need) + 2
    ids = iter(rng.permutation(total))
    t = np.full((len(lens), width), -1, np.int32)
    for b, n in enumerate(need):
        for i in range(n):
            t[b, i] = next(ids)
    return t, total


def _stale(pages, hk, page, d, seed):
    rng = np.random.default_rng(seed)
    codes = [rng.integers(0, 256, (pages, hk, page, d)).astype(np.uint8) for _ in range(2)]
    scales = [rng.integers(110, 130, (pages, hk, page // 16)).astype(np.uint8) for _ in range(2)]
    return codes, scales


# ------------------------------------------------------------------ append

APPEND = [
    # hq, hk, d, page, rot, interleaved, new tokens, tokens before
    (4, 2, 128, 16, 128, False, [1, 1, 1], [0, 15, 16]),
    (8, 1, 64, 32, 64, True, [1, 0, 17, 16, 15], [31, 5, 1, 0, 16]),
    (3, 3, 96, 64, 48, False, [33, 2, 70], [0, 63, 9]),
    (5, 1, 80, 128, 16, True, [3, 5, 130], [1, 126, 250]),
    (2, 2, 16, 16, 16, False, [20, 7], [3, 0]),
    (6, 2, 112, 32, 0, False, [18], [14]),
    (32, 8, 128, 64, 64, False, [0, 200, 1, 0], [40, 7, 64, 0]),
]


def _append_case(hq, hk, d, page, rot, inter, new, ctx, seed, fill=None, stride_pages=False):
    g = _gen(seed)
    T = sum(new)
    x = torch.randn(T, hq + 2 * hk, d, generator=g)
    x[:, hq:] *= torch.exp(torch.randn(1, 2 * hk, d, generator=g))
    x *= torch.exp(torch.randn(T, 1, 1, generator=g))
    if fill:
        fill(x, hq, hk)
    x = x.bfloat16().cuda()
    table, pages = _table([a + b for a, b in zip(new, ctx)], page, seed)
    codes, scales = _stale(pages, hk, page, d, seed)
    pkg = _pkg()
    cs = pkg.rotary_table(max(a + b for a, b in zip(new, ctx)) + 1, rot, base=1000.0) if rot else None
    plan = pkg.PagedAttention(hq, hk, d, page, rotary=cs, interleaved=inter)
    dc = [_dev(c) for c in codes]
    if stride_pages:  # keys and values of a page next to each other, and a gap
        both = torch.full((pages, 2, hk, page, d), 0xA5, dtype=torch.uint8, device="cuda")
        both = torch.cat([both, torch.full((pages, 1, hk, page, d), 0xA5, dtype=torch.uint8, device="cuda")], 1)
        both[:, 0], both[:, 1] = dc[0], dc[1]
        dc = [both[:, 0], both[:, 1]]
    ds = [_dev(s) for s in scales]
    cache = pkg.KVCache(dc[0], dc[1], ds[0], ds[1])
    return plan, cache, x, table, codes, scales, cs


@pytest.mark.parametrize("case", range(len(APPEND)))
@pytest.mark.parametrize("k_out", [False, True])
def test_append_is_bit_exact(case, k_out):
    hq, hk, d, page, rot, inter, new, ctx = APPEND[case]
    plan, cache, x, table, codes, scales, cs = _append_case(hq, hk, d, page, rot, inter, new, ctx, 100 + case,
                                                            stride_pages=k_out)
    q, k = plan.append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], cache, _dev(table), _dev(np.array(ctx, np.int32)),
                       _dev(_cum(new)), k_out=k_out)
    torch.cuda.synchronize()
    h = x.float().cpu().numpy()
    rq, rk = ref.append(h[:, :hq], h[:, hq:hq + hk], h[:, hq + hk:], codes, scales, table, ctx, _cum(new),
                        None if cs is None else cs.cpu().numpy(), inter)
    assert torch.equal(q.cpu(), torch.from_numpy(rq).bfloat16())
    assert (k is None) == (not k_out)
    if k_out:
        assert torch.equal(k.cpu(), torch.from_numpy(rk).bfloat16())
    for got, want in ((cache.k_scale, scales[0]), (cache.v_scale, scales[1])):
        assert np.array_equal(got.cpu().numpy(), want)
    for got, want in ((cache.k, codes[0]), (cache.v, codes[1])):
        bad = np.argwhere(got.cpu().numpy() != want)
        # a NaN's sign is not kept when its block grows
        assert all((want[tuple(i)] & 127) == 127 and (int(got[tuple(i)]) & 127) == 127 for i in bad), bad[:5]
    if k_out:  # the gap between strided pages is untouched
        base = cache.k._base if cache.k._base is not None else cache.k
        assert bool((base[:, 2] == 0xA5).all())


def test_append_token_by_token_grows_scales_and_keeps_older_tokens():
    # one token at a time, each larger than the last: every append grows the block's
    # scale and rounds the older codes again
    hq, hk, d, page, n = 2, 2, 64, 16, 37
    plan, cache, x, table, codes, scales, _ = _append_case(hq, hk, d, page, 0, False, [n], [0], 7)
    x = (torch.randn(n, hq + 2 * hk, d, generator=_gen(3)) * torch.exp2(torch.arange(n).float() / 2 - 12)[:, None, None]).bfloat16().cuda()
    h = x.float().cpu().numpy()
    for t in range(n):
        plan.append(x[t:t + 1, :hq], x[t:t + 1, hq:hq + hk], x[t:t + 1, hq + hk:], cache, _dev(table),
                    _dev(np.array([t], np.int32)), _dev(_cum([1])))
        ref.append(h[t:t + 1, :hq], h[t:t + 1, hq:hq + hk], h[t:t + 1, hq + hk:], codes, scales, table, [t], _cum([1]), None, False)
    torch.cuda.synchronize()
    for got, want in ((cache.k_scale, scales[0]), (cache.v_scale, scales[1]), (cache.k, codes[0]), (cache.v, codes[1])):
        assert np.array_equal(got.cpu().numpy(), want)


def test_append_zeros_infinities_and_nan():
    def fill(x, hq, hk):
        x[0:16, hq] = 0            # a whole block of zeros
        x[3, hq + 1, 5] = float("nan")
        x[5, hq + 2, 7] = float("inf")
        x[6, hq + 2, 8] = -float("inf")
        x[17, hq:] = 1e-38         # the smallest scales
        x[33, hq:] = 3e38          # the largest

    hq, hk, d, page = 2, 2, 64, 32
    new, ctx = [16, 1, 16, 1], [0, 16, 48, 0]
    plan, cache, x, table, codes, scales, _ = _append_case(hq, hk, d, page, 0, False, new, ctx, 11, fill)
    plan.append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], cache, _dev(table), _dev(np.array(ctx, np.int32)), _dev(_cum(new)))
    torch.cuda.synchronize()
    h = x.float().cpu().numpy()
    ref.append(h[:, :hq], h[:, hq:hq + hk], h[:, hq + hk:], codes, scales, table, ctx, _cum(new), None, False)
    for got, want in ((cache.k_scale, scales[0]), (cache.v_scale, scales[1])):
        assert np.array_equal(got.cpu().numpy(), want)
    for got, want in ((cache.k, codes[0]), (cache.v, codes[1])):
        got = got.cpu().numpy()
        nan = (want & 127) == 127
        assert np.array_equal(got[~nan], want[~nan]) and bool(((got[nan] & 127) == 127).all())
    assert bool((cache.k_scale == 0).any())


def test_append_without_a_page_writes_nothing_there():
    hq, hk, d, page = 2, 1, 64, 16
    new, ctx = [40, 20], [0, 0]
    plan, cache, x, table, codes, scales, _ = _append_case(hq, hk, d, page, 64, False, new, ctx, 12)
    table[0, 1] = -1
    table[1, 0] = 1 << 30          # outside the cache
    table = table[:, :2]           # the first sequence's third page is past the table
    pkg = _pkg()
    cs = plan.rotary.cpu().numpy()
    plan.append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], cache, _dev(table), _dev(np.array(ctx, np.int32)), _dev(_cum(new)))
    torch.cuda.synchronize()
    h = x.float().cpu().numpy()
    ref.append(h[:, :hq], h[:, hq:hq + hk], h[:, hq + hk:], codes, scales, table, ctx, _cum(new), cs, False)
    for got, want in ((cache.k_scale, scales[0]), (cache.v_scale, scales[1]), (cache.k, codes[0]), (cache.v, codes[1])):
        assert np.array_equal(got.cpu().numpy(), want)
    assert pkg is not None


def test_append_in_place_and_past_the_rotary_table():
    hq, hk, d, page = 4, 4, 128, 64
    new, ctx = [30], [100]
    pkg = _pkg()
    cs = pkg.rotary_table(110, d)   # positions 110 .. 129 use its last row
    plan = pkg.PagedAttention(hq, hk, d, page, rotary=cs)
    q = torch.randn(30, hq, d, generator=_gen(1)).bfloat16().cuda()
    k = torch.randn(30, hk, d, generator=_gen(2)).bfloat16().cuda()
    v = torch.randn(30, hk, d, generator=_gen(3)).bfloat16().cuda()
    table, pages = _table([130], page, 1)
    codes, scales = _stale(pages, hk, page, d, 5)
    cache = pkg.KVCache(*[_dev(c) for c in codes], *[_dev(s) for s in scales])
    h = [t.float().cpu().numpy() for t in (q, k, v)]
    rq, rk = ref.append(*h, codes, scales, table, ctx, _cum(new), cs.cpu().numpy(), False)
    plan.append(q, k, v, cache, _dev(table), _dev(np.array(ctx, np.int32)), _dev(_cum(new)), k_out=k, q_out=q)
    torch.cuda.synchronize()
    assert torch.equal(q.cpu(), torch.from_numpy(rq).bfloat16()) and torch.equal(k.cpu(), torch.from_numpy(rk).bfloat16())
    for got, want in ((cache.k_scale, scales[0]), (cache.v_scale, scales[1])):
        assert np.array_equal(got.cpu().numpy(), want)


def test_append_many_sequences():
    # more sequences than threads of a block, some empty
    rng = np.random.default_rng(4)
    new = [int(n) for n in rng.integers(0, 4, 700)]
    ctx = [int(n) for n in rng.integers(0, 40, 700)]
    hq, hk, d, page = 2, 1, 64, 16
    plan, cache, x, table, codes, scales, cs = _append_case(hq, hk, d, page, 64, True, new, ctx, 13)
    q, _ = plan.append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], cache, _dev(table), _dev(np.array(ctx, np.int32)), _dev(_cum(new)))
    torch.cuda.synchronize()
    h = x.float().cpu().numpy()
    rq, _ = ref.append(h[:, :hq], h[:, hq:hq + hk], h[:, hq + hk:], codes, scales, table, ctx, _cum(new), cs.cpu().numpy(), True)
    assert torch.equal(q.cpu(), torch.from_numpy(rq).bfloat16())
    for got, want in ((cache.k_scale, scales[0]), (cache.v_scale, scales[1])):
        assert np.array_equal(got.cpu().numpy(), want)


# ------------------------------------------------------------------ decode


def _live_cache(lens, hk, page, d, seed, scale=(114, 124)):
    table, pages = _table(lens, page, seed)
    rng = np.random.default_rng(seed)
    codes = [ref.e4m3_round(rng.normal(size=(pages, hk, page, d)) * 100) for _ in range(2)]
    scales = [rng.integers(scale[0], scale[1], (pages, hk, page // 16)).astype(np.uint8) for _ in range(2)]
    for b, n in enumerate(lens):       # what lies past a sequence's end is stale, NaN codes among it
        if n % page:
            for c in codes:
                c[table[b, n // page], :, n % page:] = 0x7F
    used = set(table[table >= 0].tolist())
    for pg in set(range(pages)) - used:
        for c in codes:
            c[pg] = 0xFF
    return table, codes, scales


def _decode(lens, hq, hk, d, page, qn, seed, edit=None, scale=None, q_scale=2.0, **kw):
    pkg = _pkg()
    table, codes, scales = _live_cache(lens, hk, page, d, seed, **kw)
    if edit:
        edit(table, codes, scales)
    plan = pkg.PagedAttention(hq, hk, d, page)
    cache = pkg.KVCache(*[_dev(c) for c in codes], *[_dev(s) for s in scales])
    q = (torch.randn(len(lens) * qn, hq + 1, d, generator=_gen(seed)) * q_scale).bfloat16().cuda()[:, :hq]
    args = (q, cache, _dev(table), _dev(np.array(lens, np.int32)))
    out, lse = plan.decode(*args, q_tokens=qn, scale=scale)
    torch.cuda.synchronize()
    return plan, args, (table, codes, scales), out, lse


def _check_decode(lens, hq, hk, d, page, qn, host, q, out, lse, scale=None):
    table, codes, scales = host
    sc = d ** -0.5 if scale is None else scale
    go, gl, qh = _f64(out), _f64(lse), _f64(q)
    for b, n in enumerate(lens):
        n = min(max(n, 0), table.shape[1] * page)
        k, has = ref.cached(codes[0], scales[0], table[b], hk, page, n)
        v, _ = ref.cached(codes[1], scales[1], table[b], hk, page, n)
        see = np.array([max(n - (qn - 1 - i), 0) for i in range(qn)])
        vis = (np.arange(n)[None, :] < see[:, None]) & has[None, :]
        r = slice(b * qn, (b + 1) * qn)
        o, ls, mag, big = ref.attend(qh[r], k, v, vis, sc)
        err, tol = np.abs(go[r] - o), ref.out_tolerance(o, mag, 11)
        assert (err <= tol).all(), (b, n, float((err / tol).max()))
        assert np.array_equal(np.isinf(gl[r]), np.isinf(ls)), (b, n)
        fin = np.isfinite(ls)
        assert (np.abs(gl[r][fin] - ls[fin]) <= ref.lse_tolerance(ls, big)[fin]).all(), (b, n)


DECODE = [
    # lens, hq, hk, d, page, qn
    ([1, 15, 16, 17, 31, 32, 33], 4, 2, 128, 16, 1),
    ([0, 64, 65, 0, 100, 127, 128, 129], 8, 1, 64, 64, 1),
    ([1000, 3, 517], 5, 5, 128, 128, 1),
    ([40, 200], 16, 1, 96, 32, 1),
    ([70], 40, 1, 128, 64, 1),              # more rows than a 16-row tile
    ([5, 2, 0, 300, 33], 8, 2, 64, 16, 4),  # drafts, some longer than their sequence
    ([90, 16], 6, 2, 128, 32, 17),
    ([77, 4], 7, 1, 80, 16, 3),
    ([50, 1], 3, 3, 16, 16, 1),
    ([2500], 2, 1, 48, 32, 2),
    ([257] * 40, 4, 4, 64, 32, 1),
    ([31, 700, 2, 90, 1500, 16, 5, 64], 12, 4, 112, 64, 1),
]


@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode(case):
    lens, hq, hk, d, page, qn = DECODE[case]
    plan, args, host, out, lse = _decode(lens, hq, hk, d, page, qn, 200 + case)
    _check_decode(lens, hq, hk, d, page, qn, host, args[0], out, lse)
    out2, lse2 = plan.decode(*args, q_tokens=qn)  # the same bits again
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    from fp8_scaled_gemm_sm_gb300 import binding

    assert binding.scaled_attn_debug_status(plan.handle)[0] == 0


@pytest.mark.parametrize("B,hq,hk,d,qn,long", [
    (70, 32, 32, 128, 1, 3000),     # 2240 segments on 152 x 12 ranges
    (90, 32, 32, 64, 1, 3000),      # 2880 on 152 x 16
    (60, 64, 32, 128, 5, 2000),     # 1920 of two row tiles each on 152 x 8
    (700, 2, 1, 128, 1, 900),       # more sequences than a block has threads
    (1500, 1, 1, 32, 2, 500),
    (2600, 2, 2, 64, 1, 70),
])
def test_decode_many_short_sequences_and_a_few_long(B, hq, hk, d, qn, long):
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(0, 40, B)]
    for b in (0, B // 2, B - 1):
        lens[b] = long + b % 17
    lens[1], lens[2] = 0, 1
    _, args, host, out, lse = _decode(lens, hq, hk, d, 16, qn, 800 + B)
    _check_decode(lens, hq, hk, d, 16, qn, host, args[0], out, lse)


def test_decode_one_long_sequence():
    lens = [20011]
    _, args, host, out, lse = _decode(lens, 4, 1, 128, 64, 1, 31)
    _check_decode(lens, 4, 1, 128, 64, 1, host, args[0], out, lse)


def test_decode_missing_pages_are_not_seen():
    lens = [100, 130, 48]

    def edit(table, codes, scales):
        table[0, 1] = -1
        table[1, 0] = codes[0].shape[0]     # one past the cache
        table[1, 3] = -7
        table[2, :] = -1                    # nothing left: zero and -infinity

    _, args, host, out, lse = _decode(lens, 4, 2, 64, 16, 1, 32, edit)
    _check_decode(lens, 4, 2, 64, 16, 1, host, args[0], out, lse)
    assert bool((out[2] == 0).all()) and bool(torch.isinf(lse[2]).all())


def test_decode_lengths_outside_the_table():
    lens = [64, 40]
    plan, args, host, _, _ = _decode(lens, 4, 2, 64, 32, 1, 33)
    out, lse = plan.decode(args[0], args[1], args[2], _dev(np.array([5000, -3], np.int32)))
    torch.cuda.synchronize()
    _check_decode([5000, -3], 4, 2, 64, 32, 1, host, args[0], out, lse)


@pytest.mark.parametrize("kind", ["value scales far apart", "zero blocks", "large scores", "equal scores"])
def test_decode_extreme_scales(kind):
    lens = [150, 33, 16]

    def edit(table, codes, scales):
        if kind == "value scales far apart":
            scales[1][:] = np.random.default_rng(1).integers(60, 190, scales[1].shape)
        elif kind == "zero blocks":
            for n in (0, 1):
                codes[n][table[0, 1]] = 0
                scales[n][table[0, 1]] = 0
            codes[1][table[1, 0]] = 0
            scales[1][table[1, 0]] = 0
        elif kind == "large scores":
            scales[0][:] = 126
        else:
            codes[0][:] = 0

    _, args, host, out, lse = _decode(lens, 4, 2, 64, 16, 1, 34, edit, q_scale=0.5 if kind == "large scores" else 2.0)
    _check_decode(lens, 4, 2, 64, 16, 1, host, args[0], out, lse)


def test_decode_rows_of_very_different_size():
    # tiny, ordinary and huge queries, a row of zeros, in one group
    lens = [90]
    pkg = _pkg()
    table, codes, scales = _live_cache(lens, 1, 32, 128, 35)
    plan = pkg.PagedAttention(6, 1, 128, 32)
    cache = pkg.KVCache(*[_dev(c) for c in codes], *[_dev(s) for s in scales])
    size = torch.tensor([1e-30, 1e-6, 1.0, 30.0, 0.0, 1e-2])[None, :, None]
    q = (torch.randn(1, 6, 128, generator=_gen(9)) * size).bfloat16().cuda()
    out, lse = plan.decode(q, cache, _dev(table), _dev(np.array(lens, np.int32)))
    torch.cuda.synchronize()
    _check_decode(lens, 6, 1, 128, 32, 1, (table, codes, scales), q, out, lse)


def test_decode_rows_that_are_not_finite_stay_alone():
    lens = [70, 40]
    plan, args, host, _, _ = _decode(lens, 6, 2, 64, 16, 1, 36)
    q = args[0].clone()
    q[0, 1, 3] = float("nan")
    q[1, 5, 0] = float("inf")
    out, lse = plan.decode(q, *args[1:])
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[0, 1].float()).all()) and bool(torch.isnan(out[1, 5].float()).all())
    q[0, 1], q[1, 5] = args[0][0, 1], args[0][1, 5]
    out[0, 1], lse[0, 1], out[1, 5], lse[1, 5] = (t for o in [plan.decode(q, *args[1:])] for t in (o[0][0, 1], o[1][0, 1], o[0][1, 5], o[1][1, 5]))
    _check_decode(lens, 6, 2, 64, 16, 1, host, q, out, lse)


def test_decode_cache_offsets_past_32_bits():
    # pages far apart: the last ones start beyond 4 GiB of codes
    pkg = _pkg()
    hk, page, d = 1, 128, 128
    pages, lens = 70, [300, 257]
    step = 80 << 20
    big = [torch.empty(pages * step, dtype=torch.uint8, device="cuda") for _ in range(2)]
    views = [b.as_strided((pages, hk, page, d), (step, page * d, d, 1)) for b in big]
    table = np.array([[69, 1, 68], [67, 66, 2]], np.int32)
    rng = np.random.default_rng(3)
    codes = [ref.e4m3_round(rng.normal(size=(pages, hk, page, d)) * 100) for _ in range(2)]
    scales = [rng.integers(114, 122, (pages, hk, page // 16)).astype(np.uint8) for _ in range(2)]
    for v, c in zip(views, codes):
        v.copy_(_dev(c))
    cache = pkg.KVCache(views[0], views[1], _dev(scales[0]), _dev(scales[1]))
    plan = pkg.PagedAttention(2, hk, d, page)
    q = torch.randn(2, 2, d, generator=_gen(1)).bfloat16().cuda()
    out, lse = plan.decode(q, cache, _dev(table), _dev(np.array(lens, np.int32)))
    torch.cuda.synchronize()
    _check_decode(lens, 2, hk, d, page, 1, (table, codes, scales), q, out, lse)
    # and the append there
    x = torch.randn(2, 4, d, generator=_gen(2)).bfloat16().cuda()
    plan.append(x[:, :2], x[:, 2:3], x[:, 3:], cache, _dev(table), _dev(np.array([299, 256], np.int32)), _dev(_cum([1, 1])))
    h = x.float().cpu().numpy()
    ref.append(h[:, :2], h[:, 2:3], h[:, 3:], codes, scales, table, [299, 256], _cum([1, 1]), None, False)
    torch.cuda.synchronize()
    for v, c in zip(views, codes):
        assert np.array_equal(v[[66, 67, 68, 69, 1, 2]].cpu().numpy(), c[[66, 67, 68, 69, 1, 2]])


# ------------------------------------------------------------------ prompt

PROMPT = [
    # queries, keys (None: the same), hq, hk, d, causal
    ([1], None, 4, 2, 128, True),
    ([77, 1, 0, 128, 129], None, 4, 1, 128, True),
    ([300], None, 8, 2, 64, True),
    ([127, 255, 2], None, 3, 3, 64, True),
    ([200, 5], None, 6, 2, 96, False),
    ([40, 130], [200, 131], 5, 1, 128, True),
    ([70, 3], [300, 0], 7, 1, 80, True),          # a sequence without keys
    ([150, 20], [30, 20], 4, 4, 128, True),       # the first 120 queries see nothing
    ([90, 33], [257, 400], 16, 1, 48, False),
    ([520], None, 16, 1, 128, True),
    ([33, 64, 1, 17, 250, 16], None, 32, 8, 128, True),
    ([10, 20], None, 2, 1, 16, True),
    ([0, 0, 9], [5, 0, 9], 2, 2, 64, True),
    ([260], [700], 12, 4, 128, True),
    ([600, 1], [600, 900], 1, 1, 128, True),
    # more keys a sequence on average: two row tiles a CTA where heads are over 64 wide
    ([40, 1, 0, 130, 3, 257], [1200, 1, 0, 130, 900, 700], 4, 1, 128, True),
    ([40, 1, 0, 130, 3, 257], [1200, 1, 0, 130, 900, 700], 3, 3, 128, False),
    ([33, 300, 5], [1000, 120, 403], 10, 2, 96, True),       # the first 180 queries of the second see nothing
    ([1, 257], [2049, 513], 16, 1, 80, True),
    ([70, 64], [1408, 16], 32, 4, 112, True),
    ([200], [0], 2, 1, 128, True),
    ([9, 500], [1500, 0], 2, 1, 128, False),
    ([40, 1, 0, 130, 3, 257], [2000, 1, 0, 130, 1500, 700], 4, 1, 128, True),
    ([40, 1, 0, 130, 3, 257], [2000, 1, 0, 130, 1500, 700], 3, 3, 128, False),
    ([33, 300, 5], [1300, 120, 603], 10, 2, 96, True),
    ([300, 2], [1009, 1030], 6, 2, 128, True),
]


def _check_prompt(ql, kl, hq, hk, d, causal, q, k, v, out, lse, scale=None):
    sc = d ** -0.5 if scale is None else scale
    go, gl, qh, kh, vh = _f64(out), _f64(lse), _f64(q), _f64(k), _f64(v)
    cq, ck = _cum(ql), _cum(kl)
    for b in range(len(ql)):
        n, m = ql[b], kl[b]
        see = np.clip(np.arange(n) + 1 + m - n, 0, m) if causal else np.full(n, m)
        r = slice(cq[b], cq[b + 1])
        o, ls, mag, big = ref.attend(qh[r], kh[ck[b]:ck[b + 1]], vh[ck[b]:ck[b + 1]], see, sc)
        err, tol = np.abs(go[r] - o), ref.out_tolerance(o, mag, 8)
        assert (err <= tol).all(), (b, n, m, float((err / tol).max()), np.argwhere(~(err <= tol))[:4])
        assert np.array_equal(np.isinf(gl[r]), np.isinf(ls)), (b, n, m)
        fin = np.isfinite(ls)
        assert (np.abs(gl[r][fin] - ls[fin]) <= ref.lse_tolerance(ls, big)[fin]).all(), (b, n, m)


def _prompt_inputs(ql, kl, hq, hk, d, seed):
    T, Tk = sum(ql), sum(kl)
    x = torch.randn(max(T, Tk), hq + 2 * hk + 1, d, generator=_gen(seed)).bfloat16().cuda()
    return x[:T, 1:hq + 1], x[:Tk, hq + 1:hq + 1 + hk], x[:Tk, hq + 1 + hk:]


@pytest.mark.parametrize("case", range(len(PROMPT)))
def test_prompt(case):
    ql, kl, hq, hk, d, causal = PROMPT[case]
    kl = ql if kl is None else kl
    q, k, v = _prompt_inputs(ql, kl, hq, hk, d, 300 + case)
    plan = _pkg().PagedAttention(hq, hk, d)
    out = torch.full((sum(ql), hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    cu = _dev(_cum(ql)), _dev(_cum(kl))
    _, lse = plan.prompt(q, k, v, *cu, causal=causal, out=out)
    torch.cuda.synchronize()
    _check_prompt(ql, kl, hq, hk, d, causal, q, k, v, out, lse)
    out2, lse2 = plan.prompt(q, k, v, *cu, causal=causal)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    from fp8_scaled_gemm_sm_gb300 import binding

    assert binding.scaled_attn_debug_status(plan.handle)[0] == 0


@pytest.mark.parametrize("B", [40, 128, 150])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_many_sequences(B, causal, d):
    # units are dealt out by the keys they see, up to 128 sequences, in their order beyond
    rng = np.random.default_rng(B)
    ql = [int(n) for n in rng.integers(0, 12, B)]
    kl = [n + int(m) for n, m in zip(ql, rng.integers(0, 9, B))]
    ql[7], kl[7], ql[B - 3], kl[B - 3], kl[5] = 290, 300, 140, 600, 0
    hq, hk = 2, 1
    q, k, v = _prompt_inputs(ql, kl, hq, hk, d, 60 + B)
    plan = _pkg().PagedAttention(hq, hk, d)
    out = torch.full((sum(ql), hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    _, lse = plan.prompt(q, k, v, _dev(_cum(ql)), _dev(_cum(kl)), causal=causal, out=out)
    torch.cuda.synchronize()
    _check_prompt(ql, kl, hq, hk, d, causal, q, k, v, out, lse)


@pytest.mark.parametrize("B", [33, 130])
def test_prompt_many_sequences_behind_contexts(B):
    rng = np.random.default_rng(B)
    ql = [int(n) for n in rng.integers(0, 12, B)]
    kl = [n + 700 + int(m) for n, m in zip(ql, rng.integers(0, 300, B))]
    ql[7], kl[7], ql[B - 3], kl[B - 3], kl[5] = 290, 300, 140, 600, 0
    hq, hk, d = 2, 1, 128
    q, k, v = _prompt_inputs(ql, kl, hq, hk, d, 70 + B)
    plan = _pkg().PagedAttention(hq, hk, d)
    out = torch.full((sum(ql), hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    _, lse = plan.prompt(q, k, v, _dev(_cum(ql)), _dev(_cum(kl)), out=out)
    torch.cuda.synchronize()
    _check_prompt(ql, kl, hq, hk, d, True, q, k, v, out, lse)


@pytest.mark.parametrize("group", [3, 6, 11, 13, 24, 39, 60, 129])
@pytest.mark.parametrize("d,ctx", [(64, 0), (128, 0), (128, 700)])
def test_prompt_heads_of_a_group_share_rows(group, d, ctx):
    # heads times tokens of a tile need not fill its rows
    ql = [45, 1, 0, 23]
    kl = [n + ctx for n in ql]
    q, k, v = _prompt_inputs(ql, kl, group, 1, d, 90 + group)
    plan = _pkg().PagedAttention(group, 1, d)
    out = torch.full((sum(ql), group, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    _, lse = plan.prompt(q, k, v, _dev(_cum(ql)), _dev(_cum(kl)), out=out)
    torch.cuda.synchronize()
    _check_prompt(ql, kl, group, 1, d, True, q, k, v, out, lse)


@pytest.mark.parametrize("hq,hk", [(64, 64), (120, 40)])
def test_prompt_many_short_ones_of_many_heads(hq, hk):
    ql = [129, 0, 257, 1, 130, 300, 128, 96, 127, 200, 256, 31]
    q, k, v = _prompt_inputs(ql, ql, hq, hk, 128, 80 + hq)
    plan = _pkg().PagedAttention(hq, hk, 128)
    out = torch.full((sum(ql), hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    _, lse = plan.prompt(q, k, v, _dev(_cum(ql)), out=out)
    torch.cuda.synchronize()
    _check_prompt(ql, ql, hq, hk, 128, True, q, k, v, out, lse)


def test_prompt_sampled_rows_of_a_long_one():
    # long enough for several key tiles a row; a sample of rows against 64 bits
    hq, hk, d, n = 4, 1, 128, 3001
    q, k, v = _prompt_inputs([n], [n], hq, hk, d, 41)
    plan = _pkg().PagedAttention(hq, hk, d)
    out, lse = plan.prompt(q, k, v, _dev(_cum([n])))
    torch.cuda.synchronize()
    rows = np.array([0, 1, 127, 128, 255, 256, 1000, 1535, 2047, 2048, 2999, 3000])
    o, ls, mag, big = ref.attend(_f64(q)[rows], _f64(k), _f64(v), rows + 1, d ** -0.5)
    err = np.abs(_f64(out)[rows] - o)
    assert (err <= ref.out_tolerance(o, mag, 8)).all()
    assert (np.abs(_f64(lse)[rows] - ls) <= ref.lse_tolerance(ls, big)).all()


def test_prompt_sequences_do_not_reach_each_other():
    # the middle sequence is all NaN and infinity: only its own rows may show it
    hq, hk, d = 4, 2, 128
    for ql, more in (([50, 60, 200], 0), ([129, 1, 127], 0), ([16, 300, 17], 0), ([50, 60, 200], 503), ([129, 1, 3], 450)):
        kl = [n + more for n in ql]
        q, k, v = _prompt_inputs(ql, kl, hq, hk, d, 42)
        cq, ck = _cum(ql), _cum(kl)
        for t, c in ((q, cq), (k, ck), (v, ck)):
            t[c[1]:c[2]] = float("nan")
            t[c[1]:c[2], :, ::3] = float("inf")
        plan = _pkg().PagedAttention(hq, hk, d)
        out, lse = plan.prompt(q, k, v, _dev(cq), _dev(ck))
        torch.cuda.synchronize()
        for b in (0, 2):
            r, rk = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
            _check_prompt([ql[b]], [kl[b]], hq, hk, d, True, q[r], k[rk], v[rk], out[r], lse[r])


@pytest.mark.parametrize("d,ctx", [(64, 0), (128, 0), (128, 400)])
def test_prompt_masked_keys_may_be_nan_and_scores_may_be_large(d, ctx):
    hq, hk, n = 2, 1, 140
    q, k, v = _prompt_inputs([n], [ctx + n], hq, hk, d, 43)
    k[ctx + 100:] = float("nan")     # rows below 100 see none of them
    q[:, 1] *= 100                   # scores of several hundred
    plan = _pkg().PagedAttention(hq, hk, d)
    out, lse = plan.prompt(q, k, v, _dev(_cum([n])), _dev(_cum([ctx + n])))
    torch.cuda.synchronize()
    o, ls, mag, big = ref.attend(_f64(q)[:100], _f64(k), _f64(v), ctx + np.arange(1, 101), d ** -0.5)
    # scores of up to 2^big are known to 2^-22 of themselves: weights move by that much
    tol = ref.out_tolerance(o, mag, 8) + (2.0 ** -20 * big)[..., None] * mag
    assert (np.abs(_f64(out)[:100] - o) <= tol).all()
    assert (np.abs(_f64(lse)[:100] - ls) <= ref.lse_tolerance(ls, big)).all()
    assert bool(torch.isnan(out[100:].float()).all())


def test_prompt_row_offsets_past_32_bits():
    hq, hk, d, n = 2, 1, 64, 150
    step = 1 << 24                   # elements between rows: 150 rows span 5 GiB
    big = torch.empty(n * step, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((n, hq + 2 * hk, d), (step, d, 1))
    x.copy_(torch.randn(n, hq + 2 * hk, d, generator=_gen(5)).bfloat16())
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    plan = _pkg().PagedAttention(hq, hk, d)
    out, lse = plan.prompt(q, k, v, _dev(_cum([n])))
    torch.cuda.synchronize()
    _check_prompt([n], [n], hq, hk, d, True, q, k, v, out, lse)


# ------------------------------------------------------------------ streams, graphs


def test_operators_follow_their_stream_and_capture():
    # append, decode and prompt chained on a side stream, then in a CUDA graph with new inputs
    hq, hk, d, page = 8, 2, 128, 32
    pkg = _pkg()
    new, ctx = [40, 3, 100], [0, 30, 5]
    lens = [a + b for a, b in zip(new, ctx)]
    cs = pkg.rotary_table(max(lens) + 1, d)
    plan = pkg.PagedAttention(hq, hk, d, page, rotary=cs)
    table, codes, scales = _live_cache(lens, hk, page, d, 51)
    for c in codes:
        c[(c & 127) == 127] = 0
    cache = pkg.KVCache(*[_dev(c) for c in codes], *[_dev(s) for s in scales])
    T = sum(new)
    x = torch.randn(T, hq + 2 * hk, d, generator=_gen(6)).bfloat16().cuda()
    tab, dctx, dcu, dlen = _dev(table), _dev(np.array(ctx, np.int32)), _dev(_cum(new)), _dev(np.array(lens, np.int32))
    last = _dev(_cum(new)[1:] - 1).long()

    def step():
        q, k = plan.append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], cache, tab, dctx, dcu, k_out=True)
        o, l = plan.prompt(q, k, x[:, hq + hk:], dcu)
        od, ld = plan.decode(q[last], cache, tab, dlen)
        return q, k, o, l, od, ld

    def check(r):
        torch.cuda.synchronize()
        q, k, o, l, od, ld = r
        _check_prompt(new, new, hq, hk, d, True, q, k, x[:, hq + hk:], o, l)
        host = (table, [c.cpu().numpy() for c in (cache.k, cache.v)], [s.cpu().numpy() for s in (cache.k_scale, cache.v_scale)])
        _check_decode(lens, hq, hk, d, page, 1, host, q[last], od, ld)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r = step()
    check(r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step()
    x.copy_(torch.randn(T, hq + 2 * hk, d, generator=_gen(7)).bfloat16())
    graph.replay()
    check(r)


# ------------------------------------------------------------------ refusals


def test_refusals():
    pkg = _pkg()
    plan = pkg.PagedAttention(4, 2, 64, 32)
    cache = plan.new_cache(4)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    n3, n4 = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (3, 4))
    bad = [
        lambda: plan.decode(q.float(), cache, table, n3),
        lambda: plan.decode(q[:, :3], cache, table, n3),
        lambda: plan.decode(q, cache, table, n4),
        lambda: plan.decode(q, cache, table.long(), n3),
        lambda: plan.decode(q, cache, table, n3.long()),
        lambda: plan.decode(q.transpose(1, 2).contiguous().transpose(1, 2), cache, table, n3),
        lambda: plan.decode(q, cache, table, n3, out=q.float()),
        lambda: plan.decode(q, pkg.KVCache.new(4, 2, 16, 64), table, n3),
        lambda: plan.decode(q.cpu(), cache, table, n3),
        lambda: plan.append(q, kv[:2], kv, cache, table, n3, n4),
        lambda: plan.append(q, kv, kv, cache, table, n3, n3),
        lambda: plan.prompt(q, kv, kv[:2], n4),
        lambda: plan.prompt(q, kv, kv, n4, n3),
        lambda: pkg.KVCache(cache.k, cache.v, cache.k_scale, cache.v_scale[:, :1]),
        lambda: pkg.KVCache(cache.k.transpose(2, 3), cache.v, cache.k_scale, cache.v_scale),
        lambda: pkg.rotary_table(10, 12),
        lambda: pkg.rotary_table(10, 16, scaling=("spiral", 2)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was not refused" % i)
    from fp8_scaled_gemm_sm_gb300 import ScaledGemmError

    odd = torch.zeros(3 * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(3, 4, 64)
    for status, f in [
        (3, lambda: plan.decode(odd, cache, table, n3)),                       # not 16-byte aligned
        (1, lambda: plan.decode(q, cache, table, n3, out=q)),                  # overlap
        (1, lambda: plan.prompt(q, kv, kv, n4, out=q)),
        (1, lambda: plan.append(q, kv, kv, cache, table, n3, n4, k_out=kv)),   # k_out is v too
        (1, lambda: plan.decode(q, cache, table, n3, scale=0.0)),
        (1, lambda: plan.prompt(q, kv, kv, n4, scale=-1.0)),
        (1, lambda: plan.prompt(q, kv, kv, n4, scale=float("inf"))),
        (2, lambda: pkg.PagedAttention(4, 2, 64, 48)),
        (2, lambda: pkg.PagedAttention(4, 3, 64, 32)),
        (2, lambda: pkg.PagedAttention(4, 2, 144, 32)),
        (2, lambda: pkg.PagedAttention(4, 2, 64, 32, rotary=pkg.rotary_table(8, 128)).append(q, kv, kv.clone(), cache, table, n3, n4)),
    ]:
        with pytest.raises(ScaledGemmError) as e:
            f()
        assert e.value.status == status


def test_empty_calls():
    pkg = _pkg()
    plan = pkg.PagedAttention(4, 2, 64, 32)
    cache = plan.new_cache(4)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, kv = (torch.zeros(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    plan.decode(q, cache, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), none)
    plan.append(q, kv, kv, cache, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), none, one)
    out, lse = plan.prompt(q, kv, kv, one)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # no pages at all: every row is empty
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = plan.decode(q, cache, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), torch.full((2,), 9, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool(torch.isinf(lse).all())
    # queries without keys
    kv = kv[:0]
    out, lse = plan.prompt(q, kv, kv, torch.tensor([0, 2], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool(torch.isinf(lse).all())
