"""GPU tests of the attention operators at the limits of what they are given, against the 64-bit implementations of attn_ref."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from test_gpu_attention import _check_decode, _check_prompt, _cum, _decode, _dev, _f64, _pkg, _prompt_inputs, _table, lib  # noqa: F401

pytestmark = pytest.mark.gpu


# A block that no token has been appended to may hold any scale byte; 255 is NaN.
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hk,d,qn", [(4, 2, 64, 1), (8, 1, 128, 1), (16, 1, 128, 1), (6, 2, 96, 4)])
def test_decode_scales_of_blocks_that_nothing_wrote(page, hq, hk, d, qn):
    lens = [7, 16, 33, 48, 65, 100, 129, 300]

    def edit(table, codes, scales):
        for s in scales:
            written = np.zeros(s.shape, bool)
            for b, n in enumerate(lens):
                for p in range(0, n, 16):
                    written[table[b, p // page], :, p % page // 16] = True
            s[~written] = 255

    _, args, host, out, lse = _decode(lens, hq, hk, d, page, qn, 400 + page, edit)
    _check_decode(lens, hq, hk, d, page, qn, host, args[0], out, lse)


@pytest.mark.parametrize("hq,qn", [(2, 1), (12, 3)])
def test_decode_lengths_up_to_31_bits(hq, qn):
    # a table of 2^24 - 1 entries that name three pages over and over: 2^31 - 128 tokens, the most that there can be
    page, d, pages = 128, 16, 3
    pkg = _pkg()
    plan = pkg.PagedAttention(hq, 1, d, page)
    rng = np.random.default_rng(8)
    codes = [ref.e4m3_round(rng.normal(size=(pages, 1, page, d)) * 100) for _ in range(2)]
    scales = [rng.integers(116, 121, (pages, 1, page // 16)).astype(np.uint8) for _ in range(2)]
    width = (1 << 24) - 1
    table = (torch.arange(width, dtype=torch.int32, device="cuda") % pages)[None]
    n = width * page
    for length in (n, n - 1, n - 113, 2 ** 31 - 1, n - 4000):
        q = torch.randn(qn, hq, d, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
        cache = pkg.KVCache(*[_dev(c) for c in codes], *[_dev(s) for s in scales])
        out, lse = plan.decode(q, cache, table, _dev(np.array([length], np.int32)), q_tokens=qn)
        torch.cuda.synchronize()
        for i in range(qn):
            see = min(length, n) - (qn - 1 - i)
            full, rest = divmod(see, page)
            times = np.array([(full - p + pages - 1) // pages for p in range(pages)])[:, None] + (np.arange(pages) == full % pages)[:, None] * (np.arange(page) < rest)
            k, v = (ref.E4M3[c[:, 0]] * np.repeat(ref.pow2(s[:, 0]), 16, -1)[..., None] for c, s in zip(codes, scales))
            x = k @ _f64(q)[i].T * d ** -0.5                       # [pages, page, hq]
            w = np.exp(x - x.max((0, 1))) * times[..., None]
            o = np.einsum("pth,ptd->hd", w, v) / w.sum((0, 1))[:, None]
            mag = np.einsum("pth,ptd->hd", w, np.abs(v)) / w.sum((0, 1))[:, None]
            # a warp adds up 2^31 / 1216 keys at most, in four fp32 sums a lane group of eight: 2^17 roundings of 2^-24 each
            assert (np.abs(_f64(out)[i] - o) <= ref.out_tolerance(o, mag, 11) + 2.0 ** -7 * mag).all()
            ls = x.max((0, 1)) + np.log(w.sum((0, 1)))
            assert (np.abs(_f64(lse)[i] - ls) <= 2.0 ** -7 + ref.lse_tolerance(ls, np.abs(x).max())).all()


def _sure(q, k, vis, scale):
    """[n, Hq]: rows whose largest score is ahead of the others by more than scores summed in fp32 can be off
    (2^-18 of sum |q k| each, as lse_tolerance has it) and another 32."""
    g = q.shape[1] // k.shape[1]
    kk = np.repeat(k, g, 1)
    s = np.where(vis[:, None, :], np.einsum("nhd,mhd->nhm", q, kk) * scale, -np.inf)
    big = np.einsum("nhd,mhd->nhm", np.abs(q), np.abs(kk)).max(-1) * scale
    top = -np.sort(-s, -1)[..., :2]
    return top[..., 0] - top[..., 1] > 2 * 2.0 ** -18 * big + 32 if top.shape[-1] > 1 else np.ones(s.shape[:2], bool)


def _check_large(q, k, v, vis, scale, out, lse, bits):
    """Of rows that are sure of their key, the output; of all, the logarithm of the sum."""
    o, ls, mag, big = ref.attend(q, k, v, vis, scale)
    sure = _sure(q, k, vis, scale)
    assert sure.any()
    assert np.isfinite(out).all()
    err = np.abs(out - o)
    assert (err <= ref.out_tolerance(o, mag, bits))[sure].all(), float((err / ref.out_tolerance(o, mag, bits))[sure].max())
    assert (np.abs(lse - ls) <= ref.lse_tolerance(ls, big)).all()


@pytest.mark.parametrize("scale", [1e4, 1e5, 1e7, 1e12, 1e24])
@pytest.mark.parametrize("lens,hq,hk,d,qn", [([150, 33, 16], 4, 2, 64, 1), ([260, 40], 6, 2, 128, 3), ([90], 24, 1, 96, 1), ([6011], 2, 1, 128, 1)])
def test_decode_scores_of_any_size(lens, hq, hk, d, qn, scale):
    page = 16
    _, args, host, out, lse = _decode(lens, hq, hk, d, page, qn, 500, scale=scale)
    table, codes, scales = host
    q, go, gl = _f64(args[0]), _f64(out), _f64(lse)
    for b, n in enumerate(lens):
        k, _ = ref.cached(codes[0], scales[0], table[b], hk, page, n)
        v, _ = ref.cached(codes[1], scales[1], table[b], hk, page, n)
        vis = np.arange(n)[None, :] < np.array([n - (qn - 1 - i) for i in range(qn)])[:, None]
        r = slice(b * qn, (b + 1) * qn)
        _check_large(q[r], k, v, vis, np.float64(np.float32(scale)), go[r], gl[r], 11)


# Values of a whole sequence near the ends of fp32's range: e4m3 codes at scales of 2^-127 .. 2^-110 and 2^112 .. 2^118.
@pytest.mark.parametrize("low,high", [(0, 6), (6, 17), (239, 245)])
@pytest.mark.parametrize("lens,hq,hk,d,qn", [([150, 33, 16], 4, 2, 64, 1), ([260, 40], 6, 2, 128, 3), ([90], 24, 1, 96, 1), ([6011], 2, 1, 128, 1)])
def test_decode_values_at_the_ends_of_the_range(lens, hq, hk, d, qn, low, high):
    def edit(table, codes, scales):
        scales[1][:] = np.random.default_rng(3).integers(low, high, scales[1].shape)
        codes[1][:] = ref.e4m3_round(np.random.default_rng(4).uniform(64, 400, codes[1].shape))   # one sign: sums do not cancel

    _, args, host, out, lse = _decode(lens, hq, hk, d, 16, qn, 505, edit)
    table, codes, scales = host
    q, go = _f64(args[0]), _f64(out)
    for b, n in enumerate(lens):
        k, _ = ref.cached(codes[0], scales[0], table[b], hk, 16, n)
        v, _ = ref.cached(codes[1], scales[1], table[b], hk, 16, n)
        r = slice(b * qn, (b + 1) * qn)
        o, _, mag, _ = ref.attend(q[r], k, v, np.array([n - (qn - 1 - i) for i in range(qn)]), d ** -0.5)
        assert o.min() > 2.0 ** -126
        # as out_tolerance, without its allowance of 1e-30
        assert (np.abs(go[r] - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -13) * mag).all(), float((np.abs(go[r] - o) / o).max())


@pytest.mark.parametrize("scale", [1e4, 1e6, 1e7, 1e8, 1e9, 1e12, 1e24])
@pytest.mark.parametrize("n,m,hq,hk,d", [(140, 140, 4, 1, 64), (70, 200, 2, 2, 128), (140, 840, 4, 1, 128), (130, 130, 5, 1, 128)])
def test_prompt_large_scores_are_right_or_nan(n, m, hq, hk, d, scale):
    q, k, v = _prompt_inputs([n], [m], hq, hk, d, 510)
    plan = _pkg().PagedAttention(hq, hk, d)
    out, lse = plan.prompt(q, k, v, _dev(_cum([n])), _dev(_cum([m])), scale=scale)
    torch.cuda.synchronize()
    vis = np.arange(m)[None, :] < np.arange(n)[:, None] + 1 + m - n
    q, k, v, out, lse, scale = _f64(q), _f64(k), _f64(v), _f64(out), _f64(lse), np.float64(np.float32(scale))
    o, ls, mag, big = ref.attend(q, k, v, vis, scale)
    top = np.abs(np.where(vis[:, None, :], np.einsum("nhd,mhd->nhm", q, np.repeat(k, hq // hk, 1)) * scale, -np.inf).max(-1))
    near, far = top <= 2.0 ** 29, top > 2.0 ** 30
    assert np.isnan(out[far]).all() and np.isnan(lse[far]).all()
    sure = near & _sure(q, k, vis, scale)
    assert (np.abs(out - o) <= ref.out_tolerance(o, mag, 8))[sure].all()
    assert (np.abs(lse - ls) <= ref.lse_tolerance(ls, big))[near].all()
    assert sure.any() if scale < 1e8 else far.any()


# The rows that a non-finite value behind the causal edge may reach: those whose last key is up to 142 before it.
@pytest.mark.parametrize("back", [1, 17, 90, 130, 255])
@pytest.mark.parametrize("n,m,hq,hk,d", [(300, 300, 1, 1, 64), (300, 300, 4, 1, 64), (260, 330, 1, 1, 128), (300, 300, 5, 1, 128),
                                         (300, 900, 2, 1, 128), (300, 907, 1, 1, 128), (400, 800, 3, 1, 96)])
def test_prompt_values_that_are_not_finite(n, m, hq, hk, d, back):
    q, k, v = _prompt_inputs([n], [m], hq, hk, d, 520)
    plan = _pkg().PagedAttention(hq, hk, d)
    cu = _dev(_cum([n])), _dev(_cum([m]))
    clean, clean_lse = plan.prompt(q, k, v, *cu)
    at = m - back
    for value in (float("inf"), float("nan")):
        v = v.clone()
        v[at, :, 3] = value
        out, lse = plan.prompt(q, k, v, *cu)
        torch.cuda.synchronize()
        last = np.arange(n) + m - n                       # the last key that a row sees
        bad = ~torch.isfinite(out).cpu().numpy()
        assert bad[last >= at][:, :, 3].all()             # who sees it shows it
        assert not bad[last + 142 < at].any()             # who is far before it does not
        bad[:, :, 3] = False
        assert not bad.any()                              # nor does any other dimension
        same = torch.isfinite(out)
        assert torch.equal(out[same], clean[same]) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("qn", [1, 4, 40])
@pytest.mark.parametrize("hq,hk,d,page", [(4, 2, 64, 16), (8, 1, 128, 64)])
def test_decode_values_that_are_not_finite(hq, hk, d, page, qn):
    lens = [90, 200]
    plan, (q, cache, table, dl), host, clean, clean_lse = _decode(lens, hq, hk, d, page, qn, 530)
    for back in (1, 2, qn, qn + 1):
        at = lens[0] - back
        kept = cache.v.clone()
        cache.v[int(table[0, at // page]), :, at % page, 5] = 0x7F
        out, lse = plan.decode(q, cache, table, dl, q_tokens=qn)
        torch.cuda.synchronize()
        bad = torch.isnan(out).cpu().numpy()
        last = lens[0] - 1 - (qn - 1 - np.arange(qn))
        assert bad[:qn][last >= at][:, :, 5].all()
        if back > qn - 1:                                 # every row sees it: nothing else to say
            assert bad[:qn, :, 5].all()
        assert not bad[qn:].any()                         # the other sequence
        bad[:, :, 5] = False
        assert not bad.any()
        same = ~torch.isnan(out)
        assert torch.equal(out[same], clean[same]) and torch.equal(lse, clean_lse)
        cache.v.copy_(kept)


def test_cache_without_pages():
    pkg = _pkg()
    plan = pkg.PagedAttention(4, 2, 64, 32)
    cache = plan.new_cache(0)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for width in (0, 3):
        table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
        lens = torch.tensor([9, 0], dtype=torch.int32, device="cuda")
        out, lse = plan.decode(q, cache, table, lens)
        rotated, _ = plan.append(q, kv, kv, cache, table, lens, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert bool((out == 0).all()) and bool(torch.isinf(lse).all()) and torch.equal(rotated, q)


def _calls(seed):
    """append, decode and prompt on inputs of their own: functions of (stream) that return their outputs."""
    pkg = _pkg()
    hq, hk, d, page, n = 8, 2, 128, 32, 96
    plan = pkg.PagedAttention(hq, hk, d, page, rotary=pkg.rotary_table(n, d))
    cache = plan.new_cache(3)
    x = torch.randn(n, hq + 2 * hk, d, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    table, cu = _dev(np.array([[2, 0, 1]], np.int32)), _dev(_cum([n]))
    each, lens = _dev(np.array([0], np.int32)), _dev(np.array([n], np.int32))
    plan.append(q, k, v, cache, table, each, cu)
    many, ones = table.expand(n, 3).contiguous(), lens.expand(n).contiguous()
    return [lambda s: plan.append(q, k, v, cache, table, each, cu, k_out=True, stream=s),
            lambda s: plan.decode(q, cache, many, ones, stream=s),
            lambda s: plan.prompt(q, k, v, cu, stream=s)]


@pytest.mark.parametrize("op", range(3))
def test_outputs_on_a_stream_of_the_callers(op):
    # the side stream is kept busy, so that its kernels run after the host has gone on
    call, other = _calls(1)[op], _calls(2)[op]
    want = [t.clone() for t in call(None)]
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    side.wait_stream(current)
    torch.cuda.synchronize()

    def wait_on(stream):
        with torch.cuda.stream(stream):
            torch.cuda._sleep(50_000_000)

    # an output that is dropped at once is still the kernel's
    wait_on(side)
    first, _ = call(side.cuda_stream)
    del _
    fresh = [torch.full_like(t, 7.0) for t in want for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(first, want[0]) and all(bool((t == 7.0).all()) for t in fresh)
    del fresh, first

    # memory that the current stream still reads is not the kernel's
    old = [torch.full_like(t, 3.0) for t in want]
    wait_on(current)
    read = [t.clone() for t in old]
    del old
    got = call(side.cuda_stream)
    torch.cuda.synchronize()
    assert all(bool((t == 3.0).all()) for t in read) and all(torch.equal(a, b) for a, b in zip(got, want))

    # results that the current stream reads may be dropped before it has
    current.wait_stream(side)
    wait_on(current)
    read = [t.clone() for t in got]
    del got
    other(side.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want))


TIMEOUT = 6  # SG_ERR_TIMEOUT


def _large(lens, hq, hk, d, page, qn, seed):
    """A plan and a decode's arguments, made on the GPU."""
    pkg = _pkg()
    plan = pkg.PagedAttention(hq, hk, d, page)
    table, pages = _table(lens, page, seed)
    cache = plan.new_cache(pages)
    g = torch.Generator("cuda").manual_seed(seed)
    for codes, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes.copy_(torch.randint(0, 127, codes.shape, generator=g, device="cuda") | torch.randint(0, 2, codes.shape, generator=g, device="cuda") << 7)
        scales.copy_(torch.randint(116, 120, scales.shape, generator=g, device="cuda"))
    q = torch.randn(len(lens) * qn, hq, d, generator=g, device="cuda").bfloat16()
    return plan, (q, cache, _dev(table), _dev(np.array(lens, np.int32)))


@pytest.mark.parametrize("hq,hk,d", [(4, 1, 128), (4, 1, 64), (16, 1, 128), (16, 1, 64), (32, 8, 128)])
def test_decode_that_gives_up_leaves_other_memory_alone(hq, hk, d):
    # a call over many sequences, then one over two of them, where a tile never comes: what the first left in the plan's
    # workspace (parts of cut segments of sequences that the second does not have) must not be joined into outputs that are not there
    from fp8_scaled_gemm_sm_gb300 import binding

    B, n, page = 60, 1700, 64
    plan, args = _large([n] * B, hq, hk, d, page, 1, 600)
    q, cache, table, lens = args
    keep = plan.decode(*args)
    buf = torch.full((B + 4, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    lbuf = torch.full((B + 4, hq), 5.0, device="cuda")
    two = (q[:2].contiguous(), cache, table[:2].contiguous(), lens[:2].contiguous())
    host = (table.cpu().numpy(), [t.cpu().numpy() for t in (cache.k, cache.v)], [t.cpu().numpy() for t in (cache.k_scale, cache.v_scale)])
    for tile in (0, 40):
        plan.decode(*args)
        binding.scaled_attn_set_debug(plan.handle, 50_000_000, tile)
        plan.decode(*two, out=buf[:2], lse=lbuf[:2])
        torch.cuda.synchronize()
        code, where = binding.scaled_attn_debug_status(plan.handle)
        assert code == TIMEOUT and where != 0
        assert bool((buf[2:] == 5.0).all()) and bool((lbuf[2:] == 5.0).all())
        # the context and the plan are as before
        binding.scaled_attn_set_debug(plan.handle)
        plan.decode(*two, out=buf[:2], lse=lbuf[:2])
        out, lse = plan.decode(*args)
        torch.cuda.synchronize()
        assert binding.scaled_attn_debug_status(plan.handle)[0] == 0
        assert torch.equal(out, keep[0]) and torch.equal(lse, keep[1])
        _check_decode([n] * 2, hq, hk, d, page, 1, host, q[:2], buf[:2], lbuf[:2])
        buf[:2], lbuf[:2] = 5.0, 5.0


# segments by range, several to a warp, rows in two tiles
@pytest.mark.parametrize("lens,hq,hk,d,qn", [([40, 700] * 40, 64, 32, 128, 1), ([2000] * 100, 64, 32, 64, 2), ([90, 16, 500] * 40, 36, 12, 128, 5)])
def test_decode_gives_up_in_every_form(lens, hq, hk, d, qn):
    from fp8_scaled_gemm_sm_gb300 import binding

    plan, args = _large(lens, hq, hk, d, 16, qn, 610)
    keep = plan.decode(*args, q_tokens=qn)
    binding.scaled_attn_set_debug(plan.handle, 50_000_000, 1)
    plan.decode(*args, q_tokens=qn)
    torch.cuda.synchronize()
    assert binding.scaled_attn_debug_status(plan.handle)[0] == TIMEOUT
    binding.scaled_attn_set_debug(plan.handle)
    out, lse = plan.decode(*args, q_tokens=qn)
    torch.cuda.synchronize()
    assert binding.scaled_attn_debug_status(plan.handle)[0] == 0
    assert torch.equal(out, keep[0]) and torch.equal(lse, keep[1])


# one row tile a CTA, two, units taken over, sequences without keys; a block that is the only one, the second, one far in
@pytest.mark.parametrize("tile", [0, 1, 5])
@pytest.mark.parametrize("ql,more,hq,hk,d", [
    ([77], 0, 8, 2, 128), ([500, 1, 300], 0, 4, 4, 64), ([40, 1, 0, 130], 900, 4, 1, 128), ([1500] * 12, 700, 16, 8, 128), ([30] * 400, 0, 5, 1, 64),
])
def test_prompt_gives_up(ql, more, hq, hk, d, tile):
    from fp8_scaled_gemm_sm_gb300 import binding

    kl = [n + more for n in ql]
    g = torch.Generator("cuda").manual_seed(620)
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").bfloat16() for n, h in ((sum(ql), hq), (sum(kl), hk), (sum(kl), hk)))
    cq, ck = _dev(_cum(ql)), _dev(_cum(kl))
    plan = _pkg().PagedAttention(hq, hk, d)
    keep = plan.prompt(q, k, v, cq, ck)
    T = sum(ql)
    buf = torch.full((T + 64, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    lbuf = torch.full((T + 64, hq), 5.0, device="cuda")
    binding.scaled_attn_set_debug(plan.handle, 50_000_000, tile)
    plan.prompt(q, k, v, cq, ck, out=buf[:T], lse=lbuf[:T])
    torch.cuda.synchronize()
    code, where = binding.scaled_attn_debug_status(plan.handle)
    reached = max(kl) > tile * (128 if d == 128 and sum(kl) > 512 * len(kl) else 64)
    assert (code, where != 0) == ((TIMEOUT, True) if reached else (0, False))
    assert bool((buf[T:] == 5.0).all()) and bool((lbuf[T:] == 5.0).all())
    binding.scaled_attn_set_debug(plan.handle)
    out, lse = plan.prompt(q, k, v, cq, ck)
    torch.cuda.synchronize()
    assert binding.scaled_attn_debug_status(plan.handle)[0] == 0
    assert torch.equal(out, keep[0]) and torch.equal(lse, keep[1])


def test_debug_limits_are_checked():
    from fp8_scaled_gemm_sm_gb300 import binding

    plan = _pkg().PagedAttention(4, 2, 64, 32)
    for bad in ((-1, -1), (0, -2), (0, 1 << 31)):
        with pytest.raises(binding.ScaledGemmError) as e:
            binding.scaled_attn_set_debug(plan.handle, *bad)
        assert e.value.status == 1
    assert binding.lib().scaled_attn_set_debug(None, 0, -1) == 1


@pytest.mark.parametrize("d,page,rot,inter", [(128, 64, 128, 0), (64, 16, 32, 1), (96, 32, 0, 0)])
def test_raw_calls_agree_and_outputs_may_be_left_out(d, page, rot, inter):
    # the C ABI by its binding's names, with k_out and lse NULL, against the calls on tensors
    from fp8_scaled_gemm_sm_gb300 import binding

    pkg = _pkg()
    hq, hk, n = 6, 2, 75
    cs = pkg.rotary_table(n, rot) if rot else None
    plan = pkg.PagedAttention(hq, hk, d, page, rotary=cs, interleaved=bool(inter))
    x = torch.randn(n, hq + 2 * hk, d, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    pages = -(-n // page)
    table, cu = torch.arange(pages, dtype=torch.int32, device="cuda")[None], _dev(_cum([n]))
    zero, lens = _dev(np.array([0], np.int32)), _dev(np.array([n], np.int32))
    cache, other = plan.new_cache(pages), plan.new_cache(pages)
    want_q, _ = plan.append(q, k, v, cache, table, zero, cu)
    want_d, _ = plan.decode(want_q[-1:], cache, table, lens)
    want_p, _ = plan.prompt(want_q, k, v, cu)

    least = hk * page * d
    args = binding.KvCacheArgs(other.k.data_ptr(), other.v.data_ptr(), other.k_scale.data_ptr(), other.v_scale.data_ptr(), pages, least, least)
    turn = binding.RotaryArgs(cs.data_ptr() if rot else None, n if rot else 0, rot, inter)
    wide, s = x.stride(0), torch.cuda.current_stream().cuda_stream
    got_q, got_d, got_p = (torch.empty_like(t) for t in (want_q, want_d, want_p))
    binding.scaled_attn_append(plan.handle, args, turn, q.data_ptr(), wide, k.data_ptr(), wide, v.data_ptr(), wide, table.data_ptr(), pages,
                               zero.data_ptr(), cu.data_ptr(), n, 1, got_q.data_ptr(), None, s)
    binding.scaled_attn_decode(plan.handle, args, got_q[-1:].data_ptr(), hq * d, 1, table.data_ptr(), pages, lens.data_ptr(), 1, d ** -0.5,
                               got_d.data_ptr(), None, s)
    binding.scaled_attn_prompt(plan.handle, got_q.data_ptr(), hq * d, k.data_ptr(), wide, v.data_ptr(), wide, cu.data_ptr(), cu.data_ptr(), n, n, 1, 1,
                               d ** -0.5, got_p.data_ptr(), None, s)
    torch.cuda.synchronize()
    for a, b in ((got_q, want_q), (got_d, want_d), (got_p, want_p), (other.k, cache.k), (other.v, cache.v), (other.k_scale, cache.k_scale), (other.v_scale, cache.v_scale)):
        assert torch.equal(a, b)


def test_scale_and_outputs_of_the_callers():
    lens, hq, hk, d, page = [70, 33, 0], 4, 2, 64, 16
    for scale in (0.03, 1.0):
        plan, args, host, out, lse = _decode(lens, hq, hk, d, page, 1, 540, scale=scale, q_scale=0.5)
        _check_decode(lens, hq, hk, d, page, 1, host, args[0], out, lse, scale=np.float64(np.float32(scale)))
        mine = torch.full_like(out, 9.0), torch.full_like(lse, 9.0)
        got = plan.decode(*args, scale=scale, out=mine[0], lse=mine[1])
        assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, mine))
        assert torch.equal(mine[0], out) and torch.equal(mine[1], lse)
        ql = [50, 1, 90]
        q, k, v = _prompt_inputs(ql, ql, hq, hk, d, 541)
        q = q * 0.5
        cu = _dev(_cum(ql))
        out, lse = plan.prompt(q, k, v, cu, scale=scale)
        _check_prompt(ql, ql, hq, hk, d, True, q, k, v, out, lse, scale=np.float64(np.float32(scale)))
        mine = torch.full_like(out, 9.0), torch.full_like(lse, 9.0)
        plan.prompt(q, k, v, cu, scale=scale, out=mine[0], lse=mine[1])
        assert torch.equal(mine[0], out) and torch.equal(mine[1], lse)


def test_rows_past_the_last_sequence_are_not_written():
    # a batch padded for a graph: more rows than the sequences have
    pkg = _pkg()
    hq, hk, d, page, n, rows = 4, 2, 64, 16, 20, 150
    plan = pkg.PagedAttention(hq, hk, d, page, rotary=pkg.rotary_table(n, d))
    x = torch.randn(rows, hq + 2 * hk, d, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    cu, zero = _dev(np.array([0, n], np.int32)), _dev(np.array([0], np.int32))
    table = torch.arange(2, dtype=torch.int32, device="cuda")[None]
    mine = [torch.full((rows, h, d), 5.0, dtype=torch.bfloat16, device="cuda") for h in (hq, hk, hq)]
    lse = torch.full((rows, hq), 5.0, device="cuda")
    plan.append(q, k, v, plan.new_cache(2), table, zero, cu, k_out=mine[1], q_out=mine[0])
    plan.prompt(q, k, v, cu, out=mine[2], lse=lse)
    torch.cuda.synchronize()
    assert all(bool((t[n:] == 5.0).all()) and not bool((t[:n] == 5.0).all()) for t in mine + [lse])
