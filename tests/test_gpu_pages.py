"""The page pool against a model of it in Python: tables, lengths, reference counts and every byte of the caches."""
import ctypes
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")
    import gpu_util

    gpu_util.lib_ready()
    import fp8_scaled_gemm_sm_gb300 as pkg

    return pkg


class Model:
    """The header's rules, one request after another."""

    def __init__(self, rows, width, pages, page, caches):
        self.page, self.pages, self.width = page, pages, width
        self.table = np.full((rows, width), -1, np.int32)
        self.lens, self.refs = np.zeros(rows, np.int32), np.zeros(pages, np.int32)
        self.caches = caches  # arrays [pages, ...]

    def _row(self, r):
        return 0 <= r < len(self.lens)

    def _length(self, r):
        return min(max(int(self.lens[r]), 0), self.width * self.page)

    def release(self, rows):
        for r in rows:
            if self._row(r):
                for p in self.table[r]:
                    if 0 <= p < self.pages:
                        self.refs[p] -= 1
                self.table[r], self.lens[r] = -1, 0

    def _serve(self, needs):
        """needs: pages of each request or None where it is refused.  The pages of each, or None."""
        free, out, upto = list(np.flatnonzero(self.refs <= 0)), [], 0
        for n in needs:
            upto += n or 0
            out.append(None if n is None or (n > 0 and upto > len(free)) else free[upto - n:upto])
        return out

    def grow(self, rows, add):
        needs, seen = [], set()
        for r, a in zip(rows, add):
            ok = self._row(r) and r not in seen and a >= 0 and self._length(r) + a <= self.width * self.page
            if self._row(r):
                seen.add(r)
            needs.append(-(-(self._length(r) + a) // self.page) + (-self._length(r) // self.page) if ok else None)
        for r, a, got in zip(rows, add, served := self._serve(needs)):
            if got is not None:
                at = -(-self._length(r) // self.page)
                self.table[r, at:at + len(got)] = got
                self.refs[got] = 1
                self.lens[r] = self._length(r) + a
        return [int(g is not None) for g in served]

    def fork(self, src, dst):
        needs, last, seen = [], [], set()
        for s, d in zip(src, dst):
            ok = self._row(s) and self._row(d) and d not in seen and self.lens[d] <= 0
            if self._row(d):
                seen.add(d)
            n = self._length(s) if ok else 0
            p = self.table[s, n // self.page] if n % self.page else -1
            last.append(int(p) if 0 <= p < self.pages else -1)
            needs.append(int(last[-1] >= 0) if ok else None)
        before = self.table.copy(), self.lens.copy()
        for s, d, p, got in zip(src, dst, last, served := self._serve(needs)):
            if got is None:
                continue
            n = min(max(int(before[1][s]), 0), self.width * self.page)
            if n == 0:
                continue
            for e in range(n // self.page):
                q = self.table[d, e] = before[0][s, e]
                if 0 <= q < self.pages:
                    self.refs[q] += 1
            if got:
                self.table[d, n // self.page] = got[0]
                self.refs[got[0]] = 1
                for c in self.caches:
                    c[got[0]] = c[p]
            self.lens[d] = n
        return [int(g is not None) for g in served]

    def compact(self):
        used = int((self.refs > 0).sum())
        to = [p for p in range(used) if self.refs[p] <= 0]
        frm = [p for p in range(used, self.pages) if self.refs[p] > 0]
        new = {a: b for a, b in zip(frm, to)}
        for i, p in np.ndenumerate(self.table):
            self.table[i] = new.get(int(p), p)
        for a, b in new.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            for c in self.caches:
                c[b] = c[a]
        return used


def _setup(pkg, rows, width, pages, page=16, hk=2, d=64, layers=2, gap=0, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    plan = pkg.PagedAttention(2 * hk, hk, d, page)
    caches, arrays, whole = [], [], []
    for _ in range(layers):
        t = []
        for _ in range(2):
            # pages `gap` bytes apart: what lies between has to stay
            buf = torch.randint(0, 256, (pages, hk * page * d + gap), dtype=torch.uint8, generator=g, device="cuda")
            whole.append(buf)
            t.append(buf[:, :hk * page * d].view(pages, hk, page, d) if not gap else buf.as_strided((pages, hk, page, d), (buf.stride(0), page * d, d, 1)))
        t += [torch.randint(0, 256, (pages, hk, page // 16), dtype=torch.uint8, generator=g, device="cuda") for _ in range(2)]
        caches.append(pkg.KVCache(*t))
        arrays += t
    if caches:
        pool = pkg.PagePool.new(plan, caches, rows, width)
    else:  # bookkeeping alone
        pool = pkg.PagePool(plan, [], torch.full((rows, width), -1, dtype=torch.int32, device="cuda"),
                            *(torch.zeros(n, dtype=torch.int32, device="cuda") for n in (rows, pages)))
    model = Model(rows, width, pages, page, [a.cpu().numpy().copy() for a in arrays])
    gaps = [(w, w[:, hk * page * d:].clone()) for w in whole]
    return pool, model, arrays, gaps


def _same(pool, model, arrays, gaps=()):
    assert np.array_equal(pool.table.cpu().numpy(), model.table)
    assert np.array_equal(pool.lens.cpu().numpy(), model.lens)
    assert np.array_equal(pool.refs.cpu().numpy(), model.refs)
    for a, b in zip(arrays, model.caches):
        assert np.array_equal(a.cpu().numpy(), b)
    for w, g in gaps:
        assert torch.equal(w[:, w.shape[1] - g.shape[1]:], g)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows,width,pages,page,hk,d,layers,gap", [
    (6, 9, 31, 16, 2, 64, 2, 0), (40, 5, 77, 64, 1, 128, 1, 48), (5, 40, 300, 32, 3, 96, 3, 0), (1300, 3, 5000, 16, 1, 16, 1, 0), (3, 4, 9, 128, 8, 128, 33, 0),
    (2, 2, 3, 16, 1, 16, 0, 0)])
def test_random_calls(pkg, rows, width, pages, page, hk, d, layers, gap):
    pool, model, arrays, gaps = _setup(pkg, rows, width, pages, page, hk, d, layers, gap)
    rng = random.Random(rows)
    pick = lambda: rng.randint(-1, rows) if rng.random() < 0.1 else rng.randrange(rows)  # noqa: E731
    for step in range(30):
        n = rng.randint(1, min(rows, 1200))
        kind = rng.choice(["grow", "grow", "fork", "fork", "release", "compact"])
        if kind == "grow":
            a, b = [pick() for _ in range(n)], [rng.choice([0, 1, page, rng.randint(-1, width * page // 2)]) for _ in range(n)]
            assert pool.grow(ints(a), ints(b)).tolist() == model.grow(a, b)
        elif kind == "fork":
            a, b = [pick() for _ in range(n)], [pick() for _ in range(n)]
            assert pool.fork(ints(a), ints(b)).tolist() == model.fork(a, b)
        elif kind == "release":
            a = [pick() for _ in range(rng.randint(1, n))]
            pool.release(ints(a))
            model.release(a)
        else:
            assert pool.compact().tolist() == [model.compact()]
        _same(pool, model, arrays, gaps)


def test_pages_run_out(pkg):
    pool, model, arrays, _ = _setup(pkg, 8, 4, 10)
    for a, b in (([0, 1, 2, 3], [40, 64, 33, 0]), ([4, 0, 5], [5, 1, 1]), ([3, 0], [64, 64])):
        assert pool.grow(ints(a), ints(b)).tolist() == model.grow(a, b)
        _same(pool, model, arrays)
    assert pool.fork(ints([0, 1, 0]), ints([5, 6, 7])).tolist() == model.fork([0, 1, 0], [5, 6, 7])
    _same(pool, model, arrays)


def test_names_outside_the_pool(pkg):
    """Entries that name no page, and lengths that no row has."""
    pool, model, arrays, _ = _setup(pkg, 5, 4, 12)
    for t, m in ((pool.table, model.table), (pool.lens, model.lens)):
        m[0] = [3, 99, -7, 5] if m.ndim == 2 else 60
        m[1] = [-1, -1, -1, -1] if m.ndim == 2 else -5
        m[2] = [1, 2, 4, 6] if m.ndim == 2 else 10 ** 9
        t.copy_(torch.from_numpy(m))
    for p in (1, 2, 3, 4, 5, 6):
        model.refs[p] = 1
    pool.refs.copy_(torch.from_numpy(model.refs))
    assert pool.fork(ints([0, 1, 2]), ints([3, 4, 1])).tolist() == model.fork([0, 1, 2], [3, 4, 1])
    _same(pool, model, arrays)
    assert pool.grow(ints([1, 2]), ints([3, 1])).tolist() == model.grow([1, 2], [3, 1])
    _same(pool, model, arrays)
    pool.release(ints([0, 0, 2, 77, -3]))
    model.release([0, 2])
    _same(pool, model, arrays)


def test_compaction_leaves_entries_of_free_pages(pkg):
    pool, model, arrays, _ = _setup(pkg, 3, 3, 12)
    model.table[:] = [[9, 11, -1], [2, 10, 7], [6, 99, -5]]
    model.refs[[9, 2]] = 1  # 11, 10, 7 and 6 are free
    pool.table.copy_(torch.from_numpy(model.table))
    pool.refs.copy_(torch.from_numpy(model.refs))
    pool.scratch.fill_(0x55)
    assert pool.compact().tolist() == [model.compact()]
    _same(pool, model, arrays)


def test_captured(pkg):
    """Grow, fork, release and compact as one graph, replayed from other states."""
    pool, model, arrays, _ = _setup(pkg, 6, 6, 40)
    rows, add, src, dst, drop = ints([0, 1, 2]), ints([20, 7, 33]), ints([0, 1]), ints([3, 4]), ints([3, 4, 1])
    ok, ok2, used = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (3, 2, 1))

    def step():
        pool.grow(rows, add, ok=ok)
        pool.fork(src, dst, ok=ok2)
        pool.release(drop)
        pool.compact(in_use=used)

    def expect():
        return [model.grow([0, 1, 2], [20, 7, 33]), model.fork([0, 1], [3, 4]), model.release([3, 4, 1]), [model.compact()]]

    step()
    want = expect()
    _same(pool, model, arrays)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
        want = expect()
        assert [ok.tolist(), ok2.tolist(), used.tolist()] == [want[0], want[1], want[3]]
        _same(pool, model, arrays)


def test_another_stream(pkg):
    pool, model, arrays, _ = _setup(pkg, 6, 6, 40)
    side = torch.cuda.Stream()
    a, b = ints([0, 1, 2]), ints([20, 7, 33])
    side.wait_stream(torch.cuda.current_stream())
    ok = pool.grow(a, b, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert ok.tolist() == model.grow([0, 1, 2], [20, 7, 33])
    _same(pool, model, arrays)


def test_refusals(pkg):
    pool, model, arrays, _ = _setup(pkg, 4, 3, 9)
    a = ints([0, 1])
    for bad in (lambda: pool.release(a.long()), lambda: pool.grow(a, a[:1]), lambda: pool.grow(a.cpu(), a), lambda: pool.fork(a, a[:1]),
                lambda: pool.grow(a, a, ok=a[:1]), lambda: pool.compact(in_use=a), lambda: pkg.PagePool(pool.plan, pool.caches, pool.table, pool.lens[:2], pool.refs),
                lambda: pkg.PagePool(pool.plan, pool.caches, pool.table, pool.lens, torch.zeros(10, dtype=torch.int32, device="cuda")),
                lambda: pkg.PagePool(pool.plan, pool.caches, pool.table.long(), pool.lens, pool.refs),
                lambda: pkg.PagePool.new(pool.plan, [], 4, 4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pkg.ScaledGemmError):
        pool.grow(ints([0] * 5), ints([1] * 5))  # more requests than rows
    _same(pool, model, arrays)


def test_c_abi_refusals(pkg):
    from fp8_scaled_gemm_sm_gb300 import binding as b

    pool, model, arrays, _ = _setup(pkg, 4, 3, 9, layers=1)
    L, h = b.lib(), pool.plan.handle
    word = pool.lens.data_ptr()
    args = lambda **k: b.PagePoolArgs(**dict(dict(table=pool.table.data_ptr(), lens=word, refs=pool.refs.data_ptr(), rows=4, table_stride=3, num_pages=9,  # noqa: E731
                                                  scratch=pool.scratch.data_ptr()), **k))
    for k, status in ((dict(table=None), 1), (dict(rows=-1), 1), (dict(refs=pool.refs.data_ptr() + 4), 3), (dict(scratch=None), 1), (dict(lens=word + 1), 3),
                      (dict(num_pages=1 << 31), 2), (dict(rows=1 << 20, table_stride=1 << 20), 2)):
        assert L.scaled_attn_pool_release(h, ctypes.byref(args(**k)), word, 1, None) == status, k
        assert L.scaled_attn_pool_grow(h, ctypes.byref(args(**k)), word, word, 1, word, None) == status, k
        assert L.scaled_attn_pool_compact(h, ctypes.byref(args(**k)), None, 0, word, None) == status, k
    ok = args()
    assert L.scaled_attn_pool_release(h, ctypes.byref(ok), None, 1, None) == 1
    assert L.scaled_attn_pool_release(h, ctypes.byref(ok), word, -1, None) == 1
    assert L.scaled_attn_pool_grow(h, ctypes.byref(ok), word, word, 5, word, None) == 1
    assert L.scaled_attn_pool_fork(h, ctypes.byref(ok), None, 1, word, word, 1, word, None) == 1
    assert L.scaled_attn_pool_fork(h, ctypes.byref(ok), None, -1, word, word, 1, word, None) == 1
    c = b.KvCacheArgs(*(t.data_ptr() for t in (arrays[0], arrays[1], arrays[2], arrays[3])), 8, arrays[0].stride(0), arrays[1].stride(0))
    assert L.scaled_attn_pool_compact(h, ctypes.byref(ok), ctypes.byref(c), 1, word, None) == 1  # fewer pages than the pool
    assert L.scaled_attn_pool_compact(h, ctypes.byref(ok), None, 0, None, None) == 1
    _same(pool, model, arrays)


def test_one_sequence_after_a_fork(pkg):
    """Append through a forked row leaves the other's tokens alone, and both read the shared part."""
    plan = pkg.PagedAttention(4, 2, 64, 16)
    cache = plan.new_cache(20)
    pool = pkg.PagePool.new(plan, cache, 3, 6)
    g = torch.Generator("cuda").manual_seed(1)
    rows = lambda n: [torch.randn(n, h, 64, generator=g, device="cuda").bfloat16() for h in (4, 2, 2)]  # noqa: E731

    def append(row, x):
        n, ctx = x[0].shape[0], pool.lens[row:row + 1].clone()
        assert pool.grow(ints([row]), ints([n])).tolist() == [1]
        plan.append(*x, cache, pool.table[row:row + 1], ctx, ints([0, n]))

    first, second, third = rows(41), rows(9), rows(30)
    append(0, first)
    assert pool.fork(ints([0, 0]), ints([1, 2])).tolist() == [1, 1]
    q = rows(3)[0]
    same, _ = plan.decode(q, cache, pool.table, pool.lens)
    one = torch.cat([plan.decode(q[i:i + 1], cache, pool.table[:1], pool.lens[:1])[0] for i in range(3)])
    assert torch.equal(same, one)
    append(1, second)
    append(2, third)
    after, _ = plan.decode(q[:1], cache, pool.table[:1], pool.lens[:1])
    assert torch.equal(after, one[:1])
    # each fork is what a sequence of its own would be: the scale of the block that both wrote behind 41 tokens included
    alone = plan.new_cache(6)
    table = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    plan.append(*first, alone, table, ints([0]), ints([0, 41]))
    plan.append(*third, alone, table, ints([41]), ints([0, 30]))
    want, _ = plan.decode(q[2:], alone, table, ints([71]))
    got, _ = plan.decode(q[2:], cache, pool.table[2:], pool.lens[2:])
    assert torch.equal(got, want)
    pool.release(ints([0, 1]))
    pool.compact()
    got, _ = plan.decode(q[2:], cache, pool.table[2:], pool.lens[2:])
    assert torch.equal(got, want)


def test_requests_and_answers_that_the_call_changes_are_refused(pkg):
    """Requests are read while the pool and the answer are written."""
    pool, model, arrays, _ = _setup(pkg, 6, 6, 40)
    a, b = ints([0, 1, 2]), ints([20, 7, 33])
    assert pool.grow(a, b).tolist() == model.grow([0, 1, 2], [20, 7, 33])
    words = pool.scratch.view(torch.int32)
    for bad in (lambda: pool.grow(a, b, ok=b), lambda: pool.grow(a, b, ok=a), lambda: pool.grow(a, pool.lens[:3]), lambda: pool.grow(pool.table[0, :3], b),
                lambda: pool.grow(a, b, ok=pool.lens[3:]), lambda: pool.grow(a, b, ok=pool.refs[-3:]), lambda: pool.grow(words[-3:], b),
                lambda: pool.fork(a, a + 3, ok=a), lambda: pool.fork(pool.lens[3:], a), lambda: pool.fork(a, pool.refs[:3]),
                lambda: pool.release(pool.lens), lambda: pool.release(pool.table[1]), lambda: pool.compact(in_use=pool.table[5, 5:]),
                lambda: pool.compact(in_use=words[:1]), lambda: pool.compact(in_use=pool.refs[39:])):
        with pytest.raises(pkg.ScaledGemmError):
            bad()
    _same(pool, model, arrays)
    both = ints([0, 1, 2, 3, 4, 5])  # of one tensor, side by side
    assert pool.fork(both[:3], both[3:]).tolist() == model.fork([0, 1, 2], [3, 4, 5])
    assert pool.grow(both[:3], both[:3]).tolist() == model.grow([0, 1, 2], [0, 1, 2])
    _same(pool, model, arrays)


@pytest.mark.parametrize("rows,entries,pages", [(0, 4, 5), (3, 0, 5), (3, 4, 0), (0, 0, 0)])
def test_pools_without_rows_entries_or_pages(pkg, rows, entries, pages):
    """Torch's empty tensors have no address.  What needs none of what is missing is carried out."""
    plan = pkg.PagedAttention(4, 2, 64, 16)
    pool = pkg.PagePool.new(plan, plan.new_cache(pages), rows, entries)
    pool.release(ints([0, 2, 7]))
    assert pool.compact().tolist() == [0]
    if rows:
        assert pool.grow(ints([0, 1, 2]), ints([0, 1, 0])).tolist() == [1, int(entries > 0 and pages > 0), 1]
        assert pool.fork(ints([0, 2]), ints([2, 0])).tolist() == [1, 1]
        assert pool.lens.tolist() == [0, 0, 0]
    none = ints([])
    assert pool.grow(none, none).tolist() == [] and pool.fork(none, none).tolist() == []


def test_plans_of_another_layout_are_refused(pkg):
    """Pages of another size would be counted and moved with the plan's; one of the same layout serves."""
    pool, model, arrays, _ = _setup(pkg, 4, 3, 9)
    a, b = ints([0, 1]), ints([20, 30])
    own = pool.plan
    for other in (pkg.PagedAttention(4, 2, 64, 32), pkg.PagedAttention(4, 4, 64, 16), pkg.PagedAttention(4, 2, 128, 16)):
        pool.plan = other
        for call in (lambda: pool.grow(a, b), lambda: pool.fork(a, a + 2), lambda: pool.release(a), lambda: pool.compact()):
            with pytest.raises(ValueError):
                call()
    pool.plan = pkg.PagedAttention(8, 2, 64, 16)
    assert pool.grow(a, b).tolist() == model.grow([0, 1], [20, 30])
    pool.plan = own
    assert pool.fork(a, a + 2).tolist() == model.fork([0, 1], [2, 3])
    _same(pool, model, arrays)


def test_a_cache_given_twice(pkg):
    """As given once."""
    pool, model, arrays, _ = _setup(pkg, 6, 6, 40, layers=1)
    pool = pkg.PagePool.new(pool.plan, pool.caches * 34, 6, 6)
    assert pool.grow(ints([0, 1, 2]), ints([20, 7, 33])).tolist() == model.grow([0, 1, 2], [20, 7, 33])
    assert pool.fork(ints([0, 2, 1]), ints([3, 4, 5])).tolist() == model.fork([0, 2, 1], [3, 4, 5])
    _same(pool, model, arrays)
    pool.release(ints([0, 4]))
    model.release([0, 4])
    assert pool.compact().tolist() == [model.compact()]
    _same(pool, model, arrays)


def test_tensors_of_a_pool_cannot_be_exchanged(pkg):
    """The calls go by their addresses: another tensor in one's place would leave them memory that has been given away."""
    pool, model, arrays, _ = _setup(pkg, 4, 3, 9)
    for name in ("table", "lens", "refs", "scratch", "caches"):
        with pytest.raises(AttributeError):
            setattr(pool, name, getattr(pool, name))
    pool.caches.clear()
    assert pool.grow(ints([0, 3]), ints([20, 7])).tolist() == model.grow([0, 3], [20, 7])
    _same(pool, model, arrays)


def test_memory_that_the_calls_have_is_kept(pkg):
    """Another tensor under a cache's or a plan's name does not give the first one's memory away."""
    from fp8_scaled_gemm_sm_gb300 import rotary_table

    plan = pkg.PagedAttention(4, 2, 64, 16, rotary=rotary_table(5000, 64))
    cache = plan.new_cache(500)
    for owner, name in ((cache, "k"), (cache, "v"), (cache, "k_scale"), (cache, "v_scale"), (plan, "rotary")):
        t = getattr(owner, name)
        at, shape, dtype = t.data_ptr(), t.shape, t.dtype
        del t
        setattr(owner, name, None)
        assert all(torch.empty(shape, dtype=dtype, device="cuda").data_ptr() != at for _ in range(3))
