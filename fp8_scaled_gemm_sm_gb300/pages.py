"""Pages of a key/value cache among sequences, for torch CUDA tensors (C ABI: ``scaled_attn_pool_*``
in ``include/scaled_attention.h``)."""
import torch

from . import binding
from .attention import KVCache, _ext


class PagePool:
    """The pages of `caches` (a ``KVCache``, or one for each layer of a model: a page number means that page of
    each) and the rows that hold them.

    `table` int32 [rows, entries] lists each row's pages in order, -1 past the last; `lens` int32 [rows] counts
    the tokens that each row holds (these calls alone change it; a sequence of which fewer are to be seen takes kv_lens of its own); `refs` int32 [num_pages] counts the entries that name a page.  The calls change them in
    place on torch's current stream, or on `stream` (a CUDA stream's number); nothing synchronises, so all can be captured in
    a CUDA graph.  Calls on one pool have to be ordered, with one another and with attention over the rows that they
    change.  Requests are int32 tensors on the pool's device, carried out in their order, the lowest free pages
    first; an answer is an int32 tensor, 1 where a request was carried out and 0 where it was refused.
    None of them may share memory with what a call changes (the pool's tensors, the answer).
    """

    def __init__(self, plan, caches, table, lens, refs):
        caches = [caches] if isinstance(caches, KVCache) else list(caches)
        for t, dims, name in ((table, 2, "table"), (lens, 1, "lens"), (refs, 1, "refs")):
            if t.dtype != torch.int32 or t.dim() != dims or t.device != plan.device or not t.is_contiguous():
                raise ValueError("%s must be a contiguous %d-D int32 tensor on the plan's device" % (name, dims))
        if lens.shape[0] != table.shape[0]:
            raise ValueError("table and lens must have as many rows")
        if any(c.k.shape[0] < refs.shape[0] for c in caches):
            raise ValueError("every cache must have the pool's pages")
        self.plan, self._caches, self._table, self._lens, self._refs = plan, tuple(caches), table, lens, refs
        self._scratch = torch.empty(binding.scaled_attn_pool_scratch_bytes(table.shape[0], refs.shape[0]), dtype=torch.uint8,
                                    device=plan.device)
        ext = _ext()
        self._p = ext.pool(plan._p, table, lens, refs, self._scratch, [c._c for c in caches])
        self._release, self._grow, self._fork, self._compact = ext.pool_release, ext.pool_grow, ext.pool_fork, ext.pool_compact

    # The calls have the tensors' addresses: others cannot take their places.
    caches = property(lambda self: list(self._caches))
    table = property(lambda self: self._table)
    lens = property(lambda self: self._lens)
    refs = property(lambda self: self._refs)
    scratch = property(lambda self: self._scratch)

    @classmethod
    def new(cls, plan, caches, rows, entries):
        """An empty pool for `rows` sequences of up to `entries` pages."""
        caches = [caches] if isinstance(caches, KVCache) else list(caches)
        if not caches:
            raise ValueError("a new pool needs a cache")
        pages = min(c.k.shape[0] for c in caches)
        return cls(plan, caches, torch.full((rows, entries), -1, dtype=torch.int32, device=plan.device),
                   *(torch.zeros(n, dtype=torch.int32, device=plan.device) for n in (rows, pages)))

    def release(self, rows, stream=None):
        """The rows give their pages back and are empty."""
        return self._release(self.plan._p, self._p, rows, stream)

    def grow(self, rows, tokens, ok=None, stream=None):
        """Pages for tokens[i] more tokens of rows[i], whose length grows by them.  Returns the answer."""
        return self._grow(self.plan._p, self._p, rows, tokens, ok, stream)

    def fork(self, src, dst, ok=None, stream=None):
        """Row dst[i], which is empty, becomes a copy of row src[i] as it was before the call: full pages are shared, a last
        page that is not full is copied in every cache.  Returns the answer."""
        return self._fork(self.plan._p, self._p, src, dst, ok, stream)

    def compact(self, in_use=None, stream=None):
        """Moves the pages in use to the lowest numbers.  Returns how many they are, int32 [1]."""
        return self._compact(self.plan._p, self._p, in_use, stream)
