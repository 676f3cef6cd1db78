"""Attention over a paged 8-bit cache, for torch CUDA tensors (C ABI:
``include/scaled_attention.h``).

``PagedAttention`` is a plan for one head layout; ``KVCache`` the cache it works
on; ``rotary_table`` the positions' cosines and sines.  As in ``binding``, this
is argument marshalling: every step runs in the library's kernels, launched on
torch's current stream, and nothing synchronises.
"""
import ctypes
import math

import torch

from . import binding

BLOCK = 16  # tokens that share a scale

# torch's current stream as a number; without the Stream object, building which takes longer than a launch
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class KVCache:
    """Keys and values of ``num_pages`` pages: e4m3 codes uint8 [num_pages, Hk, page, D]
    (pages may be strided) and e8m0 scales uint8 [num_pages, Hk, page / 16]."""

    def __init__(self, k, v, k_scale, v_scale):
        codes = (torch.uint8, torch.float8_e4m3fn)
        for t in (k, v, k_scale, v_scale):
            if not t.is_cuda or t.device != k.device:
                raise ValueError("cache tensors must be CUDA tensors on one device")
        if k.dim() != 4 or v.shape != k.shape or k.dtype not in codes or v.dtype not in codes:
            raise ValueError("cache codes must be uint8 or float8_e4m3fn [num_pages, Hk, page, D], k and v alike")
        pages, hk, page, d = k.shape
        if page % BLOCK:
            raise ValueError("page must be a multiple of %d" % BLOCK)
        for t in (k, v):
            if t.stride()[1:] != (page * d, d, 1):
                raise ValueError("cache codes must be contiguous within a page")
        for t in (k_scale, v_scale):
            if t.dtype != torch.uint8 or t.shape != (pages, hk, page // BLOCK) or not t.is_contiguous():
                raise ValueError("cache scales must be contiguous uint8 [num_pages, Hk, page / %d]" % BLOCK)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.heads, self.page, self.dim, self.device = hk, page, d, k.device
        least = hk * page * d
        self.args = binding.KvCacheArgs(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages,
                                        k.stride(0) if pages > 1 else least, v.stride(0) if pages > 1 else least)

    @classmethod
    def new(cls, num_pages, heads, page, dim, device="cuda"):
        """An empty cache (scales are written by the first append to a block)."""
        codes = [torch.zeros(num_pages, heads, page, dim, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.zeros(num_pages, heads, page // BLOCK, dtype=torch.uint8, device=device) for _ in range(2)]
        return cls(*codes, *scales)


def rotary_table(max_pos, rot, base=10000.0, scaling=None, device="cuda"):
    """float32 [max_pos, 2, rot / 2]: cosines and sines of position * frequency, the
    frequency of pair i being base^(-2 i / rot).

    ``scaling`` stretches the positions for contexts longer than the model was
    trained on: ("linear", f) divides every frequency by f; ("parts", f, low, high,
    original) divides by f only the frequencies that turn fewer than `low` times within
    `original` positions, leaves those that turn more than `high` times, and
    blends linearly in the number of turns between them.  Angles are formed in 64 bits.
    """
    if rot % 16 or rot < 0 or max_pos < 1:
        raise ValueError("rot must be a multiple of 16 and max_pos positive")
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    if scaling is not None:
        kind, f = scaling[0], float(scaling[1])
        if kind == "linear":
            freq = freq / f
        elif kind == "parts":
            low, high, original = (float(x) for x in scaling[2:])
            turns = original * freq / (2 * math.pi)
            keep = ((turns - low) / (high - low)).clamp(0, 1)
            freq = freq * keep + freq / f * (1 - keep)
        else:
            raise ValueError("scaling must be ('linear', f) or ('parts', f, low, high, original)")
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], 1).float().contiguous().to(device)


class PagedAttention:
    """A plan for `q_heads` query heads over `kv_heads` key/value heads of `dim`
    dimensions and a cache of pages of `page_size` tokens.

    `rotary` is a table from ``rotary_table`` (None: positions are not rotated);
    `interleaved` rotates pairs (2i, 2i + 1) instead of (i, i + rot / 2).  q, k and v
    are bfloat16 [tokens, heads, dim], possibly views of a projection's rows.
    """

    def __init__(self, q_heads, kv_heads, dim, page_size=64, rotary=None, interleaved=False, device=None):
        self.q_heads, self.kv_heads, self.dim, self.page_size = int(q_heads), int(kv_heads), int(dim), int(page_size)
        dev = torch.cuda.current_device() if device is None else torch.device("cuda", device).index
        self.device = torch.device("cuda", dev)
        self.rotary = rotary
        if rotary is None:
            self._rot = binding.RotaryArgs(None, 0, 0, 0)
        else:
            if rotary.dtype != torch.float32 or rotary.dim() != 3 or rotary.shape[1] != 2 or not rotary.is_contiguous():
                raise ValueError("rotary must be a contiguous float32 [max_pos, 2, rot / 2] tensor")
            if rotary.device != self.device:
                raise ValueError("rotary must be on the plan's device")
            self._rot = binding.RotaryArgs(rotary.data_ptr(), rotary.shape[0], 2 * rotary.shape[2], int(interleaved))
        self.handle = binding.scaled_attn_create(q_heads, kv_heads, dim, page_size, dev)

    def new_cache(self, num_pages):
        return KVCache.new(num_pages, self.kv_heads, self.page_size, self.dim, self.device)

    # -- checks -------------------------------------------------------------------

    def _rows(self, t, heads, what):
        if t.dim() != 3 or t.dtype != torch.bfloat16 or t.device != self.device:
            raise ValueError("%s must be a bfloat16 [tokens, heads, dim] tensor on the plan's device" % what)
        n, h, d = t.shape
        s = t.stride()
        if h != heads or d != self.dim or s[2] != 1 or (h > 1 and s[1] != d):
            raise ValueError("%s must be [tokens, %d, %d] with its heads next to each other" % (what, heads, self.dim))
        return n, (s[0] if n > 1 else heads * d)

    def _cache(self, cache):
        if cache.heads != self.kv_heads or cache.page != self.page_size or cache.dim != self.dim or cache.device != self.device:
            raise ValueError("the cache's layout differs from the plan's")
        return cache.args

    def _ints(self, t, n, what):
        if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != n or t.device != self.device or not t.is_contiguous():
            raise ValueError("%s must be a contiguous int32 [%d] tensor on the plan's device" % (what, n))
        return t.data_ptr()

    def _table(self, t, batch):
        if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != batch or t.device != self.device or not t.is_contiguous():
            raise ValueError("block_table must be a contiguous int32 [%d, pages] tensor on the plan's device" % batch)
        return t.data_ptr(), t.shape[1]

    def _out(self, t, shape, dtype, what):
        if t is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        if t.shape != shape or t.dtype != dtype or t.device != self.device or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s %s tensor on the plan's device" % (what, dtype, tuple(shape)))
        return t

    def _stream(self, stream):
        return _current_stream(self.device.index) if stream is None else stream

    # -- operators ----------------------------------------------------------------

    def append(self, q, k, v, cache, block_table, ctx_lens, cu_seqlens, k_out=False, q_out=None, stream=None):
        """Rotate q and k, append k and v to the cache behind the ctx_lens [B] tokens that
        each sequence has there; sequence b's new rows are cu_seqlens[b] .. cu_seqlens[b + 1].
        Returns (rotated q, rotated k or None)."""
        T, qs = self._rows(q, self.q_heads, "q")
        tk, ks = self._rows(k, self.kv_heads, "k")
        tv, vs = self._rows(v, self.kv_heads, "v")
        if tk != T or tv != T:
            raise ValueError("q, k and v must have the same number of rows")
        B = ctx_lens.shape[0]
        table, width = self._table(block_table, B)
        q_out = self._out(q_out, (T, self.q_heads, self.dim), torch.bfloat16, "q_out")
        if k_out is True or isinstance(k_out, torch.Tensor):
            k_out = self._out(None if k_out is True else k_out, (T, self.kv_heads, self.dim), torch.bfloat16, "k_out")
        else:
            k_out = None
        binding.scaled_attn_append(
            self.handle, self._cache(cache), self._rot, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, table, width,
            self._ints(ctx_lens, B, "ctx_lens"), self._ints(cu_seqlens, B + 1, "cu_seqlens"), T, B, q_out.data_ptr(),
            None if k_out is None else k_out.data_ptr(), self._stream(stream))
        return q_out, k_out

    def decode(self, q, cache, block_table, kv_lens, q_tokens=1, scale=None, out=None, lse=None, stream=None):
        """Attention of each sequence's newest q_tokens tokens (q [B * q_tokens, Hq, dim]) over its
        first kv_lens [B] tokens in the cache, themselves included.  Returns (out, lse)."""
        n, qs = self._rows(q, self.q_heads, "q")
        B = kv_lens.shape[0]
        if n != B * q_tokens:
            raise ValueError("q must have q_tokens = %d rows for each of %d sequences" % (q_tokens, B))
        table, width = self._table(block_table, B)
        out = self._out(out, (n, self.q_heads, self.dim), torch.bfloat16, "out")
        lse = self._out(lse, (n, self.q_heads), torch.float32, "lse")
        binding.scaled_attn_decode(
            self.handle, self._cache(cache), q.data_ptr(), qs, q_tokens, table, width, self._ints(kv_lens, B, "kv_lens"), B,
            self.dim ** -0.5 if scale is None else scale, out.data_ptr(), lse.data_ptr(), self._stream(stream))
        return out, lse

    def prompt(self, q, k, v, cu_q, cu_k=None, causal=True, scale=None, out=None, lse=None, stream=None):
        """Attention within each of the packed sequences: queries cu_q[b] .. cu_q[b + 1] over keys
        cu_k[b] .. cu_k[b + 1] (cu_k None: the same).  causal: the last query sees every
        key.  Returns (out, lse)."""
        n, qs = self._rows(q, self.q_heads, "q")
        m, ks = self._rows(k, self.kv_heads, "k")
        mv, vs = self._rows(v, self.kv_heads, "v")
        if mv != m:
            raise ValueError("k and v must have the same number of rows")
        cu_k = cu_q if cu_k is None else cu_k
        B = cu_q.shape[0] - 1
        out = self._out(out, (n, self.q_heads, self.dim), torch.bfloat16, "out")
        lse = self._out(lse, (n, self.q_heads), torch.float32, "lse")
        binding.scaled_attn_prompt(
            self.handle, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, self._ints(cu_q, B + 1, "cu_q"),
            self._ints(cu_k, B + 1, "cu_k"), n, m, B, int(causal), self.dim ** -0.5 if scale is None else scale,
            out.data_ptr(), lse.data_ptr(), self._stream(stream))
        return out, lse

    def close(self):
        if getattr(self, "handle", None):
            binding.scaled_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
