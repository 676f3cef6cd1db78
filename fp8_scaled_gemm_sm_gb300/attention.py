"""Attention over a paged 8-bit cache, for torch CUDA tensors (C ABI:
``include/scaled_attention.h``).

``PagedAttention`` is a plan for one head layout; ``KVCache`` the cache it works
on; ``rotary_table`` the positions' cosines and sines.  As in ``binding``, this
is argument marshalling: every step runs in the library's kernels, launched on
torch's current stream, and nothing synchronises.  The calls themselves are in
``_attn.so`` (``csrc/sg_attn_torch.cpp``): checks, outputs and launch in one step.
"""
import math

import torch

from . import binding

BLOCK = 16  # tokens that share a scale


_EXT = None


def _ext():
    """The calls on tensors (built by ``fp8_scaled_gemm_sm_gb300.build``)."""
    global _EXT
    if _EXT is None:
        binding.lib()
        try:
            from . import _attn
        except ImportError as e:
            raise RuntimeError("_attn.so is not built; run `python -c 'import __graft_entry__ as g; g.build()'` (%s)" % e)
        _attn.set_error(binding.ScaledGemmError)
        _EXT = _attn
    return _EXT


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
        self._held = (k, v, k_scale, v_scale)  # the calls have their addresses, whatever becomes of the names
        self.heads, self.page, self.dim, self.device = hk, page, d, k.device
        least = hk * page * d
        self._c = _ext().cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages,
                               k.stride(0) if pages > 1 else least, v.stride(0) if pages > 1 else least, hk, page, d, k.device.index)

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

    Calls run on torch's current stream, or on `stream` (a CUDA stream's number, such as
    ``torch.cuda.Stream.cuda_stream``).  Outputs that a call allocates may be dropped at
    once either way.  What the caller passes (inputs, the cache, outputs of its own) has to
    be ready on `stream` and to live until that has used it: ``wait_stream`` and
    ``record_stream`` are the caller's.

    A plan owns a workspace that ``decode`` and ``chunk`` use, so those calls on one plan have to be ordered
    (one stream, ordered streams, or a plan a stream); ``append`` and ``prompt`` may
    overlap with anything that leaves their buffers alone.  Nothing here has a backward
    pass: results carry no gradient, whatever the inputs do.  Output rows past
    cu_seqlens[B] (a batch padded for a graph) are not written.
    """

    def __init__(self, q_heads, kv_heads, dim, page_size=64, rotary=None, interleaved=False, device=None):
        self.q_heads, self.kv_heads, self.dim, self.page_size = int(q_heads), int(kv_heads), int(dim), int(page_size)
        dev = torch.cuda.current_device() if device is None else torch.device("cuda", device).index
        self.device = torch.device("cuda", dev)
        self.rotary = self._held = rotary  # the calls have its address, whatever becomes of the name
        rot = (0, 0, 0, 0)
        if rotary is not None:
            if rotary.dtype != torch.float32 or rotary.dim() != 3 or rotary.shape[1] != 2 or not rotary.is_contiguous():
                raise ValueError("rotary must be a contiguous float32 [max_pos, 2, rot / 2] tensor")
            if rotary.device != self.device:
                raise ValueError("rotary must be on the plan's device")
            rot = (rotary.data_ptr(), rotary.shape[0], 2 * rotary.shape[2], int(interleaved))
        ext = _ext()
        self.handle = binding.scaled_attn_create(q_heads, kv_heads, dim, page_size, dev)
        self._p = ext.plan(self.handle, self.q_heads, self.kv_heads, self.dim, self.page_size, dev, *rot)
        self._append, self._decode, self._chunk, self._prompt = ext.append, ext.decode, ext.chunk, ext.prompt

    def new_cache(self, num_pages):
        return KVCache.new(num_pages, self.kv_heads, self.page_size, self.dim, self.device)

    # -- operators ----------------------------------------------------------------

    def append(self, q, k, v, cache, block_table, ctx_lens, cu_seqlens, k_out=False, q_out=None, stream=None):
        """Rotate q and k, append k and v to the cache behind the ctx_lens [B] tokens that
        each sequence has there; sequence b's new rows are cu_seqlens[b] .. cu_seqlens[b + 1].
        Returns (rotated q, rotated k or None)."""
        return self._append(self._p, q, k, v, cache._c, block_table, ctx_lens, cu_seqlens, k_out, q_out, stream)

    def decode(self, q, cache, block_table, kv_lens, q_tokens=1, scale=None, out=None, lse=None, stream=None):
        """Attention of each sequence's newest q_tokens tokens (q [B * q_tokens, Hq, dim]) over its
        first kv_lens [B] tokens in the cache, themselves included.  Returns (out, lse)."""
        return self._decode(self._p, q, cache._c, block_table, kv_lens, q_tokens, scale, out, lse, stream)

    def chunk(self, q, cache, block_table, kv_lens, cu_q, scale=None, out=None, lse=None, stream=None):
        """Attention of chunks of new tokens over the cache, as many for each sequence as there are: rows cu_q[b] .. cu_q[b + 1]
        of q are sequence b's newest tokens, over its first kv_lens [B] tokens in the cache, themselves
        included (causal).  Returns (out, lse)."""
        return self._chunk(self._p, q, cache._c, block_table, kv_lens, cu_q, scale, out, lse, stream)

    def prompt(self, q, k, v, cu_q, cu_k=None, causal=True, scale=None, out=None, lse=None, stream=None):
        """Attention within each of the packed sequences: queries cu_q[b] .. cu_q[b + 1] over keys
        cu_k[b] .. cu_k[b + 1] (cu_k None: the same).  causal: the last query sees every
        key.  Returns (out, lse)."""
        return self._prompt(self._p, q, k, v, cu_q, cu_k, causal, scale, out, lse, stream)

    def close(self):
        if getattr(self, "handle", None):
            self._p = None  # calls after this are refused
            binding.scaled_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
