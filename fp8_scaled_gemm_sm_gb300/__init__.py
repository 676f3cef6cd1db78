"""GB300 (sm_103a) scaled FP8 / BF16 GEMM.

``C[M,N] = bf16((A[M,K] . B[N,K]^T) scaled)`` with fp32 accumulation, in the
ptpc, blockscale, mxfp8 and bf16 modes, computed by hand-written tcgen05 / TMA
kernels in ``libscaledgemm.so`` (C ABI: ``include/scaled_gemm.h``).

``binding`` is a thin ctypes layer with the C ABI's names; ``ScaledGemm`` wraps
it for torch CUDA tensors.  There is no fallback: if the library is missing or
the device is not sm_103, calls raise.  Importing the package loads nothing;
the library is loaded by the first call.

``PagedAttention`` is the attention between two such GEMMs: rotary positions and
append to a paged 8-bit key/value cache, attention of the newest tokens over it,
and attention over whole prompts (``include/scaled_attention.h``); ``PagePool`` shares
the cache's pages out among sequences.  ``norm_quantize`` is the step before a GEMM: a residual's
addition, root-mean-square norm and quantisation.
"""
from .binding import MODES, ScaledGemm, ScaledGemmError  # noqa: F401


def __getattr__(name):
    # the attention layer imports torch, so it is loaded when first asked for
    if name in ("KVCache", "PagedAttention", "rotary_table"):
        from . import attention

        return getattr(attention, name)
    if name == "PagePool":
        from .pages import PagePool

        return PagePool
    if name == "norm_quantize":
        from .norm import norm_quantize

        return norm_quantize
    raise AttributeError("module %r has no attribute %r" % (__name__, name))
