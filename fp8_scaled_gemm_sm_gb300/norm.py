"""A residual's addition, root-mean-square norm and quantisation before a scaled GEMM, for
torch CUDA tensors (C ABI: ``scaled_gemm_norm_quantize`` in ``include/scaled_gemm.h``)."""
from . import binding
from .attention import _ext


def norm_quantize(mode, x, weight, eps=1e-6, residual=None, residual_out=None, stream=None):
    """r = x + residual, rounded to x's type; y = r / sqrt(mean(r^2) + eps) * weight over each row of
    x [R, C] (bfloat16 or float32, as residual and weight [C]); y quantised for a GEMM of `mode`.

    Returns (codes, scales, r): codes uint8 [R, C] and scales as ``binding.quantize`` gives them, or for
    mode "bf16" y in bfloat16 and None.  Without a residual r is x.  `residual_out` takes r
    (it may be x or residual itself; None: a new tensor).  Runs on torch's current stream or on
    `stream` (a CUDA stream's number), as the calls of ``PagedAttention`` do; no backward pass.
    """
    if mode not in binding.MODES:
        raise ValueError("norm_quantize: mode must be bf16, ptpc, blockscale or mxfp8")
    return _ext().norm_quantize(binding.MODES[mode], x, weight, eps, residual, residual_out, stream)
