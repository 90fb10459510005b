"""SVDQuant W4A4 linear layer for NVIDIA B200 (sm_100a).

    Y = Xh L1 L2 + Q(Xh) Q(R) + bias,   Xh = X diag(lambda)^-1

Beside it an 8-bit layer (FP8 codes, one scale per 128) with its norm, GELU
and quantisers fused: ``rmsnorm``, ``linear_fp8_gelu``, ``linear_fp8``,
``quantize_fp8``, ``pack_weight_fp8``.

The product is the C-ABI library ``libsvdq.so`` (include/svdq.h); this
package is a thin ctypes binding with the same call names.  Every step of the
layer runs in the library's CUDA kernels; there is no CPU fallback, and the
binding raises if the library is missing.
"""

from .binding import (  # noqa: F401
    SvdqError,
    attach_lora,
    channel_absmax,
    fp8_sizes,
    lib_path,
    linear,
    linear_fp8,
    linear_fp8_gelu,
    load,
    pack_residual,
    pack_weight_fp8,
    packed_sizes,
    quantize_act,
    quantize_fp8,
    rmsnorm,
    selftest_wait_timeout,
    set_launch_overlap,
    set_linear_fp8_path,
    set_linear_fp8_splits,
    set_linear_path,
    set_wait_timeout,
    status_string,
    sync_status,
)
