"""Grouped-convolution forward engine for AMD Instinct MI355X (gfx950), with the
backward of the (batch, steps, channels) depthwise conv1d, and the sequence operators
beside that conv in a mixing block: its causal form with a carried state, linear
attention with a decay for each head, and RMS norm with the residual's addition.

The compute runs in libgconv.so (hand-written HIP kernels behind the C ABI in
include/gconv.h); this package is its Python binding.  Importing the package
does not load the library; the first call does, and raises if it is missing.
"""
from ._binding import (  # noqa: F401
    DW1D_BWD_FILTER_SCRATCH_BYTES,
    EXPORTS,
    GconvError,
    GconvLaunchError,
    PreparedCall,
    conv2d,
    conv2d_nhwc,
    dwconv1d_btc,
    dwconv1d_btc_backward,
    gconv_autotune,
    gconv_autotune_clear,
    gconv_dw1d_bwd_data,
    gconv_dw1d_bwd_filter,
    gconv_dw1d_bwd_filter_noalloc,
    gconv_dw1d_bwd_filter_workspace,
    gconv_fwd,
    gconv_fwd_ex,
    gconv_fwd_route,
    gconv_last_error,
    gconv_last_kernel,
    gconv_out_shape,
    gconv_select_route,
    gconv_status_string,
    lib,
    lib_path,
)
from ._sequence import (  # noqa: F401
    dwconv1d_causal,
    dwconv1d_causal_backward,
    dwconv1d_causal_step,
    linear_attention,
    linear_attention_backward,
    linear_attention_step,
    linear_attention_workspace,
    rms_norm,
    rms_norm_backward,
    rms_norm_e4m3,
)
