"""integer_quantized_nn_amd -- integer-quantized convolution and GEMM on MI355X.

The compute path is libiqnn.so (HIP kernels for gfx950 behind the C ABI in
include/iqnn.h); this package is its Python binding.  Importing the package
does not load the library; the first call does, and raises if it is missing.
"""
from .binding import (  # noqa: F401
    ACT_GELU, ACT_GELU_TANH, ACT_RELU, ACT_SILU, BFLOAT16, EPI_ADD, EPI_ADD_RELU, EPI_NONE, EPI_RAW_INT32, EPI_RELU, FLOAT16, FLOAT32, INT4, INT8, INT32,
    UINT4, UINT8, CkptWgradDesc, ConvDesc, GemmDesc, IqnnError, W4Desc, iqnn_abi_version, iqnn_choose_qparams, iqnn_dequantize, iqnn_maxpool2d, iqnn_qconv_fwd,
    iqnn_qconv_pair_fwd,
    iqnn_qconv_packed_size, iqnn_qconv_prepack, iqnn_qconv_prepack_host, iqnn_qgemm_fwd, iqnn_qgemm_packed_size,
    iqnn_qgemm_prepack, iqnn_qgemm_prepack_host,
    iqnn_quantize, iqnn_quantize_pad,
    iqnn_ckpt_act_bwd, iqnn_ckpt_act_fwd, iqnn_ckpt_wgrad, iqnn_ckpt_wgrad_workspace, iqnn_dequantize_groups,
    iqnn_quantize_groups, iqnn_w4_fwd, iqnn_w4_kernel, iqnn_w4_packed_size, iqnn_w4_prepack,
)
