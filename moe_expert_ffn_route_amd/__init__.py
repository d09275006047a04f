"""MI355X (gfx950) fused W8A8 MoE expert block, and the pre-norm, router and
4-bit dense products around it.

The compute lives in libmoe_w8a8.so (hand-written HIP kernels behind the C ABI
of include/moe_w8a8.h); `binding` is its ctypes front end and `synth` draws
seeded synthetic inputs.
"""
from .binding import (Debug, Dims, MoeError, Runner, debug_buffers, dims_of_case, library, make_dims,  # noqa: F401
                      moe_w8a8_forward, moe_w8a8_forward_noalloc, moe_w8a8_pack_weights, moe_w8a8_pack_weights_mx,
                      moe_w8a8_packed_mx_bytes, moe_w8a8_read_probe, moe_w8a8_read_write_probe,
                      moe_w8a8_status_string, moe_w8a8_warm, moe_w8a8_workspace_size,
                      pack_weights, upload, MOE_PACK_GMM1, MOE_PACK_GMM2, MOE_WEIGHT_INT8, MOE_WEIGHT_MXFP4,
                      MOE_WEIGHT_PACKED, MOE_WEIGHT_ROW_MAJOR)
from .binding import (GateDims, LinearW4Dims, NormDims, make_gate_dims, make_linear_w4_dims, make_norm_dims,  # noqa: F401
                      moe_w8a8_forward_quantized, moe_w8a8_gate, moe_w8a8_gate_workspace_size, moe_w8a8_linear_w4,
                      moe_w8a8_norm_quant, moe_w8a8_pack_weights_w4, moe_w8a8_packed_w4_bytes,
                      MOE_DTYPE_BF16, MOE_DTYPE_FP16, MOE_DTYPE_FP32, MOE_DTYPE_INT8, MOE_QUANT_E4M3,
                      MOE_QUANT_INT8, MOE_QUANT_NONE, MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, MOE_SCORE_SQRT_SOFTPLUS)
