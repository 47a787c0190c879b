"""B200-native W8A8 int8-dynamic linear layers.

Dynamic per-token symmetric int8 activation quantisation, a load-time weight
repack into tensor-core tile images, and int8 x int8 -> int32 GEMMs on the
sm_100a tensor cores (tcgen05, TMEM accumulators) with a dequantising bf16
epilogue -- exposed as the C ABI of libw8a8.so (include/w8a8.h) and bound here
with ctypes.  Beside them the same layers with both operands in microscaled
4-bit (``MX4Linear``, ``mx4_*``), and the norms around a block with its gate and
residual, which form the next layer's codes (``block_norm``).  The library is
loaded on first use; there is no CPU fallback.
"""
from .binding import (  # noqa: F401
    ACT_GELU_TANH, ACT_NONE, PATH_AUTO, PATH_LARGE, PATH_LARGE_BN128, PATH_LARGE_BN256, PATH_LARGE_PAIR, PATH_LARGE_PAIR128,
    PATH_SMALL, W8A8Error, W8A8Linear,
    gelu_tanh, gemm_kernel_name, launch_count, lib, linear, linear_act_quant,
    linear_act_quant_workspace_bytes, linear_workspace_bytes, pack_weight, pack_weight_int32, packed_weight_bytes,
    poll_status, quant_act, quant_act_static, quant_pack_weight, scaled_mm, scaled_mm_i32, scaled_mm_workspace_bytes, selftest_int8_mma_rate, selftest_wait_timeout,
    set_path, unpack_weight)
from .mx4 import (  # noqa: F401
    MX4Linear, MX4Tensor, mx4_bytes, mx4_dequant, mx4_linear, mx4_linear_quant,
    mx4_linear_workspace_bytes, mx4_pack, mx4_quant, mx4_scaled_mm, mx4_scaled_mm_quant, mx4_unpack)
from .norms import BlockNormOutput, Norm, block_norm  # noqa: F401
