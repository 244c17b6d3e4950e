"""GB300 fake-quant library: QAT fake quantization (int8/int4 symmetric and
affine per tensor / row / group, saturating FP8 E4M3/E5M2), its
straight-through-estimator backward, and the QLoRA two-level 4-bit block
format, as CUDA kernels for sm_103a behind a C ABI (include/qat.h); the
integer and FP8 maps also round stochastically with counter-based draws;
units may also be columns, and calibration takes a clip factor and binary16
scales; block-scaled floating-point formats (MX with E8M0 scales, NVFP4
with E4M3 scales under an FP32 tensor scale).  Layer operators use those
weights: products with 4-bit codes, the gated feed-forward block and layer
norm, forward and backward; attention operators serve a layer from a quantized
key-value cache: norms of queries and keys with the position rotation (forward and
backward), cache writes and reads, and the attention of single tokens over it.
"""
from ._lib import QatError, load  # noqa: F401
from .api import (DoubleQuantized4Bit, FakeQuantBlock, FakeQuantFp8, FakeQuantInt,  # noqa: F401
                  FakeQuantSTE, fake_quant_block, qat_fake_quant_block,
                  OptimizerStep, QatDataError, adam_hparams, amax_stats, calib_options,
                  dequantize_4bit_double,
                  fake_quant_backward, optimizer_step, qat_optimizer_step,
                  fake_quant_fp8, fake_quant_int, fake_quant_int_percentile, qat_amax_stats,
                  qat_dequant4_double, qat_fake_quant_int_percentile,
                  qat_percentile_workspace_bytes,
                  qat_fake_quant_fp8, qat_fake_quant_fp8_sr, qat_fake_quant_int,
                  qat_fake_quant_int_opts, qat_fake_quant_int_sr, qat_kernel_launch_count,
                  qat_quant4_double, qat_ste_backward, qat_workspace_bytes, quantize_4bit_double,
                  raise_on_flags)
from .layers import (GatedFfn, GatedFfnFunction, LayerNorm, LayerNormFunction, Weight4,  # noqa: F401
                     gated_ffn, gated_ffn4, gated_ffn_backward, layer_norm, layer_norm_backward,
                     linear4, qat_gated_ffn, qat_gated_ffn_backward,
                     qat_gated_ffn4, qat_gated_ffn4_workspace_bytes, qat_gated_ffn_workspace_bytes, qat_layer_norm, qat_layer_norm_backward,
                     qat_layer_norm_backward_workspace_bytes, qat_linear4, qat_linear4_workspace_bytes, weight4, weight4_double)
from .attention import (HeadNormRope, HeadNormRopeFunction, KeysValues, KvAttention, KVCache,  # noqa: F401
                        head_norm_rope, head_norm_rope_backward, kv_attention, kv_cache, kv_read, kv_write,
                        qat_head_norm_rope, qat_head_norm_rope_backward,
                        qat_head_norm_rope_backward_workspace_bytes, qat_kv_attention,
                        qat_kv_attention_workspace_bytes, qat_kv_read, qat_kv_write, rope_frequencies,
                        rope_turns)
