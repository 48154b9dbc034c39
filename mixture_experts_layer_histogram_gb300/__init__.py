"""Single-GPU MoE layer hot path for GB300 (sm_103a): softmax top-k routing (optionally from x and
router weights), per-expert token counting and index generation, token permutation, grouped SwiGLU
GEMM on tcgen05 tensor cores, and the weighted combine, forward and backward, behind the C ABI in
include/moe.h. MoELayer holds one layer's buffers and call order (and can record a pass as a CUDA
graph); HostPipeline runs passes from pinned host memory with the copies overlapped. Around the layer:
BlockNorms (the norms before and after it, with the gate and the residual), AdamW (one step over many
tensors, states in fp32 or 8 bits), and MoELayerFp4 / Fp4Weights (serving with MXFP4 experts)."""
from . import _lib
from ._lib import MoeError
from .block import BlockNorms
from .fp4 import Fp4Weights, MoELayerFp4, fp4_dequantize, fp4_quantize
from .layer import MoELayer
from .optim import AdamW
from .pipeline import HostPipeline

__all__ = ["MoELayer", "HostPipeline", "BlockNorms", "AdamW", "MoELayerFp4", "Fp4Weights", "fp4_quantize",
           "fp4_dequantize", "MoeError", "_lib"]
