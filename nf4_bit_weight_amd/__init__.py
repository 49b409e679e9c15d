"""MI355X (gfx950) fused NF4 dequantise-and-multiply.

The compute lives in libnf4.so (hand-written HIP kernels behind the C ABI of
include/nf4.h, include/nf4_attn.h, include/nf4_experts.h and include/nf4_int8.h).
This package is its Python binding: `api`, `attention`, `experts` and `int8` marshal
tensors to the C entry points, `autograd` wraps them as checkpoint-visible Functions.
Importing the package does not load the library; the first call does, and it
raises if the library has not been built.
"""

from .api import (NF4Weight, nf4_dequantize, nf4_grouped_matmul_bwd_input,  # noqa: F401
                  nf4_grouped_matmul_fwd, nf4_matmul_bwd_input, nf4_matmul_fwd,
                  nf4_path_counts, nf4_quantize, nf4_reset_path_counts, nf4_workspace_bytes)
from .attention import (NF4KVCache, nf4_kv_append, nf4_kv_attention, nf4_kv_attention_workspace,  # noqa: F401
                        nf4_kv_cache, nf4_kv_dequantize, nf4_prompt_attention_bwd, nf4_prompt_attention_fwd)
from .autograd import (NF4GroupedMatMul, NF4MatMul, nf4_grouped_linear, nf4_linear,  # noqa: F401
                       nf4_prompt_attention)
from .experts import (NF4Routing, nf4_expert_combine, nf4_expert_combine_bwd, nf4_expert_gather,  # noqa: F401
                      nf4_expert_gather_bwd, nf4_expert_plan, nf4_route, nf4_route_bwd)
from .int8 import (NF4Int8, nf4_int8_grouped_matmul, nf4_int8_matmul, nf4_int8_quantize,  # noqa: F401
                   nf4_int8_workspace)
