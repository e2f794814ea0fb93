"""TwELL activation-sparse gated FFN for MI355X (gfx950).

The compute path is libtwell.so (HIP kernels + C ABI, include/twell.h); the
Python module ``twell`` is its thin ctypes binding.  ``workloads`` draws the
seeded synthetic inputs.
"""
from .twell import (Act, Desc, Fp8Desc, MoeDesc, MoeOut, MoeWeights, NormDesc, Route, TokensDesc, TokensOrder,  # noqa: F401
                    TwellError, WDesc, Weights, alloc_act, alloc_fp8_weights, alloc_fp8_ws, alloc_moe_out,
                    alloc_moe_weights, alloc_moe_ws, alloc_norm_ws, alloc_route, alloc_tokens_order,
                    alloc_tokens_ws, alloc_weights, fp8_ws_bytes, library, moe_ws_bytes, sizes, status_str,
                    twell_dense_ffn_fwd, twell_ffn_bwd, twell_ffn_fwd, twell_ffn_fwd_hybrid, twell_fp8_linear_bwd,
                    twell_fp8_linear_fwd, twell_fp8_weights_pack, twell_fp8_weights_unpack, twell_layernorm_bwd,
                    twell_layernorm_fwd, twell_linear_fwd, twell_moe_fwd, twell_pack, twell_pack_classic,
                    twell_tokens_combine, twell_tokens_combine_bwd, twell_tokens_gather, twell_tokens_sort,
                    twell_weights_pack, twell_weights_unpack)
