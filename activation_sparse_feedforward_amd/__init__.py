"""TwELL activation-sparse gated FFN for MI355X (gfx950).

The compute path is libtwell.so (HIP kernels + C ABI, include/twell.h); the
Python module ``twell`` is its thin ctypes binding.  ``workloads`` draws the
seeded synthetic inputs.
"""
from .twell import (Act, Desc, MoeDesc, MoeOut, MoeWeights, Route, TwellError, WDesc, Weights,  # noqa: F401
                    alloc_act, alloc_moe_out, alloc_moe_weights, alloc_moe_ws, alloc_route, alloc_weights, library,
                    moe_ws_bytes, sizes, status_str, twell_dense_ffn_fwd, twell_ffn_bwd, twell_ffn_fwd,
                    twell_ffn_fwd_hybrid, twell_linear_fwd, twell_moe_fwd, twell_pack, twell_pack_classic,
                    twell_weights_pack, twell_weights_unpack)
