"""B200 (sm_100a) fused mixture-of-experts expert forward.

The compute lives in libmoe_b200.so (C ABI: include/moe.h); this package is a
thin binding over it (ctypes, and the compiled module _moe_torch for the operators
around the forward) plus seeded synthetic workloads.  Importing the
package does not load the library; the first call does, and raises if the
library was not built (there is no CPU fallback).
"""

from ._abi import (MoeConfig, MoeError, MoeTensor, MoeW13, align, builtin_config_count,  # noqa: F401
                   config_override, desc, device_errors, forward, forward_host, forward_status,
                   get_config, last_launch_count, load, make_config, profile_enable, profile_read,
                   quantize_mxfp4, router_status, router_topk, set_config_table, version, w13_from_packed, w13_from_views,
                   workspace_bytes, workspace_layout, debug_capture, MOE_CAPTURE_H_PREQUANT,
                   measure_mma_peak, backward, backward_input, backward_status, backward_workspace_bytes,
                   transpose_experts, host_workspace_bytes)
from .block import (SCALE_E4M3_16, SCALE_E8M0_32, layer_decode, layer_decode_workspace_bytes, linear_fp4,  # noqa: F401
                    linear_fp4_workspace_bytes, norm_after, norm_after_backward,
                    norm_backward_workspace_bytes, norm_before, norm_before_backward, quantize_nvfp4)
