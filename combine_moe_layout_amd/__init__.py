"""MI355X-native MoE token dispatch / combine (layout -> dispatch -> combine).

The compute path is a C-ABI shared library of hand-written HIP kernels for
gfx950 (``libep.so``, declared in ``include/ep.h``); ``binding`` marshals torch
tensors into it under the same names.  Importing this package loads nothing:
the library is opened on first use and a missing library is an error, never a
fallback.
"""
from .binding import (EP_ACT_GELU, EP_ACT_NONE, EP_ACT_RELU, EP_ACT_SILU, EP_ACT_SWIGLU, EP_BF16,
                      EP_F16, EP_FLAG_BAD_EXPERT, EP_FLAG_OVERFLOW, EP_FP8_E4M3,
                      EP_FP8_E4M3_POW2, EP_GRAD_ACCUMULATE, EP_GRAD_F32, EP_MXFP8_E4M3,
                      EP_SCALES_MN_MAJOR, EpError, EpGroupLayout, EpLayout, ep_act_grad,
                      ep_cast_e4m3_bits, ep_combine, ep_combine_f16, ep_combine_fp8,
                      ep_combine_grad, ep_combine_groups, ep_combine_mxfp8, ep_copy,
                      ep_dequant_fp8, ep_dequant_mxfp8, ep_dispatch, ep_expert_gemm,
                      ep_expert_gemm_grad_w, ep_expert_gemm_grad_x, ep_get_group_layout,
                      ep_get_layout, ep_layout_dispatch, ep_layout_workspace_bytes, ep_linear,
                      ep_linear_grad_w, ep_linear_grad_x, ep_num_recv_rows,
                      ep_scales_to_mn_major, ep_version)

__version__ = "0.1.0"
