"""Decode-time routed Mixture-of-Experts layer for GB300 (sm_103a).

The compute path is the C ABI of include/moe.h, implemented by hand-written CUDA kernels
in ``csrc/`` and built in-tree into ``libmoe.so``; ``moe`` is its Python binding, ``batch`` the binding of
the calls for a batch of tokens in 16-bit weights (no context).
"""
from .moe import (Config, Context, FileTier, MoeError, Stats, expert_blob_bytes, lib, route_noalloc,  # noqa: F401
                  rvq_block_split,
                  strerror, ROUTER_SOFTMAX, ROUTER_SIGMOID, W_RVQ3, W_INT4,
                  OK, EINVAL, ENOMEM, EBUDGET, ECUDA, ESTATE, ETIMEOUT, ENOTFOUND, EIO)
from .batch import (debug_batch_wait, group_route, group_route_workspace, grouped_kernel, grouped_matmul, grouped_wgrad, grouped_workspace,
                    grouped_wgrad_workspace, verify_draft,  # noqa: F401
                    GroupedArgs, GroupedWgradArgs, VerifyArgs, T_BF16, T_FP16, T_FP32, GROUP_NK, GROUP_KN,
                    ACT_NONE, ACT_SWIGLU, GROUPED_NONE, GROUPED_FEW, GROUPED_PAIR, GROUPED_ANY)
