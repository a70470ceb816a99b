"""MiniMax Sparse Attention (MSA) hot path on one B200 (sm_100a).

The work runs in libmsa.so (C ABI: include/msa.h); ``msa`` is its thin
Python binding, ``inputs`` the seeded synthetic workloads, ``build`` the nvcc
build of the library.
"""
from .msa import (MSAError, Workspace, attn_paged, attn_paged_i8, attn_paged_kernels,  # noqa: F401
                  device_status, index_topk, index_topk_i8, index_topk_paged, kv_append, kv_append_i8, kv_gather,
                  kv_gather_i8, load_library, select_invert, selftest_umma, sparse_attn,
                  sparse_attn_decode_noalloc, sparse_attn_paged, sparse_attn_paged_i8,
                  status_string, workspace_size)
