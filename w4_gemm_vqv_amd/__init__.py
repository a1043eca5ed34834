"""libvqv: W4 verify projection and greedy verify for MI355X (gfx950), and the
operators around them in a verify round and in batches of many requests.

The compute path is the HIP library ``libvqv.so`` (C ABI in include/vqv.h,
include/vqv_round.h and include/vqv_serve.h); ``w4_gemm_vqv_amd.vqv``,
``w4_gemm_vqv_amd.round`` and ``w4_gemm_vqv_amd.serve`` are its Python bindings. Build with
``python -m w4_gemm_vqv_amd.build``.
"""

from .round import (ROPE_SCALINGS, ROUND_EXPORTS, Edits, PagedCache, Pages, Rope, Sequences, vqv_cache_compact,
                    vqv_cache_copy, vqv_cache_fork, vqv_cache_reserve, vqv_cache_trim,
                    vqv_cache_workspace_bytes, vqv_logits_edit, vqv_logits_verify,
                    vqv_paged_attn, vqv_paged_attn_workspace_bytes, vqv_rope_append)
from .serve import (SERVE_EXPORTS, Adapters, PagedCacheQ4, vqv_cache_q4_read, vqv_lora_add,
                    vqv_lora_add_workspace_bytes, vqv_paged_attn_q4,
                    vqv_paged_attn_q4_workspace_bytes, vqv_q4_record_bytes, vqv_rope_append_q4,
                    vqv_verify_sampled, vqv_verify_sampled_workspace_bytes)
from .vqv import (EXPORTS, LIB_PATH, VQV_BF16, VQV_ERR_ALIGN, VQV_ERR_ARG, VQV_ERR_HIP,
                  VQV_ERR_UNSUPPORTED, VQV_ERR_WORKSPACE, VQV_FP16, VQV_FP32, VQV_OK, VqvError,
                  VQV_NOALLOC_SCRATCH_BYTES, lib, vqv_abi_version, vqv_qgemm, vqv_qgemm_kernel,
                  vqv_qgemm_swiglu,
                  vqv_qgemm_swiglu_workspace_bytes, vqv_qgemm_verify, vqv_qgemm_verify_ex,
                  vqv_qgemm_verify_ex_noalloc,
                  vqv_qgemm_verify_workspace_bytes, vqv_qgemm_workspace_bytes, vqv_status_string,
                  vqv_verify, vqv_verify_ex, vqv_verify_workspace_bytes)

__all__ = ["EXPORTS", "LIB_PATH", "VQV_BF16", "VQV_ERR_ALIGN", "VQV_ERR_ARG", "VQV_ERR_HIP",
           "VQV_ERR_UNSUPPORTED", "VQV_ERR_WORKSPACE", "VQV_FP16", "VQV_FP32", "VQV_OK",
           "VQV_NOALLOC_SCRATCH_BYTES", "VqvError", "lib", "vqv_abi_version", "vqv_qgemm",
           "vqv_qgemm_kernel", "vqv_qgemm_swiglu",
           "vqv_qgemm_swiglu_workspace_bytes", "vqv_qgemm_verify",
           "vqv_qgemm_verify_ex", "vqv_qgemm_verify_ex_noalloc",
           "vqv_qgemm_verify_workspace_bytes", "vqv_qgemm_workspace_bytes",
           "vqv_status_string", "vqv_verify", "vqv_verify_ex", "vqv_verify_workspace_bytes",
           "ROPE_SCALINGS", "ROUND_EXPORTS", "Edits", "PagedCache", "Pages", "Rope", "Sequences",
           "vqv_cache_compact", "vqv_cache_copy", "vqv_cache_fork", "vqv_cache_reserve",
           "vqv_cache_trim", "vqv_cache_workspace_bytes", "vqv_logits_edit", "vqv_logits_verify",
           "vqv_paged_attn", "vqv_paged_attn_workspace_bytes", "vqv_rope_append",
           "SERVE_EXPORTS", "Adapters", "PagedCacheQ4", "vqv_cache_q4_read", "vqv_lora_add",
           "vqv_lora_add_workspace_bytes", "vqv_paged_attn_q4",
           "vqv_paged_attn_q4_workspace_bytes", "vqv_q4_record_bytes", "vqv_rope_append_q4",
           "vqv_verify_sampled", "vqv_verify_sampled_workspace_bytes"]
