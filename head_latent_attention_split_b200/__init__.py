"""Absorbed multi-head latent attention (MLA) decode for B200 (sm_100a).

One decode step over a paged, compressed latent KV cache: every query head scores its
absorbed query against each cached token's latent c_t (plus the decoupled RoPE key)
and sums the latents back with the softmax weights, so one latent tile serves as both
key and value. The kernels live in libmla_decode.so (C ABI: include/mla_decode.h);
this package is a thin binding over it. The sparse variant (DeepSeek Sparse Attention:
FP8 lightning indexer, top-k selection, decode over the selected tokens) shares the cache.
What bounds the work and the cache of a long generation stands beside it: decode over a sliding
window with sink tokens, the attention weight of every cached token, eviction by that weight, and
the verification of drafted tokens after a multi-token decode.
"""
from .binding import (BF16, E4M3, F32, KERNELS, AppendParams, MlaError, Params, abi_version,  # noqa: F401
                      HeadGemmParams, device_status, make_append_params, mla_cache_append, mla_head_gemm,
                      host_io_workspace_size, make_params, mla_decode, mla_decode_host_io, mla_decode_timed, plan_host,
                      mla_decode_noalloc, noalloc_max_workspace, DsaParams, make_dsa_params, mla_dsa_index,
                      mla_dsa_topk, mla_sparse_decode, mla_window_decode, mla_attention_mass, EvictParams,
                      CompactParams, VerifyParams, mla_evict_select, mla_cache_compact, mla_verify_drafts,
                      plan_probe, resolve, set_wait_timeout_ns, status_string, wait_timeout_ns, workspace_size)
from .api import (attention_mass, cache_append, cache_compact, decode, decode_host_io, dsa_index,  # noqa: F401
                  dsa_params_for, dsa_topk, evict_select, head_gemm, params_for, sparse_decode, verify_drafts,
                  window_decode)
