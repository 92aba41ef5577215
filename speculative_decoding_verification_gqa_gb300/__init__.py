"""GB300-native speculative-decoding verification: GQA verify attention and greedy
acceptance as hand-written sm_103a CUDA kernels behind a C ABI (libspecverify.so).

Python entry points (argument marshalling over the C ABI; see ``api``):
``spec_verify_attn``, ``spec_verify_attn_paged``, ``spec_verify_attn_host_lengths``,
``spec_verify_attn_shared`` (groups with a common prefix),
``spec_pages_fork``, ``spec_pages_extend``, ``spec_pages_trim``, ``spec_pages_compact`` (the
pages of a paged cache), ``spec_kv4_write``, ``spec_kv4_read``, ``spec_verify_attn_kv4`` (a
cache held in 4 bits), ``spec_attn_mass``, ``spec_kv_evict`` (eviction by accumulated attention
weight), ``spec_accept``, ``spec_accept_stochastic``,
``spec_draft_signals``, ``workspace_status``, and ``plan_preview`` (the attention calls' work
plan, computed on the host).
"""
from .api import (AttnDesc, PagePools, SpecVerifyError, accept_workspace_bytes,
                  evict_workspace_bytes, kv4_workspace_bytes, load_library,
                  mass_workspace_bytes, new_workspace, page_pools, paged_attn_desc,
                  pages_workspace_bytes, plan_preview, set_attn_kernel, set_profile_events,
                  set_unit_ctas, shared_workspace_bytes, signals_workspace_bytes, spec_accept,
                  spec_accept_stochastic, spec_attn_mass, spec_draft_signals, spec_kv4_read,
                  spec_kv4_write, spec_kv_evict, spec_pages_compact, spec_pages_extend,
                  spec_pages_fork, spec_pages_trim, spec_verify_attn,
                  spec_verify_attn_host_lengths, spec_verify_attn_kv4, spec_verify_attn_paged,
                  spec_verify_attn_shared, verify_kv4_workspace_bytes, verify_workspace_bytes,
                  workspace_status)

__all__ = ["AttnDesc", "PagePools", "SpecVerifyError", "accept_workspace_bytes",
           "evict_workspace_bytes", "kv4_workspace_bytes", "load_library",
           "mass_workspace_bytes", "new_workspace", "page_pools", "paged_attn_desc",
           "pages_workspace_bytes", "plan_preview", "set_attn_kernel", "set_profile_events",
           "set_unit_ctas", "shared_workspace_bytes", "signals_workspace_bytes", "spec_accept",
           "spec_accept_stochastic", "spec_attn_mass", "spec_draft_signals", "spec_kv4_read",
           "spec_kv4_write", "spec_kv_evict", "spec_pages_compact", "spec_pages_extend",
           "spec_pages_fork", "spec_pages_trim", "spec_verify_attn",
           "spec_verify_attn_host_lengths", "spec_verify_attn_kv4", "spec_verify_attn_paged",
           "spec_verify_attn_shared", "verify_kv4_workspace_bytes", "verify_workspace_bytes",
           "workspace_status"]
