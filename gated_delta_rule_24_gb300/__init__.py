"""GB300-native chunked Gated Delta Rule (GDN) prefill, and the decay linear-attention
layer next to it (q/k norm with rotation, prefill, one-token step), and what the softmax-attention
layers between linear ones need to serve (rotation on several axes, append to a paged cache, attention over it).

The compute path is a C-ABI CUDA library (``csrc/``, built for sm_103a, C ABI
in ``include/gdn.h``); this package holds its thin Python binding and the
seeded workload generators.  The binding loads the library on first use and
fails loudly when it is missing: there is no CPU fallback.
"""
from .binding import (GdnError, chunk_gated_delta_rule, decay_linear_attention, decay_linear_step,  # noqa: F401
                      device_status, gdn_chunk_prefill, gdn_chunk_prefill_checkpointed,
                      gdn_chunk_prefill_noalloc, gdn_decay_prefill, gdn_decay_step, gdn_decay_workspace_bytes,
                      gdn_decode_step, gdn_init, gdn_norm_rope_append, gdn_paged_attention_step,
                      gdn_paged_attention_workspace_bytes, gdn_qk_norm_rope, gdn_qk_norm_rope_axes,
                      gdn_reserve_workspace, gdn_split_workspace_bytes,
                      load_library, norm_rope_append, paged_attention_step, qk_norm_rope, run_problem, testing_force_splits, testing_split_plan,
                      testing_wait_limit)
