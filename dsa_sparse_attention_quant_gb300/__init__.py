"""GB300-native (sm_103a) DSA sparse-attention indexer with IndexCache reuse.

The compute lives in ``libdsaidx.so`` (CUDA kernels behind the C ABI of
``include/dsaidx.h``); ``binding`` is its thin Python face, ``attention`` that
of the attention over the paged KV cache and of the cache's pages. ``synth``
builds seeded synthetic inputs.
"""
from .binding import (  # noqa: F401
    Batch,
    DsaError,
    LayerStack,
    cache_format,
    check_device_error,
    gather_rows,
    indexer_k_quant_write,
    indexer_k_rope_quant_write,
    indexer_logits,
    indexer_logits_topk,
    indexer_plan,
    indexer_q_quant_fold,
    indexer_q_rope_quant_fold,
    indexer_topk,
    indexer_workspace_size,
    layer_stack_run,
    layer_stack_workspace_size,
    load,
    new_k_cache,
    schedule_build,
    topk_logical_to_physical,
)
from .attention import (  # noqa: F401
    attn_decode,
    attn_decode8,
    attn_decode8_workspace_size,
    attn_decode_workspace_size,
    attn_prompt,
    attn_selected,
    attn_selected8,
    attn_selected8_workspace_size,
    attn_selected_workspace_size,
    kv_read8,
    kv_write,
    kv_write8,
    kv_write8_workspace_size,
    new_kv_cache,
    new_kv_cache8,
    pages_compact,
    pages_copy,
    pages_fork,
    pages_free,
    pages_workspace_size,
)

__version__ = "0.3.1"
