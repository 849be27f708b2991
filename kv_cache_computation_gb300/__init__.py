"""GB300 (sm_103a) MAC-Attention decode-step attention.

Match-Amend-Complete decode attention (arXiv 2604.00235) behind the C ABI of
include/mac.h, with a thin Python binding:

    from kv_cache_computation_gb300 import MacAttention
    mac = MacAttention(heads=32, kv_heads=8, ring_len=16, band_r=64, tau=0.3,
                       max_batch=1, max_ctx=8192, page_size=0)
    mac.append_kv(0, k_prefill, v_prefill)
    out, lse = mac.decode_step(q_pre_rope, q_post_rope, k_new, v_new)

Around it, for a serving loop: QkvRotary (norms, rotary embedding and split
of a QKV projection), page_step (pages, positions and slots of a step's new
tokens, on the GPU) and QuantKV (a KV store of 4 bits per value and decode
attention over it):

    step = page_step(lengths, new_tokens, page_table, *free, max_tokens=B)
    out, lse = QuantKV(32, 8, num_pages=4096, max_batch=B).decode_step_qkv(
        QkvRotary(32, 8), qkv, step.positions, step.slots, page_table, step.lengths, starts=step.starts)

The CUDA library must be built first (``kv_cache_computation_gb300.build``);
there is no CPU fallback.
"""
from .attention import MacAttention, make_config, query_sizes, status_string  # noqa: F401
from .paging import PageStep, new_page_pool, page_step  # noqa: F401
from .quant import QuantKV, quant_query_sizes  # noqa: F401
from .rotary import QkvRotary  # noqa: F401
from ._native import MacError  # noqa: F401
