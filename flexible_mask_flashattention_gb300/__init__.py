"""GB300 (sm_103a) Flex-Flash-Attention: fused softmax attention, forward and
backward, over AttnSlice masks, behind the C ABI of ``include/ffa.h``.

    plan = Plan(slices, seqlen_q, seqlen_k)      # block metadata on the GPU
    out, lse = fwd(q, k, v, plan, scale)
    dq, dk, dv = bwd(q, k, v, out, lse, dout, plan, scale)
    fwd_accumulate(q, k, v, plan_b, scale, out, lse)   # merge another key set in by LSE
    out, lse = lse_combine(out_a, lse_a, out_b, lse_b)
    out, lse = fwd_sink(q, k, v, plan, scale, sink)    # per-head attention-sink logits
    dq, dk, dv, dsink = bwd_sink(q, k, v, out, lse, dout, plan, scale, sink)
    q, k = qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions)   # before fwd; qk_norm_rope_bwd after bwd
    kv_cache_write(k, v, k_cache, v_cache, slots, k_exp, v_exp)        # paged cache, bf16 or quantised to e4m3
    k, v = kv_cache_read(k_cache, v_cache, page_table, cu_seqlens, total, k_exp=k_exp, v_exp=v_exp)
    out, lse = fwd_decode(q, k_cache, v_cache, page_table, kv_lens, scale, k_exp, v_exp)   # one new token a sequence
    bucket, chunk_area, bucket_area = dispatch_solve(slices, seqlen, seqlen, chunk_size, cp_size)   # host only
"""
from ._lib import (FFAError, MASK_BI_CAUSAL, MASK_CAUSAL, MASK_FULL, MASK_INV_CAUSAL, Plan, bwd,
                   bwd_sink, bwd_workspace_size, dispatch_solve, fwd, fwd_accumulate, fwd_decode,
                   fwd_decode_workspace_size, fwd_sink, kv_cache_read, kv_cache_write, load_library, lse_combine,
                   qk_norm_rope, qk_norm_rope_bwd, qk_norm_rope_bwd_workspace_size, range_gather,
                   range_scatter_reduce, selftest_bounded_wait)

__all__ = ["FFAError", "Plan", "fwd", "fwd_accumulate", "fwd_sink", "lse_combine", "bwd", "bwd_sink",
           "bwd_workspace_size", "dispatch_solve", "range_gather", "range_scatter_reduce", "load_library",
           "selftest_bounded_wait", "qk_norm_rope", "qk_norm_rope_bwd", "qk_norm_rope_bwd_workspace_size",
           "kv_cache_write", "kv_cache_read", "fwd_decode", "fwd_decode_workspace_size",
           "MASK_FULL", "MASK_CAUSAL", "MASK_INV_CAUSAL", "MASK_BI_CAUSAL"]
