"""prefix_shared_tree_attention_gb300 — tree training's hot path on GB300.

A thin Python binding over libtpa (include/tpa.h): argument marshalling and
torch-owned device memory only; every step runs in the library (the C++
packer on the host, CUDA kernels for sm_103a on the device). Functions keep
the C names without the ``tpa_`` prefix:

    tree = tree_pack(seqs, max_tokens_per_mb)           # host trie packer
    tree = tree_pack_padded(input_ids, attention_mask, max_tokens_per_mb)  # from a padded batch
    dtree = tree.upload(device)                         # metadata -> HBM
    mask = block_classify(dtree)                        # 128x128 tile classes + CSR
    dense = dense_mask(dtree)                           # [B, T, T] ancestor mask (Megatron-style)
    o, lse = tree_attn_fwd(dtree, mask, q, k, v)
    dq, dk, dv = tree_attn_bwd(dtree, mask, q, k, v, o, lse, dout)
    pos_logp, pos_ent, seq_logp, seq_ent = tree_logprobs_entropy(dtree, logits)
    pos_logp, pos_ent, seq_logp, seq_ent = lm_head_logprobs_entropy(dtree, hidden, weight)  # no logits tensor
    group_of, n_groups, algo = balance(weights, capacity, min_groups, 1, "kk")  # trees -> ranks
    metrics = packing_metrics(weights, group_of, n_groups, capacity)

The policy's operators, around the tree attention and for sampling:

    table = rope_table(n_positions, rot_dim)            # cos | sin, once for a model
    q, k = qk_norm_rope_fwd(dtree, q, k, table, wq, wk) # head norms and rotation at the tree's depths
    dq, dk, dwq, dwk = qk_norm_rope_bwd(dtree, dq, dk, q, k, table, wq, wk)
    q = paged_append(k_cache, v_cache, pages, offsets, kv_lens, k, v, q=q, table=table)  # new tokens
    o, lse = paged_attn_fwd(k_cache, v_cache, pages, offsets, kv_lens, q, max_q_len)
    tokens, n_accepted = verify_drafts(target_probs, draft_tokens, u_accept, u_next, draft_probs)
    tokens, logp = sample_tokens(logits, u, temperature, top_k, top_p, min_p)

A step that drafts a tree for each sequence, and the pages of the cache:

    positions, masks = draft_masks(parents, offsets, kv_lens, max_q_len)
    o, lse = paged_attn_tree_fwd(k_cache, v_cache, pages, offsets, kv_lens, q, masks, max_q_len)
    tokens, path, n_accepted = accept_drafts(parents, offsets, draft_tokens, sampled, max_path)
    kv_lens = paged_compact(k_cache, v_cache, pages, offsets, kv_lens, path, n_accepted)
    n_free = paged_resize(pages, kv_lens, refs, page_size)                     # pages handed out and given back
    n_free = paged_fork(k_cache, v_cache, pages, kv_lens, refs, src, dst)      # samples of a prompt
"""
from ._abi import BLOCK_SIZE, LOGITS_COMPACT, LOGITS_PADDED, STATUS, TpaError, lib  # noqa: F401
from .api import (  # noqa: F401
    BlockMask, DeviceTree, Tree, accept_drafts, balance, block_classify, dense_mask, device_check, draft_masks,
    extract_sequences, lm_head_logprobs_entropy, lm_head_workspace_bytes, packing_metrics, paged_append, paged_attn_fwd,
    paged_attn_tree_fwd, paged_attn_workspace_bytes, paged_compact, paged_fork, paged_resize, qk_norm_rope_bwd,
    qk_norm_rope_fwd, rope_table, sample_tokens, sync_status, tree_attn_bwd, tree_attn_bwd_workspace_bytes, tree_attn_fwd,
    tree_logprobs_entropy, tree_pack, tree_pack_padded, verify_drafts, wait_probe,
)
