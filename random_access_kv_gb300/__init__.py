"""FibQuant KV-cache codec on GB300 (sm_103a): Python face of the C ABI in include/fq.h.

    ctx = fq_codebook_load(C, Pi)                    # shared codebook [N, k] and rotation [d, d]
    fq_encode(ctx, x, M, nu, codes)                  # x fp16 [M, d] -> nu fp32 [M], packed codes
    fq_decode_gather(ctx, nu, codes, M, idx, n, out) # random-access decode -> fp16 [n, d]

    actx = fa_create(N, r, L)                        # iterated-map archive of symbol streams
    fa_encode(actx, sym, n_streams, n_new, T_cap, T_old, anchors)   # append (T_old = 0: encode)
    fa_access(actx, anchors, n_streams, T_cap, T, pos, n, out)      # random access

    qctx = qc_create("int8", d, n_heads, page_tokens)               # paged cache of quantised rows
    qc_norm_rope(qctx, q, k, w_q, w_k, eps, pos, table, rot, interleaved, q, k)
    qc_write(qctx, k, v, slots, pages)                              # quantise into token slots
    qc_attend(qctx, pages, q, page_table, lens, nodes, tree, scale, max_len, out, lse, workspace)
    qc_read(qctx, pages, slots, k_out, v_out)                       # the values the cache holds

All device buffers are torch CUDA tensors owned by the caller; ``alloc_store``,
``alloc_archive``, ``alloc_pages`` and ``alloc_attend_workspace`` size them.
``codebook`` builds the shared codebook and rotation on the host from seeded draws.
"""
from ._binding import (  # noqa: F401
    FQ_FLAG_NONFINITE, FQ_FLAG_RANGE, FQ_FLAG_TIMEOUT, Context, FQError, FQLibraryMissing,
    fq_attend, fq_centroid_sums, fq_code_words, fq_codebook_load, fq_decode, fq_decode_gather, fq_decode_gather_f32, fq_destroy,
    fq_encode, fq_encode_append, fq_record_bits, fq_selftest_wait, fq_shape, fq_status, fq_strerror, header_symbols,
    FA_FLAG_CORRUPT, FA_FLAG_RANGE, FA_FLAG_SYMBOL, ArchiveContext, fa_access, fa_create, fa_decode, fa_destroy,
    fa_encode, fa_max_segment, fa_params, fa_ratio_limit, fa_segments, fa_status, fa_vertex_table,
    QC_FLAG_NONFINITE, QC_FLAG_RANGE, QC_FLAG_TIMEOUT, CacheContext, qc_attend, qc_attend_workspace, qc_create, qc_destroy,
    qc_norm_rope, qc_page_bytes, qc_read, qc_status, qc_write,
)


def alloc_store(ctx, rows: int, device="cuda"):
    """Zeroed (nu fp32 [rows], codes int32 [fq_code_words(rows)]) torch tensors for a code store."""
    import torch
    nu = torch.zeros(rows, dtype=torch.float32, device=device)
    codes = torch.zeros(max(1, fq_code_words(ctx, rows)), dtype=torch.int32, device=device)
    return nu, codes


def alloc_archive(ctx, n_streams: int, T_cap: int, device="cuda"):
    """Zeroed anchors float64 [n_streams, fa_segments(T_cap), 2] for an archive batch."""
    import torch
    return torch.zeros((n_streams, fa_segments(ctx, T_cap), 2), dtype=torch.float64, device=device)


def alloc_pages(ctx, n_pages: int):
    """Zeroed pages uint8 [n_pages, qc_page_bytes] of a paged cache, on the context's device."""
    import torch
    return torch.zeros((n_pages, qc_page_bytes(ctx)), dtype=torch.uint8, device=f"cuda:{ctx.device}")


def alloc_attend_workspace(ctx, n_seq: int, n_nodes: int, n_q_heads: int, max_len: int):
    """Workspace for qc_attend calls of up to these sizes."""
    import torch
    return torch.empty(max(16, qc_attend_workspace(ctx, n_seq, n_nodes, n_q_heads, max_len)), dtype=torch.uint8,
                       device=f"cuda:{ctx.device}")
