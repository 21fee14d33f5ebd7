// fd_block.cu -- fd_decode_quant_block and fd_decode_quant_block_paged:
// attention over an 8-bit cache with one scale per block of tokens and kv
// head. The split kernel with QuantConsumer in its kBlock form (fd_quant.cuh).
//
// What bounds it: the cache's codes, 2 D bytes per (token, kv head) plus
// 8 / T bytes of scales, each read once. One sequence of 16384 E4M3 tokens, 32
// heads (134 MB): 27.3 us, 4.9 TB/s; 131072 int8 tokens, 64 / 8 heads (269 MB):
// 52 us in short bursts (5.1 TB/s), 56.5 us sustained, where the consumers'
// arithmetic takes over from memory; 32 uneven sequences in 64-token pages
// (268 MB): 58 to 61 us, 12 of them waiting for the block that holds the most short
// rows.
#include "fd_host.cuh"
#include "fd_quant.cuh"

namespace fdh {

int take_block_error(int *word) { return take_error_word(fd::g_fd_error_word, word); }

namespace {

// Columns to the consumer's shape as for one scale per kv head: up to 8
// columns four groups of two warps, 32 tokens per warp; 16 columns two groups
// of four.
template <bool kE4M3, bool kPaged>
int launch_block(int D, const CUtensorMap &tk, const CUtensorMap &tv, const fd::SplitParams &p, cudaStream_t st,
                 const CUtensorMap *rk, const CUtensorMap *rv) {
    if (D == 128) {
        if (p.cols <= 8)
            return launch_split_t<128, fd::QuantConsumer<128, 1, kE4M3, 32, true, kPaged>, true, kPaged>(tk, tv, p, st,
                                                                                                      rk, rv);
        return launch_split_t<128, fd::QuantConsumer<128, 2, kE4M3, 16, true, kPaged>, true, kPaged>(tk, tv, p, st, rk,
                                                                                                  rv);
    }
    if (p.cols <= 8)
        return launch_split_t<64, fd::QuantConsumer<64, 1, kE4M3, 32, true, kPaged>, true, kPaged>(tk, tv, p, st, rk,
                                                                                                rv);
    return launch_split_t<64, fd::QuantConsumer<64, 2, kE4M3, 16, true, kPaged>, true, kPaged>(tk, tv, p, st, rk, rv);
}

int run_block(const Problem &pr, int q_len, int kv_type, int block_tokens, const float *k_scale, const float *v_scale,
              const PagedLayout *pl) {
    int sms;
    int rc = device_sms(&sms);
    if (rc != FD_OK) return rc;
    fd::SplitParams p = split_params(pr, q_len, pl);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    while ((1 << p.blk_shift) < block_tokens) ++p.blk_shift;
    p.blocks = static_cast<int>(((pl ? pl->page_size : pr.max_len) + block_tokens - 1LL) / block_tokens);
    CUtensorMap tk, tv, rk, rv;
    std::memset(&tk, 0, sizeof tk);
    std::memset(&tv, 0, sizeof tv);
    if (!pl) {
        if (pr.max_len > 0) {
            const long long rows = static_cast<long long>(pr.B) * pr.Hkv;
            if ((rc = encode_cache_map(&tk, pr.k, pr.D, pr.max_len, rows, true)) != FD_OK) return rc;
            if ((rc = encode_cache_map(&tv, pr.v, pr.D, pr.max_len, rows, true)) != FD_OK) return rc;
        }
        return kv_type == FD_KV_E4M3 ? launch_block<true, false>(pr.D, tk, tv, p, pr.stream, nullptr, nullptr)
                                     : launch_block<false, false>(pr.D, tk, tv, p, pr.stream, nullptr, nullptr);
    }
    if ((rc = encode_paged_map(&tk, pr.k, pr.D, pl->page_size, pr.Hkv, pl->num_pages, pl->nhd, true)) != FD_OK)
        return rc;
    if ((rc = encode_paged_map(&tv, pr.v, pr.D, pl->page_size, pr.Hkv, pl->num_pages, pl->nhd, true)) != FD_OK)
        return rc;
    // small pages: maps of runs of consecutive pages (one box per such tile)
    const bool small = pl->page_size < fd::kTileTokens && pl->num_pages >= fd::kTileTokens / pl->page_size;
    if (small) {
        if ((rc = encode_paged_run_map(&rk, pr.k, pr.D, pl->page_size, pr.Hkv, pl->num_pages, pl->nhd, true)) != FD_OK)
            return rc;
        if ((rc = encode_paged_run_map(&rv, pr.v, pr.D, pl->page_size, pr.Hkv, pl->num_pages, pl->nhd, true)) != FD_OK)
            return rc;
    }
    const CUtensorMap *rkp = small ? &rk : nullptr, *rvp = small ? &rv : nullptr;
    return kv_type == FD_KV_E4M3 ? launch_block<true, true>(pr.D, tk, tv, p, pr.stream, rkp, rvp)
                                 : launch_block<false, true>(pr.D, tk, tv, p, pr.stream, rkp, rvp);
}

// Argument checks (no CUDA call) and the plan, for both forms.
int decode_block(int B, int q_len, int Hq, int Hkv, int D, int max_len, int block_tokens, int kv_type,
                 const uint16_t *q, const uint8_t *k, const uint8_t *v, const float *k_scale, const float *v_scale,
                 const int32_t *seqlens, float scale, float *out, float *lse, void *workspace, size_t workspace_bytes,
                 int num_splits, void *stream, const PagedLayout *pl) {
    if (q_len < 1 || q_len > FD_MAX_GROUP) return FD_ERR_SHAPE;
    if (kv_type != FD_KV_E4M3 && kv_type != FD_KV_INT8) return FD_ERR_SHAPE;
    if (!valid_block(block_tokens) || (pl && block_tokens > pl->page_size)) return FD_ERR_SHAPE;
    int rc = check_shape(B, Hq, Hkv, D, max_len);
    if (rc != FD_OK) return rc;
    if (static_cast<long long>(Hq) * q_len / Hkv > FD_MAX_GROUP) return FD_ERR_GROUP;
    if (num_splits < 0) return FD_ERR_SPLITS;
    if (pl || max_len > 0) {
        if (!k_scale || !v_scale) return FD_ERR_NULL_POINTER;
        if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return FD_ERR_ALIGNMENT;
    }
    if (pl) {
        if (!pl->block_table) return FD_ERR_NULL_POINTER;
        if (!aligned(pl->block_table, 16)) return FD_ERR_ALIGNMENT;
        // the flattened page coordinate (page * Hkv or page * page_size) must fit in int32
        if (static_cast<long long>(pl->num_pages) * (Hkv > pl->page_size ? Hkv : pl->page_size) > 0x7fffffffLL)
            return FD_ERR_SHAPE;
    }
    // the checks and the workspace see the (query, head) columns as Hq * q_len heads
    Problem pr = make_problem(B, Hq * q_len, Hkv, D, max_len, q, reinterpret_cast<const uint16_t *>(k),
                              reinterpret_cast<const uint16_t *>(v), seqlens, scale, out, lse, workspace,
                              workspace_bytes, num_splits == 0 ? 1 : num_splits, stream);
    if ((rc = check_problem(pr, true)) != FD_OK) return rc;
    if (num_splits == 0) {
        const int S = fd_plan(B, Hq, Hkv, D, max_len);
        if (S < 0) return S;
        pr.num_splits = S;
        if ((rc = check_problem(pr, true)) != FD_OK) return rc;
    }
    pr.Hq = Hq;
    return run_block(pr, q_len, kv_type, block_tokens, k_scale, v_scale, pl);
}

}  // namespace
}  // namespace fdh

extern "C" {

int fd_decode_quant_block(int B, int q_len, int Hq, int Hkv, int D, int max_len, int block_tokens, int kv_type,
                          const uint16_t *q, const uint8_t *k_codes, const uint8_t *v_codes, const float *k_scale,
                          const float *v_scale, const int32_t *seqlens, float scale, float *out, float *lse,
                          void *workspace, size_t workspace_bytes, int num_splits, void *stream) {
    return fdh::decode_block(B, q_len, Hq, Hkv, D, max_len, block_tokens, kv_type, q, k_codes, v_codes, k_scale, v_scale,
                             seqlens, scale, out, lse, workspace, workspace_bytes, num_splits, stream, nullptr);
}

int fd_decode_quant_block_paged(int B, int q_len, int Hq, int Hkv, int D, int page_size, int num_pages,
                                int max_pages_per_seq, int kv_layout, int block_tokens, int kv_type, const uint16_t *q,
                                const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scale,
                                const float *v_scale, const int32_t *block_table, const int32_t *seqlens, float scale,
                                float *out, float *lse, void *workspace, size_t workspace_bytes, int num_splits,
                                void *stream) {
    long long max_len = 0;
    const int rc = fdh::check_paged(page_size, num_pages, max_pages_per_seq, kv_layout, &max_len);
    if (rc != FD_OK) return rc;
    const fdh::PagedLayout pl{block_table, page_size, num_pages, max_pages_per_seq, kv_layout == FD_KV_NHD};
    return fdh::decode_block(B, q_len, Hq, Hkv, D, static_cast<int>(max_len), block_tokens, kv_type, q, k_pages, v_pages,
                             k_scale, v_scale, seqlens, scale, out, lse, workspace, workspace_bytes, num_splits, stream,
                             &pl);
}

}  // extern "C"
