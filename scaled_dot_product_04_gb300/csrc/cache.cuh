// Parameters and launchers of the paged key/value cache operators (cache.cu)
// and of the attention that reads the cache (tree.cu).
#pragma once
#include "common.cuh"

namespace sdpa {

// Device-side findings about the caller's tables, recorded in the error word
// like an expired wait, with this bit set in the site: the kernels skip what
// they point at (or read it as zeros) and sdpa_check_device_error reports
// SDPA_ERR_INVALID_ARG.
constexpr uint32_t kSiteBadData = 0x8000u;

// Request lengths -> pages, slots, positions and tree masks (sdpa_cache_plan).
struct PlanParams {
    const int32_t *ctx, *fresh;      // [b] cached tokens, new tokens (< 0: finished)
    const int32_t *parents;          // [max_new] or null
    const int32_t *held_in;          // [b] pages a request holds
    const int32_t *ring_in;          // {first free entry, number of free entries, -}
    int32_t *free_ring;              // [num_pages]
    int32_t *table;                  // [b, max_blocks]
    int32_t *held_out, *ring_out;    // [b], [3]
    int32_t *cu_new;                 // [b + 1]
    int32_t *kv_lens;                // [b]
    int32_t *slots, *positions;      // [max_new]
    uint32_t *mask;                  // [max_new, mask_words] or null
    int b, max_blocks, page_size, num_pages, max_new, mask_words;
};
cudaError_t launch_cache_plan(const PlanParams &p, int sm_count, cudaStream_t stream);

// New keys and values to their slots (sdpa_cache_append).
struct AppendParams {
    const void *k, *v;               // [total, h_kv, d], token strides below
    void *k_cache, *v_cache;         // [num_pages, h_kv, page_size, d]
    const int32_t *slots;            // [total], < 0: skip
    const float *scale_k, *scale_v;  // E4M3 cache only
    uint32_t *err;
    int64_t k_stride, v_stride;      // elements between tokens
    int total, h_kv, d, num_pages, page_size;
};
cudaError_t launch_cache_append(const AppendParams &p, int dtype, int cache_dtype, cudaStream_t stream);

// The accepted path of a verified tree, moved to the tree's front
// (sdpa_cache_accept).
struct AcceptParams {
    void *k_cache, *v_cache;
    const int32_t *table;            // [b, max_blocks]
    const int32_t *ctx, *fresh;      // [b]
    const int32_t *path;             // [b, max_path]
    const int32_t *path_lens;        // [b]
    int32_t *ctx_out;                // [b]
    uint32_t *err;
    int b, max_blocks, max_path, h_kv, row_bytes, num_pages, page_size;
};
constexpr int kAcceptThreads = 128;  // a 16-byte column each, of a row of the two caches
constexpr int64_t kAcceptMaxColumns = 65535ll * kAcceptThreads;  // the CTAs of a grid's y
cudaError_t launch_cache_accept(const AcceptParams &p, cudaStream_t stream);

// Attention of new tokens over the cache (sdpa_tree_fwd).
struct TreeParams {
    const void *q;                   // [total_q, h, d], q_stride elements between tokens
    const void *k_cache, *v_cache;
    void *o;                         // [total_q, h, d]
    float *lse;                      // [total_q, h] or null
    const int32_t *table, *cu_q, *kv_lens;
    const uint32_t *mask;            // [total_q, mask_words] or null: a chain
    const float *descale_k, *descale_v;  // E4M3 cache only
    uint32_t *err;
    char *workspace;
    int64_t q_stride;
    int num_seqs, total_q, max_kv, max_blocks, num_pages, page_size, mask_words;
    int h, h_kv, group, d;
    float scale_log2;                // attn_scale * log2(e)
    int chain_tokens;                // tokens of a chain's rows: tree_q_tokens
    int page_shift;                  // log2 of page_size, -1 if that is no power of two
};
constexpr int kTreeMaxCtas = 152;    // grid bound that the workspace is sized for
size_t tree_workspace_bytes(int max_q, int group, int d);
// bound of the places of the launch's list of key tiles: must fit 31 bits
int64_t tree_places(int max_q, int total_q, int num_seqs, int h_kv, int group, int max_kv);
int tree_q_tokens(int max_q, int group);  // tokens of a Q box
// tq: 3-D map over [total_q][h][d], boxes of tree_q_tokens tokens x (h / h_kv) heads (16-bit caches);
// tk, tv: 3-D maps over [num_pages * h_kv][page_size][d], boxes of min(page_size, 128) rows.
cudaError_t launch_tree_fwd(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const TreeParams &p, int max_q, int dtype, int cache_dtype, int sm_count,
                            cudaStream_t stream, const KernelTimer &timer);

}  // namespace sdpa
