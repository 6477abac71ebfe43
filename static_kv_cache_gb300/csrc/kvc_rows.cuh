// kvc_rows.cuh -- attention of several new tokens per sequence over the
// sequence's cached rows and over one another: the arguments, and what every
// kernel of it has in common.
//
// A call has, for each sequence b, c = cache_index[b] cached rows and n new
// tokens with K and V rows of their own, in one of two layouts:
//   packed  (kvc_prompt_attn) q [total, H, D], k / v [total, H_kv, D], the
//           tokens of sequence b at rows cu_seqlens[b] ... ; causal
//   dense   (kvc_tree_attn) q [B, H, T, D], k / v [B, H_kv, T, D]; new key s is
//           seen by token t where bit s of t's mask row is set (no mask: s <= t)
// Every token sees all c cached rows.
#pragma once

#include "kvc_internal.cuh"

namespace kvc {

struct RowsArgs {
    const uint8_t *K;            // layer slab [B, H_kv, max_ctx, D], or its pool
    const uint8_t *V;
    const int32_t *block_table;  // paged: [B, max_blocks]; else null
    const void *q, *k_new, *v_new;
    void *out;
    const int32_t *cu_seqlens;   // packed: [B + 1]; else null
    const int32_t *cache_index;  // [B], or null: no cached rows
    const int32_t *n_nodes;      // dense: [B], or null: T each
    const uint32_t *tree_mask;   // dense: [B, T, mask_words], or null: a chain
    int32_t *err;
    int32_t max_blocks, num_blocks;
    int32_t T, total, mask_words;
    int32_t B, H_kv, group, max_ctx;
    float scale_log2;            // log2(e) / sqrt(D)
};

// One sequence of a call.
struct RowsSeq {
    int c, n;       // cached rows, new tokens
    int64_t row0;   // packed: its first row
    bool bad;       // an argument out of range: no output, no read
};

__device__ __forceinline__ RowsSeq rows_seq(const RowsArgs &a, int b) {
    RowsSeq s;
    s.c = a.cache_index ? dev::ld(a.cache_index + b) : 0;
    s.bad = s.c < 0 || s.c > a.max_ctx;
    s.row0 = 0;
    if (a.cu_seqlens) {
        const int lo = dev::ld(a.cu_seqlens + b), hi = dev::ld(a.cu_seqlens + b + 1);
        s.bad = s.bad || lo < 0 || hi < lo || hi > a.total;
        s.row0 = lo;
        s.n = s.bad ? 0 : hi - lo;
    } else {
        s.n = a.n_nodes ? dev::ld(a.n_nodes + b) : a.T;
        s.bad = s.bad || s.n < 0 || s.n > a.T;
        if (s.bad) s.n = 0;
    }
    if (s.bad) s.c = 0;
    return s;
}

// Element offsets of token t, head h (of `heads`) of sequence b in q and out
// (heads = H) or in k_new and v_new (heads = H_kv).
__device__ __forceinline__ int64_t rows_offset(const RowsArgs &a, const RowsSeq &s, int b, int heads, int h, int t, int D) {
    return (a.cu_seqlens ? (s.row0 + t) * heads + h : (int64_t(b) * heads + h) * a.T + t) * D;
}

// What a CTA leaves for the combine when it starts an item that others go on
// with (pieces 0: it does not).
struct RowsCut {
    int pieces;
    int b, kv, t0, ntok;
};

// The tensor-core kernel's arguments (kvc_rows_tc.cuh).
constexpr int ROWS_MAX_CTAS = 160;  // sizes the workspace
// Length of the line of key tiles, at most.  (Places are 32-bit numbers; checked
// in units of 2^20 rounded down per lane, hence the distance from 2^31.)
constexpr int ROWS_MAX_LINE = 2000 << 20;
struct RowsTcArgs : RowsArgs {
    RowsCut *cuts;               // [grid]
    float *part_ml;              // [2 grid][256][2]: (max, sum) of a piece's query rows
    float *part_acc;             // [2 grid][D / 4][256][4]: their unnormalised accumulators
    int32_t item_cost;           // an item's start and end, in key tiles
    int32_t min_share;           // length of a CTA's share of the line, at least
    int32_t split_min;           // items of at most so many key tiles are not cut
    int32_t seg_base;            // tensor-map segment of the layer's first: layer * B * H_kv (paged: layer * num_blocks * H_kv)
    int32_t pool_end;            // paged: one past the map's last segment
    int32_t read_once;           // every (sequence, KV head) is one item: its cached rows are read once
    unsigned long long timeout_ns;
    CUtensorMap tm_k, tm_v;          // the cache: (D, T_max, segments) or the pool: (64, 8, D / 64, 2, H_kv blocks)
    CUtensorMap tm_k_new, tm_v_new;  // new rows: (D, H_kv, total) packed, (D, T, B H_kv) dense
    CUtensorMap tm_q;                // (D, H, total) packed, (D, H, T, B) dense: boxes of 64 columns, g heads, 128 / g tokens
};

struct RowsKernelInfo {
    cudaError_t (*set_max_smem)();
    cudaError_t (*launch)(const RowsTcArgs &a, int grid, int combine_rows, cudaStream_t s);
};
// 16-bit caches with D = 64 or 128
const RowsKernelInfo *rows_kernel_bf16_64();
const RowsKernelInfo *rows_kernel_bf16_128();
const RowsKernelInfo *rows_kernel_f16_64();
const RowsKernelInfo *rows_kernel_f16_128();

inline uint64_t rows_workspace(int D, uint64_t *ml, uint64_t *acc) {
    *ml = align256(ROWS_MAX_CTAS * sizeof(RowsCut));
    *acc = *ml + 2ull * ROWS_MAX_CTAS * 256 * 2 * 4;
    return *acc + 2ull * ROWS_MAX_CTAS * 256 * D * 4;
}

cudaError_t launch_rows_simt(const RowsArgs &a, int dtype, int D, int max_tokens, cudaStream_t s);

// Copies of new rows into the cache (kvc_ingest.cu).
struct IngestArgs {
    uint8_t *K, *V;              // layer slab (or pool) of the first layer
    float *k_scale, *v_scale;    // int8 caches
    const uint8_t *k_new, *v_new;
    const int32_t *block_table;
    const int32_t *cu_seqlens, *cache_index;  // packed append
    const int32_t *path, *n_accept;           // path commit
    int32_t *err;
    int64_t layer_bytes, layer_scales;        // from one layer's slab (scales) to the next
    int32_t n_layers, B, H_kv, max_ctx, max_blocks, num_blocks;
    int32_t total, T, P;
    int32_t row_vecs;            // 16-byte vectors of a row of k_new / v_new
};
cudaError_t launch_append_packed(const IngestArgs &a, bool int8, int num_sms, cudaStream_t s);
cudaError_t launch_tree_commit(const IngestArgs &a, bool int8, cudaStream_t s);

}  // namespace kvc
