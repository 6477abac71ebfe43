// kvc_rows_api.cu -- host side of the calls that take several new tokens per
// sequence: argument checks and launch planning of kvc_prompt_attn,
// kvc_append_packed, kvc_tree_attn and kvc_tree_commit.
#include <cmath>

#include "kvc_handle.cuh"
#include "kvc_rows.cuh"

namespace {

using kvc::device_current;

// What both attentions fill in alike.
kvc::RowsArgs rows_args(const kvc_cache *h, int32_t layer) {
    const kvc_config &c = h->cfg;
    const uint64_t slab = kvc::layer_slab_bytes(h);
    kvc::RowsArgs a{};
    a.K = h->k_base + slab * layer;
    a.V = h->v_base + slab * layer;
    a.block_table = h->block_table;
    a.max_blocks = c.max_context / 16;
    a.num_blocks = h->num_blocks;
    a.err = reinterpret_cast<int32_t *>(h->ws);
    a.B = c.batch;
    a.H_kv = c.n_kv_heads;
    a.group = h->group;
    a.max_ctx = c.max_context;
    a.scale_log2 = float(1.4426950408889634 / std::sqrt(double(c.d_head)));
    return a;
}

// A map of new rows with boxes of 128 rows x 64 columns: (D, H_kv, total) for
// packed rows (the rows are the outermost dimension), (D, T, B * H_kv) for
// dense ones.
bool encode_new_rows(const kvc_cache *h, const kvc::RowsArgs &a, const void *base, CUtensorMap *out) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = kvc::tensor_map_encoder();
    if (!encode) return false;
    const bool packed = a.cu_seqlens != nullptr;
    const cuuint64_t D = cuuint64_t(h->cfg.d_head);
    const cuuint64_t d1 = packed ? a.H_kv : a.T, d2 = packed ? a.total : int64_t(a.B) * a.H_kv;
    const cuuint64_t dims[3] = {D, d1, d2}, strides[2] = {2 * D, 2 * D * d1};
    const cuuint32_t box[3] = {64, packed ? 1u : 128u, packed ? 128u : 1u}, elem[3] = {1, 1, 1};
    return encode(out, h->cfg.dtype == KVC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<void *>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries' map, boxes of 128 / g tokens x g heads x 64 columns: a query
// tile's rows, token after token, in either layout.
bool encode_queries(const kvc_cache *h, const kvc::RowsArgs &a, CUtensorMap *out) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = kvc::tensor_map_encoder();
    if (!encode) return false;
    const bool packed = a.cu_seqlens != nullptr;
    const cuuint64_t D = cuuint64_t(h->cfg.d_head), H = cuuint64_t(h->cfg.n_heads), T = cuuint64_t(a.T);
    const cuuint64_t dims[4] = {D, H, packed ? cuuint64_t(a.total) : T, cuuint64_t(a.B)};
    const cuuint64_t strides[3] = {packed ? 2 * D : 2 * D * T, packed ? 2 * D * H : 2 * D, 2 * D * H * T};
    const cuuint32_t box[4] = {64, cuuint32_t(a.group), cuuint32_t(128 / a.group), 1}, elem[4] = {1, 1, 1, 1};
    return encode(out, h->cfg.dtype == KVC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  packed ? 3 : 4, const_cast<void *>(a.q), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// max_tokens: an upper bound on the new tokens of one sequence, max_cached on
// its cached rows.
kvc_status launch_rows(kvc_cache *h, const kvc::RowsArgs &r, int max_tokens, int max_cached, int32_t layer, void *workspace,
                       void *stream) {
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const kvc_config &c = h->cfg;
    if (!h->rows) {
        const cudaError_t e = kvc::launch_rows_simt(r, c.dtype, c.d_head, max_tokens, s);
        return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
    }
    if (c.max_context > 0x7fffffff - 256) return KVC_ERR_UNSUPPORTED;  // (a tile's last row is a 32-bit number)
    kvc::RowsTcArgs a{};
    static_cast<kvc::RowsArgs &>(a) = r;
    if (!encode_new_rows(h, r, r.k_new, &a.tm_k_new) || !encode_new_rows(h, r, r.v_new, &a.tm_v_new) ||
        !encode_queries(h, r, &a.tm_q))
        return KVC_ERR_CUDA;
    a.tm_k = h->rows_k;
    a.tm_v = h->rows_v;
    a.seg_base = layer * (h->block_table ? h->num_blocks : c.batch) * c.n_kv_heads;
    a.pool_end = c.n_layers * h->num_blocks * c.n_kv_heads;
    a.timeout_ns = kvc::WAIT_TIMEOUT_NS;
    uint64_t ml, acc;
    kvc::rows_workspace(c.d_head, &ml, &acc);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.cuts = reinterpret_cast<kvc::RowsCut *>(ws);
    a.part_ml = reinterpret_cast<float *>(ws + ml);
    a.part_acc = reinterpret_cast<float *>(ws + acc);
    // at most so many key tiles of one item, and length of the whole line (these
    // size the launch; what fits the line's limit is seen on the device, from the
    // sequences' own lengths)
    const int ti = 2 * (128 / h->group);
    const int64_t item = (max_cached + 127) / 128 + (int64_t(max_tokens) + 127) / 128;
    const int64_t blocks = r.cu_seqlens ? r.total / ti + (c.batch < r.total ? c.batch : r.total)
                                        : int64_t(c.batch) * ((int64_t(r.T) + ti - 1) / ti);
    a.read_once = !r.cu_seqlens && r.T <= ti;
    // An item's start and end take about as long as three key tiles.  (Prompts over
    // prefixes at 2, 3, 4 tiles: 231, 226, 222 us; short prompts 24.4, 23.8, 24.6; tree
    // steps on pages 67.4, 67.5, 68.2)
    a.item_cost = 3;
    // Where no item passes 8 key tiles none is cut: it would take about as long as its
    // pieces' combine.  Otherwise those past 4 are (past 8: prompts over prefixes 230
    // instead of 226 us).
    constexpr int SHORT = 8;
    a.min_share = 4;
    a.split_min = item > SHORT ? 4 : 0x7fffffff;  // (nothing is cut where no combine follows)
    const int64_t line = blocks * c.n_kv_heads * (item + a.item_cost);
    int64_t grid = h->num_sms < kvc::ROWS_MAX_CTAS ? h->num_sms : kvc::ROWS_MAX_CTAS;
    if ((line + a.min_share - 1) / a.min_share < grid) grid = (line + a.min_share - 1) / a.min_share;
    // the query tiles an item can fill
    const int rows = max_tokens >= ti ? 256 : max_tokens > ti / 2 ? 128 + (max_tokens - ti / 2) * h->group : max_tokens * h->group;
    const cudaError_t e = h->rows->launch(a, int(grid), item > SHORT ? rows : 0, s);
    return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

kvc::IngestArgs ingest_args(const kvc_cache *h, int32_t layer, const void *k, const void *v) {
    const kvc_config &c = h->cfg;
    const uint64_t slab = kvc::layer_slab_bytes(h);
    kvc::IngestArgs a{};
    a.K = h->k_base + slab * layer;
    a.V = h->v_base + slab * layer;
    a.layer_bytes = int64_t(slab);
    if (h->k_scale) {
        const uint64_t ss = kvc::layer_scale_bytes(h);
        a.k_scale = reinterpret_cast<float *>(h->k_scale + ss * layer);
        a.v_scale = reinterpret_cast<float *>(h->v_scale + ss * layer);
        a.layer_scales = int64_t(ss / 4);
    }
    a.k_new = static_cast<const uint8_t *>(k);
    a.v_new = static_cast<const uint8_t *>(v);
    a.block_table = h->block_table;
    a.max_blocks = c.max_context / 16;
    a.num_blocks = h->num_blocks;
    a.err = reinterpret_cast<int32_t *>(h->ws);
    a.B = c.batch;
    a.H_kv = c.n_kv_heads;
    a.max_ctx = c.max_context;
    a.row_vecs = c.d_head * (c.dtype == KVC_INT8 ? 2 : h->elem_bytes) / 16;
    return a;
}

}  // namespace

extern "C" {

uint64_t kvc_rows_workspace_bytes(const kvc_config *cfg) {
    if (kvc_workspace_bytes(cfg) == 0) return 0;
    // (the kernel on the CUDA cores splits nothing)
    if ((cfg->dtype != KVC_BF16 && cfg->dtype != KVC_FP16) || (cfg->d_head != 64 && cfg->d_head != 128)) return 256;
    uint64_t ml, acc;
    return kvc::rows_workspace(cfg->d_head, &ml, &acc);
}

kvc_status kvc_prompt_attn(kvc_cache *h, int32_t layer, const void *q, const void *k, const void *v,
                           const int32_t *cu_seqlens, const int32_t *cache_index, int32_t total,
                           void *workspace, uint64_t ws_bytes, void *out, void *stream) {
    if (!h || layer < 0 || layer >= h->cfg.n_layers || total < 0) return KVC_ERR_INVALID;
    if (h->cfg.dtype == KVC_INT8) return KVC_ERR_UNSUPPORTED;
    if (total == 0) return KVC_OK;
    if (!q || !k || !v || !cu_seqlens || !out || !device_current(h)) return KVC_ERR_INVALID;
    if (!kvc::aligned16(q) || !kvc::aligned16(k) || !kvc::aligned16(v) || !kvc::aligned16(out)) return KVC_ERR_ALIGNMENT;
    if (!workspace || ws_bytes < kvc_rows_workspace_bytes(&h->cfg)) return KVC_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KVC_ERR_ALIGNMENT;
    kvc::RowsArgs a = rows_args(h, layer);
    a.q = q;
    a.k_new = k;
    a.v_new = v;
    a.out = out;
    a.cu_seqlens = cu_seqlens;
    a.cache_index = cache_index;
    a.total = total;
    return launch_rows(h, a, total, cache_index ? h->cfg.max_context : 0, layer, workspace, stream);
}

kvc_status kvc_append_packed(kvc_cache *h, int32_t layer, const void *k, const void *v,
                             const int32_t *cu_seqlens, const int32_t *cache_index, int32_t total,
                             void *stream) {
    if (!h || layer < 0 || layer >= h->cfg.n_layers || total < 0) return KVC_ERR_INVALID;
    if (total == 0) return KVC_OK;
    if (!k || !v || !cu_seqlens || !device_current(h)) return KVC_ERR_INVALID;
    if (!kvc::aligned16(k) || !kvc::aligned16(v)) return KVC_ERR_ALIGNMENT;
    kvc::IngestArgs a = ingest_args(h, layer, k, v);
    a.cu_seqlens = cu_seqlens;
    a.cache_index = cache_index;
    a.total = total;
    const cudaError_t e = kvc::launch_append_packed(a, h->cfg.dtype == KVC_INT8, h->num_sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

kvc_status kvc_tree_attn(kvc_cache *h, int32_t layer, const void *q, const void *k_new, const void *v_new,
                         const int32_t *cache_index, const int32_t *n_nodes, const uint32_t *tree_mask, int32_t T,
                         int32_t max_index_hint, void *workspace, uint64_t ws_bytes, void *out, void *stream) {
    if (!h || layer < 0 || layer >= h->cfg.n_layers || T < 1 || max_index_hint < 0 || max_index_hint > h->cfg.max_context)
        return KVC_ERR_INVALID;
    if (h->cfg.dtype == KVC_INT8) return KVC_ERR_UNSUPPORTED;
    if (!q || !k_new || !v_new || !cache_index || !out || !device_current(h)) return KVC_ERR_INVALID;
    if (!kvc::aligned16(q) || !kvc::aligned16(k_new) || !kvc::aligned16(v_new) || !kvc::aligned16(out)) return KVC_ERR_ALIGNMENT;
    if (!workspace || ws_bytes < kvc_rows_workspace_bytes(&h->cfg)) return KVC_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KVC_ERR_ALIGNMENT;
    kvc::RowsArgs a = rows_args(h, layer);
    a.q = q;
    a.k_new = k_new;
    a.v_new = v_new;
    a.out = out;
    a.cache_index = cache_index;
    a.n_nodes = n_nodes;
    a.tree_mask = tree_mask;
    a.T = T;
    a.mask_words = int((int64_t(T) + 31) / 32);
    return launch_rows(h, a, T, max_index_hint ? max_index_hint : h->cfg.max_context, layer, workspace, stream);
}

kvc_status kvc_tree_commit(kvc_cache *h, int32_t layer, int32_t n_layers, const void *k_new, const void *v_new,
                           const int32_t *cache_index, const int32_t *path, const int32_t *n_accept, int32_t T,
                           int32_t P, void *stream) {
    if (!h || layer < 0 || n_layers < 1 || n_layers > h->cfg.n_layers - layer || T < 1 || P < 1) return KVC_ERR_INVALID;
    if (!k_new || !v_new || !cache_index || !path || !n_accept || !device_current(h)) return KVC_ERR_INVALID;
    if (!kvc::aligned16(k_new) || !kvc::aligned16(v_new)) return KVC_ERR_ALIGNMENT;
    kvc::IngestArgs a = ingest_args(h, layer, k_new, v_new);
    a.cache_index = cache_index;
    a.path = path;
    a.n_accept = n_accept;
    a.n_layers = n_layers;
    a.T = T;
    a.P = P;
    const cudaError_t e = kvc::launch_tree_commit(a, h->cfg.dtype == KVC_INT8, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

}  // extern "C"
