// kvc_e4m3_api.cu -- host side of the 8-bit paged cache and of the rotated append:
// argument checks and launches of kvc_alloc_paged_scaled, kvc_append_rope and
// kvc_packed_attn, and of the older calls on a KVC_E4M3 handle.
#include <cmath>
#include <new>

#include "kvc_e4m3.cuh"
#include "kvc_handle.cuh"

namespace {

using kvc::aligned16;
using kvc::device_current;

int row_bytes_of(const kvc_cache *h) { return h->row_dtype == KVC_FP32 ? 4 : 2; }

bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a_bytes > 0 && b_bytes > 0 && (x < y ? y - x < uintptr_t(a_bytes) : x - y < uintptr_t(b_bytes));
}

// What every append fills in alike.
kvc::RopeArgs rope_args(const kvc_cache *h, int32_t layer) {
    const kvc_config &c = h->cfg;
    const uint64_t slab = kvc::layer_slab_bytes(h);
    kvc::RopeArgs a{};
    a.K = h->k_base + slab * layer;
    a.V = h->v_base + slab * layer;
    if (h->k_scale) {
        const uint64_t ss = kvc::layer_scale_bytes(h);
        a.k_scale = reinterpret_cast<float *>(h->k_scale + ss * layer);
        a.v_scale = reinterpret_cast<float *>(h->v_scale + ss * layer);
    }
    a.block_table = h->block_table;
    a.max_blocks = c.max_context / 16;
    a.num_blocks = h->num_blocks;
    a.err = reinterpret_cast<int32_t *>(h->ws);
    a.B = c.batch;
    a.H = c.n_heads;
    a.H_kv = c.n_kv_heads;
    a.D = c.d_head;
    a.max_ctx = c.max_context;
    a.kv_head = int64_t(c.d_head) * row_bytes_of(h);
    a.k_token = a.v_token = a.kv_head * c.n_kv_heads;
    a.T = 1;
    return a;
}

kvc_status launch(const kvc_cache *h, const kvc::RopeArgs &a, void *stream) {
    const cudaError_t e = kvc::launch_rope(a, h->row_dtype, h->cfg.dtype, h->num_sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

// Boxes of 1, 2, 4 and 8 KV heads of a block (those that the cache has), 16 rows
// of 128 bytes each, 128-byte swizzle.
bool encode_pools(kvc_cache *h) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = kvc::tensor_map_encoder();
    if (!encode) return false;
    const kvc_config &c = h->cfg;
    const cuuint64_t D = kvc::E4M3_D, G = cuuint64_t(c.n_kv_heads);
    const cuuint64_t dims[4] = {D, 16, G, cuuint64_t(c.n_layers) * h->num_blocks}, strides[3] = {D, 16 * D, 16 * D * G};
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4 && (1u << i) <= G; ++i) {
        const cuuint32_t box[4] = {cuuint32_t(D), 16, 1u << i, 1};
        for (int v = 0; v < 2; ++v)
            if (encode(v ? &h->pool_v[i] : &h->pool_k[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, v ? h->v_base : h->k_base, dims, strides, box, elem,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return false;
    }
    return true;
}

// What an attention call refuses, looked at before anything is enqueued.
kvc_status refusal(const kvc_cache *h, const void *q, const void *out, int32_t total) {
    if (!device_current(h)) return KVC_ERR_INVALID;
    if (!aligned16(q) || !aligned16(out)) return KVC_ERR_ALIGNMENT;  // (pieces are joined 8 bytes at a time)
    const int64_t rows = int64_t(total) * h->cfg.n_heads;
    if (rows > 0x7fffffff) return KVC_ERR_UNSUPPORTED;
    // (a row's pieces are several CTAs', which read its queries)
    const int64_t bytes = rows * kvc::E4M3_D * row_bytes_of(h);
    return overlap(q, bytes, out, bytes) ? KVC_ERR_INVALID : KVC_OK;
}

kvc_status attend(const kvc_cache *h, int32_t layer, const void *q, const int32_t *cu_seqlens, const int32_t *cache_index,
                  int index_offset, int32_t total, int32_t hint, void *out, void *stream) {
    const kvc_config &c = h->cfg;
    const uint64_t slab = kvc::layer_slab_bytes(h), ss = kvc::layer_scale_bytes(h);
    kvc::E4m3TcArgs a{};
    a.K = h->k_base + slab * layer;
    a.V = h->v_base + slab * layer;
    a.k_scale = reinterpret_cast<const float *>(h->k_scale + ss * layer);
    a.v_scale = reinterpret_cast<const float *>(h->v_scale + ss * layer);
    a.block_table = h->block_table;
    a.q = q;
    a.out = out;
    a.cu_seqlens = cu_seqlens;
    a.cache_index = cache_index;
    a.index_offset = index_offset;
    a.total = total;
    a.bf16 = h->row_dtype == KVC_BF16;
    a.err = reinterpret_cast<int32_t *>(h->ws);
    a.B = c.batch;
    a.H = c.n_heads;
    a.H_kv = c.n_kv_heads;
    a.group = h->group;
    a.max_ctx = c.max_context;
    a.max_blocks = c.max_context / 16;
    a.num_blocks = h->num_blocks;
    a.scale_log2 = float(1.4426950408889634 / std::sqrt(double(c.d_head)));
    const kvc::E4m3Workspace w = kvc::e4m3_workspace();
    a.tickets = reinterpret_cast<int32_t *>(h->ws + w.tickets);
    a.part_ml = reinterpret_cast<float2 *>(h->ws + w.part_ml);
    a.part_acc = reinterpret_cast<float *>(h->ws + w.part_acc);
    a.layer_block = layer * h->num_blocks;
    a.timeout_ns = h->flag_timeout_ns;
    // Query rows of a tile: those of the tokens that a sequence has on average, up to 64.
    const int64_t tokens = cu_seqlens ? (int64_t(total) + c.batch - 1) / c.batch : 1;
    int rows = 1;
    while (rows < 64 && rows < tokens * h->group) rows *= 2;
    // Where they are more than 64, the kernel that has query rows on M: it does 256 of
    // them in the time that the other one takes for 80 (16 sequences of 2,048 rows, 32
    // heads over 8, with 16, 24, 64, 128 tokens: 48, 79, 143, 269 us with the other one,
    // 54, 57, 69, 109 with it) -- if there is a segment for six SMs at least: the pieces of
    // fewer are joined in longer than that (8 sequences of 8 tokens over 4,096 rows, 32
    // heads on one: 32 us with the other one, 46 with it).  The average is over the batch's
    // slots, as the lengths are on the device: idle slots, and single tokens beside one
    // long chunk, lower it for the chunk.
    const int g = h->group, pair_tokens = g <= 128 ? 2 * (128 / g) : 0;
    const int64_t seqs = c.batch < total ? c.batch : total;
    const bool many = tokens > 1 && tokens * g > 64 && pair_tokens && (total / pair_tokens + seqs) * c.n_kv_heads * 6 >= h->num_sms;
    // KV heads of a tile: the more, the larger the copies (32 KB of 8 or 4 heads take the
    // time of their bytes, of 2 heads 0.83 us an SM, of one 0.8), but the fewer segments to
    // cut: at least one for five SMs, or their ends, each joined by one CTA, are what the
    // call waits for (16 sequences of 1,024 - 8,192 rows, 8 heads: 40 us with 8 heads a
    // tile, 33.2 with 4, 33.5 with 2, 38 with 1; 4 sequences of 64 heads: 229, 231, 253).
    int nh = 8, map = 3;
    const int64_t row_tiles = cu_seqlens ? (int64_t(total) * h->group + rows - 1) / rows + seqs : seqs;
    while (many ? nh > 1 : (nh > 1 && nh * rows > 32) || c.n_kv_heads % nh || (nh > 1 && row_tiles * (c.n_kv_heads / nh) * 5 < h->num_sms)) nh /= 2, --map;
    a.nh = nh;
    a.gt = (g + rows - 1) / rows;
    a.tt = a.gt > 1 ? 1 : rows / g;
    a.gg = (g + a.gt - 1) / a.gt;
    if (many) a.gt = 1, a.gg = g, a.tt = pair_tokens;
    a.gg_inverse = (65536 + a.gg - 1) / a.gg;
    // A segment's start and end count as four tiles.  (32 heads on one KV head at 2, 4, 8:
    // 23.7, 22.3, 22.0 us; drafts 31.3, 29.7, 29.2; with query rows on M, at 2, 3, 4, 6:
    // prompt chunks 84, 87, 87, 86, a prompt of 4,096 tokens 204, 186, 183, 183.)
    a.cost = 4;
    a.groups = c.n_kv_heads / nh;
    a.shift = 7 - map;
    a.tm_k = h->pool_k[map];
    a.tm_v = h->pool_v[map];
    a.read_once = tokens * h->group <= rows;
    a.min_share = 1;
    int grid = h->num_splits ? h->num_splits : h->num_sms;
    if (grid > kvc::E4M3_MAX_CTAS) grid = kvc::E4M3_MAX_CTAS;
    const int64_t tiles = row_tiles * (c.n_kv_heads / nh) * ((int64_t(hint ? hint : c.max_context) * nh + 127) / 128);
    if (tiles < grid) grid = int(tiles);
    const cudaError_t e = many ? kvc::launch_e4m3_rows(a, grid, static_cast<cudaStream_t>(stream)) : kvc::launch_e4m3_attn(a, rows, grid, h->max_smem, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

}  // namespace

// The calls of kvc_api.cu on a KVC_E4M3 handle (arguments checked there).
kvc_status kvc::e4m3_append(const kvc_cache *h, int32_t layer, const void *k_new, const void *v_new, const int32_t *cache_index,
                            int index_offset, int32_t T_new, void *stream) {
    const kvc_config &c = h->cfg;
    if (!device_current(h)) return KVC_ERR_INVALID;
    if (int64_t(c.batch) * T_new > 0x7fffffff) return KVC_ERR_UNSUPPORTED;
    kvc::RopeArgs a = rope_args(h, layer);
    a.k = static_cast<const uint8_t *>(k_new);
    a.v = static_cast<const uint8_t *>(v_new);
    a.cache_index = cache_index;
    a.index_offset = index_offset;
    a.T = T_new;
    a.total = c.batch * T_new;
    a.k_token = a.v_token = int64_t(c.d_head) * row_bytes_of(h);
    a.kv_head = a.k_token * T_new;
    a.kv_seq = a.kv_head * c.n_kv_heads;
    return launch(h, a, stream);
}

kvc_status kvc::e4m3_append_packed(const kvc_cache *h, int32_t layer, const void *k, const void *v, const int32_t *cu_seqlens,
                                   const int32_t *cache_index, int32_t total, void *stream) {
    kvc::RopeArgs a = rope_args(h, layer);
    a.k = static_cast<const uint8_t *>(k);
    a.v = static_cast<const uint8_t *>(v);
    a.cu_seqlens = cu_seqlens;
    a.cache_index = cache_index;
    a.total = total;
    return launch(h, a, stream);
}

kvc_status kvc::e4m3_decode(const kvc_cache *h, int32_t layer, const void *q, const int32_t *valid_len, int32_t max_valid_hint,
                            void *out, void *stream) {
    const kvc_status st = refusal(h, q, out, h->cfg.batch);
    return st != KVC_OK ? st : attend(h, layer, q, nullptr, valid_len, -1, h->cfg.batch, max_valid_hint, out, stream);
}

kvc_status kvc::e4m3_step(const kvc_cache *h, int32_t layer, const void *q, const void *k_new, const void *v_new,
                          const int32_t *valid_len, int32_t max_valid_hint, void *out, void *stream) {
    kvc_status st = refusal(h, q, out, h->cfg.batch);
    if (st == KVC_OK) st = e4m3_append(h, layer, k_new, v_new, valid_len, -1, 1, stream);
    return st != KVC_OK ? st : attend(h, layer, q, nullptr, valid_len, -1, h->cfg.batch, max_valid_hint, out, stream);
}

extern "C" {

uint64_t kvc_pool_scale_bytes(const kvc_config *cfg, int32_t num_blocks) {
    if (!cfg || cfg->dtype != KVC_E4M3 || kvc_pool_bytes(cfg, num_blocks) == 0) return 0;
    return uint64_t(cfg->n_layers) * uint64_t(num_blocks) * uint64_t(cfg->n_kv_heads) * 4;
}

kvc_status kvc_alloc_paged_scaled(const kvc_config *cfg, void *k_pool, void *v_pool, void *k_scale, void *v_scale,
                                  int32_t num_blocks, const int32_t *block_table, int32_t row_dtype, void *workspace,
                                  uint64_t ws_bytes, kvc_cache **out) {
    if (!out || !cfg || cfg->dtype != KVC_E4M3 || !k_pool || !v_pool || !k_scale || !v_scale || !block_table || num_blocks <= 0)
        return KVC_ERR_INVALID;
    if (row_dtype != KVC_BF16 && row_dtype != KVC_FP16) return KVC_ERR_INVALID;
    const kvc_status st = kvc_check_config(cfg);
    if (st != KVC_OK) return st;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_scale) || !aligned16(v_scale) || !aligned16(block_table) ||
        (workspace && !aligned16(workspace)))
        return KVC_ERR_ALIGNMENT;
    const uint64_t need = kvc_workspace_bytes(cfg);
    if (!workspace || ws_bytes < need) return KVC_ERR_WORKSPACE;
    int dev = 0, sms = 0, smem = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
        return KVC_ERR_CUDA;
    if (int64_t(cfg->n_layers) * num_blocks > 0x7fffffff) return KVC_ERR_UNSUPPORTED;  // (places in the tensor maps)
    if (kvc::e4m3_set_max_smem(smem) != cudaSuccess || kvc::e4m3_rows_set_max_smem() != cudaSuccess) return KVC_ERR_CUDA;
    if (cudaMemsetAsync(workspace, 0, need, 0) != cudaSuccess || cudaStreamSynchronize(0) != cudaSuccess) return KVC_ERR_CUDA;
    kvc_cache *h = new (std::nothrow) kvc_cache{};
    if (!h) return KVC_ERR_INVALID;
    h->cfg = *cfg;
    h->device = dev;
    h->num_sms = sms;
    h->max_smem = smem;
    h->elem_bytes = 1;
    h->row_dtype = row_dtype;
    h->group = cfg->n_heads / cfg->n_kv_heads;
    h->flag_timeout_ns = kvc::WAIT_TIMEOUT_NS;
    h->k_base = static_cast<uint8_t *>(k_pool);
    h->v_base = static_cast<uint8_t *>(v_pool);
    h->k_scale = static_cast<uint8_t *>(k_scale);
    h->v_scale = static_cast<uint8_t *>(v_scale);
    h->block_table = block_table;
    h->num_blocks = num_blocks;
    h->kv_pair = 1;
    h->ws = static_cast<uint8_t *>(workspace);
    h->ws_bytes = ws_bytes;
    const kvc::E4m3Workspace w = kvc::e4m3_workspace();
    h->wl.tickets = w.tickets;  // (what kvc_get_error clears after a time-out)
    h->wl.part_ml = w.part_ml;
    if (!encode_pools(h)) {
        delete h;
        return KVC_ERR_CUDA;
    }
    *out = h;
    return KVC_OK;
}

kvc_status kvc_append_rope(kvc_cache *h, int32_t layer, const kvc_rope *rope, const void *q, int64_t q_stride, const void *k,
                           int64_t k_stride, const void *v, int64_t v_stride, const int32_t *cu_seqlens,
                           const int32_t *cache_index, int32_t total, void *q_out, void *k_out, void *stream) {
    if (!h || layer < 0 || layer >= h->cfg.n_layers || total < 0) return KVC_ERR_INVALID;
    const kvc_config &c = h->cfg;
    if (rope) {
        if (rope->d_rot < 0 || rope->d_rot > c.d_head || rope->d_rot % 8) return KVC_ERR_INVALID;
        if (rope->d_rot > 0 && (!rope->cos_sin || rope->n_positions <= 0)) return KVC_ERR_INVALID;
        if (rope->d_rot > 0 && !aligned16(rope->cos_sin)) return KVC_ERR_ALIGNMENT;
    }
    if (!cu_seqlens && total != c.batch) return KVC_ERR_INVALID;
    if (total == 0) return KVC_OK;
    if (!k || !v || !q != !q_out || !device_current(h)) return KVC_ERR_INVALID;
    if (k_out == k && c.dtype == KVC_E4M3) return KVC_ERR_INVALID;  // (the keys are read twice)
    const int eb = row_bytes_of(h);
    const int64_t kv_row = int64_t(c.n_kv_heads) * c.d_head, q_row = int64_t(c.n_heads) * c.d_head;
    if (k_stride < kv_row || v_stride < kv_row || (q && q_stride < q_row)) return KVC_ERR_INVALID;
    if (!aligned16(k) || !aligned16(v) || (q && (!aligned16(q) || !aligned16(q_out))) || (k_out && !aligned16(k_out)))
        return KVC_ERR_ALIGNMENT;
    if (k_stride * eb % 16 || v_stride * eb % 16 || (q && q_stride * eb % 16)) return KVC_ERR_ALIGNMENT;
    if ((q && q_out == q && q_stride != q_row) || (k_out == k && k_stride != kv_row)) return KVC_ERR_INVALID;  // (over rows not read yet)
    const auto bytes = [&](int64_t stride, int64_t row) { return ((total - 1) * stride + row) * eb; };
    const int64_t qn = q ? bytes(q_stride, q_row) : 0, kn = bytes(k_stride, kv_row), vn = bytes(v_stride, kv_row);
    const int64_t qon = q ? bytes(q_row, q_row) : 0, kon = k_out ? bytes(kv_row, kv_row) : 0;
    if ((q_out != q && overlap(q_out, qon, q, qn)) || overlap(q_out, qon, k, kn) || overlap(q_out, qon, v, vn) || overlap(q_out, qon, k_out, kon) ||
        (k_out != k && overlap(k_out, kon, k, kn)) || overlap(k_out, kon, q, qn) || overlap(k_out, kon, v, vn))
        return KVC_ERR_INVALID;
    kvc::RopeArgs a = rope_args(h, layer);
    a.q = static_cast<const uint8_t *>(q);
    a.k = static_cast<const uint8_t *>(k);
    a.v = static_cast<const uint8_t *>(v);
    a.q_out = static_cast<uint8_t *>(q_out);
    a.k_out = static_cast<uint8_t *>(k_out);
    a.q_token = q_stride * eb;
    a.k_token = k_stride * eb;
    a.v_token = v_stride * eb;
    a.cu_seqlens = cu_seqlens;
    a.cache_index = cache_index;
    a.total = total;
    if (rope && rope->d_rot > 0) {
        a.cos_sin = rope->cos_sin;
        a.positions = rope->positions;
        a.n_positions = rope->n_positions;
        a.half = rope->d_rot / 2;
        a.interleaved = rope->interleaved != 0;
    }
    return launch(h, a, stream);
}

kvc_status kvc_packed_attn(kvc_cache *h, int32_t layer, const void *q, const int32_t *cu_seqlens, const int32_t *cache_index,
                           int32_t total, int32_t max_rows_hint, void *out, void *stream) {
    if (!h || layer < 0 || layer >= h->cfg.n_layers || total < 0 || max_rows_hint < 0 || max_rows_hint > h->cfg.max_context)
        return KVC_ERR_INVALID;
    if (h->cfg.dtype != KVC_E4M3) return KVC_ERR_UNSUPPORTED;
    if (!cu_seqlens && total != h->cfg.batch) return KVC_ERR_INVALID;
    if (total == 0) return KVC_OK;
    if (!q || !out) return KVC_ERR_INVALID;
    const kvc_status st = refusal(h, q, out, total);
    return st != KVC_OK ? st : attend(h, layer, q, cu_seqlens, cache_index, 0, total, max_rows_hint, out, stream);
}

}  // extern "C"
