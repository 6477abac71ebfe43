// kvc_handle.cuh -- the cache handle and the host helpers that the API files
// share.  Not part of the public ABI (see include/kvc.h).
#pragma once

#include <mutex>

#include <cudaTypedefs.h>

#include "../../include/kvc.h"
#include "kvc_internal.cuh"
#include "kvc_rows.cuh"

struct kvc_cache {
    kvc_config cfg;
    int device;
    int num_sms;
    int max_smem;            // opt-in dynamic shared memory per block
    int elem_bytes;
    int group;               // n_heads / n_kv_heads
    int num_splits;          // 0: automatic
    uint64_t flag_timeout_ns;  // limit of the split combine's wait for the other splits
    uint8_t *k_base;
    uint8_t *v_base;
    uint8_t *k_scale;        // int8 caches: per-row fp32 scales [L, B, H_kv, T_max]; else null
    uint8_t *v_scale;
    const int32_t *block_table;  // paged caches: [B, max_blocks]; else null
    int32_t num_blocks;          // paged: physical blocks per layer pool
    int32_t kv_pair;             // paged: KV heads read per tile (1, or 2 with the pair kernel)
    uint8_t *ws;
    uint64_t ws_bytes;
    kvc::WorkspaceLayout wl;
    const kvc::DecodeKernelInfo *decode;
    const kvc::PrefillKernelInfo *prefill;  // nullptr where chunked prefill is not built
    int n_stages;
    int smem_bytes;
    CUtensorMap tm_k32, tm_k8, tm_v32, tm_v8;  // used by kernels with info->tensor_maps
    CUtensorMap pf_k32, pf_k8, pf_v32, pf_v8;  // the chunked prefill's (64-column blocks)
    CUtensorMap pf_k128, pf_v128;             // and its whole-tile boxes (128 rows)
    CUtensorMap rb_k64, rb_v64, rb_k32, rb_v32;  // kernels with info->ragged_maps: 64- and 32-row boxes
    const kvc::RowsKernelInfo *rows;          // prompts and trees on the tensor cores; nullptr: on the CUDA cores
    CUtensorMap rows_k, rows_v;               // its maps of the cache: 128-row boxes, or whole blocks of one KV head
};

namespace kvc {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Is the handle's device the calling thread's?
inline bool device_current(const kvc_cache *h) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == h->device;
}

inline uint64_t layer_scale_bytes(const kvc_cache *h) {
    const kvc_config &c = h->cfg;
    return uint64_t(c.batch) * c.n_kv_heads * uint64_t(c.max_context) * 4;
}

inline uint64_t layer_slab_bytes(const kvc_cache *h) {
    const kvc_config &c = h->cfg;
    if (h->block_table)  // paged: one pool of num_blocks blocks of 16 rows per KV head
        return uint64_t(h->num_blocks) * c.n_kv_heads * 16ull * c.d_head * h->elem_bytes;
    return uint64_t(c.batch) * c.n_kv_heads * uint64_t(c.max_context) * c.d_head * h->elem_bytes;
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

}  // namespace kvc
