// kvc_pages.cu -- the pages of a paged cache: forked, made writable, freed,
// copied and compacted.
//
// "10.3 -- KV cache implementation details", section 7: a block table makes
// fixed-size blocks logically contiguous, and sequences with a common prefix
// share its blocks.  The state is the table and one reference count per block
// (0: free); there is no free list, so that the outcome of a call depends on
// nothing but the state: new pages are the lowest-numbered free blocks, handed
// out in the order of (sequence, logical block).
//
// Sharing is copy-on-write: a fork copies table rows and counts them; the
// reserve that precedes an append splits the shared page that the append would
// write, copying only its live rows.
#include "kvc_handle.cuh"

namespace kvc {
namespace {

constexpr int PAGE = 16;
constexpr int MAX_SEQS = 8192;

struct PagesArgs {
    int32_t *table;        // [B, max_blocks]
    int32_t *refs;         // [num_blocks]
    int32_t *err;
    int32_t B, max_blocks, num_blocks, max_ctx;
    // copies: pools of all layers
    uint8_t *K, *V;
    int32_t n_layers, H_kv, row_vecs;
    int64_t layer_vecs;    // vectors of a layer's pool
    // workspace: the number of copies, then their (src, dst, rows)
    int32_t *n_copies, *src, *dst, *rows;
    int32_t *list;         // [num_blocks]: blocks in hand-out (or moving) order
    int32_t *where;        // [num_blocks]: reserve, the places they go to; compact, where each block goes
};

// An entry as the calls take it: a block, or -1 (anything else is recorded).
__device__ __forceinline__ int entry(const PagesArgs &a, int x) {
    if (x >= 0 && x < a.num_blocks) return x;
    if (x != -1) dev::record_error(a.err, ERR_DEVICE_INDEX);
    return -1;
}

// ---- fork ------------------------------------------------------------------
// A block owns `cols` columns of the table: it keeps all B rows of them in
// shared memory, so that the gather over parents can go in place.  Counts
// change only where an entry does; integer sums do not depend on their order.
__global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ PagesArgs a, const int32_t *parent,
                                                   int cols) {
    extern __shared__ int32_t old[];  // [B][cols]
    dev::allow_dependents();
    dev::grid_dependency_wait();
    const int c0 = blockIdx.x * cols, nc = min(cols, a.max_blocks - c0);
    for (int x = threadIdx.x; x < a.B * nc; x += blockDim.x) {
        const int b = x / nc, j = x - b * nc;
        old[b * cols + j] = a.table[int64_t(b) * a.max_blocks + c0 + j];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < a.B * nc; x += blockDim.x) {
        const int b = x / nc, j = x - b * nc;
        const int p = dev::ld(parent + b);
        if (p < -1 || p >= a.B) {
            dev::record_error(a.err, ERR_DEVICE_INDEX);
            continue;
        }
        if (p == b) continue;
        const int was = entry(a, old[b * cols + j]), now = p < 0 ? -1 : entry(a, old[p * cols + j]);
        a.table[int64_t(b) * a.max_blocks + c0 + j] = now;
        if (was == now) continue;
        if (now >= 0) atomicAdd(a.refs + now, 1);
        if (was >= 0) atomicSub(a.refs + was, 1);
    }
}

// ---- free ------------------------------------------------------------------
__global__ void __launch_bounds__(256) free_kernel(const __grid_constant__ PagesArgs a, const int32_t *keep) {
    dev::allow_dependents();
    dev::grid_dependency_wait();
    const int64_t total = int64_t(a.B) * a.max_blocks;
    for (int64_t x = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; x < total; x += int64_t(gridDim.x) * blockDim.x) {
        const int b = int(x / a.max_blocks), j = int(x - int64_t(b) * a.max_blocks);
        const int n = dev::ld(keep + b);
        if (n < 0 || n > a.max_ctx) {
            if (j == 0) dev::record_error(a.err, ERR_DEVICE_INDEX);
            continue;
        }
        if (j < (n + PAGE - 1) / PAGE) continue;
        const int was = a.table[x];
        if (was == -1) continue;
        a.table[x] = -1;
        const int page = entry(a, was);
        if (page >= 0) atomicSub(a.refs + page, 1);
    }
}

// ---- block-wide prefix sums ----------------------------------------------------
// Exclusive prefix sum of x over the 1024 threads of the block; `all` receives
// the total.  part: 32 ints of shared memory.
__device__ __forceinline__ int block_scan(int x, int *part, int &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    __syncthreads();  // part is free again
    if (lane == 31) part[warp] = y;
    __syncthreads();
    int t = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += z;
    }
    all = __shfl_sync(0xffffffffu, t, 31);
    const int before = __shfl_sync(0xffffffffu, t, warp ? warp - 1 : 0);
    return y - x + (warp ? before : 0);
}

// ---- reserve ----------------------------------------------------------------
// The range of sequence b is its logical blocks [len / 16, ceil(new_len / 16)):
// pages missing there are added, shared ones replaced.  A shared page: of its holders that reserve it in
// this call the first ones (by sequence) leave it while its count is above 1.
struct Reserve {
    const int32_t *len, *new_len;
};

// Does sequence b need a fresh page at logical block j of its range, which is x
// now?
__device__ __forceinline__ bool wants(const PagesArgs &a, const int32_t *first, const int32_t *offset, int b, int j, int x) {
    if (x < 0 || x >= a.num_blocks) return true;
    int held = a.refs[x];
    if (held <= 1) return false;
    for (int k = 0; k < b; ++k)  // earlier holders that leave it
        if (first[k] <= j && j < first[k] + offset[k + 1] - offset[k] && a.table[int64_t(k) * a.max_blocks + j] == x) --held;
    return held > 1;
}

// One block of 1024 threads.  The logical blocks of all ranges, sequence after
// sequence, are one list of places; a prefix sum over the places that want a
// page gives each its number in the order of hand-out, another one over the
// counts finds the lowest free blocks.  Only if those suffice is anything changed.
// Bound by the latency of its passes: 10 us for 64 sequences.  `wants` walks the
// earlier sequences of a shared page one by one: beams of one parent that all
// write their shared page take 0.1 ms at 1,024 sequences and 6.8 ms at 8,192.
__global__ void __launch_bounds__(1024) reserve_kernel(const __grid_constant__ PagesArgs a, const Reserve r) {
    extern __shared__ int32_t dyn[];
    int32_t *first = dyn, *offset = dyn + a.B;  // [B] first logical block, [B + 1] first place
    __shared__ int part[32];
    __shared__ int copies;
    dev::allow_dependents();
    dev::grid_dependency_wait();
    const int tid = threadIdx.x;
    int4 count4 = make_int4(1, 1, 1, 1);  // the first 4096 counts: on their way meanwhile
    if (4 * tid + 3 < a.num_blocks) count4 = *reinterpret_cast<const int4 *>(a.refs + 4 * tid);
    if (tid == 0) copies = 0;
    int places = 0;
    for (int b0 = 0; b0 < a.B; b0 += 1024) {
        const int b = b0 + tid;
        int j0 = 0, length = 0;
        if (b < a.B) {
            const int len = dev::ld(r.len + b), grown = dev::ld(r.new_len + b);
            bool ok = len >= 0 && grown >= len && grown <= a.max_ctx;
            j0 = ok ? len / PAGE : 0;
            if (ok && grown > len) {
                length = (grown + PAGE - 1) / PAGE - j0;
                if (len % PAGE != 0) {  // the page of the rows below len
                    const int x = a.table[int64_t(b) * a.max_blocks + j0];
                    ok = x >= 0 && x < a.num_blocks;
                }
            }
            if (!ok) {
                dev::record_error(a.err, ERR_DEVICE_INDEX);
                length = 0;
            }
        }
        int all;
        const int before = places + block_scan(length, part, all);
        if (b < a.B) first[b] = j0, offset[b] = before;
        places += all;
    }
    if (tid == 0) offset[a.B] = places;
    __syncthreads();
    // the sequence of a place
    auto sequence = [&](int place) {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (offset[mid] <= place) lo = mid; else hi = mid - 1;
        }
        return lo;
    };
    int total = 0;
    for (int p0 = 0; p0 < places; p0 += 1024) {
        const int place = p0 + tid;
        bool w = false;
        if (place < places) {
            const int b = sequence(place), j = first[b] + place - offset[b];
            w = wants(a, first, offset, b, j, a.table[int64_t(b) * a.max_blocks + j]);
        }
        int all;
        const int at = total + block_scan(w, part, all);
        if (w && at < a.num_blocks) a.where[at] = place;
        total += all;
    }
    // the lowest `total` free blocks, in order
    int found = 0;
    for (int x0 = 0; x0 < a.num_blocks && found < total; x0 += 4096) {
        const int x = x0 + 4 * tid;
        if (x0 > 0 && x + 3 < a.num_blocks) count4 = *reinterpret_cast<const int4 *>(a.refs + x);
        int c[4] = {count4.x, count4.y, count4.z, count4.w};
        if (x + 3 >= a.num_blocks)  // the end
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = x + e < a.num_blocks ? a.refs[x + e] : 1;
        int all;
        int at = found + block_scan((c[0] == 0) + (c[1] == 0) + (c[2] == 0) + (c[3] == 0), part, all);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c[e] == 0) {
                if (at < total) a.list[at] = x + e;
                ++at;
            }
        found += all;
    }
    __syncthreads();
    if (found < total) {  // (the whole block agrees)
        if (tid == 0) {
            dev::record_error(a.err, ERR_CAPACITY);
            *a.n_copies = 0;
        }
        return;
    }
    for (int i = tid; i < total; i += 1024) {
        const int place = a.where[i], page = a.list[i], b = sequence(place), j = first[b] + place - offset[b];
        int32_t *at = a.table + int64_t(b) * a.max_blocks + j;
        const int was = *at;
        *at = page;
        a.refs[page] = 1;
        if (entry(a, was) < 0) continue;
        atomicSub(a.refs + was, 1);
        const int len = dev::ld(r.len + b);
        if (j == len / PAGE && len % PAGE != 0) {  // (at most one page of a sequence)
            const int c = atomicAdd(&copies, 1);
            a.src[c] = was;
            a.dst[c] = page;
            a.rows[c] = len % PAGE;
        }
    }
    __syncthreads();
    if (tid == 0) *a.n_copies = copies;
}

// ---- compact ----------------------------------------------------------------
// One block.  With `live` pages in all, the free blocks below `live` and the
// live ones from there on are equally many; in one ascending pass over the
// counts the former come first, so that one list holds the targets and behind
// them the pages that move.
__global__ void __launch_bounds__(1024) compact_plan_kernel(const __grid_constant__ PagesArgs a, int32_t *n_live) {
    __shared__ int part[32];
    dev::allow_dependents();
    dev::grid_dependency_wait();
    const int tid = threadIdx.x;
    int n = 0;
    for (int x = tid; x < a.num_blocks; x += 1024) n += a.refs[x] > 0;
    int live;
    block_scan(n, part, live);
    int found = 0;
    for (int x0 = 0; x0 < a.num_blocks; x0 += 4096) {
        const int x = x0 + 4 * tid;
        int marks = 0, k = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (x + e < a.num_blocks) {
                const bool used = a.refs[x + e] > 0;
                a.where[x + e] = x + e;  // where a page goes: nowhere, so far
                if (used == (x + e >= live)) marks |= 1 << e, ++k;
            }
        int all, at = found + block_scan(k, part, all);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (marks >> e & 1) a.list[at++] = x + e;
        found += all;
    }
    __syncthreads();
    const int moves = found / 2;
    for (int i = tid; i < moves; i += 1024) {
        const int to = a.list[i], from = a.list[moves + i];
        a.src[i] = from;
        a.dst[i] = to;
        a.where[from] = to;
        a.refs[to] = a.refs[from];
        a.refs[from] = 0;
    }
    if (tid == 0) {
        *a.n_copies = moves;
        *n_live = live;
    }
}

// ---- copies ----------------------------------------------------------------
// Pairs (src[i], dst[i]) of blocks, every layer, K and V; the first rows[i] of
// the 16 rows of each KV head (all of them without `rows`).  A warp takes the
// rows of one KV head, contiguous on both sides.  Bound by the bytes: a compaction
// that moves 434 MB of reads and writes takes 63 us, 6.9 TB/s.  REMAP: also sends
// every table entry through `where`.
template <bool REMAP>
__global__ void __launch_bounds__(256) copy_kernel(const __grid_constant__ PagesArgs a, int n_pairs) {
    dev::allow_dependents();
    dev::grid_dependency_wait();
    if constexpr (REMAP) {
        const int64_t total = int64_t(a.B) * a.max_blocks;
        for (int64_t x = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; x < total; x += int64_t(gridDim.x) * blockDim.x) {
            const int was = a.table[x];
            if (was != -1) {
                const int page = entry(a, was);
                if (page >= 0 && a.where[page] != was) a.table[x] = a.where[page];
            }
        }
    }
    const int lane = threadIdx.x & 31;
    const int n = n_pairs >= 0 ? n_pairs : *a.n_copies;
    const int64_t per = 2ll * a.n_layers * a.H_kv, units = n * per;
    for (int64_t u = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units; u += int64_t(gridDim.x) * 8) {
        const int i = int(u / per), w = int(u - i * per);
        const int src = a.src[i], dst = a.dst[i], rows = a.rows ? a.rows[i] : PAGE;
        if (src < 0 || src >= a.num_blocks || dst < 0 || dst >= a.num_blocks) {
            if (w == 0 && lane == 0) dev::record_error(a.err, ERR_DEVICE_INDEX);
            continue;
        }
        const int kv = w % a.H_kv, lt = w / a.H_kv;  // lt = 2 * layer + (0: K, 1: V)
        uint4 *pool = reinterpret_cast<uint4 *>(lt & 1 ? a.V : a.K) + (lt >> 1) * a.layer_vecs;
        const uint4 *from = pool + (int64_t(src) * a.H_kv + kv) * PAGE * a.row_vecs;
        uint4 *to = pool + (int64_t(dst) * a.H_kv + kv) * PAGE * a.row_vecs;
        const int vecs = rows * a.row_vecs;
        for (int x = lane; x < vecs; x += 256) {  // eight vectors in flight
            uint4 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (x + 32 * e < vecs) v[e] = __ldcs(from + x + 32 * e);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (x + 32 * e < vecs) to[x + 32 * e] = v[e];
        }
    }
}

struct Workspace {
    uint64_t src, dst, rows, list, where, total;
};

Workspace pages_workspace(const kvc_config *c, int32_t num_blocks) {
    Workspace w;
    const uint64_t blocks = align256(4ull * num_blocks), seqs = align256(4ull * c->batch);
    const uint64_t pairs = blocks > seqs ? blocks : seqs;  // a sequence copies one page, a compaction any number
    w.src = 256;                                           // (the number of copies is at byte 0)
    w.dst = w.src + pairs;
    w.rows = w.dst + pairs;
    w.list = w.rows + seqs;
    w.where = w.list + blocks;
    w.total = w.where + blocks;
    return w;
}

// What every call fills in: the pools, and the shape of the table.
kvc_status pages_args(const kvc_cache *h, PagesArgs &a) {
    if (!h) return KVC_ERR_INVALID;
    if (!h->block_table) return KVC_ERR_UNSUPPORTED;
    if (!device_current(h)) return KVC_ERR_INVALID;
    const kvc_config &c = h->cfg;
    a = PagesArgs{};
    a.err = reinterpret_cast<int32_t *>(h->ws);
    a.B = c.batch;
    a.max_blocks = c.max_context / PAGE;
    a.num_blocks = h->num_blocks;
    a.max_ctx = c.max_context;
    a.K = h->k_base;
    a.V = h->v_base;
    a.n_layers = c.n_layers;
    a.H_kv = c.n_kv_heads;
    a.row_vecs = c.d_head * h->elem_bytes / 16;
    a.layer_vecs = int64_t(layer_slab_bytes(h) / 16);
    return KVC_OK;
}

// The same with the state: the table has to be the handle's.
kvc_status pages_args(const kvc_cache *h, int32_t *block_table, int32_t *refcount, PagesArgs &a) {
    const kvc_status st = pages_args(h, a);
    if (st != KVC_OK) return st;
    // (places in the list of all ranges are 32-bit numbers)
    if (a.B > MAX_SEQS || int64_t(a.B) * a.max_blocks > 0x7fffffff) return KVC_ERR_UNSUPPORTED;
    if (block_table != h->block_table || !refcount) return KVC_ERR_INVALID;
    if (!aligned16(refcount)) return KVC_ERR_ALIGNMENT;
    a.table = block_table;
    a.refs = refcount;
    return KVC_OK;
}

kvc_status bind_workspace(const kvc_cache *h, void *workspace, uint64_t ws_bytes, PagesArgs &a) {
    const Workspace w = pages_workspace(&h->cfg, h->num_blocks);
    if (!workspace || ws_bytes < w.total) return KVC_ERR_WORKSPACE;
    if (!aligned16(workspace)) return KVC_ERR_ALIGNMENT;
    uint8_t *p = static_cast<uint8_t *>(workspace);
    a.n_copies = reinterpret_cast<int32_t *>(p);
    a.src = reinterpret_cast<int32_t *>(p + w.src);
    a.dst = reinterpret_cast<int32_t *>(p + w.dst);
    a.rows = reinterpret_cast<int32_t *>(p + w.rows);
    a.list = reinterpret_cast<int32_t *>(p + w.list);
    a.where = reinterpret_cast<int32_t *>(p + w.where);
    return KVC_OK;
}

kvc_status done(cudaError_t e) { return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA; }

template <bool REMAP>
cudaError_t launch_copies(const kvc_cache *h, const PagesArgs &a, int n, int64_t most, cudaStream_t s) {
    const int64_t want = (most * 2 * a.n_layers * a.H_kv + 7) / 8, cap = int64_t(h->num_sms) * 8;
    return launch_pdl(copy_kernel<REMAP>, dim3(unsigned(want < cap ? want : cap)), dim3(256), 0, s, a, n);
}

}  // namespace
}  // namespace kvc

extern "C" {

uint64_t kvc_pages_workspace_bytes(const kvc_config *cfg, int32_t num_blocks) {
    if (kvc_pool_bytes(cfg, num_blocks) == 0) return 0;
    return kvc::pages_workspace(cfg, num_blocks).total;
}

kvc_status kvc_pages_fork(kvc_cache *h, int32_t *block_table, int32_t *refcount, const int32_t *parent, void *stream) {
    kvc::PagesArgs a;
    const kvc_status st = kvc::pages_args(h, block_table, refcount, a);
    if (st != KVC_OK) return st;
    if (!parent) return KVC_ERR_INVALID;
    // the columns of a block's table rows: four entries a thread, whole 32-byte
    // sectors, no more than 48 KB
    int cols = 1024 / a.B, most = 48 * 1024 / (4 * a.B);
    cols = cols < 8 ? 8 : cols > 32 ? 32 : cols & ~7;
    if (cols > most) cols = most < 1 ? 1 : most;
    const int grid = (a.max_blocks + cols - 1) / cols;
    return kvc::done(kvc::launch_pdl(kvc::fork_kernel, dim3(grid), dim3(256), cols * a.B * 4, static_cast<cudaStream_t>(stream),
                                     a, parent, cols));
}

kvc_status kvc_pages_reserve(kvc_cache *h, int32_t *block_table, int32_t *refcount, const int32_t *len,
                             const int32_t *new_len, void *workspace, uint64_t ws_bytes, void *stream) {
    kvc::PagesArgs a;
    kvc_status st = kvc::pages_args(h, block_table, refcount, a);
    if (st != KVC_OK) return st;
    if (!len || !new_len) return KVC_ERR_INVALID;
    st = kvc::bind_workspace(h, workspace, ws_bytes, a);
    if (st != KVC_OK) return st;
    const int smem = 4 * (2 * a.B + 1);
    // (the kernel's own static shared memory counts towards the 48 KB too)
    if (smem > 47 * 1024 &&
        cudaFuncSetAttribute(kvc::reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * (2 * kvc::MAX_SEQS + 1)) != cudaSuccess)
        return KVC_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kvc::launch_pdl(kvc::reserve_kernel, dim3(1), dim3(1024), smem, s, a, kvc::Reserve{len, new_len});
    if (e != cudaSuccess) return KVC_ERR_CUDA;
    return kvc::done(kvc::launch_copies<false>(h, a, -1, a.B, s));
}

kvc_status kvc_pages_free(kvc_cache *h, int32_t *block_table, int32_t *refcount, const int32_t *keep_len, void *stream) {
    kvc::PagesArgs a;
    const kvc_status st = kvc::pages_args(h, block_table, refcount, a);
    if (st != KVC_OK) return st;
    if (!keep_len) return KVC_ERR_INVALID;
    const int64_t want = (int64_t(a.B) * a.max_blocks + 255) / 256, cap = int64_t(h->num_sms) * 8;
    return kvc::done(kvc::launch_pdl(kvc::free_kernel, dim3(unsigned(want < cap ? want : cap)), dim3(256), 0,
                                     static_cast<cudaStream_t>(stream), a, keep_len));
}

kvc_status kvc_pages_copy(kvc_cache *h, const int32_t *src, const int32_t *dst, int32_t n, void *stream) {
    if (!h || n < 0) return KVC_ERR_INVALID;
    if (!h->block_table) return KVC_ERR_UNSUPPORTED;
    if (n == 0) return KVC_OK;
    if (!src || !dst) return KVC_ERR_INVALID;
    kvc::PagesArgs a;
    const kvc_status st = kvc::pages_args(h, a);
    if (st != KVC_OK) return st;
    a.src = const_cast<int32_t *>(src);
    a.dst = const_cast<int32_t *>(dst);
    return kvc::done(kvc::launch_copies<false>(h, a, n, n, static_cast<cudaStream_t>(stream)));
}

kvc_status kvc_pages_compact(kvc_cache *h, int32_t *block_table, int32_t *refcount, int32_t *block_map,
                             int32_t *n_live, void *workspace, uint64_t ws_bytes, void *stream) {
    kvc::PagesArgs a;
    kvc_status st = kvc::pages_args(h, block_table, refcount, a);
    if (st != KVC_OK) return st;
    if (!n_live) return KVC_ERR_INVALID;
    st = kvc::bind_workspace(h, workspace, ws_bytes, a);
    if (st != KVC_OK) return st;
    a.rows = nullptr;  // whole blocks
    if (block_map) a.where = block_map;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kvc::launch_pdl(kvc::compact_plan_kernel, dim3(1), dim3(1024), 0, s, a, n_live);
    if (e != cudaSuccess) return KVC_ERR_CUDA;
    return kvc::done(kvc::launch_copies<true>(h, a, -1, a.num_blocks, s));
}

}  // extern "C"
