// kvc_ingest.cu -- new rows into the cache other than one run per sequence:
// packed prompts of different lengths, and the accepted path of a drafted tree.
//
// Both are copies of whole rows (row_vecs 16-byte vectors, consecutive lanes
// on consecutive vectors on both sides) whose destination is looked up once per
// row; K and V go in one launch, the path commit takes every layer in one.  Of
// an int8 cache each row is quantised by one warp as kvc_append does it.
#include <cuda_bf16.h>

#include "kvc_rows.cuh"

namespace kvc {
namespace {

constexpr int TOKENS = 8;  // tokens of a packed-append block

// Cache row (in rows of a layer's slab or pool, KV head 0) of position pos of
// sequence b and the distance between KV heads; false where the table has none.
__device__ __forceinline__ bool cache_row(const IngestArgs &a, int b, int pos, int64_t &row, int64_t &head_step) {
    if (!a.block_table) {
        row = int64_t(b) * a.H_kv * a.max_ctx + pos;
        head_step = a.max_ctx;
        return true;
    }
    const int phys = dev::ld(a.block_table + int64_t(b) * a.max_blocks + pos / 16);
    row = int64_t(phys) * a.H_kv * 16 + pos % 16;
    head_step = 16;
    return phys >= 0 && phys < a.num_blocks;
}

// One row of D bf16 elements, quantised by a warp into codes and a scale.
template <int D>
__device__ __forceinline__ void store_q8(const uint8_t *src, uint8_t *codes, float *scale, int lane) {
    constexpr int EPL = D / 32;
    const __nv_bfloat16 *x16 = reinterpret_cast<const __nv_bfloat16 *>(src) + lane * EPL;
    float x[EPL], sc;
#pragma unroll
    for (int e = 0; e < EPL; ++e) x[e] = __bfloat162float(x16[e]);
    const uint32_t packed = dev::quantise_row_q8<EPL>(x, sc);
    static_assert(EPL == 4, "four codes per lane");
    reinterpret_cast<uint32_t *>(codes)[lane] = packed;
    if (lane == 0) *scale = sc;
}

// The sequences' tokens in chunks of TOKENS, sequence after sequence: a block
// finds its chunk by a prefix sum over the sequences' chunk counts, 256
// sequences at a time.  Bound by the bytes: 675 MB (16 prompts of 64-8,000 tokens
// into pages, 8 KV heads of 128) in 109 us, 6.2 TB/s.
template <bool INT8>
__global__ void __launch_bounds__(256) append_packed_kernel(const __grid_constant__ IngestArgs a) {
    __shared__ int warp_sum[8];
    __shared__ int found_s[4];  // sequence, first token of the chunk in it, tokens, cache position of that token
    __shared__ int64_t row_s[TOKENS], step_s[TOKENS];
    dev::allow_dependents();
    dev::grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // sequence b's first row, its tokens and its cache position; none where they do not fit
    auto sequence = [&](int64_t chunk, int b, int &lo, int &n, int &c) {
        lo = dev::ld(a.cu_seqlens + b);
        const int hi = dev::ld(a.cu_seqlens + b + 1);
        c = a.cache_index ? dev::ld(a.cache_index + b) : 0;
        const bool bad = lo < 0 || hi < lo || hi > a.total || c < 0 || c > a.max_ctx || hi - lo > a.max_ctx - c;
        if (bad && chunk == 0) dev::record_error(a.err, ERR_DEVICE_INDEX);
        n = bad ? 0 : hi - lo;
    };
    for (int64_t chunk = blockIdx.x;; chunk += gridDim.x) {
        int64_t base = 0;  // chunks of the sequences before this batch
        bool found = false;
        int b0 = 0;
        for (; b0 < a.B && !found; b0 += 256) {
            const int b = b0 + threadIdx.x;
            int lo = 0, n = 0, c = 0;
            if (b < a.B) sequence(chunk, b, lo, n, c);
            const int mine = (n + TOKENS - 1) / TOKENS;
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            __syncthreads();  // the last batch's (chunk's) shared values are read
            if (lane == 31) warp_sum[warp] = incl;
            __syncthreads();
            int64_t first = base + incl - mine, all = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                if (w < warp) first += warp_sum[w];
                all += warp_sum[w];
            }
            if (chunk >= first && chunk < first + mine) {
                const int t = int(chunk - first) * TOKENS;
                found_s[0] = b;
                found_s[1] = lo + t;
                found_s[2] = n - t < TOKENS ? n - t : TOKENS;
                found_s[3] = c + t;
            }
            base += all;
            found = chunk < base;
        }
        if (chunk == 0)  // the sequences behind the batch that holds the first chunk: recorded too
            for (int b = b0 + threadIdx.x; b < a.B; b += 256) {
                int lo, n, c;
                sequence(chunk, b, lo, n, c);
            }
        if (!found) return;
        __syncthreads();
        const int t0 = found_s[1], nt = found_s[2];
        if (threadIdx.x < nt) {
            int64_t row, step;
            if (!cache_row(a, found_s[0], found_s[3] + threadIdx.x, row, step)) {
                dev::record_error(a.err, ERR_DEVICE_INDEX);
                row = -1;
            }
            row_s[threadIdx.x] = row;
            step_s[threadIdx.x] = step;
        }
        __syncthreads();
        if constexpr (INT8) {
            for (int x = warp; x < nt * a.H_kv * 2; x += 8) {
                const int i = x / (2 * a.H_kv), j = (x >> 1) % a.H_kv;
                const bool is_v = x & 1;
                const int64_t row = row_s[i] + j * step_s[i];
                store_q8<128>((is_v ? a.v_new : a.k_new) + ((int64_t(t0) + i) * a.H_kv + j) * 256, (is_v ? a.V : a.K) + row * 128,
                              (is_v ? a.v_scale : a.k_scale) + row, lane);
            }
        } else {
            // four vectors of K and four of V in flight per thread
            const int per = a.H_kv * a.row_vecs, all = nt * per;  // vectors of a token, of the chunk
            const uint4 *ks = reinterpret_cast<const uint4 *>(a.k_new) + int64_t(t0) * per, *vs = reinterpret_cast<const uint4 *>(a.v_new) + int64_t(t0) * per;
            for (int x0 = threadIdx.x; x0 < all; x0 += 4 * 256) {
                uint4 k[4], v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int x = x0 + 256 * e;
                    if (x < all) k[e] = __ldcs(ks + x), v[e] = __ldcs(vs + x);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int x = x0 + 256 * e, i = x / per, y = x - i * per, j = y / a.row_vecs;
                    if (x >= all || row_s[i] < 0) continue;
                    const int64_t to = (row_s[i] + j * step_s[i]) * a.row_vecs + y - j * a.row_vecs;
                    reinterpret_cast<uint4 *>(a.K)[to] = k[e];
                    reinterpret_cast<uint4 *>(a.V)[to] = v[e];
                }
            }
        }
    }
}

// A warp takes 16 path positions of one (layer, sequence, KV head), K and V:
// one lane each looks up a position's source and destination, then the rows
// move with four vectors of K and four of V in flight per lane.  The path
// entries of the check are the ones that are used, so that three dependent loads
// (counts; path and table; rows) stand between the launch and the stores: at
// 78 MB they, not the 12 us of the bytes, are most of the 20 us.
constexpr int STEPS = 16;

template <bool INT8>
__global__ void __launch_bounds__(256) tree_commit_kernel(const __grid_constant__ IngestArgs a) {
    dev::allow_dependents();
    dev::grid_dependency_wait();
    const int lane = threadIdx.x & 31, layer = blockIdx.y;
    const unsigned chunks = unsigned(a.P + STEPS - 1) / STEPS, segs = unsigned(a.B) * a.H_kv;
    const unsigned u = blockIdx.x * 8 + (threadIdx.x >> 5);  // (sequence, KV head, chunk)
    if (u >= segs * chunks) return;
    const unsigned seg = u / chunks, chunk = u - seg * chunks, b = seg / a.H_kv, kv = seg - b * a.H_kv;
    const int n = dev::ld(a.n_accept + b), c = dev::ld(a.cache_index + b), i0 = int(chunk) * STEPS;
    bool bad = n < 0 || n > a.P || c < 0 || c > a.max_ctx || n > a.max_ctx - c;
    int node = 0;  // path entry 32 (i0 / 32) + lane
    if (!bad && (i0 < n || chunk == 0)) {
        for (int i = lane; i < n; i += 32) {
            const int s = dev::ld(a.path + int64_t(b) * a.P + i);
            bad = bad || s < 0 || s >= a.T;
            if (i / 32 == i0 / 32) node = s;
        }
        bad = __any_sync(0xffffffffu, bad);
    }
    if (bad) {
        if (chunk == 0 && kv == 0 && layer == 0 && lane == 0) dev::record_error(a.err, ERR_DEVICE_INDEX);
        return;
    }
    const int steps = min(STEPS, n - i0);
    if (steps <= 0) return;
    int64_t to = -1, from = 0;  // lane i: row of position i0 + i in the cache and in k_new / v_new
    node = __shfl_sync(0xffffffffu, node, (i0 & 31) + (lane & (STEPS - 1)));
    if (lane < steps) {
        int64_t row, step;
        from = (int64_t(layer) * segs + seg) * a.T + node;
        if (cache_row(a, b, c + i0 + lane, row, step))
            to = row + kv * step;
        else
            dev::record_error(a.err, ERR_DEVICE_INDEX);
    }
    uint8_t *K = a.K + layer * a.layer_bytes, *V = a.V + layer * a.layer_bytes;
    if constexpr (INT8) {
        for (int i = 0; i < steps; ++i) {
            const int64_t d = __shfl_sync(0xffffffffu, to, i), f = __shfl_sync(0xffffffffu, from, i);
            store_q8<128>(a.k_new + f * 256, K + d * 128, a.k_scale + layer * a.layer_scales + d, lane);
            store_q8<128>(a.v_new + f * 256, V + d * 128, a.v_scale + layer * a.layer_scales + d, lane);
        }
    } else {
        const int vecs = steps * a.row_vecs;
        for (int x0 = 0; x0 < vecs; x0 += 128) {
            uint4 k[4], v[4];
            int64_t at[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int x = x0 + 32 * e + lane, i = min(x / a.row_vecs, steps - 1), w = x % a.row_vecs;
                const int64_t d = __shfl_sync(0xffffffffu, to, i), f = __shfl_sync(0xffffffffu, from, i);
                at[e] = x < vecs && d >= 0 ? d * a.row_vecs + w : -1;
                if (at[e] >= 0) {
                    k[e] = dev::ld(reinterpret_cast<const uint4 *>(a.k_new) + f * a.row_vecs + w);
                    v[e] = dev::ld(reinterpret_cast<const uint4 *>(a.v_new) + f * a.row_vecs + w);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (at[e] >= 0) {
                    reinterpret_cast<uint4 *>(K)[at[e]] = k[e];
                    reinterpret_cast<uint4 *>(V)[at[e]] = v[e];
                }
        }
    }
}

int grid_of(int64_t want, int num_sms) {
    const int64_t cap = int64_t(num_sms) * 8;
    return int(want < cap ? want : cap);
}

}  // namespace

cudaError_t launch_append_packed(const IngestArgs &a, bool int8, int num_sms, cudaStream_t s) {
    // (every sequence may end inside a chunk)
    const dim3 grid(grid_of(int64_t(a.total) / TOKENS + (a.B < a.total ? a.B : a.total), num_sms));
    return int8 ? launch_pdl(append_packed_kernel<true>, grid, dim3(256), 0, s, a)
                : launch_pdl(append_packed_kernel<false>, grid, dim3(256), 0, s, a);
}

cudaError_t launch_tree_commit(const IngestArgs &a, bool int8, cudaStream_t s) {
    const int64_t units = int64_t(a.B) * a.H_kv * ((a.P + STEPS - 1) / STEPS);
    if (units > 0x7fffffff || a.n_layers > 65535) return cudaErrorInvalidValue;
    const dim3 grid(unsigned((units + 7) / 8), unsigned(a.n_layers));
    return int8 ? launch_pdl(tree_commit_kernel<true>, grid, dim3(256), 0, s, a)
                : launch_pdl(tree_commit_kernel<false>, grid, dim3(256), 0, s, a);
}

}  // namespace kvc
