// kvc_rows_simt.cu -- attention of several new tokens per sequence on the CUDA
// cores, for the contiguous caches that the tensor-core kernel does not take:
// fp32 of every head width, 16-bit types of 32 and 256.
//
// A block of four warps takes 16 query rows of one (sequence, KV head) -- row
// r = i * n + t is head i of the group, token t -- and walks the keys 32 at a
// time.  Per step the block brings 32 K and V rows into shared memory; a warp
// takes four query rows: lane j forms the four scores of key j (fp32 products
// and sums, K read once for the four rows), the rows' running maximum and sum
// are kept in the log2 domain, and the probabilities meet V with the lanes on
// the head's columns.  Bound by the CUDA cores and by copies that nothing overlaps:
// 4,096 tokens in fp32, 32 heads over 8 of 128, take 10.4 ms, 13 TFLOP/s; in bf16,
// 16 heads over 4 of 256, 8.8 ms, 16 TFLOP/s; 16 trees of 16 tokens over 8,192 fp32
// rows, 32 heads over 8 of 128, 3.8 ms.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/kvc.h"
#include "kvc_rows.cuh"

namespace kvc {
namespace {

constexpr int WARPS = 4, RW = 4, ROWS = WARPS * RW, KEYS = 32;

template <typename T>
__device__ __forceinline__ void widen16(const uint4 &v, float *x);  // a 16-byte vector to floats
template <>
__device__ __forceinline__ void widen16<float>(const uint4 &v, float *x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}
template <>
__device__ __forceinline__ void widen16<__nv_bfloat16>(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
template <>
__device__ __forceinline__ void widen16<__half>(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

template <typename T, int D>
__global__ void __launch_bounds__(WARPS * 32) rows_simt_kernel(const __grid_constant__ RowsArgs a, int parts) {
    constexpr int VEC = 16 / sizeof(T);      // elements of a 16-byte vector
    constexpr int CH = D / VEC;              // vectors of a row
    constexpr int EPL = D / 32;              // columns of the head per lane
    // rows padded by one vector, so that 32 lanes on 32 rows meet 32 banks
    __shared__ __align__(16) uint4 ks[KEYS * (CH + 1)];
    __shared__ __align__(16) T vs[KEYS * D];
    __shared__ __align__(16) float qs[ROWS * D];
    dev::allow_dependents();
    dev::grid_dependency_wait();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // `parts` blocks share the rows of a segment
    const int seg = blockIdx.x / parts, part = blockIdx.x - seg * parts, b = seg / a.H_kv, kv = seg - b * a.H_kv;
    const int H = a.H_kv * a.group;
    const RowsSeq s = rows_seq(a, b);
    if (s.bad && part == 0 && kv == 0 && threadIdx.x == 0) dev::record_error(a.err, ERR_DEVICE_INDEX);
    const int64_t rows = int64_t(s.n) * a.group;
    for (int64_t r0 = int64_t(part) * ROWS; r0 < rows; r0 += int64_t(parts) * ROWS) {
        __syncthreads();
        for (int x = threadIdx.x; x < ROWS * D; x += blockDim.x) {
            const int64_t r = r0 + x / D;
            float y = 0.f;
            if (r < rows) {
                const int i = int(r / s.n), t = int(r - int64_t(i) * s.n);
                y = to_float(reinterpret_cast<const T *>(a.q)[rows_offset(a, s, b, H, kv * a.group + i, t, D) + x % D]);
            }
            qs[x] = y * a.scale_log2;
        }
        int tok[RW];
        float m[RW], l[RW], acc[RW][EPL];
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            const int64_t r = r0 + warp * RW + k;
            tok[k] = r < rows ? int(r % s.n) : -1;
            m[k] = -INFINITY, l[k] = 0.f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) acc[k][e] = 0.f;
        }
        // causal: no key past the block's last token; rows of several heads
        // reach the last token
        const int64_t r_last = r0 + ROWS - 1 < rows ? r0 + ROWS - 1 : rows - 1;
        const bool one_head = r0 / s.n == r_last / s.n;
        const int new_end = a.tree_mask || !one_head ? s.n : int(r_last % s.n) + 1;
        const int end = s.c + new_end;  // keys: cached rows, then new ones
        for (int j0 = 0; j0 < end; j0 += KEYS) {
            // vector x of the step's K and V rows
            auto fetch = [&](int x, uint4 &kk, uint4 &vv) {
                const int c16 = x % CH, key = j0 + x / CH;
                kk = vv = make_uint4(0, 0, 0, 0);
                if (key >= end) return;
                const bool cached = key < s.c;
                const uint8_t *kp = cached ? a.K : static_cast<const uint8_t *>(a.k_new);
                const uint8_t *vp = cached ? a.V : static_cast<const uint8_t *>(a.v_new);
                // the row's element offset over D
                const int64_t row = cached ? (int64_t(b) * a.H_kv + kv) * a.max_ctx + key
                                           : rows_offset(a, s, b, a.H_kv, kv, key - s.c, 1);
                kk = dev::ld(reinterpret_cast<const uint4 *>(kp) + row * CH + c16);
                vv = dev::ld(reinterpret_cast<const uint4 *>(vp) + row * CH + c16);
            };
            auto store = [&](int x, const uint4 &kk, const uint4 &vv) {
                const int j = x / CH, c16 = x % CH;
                ks[j * (CH + 1) + c16] = kk;
                *reinterpret_cast<uint4 *>(vs + j * D + c16 * VEC) = vv;
            };
            constexpr int PER = KEYS * CH / (WARPS * 32);  // vectors of K, and of V, per thread
            if constexpr (PER <= 2) {  // (few enough to be on their way while other warps end the step before)
                uint4 kk[PER], vv[PER];
#pragma unroll
                for (int i = 0; i < PER; ++i) fetch(threadIdx.x + i * WARPS * 32, kk[i], vv[i]);
                __syncthreads();
#pragma unroll
                for (int i = 0; i < PER; ++i) store(threadIdx.x + i * WARPS * 32, kk[i], vv[i]);
            } else {
                __syncthreads();
                for (int x = threadIdx.x; x < KEYS * CH; x += blockDim.x) {
                    uint4 kk, vv;
                    fetch(x, kk, vv);
                    store(x, kk, vv);
                }
            }
            __syncthreads();
            float sc[RW];
#pragma unroll
            for (int k = 0; k < RW; ++k) sc[k] = 0.f;
            for (int c16 = 0; c16 < CH; ++c16) {
                float kx[VEC];
                widen16<T>(ks[lane * (CH + 1) + c16], kx);
#pragma unroll
                for (int k = 0; k < RW; ++k) {
                    const float *qr = qs + (warp * RW + k) * D + c16 * VEC;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) sc[k] = fmaf(kx[e], qr[e], sc[k]);
                }
            }
            const int key = j0 + lane;
#pragma unroll
            for (int k = 0; k < RW; ++k) {
                bool see = tok[k] >= 0 && key < end;
                if (see && key >= s.c) {
                    const int sn = key - s.c;
                    see = a.tree_mask ? (dev::ld(a.tree_mask + (int64_t(b) * a.T + tok[k]) * a.mask_words + (sn >> 5)) >> (sn & 31)) & 1
                                      : sn <= tok[k];
                }
                const float x = see ? sc[k] : -INFINITY;
                float mx = x;
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float m_new = fmaxf(m[k], mx);
                const float ref = m_new == -INFINITY ? 0.f : m_new;  // (nothing seen so far, or only NaN, which stays)
                const float corr = exp2f(m[k] - ref);
                const float p = see ? exp2f(x - ref) : 0.f;
                m[k] = m_new;
                l[k] = l[k] * corr + p;
#pragma unroll
                for (int e = 0; e < EPL; ++e) acc[k][e] *= corr;
                unsigned live = __ballot_sync(0xffffffffu, see);  // rows that are not seen do not meet p
                while (live) {
                    const int j = __ffs(live) - 1;
                    live &= live - 1;
                    const float pj = __shfl_sync(0xffffffffu, p, j);
#pragma unroll
                    for (int e = 0; e < EPL; ++e) acc[k][e] = fmaf(pj, to_float(vs[j * D + lane + 32 * e]), acc[k][e]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            float sum = l[k];
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that sees nothing: zeros
            if (tok[k] >= 0) {
                const int i = int((r0 + warp * RW + k) / s.n);
                T *o = reinterpret_cast<T *>(a.out) + rows_offset(a, s, b, H, kv * a.group + i, tok[k], D);
#pragma unroll
                for (int e = 0; e < EPL; ++e) o[lane + 32 * e] = from_float<T>(acc[k][e] * inv);
            }
        }
    }
}

template <typename T>
cudaError_t launch_type(const RowsArgs &a, int D, int parts, cudaStream_t s) {
    const dim3 grid(unsigned(int64_t(a.B) * a.H_kv * parts));
    switch (D) {
        case 32: return launch_pdl(rows_simt_kernel<T, 32>, grid, dim3(WARPS * 32), 0, s, a, parts);
        case 256: return launch_pdl(rows_simt_kernel<T, 256>, grid, dim3(WARPS * 32), 0, s, a, parts);
    }
    if constexpr (sizeof(T) == 4) {
        if (D == 64) return launch_pdl(rows_simt_kernel<T, 64>, grid, dim3(WARPS * 32), 0, s, a, parts);
        if (D == 128) return launch_pdl(rows_simt_kernel<T, 128>, grid, dim3(WARPS * 32), 0, s, a, parts);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

// max_tokens: an upper bound on the new tokens of one sequence.
cudaError_t launch_rows_simt(const RowsArgs &a, int dtype, int D, int max_tokens, cudaStream_t s) {
    const int64_t x = (int64_t(max_tokens) * a.group + ROWS - 1) / ROWS;
    const int64_t segs = int64_t(a.B) * a.H_kv;
    if (segs > 0x7fffffff) return cudaErrorInvalidValue;
    // (packed calls: max_tokens is the total; blocks past a sequence's rows leave at once)
    const int64_t cap = segs >= 1048576 ? 1 : 1048576 / segs;
    const int parts = int(x < cap ? x : cap);
    switch (dtype) {
        case KVC_BF16: return launch_type<__nv_bfloat16>(a, D, parts, s);
        case KVC_FP16: return launch_type<__half>(a, D, parts, s);
        case KVC_FP32: return launch_type<float>(a, D, parts, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvc
