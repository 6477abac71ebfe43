// kvc_e4m3.cuh -- the 8-bit paged cache (KVC_E4M3) and the rotated append: what
// their kernels and the host API share.
//
// A pool holds e4m3 codes, [num_blocks, H_kv, 16, 128] bytes per layer, and one
// fp32 scale per (block, KV head) in an array [num_blocks, H_kv]; a row's values
// are code * scale.  Scales that the append chooses are powers of two, so that a
// block whose scale grows keeps its older codes exactly, but for those that leave
// the format's normal range.
#pragma once

#include "kvc_internal.cuh"

namespace kvc {

// ---- the rotated append (kvc_rope.cu) ----------------------------------------
struct RopeArgs {
    uint8_t *K, *V;              // layer slab or pool
    float *k_scale, *v_scale;    // int8: per row; e4m3: per (block, KV head); else null
    const int32_t *block_table;
    const uint8_t *q, *k, *v;
    uint8_t *q_out, *k_out;      // dense [total, heads, D], or null
    const float *cos_sin;        // [n_positions, 2 * half]; null: no rotation
    const int32_t *positions;    // [total], or null: the cache position
    const int32_t *cu_seqlens;   // [B + 1], or null: T tokens of each sequence
    const int32_t *cache_index;  // [B], or null: 0
    int32_t *err;
    int64_t q_token, k_token, v_token;  // bytes from one token to the next
    int64_t kv_seq, kv_head;     // bytes: rows [B, H_kv, T, D] (kv_seq > 0), or from one KV head to the next
    int32_t index_offset;        // added to cache_index
    int32_t T, total;
    int32_t n_positions, half, interleaved;  // half: rotated elements / 2
    int32_t B, H, H_kv, D, max_ctx, max_blocks, num_blocks;
    int32_t n_heads;             // rows of a token that the row items take
    int32_t parts, per_part;     // row items per token, and their heads
    int32_t range, both;         // tokens of a page item; K and V in one
    int32_t page_items;
};
// rows: element type of q, k, v (KVC_BF16, KVC_FP16, KVC_FP32); cache: the handle's dtype
cudaError_t launch_rope(RopeArgs a, int rows, int cache, int num_sms, cudaStream_t s);

// ---- attention over the 8-bit cache (kvc_e4m3_attn.cu, kvc_e4m3_rows.cu) -----------------------
constexpr int E4M3_D = 128;
struct E4m3Args {
    const uint8_t *K, *V;        // the layer's pools
    const float *k_scale, *v_scale;
    const int32_t *block_table;
    const void *q;               // [total, H, 128]
    void *out;
    const int32_t *cu_seqlens;   // [B + 1], or null: one token of each sequence
    const int32_t *cache_index;  // [B]: rows before the call's tokens (+ index_offset)
    int32_t *err;
    int32_t index_offset, total, bf16;
    int32_t B, H, H_kv, group, max_ctx, max_blocks, num_blocks;
    float scale_log2;            // log2(e) / sqrt(128)
};

constexpr int E4M3_MAX_CTAS = 160, E4M3_SLOT = 256;  // size the workspace: CTAs, query rows of a piece
struct E4m3TcArgs : E4m3Args {
    int32_t *tickets;            // [E4M3_MAX_CTAS], zero between launches: pieces of the segment that a CTA starts
    float2 *part_ml;             // [2 E4M3_MAX_CTAS][E4M3_SLOT]: reference and sum of a piece's pairs (head, query row)
    float *part_acc;             // [2 E4M3_MAX_CTAS][E4M3_SLOT][128]: their accumulators
    int32_t nh;                  // KV heads of a tile: 1, 2, 4 or 8
    // How a head's query rows are cut: tt tokens of all g heads (gg = g, gt = 1), or,
    // where g passes the rows of a tile, gt parts of gg of one token's heads.
    int32_t tt, gt, gg;
    int32_t gg_inverse;          // 2^16 / gg, rounded up: r / gg = r * gg_inverse >> 16 for r < 64
    int32_t cost;                // places of the line for a segment's start and end
    int32_t groups, shift;       // H_kv / nh; log2 of the keys of a tile
    int32_t n_stages, min_share; // tiles of a CTA's share, at least
    int32_t layer_block;         // first block of the layer in the maps
    int32_t read_once;           // no two segments read the same rows
    unsigned long long timeout_ns;  // limit of a wait, but for those before the block leaves
    CUtensorMap tm_k, tm_v;      // (128, 16 rows, H_kv, L * num_blocks), boxes of nh heads of a block
};

struct E4m3Workspace {
    uint64_t tickets, part_ml, part_acc, total;
};
inline E4m3Workspace e4m3_workspace() {
    E4m3Workspace w;
    w.tickets = 256;
    w.part_ml = align256(w.tickets + 4 * E4M3_MAX_CTAS);
    w.part_acc = w.part_ml + 2ull * E4M3_MAX_CTAS * E4M3_SLOT * 8;
    w.total = w.part_acc + 2ull * E4M3_MAX_CTAS * E4M3_SLOT * E4M3_D * 4;
    return w;
}

// rows: query rows that a tile has per head, a power of two up to 64; nh * rows <= 32, or nh = 1
cudaError_t e4m3_set_max_smem(int max_smem);  // once per handle
cudaError_t launch_e4m3_attn(E4m3TcArgs &a, int rows, int grid, int max_smem, cudaStream_t s);
// nh = 1, tt = 2 (128 / group), gt = 1
cudaError_t e4m3_rows_set_max_smem();
cudaError_t launch_e4m3_rows(const E4m3TcArgs &a, int grid, cudaStream_t s);

#ifdef __CUDACC__
namespace dev {

// Two floats to e4m3 codes, round to nearest even, saturating; lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two codes as an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(c)));
    return r;
}

// Two fp32 operations in one instruction, each rounded to nearest.
#define KVC_PAIR_OP(NAME, OP)                                                                                         \
    __device__ __forceinline__ float2 NAME(float2 a, float2 b) {                                                      \
        float2 d;                                                                                                     \
        asm(OP ".rn.f32x2 %0, %1, %2;"                                                                                \
            : "=l"(reinterpret_cast<uint64_t &>(d))                                                                   \
            : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));                            \
        return d;                                                                                                     \
    }
KVC_PAIR_OP(mul2, "mul")
KVC_PAIR_OP(add2, "add")
KVC_PAIR_OP(sub2, "sub")
#undef KVC_PAIR_OP
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}

// Two products that are rounded by themselves: the compiler contracts a paired product
// with a sum behind it, whatever its rounding says.
__device__ __forceinline__ float2 product2(float2 a, float2 b) { return make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y)); }

// The larger magnitude; a NaN stays.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}

// One sequence of a packed call.
struct PackedSeq {
    int lo, n, c;  // first packed row, tokens, cached rows
    bool bad;
};

// cu null: T tokens of each sequence.
template <class A>
__device__ __forceinline__ PackedSeq packed_seq(const A &a, int T, int b) {
    PackedSeq s;
    s.c = a.cache_index ? ld(a.cache_index + b) : 0;
    s.bad = s.c < 0;  // (before the offset, which may leave the 32 bits)
    if (!s.bad) s.c += a.index_offset;
    int hi;
    if (a.cu_seqlens) {
        s.lo = ld(a.cu_seqlens + b);
        hi = ld(a.cu_seqlens + b + 1);
    } else {
        s.lo = b * T;
        hi = s.lo + T;
    }
    s.bad = s.bad || s.lo < 0 || hi < s.lo || hi > a.total || s.c < 0 || s.c > a.max_ctx || hi - s.lo > a.max_ctx - s.c;
    s.n = s.bad ? 0 : hi - s.lo;
    return s;
}

}  // namespace dev
#endif

}  // namespace kvc
