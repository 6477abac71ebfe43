// kvc_rows_tc.cuh -- attention of several new tokens per sequence on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory):
// packed prompts and drafted trees over contiguous or paged caches, 16-bit
// types, head widths 64 and 128.
//
// Work item: up to 2 TB new tokens (TB = 128 / g) of one (sequence, KV head)
// as two tiles of 128 query rows -- tile x holds tokens [t0 + x TB, t0 + (x + 1)
// TB), row r = tt g + i of it is token tt, head i of the group, which is how
// one box of a tensor map brings them in either layout -- and the keys they can
// see in tiles of 128: the cached rows, then the new rows.  Both query tiles
// share every K and V tile; an item with at most TB tokens has one query tile,
// and two streams x share its key tiles instead, even ones and odd ones
// ("folded": their accumulators are added at the end).  Per key tile j and
// stream x:
//   S_x = Q_x . K_j^T    tcgen05.mma, M = 128, N = 128, K = d_h; both operands
//                        K-major in shared memory
//   softmax              one thread per query row (its TMEM lane): the row's
//                        128 scores in registers, mask, running max and sum
//                        in fp32 (log2 domain); the probabilities, rounded to
//                        the cache type, overwrite S_x's columns
//   O_x += P_x . V_j     tcgen05.mma with A = P_x from tensor memory, B = V_j
//                        as stored (MN-major)
// One warp issues all MMAs, in the order PV_A(j) S_A(j+1) PV_B(j) S_B(j+1)
// (folded: PV_A(j) S_A(j+2) PV_B(j+1) S_B(j+3)): while one stream is in its
// softmax the tensor cores work on the other.  P is handed over in halves: PV is
// at the first 64 keys while the softmax is at the others.  MMAs of one thread
// complete in order, so the barrier of a stream's next S also says that its PV is
// done: the softmax may rescale O_x then, which it does only when a tile's maximum
// exceeds the reference by more than 2^8.
//
// Split: all key tiles of all items form one line (item order: sequence, KV
// head, token block) that is cut into equal shares, one per CTA, so that
// ragged batches, long contexts with few rows and causal triangles all balance
// with no planning on the host.  An item cut by a boundary leaves its
// unnormalised accumulator and (max, sum) per piece in the workspace, and
// rows_combine_kernel folds the pieces.
//
// Warps: 0-3 softmax and epilogue of stream A, 4-7 of stream B; 8 copies K and 11
// V (one ring, in the order in which the MMAs take them); 9 issues the MMAs and
// owns tensor memory; 10 walks the items, hands them to the others and copies
// their query rows.  Cached rows of a contiguous cache and new rows come as
// boxes of 128 rows x 64 columns.  A page of 16 rows (of one KV head) comes as one
// box of half pages x column blocks x 8 rows x 64 columns: the eight-row groups
// of a column block then lie 2048 bytes apart (d_h = 128) across all pages of a
// tile, which the MMA's descriptors take as they are.
//
// A tile that is not full holds foreign rows behind its own: their scores are
// masked, and their V rows are zeroed in shared memory before the PV (0 times
// an infinity or NaN would not be 0).  In the same way the rows of a
// partly visible tile are searched for infinities and NaN, which must reach
// only the rows that see them: such elements are zeroed, and the epilogue of
// the rows that see them adds them back.
//
// Measured (bf16, 32 heads over 8, d_h 128): 16,384 tokens 1.47 ms, 1.50 PFLOP/s,
// bound by the hand-overs between a stream's MMAs and its softmax; 8 prompts of
// 64-2,048 tokens over up to 1,500 rows in pages 222 us, the same and about 5 us
// at each item's ends; 16 trees of 32 tokens over 1,024-8,192 rows in pages 68 us,
// 5.0 TB/s, bound by the copies and the start and end of the launch.
//
// Every wait is bounded; a timeout records KVC_ERR_TIMEOUT, every role leaves
// its loop, MMAs and copies in flight are waited for and tensor memory is freed
// before the CTA exits.
#pragma once

#include <type_traits>

#include "kvc_decode_mma.cuh"
#include "kvc_prefill_tc.cuh"
#include "kvc_rows.cuh"
#include "kvc_tcgen05.cuh"

namespace kvc {

template <int D>
struct RowsTcCfg {
    static constexpr int BM = 128, BN = 128;
    static constexpr int CB = D / 64;              // 128-byte column blocks of a row
    static constexpr int ROW_BYTES = D * 2;
    static constexpr int CHUNKS = ROW_BYTES / 16;
    static constexpr int BLK = 128 * 128;          // one column block of a 128-row tile
    static constexpr int TILE_BYTES = CB * BLK;    // a Q, K or V tile
    static constexpr int NS = D == 64 ? 10 : 5;    // stages of the K / V ring
    static constexpr int RING_OFF = 2 * TILE_BYTES;
    static constexpr int BAR_OFF = RING_OFF + NS * TILE_BYTES;
    // full[NS], empty[NS], s_full[2], p_full[2], o_full[2], o_free[2], q_full,
    // q_empty, item_full[2], item_empty[2], fold, mma_done, p_half[2]
    static constexpr int NBAR = 2 * NS + 18;
    static constexpr int ITEM_OFF = BAR_OFF + 8 * NBAR + 8 + 24;  // after the TMEM address and the flags
    static constexpr int FOLD_OFF = ITEM_OFF + 2 * 64;            // folded items: stream A's (max, sum) of each row
    static constexpr int SMEM = 1024 + FOLD_OFF + 128 * 8;
    static constexpr int K_WARP = 8, MMA_WARP = 9, ITEM_WARP = 10, V_WARP = 11;
    static constexpr int THREADS = 12 * 32;
    // registers: 168 a thread at launch; the softmax warpgroups take from the third
    static constexpr int REGS_SOFTMAX = 208, REGS_OTHER = 88;
    static_assert(2 * REGS_SOFTMAX + REGS_OTHER == 3 * 168, "the launch's registers");
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t S_COL = 0, O_COL = 256;  // S_A, S_B (128 columns each), O_A, O_B (D each)
    static constexpr float RESCALE_LOG2 = 8.f;
    // fp16 probabilities are held 2^7 times as large, next to the type's end (at
    // most 2^(7 + RESCALE_LOG2) of 65504): at their own size those below 2^-25 of the
    // reference would be zeros for V, though not in the sum, and 32,000 of them
    // beside one dominant key as much as 2^-10 of the result.
    static constexpr float P_SHIFT_LOG2_F16 = 7.f;
    static_assert(NS >= 5, "the copy warps' waits (below)");
    static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");

    // 16-byte chunk c of row r of a tile of 128 consecutive rows
    __device__ __forceinline__ static uint32_t swz(uint32_t tile, int r, int c) {
        return tile + uint32_t(c >> 3) * BLK + uint32_t(r) * 128 + (uint32_t((c & 7) ^ (r & 7)) << 4);
    }
    // the same for a tile of eight pages, each as half pages of CB column blocks of eight rows
    __device__ __forceinline__ static uint32_t swz_paged(uint32_t tile, int r, int c) {
        return tile + uint32_t(r >> 3) * (CB * 1024) + uint32_t(c >> 3) * 1024 + uint32_t(r & 7) * 128 +
               (uint32_t((c & 7) ^ (r & 7)) << 4);
    }
};

// dev::mbar_wait_bounded, but a try may suspend the warp for up to 100 us, and 64
// tries pass before the abort flag and the timer are looked at: reading them
// between tries cost each hand-over between the softmax and the MMAs about 400
// cycles, a tenth of a key tile's time, and tries that return sooner take issue
// slots from the softmax (one user's tree 14.77 -> 14.59 us, long prompt 1 %).
__device__ __forceinline__ bool rows_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 100000;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}
__device__ __forceinline__ bool rows_wait(uint32_t bar, uint32_t parity, const volatile int *abort, unsigned long long timeout_ns) {
    if (rows_try(bar, parity)) return true;
    const uint64_t t0 = dev::global_timer_ns();
    for (uint32_t it = 0; it < (1u << 24); ++it) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (rows_try(bar, parity)) return true;
        if (*abort) return false;
        if (dev::global_timer_ns() - t0 > timeout_ns) return false;
    }
    return false;
}

// A piece of work as the roles see it: tokens [t0, t0 + ntok) of (b, kv) against
// key tiles [j0, j1).  b < 0: no more work.
struct RowsItem {
    int b, kv, t0, ntok;
    int c, n, row0;   // the sequence: cached rows, new tokens, first packed row
    int vis;          // new keys some row of the item sees: [0, vis)
    int j0, j1;
    int np;           // tiles of cached rows: tile j < np holds rows [128 j, ...), the others new rows
    int slot;         // partial slot of a piece, -1: the whole item
};
static_assert(sizeof(RowsItem) <= 64, "item slot");

// ---- the line of key tiles ------------------------------------------------------

// Length on the line of the first q token blocks (of ti tokens) of one KV head
// of a sequence: a.item_cost each for an item's start and end, and its key
// tiles -- the cached ones, and of the new ones all under a mask, otherwise
// those up to its last token.  (Int: 64 bits where the line is measured, 32 in
// one that is known to stay below ROWS_MAX_LINE.)
template <typename Int>
__device__ __forceinline__ Int rows_prefix(const RowsTcArgs &a, const RowsSeq &s, int ti, int q) {
    const Int base = Int(q) * (a.item_cost + (s.c + 127) / 128), kt = (s.n + 127) / 128;
    if (a.tree_mask) return base + q * kt;
    if (ti > 128) {  // 256 tokens: block k (from 1) sees 2 k tiles, the last one kt
        const Int nblk = (s.n + ti - 1) / ti;
        return base + (q < nblk ? Int(q) * (q + 1) : nblk * (nblk - 1) + kt);
    }
    const int m = 128 / ti;
    if (m * ti == 128) {  // m blocks a tile
        const Int full = q / m, rest = q - full * m;
        return base + m * full * (full + 1) / 2 + rest * (full + 1);
    }
    Int sum = base;
    for (int k = 1; k <= q; ++k) sum += (min(s.n, k * ti) + 127) / 128;
    return sum;
}

template <typename Int>
__device__ __forceinline__ Int rows_seq_length(const RowsTcArgs &a, const RowsSeq &s, int ti) {
    return s.n == 0 ? 0 : rows_prefix<Int>(a, s, ti, (s.n + ti - 1) / ti);
}

__device__ __forceinline__ int rows_block_tiles(const RowsArgs &a, const RowsSeq &s, int ti, int qb) {
    const int end = a.tree_mask ? s.n : min(s.n, (qb + 1) * ti);
    return (s.c + 127) / 128 + (end + 127) / 128;
}

// A place on the line: token block qb of (b, kv), an item that starts at item0.
struct RowsPlace {
    int b, kv, qb, item0;
    RowsSeq s;

    __device__ __forceinline__ void next(const RowsTcArgs &a, int ti) {
        item0 += a.item_cost + rows_block_tiles(a, s, ti, qb);
        ++qb;
        if (qb * int64_t(ti) < s.n) return;
        qb = 0;
        if (++kv < a.H_kv) return;
        kv = 0;
        do {
            if (++b >= a.B) return;
            s = rows_seq(a, b);
        } while (s.n == 0);
    }
};

// This CTA's stretch [begin, end) of the line, `place` at its start, and the
// share that cuts the line.  Boundary i is at i shares, moved back to the start
// of its item if that is too short to be worth cutting or the boundary lies
// before its first tile; even lanes of the warp work out this CTA's boundary,
// odd lanes the next one's.
__device__ __forceinline__ void rows_plan(const RowsTcArgs &a, int ti, int lane, int &share, int &begin, int &end, RowsPlace &place) {
    constexpr unsigned FULL = 0xffffffffu;
    int mine = 0;  // length of this lane's sequence (of the last batch of 32)
    int64_t sum = 0;  // (capped, so that it cannot overflow)
    for (int i = lane; i < a.B; i += 32) {
        const int64_t length = rows_seq_length<int64_t>(a, rows_seq(a, i), ti) * a.H_kv;
        sum += min(length, int64_t(1) << 32);
        mine = int(length);
    }
    // A line past ROWS_MAX_LINE is recorded, and no item taken.
    if (__reduce_add_sync(FULL, int(min(sum >> 20, int64_t(1) << 20))) > (ROWS_MAX_LINE >> 20)) {
        if (blockIdx.x == 0 && lane == 0) dev::record_error(a.err, ERR_DEVICE_INDEX);
        share = a.min_share;
        begin = end = 0;
        return;
    }
    const int total = __reduce_add_sync(FULL, int(sum));
    share = (total + int(gridDim.x) - 1) / int(gridDim.x);
    if (share < a.min_share) share = a.min_share;
    const int64_t at64 = int64_t(share) * (blockIdx.x + (lane & 1));
    const int at = at64 < total ? int(at64) : total;
    // the sequence that holds it
    int base = 0, seq0 = 0, per = 1, b = -1;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        if (a.B > 32) mine = b0 + lane < a.B ? rows_seq_length<int>(a, rows_seq(a, b0 + lane), ti) * a.H_kv : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += y;
        }
        incl += base;
        const int at_a = __shfl_sync(FULL, at, 0), at_b = __shfl_sync(FULL, at, 1);
        const unsigned hit_a = __ballot_sync(FULL, incl > at_a), hit_b = __ballot_sync(FULL, incl > at_b);
        const unsigned hit = lane & 1 ? hit_b : hit_a;
        const int l = hit ? __ffs(hit) - 1 : 0;
        const int length = __shfl_sync(FULL, mine, l), last = __shfl_sync(FULL, incl, l);
        if (hit && b < 0) {
            b = b0 + l;
            per = length / a.H_kv;
            seq0 = last - length;
        }
        base = __shfl_sync(FULL, incl, 31);
        if (hit_a && hit_b) break;
    }
    RowsPlace p;
    p.b = b;
    p.kv = p.qb = p.item0 = 0;
    int bound = total;
    if (b >= 0) {
        p.s = rows_seq(a, b);
        p.kv = (at - seq0) / per;
        p.item0 = seq0 + p.kv * per;
        // the last block that starts at or before `at`
        if (a.tree_mask) {
            p.qb = (at - p.item0) / (a.item_cost + rows_block_tiles(a, p.s, ti, 0));
            p.item0 += rows_prefix<int>(a, p.s, ti, p.qb);
        } else if (128 % ti == 0 || ti > 128) {
            int lo = 0, hi = (p.s.n + ti - 1) / ti - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.item0 + rows_prefix<int>(a, p.s, ti, mid) <= at) lo = mid; else hi = mid - 1;
            }
            p.qb = lo;
            p.item0 += rows_prefix<int>(a, p.s, ti, lo);
        } else {
            for (;; ++p.qb) {
                const int t = a.item_cost + rows_block_tiles(a, p.s, ti, p.qb);
                if (at < p.item0 + t) break;
                p.item0 += t;
            }
        }
        bound = rows_block_tiles(a, p.s, ti, p.qb) <= a.split_min || at <= p.item0 + a.item_cost ? p.item0 : at;
    }
    begin = __shfl_sync(FULL, bound, 0);
    end = __shfl_sync(FULL, bound, 1);
    place.b = __shfl_sync(FULL, p.b, 0);
    place.kv = __shfl_sync(FULL, p.kv, 0);
    place.qb = __shfl_sync(FULL, p.qb, 0);
    place.item0 = __shfl_sync(FULL, p.item0, 0);
    if (begin < end) place.s = rows_seq(a, place.b);
}

// 16 lanes x 32 columns of tensor memory, as accumulator fragments: thread i
// receives, of column block n (8 columns), lane i / 4 columns 2 (i mod 4), + 1 in
// r[4 n], r[4 n + 1], and lane i / 4 + 8 in r[4 n + 2], r[4 n + 3].
__device__ __forceinline__ void rows_tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void rows_reg_fence16(uint32_t (&r)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(r[e]));
}
// Transposes the 4 x 4 words that the four lanes of a quad hold.
__device__ __forceinline__ void rows_quad_transpose(uint32_t (&w)[4], int lane) {
    const bool odd = lane & 1, up = lane & 2;
    uint32_t x = odd ? w[0] : w[1], y = odd ? w[2] : w[3];
    x = __shfl_xor_sync(0xffffffffu, x, 1);
    y = __shfl_xor_sync(0xffffffffu, y, 1);
    (odd ? w[0] : w[1]) = x;
    (odd ? w[2] : w[3]) = y;
    x = up ? w[0] : w[2], y = up ? w[1] : w[3];
    x = __shfl_xor_sync(0xffffffffu, x, 2);
    y = __shfl_xor_sync(0xffffffffu, y, 2);
    (up ? w[0] : w[2]) = x;
    (up ? w[1] : w[3]) = y;
}

__device__ __forceinline__ void rows_tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void rows_tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Folded items take the tiles in the order K_0 K_1 V_0 K_2 V_1 ... V_(n-2) V_(n-1),
// the others K_0 V_0 K_1 V_1 ...: places of tile j's K and V among the item's 2 n.
__device__ __forceinline__ int rows_k_place(bool fold, int j) { return fold && j > 0 ? 2 * j - 1 : 2 * j; }
__device__ __forceinline__ int rows_v_place(bool fold, int j, int n) { return fold ? min(2 * j + 2, 2 * n - 1) : 2 * j + 1; }

// One bit per score column of a tile: the keys [0, lim) of 128.
__device__ __forceinline__ uint32_t lead_word(int lim, int k) {
    const int m = lim - 32 * k;
    return m >= 32 ? 0xffffffffu : m <= 0 ? 0u : (1u << m) - 1u;
}
// Infinities and NaN among the eight 16-bit elements of a vector.
template <typename T>
__device__ __forceinline__ bool not_finite(const uint4 &v) {
    constexpr uint32_t E = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad = bad || (w[i] & E) == E || ((w[i] >> 16) & E) == E;
    return bad;
}
template <typename T>
__device__ __forceinline__ uint4 finite_only(uint4 v) {
    constexpr uint32_t E = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    uint32_t *w = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & E) == E) w[i] &= 0xffff0000u;
        if (((w[i] >> 16) & E) == E) w[i] &= 0x0000ffffu;
    }
    return v;
}

// Shared-memory descriptors (kvc_tcgen05.cuh) with the 128-byte swizzle in two
// halves: the start address (and leading offset), and the rest.
__host__ __device__ constexpr uint32_t rows_desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }
__device__ __forceinline__ uint64_t rows_desc(uint32_t lo, uint32_t hi) { return (uint64_t(hi) << 32) | lo; }

__device__ __forceinline__ bool rows_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(RowsTcCfg<D>::THREADS, 1) rows_tc_kernel(const __grid_constant__ RowsTcArgs a) {
    using C = RowsTcCfg<D>;
    using Ops = MmaOps<T>;
    constexpr int BN = C::BN, CB = C::CB, NS = C::NS, BLK = C::BLK;
    constexpr unsigned FULL = 0xffffffffu;
    constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t IDESC_S = tc::idesc_f16_f32acc(BF16, 128, BN, false, false);
    constexpr uint32_t IDESC_O = tc::idesc_f16_f32acc(BF16, 128, D, false, true);

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (dev::smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = dev::smem_addr(smem);
    const uint32_t ring = sb + C::RING_OFF;
    const uint32_t full = sb + C::BAR_OFF, empty = full + 8 * NS, s_full = empty + 8 * NS, p_full = s_full + 16,
                   o_full = p_full + 16, o_free = o_full + 16, q_full = o_free + 16, q_empty = q_full + 8,
                   item_full = q_empty + 8, item_empty = item_full + 16, fold_bar = item_empty + 16, mma_done = fold_bar + 8, p_half = mma_done + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::BAR_OFF + 8 * C::NBAR);
    volatile int *flags = reinterpret_cast<volatile int *>(smem + C::BAR_OFF + 8 * C::NBAR + 8);  // abort, then odd[4]
    volatile int *odd = flags + 1;  // item i met infinities or NaN: odd[i % 4]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.group, TB = 128 / G, TI = 2 * TB;

    if (threadIdx.x == 32) {
        dev::prefetch_tensormap(&a.tm_q);
        dev::prefetch_tensormap(&a.tm_k);
        dev::prefetch_tensormap(&a.tm_v);
        dev::prefetch_tensormap(&a.tm_k_new);
        dev::prefetch_tensormap(&a.tm_v_new);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            dev::mbar_init(full + 8 * s, 1);
            dev::mbar_init(empty + 8 * s, 1);  // the commit behind the stage's last MMA
        }
        for (int x = 0; x < 2; ++x) {
            dev::mbar_init(s_full + 8 * x, 1);       // S_x is in tensor memory, PV_x before it done
            dev::mbar_init(p_full + 8 * x, 4);       // the four softmax warps wrote P_x
            dev::mbar_init(p_half + 8 * x, 4);       // its first 64 columns
            dev::mbar_init(o_full + 8 * x, 1);       // the item's last PV_x is done
            dev::mbar_init(o_free + 8 * x, 4);       // its accumulator is read (folded items: by stream B's warps)
            dev::mbar_init(item_full + 8 * x, 1);
            dev::mbar_init(item_empty + 8 * x, 11);  // every other warp has read the item
        }
        dev::mbar_init(q_full, 1);
        dev::mbar_init(q_empty, 1);   // the item's last S has read Q
        dev::mbar_init(fold_bar, 4);  // stream A's (max, sum) are in shared memory
        dev::mbar_init(mma_done, 1);
        for (int i = 0; i < 5; ++i) flags[i] = 0;
        dev::fence_mbar_init();
    }
    if (warp == C::MMA_WARP) {
        tc::tmem_alloc(dev::smem_addr(tmem_slot), C::TMEM_COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    dev::allow_dependents();
    dev::grid_dependency_wait();

    auto give_up = [&]() {
        if (lane == 0) {
            if (!flags[0]) dev::record_error(a.err, ERR_TIMEOUT);
            flags[0] = 1;
        }
    };
    // the k-th item (k = 0, 1, ...) out of its slot; false on a timeout
    auto take_item = [&](int k, RowsItem &it) {
        const bool w = rows_wait(item_full + 8 * (k & 1), uint32_t(k >> 1) & 1, flags, a.timeout_ns);
        if (!w) return false;
        it = *reinterpret_cast<const RowsItem *>(smem + C::ITEM_OFF + 64 * (k & 1));
        return true;
    };
    uint32_t filled = 0, filled_phase = 0;  // copy warps: stages filled, and the phase of each last filling
    int queries = 0;                        // items whose queries were copied
    if (warp >= C::K_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
        if (warp == C::ITEM_WARP) {
            // ------------------------------------------------------------ items and their queries
            int share, begin, end;
            RowsPlace w;
            rows_plan(a, TI, lane, share, begin, end, w);
            const int me = int(blockIdx.x);
            RowsCut cut = {0, 0, 0, 0, 0};
            bool ok = true;
            int at = begin;
            for (int k = 0; ok; ++k) {
                RowsItem it;
                it.b = -1;
                if (at < end) {
                    const int tiles = rows_block_tiles(a, w.s, TI, w.qb);
                    it.b = w.b;
                    it.kv = w.kv;
                    it.t0 = w.qb * TI;
                    it.ntok = min(TI, w.s.n - it.t0);
                    it.c = w.s.c;
                    it.n = w.s.n;
                    it.row0 = int(w.s.row0);
                    it.vis = a.tree_mask ? w.s.n : it.t0 + it.ntok;
                    it.np = (w.s.c + 127) / 128;
                    it.j0 = max(0, at - w.item0 - a.item_cost);
                    it.j1 = min(end - w.item0 - a.item_cost, tiles);
                    // pieces: the one that starts an item takes the CTA's second slot,
                    // one that goes on with it the first
                    it.slot = it.j0 == 0 && it.j1 == tiles ? -1 : 2 * me + (it.j0 == 0 ? 1 : 0);
                    if (it.j0 == 0 && it.j1 < tiles)
                        cut = {(w.item0 + a.item_cost + tiles - 1) / share - me + 1, it.b, it.kv, it.t0, it.ntok};
                    at = w.item0 + a.item_cost + it.j1;
                }
                if (k >= 2) ok = __all_sync(FULL, rows_wait(item_empty + 8 * (k & 1), uint32_t((k >> 1) - 1) & 1, flags, a.timeout_ns));
                if (!ok) break;
                if (lane == 0) {
                    odd[k & 3] = 0;  // (every role has left item k - 2)
                    *reinterpret_cast<RowsItem *>(smem + C::ITEM_OFF + 64 * (k & 1)) = it;
                    dev::mbar_arrive(item_full + 8 * (k & 1));
                }
                if (it.b < 0) break;
                if (k >= 1) ok = __all_sync(FULL, rows_wait(q_empty, uint32_t(k - 1) & 1, flags, a.timeout_ns));
                if (!ok) break;
                if (lane == 0) {
                    // one box of TB tokens x g heads per column block and query tile
                    const int nx = it.ntok > TB ? 2 : 1;
                    dev::mbar_arrive_expect_tx(q_full, uint32_t(nx * CB * G * TB) * 128);
                    for (int x = 0; x < nx; ++x)
#pragma unroll
                        for (int cb = 0; cb < CB; ++cb) {
                            const uint32_t dst = sb + x * C::TILE_BYTES + cb * BLK;
                            if (a.cu_seqlens)
                                dev::tma_load_3d(dst, &a.tm_q, cb * 64, it.kv * G, it.row0 + it.t0 + x * TB, q_full);
                            else
                                dev::tma_load_4d(dst, &a.tm_q, cb * 64, it.kv * G, it.t0 + x * TB, it.b, q_full);
                        }
                }
                queries = k + 1;
                __syncwarp();
                if (at < end) w.next(a, TI);
            }
            if (lane == 0) a.cuts[me] = cut;
            if (me == 0)  // sequences whose arguments are out of range
                for (int i = lane; i < a.B; i += 32)
                    if (rows_seq(a, i).bad) dev::record_error(a.err, ERR_DEVICE_INDEX);
            if (!ok) give_up();
        } else if (warp == C::K_WARP || warp == C::V_WARP) {
            // ------------------------------------------------------------ K and V copies
            // One warp each: sixteen boxes of pages a tile pair from one warp were too
            // slow (tree steps of 16 users on pages 71 -> 67 us).  The waits: stages
            // are let go in ring order and a warp's places are at most three apart, so
            // when it waits for place p - NS, place p - 2 NS is known to be free.
            const bool v = warp == C::V_WARP;
            // cached rows that one item reads leave L2 to what is read again
            const uint64_t pol = a.read_once ? dev::l2_evict_first_policy() : dev::l2_evict_normal_policy();
            const CUtensorMap *m_cache = v ? &a.tm_v : &a.tm_k, *m_new = v ? &a.tm_v_new : &a.tm_k_new;
            bool ok = true;
            RowsItem it;
            uint32_t base = 0;  // ring places of the items before
            for (int k = 0; ok; ++k) {
                ok = __all_sync(FULL, take_item(k, it));
                __syncwarp();
                if (!ok) break;
                if (lane == 0) dev::mbar_arrive(item_empty + 8 * (k & 1));
                if (it.b < 0) break;
                const int n = it.j1 - it.j0;
                const bool fold = it.ntok <= TB && n > 1;
                // a page's number is looked up a tile ahead
                auto page_of = [&](int jt) {
                    const int blk = 8 * jt + lane;
                    if (!a.block_table || lane >= 8 || jt >= it.np || blk * 16 >= it.c) return 0;
                    return dev::ld(a.block_table + int64_t(it.b) * a.max_blocks + blk);
                };
                int next_page = page_of(it.j0);
                for (int j = 0; j < n; ++j) {
                    const int page = next_page, jt = it.j0 + j;
                    next_page = page_of(jt + 1);
                    const uint32_t place = base + (v ? rows_v_place(fold, j, n) : rows_k_place(fold, j));
                    const uint32_t s = place % NS, gen = place / NS;
                    if (gen > 0) ok = __all_sync(FULL, rows_wait(empty + 8 * s, (gen - 1) & 1, flags, a.timeout_ns));
                    if (!ok) break;
                    filled |= 1u << s;
                    filled_phase = (filled_phase & ~(1u << s)) | ((gen & 1) << s);
                    const uint32_t dst = ring + s * C::TILE_BYTES, bar = full + 8 * s;
                    if (jt >= it.np) {  // new rows
                        const int row = 128 * (jt - it.np);
                        if (lane == 0) {
                            dev::mbar_arrive_expect_tx(bar, C::TILE_BYTES);
#pragma unroll
                            for (int cb = 0; cb < CB; ++cb)
                                if (a.cu_seqlens)
                                    dev::tma_load_3d(dst + cb * BLK, m_new, cb * 64, it.kv, it.row0 + row, bar);
                                else
                                    dev::tma_load_3d(dst + cb * BLK, m_new, cb * 64, row, it.b * a.H_kv + it.kv, bar);
                        }
                    } else if (!a.block_table) {
                        if (lane == 0) {
                            dev::mbar_arrive_expect_tx(bar, C::TILE_BYTES);
#pragma unroll
                            for (int cb = 0; cb < CB; ++cb)
                                dev::tma_load_3d(dst + cb * BLK, m_cache, cb * 64, 128 * jt, a.seg_base + it.b * a.H_kv + it.kv, bar, pol);
                        }
                    } else {
                        // the pages that hold cached rows, one lane each; a page out of
                        // range is recorded and read as zeros (behind the pool's end)
                        const int pages = min(8, (it.c - 128 * jt + 15) / 16);
                        if (lane == 0) dev::mbar_arrive_expect_tx(bar, uint32_t(pages) * CB * 2048);
                        __syncwarp();
                        if (lane < pages) {
                            const bool in = page >= 0 && page < a.num_blocks;
                            if (!in) dev::record_error(a.err, ERR_DEVICE_INDEX);
                            dev::tma_load_5d(dst + lane * (CB * 2048), m_cache, 0, 0, 0, 0,
                                             in ? a.seg_base + page * a.H_kv + it.kv : a.pool_end, bar, pol);
                        }
                    }
                    __syncwarp();
                }
                base += 2 * n;
            }
            if (!ok) give_up();
        } else {
            // ------------------------------------------------------------ MMAs
            // One thread waits and issues.  Tiles are taken in ring order, ahead of
            // the wait for P: what stands between that wait and the MMAs is idle time
            // of the tensor cores.  (A whole warp with one elected lane issuing has
            // to be brought together behind every wait and issue -- operands are in
            // registers that the warp shares -- and measured 2 % slower.)
            if (rows_elect()) {
                constexpr uint32_t HI1 = rows_desc_hi(1024), HI2 = rows_desc_hi(2048);
                bool ok = true;
                RowsItem it;
                uint32_t stage = 0, phase = 0;                                   // next tile of the ring
                uint32_t tiles_a = 0, tiles_b = 0, items_a = 0, items_b = 0;     // of each stream
                auto wait = [&](uint32_t bar, uint32_t parity) { ok = ok && rows_wait(bar, parity, flags, a.timeout_ns); };
                auto take_tile = [&]() {
                    wait(full + 8 * stage, phase);
                    const uint32_t s = stage;
                    if (++stage == NS) stage = 0, phase ^= 1;
                    return s;
                };
                auto issue_s = [&](int x, int qx, uint32_t s, bool paged) {
                    const uint32_t kt = (ring + s * C::TILE_BYTES) >> 4, qt = (sb + qx * C::TILE_BYTES) >> 4, s_t = tmem + C::S_COL + 128 * x;
                    if (CB == 2 && paged) {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            tc::mma_f16_ss(s_t, rows_desc(qt + (((ks >> 2) * BLK + (ks & 3) * 32) >> 4), HI1),
                                           rows_desc(kt + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), HI2), IDESC_S, ks > 0);
                    } else {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            tc::mma_f16_ss(s_t, rows_desc(qt + (((ks >> 2) * BLK + (ks & 3) * 32) >> 4), HI1),
                                           rows_desc(kt + (((ks >> 2) * BLK + (ks & 3) * 32) >> 4), HI1), IDESC_S, ks > 0);
                    }
                    tc::commit(s_full + 8 * x);
                };
                auto issue_pv = [&](int x, uint32_t s, bool paged, bool first, auto half) {  // 64 of the tile's keys
                    constexpr int K0 = 4 * decltype(half)::value;
                    const uint32_t vt = (ring + s * C::TILE_BYTES) >> 4, p_t = tmem + C::S_COL + 128 * x, o_t = tmem + C::O_COL + D * x;
                    if (CB == 2 && paged) {
#pragma unroll
                        for (int ks = K0; ks < K0 + 4; ++ks)
                            tc::mma_f16_ts(o_t, p_t + 8 * ks, rows_desc(vt + ((ks * 4096) >> 4) + ((1024 >> 4) << 16), HI2),
                                           IDESC_O, ks > 0 || !first);
                    } else {
#pragma unroll
                        for (int ks = K0; ks < K0 + 4; ++ks)
                            tc::mma_f16_ts(o_t, p_t + 8 * ks, rows_desc(vt + ((ks * 2048) >> 4) + ((BLK >> 4) << 16), HI1), IDESC_O, ks > 0 || !first);
                    }
                };
                for (int k = 0; ok; ++k) {
                    ok = take_item(k, it);
                    if (!ok) break;
                    dev::mbar_arrive(item_empty + 8 * (k & 1));
                    if (it.b < 0) break;
                    const int n = it.j1 - it.j0, nx = it.ntok > TB ? 2 : 1;
                    const bool fold = nx == 1 && n > 1;
                    const int cached = a.block_table ? it.np - it.j0 : 0;  // the item's tiles j < cached are pages
                    wait(q_full, uint32_t(k) & 1);
                    uint32_t sk = take_tile(), sv = 0;
                    if (!ok) break;
                    tc::fence_after();
                    issue_s(0, 0, sk, 0 < cached);
                    if (fold) {
                        tc::commit(empty + 8 * sk);
                        sk = take_tile();
                        if (!ok) break;
                        tc::fence_after();
                        issue_s(1, 0, sk, 1 < cached);
                    } else if (nx == 2) {
                        issue_s(1, 1, sk, 0 < cached);
                    }
                    tc::commit(empty + 8 * sk);
                    if (n == (fold ? 2 : 1)) tc::commit(q_empty);
                    const int steps = fold ? n : n * nx;
                    for (int u = 0; u < steps; ++u) {
                        const int x = fold || nx == 2 ? u & 1 : 0, j = fold || nx == 1 ? u : u >> 1;
                        const int jn = fold ? j + 2 : j + 1;  // the stream's next tile
                        const bool first = fold ? j < 2 : j == 0, take = fold || x == 0, release = fold || x == nx - 1;
                        if (take) {
                            sv = take_tile();
                            if (jn < n) sk = take_tile();
                        }
                        const uint32_t items = x ? items_b : items_a;
                        if (first && items > 0) wait(o_free + 8 * x, (items - 1) & 1);
                        const uint32_t ph = (x ? tiles_b : tiles_a)++ & 1;
                        wait(p_half + 8 * x, ph);
                        if (!ok) break;
                        tc::fence_after();
                        issue_pv(x, sv, j < cached, first, std::integral_constant<int, 0>());
                        wait(p_full + 8 * x, ph);
                        if (!ok) break;
                        tc::fence_after();
                        issue_pv(x, sv, j < cached, first, std::integral_constant<int, 1>());
                        if (jn < n) {
                            if (release) tc::commit(empty + 8 * sv);
                            issue_s(x, fold ? 0 : x, sk, jn < cached);
                            if (release) {
                                tc::commit(empty + 8 * sk);
                                if (jn == n - 1) tc::commit(q_empty);
                            }
                        } else {
                            tc::commit(o_full + 8 * x);
                            if (release) tc::commit(empty + 8 * sv);
                            ++(x ? items_b : items_a);
                        }
                    }
                }
                if (!ok) {
                    if (!flags[0]) dev::record_error(a.err, ERR_TIMEOUT);
                    flags[0] = 1;
                }
                tc::commit(mma_done);  // every MMA is done before tensor memory is freed
                const volatile int never = 0;
                rows_wait(mma_done, 0, &never, a.timeout_ns);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
        const int x = warp >> 2, qd = warp & 3;
        const int r = 32 * qd + lane;           // query row = TMEM lane
        const int tt = r / G, head = r - tt * G;
        int frag_tok[4], frag_head[4];  // token and head of query row 8 i + lane / 4 of the warp's 32
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rr = 32 * qd + 8 * i + (lane >> 2);
            frag_tok[i] = rr / G;
            frag_head[i] = rr - frag_tok[i] * G;
        }
        const int H = a.H_kv * G;
        const uint32_t lane_base = uint32_t(qd * 32) << 16;
        const uint32_t s_t = tmem + lane_base + C::S_COL + 128 * x, o_t = tmem + lane_base + C::O_COL + D * x;
        const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
        bool ok = true;
        uint32_t st = 0, gt = 0, gi = 0, folds = 0;  // ring position; tiles, items and folded items of this stream so far
        for (int k = 0; ok; ++k) {
            // (the item is read where it is, which spares registers, and let go at its end)
            ok = __all_sync(FULL, rows_wait(item_full + 8 * (k & 1), uint32_t(k >> 1) & 1, flags, a.timeout_ns));
            if (!ok) break;
            const RowsItem &it = *reinterpret_cast<const RowsItem *>(smem + C::ITEM_OFF + 64 * (k & 1));
            if (it.b < 0) break;
            auto leave = [&]() {
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(item_empty + 8 * (k & 1));
            };
            const int n = it.j1 - it.j0;
            const bool two = it.ntok > TB, fold = !two && n > 1;
            if (x == 1 && !two && !fold) {  // nothing for stream B
                st += 2 * n;
                leave();
                continue;
            }
            const int qx = two ? x : 0;  // query tile of this stream
            const int t = it.t0 + qx * TB + tt;              // token
            const bool row_ok = tt < TB && qx * TB + tt < it.ntok;
            const bool warp_ok = __any_sync(FULL, row_ok);  // else the warp's lanes hold no query row
            float m_run = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            const int j_first = fold ? x : 0;
            for (int j = j_first; j < n; j += fold ? 2 : 1, ++gt) {
                // the V rows that a partly visible tile has to be rid of (below)
                const int jt = it.j0 + j;
                const bool is_new = jt >= it.np;
                const int key0 = 128 * (is_new ? jt - it.np : jt);         // first key, among the cached or the new rows
                const int nv = min(128, (is_new ? it.vis : it.c) - key0);  // the tile's own rows
                // does every row of the item see the whole tile?
                const bool partial = nv < 128 || (is_new && (a.tree_mask || key0 + 127 > it.t0));
                // V rows behind the tile's own are zeroed, infinities and NaN of rows that
                // not everybody sees set aside
                auto clean = [&]() {
                    const uint32_t sv = st + rows_v_place(fold, j, n);
                    if (!__all_sync(FULL, rows_wait(full + 8 * (sv % NS), (sv / NS) & 1, flags, a.timeout_ns))) return false;
                    const uint32_t vt = ring + (sv % NS) * C::TILE_BYTES;
                    const bool paged = a.block_table && !is_new;
                    for (int i = is_new ? r : r + nv * C::CHUNKS; i < 128 * C::CHUNKS; i += 128) {
                        const int row = i / C::CHUNKS, c16 = i % C::CHUNKS;
                        const uint32_t at = paged ? C::swz_paged(vt, row, c16) : C::swz(vt, row, c16);
                        if (row >= nv) {
                            dev::st_shared_v4(at, make_uint4(0u, 0u, 0u, 0u));
                        } else {
                            uint4 v;
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
                            if (not_finite<T>(v)) {
                                odd[k & 3] = 1;
                                dev::st_shared_v4(at, finite_only<T>(v));
                            }
                        }
                    }
                    dev::fence_proxy_async_smem();
                    return true;
                };
                // With two query tiles stream A's warps do it for both (PV_B follows PV_A,
                // which waits for them), while the tile's S is on its way: what the V
                // tile's stage held before is known to have arrived, as a later place's
                // has.  Not so ahead of an item's first S, nor in folded items, where the
                // other stream's tiles lie between.
                const bool to_clean = partial && (x == 0 || fold), early = j > j_first && !fold;
                if (to_clean && early) ok = clean();
                ok = ok && __all_sync(FULL, rows_wait(s_full + 8 * x, gt & 1, flags, a.timeout_ns));
                if (!ok) break;
                if (to_clean && !early) ok = clean();
                if (!ok) break;
                tc::fence_after();
                if (!warp_ok) {
                    __syncwarp();
                    if (lane == 0) {
                        dev::mbar_arrive(p_half + 8 * x);
                        dev::mbar_arrive(p_full + 8 * x);
                    }
                    continue;
                }
                // the columns that this row does not see
                uint32_t w[4];
                if (partial) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (!is_new)
                            w[q] = lead_word(nv, q);
                        else if (a.tree_mask)
                            w[q] = row_ok && key0 / 32 + q < a.mask_words
                                       ? dev::ld(a.tree_mask + (int64_t(it.b) * a.T + t) * a.mask_words + key0 / 32 + q) & lead_word(nv, q)
                                       : 0u;
                        else
                            w[q] = lead_word(min(nv, t - key0 + 1), q);
                    }
                }
                // two halves of the scores: the first one's maximum is taken while
                // the second is on its way from tensor memory
                uint32_t sr[4][32];
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                tc::tmem_ld32(s_t, sr[0]);
                tc::tmem_ld32(s_t + 32, sr[1]);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    tc::tmem_ld_wait();
                    tc::reg_fence(sr[2 * hh]);
                    tc::reg_fence(sr[2 * hh + 1]);
                    if (hh == 0) {
                        tc::tmem_ld32(s_t + 64, sr[2]);
                        tc::tmem_ld32(s_t + 96, sr[3]);
                    }
                    if (partial) {
#pragma unroll
                        for (int q = 2 * hh; q < 2 * hh + 2; ++q)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(w[q] >> e & 1u)) sr[q][e] = __float_as_uint(-INFINITY);
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
#pragma unroll
                        for (int q = 2 * hh; q < 2 * hh + 2; ++q) {
                            m4[2 * (q & 1)] = fmax3(m4[2 * (q & 1)], __uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1]));
                            m4[2 * (q & 1) + 1] = fmax3(m4[2 * (q & 1) + 1], __uint_as_float(sr[q][e + 2]), __uint_as_float(sr[q][e + 3]));
                        }
                }
                // (a TMEM lane without a query row: whatever it holds stays in its lane)
                const float m_tile = row_ok ? fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * a.scale_log2 : -INFINITY;
                if (__any_sync(FULL, m_tile > m_run + C::RESCALE_LOG2)) {
                    const float m_new = m_tile > m_run + C::RESCALE_LOG2 ? m_tile : m_run;
                    const float corr = m_new == m_run ? 1.f : ex2_approx(m_run - m_new);
                    const float2 c2 = make_float2(corr, corr);
                    m_run = m_new;
                    l2 = __fmul2_rn(l2, c2);
                    if (j > j_first) {
                        // PV of the tile before is done (it precedes this S), the next waits for P
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {
                            uint32_t o[16];
                            rows_tmem_ld16(o_t + 16 * q, o);
                            tc::tmem_ld_wait();
                            rows_reg_fence16(o);
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), c2);
                                o[e] = __float_as_uint(y.x);
                                o[e + 1] = __float_as_uint(y.y);
                            }
                            rows_tmem_st16(o_t + 16 * q, o);
                        }
                    }
                }
                const float negm = m_run == -INFINITY ? 0.f : BF16 ? -m_run : C::P_SHIFT_LOG2_F16 - m_run;
                const float2 neg2 = make_float2(negm, negm);
                float2 ps[4] = {l2, make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 y = __ffma2_rn(make_float2(__uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1])), scale2, neg2);
                        sr[q][e] = __float_as_uint(y.x);
                        sr[q][e + 1] = __float_as_uint(y.y);
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float p0 = ex2_approx(__uint_as_float(sr[q][e])), p1 = ex2_approx(__uint_as_float(sr[q][e + 1]));
                        ps[(e >> 1) & 3] = __fadd2_rn(ps[(e >> 1) & 3], make_float2(p0, p1));
                        pk[e / 2] = Ops::pack(p0, p1);
                    }
                    rows_tmem_st16(s_t + 16 * q, pk);  // over scores that are in registers
                    if (q == 1) {  // P.V starts on these 64 keys (long prompt 1623 -> 1583 us)
                        tc::tmem_st_wait();
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) dev::mbar_arrive(p_half + 8 * x);
                    }
                }
                l2 = __fadd2_rn(__fadd2_rn(ps[0], ps[1]), __fadd2_rn(ps[2], ps[3]));
                tc::tmem_st_wait();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(p_full + 8 * x);
            }
            if (!ok) break;
            st += 2 * n;
            // ---- epilogue
            float l = l2.x + l2.y, f_a = 0.f, f_b = 1.f;  // folded items: factors of the two accumulators
            float2 *fold_ml = reinterpret_cast<float2 *>(smem + C::FOLD_OFF);
            if (fold && x == 0) {
                // stream B reads both accumulators (and lets them go; those of the
                // item before, too, before its values here are overwritten)
                ok = k == 0 || __all_sync(FULL, rows_wait(o_free, uint32_t(k - 1) & 1, flags, a.timeout_ns));
                if (!ok) break;
                fold_ml[r] = make_float2(m_run, l);
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(fold_bar);
                ++gi;
                leave();
                continue;
            }
            ok = rows_wait(o_full + 8 * x, gi & 1, flags, a.timeout_ns);
            if (fold) {  // (stream A has a part in every item: its phase is k's)
                ok = ok && rows_wait(fold_bar, folds & 1, flags, a.timeout_ns) &&
                     rows_wait(o_full, uint32_t(k) & 1, flags, a.timeout_ns);
                ++folds;
            }
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            ++gi;
            tc::fence_after();
            if (fold) {
                const float2 ml = fold_ml[r];
                const float M = fmaxf(m_run, ml.x);
                f_a = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
                f_b = m_run == -INFINITY ? 0.f : ex2_approx(m_run - M);
                l = l * f_b + ml.y * f_a;
                m_run = M;
            }
            const bool any_odd = odd[k & 3] != 0;
            const float inv = l == 0.f ? 0.f : 1.f / l;  // (a NaN, of a key row that is seen, passes)
            RowsSeq sq;
            sq.row0 = it.row0;
            auto release = [&]() {  // the accumulators are read: the next item's PV may overwrite them
                tc::fence_before();
                __syncwarp();
                if (lane == 0) {
                    dev::mbar_arrive(o_free + 8 * x);
                    if (fold) dev::mbar_arrive(o_free);
                }
            };
            if (it.slot < 0 && !any_odd && !fold) {
                // the whole item, as fragments of 16 query rows x D columns: four
                // lanes hold 32 columns of a row and, transposed, write 64
                // contiguous bytes (a row per lane, 16 bytes at a time, would keep
                // the store path busy four times as long).  A row of zeros where
                // nothing was seen, whatever the accumulator holds
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[D / 32][16];
                    const uint32_t at = o_t + (uint32_t(16 * h) << 16);
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) rows_tmem_ld_frag(at + 32 * q, o[q]);
                    float2 g[2];
                    T *to[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float gi2 = __shfl_sync(FULL, inv, 16 * h + 8 * i + (lane >> 2));
                        g[i] = make_float2(gi2, gi2);
                        const int tok = qx * TB + frag_tok[2 * h + i];
                        to[i] = frag_tok[2 * h + i] < TB && tok < it.ntok
                                    ? reinterpret_cast<T *>(a.out) + rows_offset(a, sq, it.b, H, it.kv * G + frag_head[2 * h + i], it.t0 + tok, D) + 8 * (lane & 3)
                                    : nullptr;
                    }
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) rows_reg_fence16(o[q]);
                    if (h == 1) release();
#pragma unroll
                    for (int q = 0; q < D / 32; ++q)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int n4 = 0; n4 < 4; ++n4) {
                                const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[q][4 * n4 + 2 * i]), __uint_as_float(o[q][4 * n4 + 2 * i + 1])), g[i]);
                                w[n4] = g[i].x != 0.f ? Ops::pack(y.x, y.y) : 0u;
                            }
                            rows_quad_transpose(w, lane);
                            if (to[i]) *reinterpret_cast<uint4 *>(to[i] + 32 * q) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                }
                leave();
                continue;
            }
            // a piece: its accumulator, four columns of the tile's rows after one
            // another; or a whole item that is folded or has infinities or NaN among
            // its V rows, a row per lane
            float *prow = nullptr;
            if (row_ok && it.slot >= 0) {
                prow = a.part_acc + int64_t(it.slot) * 256 * D + 4 * (128 * qx + r);
                reinterpret_cast<float2 *>(a.part_ml)[int64_t(it.slot) * 256 + 128 * qx + r] = make_float2(m_run, l);
            }
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tc::tmem_ld32(o_t + 32 * q, o);
                if (fold) {
                    uint32_t oa[32];
                    tc::tmem_ld32(o_t - D + 32 * q, oa);
                    tc::tmem_ld_wait();
                    tc::reg_fence(oa);
                    tc::reg_fence(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(fmaf(__uint_as_float(o[e]), f_b, __uint_as_float(oa[e]) * f_a));
                } else {
                    tc::tmem_ld_wait();
                    tc::reg_fence(o);
                }
                if (q == D / 32 - 1) release();
                if (any_odd && row_ok) {
                    // add them back where the row sees them (of the tiles that were
                    // searched: those some row does not see whole)
                    for (int jt = max(it.j0, it.np); jt < it.j1; ++jt) {
                        const int key0 = 128 * (jt - it.np), nv = min(128, it.vis - key0);
                        if (!(nv < 128 || a.tree_mask || key0 + 127 > it.t0)) continue;
                        for (int key = key0; key < key0 + nv; ++key) {
                            const bool see = a.tree_mask ? dev::ld(a.tree_mask + (int64_t(it.b) * a.T + t) * a.mask_words + (key >> 5)) >> (key & 31) & 1u
                                                         : key <= t;
                            if (!see) continue;
                            const T *v = reinterpret_cast<const T *>(a.v_new) + rows_offset(a, sq, it.b, a.H_kv, it.kv, key, D) + 32 * q;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float y = float(v[e]);
                                if (!isfinite(y)) o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
                            }
                        }
                    }
                }
                if (prow) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4 *>(prow + int64_t(8 * q + e / 4) * 1024) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                } else if (row_ok) {
                    T *orow = reinterpret_cast<T *>(a.out) + rows_offset(a, sq, it.b, H, it.kv * G + head, t, D) + 32 * q;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t u[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            u[i] = l != 0.f ? Ops::pack(__uint_as_float(o[e + 2 * i]) * inv, __uint_as_float(o[e + 2 * i + 1]) * inv) : 0u;
                        *reinterpret_cast<uint4 *>(orow + e) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            }
            leave();
        }
        if (!ok) give_up();
    }

    // ---- teardown
    tc::fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, C::TMEM_COLS);
    }
    // after an abort, wait (bounded) for the copies that may still land
    if (warp == C::ITEM_WARP && lane == 0 && flags[0] && queries > 0) {
        const volatile int never = 0;
        rows_wait(q_full, uint32_t(queries - 1) & 1, &never, a.timeout_ns);
    }
    if ((warp == C::K_WARP || warp == C::V_WARP) && lane == 0 && flags[0]) {
        const volatile int never = 0;
        for (int s = 0; s < NS; ++s)
            if (filled >> s & 1) rows_wait(full + 8 * s, filled_phase >> s & 1, &never, a.timeout_ns);
    }
}

// Folds the pieces of the items that CTA boundaries cut.  Block (i, y): 64 query
// rows x 64 columns of the item that CTA i started; a thread takes eight columns
// of a row, consecutive threads consecutive rows, as the pieces are laid out:
// out = sum_p O_p 2^(m_p - M) / sum_p l_p 2^(m_p - M).
template <typename T, int D>
__global__ void __launch_bounds__(512) rows_combine_kernel(const __grid_constant__ RowsTcArgs a) {
    dev::allow_dependents();
    dev::grid_dependency_wait();
    const int i = blockIdx.x;
    const RowsCut cut = a.cuts[i];
    if (cut.pieces == 0) return;
    const int G = a.group, TB = 128 / G;
    const int yr = blockIdx.y / (D / 64), yc = blockIdx.y % (D / 64);
    const int r = 64 * yr + (threadIdx.x & 63), col = 64 * yc + 8 * (threadIdx.x >> 6);
    const int x = r >> 7, rt = (r & 127) / G, head = (r & 127) - rt * G, tok = x * TB + rt;
    if (rt >= TB || tok >= cut.ntok) return;
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + r;
    const float *acc = a.part_acc + 4 * r + (col / 4) * 1024;
    auto slot = [&](int p) { return int64_t(p == 0 ? 2 * i + 1 : 2 * (i + p)) * 256; };
    float M = -INFINITY, L = 0.f, o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int p = 0; p < cut.pieces; ++p) {
        const float2 y = __ldcg(ml + slot(p));
        const float4 u = __ldcg(reinterpret_cast<const float4 *>(acc + slot(p) * D));
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(acc + slot(p) * D + 1024));
        if (y.y == 0.f) continue;  // the row sees nothing of this piece
        const float m = fmaxf(M, y.x), fo = M == -INFINITY ? 0.f : ex2_approx(M - m), f = ex2_approx(y.x - m);
        M = m;
        L = L * fo + y.y * f;
        const float w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(w[e], f, o[e] * fo);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const RowsSeq s = rows_seq(a, cut.b);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = MmaOps<T>::pack(o[2 * e] * inv, o[2 * e + 1] * inv);
    T *to = reinterpret_cast<T *>(a.out) + rows_offset(a, s, cut.b, a.H_kv * G, cut.kv * G + head, cut.t0 + tok, D) + col;
    *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int D>
cudaError_t set_rows_tc_max_smem() {
    return cudaFuncSetAttribute(rows_tc_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, RowsTcCfg<D>::SMEM);
}

// combine_rows: rows of the two query tiles that an item can use; 0 where no
// item can be cut.
template <typename T, int D>
cudaError_t launch_rows_tc(const RowsTcArgs &a, int grid, int combine_rows, cudaStream_t s) {
    const cudaError_t e = launch_pdl(rows_tc_kernel<T, D>, dim3(grid), dim3(RowsTcCfg<D>::THREADS), RowsTcCfg<D>::SMEM, s, a);
    if (e != cudaSuccess || combine_rows == 0 || grid == 1) return e;
    return launch_pdl(rows_combine_kernel<T, D>, dim3(grid, (combine_rows + 63) / 64 * (D / 64)), dim3(512), 0, s, a);
}

template <typename T, int D>
const RowsKernelInfo *rows_tc_info() {
    static const RowsKernelInfo info = {&set_rows_tc_max_smem<T, D>, &launch_rows_tc<T, D>};
    return &info;
}

}  // namespace kvc
