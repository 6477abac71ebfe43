// kvc_e4m3_tc.cuh -- attention of packed new tokens over the 8-bit paged cache on
// the fifth-generation tensor cores, which take the e4m3 codes as they are stored.
//
// Token i of sequence b, whose rows are in the cache already, attends over rows
// j <= cache_index[b] + i:
//   out = softmax_j(q . (kc_j ks_j) / sqrt(128)) . (vc_j vs_j)
// with the codes kc, vc and the scales ks, vs of the rows' blocks.  A scale is
// constant over a block and factors out of its scores; vs goes into the
// probabilities.  So both products run on codes (tcgen05.mma kind::f8f6f4), and no
// code is ever widened by a thread:
//   S[128 keys x N]  = Kc . Q'     A = the K codes as copied (K-major)
//   O[128 x N]      += Vc^T . P'   A = the V codes as copied (MN-major)
// The other operand has 3 bits of mantissa too, so a query element is taken as the
// sum of three of them, each what the ones before leave (off by 2^-12, or by 2^-17 of
// the row's largest): three columns, added up as they are read, or, where a tile has
// many query rows, three products into one column.  A probability is split in
// four, each 32 times what the ones before leave (off by 2^-15, or by 2^-25 of 1; the
// softmax's sum takes it as it is): four columns, added up at a piece's end with the
// factors 1, 2^-5, 2^-10 and 2^-15.  With three, 16 times what is left, whatever was 2^-18
// of a row's first maximum was lost, and with it, beside one key with 97 % of the weight,
// much of what 16,384 others add up to (the fourth costs 3 %: 32 heads on one KV head 20.9
// -> 21.4 us, drafts 27.8 -> 28.8).  The tensor cores have the time: they read A for as
// long as N = 64 takes them.
//
// A tile is 128 rows: the blocks of 16 rows of NH KV heads that lie one behind
// another in the pool, of 8 / NH pages.  One box brings a page's NH heads (NH * 2
// KB; the V of one head is copied by threads).  A tile's columns belong to NH heads;
// of S a thread reads those of its own row's head, and P' is zero where row and column
// are of different heads (those bytes are zeroed once, at the start, and never
// written).  Codes are finite, so zeros keep the heads apart.
//
// Softmax.  Two groups of warps take the tiles in turn, each with its own
// running references, sums and accumulator O, joined at the end of a piece; or, where
// a head has more query rows than a tile's 32 (WIDE), both take every tile, each for
// 32 rows of its own, so that a tile that was copied once serves 64.  A
// thread has one key.  P' is MN-major, so that a thread's probabilities, of all its
// head's query rows, are neighbouring bytes.  A pair (head, query row) has one
// reference mo, of the scores with the values' scale in them: P' = 2^(s + log2 vs -
// mo) stays within the range of the four values (up to 2^8, down to 2^-24) whatever the
// blocks' scales, and P' / vs sums up to what the output is divided by.
// (Scales of values below 2^-90, zeros among them, count as that in a reference, so
// that no sum overflows; below 2^-40 the sum has an exponential of its own, as P' may
// be flushed to zero beside values of common size; and where references differ, sums
// take the factor in two steps, as one may be below what fp32 has.)  The references
// are raised, and the maxima taken at all, only where a P' would pass 2^8: else a tile
// costs the group one barrier that carries the question.  A reference is set so that
// the row's largest P' is 2^r.  What is cut off below the four values is 2^-(25 + r) of
// that at most, and a later score has 8 - r bits to go.  r grows with the rows that the
// segment sees, 0 below 1,024, 4 from 8,192, 6 from 32,768 on, so that all they lose is
// 2^-15 of the largest: short segments have no time to raise references, long ones
// hardly notice (r always 0, as it is, always 4: 1,216 sequences of 512 rows 76, 76, 84
// us, 32 heads on one KV head 21.4, 22.3, 22.6, a batch 33.0, 33.3, 33.8, long MHA 233).
//
// The line of all tiles (sequence after sequence, head group, query rows) is cut
// into equal shares; a cut segment's pieces go to the workspace as partial results,
// and the CTA that finds itself the last of them (a counter) joins them.  No CTA
// waits for another.
//
// Warps: 0 copies, 1 issues S, 2 issues O, the others softmax and epilogue.  After a wait
// that ran out (KVC_ERR_TIMEOUT) the softmax warps go through the rest of their
// tiles without waiting, so that all meet at the same barriers.  The waits for copies and
// products in flight before the block leaves keep their limit, whatever the handle's is.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvc_e4m3.cuh"
#include "kvc_tcgen05.cuh"

namespace kvc {
namespace e4 {

constexpr unsigned FULL = 0xffffffffu;
constexpr int TILE = 128, TILE_BYTES = TILE * E4M3_D, STAGE_BYTES = 2 * TILE_BYTES;
constexpr int MAX_STAGES = 6;
constexpr uint32_t TMEM_COLS = 512, S_COL = 0, S_NEXT = 128, O_COL = 256, O_NEXT = 128;  // (a group's)
constexpr float RESCALE_LOG2 = 8.f, SMALL_LOG2 = -40.f;
constexpr int64_t MAX_LINE = 1 << 30;  // tiles of a call (places are 32-bit numbers)
constexpr int GROUPS = 2;
// Softmax warps: two groups of 4, or of 8 where a tile has 16 or 32 query rows per
// head: two warps then share each key, a half of the rows each (the exponents, sums and
// bytes of 32 rows are more than one thread has registers for; with 16, two warps take
// what one does or 3 % more where tiles are many, 64 sequences of 4,000 rows with 16 heads
// on one KV head 25.3 us and 24.9, and less where a call waits for its last pieces, one
// sequence of 8,048 rows 13.2 us and 14.4).
// Before them: copies, the issuers of S and O, and, where a tile is of one head, a
// warp that copies V 16 bytes a lane: 16 boxes of 2 KB a tile take 1.1 us (a box about
// 50 cycles and five for each of its rows), eight of them beside the warp 0.8.
template <int RT, bool ONE>
struct Warps {
    static constexpr int SOFT0 = ONE ? 4 : 3;
    static constexpr int SPLIT = RT >= 16 ? 2 : 1, RW = RT / SPLIT;  // RW: query rows of a thread
    // The three values of a query element: columns of one product (whose latency is that
    // of four instructions, not twelve: one user 8.4 us and 8.7) or three products.
    static constexpr bool COLUMNS = RT <= 4;
    static constexpr int SETS = GROUPS * SPLIT, NSOFT = 4 * SETS, THREADS = 32 * (SOFT0 + NSOFT);
};

// Shared memory behind the stages (all of it 1024-byte aligned at first): Q'
// [2][N rows][128] by piece, P' [2][128 keys][4 ps] by group, then the small arrays.
struct Small {
    float k_scale[MAX_STAGES][8], v_scale[MAX_STAGES][8];  // of the stage's blocks
    float red[GROUPS][8][32];       // maxima of a block's keys, [block][query row]
    float sums[2][GROUPS][128];     // [piece parity]: sums of a half-warp's keys (one head: of a warp's)
    float ref[2][GROUPS][32];       // [piece parity]: references of the pairs
    float neg[GROUPS][32];          // by pair: -mo
    float delta[GROUPS][32], corr[GROUPS][32];  // what it has just been raised by, and 2 to the minus half of that
    float qf[2][64];                // factor of a pair's scores, [piece parity]
    int32_t lim[2][64];             // keys that a pair's query row sees
    int64_t out_row[2][64];         // its row of out, or -1
    uint64_t full[MAX_STAGES], empty[MAX_STAGES], v_full[MAX_STAGES];
    uint64_t s_full[2], s_free[2], p_full[2], p_free[2];
    uint64_t q_full[2], o_free, mma_done;
    int64_t plan[20];               // the warps' parts of the line
    uint32_t tmem;
    int32_t flags[2];               // abort; last of the pieces
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t *r) {
    if constexpr (N == 1)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[0]) : "r"(t) : "memory");
    else if constexpr (N == 2)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(t) : "memory");
    else if constexpr (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(t)
                     : "memory");
    else if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(t)
                     : "memory");
    else {
        tmem_ld<8>(t, r);
        tmem_ld<8>(t + 8, r + 8);
        if constexpr (N == 32) tmem_ld<16>(t + 16, r + 16);
    }
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
template <int N>
__device__ __forceinline__ void reg_fence(uint32_t *r) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Does any thread say so?  By all `threads` of the barrier.
__device__ __forceinline__ bool barrier_or(int id, int threads, bool x) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(uint32_t(x)), "r"(id), "r"(threads)
        : "memory");
    return any != 0;
}

// Descriptor of an MN-major operand whose rows (of one key) are 4 ps = 32, 64 or
// 128 bytes, one swizzle of that width: bits 61-63 are 6, 4, 2; 8 rows to the next.
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, int ps) {
    const uint64_t layout = ps == 32 ? 2 : ps == 16 ? 4 : 6;
    return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(uint32_t(ps) * 32 >> 4) << 32) | (uint64_t(1) << 46) | (layout << 61);
}

// D[tmem] = A B (+ D), e4m3 codes, fp32 accumulation; issued by one thread.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

struct Piece {
    int b, lo, n, c;     // the sequence: first packed row, tokens, cached rows
    int hg, j, part;     // head group, row tile (tokens j tt ...), part of the heads
    int first, last;     // tiles [first, last)
    int tiles;           // of the whole segment
    int keys;            // that its last token sees
    int start;           // place of the segment's first tile in the line
};

// The line: each segment's tiles behind `cost` places that hold none, which stand for
// its start and end, so that shares with many short segments are no longer.  All of
// it by whole warps: the lanes hold the sequences [from, from + 32).
struct Walker {
    int b, hg, j, part, tiles;
    dev::PackedSeq s, mine;
    int from, start, at, end, share;

    __device__ __forceinline__ int keys(const E4m3TcArgs &a) const { return s.c + min(s.n, (j + 1) * a.tt); }
    __device__ __forceinline__ void measure(const E4m3TcArgs &a) { tiles = (keys(a) + (1 << a.shift) - 1) >> a.shift; }

    // length of a sequence's part of the line (at most 2^31 - 1: a longer one counts as
    // that; one row tile's is within 2^30, as the configuration's check has it)
    __device__ __forceinline__ int length(const E4m3TcArgs &a, const dev::PackedSeq &q) const {
        const int add = (1 << a.shift) - 1, per = a.gt * a.groups;
        if (q.n <= a.tt) return q.n ? (((q.c + q.n + add) >> a.shift) + a.cost) * per : 0;
        int64_t sum = 0;
        for (int t = a.tt; t < q.n + a.tt; t += a.tt) sum += ((q.c + min(q.n, t) + add) >> a.shift) + a.cost;
        return int(min(sum * per, int64_t(0x7fffffff)));
    }

    // The 32 sequences from `at` on into the lanes; returns this lane's length.
    __device__ __forceinline__ int look(const E4m3TcArgs &a, int at, int lane) {
        from = at;
        mine = dev::PackedSeq{};
        if (at + lane < a.B) mine = dev::packed_seq(a, 1, at + lane);
        return length(a, mine);
    }
    __device__ __forceinline__ static int64_t total(int len) {
        return __reduce_add_sync(FULL, unsigned(len) & 0xffffu) + (int64_t(__reduce_add_sync(FULL, unsigned(len) >> 16)) << 16);
    }
    __device__ __forceinline__ void take(int src) {
        b = from + src;
        s.lo = __shfl_sync(FULL, mine.lo, src);
        s.n = __shfl_sync(FULL, mine.n, src);
        s.c = __shfl_sync(FULL, mine.c, src);
    }

    // This CTA's share; by all its warps (`warp` of `warps`; sums: a place for each).  False: it has none.
    __device__ __forceinline__ bool init(const E4m3TcArgs &a, int64_t *sums, int warp, int warps, int lane) {
        int len = 0, first = 0, per = 32;  // sequences of a warp
        int64_t all = 0, before = 0;
        if (a.B <= 32) {
            len = look(a, 0, lane);
            all = total(len);
        } else {
            per = ((a.B + warps - 1) / warps + 31) & ~31;
            for (int i = warp * per; i < min(a.B, (warp + 1) * per); i += 32) all += total(look(a, i, lane));
            if (lane == 0) sums[warp] = all;
            __syncthreads();
            all = 0;
            for (int w = 0; w < warps; ++w) all += sums[w];
        }
        if (all > MAX_LINE) {
            if (blockIdx.x == 0 && lane == 0) dev::record_error(a.err, ERR_DEVICE_INDEX);
            return false;
        }
        share = max(int(unsigned(all + gridDim.x - 1) / gridDim.x), a.min_share);
        const int64_t place = int64_t(share) * blockIdx.x;
        if (place >= all) return false;
        at = int(place);
        end = min(int(all), at + share);
        if (a.B > 32) {  // on to the warp's part that holds it
            for (int w = 0; before + sums[w] <= at; ++w) {
                before += sums[w];
                first += per;
            }
            len = look(a, first, lane);
        }
        for (start = int(before);; len = look(a, from + 32, lane)) {
            int incl = len;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(FULL, incl, o);
                if (lane >= o) incl += y;
            }
            const unsigned hit = __ballot_sync(FULL, start + incl - len <= at && at < start + incl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                take(src);
                start += __shfl_sync(FULL, incl - len, src);
                const int one = __shfl_sync(FULL, len, src) / a.groups;
                hg = (at - start) / one;
                start += hg * one;
                break;
            }
            start += __shfl_sync(FULL, incl, 31);
        }
        j = part = 0;
        for (measure(a); at >= start + a.gt * (tiles + a.cost); ++j, measure(a)) start += a.gt * (tiles + a.cost);
        if (a.gt > 1) part = (at - start) / (tiles + a.cost);
        start += part * (tiles + a.cost);
        return true;
    }

    __device__ __forceinline__ bool next(const E4m3TcArgs &a, Piece &p, int lane) {
        do {
            if (at >= end) return false;
            if (at >= start + a.cost + tiles) {  // on to the next segment
                start += a.cost + tiles;
                if (++part == a.gt) {
                    part = 0;
                    if (++j * a.tt >= s.n) {
                        j = 0;
                        if (++hg == a.groups) {
                            hg = 0;
                            unsigned later = __ballot_sync(FULL, mine.n > 0) & (~1u << (b - from));
                            while (!later) {
                                if (from + 32 >= a.B) return false;
                                look(a, from + 32, lane);
                                later = __ballot_sync(FULL, mine.n > 0);
                            }
                            take(__ffs(later) - 1);
                        }
                    }
                    measure(a);
                }
            }
            p.first = max(0, at - start - a.cost);
            p.last = min(tiles, end - start - a.cost);
            at = min(end, start + a.cost + tiles);
        } while (p.last <= 0);
        p.b = b, p.lo = s.lo, p.n = s.n, p.c = s.c;
        p.hg = hg, p.j = j, p.part = part;
        p.tiles = tiles;
        p.keys = keys(a);
        p.start = start + a.cost;
        return true;
    }
};

// The piece's query rows as three e4m3 values per element, [value][pr rows][128], and
// what the softmax warps know of each; by all of them (w).
template <int RT, bool WIDE>
__device__ __forceinline__ void load_queries(const E4m3TcArgs &a, const Piece &p, Small &sm, uint32_t q_s, int np, int pr, int w, int lane) {
    constexpr int NSOFT = Warps<RT, false>::NSOFT, BATCH = (WIDE ? 64 : 32) / NSOFT;
    const int pairs = WIDE ? 2 * RT : a.nh * RT, x = np & 1;
    uint2 raw[BATCH];
    int64_t row[BATCH];
    int lim[BATCH];
#pragma unroll
    for (int e = 0; e < BATCH; ++e) {  // all loads in flight
        const int pair = w + NSOFT * e, h = WIDE ? 0 : pair / RT, r = WIDE ? pair : pair % RT;
        const int tt = (r * a.gg_inverse) >> 16, gi = p.part * a.gg + r - tt * a.gg, t = p.j * a.tt + tt;
        const bool live = pair < pairs && tt < a.tt && gi < a.group && t < p.n;
        row[e] = live ? (int64_t(p.lo) + t) * a.H + (p.hg * a.nh + h) * a.group + gi : -1;
        lim[e] = live ? p.c + t + 1 : 0;
        raw[e] = make_uint2(0, 0);
        if (live) raw[e] = dev::ld(static_cast<const uint2 *>(a.q) + row[e] * 32 + lane);
    }
#pragma unroll
    for (int e = 0; e < BATCH; ++e) {
        const int pair = w + NSOFT * e;
        if (pair >= pairs) break;
        float y[4];
        if (a.bf16) {
            y[0] = __uint_as_float(raw[e].x << 16), y[1] = __uint_as_float(raw[e].x & 0xffff0000u);
            y[2] = __uint_as_float(raw[e].y << 16), y[3] = __uint_as_float(raw[e].y & 0xffff0000u);
        } else {
            const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(&raw[e].x)), v = __half22float2(*reinterpret_cast<const __half2 *>(&raw[e].y));
            y[0] = u.x, y[1] = u.y, y[2] = v.x, y[3] = v.y;
        }
        // the exponent field of the row's largest element (as integers: those of
        // infinities and NaN are above all others')
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(y[k]) & 0x7fffffffu);
        top = __reduce_max_sync(FULL, top) >> 23;
        const bool odd = top == 255;
        const uint32_t ex = max(top, 8u);
        const float up = __uint_as_float((261u - (odd ? 8u : ex)) << 23);  // 2^(134 - ex): the largest becomes 128 ... 256
        if (lane == 0) {
            sm.qf[x][pair] = odd ? __int_as_float(0x7fffffff) : __uint_as_float((ex - 7u) << 23) * a.scale_log2;
            sm.lim[x][pair] = lim[e];
            sm.out_row[x][pair] = row[e];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = odd ? 0.f : y[k] * up;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uint32_t lo = dev::e4m3x2(y[0], y[1]), hi = dev::e4m3x2(y[2], y[3]);
            dev::st_shared_u32(q_s + uint32_t(i * pr + pair) * 128 + (uint32_t((lane >> 2) ^ (pair & 7)) << 4) + uint32_t(lane & 3) * 4, lo | hi << 16);
            if (i < 2) {
                const uint32_t bl = dev::e4m3x2_to_f16x2(lo), bh = dev::e4m3x2_to_f16x2(hi);
                const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(&bl)), v = __half22float2(*reinterpret_cast<const __half2 *>(&bh));
                y[0] -= u.x, y[1] -= u.y, y[2] -= v.x, y[3] -= v.y;
            }
        }
    }
    dev::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(dev::smem_addr(&sm.q_full[x]));
}

// Max or sum of v[0 .. R) over the 16 lanes of a half-warp; v[0] of lane l (of 16) is
// then row l * R / 16's.
template <int R, bool SUM>
__device__ __forceinline__ void reduce16(float (&v)[R], int lane) {
    static_assert(R <= 16, "a row per lane");
    int bit = 8;
#pragma unroll
    for (int s = R / 2; s >= 1; s >>= 1, bit >>= 1) {
        const bool up = (lane & bit) != 0;
#pragma unroll
        for (int i = 0; i < s; ++i) {
            const float send = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
            const float got = __shfl_xor_sync(FULL, send, bit);
            v[i] = SUM ? keep + got : fmaxf(keep, got);
        }
    }
    for (; bit >= 1; bit >>= 1) {
        const float got = __shfl_xor_sync(FULL, v[0], bit);
        v[0] = SUM ? v[0] + got : fmaxf(v[0], got);
    }
}
template <int R>
__device__ __forceinline__ void store_reduced(float *to, const float (&v)[R], int lane) {
    const int l = lane & 15;
    if (l % (16 / R) == 0) to[l / (16 / R)] = v[0];
}

// Max of v[0 .. RT) over the warp; lane l has row l's.
template <int RT>
__device__ __forceinline__ float max_rows(const float (&v)[RT], int lane) {
    float mine = -INFINITY;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        float y;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(v[r]));
        mine = lane == r ? y : mine;
    }
    return mine;
}

// The partial results of CTAs c0 ... c1 joined into the pairs' output rows, by all
// of NSOFT warps (sw; `first`: the first of their pairs): a warp has every NSOFT-th
// pair, a lane four of its elements and one piece's reference and sum.
template <int NSOFT>
__device__ __forceinline__ void join(const E4m3TcArgs &a, int64_t out_row, int first, int pairs, int c0, int c1, int sw, int lane) {
    constexpr int BATCH = 8;
    const auto slot_of = [&](int c) { return 2 * int64_t(c) + (c == c0); };
    float4 z[BATCH];
    const auto fetch = [&](int pair, int b) {  // eight pieces' loads in flight
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (b + i <= c1) z[i] = __ldcg(reinterpret_cast<const float4 *>(a.part_acc + (slot_of(b + i) * E4M3_SLOT + first + pair) * E4M3_D) + lane);
        }
    };
#pragma unroll 1
    for (int pair = sw; pair < pairs; pair += NSOFT) {
        float M = -INFINITY, L = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int b = c0; b <= c1; b += 32) {  // (a lane per piece)
            float2 ml = make_float2(-INFINITY, 0.f);
            if (b + lane <= c1) ml = __ldcg(a.part_ml + slot_of(b + lane) * E4M3_SLOT + first + pair);
            fetch(pair, b);
            float m;
            asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(ml.x));
            m = fmaxf(M, m);
            const float old2 = M == -INFINITY ? 0.f : ex2(0.5f * (M - m)), e2 = ml.x == -INFINITY ? 0.f : ex2(0.5f * (ml.x - m));
            const float old = old2 * old2, e = e2 * e2;
            M = m;
            float l = ml.x == -INFINITY ? ml.y : ml.y * e2 * e2;  // (0, or a NaN that stays)
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(FULL, l, o);
            L = L * old2 * old2 + l;
            y.x *= old, y.y *= old, y.z *= old, y.w *= old;
            for (int q = b; q <= min(c1, b + 31); q += BATCH) {
                if (q > b) fetch(pair, q);
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const float f = __shfl_sync(FULL, e, (q - b + i) & 31);
                    y = make_float4(fmaf(z[i].x, f, y.x), fmaf(z[i].y, f, y.y), fmaf(z[i].z, f, y.z), fmaf(z[i].w, f, y.w));
                }
            }
        }
        const float f = L == 0.f ? 0.f : 1.f / L;
        const int64_t r = __shfl_sync(FULL, out_row, pair);
        if (r < 0) continue;
        uint2 u;
        if (a.bf16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x * f, y.y * f), hi = __floats2bfloat162_rn(y.z * f, y.w * f);
            u = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        } else {
            const __half2 lo = __floats2half2_rn(y.x * f, y.y * f), hi = __floats2half2_rn(y.z * f, y.w * f);
            u = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        }
        reinterpret_cast<uint2 *>(a.out)[r * 32 + lane] = u;
    }
}

// Two numbers up to 2^8 as four e4m3 values each, the next 32 times what the ones before
// leave.  A value leaves at most 2^-4 of what it is of, 8 of 2^8, so the next is 2^8 at
// most too.  What the first leaves is rounded to fp16 (2^-15 of the number), whose 11 bits the
// other three hold, but for what is below half of the last one's smallest step, 2^-25.
// (The number itself rounded to fp16 first: 2^-11 of it, the error against 64 bits with
// fp16 queries a fifth larger, and at most 2 % in time, 32 query rows a tile.)
__device__ __forceinline__ void split4(float2 f, uint32_t (&c)[4]) {
    const __half2 minus = __float2half2_rn(-32.f), times = __float2half2_rn(32.f);
    c[0] = dev::e4m3x2(f.x, f.y);
    const uint32_t b0 = dev::e4m3x2_to_f16x2(c[0]);
    const float2 r = dev::fma2(__half22float2(*reinterpret_cast<const __half2 *>(&b0)), make_float2(-32.f, -32.f), dev::mul2(f, make_float2(32.f, 32.f)));
    __half2 x = __floats2half2_rn(r.x, r.y);
#pragma unroll
    for (int k = 1; k < 4; ++k) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
        c[k] = r;
        if (k < 3) {
            const uint32_t back = dev::e4m3x2_to_f16x2(c[k]);
            x = __hfma2(*reinterpret_cast<const __half2 *>(&back), minus, __hmul2(x, times));
        }
    }
}

// RT consecutive floats of shared memory (16-byte aligned where RT >= 4)
template <int RT>
__device__ __forceinline__ void load_row(const float *p, float (&y)[RT]) {
    if constexpr (RT >= 4) {
#pragma unroll
        for (int r = 0; r < RT; r += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(p + r);
            y[r] = x.x, y[r + 1] = x.y, y[r + 2] = x.z, y[r + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int r = 0; r < RT; ++r) y[r] = p[r];
    }
}

// RT: query rows per head (of a group, WIDE); ONE: a tile is of one head (nh == 1).
template <int RT, bool ONE, bool WIDE>
__global__ void __launch_bounds__(Warps<RT, ONE>::THREADS, 1) e4m3_attn_kernel(const __grid_constant__ E4m3TcArgs a) {
    using C = Warps<RT, ONE>;
    constexpr int THREADS = C::THREADS, NSOFT = C::NSOFT, SOFT0 = C::SOFT0, RW = C::RW, SETS = C::SETS;
    static_assert(!WIDE || (ONE && RT == 32), "two groups of 32 rows");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (dev::smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = dev::smem_addr(smem);
    const int nh = ONE ? 1 : a.nh, pages = 8 / nh, pairs = nh * RT, ps = pairs < 8 ? 8 : pairs;
    const int pr = WIDE ? 2 * RT : pairs < 16 ? 16 : pairs, ns = a.n_stages;  // columns of S
    const uint32_t q_bytes = uint32_t(3 * pr) * 128, p_bytes = uint32_t(ps) * 512;
    const uint32_t q_s = sb + uint32_t(ns) * STAGE_BYTES, p_s = q_s + 2 * q_bytes;
    Small &sm = *reinterpret_cast<Small *>(smem + size_t(ns) * STAGE_BYTES + 2 * (q_bytes + p_bytes));
    volatile int *flags = sm.flags;
    auto bar = [](const uint64_t &x) { return dev::smem_addr(&x); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        dev::prefetch_tensormap(&a.tm_k);
        dev::prefetch_tensormap(&a.tm_v);
        for (int s = 0; s < ns; ++s) {
            dev::mbar_init(bar(sm.full[s]), 1);
            dev::mbar_init(bar(sm.empty[s]), 1);
            dev::mbar_init(bar(sm.v_full[s]), 1);
        }
        for (int x = 0; x < 2; ++x) {
            dev::mbar_init(bar(sm.s_full[x]), 1);
            dev::mbar_init(bar(sm.s_free[x]), WIDE ? NSOFT : NSOFT / GROUPS);
            dev::mbar_init(bar(sm.p_full[x]), NSOFT / GROUPS);
            dev::mbar_init(bar(sm.p_free[x]), 1);
            dev::mbar_init(bar(sm.q_full[x]), NSOFT);
        }
        dev::mbar_init(bar(sm.o_free), NSOFT);
        dev::mbar_init(bar(sm.mma_done), 2);
        flags[0] = 0;
        dev::fence_mbar_init();
    }
    // Q' and P': the rows of no pair, and P' off the diagonal, stay zero
    for (uint32_t i = threadIdx.x * 16; i < 2 * (q_bytes + p_bytes); i += THREADS * 16) dev::st_shared_v4(q_s + i, make_uint4(0, 0, 0, 0));
    dev::fence_proxy_async_smem();
    if (warp == 1) {
        tc::tmem_alloc(dev::smem_addr(&sm.tmem), TMEM_COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sm.tmem;
    // what is above overlaps the kernel before
    dev::grid_dependency_wait();
    dev::allow_dependents();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += THREADS)
            if (dev::packed_seq(a, 1, b).bad) dev::record_error(a.err, ERR_DEVICE_INDEX);

    Walker walk;
    const bool any = walk.init(a, sm.plan, warp, THREADS / 32, lane);  // the same in every warp
    const auto wait = [&](uint32_t b, uint32_t parity) { return dev::mbar_wait_bounded(b, parity, flags, a.timeout_ns); };
    const auto fail = [&] {
        if (lane == 0) {
            if (!flags[0]) dev::record_error(a.err, ERR_TIMEOUT);
            flags[0] = 1;
        }
    };
    int issued = 0;
    Piece p;
    if (!any) {
        // no tiles for this CTA
    } else if (warp == 0) {
        // ------------------------------------------------------------ copies
        // Lanes 0-7 copy a page's K each, 8-15 its V (not ONE); 16-31 the scales of the
        // (page, head) blocks.
        const uint64_t pol = a.read_once ? dev::l2_evict_first_policy() : dev::l2_evict_normal_policy();
        const int unit = lane & 7, page_of = lane < 16 ? unit : unit / nh, head_of = unit % nh;
        const bool is_v = (lane & 8) != 0, copies = lane < (ONE ? 8 : 16) && unit < pages;
        bool ok = true;
        int s = 0;
        uint32_t round = 0;  // parity of the stage's turn
        while (ok && walk.next(a, p, lane)) {
            const int32_t *table = a.block_table + int64_t(p.b) * a.max_blocks;
            const int n_pages = (p.keys + 15) >> 4;
            auto entry = [&](int tile) {
                const int page = tile * pages + page_of;
                if (page >= n_pages || tile >= p.last) return -1;
                const int phys = dev::ld(table + page);
                if (phys >= 0 && phys < a.num_blocks) return phys;
                dev::record_error(a.err, ERR_DEVICE_INDEX);
                return -1;
            };
            int phys = entry(p.first);
            for (int t = p.first; t < p.last; ++t) {
                const int next = entry(t + 1);  // on its way meanwhile
                if (issued >= ns && !__all_sync(FULL, wait(bar(sm.empty[s]), round ^ 1))) {
                    fail();
                    ok = false;
                    break;
                }
                const uint32_t full = bar(sm.full[s]), box = uint32_t(nh) * 2048;
                const unsigned boxes = __ballot_sync(FULL, copies && phys >= 0);
                if (lane == 0) dev::mbar_expect_tx(full, uint32_t(__popc(boxes)) * box);
                __syncwarp();
                if (copies && phys >= 0)
                    dev::tma_load_4d(sb + uint32_t(s) * STAGE_BYTES + (is_v ? TILE_BYTES : 0) + uint32_t(unit) * box, is_v ? &a.tm_v : &a.tm_k, 0, 0,
                                     p.hg * nh, a.layer_block + phys, full, pol);
                if (lane >= 16 && phys >= 0) {
                    const int64_t at = int64_t(phys) * a.H_kv + p.hg * nh + head_of;
                    dev::cp_async_4(dev::smem_addr(is_v ? &sm.v_scale[s][unit] : &sm.k_scale[s][unit]), (is_v ? a.v_scale : a.k_scale) + at);
                }
                dev::cp_async_arrive(full);
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(full);
                ++issued;
                if (++s == ns) s = 0, round ^= 1;
                phys = next;
            }
        }
    } else if (ONE && warp == 3) {
        // ------------------------------------------------------------ V of one head
        // 16 bytes a lane at a time, swizzled as a box would be.
        bool ok = true;
        int s = 0, t = 0;
        uint32_t round = 0;
        const int r4 = lane >> 3, c = lane & 7;  // row (of four) and chunk of a copy
        const uint32_t even = uint32_t(r4) * 128 + (uint32_t(c ^ r4) << 4), odd = uint32_t(r4) * 128 + (uint32_t(c ^ (r4 + 4)) << 4);
        while (ok && walk.next(a, p, lane)) {
            const int32_t *table = a.block_table + int64_t(p.b) * a.max_blocks;
            const int n_pages = (p.keys + 15) >> 4;
            const auto entry = [&](int tile) {
                const int page = tile * 8 + c;
                int phys = -1;
                if (page < n_pages && tile < p.last) phys = dev::ld(table + page);
                return phys >= 0 && phys < a.num_blocks ? phys : -1;  // (recorded by warp 0)
            };
            int phys = entry(p.first);
            for (int i = p.first; i < p.last; ++i, ++t) {
                const int next = entry(i + 1);
                if (t >= ns && !__all_sync(FULL, wait(bar(sm.empty[s]), round ^ 1))) {
                    fail();
                    ok = false;
                    break;
                }
                const uint32_t dst = sb + uint32_t(s) * STAGE_BYTES + TILE_BYTES;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int block = __shfl_sync(FULL, phys, k);
                    if (block < 0) continue;
                    const uint8_t *src = a.V + (int64_t(block) * a.H_kv + p.hg) * 2048 + lane * 16;
#pragma unroll
                    for (int e = 0; e < 4; ++e) dev::cp_async_16(dst + uint32_t(k * 2048 + e * 512) + (e & 1 ? odd : even), src + e * 512);
                }
                dev::cp_async_arrive(bar(sm.v_full[s]));
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(bar(sm.v_full[s]));
                if (++s == ns) s = 0, round ^= 1;
                phys = next;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ------------------------------------------------------------ MMA issuers
        // (one thread issues; the pieces are found by the warp)
        const uint32_t idesc_s = tc::idesc_f16_f32acc(false, 128, C::COLUMNS ? 3 * pr : pr, false, false);  // (format 0 of this kind: e4m3)
        const uint32_t idesc_o = tc::idesc_f16_f32acc(false, 128, 4 * ps, true, true);
        bool ok = true;
        int t = 0, np = 0, s = 0;
        uint32_t round = 0;
        bool more = walk.next(a, p, lane);
        while (more) {
            const int tiles = p.last - p.first;
            more = walk.next(a, p, lane);  // (now, not when it is waited for)
            if (warp == 1 && tc::elect()) {
                ok = ok && wait(bar(sm.q_full[np & 1]), uint32_t(np >> 1) & 1);
                const uint32_t qt = q_s + uint32_t(np & 1) * q_bytes;
                for (int i = 0; ok && i < tiles; ++i, ++t) {
                    const int x = t & 1;
                    ok = wait(bar(sm.full[s]), round);
                    if (ok && t >= 2) ok = wait(bar(sm.s_free[x]), uint32_t((t >> 1) - 1) & 1);
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t kt = sb + uint32_t(s) * STAGE_BYTES, d = tmem + S_COL + uint32_t(x) * S_NEXT;
#pragma unroll
                    for (int i3 = 0; i3 < (C::COLUMNS ? 1 : 3); ++i3)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8(d, tc::smem_desc_sw128(kt + k * 32, 16, 1024), tc::smem_desc_sw128(qt + uint32_t(i3 * pr * 128 + k * 32), 16, 1024), idesc_s,
                                   i3 > 0 || k > 0);
                    tc::commit(bar(sm.s_full[x]));
                    if (++s == ns) s = 0, round ^= 1;
                }
            } else if (warp == 2 && tc::elect()) {
                for (int i = 0; ok && i < tiles; ++i, ++t) {
                    const uint32_t vt = sb + uint32_t(s) * STAGE_BYTES + TILE_BYTES;
#pragma unroll 1
                    for (int x = WIDE ? 0 : t & 1; x <= (WIDE ? 1 : t & 1); ++x) {  // the groups that the tile has
                        ok = wait(bar(sm.p_full[x]), uint32_t(WIDE ? t : t >> 1) & 1);
                        if (ok && i == 0 && np > 0) ok = wait(bar(sm.o_free), uint32_t(np - 1) & 1);
                        if (ok) ok = wait(bar(ONE ? sm.v_full[s] : sm.full[s]), round);
                        if (!ok) break;
                        if (ONE) dev::fence_proxy_async_smem();  // (V was written by threads' copies)
                        tc::fence_after();
                        const uint32_t pt = p_s + uint32_t(x) * p_bytes;
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 32 keys each
                            mma_f8(tmem + O_COL + uint32_t(x) * O_NEXT, tc::smem_desc_sw128(vt + k * 4096, 16, 1024),
                                   desc_rows(pt + uint32_t(k) * 32 * uint32_t(4 * ps), ps), idesc_o, i > (WIDE ? 0 : 1) || k > 0);
                        tc::commit(bar(sm.p_free[x]));
                    }
                    if (!ok) break;
                    tc::commit(bar(sm.empty[s]));
                    if (++s == ns) s = 0, round ^= 1;
                }
            }
            __syncwarp();
            ++np;
        }
        if (tc::elect()) {
            if (!ok) {
                if (!flags[0]) dev::record_error(a.err, ERR_TIMEOUT);
                flags[0] = 1;
            }
            // every MMA issued here has completed before tensor memory is freed
            tc::commit(bar(sm.mma_done));
            const volatile int never = 0;
            dev::mbar_wait_bounded(bar(sm.mma_done), 0, &never, WAIT_TIMEOUT_NS);
        }
        __syncwarp();
    } else if (warp >= SOFT0) {
        // ------------------------------------------------------------ softmax
        const int sw = warp - SOFT0, set = sw >> 2, g = set & 1, part = set >> 1;  // part: of the query rows
        const int w = warp & 3, row = 32 * w + lane;  // tensor-memory lane: the tile's row, or O's element
        const int hw = row >> 4, head = hw % nh, page_of = hw / nh, r0 = head * RT + part * RW;  // r0: this thread's first pair
        const int of_all = WIDE ? g * RT : 0;  // the group's first pair of the piece's
        const uint32_t lanes = uint32_t(w * 32) << 16;
        const int my_head = lane / RT, my_row = lane % RT;  // this lane's pair, where lane < pairs
        const int p_shift = ps == 32 ? 7 : ps == 16 ? 6 : 5;
        const uint32_t p_row = p_s + uint32_t(g) * p_bytes + (uint32_t(row) << p_shift);
        const uint32_t p_swz = (uint32_t(row) >> (7 - p_shift)) & ((1u << (p_shift - 4)) - 1);
        const auto group_sync = [&] { dev::named_barrier_sync(1 + g, NSOFT / GROUPS * 32); };
        const auto all_sync = [&] { dev::named_barrier_sync(3, NSOFT * 32); };
        // (all lanes learn of a failure)
        const auto must = [&](bool good) {
            if (!__all_sync(FULL, good)) fail();
        };
        int t0 = 0, np = 0;  // tiles before this piece, pieces
        constexpr int STEP = WIDE ? 1 : GROUPS;
        int s = WIDE ? 0 : g;  // stage of this group's next tile, and the parity of its turn
        uint32_t round = 0;
        if (s >= ns) s -= ns, round ^= 1;
        bool more = walk.next(a, p, lane);
        if (more) load_queries<RT, WIDE>(a, p, sm, q_s, 0, pr, sw, lane);
        while (more) {
            const Piece here = p;
            const int xp = np & 1, tiles = here.last - here.first;
            // The next piece and its queries (the last scores of the piece before, which
            // had the buffer, are long read); by all warps, each once, after its first tile.
            const auto look_ahead = [&] {
                more = walk.next(a, p, lane);
                if (more) load_queries<RT, WIDE>(a, p, sm, q_s + uint32_t(xp ^ 1) * q_bytes, np + 1, pr, sw, lane);
            };
            must(wait(bar(sm.q_full[xp]), uint32_t(np >> 1) & 1));  // qf, lim and out_row are there
            const int64_t out_row = lane < pairs ? sm.out_row[xp][of_all + lane] : -1;
            float mo = 0.f;  // this lane's pair
            float sum[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) sum[r] = 0.f;
            const int least = here.c + here.j * a.tt + 1;  // keys that every row of the piece sees
            const float room = float(min(max(22 - __clz(here.keys), 0), 6));  // log2 of the largest P' where a reference is set
            int i = WIDE || (t0 & 1) == g ? 0 : 1;
            const int first = i;
            for (; i < tiles; i += STEP) {
                const int t = t0 + i;
                const int x = WIDE ? t & 1 : g;  // the tile's score buffer
                const uint32_t turn = uint32_t(WIDE ? t : t >> 1) & 1;  // parity of the group's P' and O
                const int key = ((here.first + i) * pages + page_of) * 16 + (lane & 15);
                const bool masked = (here.first + i + 1) * pages * 16 > least;  // the same in every thread
                must(!flags[0] && wait(bar(sm.s_full[x]), uint32_t(t >> 1) & 1) && wait(bar(sm.full[s]), round));
                tc::fence_after();
                // v: exponents of P'
                float v[RW];
                const float ks = sm.k_scale[s][hw], lv0 = __log2f(sm.v_scale[s][hw]);
                const float lv = lv0 < -90.f ? -90.f : lv0;  // (a NaN stays)
                {
                    uint32_t raw[RW];
                    const uint32_t col = tmem + lanes + S_COL + uint32_t(x) * S_NEXT + uint32_t(of_all + part * RW);
                    float qf[RW], neg[RW];
                    constexpr int M = C::COLUMNS ? 3 : 1, HEADS = ONE ? 1 : 2;  // (a warp's rows are of two heads)
                    uint32_t in[M][HEADS][RW];
                    const int h = ONE ? 0 : 2 * w % nh;
#pragma unroll
                    for (int k = 0; k < M; ++k)
#pragma unroll
                        for (int x = 0; x < HEADS; ++x) tmem_ld<RW>(col + uint32_t(k * pr + (h + x) * RT), in[k][x]);
                    load_row<RW>(sm.qf[xp] + of_all + r0, qf);
                    load_row<RW>(sm.neg[g] + r0, neg);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < M; ++k)
#pragma unroll
                        for (int x = 0; x < HEADS; ++x) reg_fence<RW>(in[k][x]);
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        float y[M];
#pragma unroll
                        for (int k = 0; k < M; ++k) y[k] = __uint_as_float(ONE || !(lane & 16) ? in[k][0][r] : in[k][HEADS - 1][r]);
                        raw[r] = __float_as_uint(M == 1 ? y[0] : y[0] + (y[M / 2] + y[M - 1]));
                    }
                    if constexpr (RW == 1) {
                        v[0] = fmaf(__uint_as_float(raw[0]), ks * qf[0], i == first ? lv : neg[0] + lv);
                    } else {
                        const float2 ks2 = make_float2(ks, ks), lv2 = make_float2(lv, lv);
#pragma unroll
                        for (int r = 0; r < RW; r += 2) {
                            const float2 off = i == first ? lv2 : dev::add2(make_float2(neg[r], neg[r + 1]), lv2);
                            const float2 y = dev::fma2(make_float2(__uint_as_float(raw[r]), __uint_as_float(raw[r + 1])),
                                                  dev::mul2(ks2, make_float2(qf[r], qf[r + 1])), off);
                            v[r] = y.x, v[r + 1] = y.y;
                        }
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(bar(sm.s_free[x]));
                if (masked) {
                    if (ONE) must(!flags[0] && wait(bar(sm.v_full[s]), round));  // (what is zeroed must not be copied later)
#pragma unroll
                    for (int r = 0; r < RW; ++r)
                        if (key >= sm.lim[xp][of_all + r0 + r]) v[r] = -INFINITY;
                    // rows that nobody sees may hold anything
                    if (part == 0 && (!WIDE || g == 0) && key >= here.keys)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            dev::st_shared_v4(sb + uint32_t(s) * STAGE_BYTES + TILE_BYTES + uint32_t(row) * 128 + (uint32_t((k + lane) & 7) << 4),
                                              make_uint4(0, 0, 0, 0));
                }
                // Does one pass 2^8?
                bool pass = i == first;
                if (!pass) {
                    float most = v[0];
#pragma unroll
                    for (int r = 1; r < RW; ++r) most = fmaxf(most, v[r]);
                    pass = barrier_or(1 + g, NSOFT / GROUPS * 32, most > RESCALE_LOG2);
                }
                // the product that read P' (and wrote O) before is done
                if (t >= STEP) must(!flags[0] && wait(bar(sm.p_free[g]), turn ^ 1));
                if (pass) {
                    if constexpr (ONE) {
                        const float y = max_rows<RW>(v, lane);
                        if (lane < RW) sm.red[g][w][part * RW + lane] = y;
                    } else {
                        float mv[RW];
#pragma unroll
                        for (int r = 0; r < RW; ++r) mv[r] = v[r];
                        reduce16<RW, false>(mv, lane);
                        store_reduced<RW>(sm.red[g][hw] + part * RW, mv, lane);
                    }
                    group_sync();
                    // every warp of the group comes to the same references
                    float corr = 1.f;
                    if (lane < pairs) {
                        float top = -INFINITY;
                        if constexpr (ONE) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) top = fmaxf(top, sm.red[g][k][lane]);
                        } else {
                            for (int k = 0; k < pages; ++k) top = fmaxf(top, sm.red[g][k * nh + my_head][my_row]);
                        }
                        // (keys that a row sees come before those it does not: one that sees
                        // none in its first tile sees none later)
                        const float delta = i == first ? (top == -INFINITY ? 0.f : top - room) : fmaxf(top - room, 0.f);
                        corr = ex2(-0.5f * delta);
                        mo = i == first ? delta : mo + delta;
                        sm.neg[g][lane] = -mo;
                        sm.delta[g][lane] = delta;
                    }
                    sm.corr[g][lane] = corr;
                    __syncwarp();
                    {
                        float y[RW];
                        load_row<RW>(sm.delta[g] + r0, y);
#pragma unroll
                        for (int r = 0; r < RW; ++r) v[r] -= y[r];
                    }
                    if (i != first) {
                        float y[RW];
                        load_row<RW>(sm.corr[g] + r0, y);
#pragma unroll
                        for (int r = 0; r < RW; ++r) sum[r] *= y[r], sum[r] *= y[r];
                        // O of the tiles before, at the new references
                        tc::fence_after();
                        const uint32_t at = tmem + lanes + O_COL + uint32_t(g) * O_NEXT;
                        for (int c0 = 16 * part; c0 < 4 * ps; c0 += 16 * C::SPLIT) {
                            uint32_t o[16];
                            tmem_ld<16>(at + uint32_t(c0), o);
                            tc::tmem_ld_wait();
                            reg_fence<16>(o);
#pragma unroll
                            for (int k = 0; k < 16; k += 4) {
                                float y[4];
                                load_row<4>(sm.corr[g] + ((c0 + k) & (ps - 1)), y);
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[k + e] = __float_as_uint(__uint_as_float(o[k + e]) * y[e] * y[e]);
                            }
                            tmem_st8(at + uint32_t(c0), o);
                            tmem_st8(at + uint32_t(c0) + 8, o + 8);
                        }
                        tc::tmem_st_wait();
                    }
                }
                // P' of this key, and what it is of the sum
                float per = lv == lv ? ex2(-lv) : 1.f;
                if (lv < SMALL_LOG2) {
                    per = 0.f;
#pragma unroll
                    for (int r = 0; r < RW; ++r) sum[r] += ex2(v[r] - lv);
                    if (sm.v_scale[s][hw] == 0.f)
#pragma unroll
                        for (int r = 0; r < RW; ++r) v[r] = -INFINITY;  // (zeros are zeros)
                }
                constexpr int W = RW < 16 ? RW : 16;  // bytes of a store
#pragma unroll
                for (int q0 = 0; q0 < RW; q0 += W) {
                    uint32_t c[4][W < 4 ? 1 : W / 4];
#pragma unroll
                    for (int e = 0; e < W; e += 2) {
                        float2 f = make_float2(ex2(v[q0 + e]), 0.f);
                        if constexpr (W > 1) {
                            f.y = ex2(v[q0 + e + 1]);
                            const float2 y = dev::fma2(f, make_float2(per, per), make_float2(sum[q0 + e], sum[q0 + e + 1]));
                            sum[q0 + e] = y.x, sum[q0 + e + 1] = y.y;
                        } else {
                            sum[0] = fmaf(f.x, per, sum[0]);
                        }
                        uint32_t two[4];
                        split4(f, two);
#pragma unroll
                        for (int k = 0; k < 4; ++k) c[k][e / 4] = e % 4 ? __byte_perm(c[k][e / 4], two[k], 0x5410) : two[k];
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t n = uint32_t(k * ps + r0 + q0), to = p_row + (((n >> 4) ^ p_swz) << 4) + (n & 15);
                        if constexpr (W == 16)
                            dev::st_shared_v4(to, make_uint4(c[k][0], c[k][1], c[k][2], c[k][3]));
                        else if constexpr (W == 8)
                            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(to), "r"(c[k][0]), "r"(c[k][1]) : "memory");
                        else if constexpr (W == 4)
                            dev::st_shared_u32(to, c[k][0]);
                        else if constexpr (W == 2)
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(uint16_t(c[k][0])) : "memory");
                        else
                            asm volatile("st.shared.u8 [%0], %1;" ::"r"(to), "r"(c[k][0]) : "memory");
                    }
                }
                dev::fence_proxy_async_smem();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(bar(sm.p_full[g]));
                if ((s += STEP) >= ns) s -= ns, round ^= 1;
                if (i == first) look_ahead();
            }
            if (first >= tiles) look_ahead();
            // ---- the piece's end
            reduce16<RW, true>(sum, lane);
            if constexpr (ONE) {  // both halves' keys are of the one head
                sum[0] += __shfl_xor_sync(FULL, sum[0], 16);
                store_reduced<RW>(sm.sums[xp][g] + 32 * w + part * RW, sum, lane);
            } else {
                store_reduced<RW>(sm.sums[xp][g] + 16 * hw + part * RW, sum, lane);
            }
            if (w == 0 && part == 0) sm.ref[xp][g][lane] = mo;
            // the last product of each group
            t0 += tiles;
#pragma unroll
            for (int k = 1; k <= GROUPS; ++k)
                if (WIDE ? k == 1 : tiles >= k) must(!flags[0] && wait(bar(sm.p_free[WIDE ? g : (t0 - k) & 1]), uint32_t(WIDE ? t0 - k : (t0 - k) >> 1) & 1));
            all_sync();
            tc::fence_after();
            // the groups' sums and accumulators at one reference (of those that have seen a
            // key); WIDE: the rows are the group's own
            float M = -INFINITY, l = 0.f, lg[GROUPS], fo[GROUPS];
#pragma unroll
            for (int x = 0; x < GROUPS; ++x) {
                lg[x] = 0.f;
                if (lane < pairs && (!WIDE || x == g)) {
                    if constexpr (ONE) {
                        for (int k = 0; k < 4; ++k) lg[x] += sm.sums[xp][x][32 * k + lane];
                    } else {
                        for (int k = 0; k < pages; ++k) lg[x] += sm.sums[xp][x][16 * (k * nh + my_head) + my_row];
                    }
                }
                fo[x] = lg[x] == 0.f ? -INFINITY : sm.ref[xp][x][lane];
                M = fmaxf(M, fo[x]);
            }
#pragma unroll
            for (int x = 0; x < GROUPS; ++x) {
                const float half = lg[x] == 0.f ? 0.f : ex2(0.5f * (fo[x] - M));
                l += lg[x] * half * half;  // (a NaN stays)
                fo[x] = half * half;
            }
            const bool whole = here.first == 0 && here.last == here.tiles;
            const int64_t slot = 2 * int64_t(blockIdx.x) + (here.first == 0);
            float *acc = a.part_acc + (slot * E4M3_SLOT + of_all) * E4M3_D;
            if (!whole && w == 0 && part == 0 && (WIDE || g == 0) && lane < pairs) a.part_ml[slot * E4M3_SLOT + of_all + lane] = make_float2(M, l);
            const float over = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;  // (NaN sums stay)
            for (int c0 = 8 * (WIDE ? part : set); c0 < pairs; c0 += 8 * (WIDE ? C::SPLIT : SETS)) {  // eight pairs at a time, a set's
                float y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = 0.f;
#pragma unroll
                for (int x = 0; x < GROUPS; ++x) {
                    if (WIDE && x != g) continue;
                    uint32_t o[4][8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_ld<8>(tmem + lanes + O_COL + uint32_t(x) * O_NEXT + uint32_t(k * ps + c0), o[k]);
                    tc::tmem_ld_wait();
                    const bool there = WIDE || tiles > 1 || ((t0 - 1) & 1) == x;  // (a group without a tile has no accumulator)
#pragma unroll
                    for (int k = 0; k < 4; ++k) reg_fence<8>(o[k]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float z = __uint_as_float(o[3][k]);
#pragma unroll
                        for (int v = 2; v >= 0; --v) z = fmaf(z, 0x1p-5f, __uint_as_float(o[v][k]));
                        z *= __shfl_sync(FULL, fo[x], c0 + k);
                        y[k] += there ? z : 0.f;
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float z = y[k] * __shfl_sync(FULL, over, c0 + k);
                    if (c0 + k >= pairs) continue;
                    if (!whole) {
                        acc[(c0 + k) * E4M3_D + row] = z;
                    } else {
                        const int64_t r = __shfl_sync(FULL, out_row, c0 + k);
                        if (r >= 0) {
                            if (a.bf16)
                                static_cast<__nv_bfloat16 *>(a.out)[r * E4M3_D + row] = __float2bfloat16_rn(z);
                            else
                                static_cast<__half *>(a.out)[r * E4M3_D + row] = __float2half_rn(z);
                        }
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(bar(sm.o_free));
            if (!whole) {
                // the last of the segment's pieces joins them
                __threadfence();
                const int c0 = here.start / walk.share, c1 = (here.start + here.tiles - 1) / walk.share;
                all_sync();
                if (sw == 0 && lane == 0) flags[1] = atomicAdd(a.tickets + c0, 1) == c1 - c0;
                all_sync();
                if (flags[1]) {
                    __threadfence();
                    if constexpr (WIDE)
                        join<NSOFT / GROUPS>(a, out_row, of_all, pairs, c0, c1, part * 4 + (sw & 3), lane);
                    else
                        join<NSOFT>(a, out_row, 0, pairs, c0, c1, sw, lane);
                    if (sw == 0 && lane == 0) a.tickets[c0] = 0;  // as the next launch finds it
                }
            }
            ++np;
        }
    }

    // ---- teardown: every role is done; the MMAs have completed
    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, TMEM_COLS);
    }
    if (warp == 0 && lane == 0 && flags[0]) {
        // after an abort, the copies that may still land
        const volatile int never = 0;
        for (int i = issued > ns ? issued - ns : 0; i < issued; ++i)
            dev::mbar_wait_bounded(bar(sm.full[i % ns]), uint32_t(i / ns) & 1, &never, WAIT_TIMEOUT_NS);
    }
}

}  // namespace e4
}  // namespace kvc
