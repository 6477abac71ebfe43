// kvc_e4m3_rows.cu -- attention of long prompt chunks over the 8-bit paged cache:
// query rows on the tensor cores' M, codes widened to fp16 in shared memory.
//
// The kernel of kvc_e4m3_tc.cuh has keys on M, so that few query rows cost little.
// With 128 query rows and more that order pays for each row what this one pays for
// 128: a row's scores lie in one thread, so that maximum and sum need no other, and a
// probability is one fp16 value instead of four of 8 bits.
//
// A tile of the line (kvc_e4m3_tc.cuh) is 128 keys of one KV head, a segment up to
// 2 TB tokens (TB = 128 / g) of one (sequence, KV head) as two query tiles of 128 rows,
// which share each tile of keys.  Per tile and query tile x, as the kernel for 16-bit
// caches (kvc_rows_tc.cuh) has it:
//   S_x = Q_x . Kc^T      queries scaled by a power of two so that a row's largest
//                         element is 2^14 ... 2^15: exact in fp16 down to 2^-28 of it
//   P_x = 2^(s - mo + 7) vs   one thread per row; over S_x, as fp16
//   O_x += P_x . Vc
// with the codes as fp16 (exact), the blocks' scales of K in the scores and of V in P;
// 2^(s - mo + 7) sums up to what the output is divided by.  References mo (of s + log2
// vs) as in kvc_e4m3_tc.cuh; 2^7 keeps probabilities away from fp16's smallest.  A
// block whose scale is NaN makes the sum of the rows that see a key of it NaN: as a
// factor it would reach those too that do not.
//
// Warps: 0-3 softmax and epilogue of query tile 0, 4-7 of 1; 8 walks the line, hands
// the pieces to the others and copies the codes of a tile (K_0 V_0 K_1 ...) into the
// second half of its stage, row behind row: where the second halves of the rows as fp16
// are to stand, so that 10 and 11 widen each row in place (rows that nobody sees become
// zeros); 9 issues the MMAs.  A cut segment's pieces are joined by the CTA that finds
// itself the last.  Every wait is bounded, and after one that ran out every role leaves.
//
// Measured (bf16, 32 heads over 8): 8 chunks of 512 tokens over 4,096 rows 289 us, 1.01
// PFLOP/s; a prompt of 4,096 tokens 183 us; 4 chunks of 200 - 500 tokens over up to 4,000
// rows 87 us (190 with the kernel that has keys on M).  A tile of 256 query rows takes
// 2.3 us, bound by each query tile's chain: 1.2 us its softmax (half of it the maxima),
// 0.6 its MMAs, the rest hand-overs and the other query tile's MMAs; without the softmax
// it would take 1.6, without the widening 2.2.  What it took from 162 to 87: codes widened
// by threads from memory 142, copied first and widened in place 106, MMAs issued by an
// elected thread 92, maxima of blocks before their scales 86, scales waited for apart
// from V 84.
#include "kvc_e4m3_tc.cuh"
#include "kvc_rows_tc.cuh"

namespace kvc {
namespace {

using e4::FULL;
using e4::Piece;
using e4::Walker;
using e4::ex2;

using RC = RowsTcCfg<128>;
constexpr int NS = RC::NS, TILE_BYTES = RC::TILE_BYTES, BLK = RC::BLK, THREADS = RC::THREADS;
constexpr float SHIFT = 7.f;
constexpr float LEAST = 0x1p-90f, TINY = 0x1p-126f;

struct RowsSmall {
    float ks[4][8], vs[4][8], lv[4][8];  // of a tile's blocks: the scales (NaN as 0), log2 of V's
    uint32_t odd[4];                     // the blocks that have a NaN one
    uint64_t raw[NS], full[NS], empty[NS], scales[4];
    uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_free[2], q_full[2], mma_done;
    uint64_t item_full[2], item_empty[2], join_in, join_out;
    int64_t plan[THREADS / 32];
    struct Item {
        Piece p;     // b < 0: no more
        int c0, c1;  // the CTAs that have pieces of the segment
    } item[2];
    uint32_t pages[NS];  // the blocks that a stage has
    uint32_t tmem;
    int32_t flags[2];  // abort; last of the pieces
};
constexpr int SMEM = 1024 + RC::BAR_OFF + int(sizeof(RowsSmall));
static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");

// A warp's 32 query rows of a piece into their places, scaled; returns what a score of
// this lane's row has to be multiplied by.  row: this lane's row of q, or -1: zeros.
__device__ __forceinline__ float load_queries(const E4m3TcArgs &a, int row, uint32_t tile, int r0, int lane) {
    constexpr int BATCH = 16;
    const int half = lane >> 4, c = lane & 15;  // row (of two) and 16-byte chunk of a step
    float qf = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < 16; i0 += BATCH) {
        uint4 raw[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int from = __shfl_sync(FULL, row, 2 * (i0 + i) + half);
            raw[i] = from >= 0 ? dev::ld(static_cast<const uint4 *>(a.q) + int64_t(from) * 16 + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            float2 y[4];
            uint32_t top = 0;  // (as integers: infinities and NaN are above all others)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t w = (&raw[i].x)[k];
                y[k] = a.bf16 ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)) : __half22float2(*reinterpret_cast<const __half2 *>(&w));
                top = max(top, max(__float_as_uint(y[k].x) & 0x7fffffffu, __float_as_uint(y[k].y) & 0x7fffffffu));
            }
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(FULL, top, o));
            top >>= 23;
            const bool odd = top == 255;
            const uint32_t ex = odd ? 15u : max(top, 15u);
            const float up = __uint_as_float((268u - ex) << 23);  // the largest becomes 2^14 ... 2^15
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = odd ? 0u : MmaOps<__half>::pack(y[k].x * up, y[k].y * up);
            dev::st_shared_v4(RC::swz(tile, r0 + 2 * (i0 + i) + half, c), make_uint4(w[0], w[1], w[2], w[3]));
            const float f = __shfl_sync(FULL, odd ? __int_as_float(0x7fffffff) : __uint_as_float((ex - 14u) << 23) * a.scale_log2, (lane & 1) * 16);
            if (lane >> 1 == i0 + i) qf = f;
        }
    }
    return qf;
}

// 32 outputs of a row
__device__ __forceinline__ void store32(const E4m3TcArgs &a, int row, int q, const float (&y)[32]) {
    uint4 *to = static_cast<uint4 *>(a.out) + int64_t(row) * 16 + 4 * q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float u = y[8 * i + 2 * k], v = y[8 * i + 2 * k + 1];
            w[k] = a.bf16 ? MmaOps<__nv_bfloat16>::pack(u, v) : MmaOps<__half>::pack(u, v);
        }
        to[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// SHORT: for limits below those for which rows_wait suspends a warp (as an operand of the
// waits that time costs 2 % of a call).
template <bool SHORT>
__global__ void __launch_bounds__(THREADS, 1) e4m3_rows_kernel(const __grid_constant__ E4m3TcArgs a) {
    constexpr uint32_t IDESC_S = tc::idesc_f16_f32acc(false, 128, 128, false, false), IDESC_O = tc::idesc_f16_f32acc(false, 128, 128, false, true);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (dev::smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = dev::smem_addr(smem), ring = sb + RC::RING_OFF;
    RowsSmall &sm = *reinterpret_cast<RowsSmall *>(smem + RC::BAR_OFF);
    volatile int *flags = sm.flags;
    const auto bar = [](const uint64_t &x) { return dev::smem_addr(&x); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.group, TB = 128 / G;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            dev::mbar_init(bar(sm.raw[s]), 1);   // the codes are there
            dev::mbar_init(bar(sm.full[s]), 2);  // both halves of the rows are widened
            dev::mbar_init(bar(sm.empty[s]), 1);  // the commit behind the stage's last MMA
        }
        for (int x = 0; x < 2; ++x) {
            dev::mbar_init(bar(sm.s_full[x]), 1);  // S_x is there, the product before it done
            dev::mbar_init(bar(sm.p_half[x]), 4);  // P_x of 64 keys
            dev::mbar_init(bar(sm.p_full[x]), 4);
            dev::mbar_init(bar(sm.o_full[x]), 1);  // a piece's last product
            dev::mbar_init(bar(sm.o_free[x]), 4);  // its accumulator is read
            dev::mbar_init(bar(sm.q_full[x]), 4);
            dev::mbar_init(bar(sm.item_full[x]), 1);
            dev::mbar_init(bar(sm.item_empty[x]), 11);  // every other warp has read it
        }
        for (int i = 0; i < 4; ++i) dev::mbar_init(bar(sm.scales[i]), 1);
        dev::mbar_init(bar(sm.join_in), 8);   // the softmax warps' partial results are written
        dev::mbar_init(bar(sm.join_out), 1);  // the last of the pieces is known
        dev::mbar_init(bar(sm.mma_done), 1);
        flags[0] = 0;
        dev::fence_mbar_init();
    }
    if (warp == RC::MMA_WARP) {
        tc::tmem_alloc(dev::smem_addr(&sm.tmem), RC::TMEM_COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sm.tmem;
    dev::grid_dependency_wait();
    dev::allow_dependents();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += THREADS)
            if (dev::packed_seq(a, 1, b).bad) dev::record_error(a.err, ERR_DEVICE_INDEX);

    Walker walk;
    const bool any = walk.init(a, sm.plan, warp, THREADS / 32, lane);
    const auto wait = [&](uint32_t b, uint32_t parity) {
        return SHORT ? dev::mbar_wait_bounded(b, parity, flags, a.timeout_ns) : rows_wait(b, parity, flags, a.timeout_ns);
    };
    const auto fail = [&] {
        if (lane == 0) {
            if (!flags[0]) dev::record_error(a.err, ERR_TIMEOUT);
            flags[0] = 1;
        }
    };
    // query tiles of a piece
    const auto tiles_of = [&](const Piece &p) { return min(p.n - p.j * a.tt, a.tt) > TB ? 2 : 1; };
    const auto item_there = [&](int k) { return wait(bar(sm.item_full[k & 1]), uint32_t(k >> 1) & 1); };
    bool ok = true;
    uint32_t issued = 0;
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(RC::REGS_OTHER));
        if (warp == 8) {
            // ------------------------------------------------------------ pieces and copies
            Piece p;
            bool more = any && walk.next(a, p, lane);
            for (int k = 0;; ++k) {
                if (k >= 2 && !__all_sync(FULL, wait(bar(sm.item_empty[k & 1]), uint32_t((k >> 1) - 1) & 1))) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    RowsSmall::Item &it = sm.item[k & 1];
                    it.p.b = -1;
                    if (more) it = {p, p.start / walk.share, (p.start + p.tiles - 1) / walk.share};
                    dev::mbar_arrive(bar(sm.item_full[k & 1]));
                }
                __syncwarp();
                if (!more) break;
                const int32_t *table = a.block_table + int64_t(p.b) * a.max_blocks;
                const int n_pages = (p.keys + 15) >> 4;
                const auto entry = [&](int t) {
                    const int page = t * 8 + lane;
                    if (lane >= 8 || t >= p.last || page >= n_pages) return -1;
                    const int phys = dev::ld(table + page);
                    if (phys >= 0 && phys < a.num_blocks) return phys;
                    dev::record_error(a.err, ERR_DEVICE_INDEX);
                    return -1;
                };
                int phys = entry(p.first);
                for (int t = p.first; ok && t < p.last; ++t) {
                    const int next = entry(t + 1);  // on its way meanwhile
                    const int64_t at = int64_t(max(phys, 0)) * a.H_kv + p.hg;
                    float ks = 0.f, vs = 1.f;
                    if (phys >= 0) ks = dev::ld(a.k_scale + at), vs = dev::ld(a.v_scale + at);
                    const unsigned have = __ballot_sync(FULL, phys >= 0);
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const uint32_t s = issued % NS, gen = issued / NS;
                        if (gen > 0 && !__all_sync(FULL, wait(bar(sm.empty[s]), (gen - 1) & 1))) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) sm.pages[s] = have;
                        __syncwarp();
                        if (lane == 0) dev::mbar_arrive_expect_tx(bar(sm.raw[s]), uint32_t(__popc(have)) * 2048);
                        __syncwarp();
                        if (phys >= 0) dev::bulk_copy_g2s(ring + s * TILE_BYTES + BLK + lane * 2048, (v ? a.V : a.K) + at * 2048, 2048, bar(sm.raw[s]));
                        __syncwarp();
                        if (v == 0) {
                            // (the softmax has read what is here: where K_t's stage is free, both
                            // query tiles' products of V_(t - 3) are done)
                            const int slot = (issued >> 1) & 3;
                            const unsigned odd = __ballot_sync(FULL, ks != ks || vs != vs);
                            if (lane < 8) {
                                sm.ks[slot][lane] = ks == ks ? ks : 0.f;
                                sm.vs[slot][lane] = vs == vs ? vs : 0.f;
                                sm.lv[slot][lane] = __log2f(fmaxf(vs, LEAST));
                            }
                            if (lane == 0) sm.odd[slot] = odd;
                            __syncwarp();
                            if (lane == 0) dev::mbar_arrive(bar(sm.scales[slot]));
                        }
                        ++issued;
                    }
                    phys = next;
                }
                if (!ok) break;
                more = walk.next(a, p, lane);
            }
            if (!ok) fail();
        } else if (warp != RC::MMA_WARP) {
            // ------------------------------------------------------------ codes to fp16
            // Half of a tile's rows; lane: row (of four) and 16 codes of it.
            const int c = lane & 7, r4 = lane >> 3;
            const bool right = c >= 4;
            // chunks of the right half odd ones first, of the left one even ones: all banks
            const uint32_t to = uint32_t(right) * BLK + uint32_t(r4) * 128 + (uint32_t(((2 * (c & 3)) | int(right)) ^ r4) << 4);
            uint32_t place = 0;
            for (int k = 0;; ++k) {
                ok = __all_sync(FULL, item_there(k));
                if (!ok) break;
                const Piece &p = sm.item[k & 1].p;
                const int b = p.b, n = 2 * (p.last - p.first), keys = p.keys - 128 * p.first;
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(bar(sm.item_empty[k & 1]));
                if (b < 0) break;
                for (int i = 0; i < n; ++i, ++place) {
                    const uint32_t s = place % NS;
                    ok = __all_sync(FULL, wait(bar(sm.raw[s]), (place / NS) & 1));
                    if (!ok) break;
                    const uint32_t pages = sm.pages[s];
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        const int page = 4 * (warp - 10) + h;
                        const int seen = pages >> page & 1 ? keys - 128 * (i >> 1) - 16 * page : 0;  // rows
                        const uint32_t at = ring + s * TILE_BYTES + uint32_t(page) * 2048;
                        uint4 w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(w[e].x), "=r"(w[e].y), "=r"(w[e].z), "=r"(w[e].w)
                                         : "r"(at + BLK + uint32_t(e) * 512 + uint32_t(lane) * 16)
                                         : "memory");
                        if (seen < 16) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (4 * e + r4 >= seen) w[e] = make_uint4(0, 0, 0, 0);
                        }
                        __syncwarp();  // every lane has read what the others write over
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t x0 = right ? w[e].z : w[e].x, x1 = right ? w[e].w : w[e].y, y0 = right ? w[e].x : w[e].z, y1 = right ? w[e].y : w[e].w;
                            const uint32_t dst = (at + uint32_t(e) * 512 + to) ^ (e & 1 ? 64u : 0u);
                            dev::st_shared_v4(dst, make_uint4(dev::e4m3x2_to_f16x2(x0 & 0xffffu), dev::e4m3x2_to_f16x2(x0 >> 16),
                                                              dev::e4m3x2_to_f16x2(x1 & 0xffffu), dev::e4m3x2_to_f16x2(x1 >> 16)));
                            dev::st_shared_v4(dst ^ 16, make_uint4(dev::e4m3x2_to_f16x2(y0 & 0xffffu), dev::e4m3x2_to_f16x2(y0 >> 16),
                                                                   dev::e4m3x2_to_f16x2(y1 & 0xffffu), dev::e4m3x2_to_f16x2(y1 >> 16)));
                        }
                    }
                    dev::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) dev::mbar_arrive(bar(sm.full[s]));
                }
                if (!ok) break;
            }
            if (!ok) fail();
        } else if (tc::elect()) {
            // ------------------------------------------------------------ MMAs
            constexpr uint32_t HI = rows_desc_hi(1024);
            uint32_t stage = 0, phase = 0, tiles[2] = {0, 0}, pieces[2] = {0, 0};
            const auto must = [&](uint32_t b, uint32_t parity) { ok = ok && wait(b, parity); };
            const auto take = [&] {
                must(bar(sm.full[stage]), phase);
                const uint32_t s = stage;
                if (++stage == NS) stage = 0, phase ^= 1;
                return s;
            };
            const auto issue_s = [&](int x, uint32_t s) {
                const uint32_t kt = (ring + s * TILE_BYTES) >> 4, qt = (sb + x * TILE_BYTES) >> 4;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    tc::mma_f16_ss(tmem + RC::S_COL + 128 * x, rows_desc(qt + (((k >> 2) * BLK + (k & 3) * 32) >> 4), HI),
                                   rows_desc(kt + (((k >> 2) * BLK + (k & 3) * 32) >> 4), HI), IDESC_S, k > 0);
                tc::commit(bar(sm.s_full[x]));
            };
            const auto issue_o = [&](int x, uint32_t s, int k0, bool first) {  // 64 keys
                const uint32_t vt = (ring + s * TILE_BYTES) >> 4;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma_f16_ts(tmem + RC::O_COL + 128 * x, tmem + RC::S_COL + 128 * x + 8 * (k0 + k),
                                   rows_desc(vt + (((k0 + k) * 2048) >> 4) + ((BLK >> 4) << 16), HI), IDESC_O, k0 + k > 0 || !first);
            };
            for (int k = 0;; ++k) {
                ok = item_there(k);
                if (!ok) break;
                const Piece &p = sm.item[k & 1].p;
                const int b = p.b, n = p.last - p.first, nx = tiles_of(p);
                dev::mbar_arrive(bar(sm.item_empty[k & 1]));
                if (b < 0) break;
                {
                    must(bar(sm.q_full[0]), pieces[0] & 1);
                    uint32_t sk = take(), sv = 0;
                    if (ok) {
                        tc::fence_after();
                        issue_s(0, sk);
                    }
                    if (nx == 2) {
                        must(bar(sm.q_full[1]), pieces[1] & 1);
                        if (ok) {
                            tc::fence_after();
                            issue_s(1, sk);
                        }
                    }
                    if (ok) tc::commit(bar(sm.empty[sk]));
                    for (int j = 0; ok && j < n; ++j) {
                        sv = take();
                        if (j + 1 < n) sk = take();
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if (x == nx) break;
                            if (j == 0 && pieces[x] > 0) must(bar(sm.o_free[x]), (pieces[x] - 1) & 1);
                            const uint32_t turn = tiles[x]++ & 1;
                            must(bar(sm.p_half[x]), turn);
                            if (!ok) break;
                            tc::fence_after();
                            issue_o(x, sv, 0, j == 0);
                            must(bar(sm.p_full[x]), turn);
                            if (!ok) break;
                            tc::fence_after();
                            issue_o(x, sv, 4, j == 0);
                            if (j + 1 < n) {
                                if (x == nx - 1) tc::commit(bar(sm.empty[sv]));
                                issue_s(x, sk);
                                if (x == nx - 1) tc::commit(bar(sm.empty[sk]));
                            } else {
                                tc::commit(bar(sm.o_full[x]));
                                if (x == nx - 1) tc::commit(bar(sm.empty[sv]));
                                ++pieces[x];
                            }
                        }
                    }
                }
                if (!ok) break;
            }
            if (!ok) {
                if (!flags[0]) dev::record_error(a.err, ERR_TIMEOUT);
                flags[0] = 1;
            }
            // every MMA is done before tensor memory is freed
            tc::commit(bar(sm.mma_done));
            const volatile int never = 0;
            rows_wait(bar(sm.mma_done), 0, &never, WAIT_TIMEOUT_NS);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(RC::REGS_SOFTMAX));
        const int x = warp >> 2, r = threadIdx.x & 127;  // query tile; query row: tensor-memory lane
        const int tt = r / G;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const uint32_t s_t = tmem + lanes + RC::S_COL + 128 * x, o_t = tmem + lanes + RC::O_COL + 128 * x;
        float qf = 0.f;    // what its scores have to be multiplied by
        bool nan = false;  // it has an infinity or NaN
        int row = -1;      // of q and out
        int lim = 0;       // keys that it sees
        // the k-th piece, and its queries
        RowsSmall::Item it;
        const auto take = [&](int k) {
            ok = __all_sync(FULL, item_there(k));
            if (!ok) return false;
            it = sm.item[k & 1];
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(bar(sm.item_empty[k & 1]));
            const Piece &p = it.p;
            if (p.b < 0) return false;
            if (x >= tiles_of(p)) return true;
            const int t = p.j * a.tt + x * TB + tt;
            const bool live = tt < TB && t < p.n;
            row = live ? (p.lo + t) * a.H + p.hg * G + (r - tt * G) : -1;
            lim = live ? p.c + t + 1 : 0;
            qf = load_queries(a, row, sb + x * TILE_BYTES, r - lane, lane);
            nan = qf != qf;
            if (nan) qf = 0.f;
            dev::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(bar(sm.q_full[x]));
            return true;
        };
        uint32_t tile = 0, gt = 0, gp = 0, joins = 0;  // tiles so far; this query tile's, and its pieces
        bool more = take(0);
        for (int k = 1; more; ++k) {
            const int n = it.p.last - it.p.first, first = it.p.first, least = it.p.c + it.p.j * a.tt + 1, c0 = it.c0, c1 = it.c1;
            const bool works = x < tiles_of(it.p), whole = n == it.p.tiles;
            float m = 0.f;
            float2 sum[2] = {make_float2(nan ? __int_as_float(0x7fffffff) : 0.f, 0.f), make_float2(0.f, 0.f)};
            const int out_row = row;
            if (works) {
                const bool warp_ok = __any_sync(FULL, row >= 0);
                for (int i = 0; i < n; ++i, ++gt, ++tile) {
                    // (S first: query tile 1 may have skipped pieces, and only S tells it that the
                    // scales of four tiles ago, whose parity is the other one, are done)
                    ok = __all_sync(FULL, wait(bar(sm.s_full[x]), gt & 1) && wait(bar(sm.scales[tile & 3]), (tile >> 2) & 1));
                    if (!ok) break;
                    tc::fence_after();
                    if (!warp_ok) {
                        __syncwarp();
                        if (lane == 0) {
                            dev::mbar_arrive(bar(sm.p_half[x]));
                            dev::mbar_arrive(bar(sm.p_full[x]));
                        }
                        continue;
                    }
                    const int sees = lim - 128 * (first + i), slot = tile & 3;  // keys of the tile
                    const bool partial = 128 * (first + i + 1) > least;  // does not every row of the piece see all?
                    uint32_t sr[4][32];
                    float top = -INFINITY;  // of s + log2 vs
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
                                    if (32 * q + e >= sees) sr[q][e] = __float_as_uint(-INFINITY);
                        }
                        const float4 ks = *reinterpret_cast<const float4 *>(&sm.ks[slot][4 * hh]), lv = *reinterpret_cast<const float4 *>(&sm.lv[slot][4 * hh]);
#pragma unroll
                        for (int b = 4 * hh; b < 4 * hh + 4; ++b) {
                            const uint32_t *v = &sr[b >> 1][16 * (b & 1)];
                            float most[2] = {__uint_as_float(v[0]), __uint_as_float(v[1])};
#pragma unroll
                            for (int e = 2; e < 14; e += 4) {
                                most[0] = fmax3(most[0], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                                most[1] = fmax3(most[1], __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                            }
                            most[0] = fmax3(most[0], __uint_as_float(v[14]), __uint_as_float(v[15]));
                            top = fmaxf(top, fmaf(fmaxf(most[0], most[1]), fmaxf((&ks.x)[b & 3] * qf, TINY), (&lv.x)[b & 3]));
                        }
                    }
                    // The reference: the first tile's maximum; later raised where one passes it
                    // by 2^8.  (A row that sees none of its first tile sees none later.)
                    const bool raise = i == 0 ? top > -INFINITY : top > m + e4::RESCALE_LOG2;
                    if (__any_sync(FULL, raise)) {
                        const float half = raise ? ex2(0.5f * (m - top)) : 1.f;
                        if (raise) m = top;
                        if (i > 0) {
                            const float2 h2 = make_float2(half, half), c2 = make_float2(half * half, half * half);
                            sum[0] = __fmul2_rn(__fmul2_rn(sum[0], h2), h2);
                            sum[1] = __fmul2_rn(__fmul2_rn(sum[1], h2), h2);
#pragma unroll 1
                            for (int q = 0; q < 8; ++q) {
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
                    // (blocks [0, (sees + 15) / 16) are this row's)
                    if (const uint32_t odd = sm.odd[slot]; odd && sees > 0 && (odd & ((2u << min((sees - 1) >> 4, 7)) - 1))) sum[0].x = __int_as_float(0x7fffffff);
                    const float2 off = make_float2(SHIFT - m, SHIFT - m);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 ks = *reinterpret_cast<const float2 *>(&sm.ks[slot][2 * q]), vs = *reinterpret_cast<const float2 *>(&sm.vs[slot][2 * q]);
                        uint32_t pk[16];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const float f = fmaxf((b ? ks.y : ks.x) * qf, TINY), w = b ? vs.y : vs.x;  // (f not 0: it meets the masked scores' -inf)
#pragma unroll
                            for (int e = 16 * b; e < 16 * b + 16; e += 2) {
                                float2 y = __ffma2_rn(make_float2(__uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1])), make_float2(f, f), off);
                                y = make_float2(ex2(y.x), ex2(y.y));
                                sum[(e >> 1) & 1] = __fadd2_rn(sum[(e >> 1) & 1], y);
                                y = __fmul2_rn(y, make_float2(w, w));
                                pk[e / 2] = MmaOps<__half>::pack(y.x, y.y);
                            }
                        }
                        rows_tmem_st16(s_t + 16 * q, pk);  // over scores that are in registers
                        if (q & 1) {
                            tc::tmem_st_wait();
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) dev::mbar_arrive(bar(q == 1 ? sm.p_half[x] : sm.p_full[x]));
                        }
                    }
                }
            } else {
                tile += n;
            }
            if (!ok) break;
            more = take(k);  // the next one's queries: this one's scores are all there
            if (!ok) break;
            // ---- the piece's end
            const float2 two = __fadd2_rn(sum[0], sum[1]);
            const float l = two.x + two.y;
            const int64_t slot = 2 * int64_t(blockIdx.x) + (first == 0);
            const int at = x * 128 + r;
            if (works) {
                ok = __all_sync(FULL, wait(bar(sm.o_full[x]), gp & 1));
                if (!ok) break;
                ++gp;
                tc::fence_after();
                const float f = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;  // (NaN sums stay)
                if (!whole) a.part_ml[slot * E4M3_SLOT + at] = make_float2(l == 0.f ? -INFINITY : m, l);
                float4 *acc = reinterpret_cast<float4 *>(a.part_acc) + slot * (E4M3_SLOT * 32) + at;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t o[32];
                    tc::tmem_ld32(o_t + 32 * q, o);
                    tc::tmem_ld_wait();
                    tc::reg_fence(o);
                    float y[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(o[e]) * f;
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[(8 * q + e) * E4M3_SLOT] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                    } else if (out_row >= 0) {
                        store32(a, out_row, q, y);
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(bar(sm.o_free[x]));
            }
            if (!whole) {
                // the last of the segment's pieces joins them
                __threadfence();
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(bar(sm.join_in));
                if (warp == 0) {
                    ok = __all_sync(FULL, wait(bar(sm.join_in), joins & 1));
                    if (!ok) break;
                    if (lane == 0) {
                        flags[1] = atomicAdd(a.tickets + c0, 1) == c1 - c0;
                        dev::mbar_arrive(bar(sm.join_out));
                    }
                }
                ok = __all_sync(FULL, wait(bar(sm.join_out), joins & 1));
                if (!ok) break;
                ++joins;
                if (flags[1]) {
                    __threadfence();
                    const auto slot_of = [&](int c) { return 2 * int64_t(c) + (c == c0); };
                    if (works && out_row >= 0) {
                        float M = -INFINITY, L = 0.f;
                        for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(a.part_ml + slot_of(c) * E4M3_SLOT + at).x);
                        for (int c = c0; c <= c1; ++c) {
                            const float2 ml = __ldcg(a.part_ml + slot_of(c) * E4M3_SLOT + at);
                            const float half = ex2(0.5f * (ml.x - M));
                            L += ml.x == -INFINITY ? ml.y : ml.y * half * half;  // (0, or a NaN that stays)
                        }
                        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            float y[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) y[e] = 0.f;
                            for (int c = c0; c <= c1; ++c) {
                                const float mc = __ldcg(a.part_ml + slot_of(c) * E4M3_SLOT + at).x;
                                const float f = mc == -INFINITY ? 0.f : ex2(mc - M) * inv;
                                const float4 *acc = reinterpret_cast<const float4 *>(a.part_acc) + slot_of(c) * (E4M3_SLOT * 32) + at;
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float4 z = __ldcg(acc + (8 * q + e) * E4M3_SLOT);
                                    y[4 * e] = fmaf(z.x, f, y[4 * e]), y[4 * e + 1] = fmaf(z.y, f, y[4 * e + 1]);
                                    y[4 * e + 2] = fmaf(z.z, f, y[4 * e + 2]), y[4 * e + 3] = fmaf(z.w, f, y[4 * e + 3]);
                                }
                            }
                            store32(a, out_row, q, y);
                        }
                    }
                    if (threadIdx.x == 0) a.tickets[c0] = 0;  // as the next launch finds it
                }
            }
        }
        if (!ok) fail();
    }

    // ---- teardown: every role is done; the MMAs have completed
    tc::fence_before();
    __syncthreads();
    if (warp == RC::MMA_WARP) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, RC::TMEM_COLS);
    }
    if (warp == 8 && lane == 0 && flags[0]) {
        // after an abort, the copies that may still land
        const volatile int never = 0;
        for (uint32_t i = issued > NS ? issued - NS : 0; i < issued; ++i) rows_wait(bar(sm.raw[i % NS]), (i / NS) & 1, &never, WAIT_TIMEOUT_NS);
    }
}

}  // namespace

cudaError_t e4m3_rows_set_max_smem() {
    const cudaError_t e = cudaFuncSetAttribute(e4m3_rows_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(e4m3_rows_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
}

cudaError_t launch_e4m3_rows(const E4m3TcArgs &a, int grid, cudaStream_t s) {
    return launch_pdl(a.timeout_ns < WAIT_TIMEOUT_NS / 100 ? e4m3_rows_kernel<true> : e4m3_rows_kernel<false>, dim3(grid), dim3(THREADS), SMEM, s, a);
}

}  // namespace kvc
