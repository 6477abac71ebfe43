// kvc_rope.cu -- new tokens' queries and keys rotated by their positions, and
// their keys and values stored in the cache.
//
// A pair (x, y) of a row's elements turns by the angle of the token's position:
//   x' = x cos - y sin,  y' = y cos + x sin
// in fp32, each product and sum rounded by itself, so that the result does not
// depend on how the compiler contracts them (codes of 8 bits are chosen from it).
// The pairs are (i, i + half) of the first 2 half elements, or (2 i, 2 i + 1).
//
// Warps take items.  A row item is a token and some of its heads: a lane holds the
// two vectors of its pairs, keeps their cosines and sines, and goes over the heads.
// A page item (8-bit caches) is a range of tokens of one KV head, K or V (16 tokens:
// K and V): the warp that has a block's first new token takes all of the block's new
// rows at once, so that the scale is chosen, the older rows' codes follow it and the
// block is written by one warp, whatever the order of the others.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/kvc.h"
#include "kvc_e4m3.cuh"

namespace kvc {
namespace {

// What a kernel does: rows of caches of the rows' own type, or of no cache; of int8
// ones; blocks of 8-bit ones, and rows of no cache in every second thread block.
enum Mode { PLAIN, INT8, BLOCKS };
constexpr unsigned FULL = 0xffffffffu;

template <int BYTES>
struct Vec;
template <>
struct Vec<16> {
    using type = uint4;
};
template <>
struct Vec<8> {
    using type = uint2;
};

// Two neighbouring elements, and back.
template <typename T>
__device__ __forceinline__ float2 widen2(const T *p);
template <>
__device__ __forceinline__ float2 widen2(const float *p) { return make_float2(p[0], p[1]); }
template <>
__device__ __forceinline__ float2 widen2(const __nv_bfloat16 *p) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 widen2(const __half *p) { return __half22float2(*reinterpret_cast<const __half2 *>(p)); }
__device__ __forceinline__ void narrow2(float *p, float2 x) { p[0] = x.x, p[1] = x.y; }
__device__ __forceinline__ void narrow2(__nv_bfloat16 *p, float2 x) { *reinterpret_cast<__nv_bfloat162 *>(p) = __float22bfloat162_rn(x); }
__device__ __forceinline__ void narrow2(__half *p, float2 x) { *reinterpret_cast<__half2 *>(p) = __float22half2_rn(x); }

// The two vectors of VE elements that lane unit u of a row holds, and its pairs.
template <typename T, int VE>
struct Unit {
    using V = typename Vec<sizeof(T) * VE>::type;
    int at[2];      // first elements
    bool turns;     // are they rotated?
    int angle;      // first of its VE pairs
    bool side;      // pairs (i, i + half): one element of each vector; else neighbours

    __device__ __forceinline__ Unit(const RopeArgs &a, int u) {
        const int ru = a.half / VE;  // units that rotate
        turns = u < ru;
        angle = u * VE;
        side = !a.interleaved;
        if (side && turns) {
            at[0] = u * VE;
            at[1] = a.half + u * VE;
        } else {
            at[0] = 2 * u * VE;  // (units behind the rotated ones: 2 ru VE + 2 (u - ru) VE)
            at[1] = at[0] + VE;
        }
    }
    __device__ __forceinline__ void angles(const RopeArgs &a, int place, float (&cs)[VE], float (&sn)[VE]) const {
        if (!turns) return;
        const float *t = a.cos_sin + int64_t(place) * 2 * a.half + angle;
#pragma unroll
        for (int e = 0; e < VE; e += 4) {
            const float4 c = dev::ld(reinterpret_cast<const float4 *>(t + e)), s = dev::ld(reinterpret_cast<const float4 *>(t + a.half + e));
            cs[e] = c.x, cs[e + 1] = c.y, cs[e + 2] = c.z, cs[e + 3] = c.w;
            sn[e] = s.x, sn[e + 1] = s.y, sn[e + 2] = s.z, sn[e + 3] = s.w;
        }
    }
    __device__ __forceinline__ void load(const uint8_t *row, V (&raw)[2]) const {
        raw[0] = dev::ld(reinterpret_cast<const V *>(row + at[0] * int(sizeof(T))));
        raw[1] = dev::ld(reinterpret_cast<const V *>(row + at[1] * int(sizeof(T))));
    }
    // the same bits, as far as the compiler knows others
    __device__ __forceinline__ static void keep(V (&raw)[2]) {
        uint32_t *w = reinterpret_cast<uint32_t *>(raw);
#pragma unroll
        for (int i = 0; i < int(sizeof(raw) / 4); ++i) asm volatile("" : "+r"(w[i])::"memory");
    }
    // x: the elements of both vectors, rotated, in pairs of neighbours
    __device__ __forceinline__ void turn(const V (&raw)[2], const float (&cs)[VE], const float (&sn)[VE], bool rotate,
                                         float2 (&x)[VE]) const {
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int e = 0; e < VE / 2; ++e) x[v * VE / 2 + e] = widen2<T>(reinterpret_cast<const T *>(&raw[v]) + 2 * e);
        if (!turns || !rotate) return;
        if (side) {
#pragma unroll
            for (int e = 0; e < VE / 2; ++e) {
                const float2 c = make_float2(cs[2 * e], cs[2 * e + 1]), s = make_float2(sn[2 * e], sn[2 * e + 1]), p = x[e], q = x[VE / 2 + e];
                x[e] = dev::sub2(dev::product2(p, c), dev::product2(q, s));
                x[VE / 2 + e] = dev::add2(dev::product2(q, c), dev::product2(p, s));
            }
        } else {
#pragma unroll
            for (int e = 0; e < VE; ++e) {  // (x, y) (c, c), then -/+ (y, x) (s, s)
                const float2 p = x[e], c = dev::product2(p, make_float2(cs[e], cs[e])), s = dev::product2(make_float2(-p.y, p.x), make_float2(sn[e], sn[e]));
                x[e] = dev::add2(c, s);
            }
        }
    }
    __device__ __forceinline__ void store(uint8_t *row, const float2 (&x)[VE]) const {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            V raw;
#pragma unroll
            for (int e = 0; e < VE / 2; ++e) narrow2(reinterpret_cast<T *>(&raw) + 2 * e, x[v * VE / 2 + e]);
            *reinterpret_cast<V *>(row + at[v] * int(sizeof(T))) = raw;
        }
    }
    // VE one-byte codes of vector i
    __device__ __forceinline__ void store_codes(uint8_t *row, int i, const uint32_t *c) const {
        if constexpr (VE == 8)
            *reinterpret_cast<uint2 *>(row + at[i]) = make_uint2(c[0], c[1]);
        else
            *reinterpret_cast<uint32_t *>(row + at[i]) = c[0];
    }
};

// Position of packed row r of sequence s in the cache, and for the rotation;
// false (recorded) where the table of angles has none.
__device__ __forceinline__ bool place_of(const RopeArgs &a, int r, int pos, int &place) {
    place = a.positions ? dev::ld(a.positions + r) : pos;
    if (!a.cos_sin || (place >= 0 && place < a.n_positions)) return true;
    dev::record_error(a.err, ERR_DEVICE_INDEX);
    return false;
}

__device__ __forceinline__ const uint8_t *kv_row(const RopeArgs &a, const uint8_t *x, int64_t token, int b, int i, int r, int j) {
    return x + (a.kv_seq ? b * a.kv_seq + i * token : r * token) + j * a.kv_head;
}

template <typename T, int VE, Mode M>
__device__ __forceinline__ void row_item(const RopeArgs &a, unsigned item, int lane) {
    constexpr int STEP = 4;  // rows in flight per lane
    const int r = a.parts == 1 ? int(item) : int(item / unsigned(a.parts)), part = int(item) - r * a.parts;
    const int U = a.D / (2 * VE), u = lane % U, slot = lane / U, SL = 32 / U;
    const Unit<T, VE> unit(a, u);
    const int row_bytes = a.D * int(sizeof(T));
    // the token's heads: those of q, of k and of v, one behind another
    const int nq = a.q ? a.H : 0, nk = nq + a.H_kv;
    const int end = min(a.n_heads, (part + 1) * a.per_part);
    const uint8_t *qs = a.q + r * a.q_token, *ks = a.k + r * a.k_token - nq * row_bytes, *vs = a.v + r * a.v_token - nk * row_bytes;
    typename Unit<T, VE>::V raw[STEP][2];
    const auto fetch = [&](int h0) {
#pragma unroll
        for (int e = 0; e < STEP; ++e) {
            const int h = h0 + e * SL + slot;
            if (h < end) unit.load((h < nq ? qs : h < nk ? ks : vs) + h * row_bytes, raw[e]);
        }
    };
    fetch(part * a.per_part);  // on their way while the token's place is looked up
    // the token's sequence
    int b = -1, pos = 0;
    if (!a.cu_seqlens) {
        b = r;
        const dev::PackedSeq s = dev::packed_seq(a, 1, b);
        if (s.bad) return;
        pos = s.c;
    } else {
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            dev::PackedSeq s{};
            if (b0 + lane < a.B) s = dev::packed_seq(a, 0, b0 + lane);
            const unsigned hit = __ballot_sync(FULL, s.lo <= r && r - s.lo < s.n);
            if (hit) {
                const int src = __ffs(hit) - 1;
                b = b0 + src;
                pos = r - __shfl_sync(FULL, s.lo, src) + __shfl_sync(FULL, s.c, src);
                break;
            }
        }
        if (b < 0) return;
    }
    int place;
    if (!place_of(a, r, pos, place)) return;
    float cs[VE], sn[VE];
    unit.angles(a, place, cs, sn);
    // the token's row in the cache (KV head 0), and the distance between KV heads
    int64_t row = -1, step = 0;
    if (M != BLOCKS) {
        if (a.block_table) {
            const int phys = dev::ld(a.block_table + int64_t(b) * a.max_blocks + pos / 16);
            if (phys >= 0 && phys < a.num_blocks)
                row = int64_t(phys) * a.H_kv * 16 + pos % 16;
            else if (lane == 0)
                dev::record_error(a.err, ERR_DEVICE_INDEX);
            step = 16;
        } else {
            row = int64_t(b) * a.H_kv * a.max_ctx + pos;
            step = a.max_ctx;
        }
    }
    uint8_t *qd = a.q_out + int64_t(r) * a.H * row_bytes, *kd = a.k_out ? a.k_out + (int64_t(r) * a.H_kv - nq) * row_bytes : nullptr;
    for (int h0 = part * a.per_part; h0 < end; h0 += STEP * SL) {
        if (h0 > part * a.per_part) fetch(h0);
#pragma unroll
        for (int e = 0; e < STEP; ++e) {
            unit.keep(raw[e]);  // (one row at a time: registers)
            const int h = h0 + e * SL + slot;
            const bool live = h < end, is_q = h < nq, is_v = h >= nk;
            const int64_t to = row + (h - (is_v ? nk : nq)) * step;  // cache row
            uint8_t *cache = is_v ? a.V : a.K, *dense = is_q ? qd : is_v ? nullptr : kd;
            float2 x[VE];
            if (live) {
                unit.turn(raw[e], cs, sn, !is_v, x);
                if (dense) unit.store(dense + h * row_bytes, x);
            }
            if constexpr (M == PLAIN) {
                if (live && !is_q && row >= 0) unit.store(cache + to * row_bytes, x);
            }
            if constexpr (M == INT8) {
                // scale = absmax / 127, code = rint(x * (127 / absmax)), as kvc_append has it
                float am = 0.f;
                if (live)
#pragma unroll
                    for (int t = 0; t < VE; ++t) am = fmaxf(am, fmaxf(fabsf(x[t].x), fabsf(x[t].y)));
                for (int o = U / 2; o >= 1; o >>= 1) am = fmaxf(am, __shfl_xor_sync(FULL, am, o));
                if (live && !is_q && row >= 0) {
                    const float inv = am > 0.f ? 127.0f / am : 0.f;
                    const auto code = [&](float y) {
                        const int c = __float2int_rn(y * inv);
                        return uint32_t(c > 127 ? 127 : c < -127 ? -127 : c) & 0xffu;
                    };
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint32_t c[VE / 4];
#pragma unroll
                        for (int t = 0; t < VE / 4; ++t) {
                            const float2 y = x[v * VE / 2 + 2 * t], z = x[v * VE / 2 + 2 * t + 1];
                            c[t] = code(y.x) | code(y.y) << 8 | code(z.x) << 16 | code(z.y) << 24;
                        }
                        unit.store_codes(cache + to * a.D, v, c);
                    }
                    if (u == 0) (is_v ? a.v_scale : a.k_scale)[to] = am / 127.0f;
                }
            }
        }
    }
}

// The smallest power of two s with top <= 448 s (from 2^-126 up); 0 for 0.
__device__ __forceinline__ float e4m3_scale(float top) {
    if (!(top > 0.f)) return 0.f;
    const uint32_t bits = __float_as_uint(top);
    const int e = int(bits >> 23) - ((bits & 0x7fffffu) > 0x600000u ? 7 : 8);  // 448 = 1.75 * 2^8
    return __uint_as_float(uint32_t(max(e, 1)) << 23);
}

// The codes of a block's first rows, times f.
__device__ __forceinline__ void rescale_rows(uint8_t *block, int rows, float f, int lane) {
    for (int x16 = lane; x16 < rows * (E4M3_D / 16); x16 += 32) {
        uint4 v = dev::ld(reinterpret_cast<const uint4 *>(block) + x16);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t l2 = dev::e4m3x2_to_f16x2(w[t] & 0xffffu), h2 = dev::e4m3x2_to_f16x2(w[t] >> 16);
            const float2 l = __half22float2(*reinterpret_cast<const __half2 *>(&l2)), h = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
            w[t] = dev::e4m3x2(__fmul_rn(l.x, f), __fmul_rn(l.y, f)) | dev::e4m3x2(__fmul_rn(h.x, f), __fmul_rn(h.y, f)) << 16;
        }
        reinterpret_cast<uint4 *>(block)[x16] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The scale that new rows with the largest element `top` make of a block's old one.  (One
// below 2^-126, which only a cache filled by other means has, is not kept: its reciprocal
// may be infinite, and a zero's code then NaN.)
__device__ __forceinline__ float next_scale(float old, float top) {
    return top <= 448.f * old && (old == 0.f || old >= 0x1p-126f) ? old : fmaxf(e4m3_scale(top), old > 0.f ? 0x1p-126f : 0.f);
}

// The scale of a block whose row `slot` has an infinity or NaN is a NaN that keeps the
// scale, a power of two or 0, of the rows before.  They are as they were as soon as that
// row or one before it is stored again: a rejected token takes no other with it.
__device__ __forceinline__ float bad_scale(float scale, int slot) { return __uint_as_float(0x7fc00000u | uint32_t(slot) << 8 | __float_as_uint(scale) >> 23); }
// What an append at row `slot` finds; NaN: rows before it are lost.
__device__ __forceinline__ float kept_scale(float scale, int slot) {
    const uint32_t bits = __float_as_uint(scale), e = bits & 0xffu;
    return scale == scale || (bits & 0xfffff000u) != 0x7fc00000u || e == 0xffu || slot > int(bits >> 8 & 15u) ? scale : __uint_as_float(e << 23);
}

// What page_rows leaves out: new rows one after the other, where one of them or the
// block's scale is not finite.
template <typename T, int VE>
__device__ __forceinline__ void odd_rows(const RopeArgs &a, int b, int lo, int c, int i0, int n, int j, bool is_v, int lane) {
    constexpr int U = E4M3_D / (2 * VE);
    const Unit<T, VE> unit(a, lane % U);
    const int phys = dev::ld(a.block_table + int64_t(b) * a.max_blocks + (c + i0) / 16);
    if (phys < 0 || phys >= a.num_blocks) return;  // (recorded)
    float *sp = (is_v ? a.v_scale : a.k_scale) + int64_t(phys) * a.H_kv + j;
    uint8_t *block = (is_v ? a.V : a.K) + (int64_t(phys) * a.H_kv + j) * (16 * E4M3_D);
    const bool rotate = !is_v && unit.turns;
    float2 x[VE];
    // row i, rotated, and its largest element; false: it is not stored
    const auto take = [&](int i, uint32_t &bits) {
        int place;
        if (!place_of(a, lo + i, c + i, place)) return false;
        typename Unit<T, VE>::V raw[2];
        float cs[VE], sn[VE];
        unit.load(is_v ? kv_row(a, a.v, a.v_token, b, i, lo + i, j) : kv_row(a, a.k, a.k_token, b, i, lo + i, j), raw);
        if (rotate) unit.angles(a, place, cs, sn);
        unit.turn(raw, cs, sn, rotate, x);
        float most = 0.f;
        for (int e = 0; e < VE; ++e) most = dev::max_abs_nan(dev::max_abs_nan(most, x[e].x), x[e].y);
        bits = __reduce_max_sync(FULL, __float_as_uint(most) & 0x7fffffffu);
        return true;
    };
    uint32_t bits;
    const float first = (c + i0) % 16 > 0 ? dev::ld(sp) : 0.f;
    bool odd = first != first;
    for (int i = i0; !odd && i < i0 + n; ++i) odd = take(i, bits) && bits >= 0x7f800000u;
    for (int i = i0; odd && i < i0 + n; ++i) {
        const int slot = (c + i) % 16;
        if (!take(i, bits)) continue;
        __syncwarp();  // (what the warp has written for the row before)
        const bool bad = bits >= 0x7f800000u;
        const float was = slot > 0 ? dev::ld(sp) : 0.f, old = kept_scale(was, slot);
        const bool lost = old != old;
        float scale = next_scale(old, bad ? 0.f : __uint_as_float(bits));
        if (bad && (__float_as_uint(scale) & 0x7fffffu))  // (one that is no power of two has no room)
            scale = fminf(__uint_as_float((__float_as_uint(scale) & 0x7f800000u) + 0x800000u), 0x1p127f);
        const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
        if (slot > 0 && !lost && scale != old) rescale_rows(block, slot, __fmul_rn(old, inv), lane);
        __syncwarp();
        if (lane < U)
            for (int v = 0; v < 2; ++v) {
                uint32_t codes[VE / 4];
                for (int t = 0; t < VE / 4; ++t) {
                    const float2 y = x[v * VE / 2 + 2 * t], z = x[v * VE / 2 + 2 * t + 1];
                    codes[t] = bad || lost ? 0u : dev::e4m3x2(y.x * inv, y.y * inv) | dev::e4m3x2(z.x * inv, z.y * inv) << 16;
                }
                unit.store_codes(block + slot * E4M3_D, v, codes);
            }
        if (lane == 0 && !lost) *sp = bad ? bad_scale(scale, slot) : scale;
        __syncwarp();
    }
}

// New rows [i0, i0 + n) of sequence b, all of one block, of KV head j of K or V; true, and
// nothing stored, where one of them or the block's scale is not finite.
// The warp holds them as they were read and rotates them twice, for the largest
// element and for the codes: as fp32 they would take the registers of two warps, and
// what bounds a prompt is how many reads are in flight.
template <typename T, int VE>
__device__ __forceinline__ bool page_rows(const RopeArgs &a, int b, int lo, int c, int i0, int n, int j, bool is_v, int lane) {
    constexpr int U = E4M3_D / (2 * VE), SL = 32 / U, P = 16 / SL;
    const int u = lane % U, slot = lane / U, pos0 = c + i0, s0 = pos0 % 16;
    const Unit<T, VE> unit(a, u);
    const int phys = dev::ld(a.block_table + int64_t(b) * a.max_blocks + pos0 / 16);
    typename Unit<T, VE>::V raw[P][2];
    int place[P];
    unsigned live = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int k = p * SL + slot, i = i0 + k;  // the k-th new row
        place[p] = 0;
        if (k < n) {
            unit.load(is_v ? kv_row(a, a.v, a.v_token, b, i, lo + i, j) : kv_row(a, a.k, a.k_token, b, i, lo + i, j), raw[p]);
            if (place_of(a, lo + i, c + i, place[p])) live |= 1u << p;
        }
    }
    if (phys < 0 || phys >= a.num_blocks) {
        if (lane == 0) dev::record_error(a.err, ERR_DEVICE_INDEX);
        return false;
    }
    if (!__any_sync(FULL, live != 0)) return false;
    float *sp = (is_v ? a.v_scale : a.k_scale) + int64_t(phys) * a.H_kv + j;
    const float old = s0 > 0 ? dev::ld(sp) : 0.f;
    uint8_t *block = (is_v ? a.V : a.K) + (int64_t(phys) * a.H_kv + j) * (16 * E4M3_D);
    const bool rotate = !is_v && unit.turns;
    float most = 0.f;  // (a NaN stays)
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if (!(live >> p & 1)) continue;
        float cs[VE], sn[VE];
        float2 x[VE];
        asm volatile("" ::: "memory");  // (one row's angles at a time: registers)
        if (rotate) unit.angles(a, place[p], cs, sn);
        unit.turn(raw[p], cs, sn, rotate, x);
#pragma unroll
        for (int e = 0; e < VE; ++e) most = dev::max_abs_nan(dev::max_abs_nan(most, x[e].x), x[e].y);
    }
    const uint32_t bits = __reduce_max_sync(FULL, __float_as_uint(most) & 0x7fffffffu);  // (infinities and NaN are above all)
    if (bits >= 0x7f800000u || old != old) return true;
    const float scale = next_scale(old, __uint_as_float(bits));
    const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
    if (s0 > 0 && scale != old) {
        // the rows before, at the new scale
        rescale_rows(block, s0, __fmul_rn(old, inv), lane);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) unit.keep(raw[p]);  // (else the compiler holds on to what it has rotated)
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if (!(live >> p & 1)) continue;
        float cs[VE], sn[VE];
        float2 x[VE];
        asm volatile("" ::: "memory");  // (one row's angles at a time: registers)
        if (rotate) unit.angles(a, place[p], cs, sn);
        unit.turn(raw[p], cs, sn, rotate, x);
        uint8_t *row = block + (s0 + p * SL + slot) * E4M3_D;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            uint32_t codes[VE / 4];
#pragma unroll
            for (int t = 0; t < VE / 4; ++t) {
                const float2 i2 = make_float2(inv, inv), y = dev::mul2(x[v * VE / 2 + 2 * t], i2), z = dev::mul2(x[v * VE / 2 + 2 * t + 1], i2);
                codes[t] = dev::e4m3x2(y.x, y.y) | dev::e4m3x2(z.x, z.y) << 16;
            }
            unit.store_codes(row, v, codes);
        }
    }
    if (lane == 0 && (s0 == 0 || scale != old)) *sp = scale;
    return false;
}

// ODD: the blocks that are not finite, else the others; are there any of those?
template <typename T, int VE, bool ODD>
__device__ __forceinline__ bool page_item(const RopeArgs &a, unsigned item, int lane) {
    // (range, KV head), K and V behind one another; where warps are many, each an item
    const unsigned per = a.both ? a.H_kv : 2 * a.H_kv, range = item / per, w = item - range * per;
    const int j = int(w) < a.H_kv ? int(w) : int(w) - a.H_kv;
    const int t0 = int(range) * a.range, t1 = min(a.total, t0 + a.range);
    // sequence after sequence, those of its blocks whose first new token is in [t0, t1)
    bool odd = false;
    dev::PackedSeq mine{};
    int b0 = a.cu_seqlens ? 0 : t0 / a.T;  // (without cu_seqlens: the first of the range on)
    for (; b0 < a.B && (a.cu_seqlens || t1 > b0 * a.T); b0 += 32) {
        mine = dev::PackedSeq{};
        if (b0 + lane < a.B && (a.cu_seqlens || t1 > (b0 + lane) * a.T)) mine = dev::packed_seq(a, a.T, b0 + lane);
        unsigned hit = __ballot_sync(FULL, mine.n > 0 && mine.lo < t1 && mine.lo + mine.n > t0);
        while (hit) {
            const int src = __ffs(hit) - 1;
            hit &= hit - 1;
            const int lo = __shfl_sync(FULL, mine.lo, src), n = __shfl_sync(FULL, mine.n, src), c = __shfl_sync(FULL, mine.c, src);
            int i = 0;
            if (lo < t0) {
                i = t0 - lo;
                i += (16 - (c + i) % 16) % 16;
            }
            while (i < n && lo + i < t1) {
                const int take = min(n - i, 16 - (c + i) % 16);
#pragma unroll 1
                for (int v = int(w) >= a.H_kv; v <= (a.both || int(w) >= a.H_kv); ++v) {
                    if constexpr (ODD)
                        odd_rows<T, VE>(a, b0 + src, lo, c, i, take, j, v, lane);
                    else if (page_rows<T, VE>(a, b0 + src, lo, c, i, take, j, v, lane))
                        odd = true;
                }
                i += take;
            }
        }
    }
    return odd;
}

// (apart from the others, which would be 3 % slower, single tokens 10 %)
template <typename T, int VE>
__device__ __noinline__ void odd_items(const RopeArgs &a, unsigned x, unsigned step, int lane) {
    for (; x < unsigned(a.page_items); x += step) page_item<T, VE, true>(a, x, lane);
}

template <typename T, int VE, Mode M>
__global__ void __launch_bounds__(256, 2) rope_kernel(const __grid_constant__ RopeArgs a) {
    dev::allow_dependents();
    dev::grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += 256)
            if (dev::packed_seq(a, a.T, b).bad) dev::record_error(a.err, ERR_DEVICE_INDEX);
    // (loops of their own: in one, each kind of item would have the other's registers spilled)
    const unsigned warp = threadIdx.x >> 5, half = gridDim.x / 2;
    if (M == BLOCKS && (blockIdx.x & 1) == 0) {
        const unsigned first = blockIdx.x / 2 * 8 + warp, step = (gridDim.x - half) * 8;
        bool odd = false;
        for (unsigned x = first; x < unsigned(a.page_items); x += step) odd |= page_item<T, VE, false>(a, x, lane);
        if (odd) odd_items<T, VE>(a, first, step, lane);
    } else {
        const unsigned block = M == BLOCKS ? blockIdx.x / 2 : blockIdx.x, blocks = M == BLOCKS ? half : gridDim.x;
        for (unsigned x = block * 8 + warp; x < unsigned(a.total) * a.parts; x += blocks * 8) row_item<T, VE, M>(a, x, lane);
    }
}

template <typename T, int VE, Mode M>
cudaError_t launch(const RopeArgs &a, int num_sms, cudaStream_t s) {
    const int64_t rows = (int64_t(a.total) * a.parts + 7) / 8, pages = (int64_t(a.page_items) + 7) / 8, cap = int64_t(num_sms) * 32;
    int64_t grid = rows < cap ? rows : cap;
    if (M == BLOCKS) {  // even blocks: pages, odd ones: rows
        const int64_t p = pages < cap ? pages : cap;
        grid = grid > p ? 2 * grid : 2 * p - (grid == 0);
    }
    return launch_pdl(rope_kernel<T, VE, M>, dim3(unsigned(grid)), dim3(256), 0, s, a);
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, int rows, int cache, int num_sms, cudaStream_t s) {
    const bool eight = cache == KVC_E4M3;
    a.n_heads = (a.q ? a.H : 0) + (eight ? (a.k_out ? a.H_kv : 0) : 2 * a.H_kv);
    // few tokens: a token's heads over several warps, sixteen vectors of a lane each
    const int64_t target = int64_t(num_sms) * 16;
    const int ve = rows == KVC_FP32 || a.half % 8 ? 4 : 8, chunk = 4 * 32 / (a.D / (2 * ve));  // heads that a warp has in flight
    a.parts = 0;
    a.per_part = 1;
    if (a.n_heads > 0) {
        const int most = (a.n_heads + chunk - 1) / chunk;
        const int64_t want = (target + a.total - 1) / a.total;
        a.parts = int(want < most ? want : most);
        a.per_part = (a.n_heads + a.parts - 1) / a.parts;
    }
    // pages: whole blocks of a prompt, or single tokens spread over the warps
    int64_t range = int64_t(a.total) * 2 * a.H_kv / target, pages = 0;
    a.range = int(range < 1 ? 1 : range > 16 ? 16 : range);
    a.both = a.range == 16;
    if (eight) pages = (int64_t(a.total) + a.range - 1) / a.range * (a.both ? 1 : 2) * a.H_kv;
    const int64_t warps = pages + int64_t(a.total) * a.parts;
    if (warps > 0x7fffffff) return cudaErrorInvalidValue;
    a.page_items = int(pages);
#define KVC_ROPE(T, VE, M) return launch<T, VE, M>(a, num_sms, s)
    if (cache == KVC_FP32) KVC_ROPE(float, 4, PLAIN);
    if (ve == 8) {
        if (cache == KVC_BF16) KVC_ROPE(__nv_bfloat16, 8, PLAIN);
        if (cache == KVC_FP16) KVC_ROPE(__half, 8, PLAIN);
        if (cache == KVC_INT8) KVC_ROPE(__nv_bfloat16, 8, INT8);
        if (rows == KVC_BF16) KVC_ROPE(__nv_bfloat16, 8, BLOCKS);
        KVC_ROPE(__half, 8, BLOCKS);
    }
    if (cache == KVC_BF16) KVC_ROPE(__nv_bfloat16, 4, PLAIN);
    if (cache == KVC_FP16) KVC_ROPE(__half, 4, PLAIN);
    if (cache == KVC_INT8) KVC_ROPE(__nv_bfloat16, 4, INT8);
    if (rows == KVC_BF16) KVC_ROPE(__nv_bfloat16, 4, BLOCKS);
    KVC_ROPE(__half, 4, BLOCKS);
#undef KVC_ROPE
}

}  // namespace kvc
