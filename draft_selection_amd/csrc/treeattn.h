// Attention of a tree of drafted tokens over a paged cache.
//
//   z_ij = scale k_scale <q_i, K_j>  for every key j that node i sees,
//   o_i  = v_scale sum_j p_ij V_j,   p_i = softmax(z_i),   lse_i = ln sum_j e^z_ij,
// in one pass over the keys with the running maximum m and sum l of the
// softmax.  Node i of row b sees the row's s cached positions and the nodes
// whose bit is set in its mask row (no mask: nodes 0..i).
//
// Rows.  The nodes of a batch row times the query heads of one K/V head are the
// rows of one product (r = node * group + head in group), in row tiles of 32 RW.
// A workgroup is RW x KW waves: RW waves of 32 rows each share the tiles of one
// of KW groups of keys, whose sums are joined through LDS at the end.  Few rows
// take many key groups (each wave then streams K and V of its own, with no
// barrier), many rows take many row waves (each tile is read once for all).
// Wide heads (256) split a row wave's output columns over CW = 2 waves, which
// both compute the scores: the sums then leave room for q in the registers.
//
// Products.  S^T = K Q^T by 32 x 32 x 16 MFMA, so a lane holds scores of one row
// (l % 32) and its softmax needs one exchange, with lane l ^ 32, for the maximum
// only.  Its 16 scores of 32 keys are those of keys 8 (i / 4) + 4 (l / 32) +
// i % 4; taken eight at a time they are already the operand of O^T = V^T P^T,
// if V^T's keys are taken in the same order.  V lies in LDS by keys; the
// transposing LDS reads deliver it by columns.
//
// Measured on an MI355X, caches in HBM, 32 query heads on 8 of 128, this kernel
// and the join together, captured, medians: 64 rows of up to 4,096 cached
// positions and chains of up to 17 nodes, 177 us (3.9 TB/s; the same keys moved
// with no arithmetic take 165); 8 rows of up to 16,384 and trees of up to 64, 141
// (510 TFLOP/s; keys alone 107, products alone 115, and at equal lengths 207, 148
// and 156: the waves stand at their LDS-DMA loads while the matrix core is free);
// 2 rows of 131,000 in 8 bits and trees of 32, 208 (660 TFLOP/s; keys alone 136,
// products alone 196: every row wave converts the tile's values for itself, on
// the vector unit that also does the softmax); one token over 333, 12.5 (a chain
// of loads: lengths, page ids, keys; then the join).
//
// Keys move from the cache into a ring of two or three LDS stages by 16-byte
// LDS-DMA loads (global_load_lds_dwordx4), one or two rounds ahead; page ids as
// many rounds before that.  16-byte chunk c of tile row `row` lies at chunk c ^ key(row); the keys
// spread what one LDS pass reads over all 64 banks.
#pragma once

#include "cache.h"
#include "project.h"

namespace dsel {

struct TreeAttnParams {
    CacheView c;
    TableView t;
    const char *q;  // bf16
    int64_t sqb, sqt, sqh;  // strides of batch, token, head in elements
    uint16_t *out;  // [B, T, Hq, D]
    float *lse;     // [B, T, Hq] or NULL
    const int32_t *mask;  // [B, T, words] or NULL
    const int32_t *len;
    int B, T, Hq, D, group, words;
    float scale;  // times log2(e)
    int wgs;      // workgroups that share the work
    bool whole;   // no tile is split (kAttnWholeKeys)
    int page_shift;  // log2 of the page size, -1 if it is no power of two
    float *part;     // partial sums
    int32_t *join;  // [wgs][kJoinWords]: the row tile that begins in a workgroup's share and ends in a later one's
};
constexpr int kJoinWords = 8;
// Rows whose table cannot hold more keys than this are not split: a unit is a
// whole tile, and there is no join.  One launch less for the host, and on the
// card, whole against split (32 query heads on 8 of 128): one token over 120
// keys 11.0 us against 12.3, over 250 12.7 against 12.5, over 500 16.4 against
// 12.6; 8 rows of 17 nodes over 120 keys 13.8 against 16.3, over 250 18.0 against
// 18.3.  (Other heads, other head sizes and 8-bit caches were not measured.)
constexpr int kAttnWholeKeys = 256;

__device__ u32x4 g_attn_zero[1];  // what a key that is none reads (never written)

// E4M3: 8-bit cache; DP: padded head dim; RW waves of 32 rows, each as CW waves
// that hold DP / CW columns of the output, by KW key groups; KT keys a tile; ST
// ring stages
template <bool E4M3_, int DP_, int RW_, int CW_, int KW_, int KT_, int ST_>
struct AttnCfg {
    static constexpr bool E4M3 = E4M3_;
    static constexpr int DP = DP_, RW = RW_, CW = CW_, KW = KW_, KT = KT_, ST = ST_;
    static constexpr int GW = RW * CW;                          // waves of a key group
    static constexpr int RB = DP * (E4M3 ? 1 : 2);              // bytes of a tile row
    static constexpr int NT = 64 * GW * KW, ROWS = 32 * RW, ROUND = KT * KW;
    static constexpr int TILE = KT * RB, GROUP = 2 * ST * TILE;  // K tiles, then V tiles of a key group
    static constexpr int SUMS = KW > 1 ? KW * GW * (DP / CW / 2 + 2) * 256 : 0;  // the groups' sums, in the ring's place
    static constexpr int RING = KW * GROUP > SUMS ? KW * GROUP : SUMS;
    static constexpr int LDS = RING + GW * KW * ST * 256;       // and page ids, per wave
    static constexpr int LOADS = TILE / 1024 / GW;              // LDS-DMA loads of a wave per K or V tile
    static constexpr int STEP = 2 * LOADS + 1;                  // and of a round: K, V, page ids
    static constexpr int PART = ROWS * (DP + 2);                // floats of one partial result
    static constexpr int NS = KT / 32, NB = DP / 32 / CW, CH = RB / 16, QUADS = NB * 4 / KW;
    // workgroups on a CU, as far as LDS (160 KB) and registers (512 a lane) allow
    static constexpr int WGS = LDS <= 80 * 1024 && NT <= 256 ? 2 : 1;
    static constexpr int WAVES = WGS * NT / 256 < 1 ? 1 : WGS * NT / 256;  // per SIMD
    static_assert(LOADS * 1024 * GW == TILE && KT <= 64 && KT % 32 == 0 && DP % 32 == 0, "tile geometry");
    static_assert((ST - 1) * STEP < 64, "outstanding loads are counted in 6 bits");

    __device__ static __forceinline__ int kkey(int row) {
        return RB >= 256 ? row & 15 : RB == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
    }
    // rows that one transposing read takes together: 4 (16 bits) or 4 + 4 eight apart (8 bits)
    __device__ static __forceinline__ int vkey(int row) {
        if constexpr (!E4M3) return RB >= 256 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
        else if constexpr (RB >= 256) return ((row & 3) | ((row >> 1) & 4)) << 1;
        else if constexpr (RB == 128) return (((row >> 1) & 1) | ((row >> 2) & 2)) << 1;
        else return ((row >> 3) & 1) << 1;
    }
};

// The work: units of one round (ROUND keys of one row tile), row by row of the
// batch, within it K/V head by head, row tile by row tile, round by round;
// each workgroup takes a share of consecutive units.  So every workgroup has
// the same number of rounds whatever the lengths, and a tile's rounds are split
// over as many workgroups as it takes; the partial sums of a split tile are
// joined by tree_attn_join_kernel.
struct AttnRow {
    int s, n;        // cached positions, nodes (0: nothing to do)
    int rts, rounds; // row tiles, rounds of each
    int units;       // units of a row tile: its rounds, or 1 (whole)
};
template <class C>
__device__ __forceinline__ AttnRow attn_row(const TreeAttnParams &p, int64_t b) {
    AttnRow r;
    r.n = block_len_of(p.len, b, p.T);
    r.s = r.n > 0 ? seq_len_of(p.t, b, r.n, p.c.page_size) : 0;
    if (r.s < 0) r.n = r.s = 0;
    r.rts = (r.n * p.group + C::ROWS - 1) / C::ROWS;
    r.rounds = (int)(((int64_t)r.s + r.n + C::ROUND - 1) / C::ROUND);
    r.units = p.whole && r.rounds ? 1 : r.rounds;
    return r;
}
__device__ __forceinline__ int64_t wave_incl_scan64(int64_t x) {
    const uint32_t lane = lane_id();
#pragma unroll
    for (uint32_t o = 1; o < 64; o <<= 1) {
        const int64_t y = (int64_t)shfl_idx64((uint64_t)x, lane >= o ? lane - o : lane);
        if (lane >= o) x += y;
    }
    return x;
}

// Shares of U units: W of them, the first U % W one unit longer.  U passes 32
// bits only in batches that no memory holds, but is counted in 64; 64-bit
// division costs a wave about a microsecond and is kept off the usual path.
constexpr int kAttnCUs = 256;
struct AttnShares {
    int64_t U, each, more;  // units, U / W, U % W
    int W;
    __device__ __forceinline__ int64_t begin(int64_t w) const { return w * each + (w < more ? w : more); }
    __device__ __forceinline__ static int64_t div(int64_t a, int64_t b) {
        return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
    }
    // the share that unit u lies in
    __device__ __forceinline__ int of(int64_t u) const {
        const int64_t longer = more * (each + 1);
        return (int)(u < longer ? div(u, each + 1) : more + div(u - longer, each));
    }
};
__device__ __forceinline__ AttnShares attn_shares(const TreeAttnParams &p, int64_t U) {
    AttnShares s;
    s.U = U;
    s.W = (int)(U < p.wgs ? U : p.wgs);
    s.each = AttnShares::div(U, s.W);
    s.more = U - s.each * s.W;
    return s;
}

// The rows of the batch, 64 at a time: lane k holds row b0 + k.  A whole wave
// calls all of this.
template <class C>
struct AttnBatch {
    int64_t incl;  // units of rows 0 .. this lane's, of the lane's range of ceil(B / 64) rows
    AttnRow mine;  // B <= 64: the lane's row
    __device__ __forceinline__ int64_t load(const TreeAttnParams &p) {
        const int64_t c = ((int64_t)p.B + 63) / 64, b0 = lane_id() * c;
        int64_t sum = 0;
        mine = AttnRow{0, 0, 0, 0, 0};
        for (int64_t k = 0; k < c; ++k)
            if (b0 + k < p.B) {
                mine = attn_row<C>(p, b0 + k);
                sum += (int64_t)mine.rts * p.c.heads * mine.units;
            }
        incl = wave_incl_scan64(sum);
        return (int64_t)readlane64((uint64_t)incl, 63);
    }
    __device__ __forceinline__ AttnRow row(const TreeAttnParams &p, int b) const {
        if (p.B > 64) return attn_row<C>(p, b);
        AttnRow r;
        r.s = __builtin_amdgcn_readlane(mine.s, b);
        r.n = __builtin_amdgcn_readlane(mine.n, b);
        r.rts = __builtin_amdgcn_readlane(mine.rts, b);
        r.rounds = __builtin_amdgcn_readlane(mine.rounds, b);
        r.units = __builtin_amdgcn_readlane(mine.units, b);
        return r;
    }
    // the row that unit u lies in, and the units before that row
    __device__ __forceinline__ int find(const TreeAttnParams &p, int64_t u, int64_t *before) const {
        const int64_t c = ((int64_t)p.B + 63) / 64;
        const int j = __builtin_ctzll(ballot(incl > u));  // u < the total, so some lane's sum passes it
        int64_t at = j ? (int64_t)readlane64((uint64_t)incl, j - 1) : 0, b = j * c;
        // that lane's own rows, 64 at a time
        for (int64_t k0 = 0; c > 1 && k0 < c; k0 += 64) {
            const int64_t k = k0 + lane_id();
            const AttnRow r = k < c && b + k < p.B ? attn_row<C>(p, b + k) : AttnRow{0, 0, 0, 0, 0};
            const int64_t x = (int64_t)r.rts * p.c.heads * r.units, sum = wave_incl_scan64(x);
            const uint64_t m = ballot(at + sum > u);
            if (m) {
                const int i = __builtin_ctzll(m);
                *before = at + (int64_t)readlane64((uint64_t)(sum - x), i);
                return (int)(b + k0 + i);
            }
            at += (int64_t)readlane64((uint64_t)sum, 63);
        }
        *before = at;
        return (int)b;
    }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ bf16x8 widen_e4m3(uint32_t a, uint32_t b) {
    const bf16x2 w0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, 1.0f, false);
    const bf16x2 w1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, 1.0f, true);
    const bf16x2 w2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, 1.0f, false);
    const bf16x2 w3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, 1.0f, true);
    return bf16x8{w0[0], w0[1], w1[0], w1[1], w2[0], w2[1], w3[0], w3[1]};
}

#define DSEL_LDS __attribute__((address_space(3)))

// 4 bytes per lane into LDS at lds_base + 4 * lane, as lds_dma16 does 16: page
// ids arrive like the keys, so that no wait of the compiler's for a load of its
// own waits for the keys in flight too
__device__ __forceinline__ void lds_dma4(const void *src, int32_t *lds_base) {
    const uint32_t m0v = (uint32_t)(uintptr_t)(DSEL_LDS void *)lds_base;
    asm volatile("global_load_lds_dword %1, off"
                 :
                 : "{m0}"(__builtin_amdgcn_readfirstlane(m0v)), "v"(src)
                 : "memory");
}

// 8 keys (16 kk + 8 (e / 4) + 4 (l / 32) + e % 4 of the 32 from tile row `sub`
// on) of V's column 32 mb + l % 32
template <class C>
__device__ __forceinline__ bf16x8 v_operand(const char *vt, int sub, int kk, int mb) {
    const int l = lane_id(), h = l >> 5;
    if constexpr (!C::E4M3) {
        const int row = sub + 16 * kk + 4 * h + ((l & 15) >> 2);
        const int chunk = 4 * mb + 2 * ((l >> 4) & 1) + ((l & 3) >> 1);
        const char *a = vt + row * C::RB + ((chunk ^ C::vkey(row)) << 4) + ((l & 1) << 3);
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DSEL_LDS s16x4 *)a);
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DSEL_LDS s16x4 *)(a + 8 * C::RB));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        const int k = (l & 15) >> 1, row = sub + 16 * kk + 8 * (k >> 2) + 4 * h + (k & 3);
        const int chunk = 2 * mb + ((l >> 4) & 1);
        const char *a = vt + row * C::RB + ((chunk ^ C::vkey(row)) << 4) + ((l & 1) << 3);
        const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((DSEL_LDS i32x2 *)a);
        return widen_e4m3((uint32_t)x[0], (uint32_t)x[1]);
    }
}

// Infinities and NaN among the values of a tile.  0 times those is no 0, so a
// row that does not see their key would catch them.  A tile in which some rows
// do not see every key is looked through for them; if it holds any they are
// taken out of the products and counted apart, among the keys that each row
// sees: +inf as 1, -inf as 32, NaN as 1024 (below 32 of each per product, so
// the sum tells them apart).  Counted so, an infinity that a row sees is one
// whatever its weight; in a tile that every row sees whole, which is not looked
// through, the product makes it NaN if its weight is 0.  Either way the element
// is not finite, which is all that is promised: looking through every tile would
// read V twice.
template <class C>
__device__ __forceinline__ bool tile_special(const char *vt) {
    bool r = false;
#pragma unroll 1
    for (int i = lane_id() * 16; i < C::TILE; i += 1024) {
        const u32x4 w = *(const u32x4 *)(vt + i);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if constexpr (C::E4M3) r |= (((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
            else r |= (w[k] & 0x7F800000u) == 0x7F800000u || (w[k] & 0x7F80u) == 0x7F80u;
    }
    return ballot(r) != 0;
}
__device__ __forceinline__ bf16x8 only_finite(const bf16x8 &v) {
    u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu;
        if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
    }
    return __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ bf16x8 special_codes(const bf16x8 &v) {
    u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t c = 0;
#pragma unroll
        for (int k = 0; k < 32; k += 16) {
            const uint32_t x = (w[i] >> k) & 0xFFFFu;
            if ((x & 0x7F80u) == 0x7F80u) c |= (x == 0x7F80u ? 0x3F80u : x == 0xFF80u ? 0x4200u : 0x4480u) << k;
        }
        w[i] = c;
    }
    return __builtin_bit_cast(bf16x8, w);
}
// Adds what the specials of a tile do to column block mb.
template <class C>
__device__ __forceinline__ void add_special(floatx16 &o, const char *vt, int mb, uint64_t see) {
    const int h = lane_id() >> 5;
#pragma unroll 1
    for (int step = 0; step < C::KT / 16; ++step) {
        const uint32_t bits = (uint32_t)(see >> (16 * step + 4 * h));
        u32x4 seen;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const int k = 8 * (e >> 2) + (e & 3);
            seen[e >> 1] = ((bits >> k) & 1 ? 0x3F80u : 0u) | ((bits >> (k + 1)) & 1 ? 0x3F800000u : 0u);
        }
        const bf16x8 code = special_codes(v_operand<C>(vt, 32 * (step >> 1), step & 1, mb));
        const floatx16 n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(code, __builtin_bit_cast(bf16x8, seen), floatx16{}, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int k = (int)n[i];
            const bool nan = k >= 1024 || ((k & 31) && k >= 32);
            if (k) o[i] += nan ? __builtin_nanf("") : k >= 32 ? -__builtin_inff() : __builtin_inff();
        }
    }
}

template <class C>
struct AttnState {
    floatx16 o[C::NB];
    float m, l;  // per lane: row l % 32; l: the sum over the lane's own keys
};
template <class C>
using AttnScores = floatx16[C::NS];

// Scores of a tile: S^T = K Q^T
template <class C>
__device__ __forceinline__ void attn_scores(AttnScores<C> &s, const bf16x8 (&q)[C::DP / 16], const char *kt) {
    const int l = lane_id(), h = l >> 5, r = l & 31, key = C::kkey(r);
#pragma unroll
    for (int sub = 0; sub < C::NS; ++sub) {
        const char *row = kt + (sub * 32 + r) * C::RB;
        s[sub] = floatx16{};
        if constexpr (!C::E4M3) {
#pragma unroll
            for (int ks = 0; ks < C::DP / 16; ++ks) {
                const bf16x8 x = *(const bf16x8 *)(row + (((2 * ks + h) ^ key) << 4));
                s[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, q[ks], s[sub], 0, 0, 0);
            }
        } else {
            // a 16-byte chunk is 16 values: two steps of the product
#pragma unroll
            for (int ks = 0; ks < C::DP / 32; ++ks) {
                const u32x4 x = *(const u32x4 *)(row + (((2 * ks + h) ^ key) << 4));
                s[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_e4m3(x[0], x[1]), q[2 * ks], s[sub], 0, 0, 0);
                s[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_e4m3(x[2], x[3]), q[2 * ks + 1], s[sub], 0, 0, 0);
            }
        }
    }
}

// Scores that a row does not see become -inf (bit j of `see`: key j of the tile).
template <class C>
__device__ __forceinline__ void attn_mask(AttnScores<C> &s, uint64_t see) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int sub = 0; sub < C::NS; ++sub) {
        const uint32_t w = (uint32_t)(see >> (32 * sub)) >> (4 * h);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (!((w >> (8 * (i >> 2) + (i & 3))) & 1)) s[sub][i] = -__builtin_inff();
    }
}

// The running maximum of a row only moves (and its sums are only scaled) when
// the row's own scores pass it by more than 8: weights stay below 2^8, as exact
// as any others.  The other rows of the wave are scaled by 1 then, so that when
// they move, and with it every rounding, depends on no row but their own.
template <class C>
__device__ __forceinline__ void attn_rescale(AttnState<C> &a, const AttnScores<C> &s, float c) {
    float top = -__builtin_inff();
#pragma unroll
    for (int sub = 0; sub < C::NS; ++sub)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[sub][i]);
    top = fmaxf(top, __uint_as_float(xor_lane32<32>(__float_as_uint(top)))) * c;
    const bool move = top > a.m + 8.0f;
    if (ballot(move)) {
        const float f = move ? __builtin_amdgcn_exp2f(a.m - top) : 1.0f;
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
            for (int i = 0; i < 16; ++i) a.o[nb][i] *= f;
        a.l *= f;
        if (move) a.m = top;
    }
}

// Weights of a tile, in place, and their sums.
template <class C>
__device__ __forceinline__ void attn_weights(AttnState<C> &a, AttnScores<C> &s, float c) {
    const float ms = a.m == -__builtin_inff() ? 0.0f : a.m;
    float sum = 0.0f;
#pragma unroll
    for (int sub = 0; sub < C::NS; ++sub)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[sub][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[sub][i], c, -ms));
            sum += s[sub][i];
        }
    a.l += sum;
}

// O^T += V^T P^T for column blocks nb0 .. of the wave, the weights rounded to
// bf16, the matrix core's type here: half a step of 2^-8 of each weight, where the
// output is rounded by as much once more (the sum of the weights, and lse with it,
// stays that of the unrounded ones).  Two operands are read together.  The branch on `special` between the
// reads and the products also keeps the compiler from reading every operand of
// the tile ahead, which costs 60 registers and spills: without it (the special
// case as a call of its own) the kernel took 15 to 25% longer.
template <class C>
__device__ __forceinline__ void attn_values(AttnState<C> &a, const AttnScores<C> &s, const char *vt, int nb0, bool special) {
#pragma unroll
    for (int sub = 0; sub < C::NS; ++sub)
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            bf16x8 w;
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = (__bf16)s[sub][8 * kk + e];
            constexpr int G = C::NB < 2 ? C::NB : 2;
#pragma unroll
            for (int n0 = 0; n0 < C::NB; n0 += G) {
                bf16x8 v[G];
#pragma unroll
                for (int nb = 0; nb < G; ++nb) v[nb] = v_operand<C>(vt, 32 * sub, kk, nb0 + n0 + nb);
                if (special) {
#pragma unroll
                    for (int nb = 0; nb < G; ++nb) v[nb] = only_finite(v[nb]);
                }
#pragma unroll
                for (int nb = 0; nb < G; ++nb) a.o[n0 + nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[nb], w, a.o[n0 + nb], 0, 0, 0);
            }
        }
}

// Which of the 32 keys from position `kb` on node t of row b sees, by its mask
__device__ __forceinline__ uint32_t sees_of(const TreeAttnParams &p, int64_t b, int t, int s, int kb) {
    const int first = kb - s;  // the node at the first of them
    if (first <= -32) return ~0u;
    if (p.mask == nullptr) {
        const int count = t + 1 - first;
        return count >= 32 ? ~0u : count <= 0 ? 0u : (1u << count) - 1;
    }
    const int32_t *w = p.mask + ((int64_t)b * p.T + t) * p.words;
    if (first < 0) return ((uint32_t)w[0] << -first) | ((1u << -first) - 1);
    const int i = first >> 5, sh = first & 31;
    uint32_t x = i < p.words ? (uint32_t)w[i] >> sh : 0u;
    if (sh && i + 1 < p.words) x |= (uint32_t)w[i + 1] << (32 - sh);
    return x;
}

template <class C>
__global__ __launch_bounds__(C::NT, C::WAVES) void tree_attn_kernel(TreeAttnParams p) {
    __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int gw = wave % C::GW, grp = wave / C::GW, rw = gw / C::CW, nb0 = gw % C::CW * C::NB, h = lane >> 5;
    int32_t *const join = p.join + blockIdx.x * kJoinWords;
    if (threadIdx.x == 0 && !p.whole) join[0] = -1;
    AttnBatch<C> batch;
    const int64_t U = batch.load(p);
    if (U == 0) return;
    // neighbouring shares on one XCD (workgroup i runs on XCD i % 8): row tiles
    // that read the same keys then find them in its L2
    const AttnShares shares = attn_shares(p, U);
    const int per = (shares.W + 7) >> 3;
    if ((int)(blockIdx.x >> 3) >= per) return;
    const int share = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (share >= shares.W) return;
    int64_t u = shares.begin(share);
    const int64_t uend = shares.begin(share + 1);
    int64_t before;
    int b = batch.find(p, u, &before);
    AttnRow row = batch.row(p, b);

    char *const kring = lds + grp * C::GROUP, *const vring = kring + C::ST * C::TILE;
    int32_t *const ids = (int32_t *)(lds + C::RING) + wave * C::ST * 64;
    while (u < uend) {
        while (u - before >= (int64_t)row.rts * p.c.heads * row.units) {  // on to the next row with work
            before += (int64_t)row.rts * p.c.heads * row.units;
            row = batch.row(p, ++b);
        }
        const int item = (int)AttnShares::div(u - before, row.units);
        const int r0 = (int)((u - before) - (int64_t)item * row.units);
        const int r1 = p.whole || (int64_t)row.rounds - r0 < uend - u ? row.rounds : (int)(r0 + (uend - u));
        const int hk = item / row.rts, rt = item - hk * row.rts;
        const int total = row.s + row.n;
        const char *const kbase = p.c.k + 16 * (hk * p.c.head_stride);
        const char *const vbase = p.c.v + 16 * (hk * p.c.head_stride);
        const int32_t *const table = p.t.table + b * p.t.ld;
        float c = p.scale;
        // c is a positive number, so that a masked score of -inf stays one times c:
        // what a scale's sign or NaN does to the scores is done to q
        uint32_t sign = 0, nan = 0;
        if (C::E4M3 && p.c.k_scale) {
            const float ks = p.c.k_scale[hk];
            sign = ks < 0.0f ? 0x80008000u : 0u;
            c = p.scale * fabsf(ks);
            if (c == 0.0f) c = 1e-37f;
            if (c != c) {
                nan = 0x7FC07FC0u;
                c = 1.0f;
            }
        }

        // the lane's rows, and their q: eight values of every 16-deep step
        const int rows = row.n * p.group, r = rt * C::ROWS + rw * 32 + (lane & 31);
        const bool live = r < rows;
        const bool idle = rt * C::ROWS + rw * 32 >= rows;  // the whole wave: it only moves keys
        const int t = live ? r / p.group : 0, head = hk * p.group + (live ? r - t * p.group : 0);
        const uint16_t *const qr = (const uint16_t *)p.q + b * p.sqb + t * p.sqt + head * p.sqh;
        bf16x8 q[C::DP / 16];
#pragma unroll
        for (int ks = 0; ks < C::DP / 16; ++ks) {
            const int d = C::E4M3 ? 32 * (ks >> 1) + 16 * h + 8 * (ks & 1) : 16 * ks + 8 * h;
            u32x4 w = live && d < p.D ? *(const u32x4 *)(qr + d) : u32x4{0, 0, 0, 0};
            if constexpr (C::E4M3) w = (w ^ sign) | nan;
            q[ks] = __builtin_bit_cast(bf16x8, w);
        }

        // The keys of a round: lane j of every wave places key j of its group's
        // tile, as a byte offset.  A key past the end, or of a page that is none,
        // has no place; it reads what the first key that has one reads, and its
        // score is masked.
        auto key_pos = [&](int round) { return (uint32_t)(round * C::ROUND + grp * C::KT + (lane & (C::KT - 1))); };
        auto page_at = [&](uint32_t k) { return p.page_shift >= 0 ? k >> p.page_shift : k / (uint32_t)p.c.page_size; };
        auto entry_of = [&](int round) -> const int32_t * {
            const uint32_t k = key_pos(round);
            return table + (k < (uint32_t)total ? page_at(k) : 0u);
        };
        auto place = [&](int round, int page, uint64_t *ok) -> int64_t {
            const uint32_t k = key_pos(round);
            const bool in = k < (uint32_t)total, good = in && page >= 0 && page < p.c.num_pages;
            if (in && !good) device_error(kErrPage);
            const uint32_t slot = k - page_at(k) * (uint32_t)p.c.page_size;
            const int64_t off = 16 * ((int64_t)page * p.c.page_stride + (int64_t)slot * p.c.slot_stride);
            const uint64_t m = ballot(good);
            *ok = m;
            if (m == ~0ull) return off;
            const int64_t first = m ? (int64_t)readlane64((uint64_t)off, __builtin_ctzll(m)) : 0;
            return good ? off : first;
        };
        const bool padded = p.c.vecs < C::CH;  // chunks past the head dim read zeros
        auto stage = [&](char *kt, char *vt, int64_t off) {
#pragma unroll
            for (int j = 0; j < C::LOADS; ++j) {
                const int pos = (gw * C::LOADS + j) * 1024, byte = pos + lane * 16;
                const int rr = byte / C::RB, ch = (byte % C::RB) / 16;
                const int64_t o = (int64_t)shfl_idx64((uint64_t)off, rr);
                const int kc = ch ^ C::kkey(rr), vc = ch ^ C::vkey(rr);
                const char *ks = kbase + 16 * kc + o, *vs = vbase + 16 * vc + o;
                if (padded) {
                    if (kc >= p.c.vecs) ks = (const char *)g_attn_zero;
                    if (vc >= p.c.vecs) vs = (const char *)g_attn_zero;
                }
                lds_dma16(ks, (uint16_t *)(kt + pos));
                lds_dma16(vs, (uint16_t *)(vt + pos));
            }
        };
        // Round i computes on its own keys and starts those of round i + A, whose
        // places it reads from page ids fetched A rounds before that.
        constexpr int A = C::ST - 1;
        auto slot = [&](int round) { return (uint32_t)(round - r0) % C::ST; };
        auto start = [&](int round, int64_t off) {
            stage(kring + slot(round) * C::TILE, vring + slot(round) * C::TILE, off);
            lds_dma4(entry_of(round + A), ids + slot(round + A) * 64);
        };
        uint64_t have[C::ST];  // at the top of round i: which keys of rounds i .. i + A - 1 have a place
        {
            int page[A];
#pragma unroll
            for (int k = 0; k < A; ++k) page[k] = *entry_of(r0 + k);
#pragma unroll
            for (int ks = 0; ks < C::DP / 16; ++ks) asm volatile("" : "+v"(q[ks]));  // q is here before the ring starts
#pragma unroll
            for (int k = 0; k < A; ++k) {
                const int64_t off = place(r0 + k, page[k], &have[k]);
                if (r0 + k < r1) start(r0 + k, off);
            }
            have[A] = 0;
        }
        AttnState<C> a;
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb) a.o[nb] = floatx16{};
        a.m = -__builtin_inff();
        a.l = 0.0f;

        constexpr uint64_t kAll = ~0ull >> (64 - C::KT);
        for (int round = r0; round < r1; ++round) {
            // this round's keys have landed, and nobody still reads the slots filled next
            if (round + A <= r1) wait_vmcnt_lgkm0<(A - 1) * C::STEP>();
            else wait_vmcnt_lgkm0<0>();
            if constexpr (C::GW > 1) wg_barrier();
            else asm volatile("" ::: "memory");
            if (round + A < r1) {
                start(round + A, place(round + A, ids[slot(round + A) * 64 + lane], &have[A]));
            }
            const uint64_t now = have[0];
#pragma unroll
            for (int k = 0; k < A; ++k) have[k] = have[k + 1];
            const int kb = round * C::ROUND + grp * C::KT;
            const bool whole = kb + C::KT <= row.s && (now & kAll) == kAll;
            if (idle || (now & kAll) == 0) continue;
            uint64_t see = now;
            if (!whole)
                see &= sees_of(p, b, t, row.s, kb) | (C::KT == 64 ? (uint64_t)sees_of(p, b, t, row.s, kb + 32) << 32 : 0);
            const char *const vt = vring + slot(round) * C::TILE;
            AttnScores<C> s;
            attn_scores<C>(s, q, kring + slot(round) * C::TILE);
            if (!whole) attn_mask<C>(s, see);
            attn_rescale<C>(a, s, c);
            attn_weights<C>(a, s, c);
            const bool special = !whole && tile_special<C>(vt);
            attn_values<C>(a, s, vt, nb0, special);
            if (special) {
#pragma unroll
                for (int nb = 0; nb < C::NB; ++nb) add_special<C>(a.o[nb], vt, nb0 + nb, see);
            }
        }

        a.l += __uint_as_float(xor_lane32<32>(__float_as_uint(a.l)));
        floatx4 mine[C::QUADS];  // the columns that this wave writes
        if constexpr (C::KW > 1) {
            // the key groups' sums, exchanged through LDS: every group joins (and
            // writes) its part of the columns
            floatx4 *const sums = (floatx4 *)lds + gw * 64 + lane;
            float2 *const stats = (float2 *)(lds + C::KW * C::GW * C::NB * 4096) + gw * 64 + lane;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < C::NB * 4; ++k)
                sums[(grp * C::NB * 4 + k) * C::GW * 64] = floatx4{a.o[k >> 2][4 * (k & 3)], a.o[k >> 2][4 * (k & 3) + 1],
                                                                 a.o[k >> 2][4 * (k & 3) + 2], a.o[k >> 2][4 * (k & 3) + 3]};
            stats[grp * C::GW * 64] = float2{a.m, a.l};
            __syncthreads();
            float m = -__builtin_inff(), f[C::KW];
            float2 st[C::KW];
#pragma unroll
            for (int g = 0; g < C::KW; ++g) {
                st[g] = stats[g * C::GW * 64];
                m = fmaxf(m, st[g].x);
            }
            const float ms = m == -__builtin_inff() ? 0.0f : m;
            a.l = 0.0f;
            a.m = m;
#pragma unroll
            for (int g = 0; g < C::KW; ++g) {
                f[g] = __builtin_amdgcn_exp2f(st[g].x - ms);
                a.l += st[g].y * f[g];
            }
#pragma unroll
            for (int k = 0; k < C::QUADS; ++k) {
                mine[k] = floatx4{0, 0, 0, 0};
#pragma unroll
                for (int g = 0; g < C::KW; ++g)
                    mine[k] += sums[(g * C::NB * 4 + grp * C::QUADS + k) * C::GW * 64] * f[g];
            }
        } else {
#pragma unroll
            for (int k = 0; k < C::QUADS; ++k)
                mine[k] = floatx4{a.o[k >> 2][4 * (k & 3)], a.o[k >> 2][4 * (k & 3) + 1], a.o[k >> 2][4 * (k & 3) + 2],
                                  a.o[k >> 2][4 * (k & 3) + 3]};
        }
        if (threadIdx.x == 0 && r0 == 0 && r1 < row.rounds) {
            // the tile goes on in the shares up to that of its last round
            join[0] = b;
            join[1] = hk;
            join[2] = rt;
            join[3] = share;
            join[4] = shares.of(u + row.rounds - 1);
            join[5] = row.n;
        }
        if (live) {
            // quad k: columns 8 k + 4 h + 0..3 of the wave's part
            const int d0 = 32 * nb0 + 8 * (grp * C::QUADS) + 4 * h;
            const bool first = h == 0 && nb0 == 0 && grp == 0;
            if (r0 == 0 && r1 == row.rounds) {
                const float vs = C::E4M3 && p.c.v_scale ? p.c.v_scale[hk] : 1.0f;
                const bool some = !(a.l <= 0.0f);  // NaN counts as something
                const float f = some ? vs / a.l : 0.0f;
                const int64_t at = ((int64_t)b * p.T + t) * p.Hq + head;
#pragma unroll
                for (int k = 0; k < C::QUADS; ++k) {
                    if (d0 + 8 * k >= p.D) continue;
                    bf16x2 y[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e >> 1][e & 1] = (__bf16)(some ? mine[k][e] * f : 0.0f);
                    *(uint2 *)(p.out + at * p.D + d0 + 8 * k) = __builtin_bit_cast(uint2, y);
                }
                if (p.lse && first)
                    p.lse[at] = some ? (a.m + __builtin_amdgcn_logf(a.l)) * 0.69314718055994531f : -__builtin_inff();
            } else {
                float *to = p.part + (int64_t)(share * 2 + (r0 == 0)) * C::PART;
                const int rr = rw * 32 + (lane & 31);
                if (first) {
                    to[rr] = a.m;
                    to[C::ROWS + rr] = a.l;
                }
#pragma unroll
                for (int k = 0; k < C::QUADS; ++k) *(floatx4 *)(to + 2 * C::ROWS + rr * C::DP + d0 + 8 * k) = mine[k];
            }
        }
        u += p.whole ? 1 : r1 - r0;
        if (u < uend) {
            // the ring (and the sums in it) are read no more
            wait_vmcnt_lgkm0<0>();
            __syncthreads();
        }
    }
}

// Joins the partial sums of the row tiles that several workgroups shared:
// workgroup (i, y) takes 1024 / DP rows of the tile that workgroup i of the
// attention began and did not end; a thread takes four columns of a row and has
// the parts of eight shares in flight at a time.  (Four rows a thread, a quarter
// of the workgroups: 25 us instead of 14 at 2 x 131,000 keys.)
template <class C>
struct AttnJoin {
    static constexpr int TR = C::DP / 4, NR = 256 / TR, Y = C::ROWS / NR;
};
template <class C>
__global__ __launch_bounds__(256) void tree_attn_join_kernel(TreeAttnParams p) {
    using J = AttnJoin<C>;
    constexpr int N = 8;
    const int32_t *const join = p.join + blockIdx.x * kJoinWords;
    const int b = join[0];
    if (b < 0) return;
    const int hk = join[1], rt = join[2], w0 = join[3], w1 = join[4], n = join[5];
    const int rr = blockIdx.y * J::NR + threadIdx.x / J::TR, d = (threadIdx.x % J::TR) * 4;
    const int r = rt * C::ROWS + rr;
    if (r >= n * p.group) return;
    float m = -__builtin_inff(), l = 0.0f;
    floatx4 o = {0, 0, 0, 0};
    for (int w = w0; w <= w1; w += N) {
        float pm[N], pl[N];
        floatx4 po[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            // the first share begins the tile (part 1), in the others it is what they begin with (part 0)
            const int v = w + k <= w1 ? w + k : w1;
            const float *x = p.part + (int64_t)(v * 2 + (v == w0)) * C::PART;
            pm[k] = w + k <= w1 ? x[rr] : -__builtin_inff();
            pl[k] = x[C::ROWS + rr];
            po[k] = *(const floatx4 *)(x + 2 * C::ROWS + rr * C::DP + d);
        }
        float mn = m;
#pragma unroll
        for (int k = 0; k < N; ++k) mn = fmaxf(mn, pm[k]);
        const float ms = mn == -__builtin_inff() ? 0.0f : mn;
        const float f0 = __builtin_amdgcn_exp2f(m - ms);
        l *= f0;
        o *= f0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (w + k > w1) continue;
            const float f = __builtin_amdgcn_exp2f(pm[k] - ms);
            l += pl[k] * f;
            o += po[k] * f;
        }
        m = mn;
    }
    const int t = r / p.group, g = r - t * p.group;
    const int64_t at = ((int64_t)b * p.T + t) * p.Hq + hk * p.group + g;
    const bool some = !(l <= 0.0f);
    const float f = some ? (C::E4M3 && p.c.v_scale ? p.c.v_scale[hk] : 1.0f) / l : 0.0f;
    if (d < p.D) {
        bf16x2 y[2];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e >> 1][e & 1] = (__bf16)(some ? o[e] * f : 0.0f);
        *(uint2 *)(p.out + at * p.D + d) = __builtin_bit_cast(uint2, y);
    }
    if (p.lse && d == 0) p.lse[at] = some ? (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f : -__builtin_inff();
}

}  // namespace dsel
