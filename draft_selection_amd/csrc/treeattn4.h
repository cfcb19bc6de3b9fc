// Attention of a tree of drafted tokens over a paged cache held in 4 bits.
//
// The same sums as treeattn.h, over the same rows, rounds and shares of work.  A
// value of the cache, 2^(s-127) times an e2m1 value, is exact in bf16, so once
// widened the products are those of a bf16 cache with the same values.
//
// A 16-byte vector is 32 values and has one scale byte.  V has to be read by
// columns, and a column's values of different keys have different scales, so its
// tile is widened to bf16 on its way into LDS (one instruction for two values, scale
// and all), from where the transposing reads deliver it as in treeattn.h.
//
// Reading half of a byte a value, this is bound by arithmetic, or for few rows by
// instructions, sooner than by memory, and there are two kernels:
//   tree_attn4_kernel, rows in tiles of 32 a wave: the row waves of a key group widen
//     a part of K's and V's tile each, for all of them;
//   tree_attn4_few_kernel, at most 32 rows (16 of head sizes past 128, where two tiles
//     of sums do not fit the registers): a wave has keys of its own, K goes straight to
//     registers, and products of 16 rows waste less of the matrix core and, what
//     counts more, half as many of the exponentials.
#pragma once

#include "treeattn.h"

namespace dsel {

// Scale byte s as 2^(s - 127); the conversions take its exponent alone, and 255 as NaN
__device__ __forceinline__ float block_scale(uint32_t s) { return __uint_as_float(s << 23); }

// Is a block of V to be kept out of the products?  255 is NaN, and under 253 and 254,
// which no call writes, the larger codes pass bf16: 0 times those is no 0 either, and a
// key that is none reads a slot that may hold anything.
__device__ __forceinline__ bool not_finite(uint32_t s) { return s > 252; }

// the 8 values of a word
__device__ __forceinline__ bf16x8 widen_fp4(uint32_t w, float s) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A piece of work: rounds [r0, r1) of row tile rt of K/V head hk of batch row b
struct AttnUnit {
    int b, hk, rt, r0, r1, share;
    int64_t u;
    AttnRow row;
};
// The pieces of this workgroup's share, one after the other (as tree_attn_kernel).
template <class C, class F>
__device__ __forceinline__ void attn_units(const TreeAttnParams &p, F work) {
    int32_t *const join = p.join + blockIdx.x * kJoinWords;
    if (threadIdx.x == 0 && !p.whole) join[0] = -1;
    AttnBatch<C> batch;
    const int64_t U = batch.load(p);
    if (U == 0) return;
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
    while (u < uend) {
        while (u - before >= (int64_t)row.rts * p.c.heads * row.units) {  // on to the next row with work
            before += (int64_t)row.rts * p.c.heads * row.units;
            row = batch.row(p, ++b);
        }
        const int item = (int)AttnShares::div(u - before, row.units);
        const int r0 = (int)((u - before) - (int64_t)item * row.units);
        const int r1 = p.whole || (int64_t)row.rounds - r0 < uend - u ? row.rounds : (int)(r0 + (uend - u));
        const int hk = item / row.rts;
        work(AttnUnit{b, hk, item - hk * row.rts, r0, r1, share, u, row}, shares, join);
        u += p.whole ? 1 : r1 - r0;
        if (u < uend) __syncthreads();  // the tiles (and the sums in them) are read no more
    }
}

// Where a key's vectors lie, and whether they do: the offset in vectors of position
// `pos` of the row, which is that of its scale bytes too.  A key past the end, or of
// a page that is none, has no place and reads the first slot of page 0; its score is
// masked.
struct Attn4Keys {
    const int32_t *table;
    int64_t head;  // offset of the K/V head
    uint32_t total;
    __device__ __forceinline__ uint32_t page_at(const TreeAttnParams &p, uint32_t k) const {
        return p.page_shift >= 0 ? k >> p.page_shift : k / (uint32_t)p.c.page_size;
    }
    // (The position is chosen and not the lookup, so that no lanes branch around it: the
    // compiler has put spills of all lanes at the join ahead of the mask's restore, and
    // lanes past a row's end lost their scale bytes.)
    __device__ __forceinline__ int page(const TreeAttnParams &p, uint32_t pos) const {
        return table[page_at(p, pos < total ? pos : 0u)];
    }
    __device__ __forceinline__ int64_t place(const TreeAttnParams &p, uint32_t pos, int page, bool *bad) const {
        const bool in = pos < total, good = in && (uint32_t)page < (uint32_t)p.c.num_pages;
        *bad = in && !good;
        const uint32_t slot = pos - page_at(p, pos) * (uint32_t)p.c.page_size;
        const int64_t off = (int64_t)page * p.c.page_stride + (int64_t)slot * p.c.slot_stride;
        return head + (good ? off : 0);
    }
};

// ---- rows in tiles of 32 a wave ---------------------------------------------------
//
// Measured on an MI355X, captured, caches in HBM (three sets in turn), heads-first
// pages, 32 query heads on 8 of 128, this kernel and the join together, medians: 64
// chains of up to 17 nodes over up to 4,096 positions 121 us (283 TFLOP/s of products
// that count: 68 of the 128 rows of a tile do); under a window of 1,024 67; 8 trees of
// up to 64 over up to 16,384, 127 us; 32 chains of up to 9 over up to 2,048 44; 2 trees
// of 32 over 131,000, 183 us (749, at 1.7 GHz: what the card's power allows).  16 heads
// on 2 of 256, 16 trees of up to 21 over up to 5,000: 81 us (69 in a loop without the
// step below, whose registers spill at that size: 176 to 196 bytes of a lane's; 24 to
// 36 at 128, none at 64).  A round of 64 keys takes 3,900 cycles for the two waves of a
// SIMD, of which the products are 2,048; the start, the parts of split tiles and the
// join take some 35 us of every call.
// On the way there: K straight to every row wave's registers (each widens the whole
// tile) 131 and 207 us; products, softmax and widening after each other 131 and 209;
// steps in one, but page ids fetched behind the vectors of a round (loads land in their
// order, so each waited for all of them) 144 and 214.

// DP: padded head dim; RW waves of 32 rows, each as CW waves that hold DP / CW
// columns of the output, by KW key groups; KT keys a round
template <bool WIN_, int DP_, int RW_, int CW_, int KW_, int KT_>
struct Attn4Cfg {
    static constexpr bool E4M3 = false, WIN = WIN_;  // (the tiles in LDS are of bf16)
    static constexpr int DP = DP_, RW = RW_, CW = CW_, KW = KW_, KT = KT_;
    static constexpr int GW = RW * CW;
    static constexpr int NT = 64 * GW * KW, ROWS = 32 * RW, ROUND = KT * KW;
    static constexpr int NS = KT / 32, NB = DP / 32 / CW, QUADS = NB * 4 / KW;
    // Rows of the tiles are padded: eight rows that a read of K takes 16 bytes of, four
    // that a transposing read of V takes 64 of, and (V's vectors turned, below) those
    // that sixteen lanes widen a vector into, lie in banks apart, and an operand's
    // place is a constant past the lane's.
    static constexpr int KB = DP * 2 + 16, VB = DP * 2 + 64;
    static constexpr int KTILE = KT * KB, VTILE = KT * VB;
    static constexpr int GROUP = 2 * (KTILE + VTILE);  // two stages of each
    static constexpr int SUMS = KW > 1 ? KW * GW * (DP / CW / 2 + 2) * 256 : 0;
    static constexpr int RING = KW * GROUP > SUMS ? KW * GROUP : SUMS;
    static constexpr int CH = DP / 32;       // vectors of a row
    static constexpr int VW = KT * CH / 64;  // a bit for each vector of a tile, in words
    static constexpr int LDS = RING + KW * 4 * VW * 8;
    static constexpr int PART = ROWS * (DP + 2);
    static constexpr int VC = (KT * CH + 64 * GW - 1) / (64 * GW);  // vectors of a tile that a lane widens
    static constexpr int QS = DP / 16, PS = 2 * NB;  // products of 32 keys: of q and K, of P and V
    static constexpr int STEPS = QS > PS ? QS : PS;
    static constexpr int WGS = LDS <= 80 * 1024 && NT <= 256 ? 2 : 1;
    static constexpr int WAVES = WGS * NT / 256 < 1 ? 1 : WGS * NT / 256;
    static_assert(DP % 64 == 0 && 16 % STEPS == 0 && (KT * CH) % 64 == 0 && (KT == 32 || KT == 64), "tile geometry");
    __device__ static __forceinline__ int turn(int row) { return DP >= 128 ? row & 3 : (row & 1) | (row >> 1 & 2); }
};

// One step of the pipeline, over three neighbouring sets of 32 keys: the scores of
// the next one are computed (into s2), the scores s of this one become weights (p,
// bf16 as in attn_values), and the products of the weights before with V are added.
// None of the three waits for another, so products and vector instructions go
// out in turn and the matrix core and the vector unit work at the same time; side(i)
// is other work of the wave's, in as many slices.  Operands are read two products
// ahead.  (The barriers hold the compiler to this order.)  Returns what o is still to
// be scaled by, as attn_rescale does it.
//   kop(j): K's operand of the j-th step of q's product; vop(j): V's of the j-th product
template <class C, class F, class G, class H>
__device__ __forceinline__ float attn4_step(AttnState<C> &a, const floatx16 &s, floatx16 &s2, bf16x8 (&p)[2],
                                            const bf16x8 (&q)[C::QS], float c, F kop, G vop, H side) {
    constexpr int QE = C::STEPS / C::QS, PE = C::STEPS / C::PS;
    // weights done after slice i: none of the first, which finds the maximum
    auto done = [](int i) { return i <= 0 ? 0 : i == C::STEPS - 1 ? 16 : (16 * i / (C::STEPS - 1) + 1) & ~1; };
    bf16x8 k[2], v[2], w[2];
    float sum = 0.0f, f = 1.0f, ms = 0.0f;
    k[0] = kop(0);
    v[0] = vop(0);
    k[1] = kop(1);
    v[1] = vop(1);
    s2 = floatx16{};
#pragma unroll
    for (int i = 0; i < C::STEPS; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        if (i % QE == 0) {
            const int j = i / QE;
            s2 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[j & 1], q[j], s2, 0, 0, 0);
            if (j + 2 < C::QS) k[j & 1] = kop(j + 2);
        }
        if (i % PE == 0) {
            const int j = i / PE;
            a.o[j % C::NB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[j & 1], p[j / C::NB], a.o[j % C::NB], 0, 0, 0);
            if (j + 2 < C::PS) v[j & 1] = vop(j + 2);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (i == 0) {
            float top = -__builtin_inff();
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[e]);
            top = fmaxf(top, __uint_as_float(xor_lane32<32>(__float_as_uint(top)))) * c;
            const bool move = top > a.m + 8.0f;
            f = move ? __builtin_amdgcn_exp2f(a.m - top) : 1.0f;
            if (move) a.m = top;
            ms = a.m == -__builtin_inff() ? 0.0f : a.m;
            a.l *= f;
        }
        side(i);
#pragma unroll
        for (int e = done(i - 1); e < done(i); ++e) {
            float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -ms));
            asm volatile("" : "+v"(x));  // here, not where it is first used
            sum += x;
            w[e >> 3][e & 7] = (__bf16)x;
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    a.l += sum;
    p[0] = w[0];
    p[1] = w[1];
    asm volatile("" : "+v"(p[0]), "+v"(p[1]));
    return f;
}

// A bit for each vector of 32 keys (vector i: key i / CH, columns 32 (i % CH) ..), as
// the waves that widen them leave it in LDS: those of K whose page is none, those of
// V that are not finite.  Both are rare, and are looked for after a step's products, when
// the words have long arrived.
template <class C>
struct Attn4Bits {
    static constexpr int N = C::VW / C::NS;
    uint64_t w[N];
    __device__ __forceinline__ void load(const uint64_t *from, int sub) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = from[sub * N + i];
    }
    __device__ __forceinline__ bool any() {
        uint64_t x = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            asm volatile("" : "+v"(w[i]));  // not waited for before
            x |= w[i];
        }
        return __builtin_amdgcn_readfirstlane((int)((uint32_t)(x >> 32) | (uint32_t)x)) != 0;
    }
    // bit k: key k's vector of column block ch
    __device__ __forceinline__ uint32_t keys(int ch) const {
        uint32_t r = 0;
#pragma unroll 1
        for (int k = 0; k < 32; ++k) {
            const int i = k * C::CH + ch;
            uint64_t x = w[0];
#pragma unroll
            for (int n = 1; n < N; ++n) x = (i >> 6) == n ? w[n] : x;
            r |= ((uint32_t)(x >> (i & 63)) & 1) << k;
        }
        return r;
    }
};
// Blocks of V that are not finite enter the products under a scale of 2^-127; a row that
// sees the key of one (bits of see) gets NaN in its columns.
template <class C>
__device__ __forceinline__ void attn4_nan(AttnState<C> &a, const Attn4Bits<C> &nan, int nb0, uint32_t see) {
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb) {
        const float add = nan.keys(nb0 + nb) & see ? __builtin_nanf("") : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a.o[nb][i] += add;
    }
}

template <class C>
__global__ __launch_bounds__(C::NT, C::WAVES) void tree_attn4_kernel(TreeAttnParams p) {
    __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int gw = wave % C::GW, grp = wave / C::GW, rw = gw / C::CW, nb0 = gw % C::CW * C::NB, h = lane >> 5;
    // K's stages, V's stages; bits of V's, of K's
    char *const kring = lds + grp * C::GROUP, *const vring = kring + 2 * C::KTILE;
    uint64_t *const bits = (uint64_t *)(lds + C::RING) + grp * 4 * C::VW;
    // vector i of a tile's that this lane loads and widens
    auto part = [&](int i) { return (i * C::GW + gw) * 64 + lane; };
    auto none = [&](int i) { return C::KT * C::CH % (64 * C::GW) && (i * C::GW + gw) * 64 >= C::KT * C::CH; };
    const int last = p.c.vecs - 1;
    // where a tile's operands lie for this lane: K's of step 0, V's of column block nb0
    const char *const kat = kring + (lane & 31) * C::KB + h * 16;
    const char *const vat = vring + (4 * h + ((lane & 15) >> 2)) * C::VB + nb0 * 64 + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    auto vop = [&](const char *vt, int j) {
        const char *const at = vt + j % C::NB * 64 + 16 * (j / C::NB) * C::VB;
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DSEL_LDS s16x4 *)at);
        const s16x4 z = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DSEL_LDS s16x4 *)(at + 8 * C::VB));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(y, z, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    attn_units<C>(p, [&](const AttnUnit &x, const AttnShares &shares, int32_t *join) {
        const AttnRow &row = x.row;
        const int b = x.b, r0 = x.r0, r1 = x.r1;
        // the lane's rows, and their q: eight values of every 16-deep step
        const int rows = row.n * p.group, r = x.rt * C::ROWS + rw * 32 + (lane & 31);
        const bool live = r < rows;
        const bool idle = x.rt * C::ROWS + rw * 32 >= rows;  // the whole wave: it only moves keys
        const int t = live ? r / p.group : 0, head = x.hk * p.group + (live ? r - t * p.group : 0);
        const uint16_t *const qr = (const uint16_t *)p.q + b * p.sqb + t * p.sqt + head * p.sqh;
        bf16x8 q[C::QS];
#pragma unroll
        for (int j = 0; j < C::QS; ++j) {
            const int d = 16 * j + 8 * h;
            q[j] = __builtin_bit_cast(bf16x8, live && d < p.D ? *(const u32x4 *)(qr + d) : u32x4{0, 0, 0, 0});
        }
        const Attn4Keys keys{p.t.table + b * p.t.ld, x.hk * p.c.head_stride, (uint32_t)(row.s + row.n)};
        auto first_key = [&](int round) { return row.at(round) * C::ROUND + grp * C::KT; };
        // (Past the last round its keys again: a load that may not be made would make
        // its registers' copies, and waits for them.)
        auto pos = [&](int round, int i) { return (uint32_t)(first_key(min(round, r1 - 1)) + part(i) / C::CH); };

        // What this lane has of the next rounds' keys, as loaded: vectors of K and V,
        // their scales, and where they lie, of an even and an odd round (counted from
        // r0).  Vectors past the head dim read the row's last one: of K they meet zeros
        // of q (and a NaN among them makes no score NaN that is not so already), and V's
        // columns there are written nowhere.
        struct Raw {
            u32x4 k[C::VC], v[C::VC];
            uint32_t ks[C::VC], vs[C::VC];
            int64_t at[C::VC];
            bool bad[C::VC];  // K's page is none
            int page[C::VC];  // of the round whose K is loaded next
        } raw[2];
        // Page ids are fetched two rounds before they are taken: loads land in their
        // order, so one fetched behind a round's vectors would have to wait for them.
        auto fetch_pages = [&](Raw &w, int round) {
#pragma unroll
            for (int i = 0; i < C::VC; ++i)
                if (!none(i)) w.page[i] = keys.page(p, pos(round, i));
        };
        auto load_k = [&](Raw &w, int round) {
#pragma unroll
            for (int i = 0; i < C::VC; ++i) {
                if (none(i)) break;
                const uint32_t k = pos(round, i);
                w.at[i] = keys.place(p, k, w.page[i], &w.bad[i]) + min(part(i) % C::CH, last);
                if (w.bad[i] && in_reach<C>(p, row.s, k)) device_error(kErrPage);
                w.k[i] = ((const u32x4 *)p.c.k)[w.at[i]];
                w.ks[i] = p.c.k_block[w.at[i]];
            }
        };
        auto load_v = [&](Raw &w) {
#pragma unroll
            for (int i = 0; i < C::VC; ++i) {
                if (none(i)) break;
                w.v[i] = ((const u32x4 *)p.c.v)[w.at[i]];
                w.vs[i] = p.c.v_block[w.at[i]];
            }
        };
        // Widening a round's K and V into stages ks and vs of LDS is cut into 8 VC pieces:
        // 16 bytes of K, then of V.  V's four chunks of a vector are written in an order
        // of the row's (chunk j ^ turn(row) in turn j), so that the rows of sixteen lanes
        // write to banks apart.
        auto widen_k = [&](const Raw &w, int st, int i, int j) {
            if (none(i)) return;
            if (j == 0) {
                const uint64_t m = ballot(w.bad[i]);
                if (lane == 0) bits[(2 + st) * C::VW + i * C::GW + gw] = m;
            }
            char *const to = kring + st * C::KTILE + part(i) / C::CH * C::KB + part(i) % C::CH * 64;
            *(bf16x8 *)(to + 16 * j) = widen_fp4(w.k[i][j], block_scale(w.ks[i]));
        };
        auto widen_v = [&](Raw &w, int st, int i, int j) {
            if (none(i)) return;
            const int rr = part(i) / C::CH, tn = C::turn(rr);
            if (j == 0) {
                const bool nan = not_finite(w.vs[i]);
                const uint64_t m = ballot(nan);
                if (lane == 0) bits[st * C::VW + i * C::GW + gw] = m;
                if (nan) w.vs[i] = 0;  // (what the block holds is still finite)
                if (tn & 1) w.v[i] = u32x4{w.v[i][1], w.v[i][0], w.v[i][3], w.v[i][2]};
                if (tn & 2) w.v[i] = u32x4{w.v[i][2], w.v[i][3], w.v[i][0], w.v[i][1]};
            }
            const uint32_t to = (uint32_t)(rr * C::VB + part(i) % C::CH * 64 + tn * 16);
            *(bf16x8 *)(vring + st * C::VTILE + (to ^ (16 * j))) = widen_fp4(w.v[i][j], block_scale(w.vs[i]));
        };
        auto meet = [&] {  // all of this wave's LDS work done, and all waves here
            wait_vmcnt_lgkm0<63>();
            wg_barrier();
        };

        // Round r works on the scores of its keys, adds the products of the 32 keys
        // before, and computes the scores of the 32 after.  Before the first step that
        // takes K of r + 1 all waves meet; the step before that widens K of r + 1 and V
        // of r (rounds of 32 keys have one step: it widens K of r + 2 and V of r, which
        // the next round takes), the other one sends out loads that have two rounds to land.
        constexpr bool LAG = C::NS == 1;
        fetch_pages(raw[0], r0);
        fetch_pages(raw[1], r0 + 1);
        load_k(raw[0], r0);
        load_v(raw[0]);
        fetch_pages(raw[0], r0 + 2);
        AttnState<C> a;
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb) a.o[nb] = floatx16{};
        a.m = -__builtin_inff();
        a.l = 0.0f;
        // the step before the first one: weights of 0, and a V of 0 for them
        for (int i = (gw * 64 + lane) * 16; i < C::VTILE; i += C::GW * 1024) *(u32x4 *)(vring + C::VTILE + i) = u32x4{0, 0, 0, 0};
        if (gw == 0 && lane < C::VW) bits[C::VW + lane] = 0;
        bf16x8 w[2];
        w[0] = w[1] = bf16x8{};
        load_k(raw[1], r0 + 1);
        load_v(raw[1]);
        fetch_pages(raw[1], r0 + 3);
#pragma unroll
        for (int j = 0; j < 4 * C::VC; ++j) widen_k(raw[0], 0, j >> 2, j & 3);
        load_k(raw[0], r0 + 2);
        fetch_pages(raw[0], r0 + 4);
        if constexpr (LAG) {
#pragma unroll
            for (int j = 0; j < 4 * C::VC; ++j) widen_k(raw[1], 1, j >> 2, j & 3);
            load_k(raw[1], r0 + 3);
            fetch_pages(raw[1], r0 + 5);
        }
        meet();
        floatx16 s = {}, s2;
        if (!idle) {
#pragma unroll
            for (int j = 0; j < C::QS; ++j) s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*(const bf16x8 *)(kat + 32 * j), q[j], s, 0, 0, 0);
        }
        uint32_t seen = 0;  // what the lane's row sees of the 32 keys before
        Attn4Bits<C> lost;  // of the 32 keys that s is of
        lost.load(bits + 2 * C::VW, 0);
        // The first round of one step widens K of r0 + 2 into the stage that these were
        // read from, which every wave has to have done.  (Rounds of two steps widen into
        // the other stage first, and meet before they come to this one.)
        if constexpr (LAG) meet();
        // One step: scores s of 32 keys from position kb on, V of the 32 before in stage
        // VST, K of the 32 after in stage KST (sub-rounds VSUB and KSUB)
        auto step = [&](floatx16 &s, floatx16 &s2, int kb, auto vst, auto vsub, auto kst, auto ksub, auto side) {
            constexpr int VST = decltype(vst)::value, VSUB = decltype(vsub)::value;
            constexpr int KST = decltype(kst)::value, KSUB = decltype(ksub)::value;
            Attn4Bits<C> nan, lost2;
            nan.load(bits + VST * C::VW, VSUB);
            uint32_t see = ~0u;
            bool whole = kb + 32 <= row.s;
            if constexpr (C::WIN) whole = whole && (kb + 32 <= p.sinks || kb > row.s + p.T - 1 - p.window);
            if (lost.any() || !whole) {
                if constexpr (C::WIN) see = sees_near(p, b, t, depth_of(p, b, t), row.s, kb);
                else see = sees_of(p, b, t, row.s, kb);
                see &= ~keys_from(kb, row.s + row.n) & ~lost.keys(0);
                const uint32_t m = see >> (4 * h);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!((m >> (8 * (i >> 2) + (i & 3))) & 1)) s[i] = -__builtin_inff();
            }
            lost2.load(bits + (2 + KST) * C::VW, KSUB);
            const char *const kt = kat + KST * C::KTILE + KSUB * 32 * C::KB, *const vt = vat + VST * C::VTILE + VSUB * 32 * C::VB;
            const float f = attn4_step<C>(a, s, s2, w, q, p.scale, [&](int j) { return *(const bf16x8 *)(kt + 32 * j); },
                                          [&](int j) { return vop(vt, j); }, side);
            if (nan.any()) attn4_nan<C>(a, nan, nb0, seen);
            if (ballot(f != 1.0f)) {
#pragma unroll
                for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) a.o[nb][i] *= f;
            }
            lost = lost2;
            seen = see;
        };
        // slice i of S of the pieces of widening K from kw to stage ks, V from vw to vs
        constexpr int S = C::STEPS, PIECES = 4 * C::VC;
        auto widen = [&](int i, const Raw &kw, int ks, Raw &vw, int vs) {
#pragma unroll
            for (int j = i * PIECES * 2 / S; j < (i + 1) * PIECES * 2 / S; ++j) {
                if (j < PIECES) widen_k(kw, ks, j >> 2, j & 3);
                else widen_v(vw, vs, (j - PIECES) >> 2, j & 3);
            }
        };
        auto go = [&](int round, floatx16 &s, floatx16 &s2, auto stage) {
            constexpr int ST = decltype(stage)::value;
            constexpr std::integral_constant<int, ST> st;
            constexpr std::integral_constant<int, 1 - ST> nx;
            constexpr std::integral_constant<int, 0> c0;
            constexpr std::integral_constant<int, 1> c1;
            const int kb = first_key(round);
            if constexpr (LAG) {
                // K of r + 2 comes from, and K of r + 4 goes to, the registers of even
                // (odd) rounds, like V of r and r + 2
                auto side = [&](int i) {
                    widen(i, raw[ST], ST, raw[ST], ST);
                    if (i == S - 1) {
                        load_v(raw[ST]);
                        load_k(raw[ST], round + 4);
                        fetch_pages(raw[ST], round + 6);
                    }
                };
                if (idle) {
#pragma unroll
                    for (int i = 0; i < S; ++i) side(i);
                } else {
                    step(s, s2, kb, nx, c0, nx, c0, side);
                }
                meet();
            } else {
                auto side = [&](int i) { widen(i, raw[1 - ST], 1 - ST, raw[ST], ST); };
                auto loads = [&](int i) {
                    if (i == 0) load_v(raw[ST]);
                    if (i == 1) {
                        load_k(raw[1 - ST], round + 3);
                        fetch_pages(raw[1 - ST], round + 5);
                    }
                };
                if (idle) {
#pragma unroll
                    for (int i = 0; i < S; ++i) side(i);
                } else {
                    step(s, s2, kb, nx, c1, st, c1, side);
                }
                meet();
                if (idle) {
                    loads(0);
                    loads(1);
                } else {
                    step(s2, s, kb + 32, st, c0, nx, c0, loads);
                }
            }
        };
        for (int round = r0; round < r1; round += 2) {
            go(round, s, s2, std::integral_constant<int, 0>{});
            if (round + 1 < r1) {
                if constexpr (LAG) go(round + 1, s2, s, std::integral_constant<int, 1>{});
                else go(round + 1, s, s2, std::integral_constant<int, 1>{});
            }
        }
        {
            // the products of the last 32 keys
            const int st = (r1 - 1 - r0) & 1;
            if (!idle) {
                Attn4Bits<C> nan;
                nan.load(bits + st * C::VW, C::NS - 1);
#pragma unroll
                for (int j = 0; j < C::PS; ++j)
                    a.o[j % C::NB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vop(vat + st * C::VTILE + (C::NS - 1) * 32 * C::VB, j),
                                                                            w[j / C::NB], a.o[j % C::NB], 0, 0, 0);
                if (nan.any()) attn4_nan<C>(a, nan, nb0, seen);
            }
        }
        const AttnPiece piece{b, x.hk, x.rt, t, head, r0, r1, live, x.share, x.u};
        attn_finish<C>(p, a, row, piece, shares, lds, join);
    });
}

// ---- at most 32 rows --------------------------------------------------------------

// RR row tiles of 16; KW waves with 64 keys a round each.  Measured as above: one token
// for each of 16 rows of up to 60,000 positions 133 to 157 us (5.1 to 4.3 TB/s; with
// products of 32 rows 190), tokens-first pages 256 to 265; one token over 333
// positions 11 us.  Two row tiles, 8 tokens for each of 32 rows of 8,192: 160 us, and
// 185 tokens-first; their registers spill (248 to 268 bytes of a lane's at 128).  Head
// size 256, one tile, 1 or 2 tokens: 136 us (4.2 TB/s).
template <bool WIN_, int DP_, int RR_, int KW_>
struct Attn4FewCfg {
    static constexpr bool E4M3 = false, WIN = WIN_;
    static constexpr int DP = DP_, RR = RR_, KW = KW_, KT = 64;
    static constexpr int RB = DP * 2, NT = 64 * KW, ROWS = 16 * RR, ROUND = KT * KW;
    static constexpr int TILE = KT * RB;             // V's
    static constexpr int NB = DP / 16, CH = DP / 32;  // blocks of 16 columns; vectors of a row
    static constexpr int VC = CH;                     // V's vectors of a tile, for a lane
    static constexpr int KS = DP / 32;                // steps of q's product
    static constexpr int KV = CH >= 4 ? CH / 4 : 1;   // K's vectors of a key, for a lane (of 64 columns: half a one)
    static constexpr int SUMS = KW * (RR * NB * 4 + RR * 2) * 256;
    static constexpr int LDS = KW * TILE > SUMS ? KW * TILE : SUMS;
    static constexpr int PART = ROWS * (DP + 2);
    static constexpr int WGS = LDS <= 80 * 1024 ? 2 : 1, WAVES = WGS * NT / 256;
    static_assert(DP % 64 == 0 && NB % KW == 0, "tile geometry");
    // of eight rows that half a wave reads 32 bytes of
    __device__ static __forceinline__ int vkey(int row) { return RB >= 256 ? (row & 7) << 1 : ((row >> 1) & 3) << 1; }
    __device__ static __forceinline__ int turn(int row) { return RB >= 256 ? (row >> 1) & 1 : 0; }
};

// S^T = K Q^T by 16 x 16 x 32 MFMA: of 16 keys lane l has the scores of keys 4 (l / 16)
// + i with row l % 16.  K's vector v of a key goes to lane group v (of 64 columns, its
// halves to groups v and v + 2), which supplies 8 values of it to each step of the
// product: no lane loads a byte that it does not use.  Two sets of 16 keys are the
// operand of O^T = V^T P^T, with V^T's keys in the same order.
template <class C>
__global__ __launch_bounds__(C::NT, C::WAVES) void tree_attn4_few_kernel(TreeAttnParams p) {
    __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
    const int lane = lane_id(), g = lane >> 4, c16 = lane & 15;
    const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char *const vt = lds + grp * C::TILE;
    const int last = p.c.vecs - 1;
    int vat[C::NB];
    const int vrow = 4 * g + (c16 >> 2);
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb)
        vat[nb] = vrow * C::RB + (((2 * nb + ((lane & 3) >> 1)) ^ C::vkey(vrow)) << 4) + ((lane & 1) << 3);
    attn_units<C>(p, [&](const AttnUnit &x, const AttnShares &shares, int32_t *join) {
        const AttnRow &row = x.row;
        const int b = x.b, r0 = x.r0, r1 = x.r1, rows = row.n * p.group;
        int t[C::RR], head[C::RR];
        bool live[C::RR];
        bf16x8 q[C::RR][C::KS];
#pragma unroll
        for (int i = 0; i < C::RR; ++i) {
            const int r = x.rt * C::ROWS + 16 * i + c16;
            live[i] = r < rows;
            t[i] = live[i] ? r / p.group : 0;
            head[i] = x.hk * p.group + (live[i] ? r - t[i] * p.group : 0);
            const uint16_t *const qr = (const uint16_t *)p.q + b * p.sqb + t[i] * p.sqt + head[i] * p.sqh;
#pragma unroll
            for (int j = 0; j < C::KS; ++j) {
                const int d = C::CH >= 4 ? 32 * (g + 4 * (j / 4)) + 8 * (j & 3) : 32 * (g & 1) + 8 * (2 * (g >> 1) + j);
                q[i][j] = __builtin_bit_cast(bf16x8, live[i] && d < p.D ? *(const u32x4 *)(qr + d) : u32x4{0, 0, 0, 0});
            }
        }
        const Attn4Keys keys{p.t.table + b * p.t.ld, x.hk * p.c.head_stride, (uint32_t)(row.s + row.n)};
        // (past the last round its keys again, as above)
        auto first_key = [&](int round) { return row.at(min(round, r1 - 1)) * C::ROUND + grp * C::KT; };
        // lane j places key j of the tile, a round ahead of its vectors
        auto page_of = [&](int round) { return keys.page(p, (uint32_t)(first_key(round) + lane)); };
        // vectors of K (4 sets of 16 keys) and V, their scales
        u32x4 k[4][C::KV], v[C::VC];
        uint32_t ks[4][C::KV], vs[C::VC];
        auto load = [&](int64_t off) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t o = (int64_t)shfl_idx64((uint64_t)off, 16 * i + c16);
#pragma unroll
                for (int j = 0; j < C::KV; ++j) {
                    const int64_t at = o + min(C::CH >= 4 ? g + 4 * j : g & 1, last);
                    if constexpr (C::CH >= 4) {
                        k[i][j] = ((const u32x4 *)p.c.k)[at];
                    } else {
                        const uint2 w = ((const uint2 *)p.c.k)[2 * at + (g >> 1)];
                        k[i][j] = u32x4{w.x, w.y, 0, 0};
                    }
                    ks[i][j] = p.c.k_block[at];
                }
            }
#pragma unroll
            for (int i = 0; i < C::VC; ++i) {
                const int part = i * 64 + lane;
                const int64_t o = (int64_t)shfl_idx64((uint64_t)off, part / C::CH) + min(part % C::CH, last);
                v[i] = ((const u32x4 *)p.c.v)[o];
                vs[i] = p.c.v_block[o];
            }
        };
        floatx4 o[C::RR][C::NB];
        float m[C::RR], l[C::RR];
#pragma unroll
        for (int i = 0; i < C::RR; ++i) {
            m[i] = -__builtin_inff();
            l[i] = 0.0f;
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb) o[i][nb] = floatx4{};
        }
        auto place = [&](int round, int page, uint64_t *ok) {
            const uint32_t pos = (uint32_t)(first_key(round) + lane);
            bool bad;
            const int64_t off = keys.place(p, pos, page, &bad);
            if (bad && in_reach<C>(p, row.s, pos)) device_error(kErrPage);
            *ok = ballot(pos < keys.total && !bad);
            return off;
        };
        uint64_t now, next = 0;
        load(place(r0, page_of(r0), &now));
        int page = page_of(r0 + 1);
        for (int round = r0; round < r1; ++round) {
            // V into LDS (this wave's own), the scores of 64 keys, and the next loads
            uint64_t nan = 0;  // lanes with a block among V's that is not finite: none, mostly
#pragma unroll
            for (int i = 0; i < C::VC; ++i) {
                const int part = i * 64 + lane, rr = part / C::CH, ch = part % C::CH, tn = C::turn(rr);
                const bool is = not_finite(vs[i]);
                nan |= ballot(is);
                const float f = block_scale(is ? 0 : vs[i]);
                u32x4 w = v[i];
                if (tn) w = u32x4{w[1], w[0], w[3], w[2]};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *(bf16x8 *)(vt + rr * C::RB + (((4 * ch + (j ^ tn)) ^ C::vkey(rr)) << 4)) = widen_fp4(w[j], f);
            }
            uint32_t vbad[C::VC];
            if (nan) {
#pragma unroll
                for (int i = 0; i < C::VC; ++i) vbad[i] = not_finite(vs[i]);
            }
            floatx4 s[C::RR][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int n = 0; n < C::RR; ++n) s[n][i] = floatx4{};
#pragma unroll
                for (int j = 0; j < C::KS; ++j) {
                    const bf16x8 kw = widen_fp4(k[i][j / 4][j & 3], block_scale(ks[i][j / 4]));
#pragma unroll
                    for (int n = 0; n < C::RR; ++n) s[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kw, q[n][j], s[n][i], 0, 0, 0);
                }
            }
            const uint64_t ok = now;
            load(place(round + 1, page, &next));
            page = page_of(round + 2);
            now = next;
            const int kb = first_key(round);
            bool whole = kb + C::KT <= row.s && ok == ~0ull;
            if constexpr (C::WIN) whole = whole && (kb + C::KT <= p.sinks || kb > row.s + p.T - 1 - p.window);
            uint64_t see[C::RR];
#pragma unroll
            for (int n = 0; n < C::RR; ++n) {
                see[n] = ok;
                if (!whole) {
                    if constexpr (C::WIN) {
                        const int d = depth_of(p, b, t[n]);
                        see[n] &= sees_near(p, b, t[n], d, row.s, kb) | (uint64_t)sees_near(p, b, t[n], d, row.s, kb + 32) << 32;
                    } else {
                        see[n] &= sees_of(p, b, t[n], row.s, kb) | (uint64_t)sees_of(p, b, t[n], row.s, kb + 32) << 32;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!((see[n] >> (16 * i + 4 * g + e)) & 1)) s[n][i][e] = -__builtin_inff();
                }
                // softmax, as attn_rescale and attn_weights
                float top = -__builtin_inff();
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, s[n][i][e]);
                top = fmaxf(top, __uint_as_float(xor_lane32<16>(__float_as_uint(top))));
                top = fmaxf(top, __uint_as_float(xor_lane32<32>(__float_as_uint(top)))) * p.scale;
                const bool move = top > m[n] + 8.0f;
                if (ballot(move)) {
                    const float f = move ? __builtin_amdgcn_exp2f(m[n] - top) : 1.0f;
#pragma unroll
                    for (int nb = 0; nb < C::NB; ++nb) o[n][nb] *= f;
                    l[n] *= f;
                    if (move) m[n] = top;
                }
                const float ms = m[n] == -__builtin_inff() ? 0.0f : m[n];
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[n][i][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][i][e], p.scale, -ms));
                        sum += s[n][i][e];
                    }
                l[n] += sum;
            }
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                bf16x8 w[C::RR];
#pragma unroll
                for (int n = 0; n < C::RR; ++n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[n][e] = (__bf16)s[n][2 * sub + (e >> 2)][e & 3];  // (as attn_values)
#pragma unroll
                for (int nb = 0; nb < C::NB; ++nb) {
                    const char *const at = vt + vat[nb] + 32 * sub * C::RB;
                    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DSEL_LDS s16x4 *)at);
                    const s16x4 z = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DSEL_LDS s16x4 *)(at + 16 * C::RB));
                    typedef short s16x8 __attribute__((ext_vector_type(8)));
                    const bf16x8 vw = __builtin_bit_cast(bf16x8, __builtin_shufflevector(y, z, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                    for (int n = 0; n < C::RR; ++n) o[n][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vw, w[n], o[n][nb], 0, 0, 0);
                }
            }
            if (nan) {
                // (as attn4_nan)
#pragma unroll
                for (int i = 0; i < C::VC; ++i)
                    for (uint64_t mm = ballot(vbad[i] != 0); mm; mm &= mm - 1) {
                        const int part = i * 64 + __builtin_ctzll(mm), key = part / C::CH, ch = part % C::CH;
#pragma unroll
                        for (int n = 0; n < C::RR; ++n)
#pragma unroll
                            for (int nb = 0; nb < C::NB; ++nb)
                                if (nb >> 1 == ch && ((see[n] >> key) & 1)) o[n][nb] += __builtin_nanf("");
                    }
            }
        }

        // the waves' sums joined through LDS: every wave joins, and writes, its part of
        // the columns
        constexpr int Q = C::NB / C::KW;
        __syncthreads();
        floatx4 *const sums = (floatx4 *)lds + lane;
        float2 *const stats = (float2 *)(lds + C::KW * C::RR * C::NB * 1024) + lane;
#pragma unroll
        for (int n = 0; n < C::RR; ++n) {
            l[n] += __uint_as_float(xor_lane32<16>(__float_as_uint(l[n])));
            l[n] += __uint_as_float(xor_lane32<32>(__float_as_uint(l[n])));
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb) sums[((grp * C::RR + n) * C::NB + nb) * 64] = o[n][nb];
            stats[(grp * C::RR + n) * 64] = float2{m[n], l[n]};
        }
        __syncthreads();
        if (threadIdx.x == 0 && r0 == 0 && r1 < row.rounds) {
            join[0] = b;
            join[1] = x.hk;
            join[2] = x.rt;
            join[3] = x.share;
            join[4] = shares.of(x.u + row.rounds - 1);
            join[5] = row.n;
        }
#pragma unroll
        for (int n = 0; n < C::RR; ++n) {
            float mm = -__builtin_inff(), ll = 0.0f, f[C::KW];
            float2 st[C::KW];
#pragma unroll
            for (int w = 0; w < C::KW; ++w) {
                st[w] = stats[(w * C::RR + n) * 64];
                mm = fmaxf(mm, st[w].x);
            }
            const float ms = mm == -__builtin_inff() ? 0.0f : mm;
#pragma unroll
            for (int w = 0; w < C::KW; ++w) {
                f[w] = __builtin_amdgcn_exp2f(st[w].x - ms);
                ll += st[w].y * f[w];
            }
            const bool first = g == 0 && grp == 0, done = r0 == 0 && r1 == row.rounds;
            const bool some = !(ll <= 0.0f);  // NaN counts as something
            const float inv = some ? 1.0f / ll : 0.0f;
            const int64_t at = ((int64_t)b * p.T + t[n]) * p.Hq + head[n];
            float *const to = p.part + (int64_t)(x.share * 2 + (r0 == 0)) * C::PART;
            const int rr = 16 * n + c16;
            if (live[n] && first) {
                if (!done) {
                    to[rr] = mm;
                    to[C::ROWS + rr] = ll;
                } else if (p.lse) {
                    p.lse[at] = some ? (mm + __builtin_amdgcn_logf(ll)) * 0.69314718055994531f : -__builtin_inff();
                }
            }
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int nb = grp * Q + i, d = 16 * nb + 4 * g;
                floatx4 y = {};
#pragma unroll
                for (int w = 0; w < C::KW; ++w) y += sums[((w * C::RR + n) * C::NB + nb) * 64] * f[w];
                if (!live[n]) continue;
                if (!done) {
                    *(floatx4 *)(to + 2 * C::ROWS + rr * C::DP + d) = y;
                } else if (d < p.D) {
                    bf16x2 z[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e >> 1][e & 1] = (__bf16)(some ? y[e] * inv : 0.0f);
                    *(uint2 *)(p.out + at * p.D + d) = __builtin_bit_cast(uint2, z);
                }
            }
        }
    });
}

}  // namespace dsel
