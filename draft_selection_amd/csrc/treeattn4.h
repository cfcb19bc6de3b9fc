// Attention of a tree of drafted tokens over a paged cache held in 4 bits.
//
// The same sums as treeattn.h, over the same rows, rounds and shares of work.  A
// value of the cache, 2^(s-127) times an e2m1 value, is exact in bf16, so once
// widened the products are those of a bf16 cache with the same values.
//
// A 16-byte vector is 32 values and has one scale byte.  K goes straight from the
// cache to registers: the operand of S^T = K Q^T wants of lane l 8 values of key
// l % 32, and a vector is 8 values for each of four steps of the product, so lane l
// loads vectors 2 c + l / 32 of its key's row and widens them (one instruction for
// two values, scale and all) on their way into the matrix core; no LDS, at a third
// of the bytes of a tile of 8 bits.  V has to be read by columns, and a column's
// values of different keys have different scales, so they cannot stay 4 bits wide
// until then: the waves of a key group widen the tile once, each its part, into a
// bf16 tile in LDS, from which the transposing reads deliver it as in treeattn.h.
// Loads go out one round ahead into registers; page ids one round before that.
#pragma once

#include "treeattn.h"

namespace dsel {

// DP: padded head dim; RW waves of 32 rows, each as CW waves that hold DP / CW
// columns of the output, by KW key groups; KT keys a tile
template <bool WIN_, int DP_, int RW_, int CW_, int KW_, int KT_>
struct Attn4Cfg {
    static constexpr bool E4M3 = false, WIN = WIN_;  // (the tile in LDS is one of bf16)
    static constexpr int DP = DP_, RW = RW_, CW = CW_, KW = KW_, KT = KT_;
    static constexpr int GW = RW * CW;
    static constexpr int RB = DP * 2;
    static constexpr int NT = 64 * GW * KW, ROWS = 32 * RW, ROUND = KT * KW;
    static constexpr int TILE = KT * RB;
    static constexpr int ST = GW > 1 ? 2 : 1;  // V tiles: a wave alone writes its next one after its own reads
    static constexpr int SUMS = KW > 1 ? KW * GW * (DP / CW / 2 + 2) * 256 : 0;
    static constexpr int RING = KW * ST * TILE > SUMS ? KW * ST * TILE : SUMS;
    static constexpr int LDS = RING;
    static constexpr int PART = ROWS * (DP + 2);
    static constexpr int NS = KT / 32, NB = DP / 32 / CW, QUADS = NB * 4 / KW;
    static constexpr int CH = DP / 32;                            // vectors of a row
    static constexpr int KC = CH / 2;                             // K vectors of a lane per 32 keys
    static constexpr int VC = (KT * CH + 64 * GW - 1) / (64 * GW);  // and V vectors of a tile
    static constexpr int WGS = LDS <= 80 * 1024 && NT <= 256 ? 2 : 1;
    static constexpr int WAVES = WGS * NT / 256 < 1 ? 1 : WGS * NT / 256;
    static_assert(KT <= 64 && KT % 32 == 0 && DP % 64 == 0, "tile geometry");
    __device__ static __forceinline__ int vkey(int row) { return RB >= 256 ? (row & 3) << 2 : ((row >> 1) & 1) << 2; }
};

// Scale byte s as 2^(s - 127); the conversions take its exponent alone, and 255 as NaN
__device__ __forceinline__ float block_scale(uint32_t s) { return __uint_as_float(s << 23); }

// the 8 values of a word
__device__ __forceinline__ bf16x8 widen_fp4(uint32_t w, float s) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// What a lane has of a round's keys, as loaded
template <class C>
struct Attn4Raw {
    u32x4 k[C::NS * C::KC], v[C::VC];
    uint32_t ks[C::NS * C::KC], vs[C::VC];
};

template <class C>
__device__ __forceinline__ void attn4_scores(AttnScores<C> &s, const bf16x8 (&q)[C::DP / 16], const Attn4Raw<C> &x) {
#pragma unroll
    for (int sub = 0; sub < C::NS; ++sub) {
        s[sub] = floatx16{};
#pragma unroll
        for (int c = 0; c < C::KC; ++c) {
            const float f = block_scale(x.ks[sub * C::KC + c]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_fp4(x.k[sub * C::KC + c][j], f), q[4 * c + j], s[sub], 0, 0, 0);
        }
    }
}

template <class C>
__global__ __launch_bounds__(C::NT, C::WAVES) void tree_attn4_kernel(TreeAttnParams p) {
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

    char *const vring = lds + grp * C::ST * C::TILE;
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
        const int64_t hv = hk * p.c.head_stride;
        const int32_t *const table = p.t.table + b * p.t.ld;

        // the lane's rows, and their q: eight values of every 16-deep step
        const int rows = row.n * p.group, r = rt * C::ROWS + rw * 32 + (lane & 31);
        const bool live = r < rows;
        const bool idle = rt * C::ROWS + rw * 32 >= rows;  // the whole wave: it only moves keys
        const int t = live ? r / p.group : 0, head = hk * p.group + (live ? r - t * p.group : 0);
        const uint16_t *const qr = (const uint16_t *)p.q + b * p.sqb + t * p.sqt + head * p.sqh;
        bf16x8 q[C::DP / 16];
#pragma unroll
        for (int ks = 0; ks < C::DP / 16; ++ks) {
            const int d = 64 * (ks >> 2) + 32 * h + 8 * (ks & 3);
            const u32x4 w = live && d < p.D ? *(const u32x4 *)(qr + d) : u32x4{0, 0, 0, 0};
            q[ks] = __builtin_bit_cast(bf16x8, w);
        }

        // The keys of a round: lane j of every wave places key j of its group's tile
        // (or, of a tile of 32, key j % 32) as an offset in vectors, which is that of
        // its scale byte too.  A key past the end, or of a page that is none, has no
        // place; it reads what the first key that has one reads, and its score is masked.
        auto key_pos = [&](int round) {
            return (uint32_t)(row.at(round) * C::ROUND + grp * C::KT + (lane & (C::KT - 1)));
        };
        auto page_at = [&](uint32_t k) { return p.page_shift >= 0 ? k >> p.page_shift : k / (uint32_t)p.c.page_size; };
        auto page_of = [&](int round) {
            const uint32_t k = key_pos(round);
            return table[k < (uint32_t)total ? page_at(k) : 0u];
        };
        auto place = [&](int round, int page, uint64_t *ok) -> int64_t {
            const uint32_t k = key_pos(round);
            const bool in = k < (uint32_t)total, good = in && page >= 0 && page < p.c.num_pages;
            if (in && !good) device_error(kErrPage);
            const uint32_t slot = k - page_at(k) * (uint32_t)p.c.page_size;
            const int64_t off = hv + (int64_t)page * p.c.page_stride + (int64_t)slot * p.c.slot_stride;
            const uint64_t m = ballot(good);
            *ok = m;
            if (m == ~0ull) return off;
            const int64_t first = m ? (int64_t)readlane64((uint64_t)off, __builtin_ctzll(m)) : hv;
            return good ? off : first;
        };
        const bool padded = p.c.vecs < C::CH;  // vectors past the head dim read zeros
        auto load = [&](Attn4Raw<C> &x, int64_t off) {
#pragma unroll
            for (int sub = 0; sub < C::NS; ++sub) {
                const int64_t o = C::NS == 1 ? off : (int64_t)shfl_idx64((uint64_t)off, 32 * sub + (lane & 31));
#pragma unroll
                for (int c = 0; c < C::KC; ++c) {
                    const bool none = padded && 2 * c + h >= p.c.vecs;
                    const int64_t at = o + 2 * c + h;
                    x.k[sub * C::KC + c] = *(none ? g_attn_zero : (const u32x4 *)p.c.k + at);
                    x.ks[sub * C::KC + c] = *(none ? (const uint8_t *)g_attn_zero : p.c.k_block + at);
                }
            }
#pragma unroll
            for (int i = 0; i < C::VC; ++i) {
                const int at = (i * C::GW + gw) * 64 + lane, rr = at / C::CH, ch = at % C::CH;
                if (C::KT * C::CH % (64 * C::GW) && (i * C::GW + gw) * 64 >= C::KT * C::CH) break;
                const int64_t o = (int64_t)shfl_idx64((uint64_t)off, rr) + ch;
                const bool none = padded && ch >= p.c.vecs;
                x.v[i] = *(none ? g_attn_zero : (const u32x4 *)p.c.v + o);
                x.vs[i] = *(none ? (const uint8_t *)g_attn_zero : p.c.v_block + o);
            }
        };
        auto widen_v = [&](char *vt, const Attn4Raw<C> &x) {
#pragma unroll
            for (int i = 0; i < C::VC; ++i) {
                const int at = (i * C::GW + gw) * 64 + lane, rr = at / C::CH, ch = at % C::CH;
                if (C::KT * C::CH % (64 * C::GW) && (i * C::GW + gw) * 64 >= C::KT * C::CH) break;
                const float f = block_scale(x.vs[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *(bf16x8 *)(vt + rr * C::RB + (((4 * ch + j) ^ C::vkey(rr)) << 4)) = widen_fp4(x.v[i][j], f);
            }
        };
        Attn4Raw<C> x;
        uint64_t now, next = 0;
        load(x, place(r0, page_of(r0), &now));
        int page = page_of(r0 + 1);
        AttnState<C> a;
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb) a.o[nb] = floatx16{};
        a.m = -__builtin_inff();
        a.l = 0.0f;

        constexpr uint64_t kAll = ~0ull >> (64 - C::KT);
        for (int round = r0; round < r1; ++round) {
            char *const vt = vring + (C::ST > 1 && ((round - r0) & 1) ? C::TILE : 0);
            widen_v(vt, x);
            Attn4Raw<C> y = x;
            if (round + 1 < r1) {
                load(y, place(round + 1, page, &next));
                page = page_of(round + 2);
            }
            const int kb = row.at(round) * C::ROUND + grp * C::KT;
            bool whole = kb + C::KT <= row.s && (now & kAll) == kAll;
            if constexpr (C::WIN) whole = whole && (kb + C::KT <= p.sinks || kb > row.s + p.T - 1 - p.window);
            const bool work = !idle && (now & kAll) != 0;
            uint64_t see = now;
            AttnScores<C> s;
            if (work) {
                if (!whole) {
                    if constexpr (C::WIN) {
                        const int d = depth_of(p, b, t);
                        see &= sees_near(p, b, t, d, row.s, kb) |
                               (C::KT == 64 ? (uint64_t)sees_near(p, b, t, d, row.s, kb + 32) << 32 : 0);
                    } else {
                        see &= sees_of(p, b, t, row.s, kb) | (C::KT == 64 ? (uint64_t)sees_of(p, b, t, row.s, kb + 32) << 32 : 0);
                    }
                }
                attn4_scores<C>(s, q, x);
                if (!whole) attn_mask<C>(s, see);
                attn_rescale<C>(a, s, p.scale);
                attn_weights<C>(a, s, p.scale);
            }
            if constexpr (C::GW > 1) {
                // the tile is whole; the one before it, which the next round writes
                // over, is read by nobody any more
                wait_vmcnt_lgkm0<63>();
                wg_barrier();
            }
            if (work) {
                const bool special = !whole && tile_special<C>(vt);
                attn_values<C>(a, s, vt, nb0, special);
                if (special) {
#pragma unroll
                    for (int nb = 0; nb < C::NB; ++nb) add_special<C>(a.o[nb], vt, nb0 + nb, see);
                }
            }
            x = y;
            now = next;
        }
        const AttnPiece piece{b, hk, rt, t, head, r0, r1, live, share, u};
        attn_finish<C>(p, a, row, piece, shares, lds, join);
        u += p.whole ? 1 : r1 - r0;
        if (u < uend) __syncthreads();  // the tiles (and the sums in them) are read no more
    }
}

}  // namespace dsel
