// The attention weight of every cached position, summed over nodes and heads.
//
//   w_p <- decay w_p + sum_{i, h} count_i e^(scale <q_ih, K_p> - lse_ih)
//
// with the lse that the attention left: the softmax is known, so one product and
// one exponential a score give it, V is not read, and no maximum runs along.
//
// S = Q K^T by 16 x 16 x 32 MFMA with the keys along the lanes: lane l has the
// scores of key l % 16 with rows 4 (l / 16) .. of a tile of 16, adds their weights up
// in one register, and the four lanes of a key join at the end.  So a position's sum
// over all rows and heads of a wave stays in a register.  (Tiles of 32 rows: 106 us
// where 36 rows are 2.25 of 16.)  Vector v of a key's row goes to lane group v % 4,
// which supplies 8 of its values to each step of the product that it feeds.  The lse
// is subtracted before the step to base 2 (its product with log2 e would be rounded
// at its own size, not the difference's); a row that counts nothing has lse +inf.
// The rows' values are spread over the registers through LDS.
//
// A wave holds the K operand of 64 keys of one head, straight from the cache, and
// runs the rows of q past it, while K of its next head is on its way: K is read
// once, q once per 64 keys from the caches.  Pairs of waves share the heads of the
// same keys.  Where that leaves CUs without work, a wave takes 16 keys and four
// share the heads: latency counts then (lengths, page ids, keys, head by head).
// Measured on an MI355X, captured, 32 query heads on 8 of 128: one token over 700
// positions 6.2 us (64 keys a wave: 14.5); 9 tokens for each of 32 rows of up to 8,192,
// 104 us (3.3 TB/s of K; 16 keys a wave: 135), in 8 bits 77, in 4 bits 58; one token for
// each of 2 rows of up to 131,000, 92 us (4.7 TB/s).
#pragma once

#include "treeattn4.h"

namespace dsel {

struct KeyWeightsParams {
    CacheView c;
    TableView t;
    const char *q;  // bf16
    int64_t sqb, sqt, sqh;
    const float *lse, *count;  // count: NULL = 1
    float *w;
    int64_t ld;
    const int32_t *len;
    int B, T, Hq, D, group;
    float scale, decay;
    int page_shift;
    int hs;  // waves that share the heads of the same keys: 4, 2 or 1
};

template <CacheType F_, int DP_, int NK_>
struct KeyWeightsCfg {
    static constexpr CacheType F = F_;
    static constexpr int DP = DP_, NK = NK_;                             // 16 NK keys a wave
    static constexpr int PER = F == kMxfp4 ? 32 : F == kE4m3 ? 16 : 8;  // values of a 16-byte vector
    static constexpr int CH = DP / PER, KC = CH >= 4 ? CH / 4 : 1;       // vectors of a row, and of a lane (of two, half a one)
    static constexpr int QS = DP / 32, S = QS / KC;                      // steps of the product, and those that a vector feeds
    static constexpr int WAVES = DP <= 128 ? 2 : 1;                      // (two heads' K of 256 values take over 256 registers)
};

template <class C>
__global__ __launch_bounds__(256, C::WAVES) void key_weights_kernel(KeyWeightsParams p) {
    __shared__ float shift[4][32];
    __shared__ float sums[4][C::NK * 16];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, c16 = lane & 15;
    const int hs = wave & (p.hs - 1), kg = wave / p.hs;
    const int b = blockIdx.y;
    const int n = block_len_of(p.len, b, p.T);
    if (n == 0) return;
    const int s = seq_len_of(p.t, b, 0, p.c.page_size);
    const int32_t *const table = p.t.table + b * p.t.ld;
    const int rows = n * p.group, last = p.c.vecs - 1;
    const int64_t keys = 4 / p.hs * 16 * C::NK;
    struct Raw {
        u32x4 k[C::NK][C::KC];
        uint32_t s[C::NK][C::KC];
    } raw[2];
    for (int64_t first = blockIdx.x * keys; first < s; first += gridDim.x * keys) {
        const int key0 = (int)first + kg * C::NK * 16;
        int64_t place[C::NK];
        bool good[C::NK];
#pragma unroll
        for (int i = 0; i < C::NK; ++i) {
            const int64_t k = (int64_t)key0 + 16 * i + c16;
            const uint32_t at = k < s ? (uint32_t)k : 0u;
            const uint32_t pg = p.page_shift >= 0 ? at >> p.page_shift : at / (uint32_t)p.c.page_size;
            const int page = table[pg];
            const bool none = page < 0 || page >= p.c.num_pages;
            if (k < s && none) device_error(kErrPage);
            good[i] = k < s && !none;
            place[i] = none ? 0 : (int64_t)page * p.c.page_stride + (int64_t)(at - pg * (uint32_t)p.c.page_size) * p.c.slot_stride;
        }
        float sum[C::NK];
#pragma unroll
        for (int i = 0; i < C::NK; ++i) sum[i] = 0.0f;
        // Vectors past the head dim read the row's last one and meet zeros of q.
        auto load = [&](Raw &w, int hk) {
#pragma unroll
            for (int i = 0; i < C::NK; ++i)
#pragma unroll
                for (int c = 0; c < C::KC; ++c) {
                    const int64_t at = place[i] + min(hk, p.c.heads - 1) * p.c.head_stride + min(C::CH >= 4 ? g + 4 * c : g & 1, last);
                    if constexpr (C::CH >= 4) {
                        w.k[i][c] = ((const u32x4 *)p.c.k)[at];
                    } else {
                        const uint2 half = ((const uint2 *)p.c.k)[2 * at + (g >> 1)];
                        w.k[i][c] = u32x4{half.x, half.y, 0, 0};
                    }
                    if constexpr (C::F == kMxfp4) w.s[i][c] = p.c.k_block[at];
                }
        };
        // K of the next head is asked for behind the last q of this one: loads land in
        // their order, and a q behind it would have to wait for it.
        auto add = [&](const Raw &w, int hk, Raw &next) {
            bf16x8 k[C::NK][C::QS];
#pragma unroll
            for (int i = 0; i < C::NK; ++i)
#pragma unroll
                for (int c = 0; c < C::KC; ++c) {
                    const u32x4 x = w.k[i][c];
                    if constexpr (C::F == kMxfp4) {
#pragma unroll
                        for (int j = 0; j < C::S; ++j) k[i][C::S * c + j] = widen_fp4(x[j], block_scale(w.s[i][c]));
                    } else if constexpr (C::F == kE4m3) {
                        k[i][2 * c] = widen_e4m3(x[0], x[1]);
                        k[i][2 * c + 1] = widen_e4m3(x[2], x[3]);
                    } else {
                        k[i][c] = __builtin_bit_cast(bf16x8, x);
                    }
                }
            const float c = C::F == kE4m3 && p.c.k_scale ? p.scale * p.c.k_scale[hk] : p.scale;
            // R tiles of 16 rows from row r0 on
            auto tiles = [&](int r0, auto count, auto last_tile) {
                constexpr int R = decltype(count)::value;
                bf16x8 q[R][C::QS];
                float L[R];
#pragma unroll
                for (int n = 0; n < R; ++n) {
                    const int r = r0 + 16 * n + c16;
                    const bool live = r < rows;
                    const int t = live ? r / p.group : 0, head = hk * p.group + (live ? r - t * p.group : 0);
                    const uint16_t *const qr = (const uint16_t *)p.q + b * p.sqb + t * p.sqt + head * p.sqh;
#pragma unroll
                    for (int j = 0; j < C::QS; ++j) {
                        const int d = C::CH >= 4 ? (g + 4 * (j / C::S)) * C::PER + 8 * (j % C::S) : 32 * (g & 1) + 8 * (2 * (g >> 1) + j);
                        q[n][j] = __builtin_bit_cast(bf16x8, live && d < p.D ? *(const u32x4 *)(qr + d) : u32x4{0, 0, 0, 0});
                    }
                    L[n] = __builtin_inff();
                    if (live) {
                        const float l = p.lse[((int64_t)b * p.T + t) * p.Hq + head];
                        const float a = p.count ? p.count[(int64_t)b * p.T + t] : 1.0f;
                        if (fabsf(l) < __builtin_inff() && a > 0.0f)
                            L[n] = p.count ? l - 0.69314718055994531f * __builtin_amdgcn_logf(a) : l;
                    }
                }
                if constexpr (decltype(last_tile)::value) {
                    __builtin_amdgcn_sched_barrier(0);
                    load(next, hk + p.hs);
                }
#pragma unroll
                for (int n = 0; n < R; ++n)
                    if (g == 0) shift[wave][16 * n + lane] = L[n];
                asm volatile("" ::: "memory");
                floatx4 Ls[R];
#pragma unroll
                for (int n = 0; n < R; ++n) Ls[n] = *(const floatx4 *)&shift[wave][16 * n + 4 * g];
#pragma unroll
                for (int i = 0; i < C::NK; ++i) {
                    floatx4 z[R];
#pragma unroll
                    for (int n = 0; n < R; ++n) z[n] = floatx4{};
#pragma unroll
                    for (int j = 0; j < C::QS; ++j)
#pragma unroll
                        for (int n = 0; n < R; ++n) z[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q[n][j], k[i][j], z[n], 0, 0, 0);
#pragma unroll
                    for (int n = 0; n < R; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = __builtin_fmaf(z[n][e], c, -Ls[n][e]);
                            // a row that counts nothing may meet infinities: its NaN is no more than 0
                            sum[i] += fmaxf(__builtin_amdgcn_exp2f(x * 1.44269504088896341f), 0.0f);
                        }
                }
                asm volatile("" ::: "memory");
            };
            constexpr std::integral_constant<int, 1> one;
            constexpr std::integral_constant<int, 2> two;
            int r0 = 0;
            for (; r0 + 32 < rows; r0 += 32) tiles(r0, two, std::integral_constant<bool, false>{});
            if (r0 + 16 < rows) tiles(r0, two, std::integral_constant<bool, true>{});
            else tiles(r0, one, std::integral_constant<bool, true>{});
        };
        load(raw[0], hs);
        for (int hk = hs; hk < p.c.heads; hk += 2 * p.hs) {
            add(raw[0], hk, raw[1]);
            if (hk + p.hs >= p.c.heads) break;
            add(raw[1], hk + p.hs, raw[0]);
        }
#pragma unroll
        for (int i = 0; i < C::NK; ++i) {
            sum[i] += __uint_as_float(xor_lane32<16>(__float_as_uint(sum[i])));
            sum[i] += __uint_as_float(xor_lane32<32>(__float_as_uint(sum[i])));
            if (g == 0) sums[wave][16 * i + lane] = sum[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < C::NK; ++i) {
            if (hs != 0 || g != 0) break;
            float x = sum[i];
            for (int k = 1; k < p.hs; ++k) x += sums[wave + k][16 * i + lane];
            if (!good[i]) continue;
            float *w = p.w + b * p.ld + key0 + 16 * i + lane;
            *w = p.decay == 0.0f ? x : __builtin_fmaf(p.decay, *w, x);
        }
        __syncthreads();  // the sums are read
    }
}

}  // namespace dsel
