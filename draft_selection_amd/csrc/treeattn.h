// Attention of a tree of drafted tokens over a paged cache.
//
//   z_ij = scale k_scale <q_i, K_j>  for every key j that node i sees,
//   o_i  = v_scale sum_j p_ij V_j,   p_i = softmax(z_i),   lse_i = ln sum_j e^z_ij,
// in one pass over the keys with the running maximum m and sum l of the
// softmax.  Node i of row b sees the row's s cached positions and the nodes
// whose bit is set in its mask row (no mask: nodes 0..i).
#pragma once

#include "cache.h"

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
};

// The simplest form: one wave per node and head; 64 keys at a time, one per
// lane for the products with q, then one after the other for the values.
template <bool E4M3>
__global__ __launch_bounds__(64) void tree_attn_simple_kernel(TreeAttnParams p) {
    __shared__ float qs[256], ps[64];
    __shared__ int64_t at[64];
    const int lane = threadIdx.x, h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    const int n = block_len_of(p.len, b, p.T);
    if (t >= n) return;
    const int s = seq_len_of(p.t, b, n, p.c.page_size);
    if (s < 0) return;
    const int hk = h / p.group;
    const uint16_t *q = (const uint16_t *)p.q + b * p.sqb + t * p.sqt + h * p.sqh;
    for (int e = lane; e < p.D; e += 64) qs[e] = __uint_as_float((uint32_t)q[e] << 16);
    const float ks = E4M3 && p.c.k_scale ? p.c.k_scale[hk] : 1.0f, vs = E4M3 && p.c.v_scale ? p.c.v_scale[hk] : 1.0f;
    float m = -__builtin_inff(), l = 0.0f, o[4] = {0, 0, 0, 0};
    const int total = s + n;
    auto value = [&](const char *row, int e) {
        if constexpr (E4M3) return __builtin_amdgcn_cvt_f32_fp8(((const uint8_t *)row)[e], 0);
        else return __uint_as_float((uint32_t)((const uint16_t *)row)[e] << 16);
    };
    for (int k0 = 0; k0 < total; k0 += 64) {
        const int k = k0 + lane;
        bool sees = k < total;
        if (sees && k >= s) {
            const int j = k - s;
            sees = p.mask ? (p.mask[((int64_t)b * p.T + t) * p.words + (j >> 5)] >> (j & 31)) & 1 : j <= t;
        }
        const int64_t a = sees ? place_of(p.c, p.t, b, k) : -1;
        sees = a >= 0;
        __syncthreads();
        at[lane] = a;
        float z = -__builtin_inff();
        if (sees) {
            const char *row = p.c.k + 16 * (a + hk * p.c.head_stride);
            float acc = 0.0f;
            for (int e = 0; e < p.D; ++e) acc += qs[e] * value(row, e);
            z = acc * p.scale * ks;
        }
        float mx = z;
        for (int x = 1; x < 64; x <<= 1) mx = fmaxf(mx, shfl_idxf(mx, lane ^ x));
        const float mn = fmaxf(m, mx), ms = mn == -__builtin_inff() ? 0.0f : mn;
        const float w = sees ? exp2f(z - ms) : 0.0f, alpha = exp2f(m - ms);
        ps[lane] = w;
        float sum = w;
        for (int x = 1; x < 64; x <<= 1) sum += shfl_idxf(sum, lane ^ x);
        l = l * alpha + sum;
        m = mn;
        __syncthreads();
        for (int i = 0; i < 4; ++i) o[i] *= alpha;
        for (int j = 0; j < 64; ++j) {
            if (at[j] < 0) continue;
            const char *row = p.c.v + 16 * (at[j] + hk * p.c.head_stride);
            for (int i = 0; i < 4; ++i)
                if (i * 64 + lane < p.D) o[i] += ps[j] * value(row, i * 64 + lane);
        }
    }
    const int64_t r = ((int64_t)b * p.T + t) * p.Hq + h;
    const float inv = l > 0.0f || l != l ? vs / l : 0.0f;
    for (int i = 0; i < 4; ++i)
        if (i * 64 + lane < p.D) {
            const __bf16 x = (__bf16)(o[i] * inv);
            p.out[r * p.D + i * 64 + lane] = __builtin_bit_cast(uint16_t, x);
        }
    if (p.lse && lane == 0) p.lse[r] = l > 0.0f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -__builtin_inff();
}

}  // namespace dsel
