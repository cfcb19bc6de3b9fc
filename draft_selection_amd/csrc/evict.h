// Rows of the pool cut down to the positions of most weight.
//
// Four launches: the positions that every row keeps and the pages it needs for
// them (one workgroup a row), the pages handed out (pool_give_kernel), the kept
// rows copied in every layer, and the pool brought up to date.  The copies go to
// fresh pages, so a page that another row holds too is only read, and every row is
// copied by as many workgroups as it takes, in no order.  The copy is bound by
// memory and is nearly all of the time where there are many layers.
#pragma once

#include "cache.h"

namespace dsel {

struct EvictParams {
    PoolParams g;
    CacheView c;
    const int32_t *budget;
    float *weights;
    int64_t ld;
    int sinks, recent;
    int32_t *need;   // [rows]: pages that the row's kept positions take, -1: it stays as it is
    int32_t *list;   // [rows][list_ld]: the kept positions
    int64_t list_ld;
    int kinds;       // 2: K and V; 1: one array is both
};

// Exclusive prefix sums of two values per thread over a workgroup of 1024.
__device__ __forceinline__ int2 block_scan1024x2(int2 v, int *part) {
    int t;
    int2 r;
    r.x = block_scan1024(v.x, part, &t);
    r.y = block_scan1024(v.y, part, &t);
    return r;
}

// The m largest of the weights of positions [lo, hi), m < hi - lo: four passes
// over 8 bits each of their order find the m-th largest, then a thread counts and
// lists the positions of a run of its own.
__global__ __launch_bounds__(1024) void evict_plan_kernel(EvictParams p) {
    __shared__ int hist[16][256];
    __shared__ int part[17], bad;
    __shared__ uint32_t found[2];
    const int r = blockIdx.x, tid = threadIdx.x, wave = tid >> 6;
    const int K = p.budget[r], n = p.g.seq_len[r];
    if (K < 0 || K >= n) {
        if (tid == 0) p.need[r] = -1;
        return;
    }
    const int P = p.g.page_size, held = p.g.row_pages[r];
    if ((int64_t)p.sinks + p.recent > K || held < 0 || held > p.g.max_pages || (int64_t)held * P < n) {
        if (tid == 0) {
            p.need[r] = -1;
            device_error(kErrSeqLen);
        }
        return;
    }
    if (tid == 0) bad = 0;
    __syncthreads();
    for (int i = tid; i < held; i += 1024) {
        const int page = p.g.table[r * p.g.ld + i];
        if (page < 0 || page >= p.g.num_pages) bad = 1;
    }
    __syncthreads();
    if (bad) {
        if (tid == 0) {
            p.need[r] = -1;
            device_error(kErrPage);
        }
        return;
    }
    if (tid == 0) p.need[r] = (int)(((int64_t)K + P - 1) / P);
    const float *w = p.weights + r * p.ld;
    const int lo = p.sinks, hi = n - p.recent;
    int m = K - p.sinks - p.recent;
    uint32_t key = 0, mask = 0;  // the digits of the m-th largest found so far
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 16 * 256; i += 1024) hist[0][i] = 0;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += 1024) {
            const uint32_t x = order_bits(w[i]);
            if ((x & mask) == key) atomicAdd(&hist[wave][x >> shift & 255], 1);
        }
        __syncthreads();
        int count = 0;
        if (tid < 256)
            for (int i = 0; i < 16; ++i) count += hist[i][255 - tid];  // from the largest digit down
        int all;
        const int above = block_scan1024(count, part, &all);
        if (tid < 256 && above < m && above + count >= m) {
            found[0] = 255 - tid;
            found[1] = above;
        }
        if (tid == 0 && m == 0) {
            found[0] = 255;
            found[1] = 0;
        }
        __syncthreads();
        key |= found[0] << shift;
        mask |= 255u << shift;
        m -= (int)found[1];
        __syncthreads();
    }
    // m of those that equal the key are kept, the first ones
    const int each = (n + 1023) / 1024, i0 = min(tid * each, n), i1 = min(i0 + each, n);
    int2 mine = {0, 0};  // always or surely kept, equal to the key
    for (int i = i0; i < i1; ++i) {
        const bool fixed = i < lo || i >= hi;
        const uint32_t x = order_bits(w[i]);
        mine.x += fixed || x > key;
        mine.y += !fixed && x == key;
    }
    const int2 before = block_scan1024x2(mine, part);
    int at = before.x + min(before.y, m), ties = before.y;
    int32_t *list = p.list + r * p.list_ld;
    for (int i = i0; i < i1; ++i) {
        const bool fixed = i < lo || i >= hi;
        const uint32_t x = order_bits(w[i]);
        const bool tie = !fixed && x == key;
        if (fixed || x > key || (tie && ties < m)) list[at++] = i;
        ties += tie;
    }
}

// Workgroup (x, y, z): every gridDim.x-th run of 64 kept positions of row z, in one
// layer's K or V.
constexpr int kEvictRows = 64;
__global__ __launch_bounds__(256) void evict_copy_kernel(EvictParams p) {
    __shared__ int64_t from[kEvictRows], to[kEvictRows];
    const int r = blockIdx.z, tid = threadIdx.x;
    if (p.need[r] <= 0 || p.g.granted[0] == 0) return;
    const int K = p.budget[r], P = p.g.page_size;
    const uint32_t lk = blockIdx.y, both = p.kinds - 1;
    const int64_t base = (lk >> both) * p.c.layer_stride;
    u32x4 *x = (u32x4 *)(lk & both ? p.c.v : p.c.k) + base;
    uint8_t *y = lk & both ? p.c.v_block : p.c.k_block;
    if (y) y += base;
    const uint32_t vecs = p.c.vecs, cols = vecs * p.c.heads;
    for (int64_t first = (int64_t)blockIdx.x * kEvictRows; first < K; first += (int64_t)gridDim.x * kEvictRows) {
        const int m = (int)min(K - first, (int64_t)kEvictRows);
        if (tid < m) {
            const int i = (int)first + tid, s = p.list[r * p.list_ld + i];
            from[tid] = p.g.table[r * p.g.ld + s / P] * p.c.page_stride + s % P * p.c.slot_stride;
            to[tid] = p.g.plan[(int64_t)r * p.g.max_pages + i / P] * p.c.page_stride + i % P * p.c.slot_stride;
        }
        __syncthreads();
        for (uint32_t i = tid; i < m * cols; i += 256) {
            const uint32_t t = i / cols, col = i - t * cols, h = col / vecs;
            const int64_t o = h * p.c.head_stride + (col - h * vecs);
            x[to[t] + o] = x[from[t] + o];
            if (y) y[to[t] + o] = y[from[t] + o];
        }
        __syncthreads();  // the places are read
    }
}

// One workgroup a row: old pages given back, the row's new entries, its weights
// moved.  list[i] >= i, so a chunk's weights are read before any of them, and
// after none of the later ones, is written.
__global__ __launch_bounds__(1024) void evict_finish_kernel(EvictParams p) {
    const int r = blockIdx.x, tid = threadIdx.x;
    const int need = p.need[r];
    if (need < 0 || p.g.granted[0] == 0) return;
    const int K = p.budget[r], n = p.g.seq_len[r], held = p.g.row_pages[r];
    int32_t *table = p.g.table + r * p.g.ld;
    for (int i = tid; i < held; i += 1024) {
        const int page = table[i];
        if (atomicSub(&p.g.refcount[page], 1) <= 0) {
            atomicAdd(&p.g.refcount[page], 1);
            device_error(kErrPage);
        }
        table[i] = i < need ? p.g.plan[(int64_t)r * p.g.max_pages + i] : -1;
    }
    float *w = p.weights + r * p.ld;
    const int32_t *list = p.list + r * p.list_ld;
    for (int i0 = 0; i0 < n; i0 += 1024) {
        const int i = i0 + tid;
        const float x = i < K ? w[list[i]] : 0.0f;
        __syncthreads();
        if (i < n) w[i] = x;
    }
    __syncthreads();  // every thread has read row_pages and seq_len
    if (tid == 0) {
        p.g.row_pages[r] = need;
        p.g.seq_len[r] = K;
    }
}

}  // namespace dsel
