// Rows of the pool cut down to the positions of most weight.
//
// Four launches: the positions that every row keeps and the pages it needs for
// them (one workgroup a row), the pages handed out (pool_give_kernel), the kept
// rows copied in every layer, and the pool brought up to date.  The copies go to
// fresh pages, so a page that another row holds too is only read, and every row is
// copied by as many workgroups as it takes, in no order.  The copy is bound by
// memory and is nearly all of the time where there are many layers.  Measured on an
// MI355X, 8 heads of 128 in bf16, kernel by kernel: 16 rows of 1,024 to 4,096 positions
// cut to 1,500 in eight layers 280 us of copying (4.9 TB/s), 15 the plan, 10 the pages, 5
// the end; two rows of 550 and 1,100 cut to 512 in one layer 6, 9, 6 and 3.  Captured,
// the four together: 312 and 28 us; two rows of 120,000 to 60,000 in one layer 461 (the
// plan reads the weights of a row past 16,384 again in every pass).
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
    // what the launches hand on
    int32_t *need;   // [rows]: pages that the row's kept positions take, -1: it stays as it is
    int32_t *len;    // [rows]: its length before
    int32_t *list;   // [rows][list_ld]: the kept positions
    int64_t list_ld;
    float *moved;    // [rows][max_len]: their weights
    int64_t moved_ld;
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
// lists the positions of a run of its own.  A row of up to 16,384 positions is read
// once, into registers.  Weights crowd into few digits (their exponents, above all):
// every wave counts in two histograms of its own, for even and odd lanes.
constexpr int kEvictHeld = 16;
__global__ __launch_bounds__(1024) void evict_plan_kernel(EvictParams p) {
    __shared__ int hist[32][256];
    __shared__ int part[17], bad;
    __shared__ uint32_t found[3];
    const int r = blockIdx.x, tid = threadIdx.x;
    int *const mine = hist[(tid >> 6) * 2 + (tid & 1)];
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
    if (tid == 0) {
        p.need[r] = (int)(((int64_t)K + P - 1) / P);
        p.len[r] = n;
    }
    const float *w = p.weights + r * p.ld;
    const int lo = p.sinks, hi = n - p.recent;
    int m = K - p.sinks - p.recent;
    // position tid + 1024 i, in the order of weights
    const bool held_all = n <= kEvictHeld * 1024;
    uint32_t x[kEvictHeld];
    if (held_all) {
#pragma unroll
        for (int i = 0; i < kEvictHeld; ++i) x[i] = tid + 1024 * i < n ? order_bits(w[tid + 1024 * i]) : 0u;
    }
    uint32_t key = 0, mask = 0;  // the digits of the m-th largest found so far
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 32 * 256; i += 1024) hist[0][i] = 0;
        __syncthreads();
        if (held_all) {
#pragma unroll
            for (int i = 0; i < kEvictHeld; ++i) {
                const int at = tid + 1024 * i;
                if (at >= lo && at < hi && (x[i] & mask) == key) atomicAdd(&mine[x[i] >> shift & 255], 1);
            }
        } else {
            for (int i = lo + tid; i < hi; i += 1024) {
                const uint32_t y = order_bits(w[i]);
                if ((y & mask) == key) atomicAdd(&mine[y >> shift & 255], 1);
            }
        }
        __syncthreads();
        int count = 0;
        if (tid < 256) {  // from the largest digit down
#pragma unroll
            for (int i = 0; i < 32; ++i) count += hist[i][255 - tid];
        }
        int all;
        const int above = block_scan1024(count, part, &all);
        if (tid < 256 && above < m && above + count >= m) {
            found[0] = 255 - tid;
            found[1] = above;
            found[2] = above + count == m;
        }
        if (tid == 0 && m == 0) {
            found[0] = 255;
            found[1] = found[2] = 0;
        }
        __syncthreads();
        key |= found[0] << shift;
        mask |= 255u << shift;
        m -= (int)found[1];
        const bool all_kept = found[2] && key;
        __syncthreads();
        if (all_kept) {  // every weight with these digits: no more are needed, and no ties
            --key;
            m = 0;
            break;
        }
    }
    // m of those that equal the key are kept, the first ones
    int32_t *list = p.list + r * p.list_ld;
    if (held_all) {
        // 1,024 positions after each other at a time
        int at = 0, ties = 0;
#pragma unroll
        for (int i = 0; i < kEvictHeld; ++i) {
            if (1024 * i >= n) break;
            const int pos = tid + 1024 * i;
            const bool fixed = pos < n && (pos < lo || pos >= hi), in = pos >= lo && pos < hi;
            const bool tie = in && x[i] == key;
            int all, ties_all;
            const int before = block_scan1024((fixed || (in && x[i] > key)) | (int)tie << 16, part, &all);
            const int tie_at = ties + (before >> 16);
            ties_all = all >> 16;
            const int take = min(max(m - ties, 0), before >> 16);  // ties taken before this one, of these
            if (fixed || (in && x[i] > key) || (tie && tie_at < m)) list[at + (before & 0xFFFF) + take] = pos;
            at += (all & 0xFFFF) + min(max(m - ties, 0), ties_all);
            ties += ties_all;
        }
        return;
    }
    const int each = (n + 1023) / 1024, i0 = min(tid * each, n), i1 = min(i0 + each, n);
    int2 own = {0, 0};  // always or surely kept, equal to the key
    for (int i = i0; i < i1; ++i) {
        const bool fixed = i < lo || i >= hi;
        const uint32_t y = order_bits(w[i]);
        own.x += fixed || y > key;
        own.y += !fixed && y == key;
    }
    const int2 before = block_scan1024x2(own, part);
    int at = before.x + min(before.y, m), ties = before.y;
    for (int i = i0; i < i1; ++i) {
        const bool fixed = i < lo || i >= hi;
        const uint32_t y = order_bits(w[i]);
        const bool tie = !fixed && y == key;
        if (fixed || y > key || (tie && ties < m)) list[at++] = i;
        ties += tie;
    }
}

// Workgroup (x, y, z): every gridDim.x-th run of 16 kept positions of row z, in one
// layer's K or V, eight vectors of a thread loaded before the first is stored (runs of
// 64, vector by vector: 14 us instead of 6 where there is one layer); the last y: their
// weights.
constexpr int kEvictRows = 16;
__global__ __launch_bounds__(256) void evict_copy_kernel(EvictParams p) {
    __shared__ int64_t from[kEvictRows], to[kEvictRows];
    const int r = blockIdx.z, tid = threadIdx.x;
    if (p.need[r] <= 0 || p.g.granted[0] == 0) return;
    const int K = p.budget[r], P = p.g.page_size;
    if (blockIdx.y == gridDim.y - 1) {
        const float *w = p.weights + r * p.ld;
        for (int64_t i = (int64_t)blockIdx.x * 256 + tid; i < K; i += (int64_t)gridDim.x * 256)
            p.moved[r * p.moved_ld + i] = w[p.list[r * p.list_ld + i]];
        return;
    }
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
        constexpr int N = 8;
        for (uint32_t i0 = tid; i0 < m * cols; i0 += 256 * N) {
            u32x4 v[N];
            uint8_t e[N];
            int64_t go[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint32_t i = i0 + 256 * n;
                if (i >= m * cols) continue;
                const uint32_t t = i / cols, col = i - t * cols, h = col / vecs;
                const int64_t o = h * p.c.head_stride + (col - h * vecs);
                go[n] = to[t] + o;
                v[n] = x[from[t] + o];
                if (y) e[n] = y[from[t] + o];
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (i0 + 256 * n >= m * cols) continue;
                x[go[n]] = v[n];
                if (y) y[go[n]] = e[n];
            }
        }
        __syncthreads();  // the places are read
    }
}

// Workgroup (0, r): row r's old pages given back and its new entries; workgroup (1 +
// i, r): a part of its weights written back, 0 behind them.  Nothing that another
// workgroup changes is read: lengths come from `len`.
constexpr int kEvictParts = 8;
__global__ __launch_bounds__(1024) void evict_finish_kernel(EvictParams p) {
    const int r = blockIdx.y, tid = threadIdx.x;
    const int need = p.need[r];
    if (need < 0 || p.g.granted[0] == 0) return;
    const int K = p.budget[r], n = p.len[r];
    if (blockIdx.x > 0) {
        float *w = p.weights + r * p.ld;
        for (int i = (blockIdx.x - 1) * 1024 + tid; i < n; i += kEvictParts * 1024)
            w[i] = i < K ? p.moved[r * p.moved_ld + i] : 0.0f;
        return;
    }
    const int held = p.g.row_pages[r];
    int32_t *table = p.g.table + r * p.g.ld;
    for (int i = tid; i < held; i += 1024) {
        const int page = table[i];
        if (atomicSub(&p.g.refcount[page], 1) <= 0) {
            atomicAdd(&p.g.refcount[page], 1);
            device_error(kErrPage);
        }
        table[i] = i < need ? p.g.plan[(int64_t)r * p.g.max_pages + i] : -1;
    }
    __syncthreads();  // every thread has read row_pages
    if (tid == 0) {
        p.g.row_pages[r] = need;
        p.g.seq_len[r] = K;
    }
}

}  // namespace dsel
