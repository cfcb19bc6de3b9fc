// The paged K/V cache: rows appended, kept rows moved together, and the pool
// of pages behind it (reserve, fork, free).
//
// Position p of batch row b lies in page table[b][p / P], slot p % P.  A page
// is held by refcount[page] rows (0 = free).  Full pages may be shared; the
// page that holds the first position past a row's length never is, because a
// fork copies the partial last page.  So appending and compacting, which write
// only at or past the length, never touch a shared page.
//
// Every kernel here moves bytes and is bound by memory (or, at the small
// sizes of one step, by its launch): 16 bytes per lane and access, neighbouring
// lanes on neighbouring 16-byte vectors of a row.  Measured on an MI355X, 36
// layers of 8 heads of 128 in bf16 (medians of a kernel trace): 64 rows of up to 17
// tokens appended in 51 us (4.7 TB/s), their kept paths compacted in 13; four prompts of
// up to 2,048 tokens into 8 layers in 4 bits in 68 (4.0 TB/s); 48 forks
// of 8 layers, pages of 64 slots, in 24 us of copying (4.2 TB/s) and 12 of handing
// out pages.
#pragma once

#include "common.h"

namespace dsel {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kErrTree = 16, kErrSeqLen = 4, kErrPage = 8, kErrPool = 32;
constexpr int kMaxTree = 256;      // DSEL_MAX_TREE
constexpr int kMaxRows = 4096;     // DSEL_MAX_ROWS
constexpr int kAppendTokens = 64;  // tokens of one append workgroup

__device__ __forceinline__ void device_error(int bit) { atomicOr(&g_device_error, bit); }

// Geometry of a cache's K and V (the same for both); strides in 16-byte vectors
struct CacheView {
    char *k, *v;
    int layers, heads, vecs;  // vecs: 16-byte vectors of one head's row
    int64_t layer_stride, page_stride;
    int64_t slot_stride, head_stride;
    int64_t num_pages;
    int page_size;
    const float *k_scale, *v_scale;  // 8 bits: [layers, heads] or NULL (1)
    uint8_t *k_block, *v_block;      // 4 bits: the scale byte of vector i is byte i; NULL otherwise
};

struct TableView {
    const int32_t *table;
    int64_t ld;
    int max_pages;
    const int32_t *seq_len;
};

// Length of row b and the n positions past it that a call uses: -1 (and
// DSEL_DEVERR_SEQ_LEN) when they do not fit the table row.
__device__ __forceinline__ int seq_len_of(const TableView &t, int64_t b, int n, int page_size) {
    const int s = t.seq_len[b];
    if (s >= 0 && (int64_t)s + n <= (int64_t)t.max_pages * page_size) return s;
    device_error(kErrSeqLen);
    return -1;
}

// Vector offset of position p of row b in K or V (layer 0, head 0), -1 (and
// DSEL_DEVERR_PAGE) when its page id is out of range.  64-bit: a cache may
// hold more than 2^32 bytes.
__device__ __forceinline__ int64_t place_of(const CacheView &c, const TableView &t, int64_t b, int p) {
    const int page = t.table[b * t.ld + p / c.page_size];
    if (page < 0 || page >= c.num_pages) {
        device_error(kErrPage);
        return -1;
    }
    return (int64_t)page * c.page_stride + (int64_t)(p % c.page_size) * c.slot_stride;
}

// ---- append -----------------------------------------------------------------

struct AppendParams {
    CacheView c;
    TableView t;
    const char *k, *v;                 // new rows, bf16
    int64_t sl, sb, st, sh;            // strides of layer, batch, token, head in 8-element vectors
    int T;
    const int32_t *len;
};

// 8 bits of an e4m3 value x / s: the quotient is rounded to fp32 once, then to
// nearest even in e4m3 by the conversion instruction; values past the largest
// finite one (448) are held to it, NaN stays NaN.
__device__ __forceinline__ float clamp_e4m3(float x) { return x != x ? x : fminf(fmaxf(x, -448.0f), 448.0f); }

__device__ __forceinline__ u32x4 to_e4m3(const u32x4 &a, const u32x4 &b, float s) {
    u32x4 r;
    float x[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t wa = a[e >> 1], wb = b[e >> 1];
        x[e] = __uint_as_float((e & 1) ? (wa & 0xFFFF0000u) : (wa << 16));
        x[8 + e] = __uint_as_float((e & 1) ? (wb & 0xFFFF0000u) : (wb << 16));
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        int o = 0;
        o = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(x[4 * w] / s), clamp_e4m3(x[4 * w + 1] / s), o, false);
        o = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(x[4 * w + 2] / s), clamp_e4m3(x[4 * w + 3] / s), o, true);
        r[w] = (uint32_t)o;
    }
    return r;
}

// 32 values in 4 bits, and their scale byte.  The scale is the least power of two
// with max |x| <= 7 2^e: for max = 2^k m, 1 <= m < 2, that is 2^(k-2) if m <= 1.75,
// else 2^(k-1), and is read off the largest pattern.  x / 2^e is exact; the
// conversion instruction divides by the scale and rounds to nearest even, and holds
// to 6.  bf16 patterns without their sign order like the values.  Subnormal inputs,
// which are 0 under the least scale there is (they are below 2^-3 of it), are
// cleared: the instruction makes nonzero codes of some of them.
__device__ __forceinline__ uint32_t no_subnormals(uint32_t w) {
    if ((w & 0x7F800000u) == 0) w &= 0x8000FFFFu;
    if ((w & 0x7F80u) == 0) w &= 0xFFFF8000u;
    return w;
}
__device__ __forceinline__ u32x4 to_mxfp4(const u32x4 (&w)[4], uint8_t *scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = pk_max_i16(top, w[i][j] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    const bool none = top >= 0x7F80u;  // an infinity or NaN
    const int e = min(max((int)((top >> 7) + ((top & 0x7Fu) > 0x60u)) - 2, 4), 252);
    *scale = (uint8_t)(none ? 255 : e);
    const float s = __uint_as_float((uint32_t)e << 23);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t o = 0;
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, no_subnormals(w[i][0])), s, 0);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, no_subnormals(w[i][1])), s, 1);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, no_subnormals(w[i][2])), s, 2);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, no_subnormals(w[i][3])), s, 3);
        r[i] = none ? 0u : o;
    }
    return r;
}

// Workgroup (x, y, z): tokens [64 x, 64 x + 64) of batch row z, layer y / 2, K
// or V by y % 2.  Of the cache's type.
enum CacheType { kBf16, kE4m3, kMxfp4 };
template <CacheType F>
__global__ __launch_bounds__(256) void cache_append_kernel(AppendParams p) {
    __shared__ int64_t place[kAppendTokens];
    const int b = blockIdx.z, layer = blockIdx.y >> 1, isv = blockIdx.y & 1;
    const int n = block_len_of(p.len, b, p.T);
    const int t0 = blockIdx.x * kAppendTokens;
    if (t0 >= n) return;
    const int s = seq_len_of(p.t, b, n, p.c.page_size);
    if (s < 0) return;
    const int m = min(n - t0, kAppendTokens);
    if ((int)threadIdx.x < m) place[threadIdx.x] = place_of(p.c, p.t, b, s + t0 + threadIdx.x);
    __syncthreads();
    const uint32_t vecs = p.c.vecs, cols = vecs * p.c.heads;
    u32x4 *dst = (u32x4 *)(isv ? p.c.v : p.c.k) + layer * p.c.layer_stride;
    const u32x4 *src = (const u32x4 *)(isv ? p.v : p.k) + layer * p.sl + b * p.sb + t0 * p.st;
    const float *scale = isv ? p.c.v_scale : p.c.k_scale;
    for (uint32_t i = threadIdx.x; i < m * cols; i += 256) {
        const uint32_t t = i / cols, col = i - t * cols, h = col / vecs, e = col - h * vecs;
        if (place[t] < 0) continue;
        const u32x4 *x = src + t * p.st + h * p.sh + (F == kMxfp4 ? 4 * e : F == kE4m3 ? 2 * e : e);
        const int64_t at = place[t] + h * p.c.head_stride + e;
        u32x4 w = x[0];
        if constexpr (F == kE4m3) w = to_e4m3(w, x[1], scale ? scale[layer * p.c.heads + h] : 1.0f);
        if constexpr (F == kMxfp4) {
            const u32x4 all[4] = {w, x[1], x[2], x[3]};
            w = to_mxfp4(all, (isv ? p.c.v_block : p.c.k_block) + layer * p.c.layer_stride + at);
        }
        dst[at] = w;
    }
}

// ---- compact ----------------------------------------------------------------

struct CompactParams {
    CacheView c;
    TableView t;
    const int32_t *path, *n_keep;
    int32_t *new_len;
    int T;
    int kinds;  // 2: K and V; 1: one array is both, and moves once
};

// Rows s + path[i] move to s + i.  path ascends, so path[i] >= i and a row
// still to be read is never one already written: each thread owns one 16-byte
// column of one layer's K or V and goes through the list in order, eight rows
// loaded before the first of them is stored.
__global__ __launch_bounds__(256) void cache_compact_kernel(CompactParams p) {
    __shared__ int64_t from[kMaxTree], to[kMaxTree];
    __shared__ int bad_path, bad_page;
    const int b = blockIdx.y, tid = threadIdx.x;
    const int n = p.n_keep[b];
    if (tid == 0) bad_path = bad_page = 0;
    __syncthreads();
    const bool fits = n >= 0 && n <= p.T;
    int s = -1;
    if (!fits) device_error(kErrTree);
    else if (n > 0) {
        int last = 0;  // the list ascends if every neighbouring pair does
        if (tid < n) {
            last = p.path[(int64_t)b * p.T + tid];
            const int before = tid ? p.path[(int64_t)b * p.T + tid - 1] : -1;
            if (last <= before || last >= p.T) bad_path = 1;
        }
        __syncthreads();
        if (!bad_path) {
            s = seq_len_of(p.t, b, p.path[(int64_t)b * p.T + n - 1] + 1, p.c.page_size);
            if (s >= 0 && tid < n) {
                from[tid] = place_of(p.c, p.t, b, s + last);
                to[tid] = place_of(p.c, p.t, b, s + tid);
                if (from[tid] < 0 || to[tid] < 0) bad_page = 1;
            }
            __syncthreads();
        }
        if (bad_path && tid == 0) device_error(kErrTree);
    }
    const bool move = fits && n > 0 && s >= 0 && !bad_path && !bad_page;
    if (blockIdx.x == 0 && tid == 0) p.new_len[b] = p.t.seq_len[b] + (move ? n : 0);
    if (!move) return;
    const uint32_t vecs = p.c.vecs, cols = vecs * p.c.heads;
    const uint32_t i = blockIdx.x * 256 + tid;
    const uint32_t lk = i / cols;
    if (lk >= (uint32_t)(p.kinds * p.c.layers)) return;
    const uint32_t col = i - lk * cols, h = col / vecs, both = p.kinds - 1;
    const int64_t at = (lk >> both) * p.c.layer_stride + h * p.c.head_stride + (col - h * vecs);
    u32x4 *x = (u32x4 *)(lk & both ? p.c.v : p.c.k) + at;
    uint8_t *y = lk & both ? p.c.v_block : p.c.k_block;  // 4 bits: a vector's scale byte goes with it
    if (y) y += at;
    for (int k = 0; k < n; k += 8) {
        u32x4 w[8];
        uint8_t s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < n) w[e] = x[from[k + e]];
        if (y) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < n) s[e] = y[from[k + e]];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < n && from[k + e] != to[k + e]) x[to[k + e]] = w[e];
        if (y) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < n && from[k + e] != to[k + e]) y[to[k + e]] = s[e];
        }
    }
}

// ---- the pool ---------------------------------------------------------------

struct PoolParams {
    int32_t *table;
    int64_t ld;
    int rows, max_pages;
    int32_t *row_pages, *seq_len, *refcount;
    int64_t num_pages;
    int page_size;
    const int32_t *arg;  // which / src / extra / pages wanted, one per row
    int32_t *granted;    // out [1]
    int32_t *plan;       // fork: workspace [rows]; cut: [rows][max_pages]
};

// Exclusive prefix sum of one value per thread over a workgroup of 1024;
// *total gets the sum.  `part` is LDS scratch of 17 words.
__device__ __forceinline__ int block_scan1024(int x, int *part, int *total) {
    const int tid = threadIdx.x;
    const int incl = wave_incl_scan(x);
    __syncthreads();
    if ((tid & 63) == 63) part[tid >> 6] = incl;
    __syncthreads();
    if (tid < 64) {
        const int w = tid < 16 ? part[tid] : 0;
        const int wi = wave_incl_scan(w);
        if (tid < 16) part[tid] = wi - w;
        if (tid == 15) part[16] = wi;
    }
    __syncthreads();
    *total = part[16];
    return part[tid >> 6] + incl - x;
}

// The free pages among the 16 from `first` on, as bits.
__device__ __forceinline__ uint32_t free_bits(const PoolParams &p, int64_t first) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (first + i < p.num_pages && p.refcount[first + i] == 0) m |= 1u << i;
    return m;
}

// One workgroup hands out pages: need[r] of them to row r, the lowest free
// pages in row order, if the pool holds enough for every row; else none.
// The pool is the refcount array itself (a page is free when its count is 0),
// so no list has to be kept in step with it and the pages handed out depend on
// nothing but the counts.  16 pages per thread and 16,384 per pass; 6 to 12 us,
// a few dependent loads and prefix sums in one workgroup.
// kFork: the one page of row r goes to plan[r]; kCut: row r's arg[r] pages (none
// if that is negative) go to its row of plan, beside those that it still holds;
// kMore: the pages follow those that the row holds already.
enum PoolGive { kMore, kFork, kCut };
template <PoolGive G>
__global__ __launch_bounds__(1024) void pool_give_kernel(PoolParams p) {
    __shared__ int start[kMaxRows], held[kMaxRows];
    __shared__ int part[17], over;
    __shared__ unsigned long long wanted;
    constexpr bool FORK = G == kFork;
    const int tid = threadIdx.x;
    if (tid == 0) {
        over = 0;
        wanted = 0;
    }
    __syncthreads();
    constexpr int R = kMaxRows / 1024;
    constexpr int64_t kPass = 1024 * 16;
    uint32_t bits = free_bits(p, tid * 16);  // the first pass's loads fly beside the rows'
    int need[R], code[R];
    // What all rows want is counted in 32 bits where that cannot overflow (1,024
    // rows of at most 2^20 pages a scan), else also in 64.
    const bool large = p.num_pages > (1 << 20);
    int64_t all = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        need[i] = 0;
        code[i] = -2;
        if (i * 1024 >= p.rows) continue;  // (the same for all threads)
        const int r = i * 1024 + tid;
        if (r < p.rows) {
            const int have = p.row_pages[r], a = p.arg[r];
            held[r] = have;
            bool bad = false;
            if constexpr (G == kCut) {
                need[i] = max(a, 0);
            } else if constexpr (FORK) {
                if (a != -1) {
                    bad = a < 0 || a >= p.rows || a == r || have != 0;
                    if (!bad) {
                        const int n = p.seq_len[a], h = p.row_pages[a];
                        bad = p.arg[a] != -1 || n < 0 || h > p.max_pages || (int64_t)n > (int64_t)h * p.page_size;
                        need[i] = !bad && n % p.page_size ? 1 : 0;
                        code[i] = bad ? -2 : -1;
                    }
                }
            } else {
                const int n = p.seq_len[r];
                bad = n < 0 || a < 0 || have < 0 || have > p.max_pages;
                if (!bad) {
                    const uint32_t keys = (uint32_t)n + (uint32_t)a, pages = keys / (uint32_t)p.page_size +
                                                                             (keys % (uint32_t)p.page_size != 0);
                    bad = pages > (uint32_t)p.max_pages;
                    if (!bad) need[i] = (int)pages > have ? (int)pages - have : 0;
                }
            }
            if (bad) device_error(kErrSeqLen);
            if (need[i] > p.num_pages) over = 1;
            if (large && need[i]) atomicAdd(&wanted, (unsigned long long)need[i]);
        }
        int here;
        const int at = block_scan1024(need[i], part, &here);
        if (r < p.rows) start[r] = (int)all + at;
        all += here;
    }
    __syncthreads();
    // more pages than the pool has, and 32 bits may count, are more than it holds
    const bool many = over || (large ? wanted > (unsigned long long)p.num_pages : all > p.num_pages);
    const int total = (int)all;
    // does the pool hold enough?  (a pool of one pass is looked at once, below)
    const bool one = p.num_pages <= kPass;
    int found = 0;
    int rank = 0;
    for (int64_t base = 0; !many && base < p.num_pages && found < total; base += kPass) {
        if (base) bits = free_bits(p, base + tid * 16);
        int here;
        rank = block_scan1024(__builtin_popcount(bits), part, &here);
        found += here;
    }
    const bool ok = !many && found >= total;
    if (tid == 0) {
        p.granted[0] = ok;
        if (!ok) device_error(kErrPool);
    }
    __syncthreads();  // start[] and held[] are whole
    if (ok && total > 0) {
        int given = 0;
        for (int64_t base = 0; given < total; base += kPass) {
            if (!one) {
                int here;
                bits = free_bits(p, base + tid * 16);
                rank = given + block_scan1024(__builtin_popcount(bits), part, &here);
                given += here;
            } else {
                given = total;
            }
            for (uint32_t m = bits; m && rank < total; m &= m - 1, ++rank) {
                const int page = (int)(base + tid * 16 + __builtin_ctz(m));
                int lo = 0, hi = p.rows - 1;  // the last row whose pages start at or before `rank`
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (start[mid] <= rank) lo = mid;
                    else hi = mid - 1;
                }
                if constexpr (FORK) p.plan[lo] = page;
                else if constexpr (G == kCut) p.plan[(int64_t)lo * p.max_pages + (rank - start[lo])] = page;
                else p.table[lo * p.ld + held[lo] + (rank - start[lo])] = page;
                p.refcount[page] = 1;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = i * 1024 + tid;
        if (r >= p.rows) continue;
        if constexpr (FORK) {
            if (!ok) p.plan[r] = -2;
            else if (!need[i]) p.plan[r] = code[i];
        } else if (G == kMore && ok && need[i]) {
            p.row_pages[r] = held[r] + need[i];
        }
    }
}

// fork, after pool_give_kernel<kFork>.  Workgroup (0, r): row r's table entries
// and counts; workgroup (1 + u, r): 16 slots of the partial last page, of one
// layer's K or V.  A source row is never itself a fork's target, so nothing
// read here is written here.
constexpr int kForkSlots = 16;
__global__ __launch_bounds__(256) void pages_fork_kernel(PoolParams p, CacheView c) {
    const int r = blockIdx.y, tid = threadIdx.x;
    const int fresh = p.plan[r];
    if (fresh < -1) return;
    const int s = p.arg[r], n = p.seq_len[s];
    const int whole = n / p.page_size, rest = n % p.page_size;
    const int32_t *from = p.table + s * p.ld;
    if (blockIdx.x == 0) {
        int32_t *to = p.table + r * p.ld;
        for (int i = tid; i < whole; i += 256) {
            const int page = from[i];
            to[i] = page;
            if (page >= 0 && page < p.num_pages) atomicAdd(&p.refcount[page], 1);
            else device_error(kErrPage);
        }
        if (tid == 0) {
            if (rest) {
                // with no page to copy, its id is taken along and the new page goes back
                const int page = from[whole];
                const bool good = page >= 0 && page < p.num_pages;
                to[whole] = good ? fresh : page;
                if (!good) p.refcount[fresh] = 0;
            }
            p.row_pages[r] = whole + (rest ? 1 : 0);
            p.seq_len[r] = n;
        }
        return;
    }
    if (!rest) return;
    const int chunks = (c.page_size + kForkSlots - 1) / kForkSlots;
    const int u = blockIdx.x - 1, lk = u / chunks, first = (u - lk * chunks) * kForkSlots;
    const int m = min(rest - first, kForkSlots);
    if (m <= 0) return;
    const int page = from[whole];
    if (page < 0 || page >= c.num_pages) {
        if (tid == 0) device_error(kErrPage);
        return;
    }
    const int64_t base = (lk >> 1) * c.layer_stride + first * c.slot_stride;
    u32x4 *x = (u32x4 *)(lk & 1 ? c.v : c.k) + base;
    uint8_t *y = lk & 1 ? c.v_block : c.k_block;  // 4 bits: the vectors' scale bytes
    if (y) y += base;
    const u32x4 *src = x + page * c.page_stride;
    u32x4 *dst = x + fresh * c.page_stride;
    const uint32_t vecs = c.vecs, cols = vecs * c.heads;
    for (uint32_t i = tid; i < m * cols; i += 256) {
        const uint32_t t = i / cols, col = i - t * cols, h = col / vecs;
        const int64_t o = t * c.slot_stride + h * c.head_stride + (col - h * vecs);
        dst[o] = src[o];
        if (y) y[fresh * c.page_stride + o] = y[page * c.page_stride + o];
    }
}

// free: one workgroup per row gives back what a marked row holds.  Counts only
// go down by atomic adds, whose order does not matter.
__global__ __launch_bounds__(256) void pages_free_kernel(PoolParams p) {
    const int r = blockIdx.x, tid = threadIdx.x;
    if (p.arg[r] == 0) return;
    const int n = p.row_pages[r];
    const bool ok = n >= 0 && n <= p.max_pages;
    if (!ok) {
        if (tid == 0) device_error(kErrSeqLen);
        return;
    }
    int32_t *t = p.table + r * p.ld;
    for (int i = tid; i < n; i += 256) {
        const int page = t[i];
        t[i] = -1;
        bool good = page >= 0 && page < p.num_pages;
        if (good && atomicSub(&p.refcount[page], 1) <= 0) {
            atomicAdd(&p.refcount[page], 1);
            good = false;
        }
        if (!good) device_error(kErrPage);
    }
    __syncthreads();  // every thread has read row_pages
    if (tid == 0) {
        p.row_pages[r] = 0;
        p.seq_len[r] = 0;
    }
}

}  // namespace dsel
