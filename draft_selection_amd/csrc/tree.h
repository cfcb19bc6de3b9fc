// Trees of drafted tokens: ancestor masks, depths, and the path that the
// target keeps.  Node 0 is the last verified token; 0 <= parent[i] < i.
#pragma once

#include "cache.h"

namespace dsel {

struct TreeParams {
    const int32_t *parent, *tok, *target;
    int64_t target_stride;
    int T;
    const int32_t *len;
    int32_t *mask, *depth;           // tree_mask
    int32_t *n_keep, *path, *out_tok;  // tree_accept
};

// Row i of the mask holds i and every node above it.  One thread per node, and
// links that double: after step k a node's words hold its nearest 2^k nodes
// upwards and `up` is the node 2^k levels above, whose words and link it then
// takes over, so a tree of 256 is done in 8 steps.  A link that goes to no
// earlier node ends its chain.  7 us for 256 trees of 256 (climbing link by
// link: 10), 3 for one of 60: the launch and one load's latency.
__global__ __launch_bounds__(kMaxTree) void tree_mask_kernel(TreeParams p) {
    constexpr int W = kMaxTree / 32, S = W + 1;  // an odd stride spreads the rows over the banks
    __shared__ int up[kMaxTree], height[kMaxTree];
    __shared__ uint32_t bits[kMaxTree * S];
    const int b = blockIdx.x, i = threadIdx.x, words = (p.T + 31) / 32;
    const int n = block_len_of(p.len, b, p.T);
    int a = -1, d = 0;
    uint32_t own[W];
#pragma unroll
    for (int w = 0; w < W; ++w) own[w] = (i >> 5) == w ? 1u << (i & 31) : 0u;
    if (i < n) {
        a = p.parent[(int64_t)b * p.T + i];
        if (i == 0 ? a != -1 : (a < 0 || a >= i)) {
            device_error(kErrTree);
            a = -1;
        }
        d = a >= 0;
    }
    for (int reach = 1; reach < n; reach *= 2) {
        up[i] = a;
        height[i] = d;
#pragma unroll
        for (int w = 0; w < W; ++w)
            if (w < words) bits[i * S + w] = own[w];
        __syncthreads();
        if (a >= 0) {
            // a node whose chain has ended keeps its height: it is the root's distance
#pragma unroll
            for (int w = 0; w < W; ++w)
                if (w < words) own[w] |= bits[a * S + w];
            d += height[a];
            a = up[a];
        }
        __syncthreads();
    }
    if (i < n && p.depth) p.depth[(int64_t)b * p.T + i] = d;
#pragma unroll
    for (int w = 0; w < W; ++w)
        if (w < words) bits[i * S + w] = own[w];
    __syncthreads();
    int32_t *m = p.mask + (int64_t)b * p.T * words;
    for (int e = i; e < n * words; e += blockDim.x) m[e] = (int32_t)bits[(e / words) * S + e % words];
}

// One wave per tree: the nodes' parents and tokens stay in registers, four per
// lane, and each step is a compare and a ballot per 64 nodes.  A child lies
// after its parent, so the walk ends.  Latency bounds it: 2 us for one tree of
// 60, 6 for 256 of 256.
__global__ __launch_bounds__(64) void tree_accept_kernel(TreeParams p) {
    const int b = blockIdx.x, lane = threadIdx.x;
    const int n = block_len_of(p.len, b, p.T);
    const int64_t base = (int64_t)b * p.T;
    constexpr int Q = kMaxTree / 64;
    int up[Q], tok[Q], want[Q], path[Q], out[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int i = q * 64 + lane;
        const bool in = i < n;
        up[q] = in ? p.parent[base + i] : -1;
        tok[q] = in ? p.tok[base + i] : 0;
        want[q] = in ? p.target[(base + i) * p.target_stride] : 0;
        if (in && (i == 0 ? up[q] != -1 : (up[q] < 0 || up[q] >= i))) {
            device_error(kErrTree);
            up[q] = -1;
        }
        if (i == 0) up[q] = -1;
        path[q] = out[q] = -1;
    }
    int cur = n > 0 ? 0 : -1, kept = 0;
    while (cur >= 0) {
        int w = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if ((cur >> 6) == q) w = __builtin_amdgcn_readlane(want[q], cur & 63);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if ((kept >> 6) == q && lane == (kept & 63)) {
                path[q] = cur;
                out[q] = w;
            }
        ++kept;
        int next = -1;
#pragma unroll
        for (int q = Q - 1; q >= 0; --q) {
            const uint64_t m = ballot(up[q] == cur && tok[q] == w);
            if (m) next = q * 64 + __builtin_ctzll(m);
        }
        cur = next;
    }
    if (lane == 0) p.n_keep[b] = kept;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int i = q * 64 + lane;
        if (i < p.T) {
            p.path[base + i] = path[q];
            p.out_tok[base + i] = out[q];
        }
    }
}

}  // namespace dsel
