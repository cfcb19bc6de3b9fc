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

// Row i of the mask holds i and every node above it.  One thread per node
// climbs its own parent links in LDS (as many steps as the node is deep; a
// link that does not go to an earlier node ends the climb), setting bits in its
// own LDS words.  A launch's latency bounds it.
__global__ __launch_bounds__(kMaxTree) void tree_mask_kernel(TreeParams p) {
    __shared__ int up[kMaxTree];
    __shared__ uint32_t bits[kMaxTree * (kMaxTree / 32 + 1)];  // an odd stride spreads the rows over the banks
    constexpr int S = kMaxTree / 32 + 1;
    const int b = blockIdx.x, i = threadIdx.x, words = (p.T + 31) / 32;
    const int n = block_len_of(p.len, b, p.T);
    if (i < n) {
        int a = p.parent[(int64_t)b * p.T + i];
        if (i == 0 ? a != -1 : (a < 0 || a >= i)) {
            device_error(kErrTree);
            a = -1;
        }
        up[i] = a;
        for (int w = 0; w < words; ++w) bits[i * S + w] = 0;
    }
    __syncthreads();
    if (i < n) {
        int d = -1;
        for (int a = i; a >= 0; a = up[a], ++d) bits[i * S + (a >> 5)] |= 1u << (a & 31);
        if (p.depth) p.depth[(int64_t)b * p.T + i] = d;
    }
    __syncthreads();
    int32_t *m = p.mask + (int64_t)b * p.T * words;
    for (int e = i; e < n * words; e += blockDim.x) m[e] = (int32_t)bits[(e / words) * S + e % words];
}

// One wave per tree: the nodes' parents and tokens stay in registers, four per
// lane, and each step is a compare and a ballot per 64 nodes.  A child lies
// after its parent, so the walk ends.
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
