// libdsel.so: the C ABI declared in include/dsel.h.  Host-side validation,
// launch geometry and status codes; the kernels live in the headers below.
// The whole library is one translation unit (so the device error word needs no
// relocatable device code).
#include <hip/hip_runtime.h>

#include <limits.h>

#include <mutex>
#include <type_traits>

#include "dsel.h"
#include "common.h"
#include "conv.h"
#include "evict.h"
#include "fused.h"
#include "keyweights.h"
#include "latency.h"
#include "lmhead.h"
#include "pairwalk.h"
#include "path.h"
#include "project.h"
#include "topk16.h"
#include "tree.h"
#include "treeattn.h"
#include "treeattn4.h"
#include "verify.h"

#define DSEL_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace dsel;

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Do the na bytes from a on and the nb bytes from b on share any?
inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    return (uintptr_t)a < (uintptr_t)b + (uintptr_t)nb && (uintptr_t)b < (uintptr_t)a + (uintptr_t)na;
}

// `rows` runs of `width` bytes, `ld` from one to the next
struct Span {
    const void *at;  // NULL: no bytes
    int64_t width, rows = 1, ld = 0;
};
// Do two of them share any bytes?  Runs may lie in each other's gaps.
inline bool overlap(const Span &a, const Span &b) {
    if (!a.at || !b.at || !overlap(a.at, (a.rows - 1) * a.ld + a.width, b.at, (b.rows - 1) * b.ld + b.width)) return false;
    for (int64_t i = 0; i < a.rows; ++i) {
        const int64_t lo = (int64_t)((uintptr_t)a.at - (uintptr_t)b.at) + i * a.ld;  // from b's begin on
        // b's first run that ends behind lo
        const int64_t j = lo < b.width ? 0 : b.rows > 1 ? (lo - b.width) / b.ld + 1 : 1;
        if (j < b.rows && j * b.ld < lo + a.width) return true;
    }
    return false;
}

inline dsel_status launch(const void *kernel, dim3 grid, dim3 block, void *arg, size_t shmem,
                          dsel_stream_t stream) {
    void *args[] = {arg};
    hipError_t e = hipLaunchKernel(kernel, grid, block, args, shmem, (hipStream_t)stream);
    return e == hipSuccess ? DSEL_OK : DSEL_E_HIP;
}

#ifndef DSEL_VERIFY_WGS
#define DSEL_VERIFY_WGS 2048
#endif


dsel_status check_walk(const dsel_walk_args *w, WalkParams *out) {
    if (!w) return DSEL_E_ARG;
    if (w->mode != DSEL_GREEDY && w->mode != DSEL_SAMPLED) return DSEL_E_DTYPE;
    if (!w->cand_id || !w->path_tok || !w->path_slot) return DSEL_E_ARG;
    if (w->mode == DSEL_SAMPLED && (!w->uniforms || !(w->temperature > 0.0f))) return DSEL_E_ARG;
    if (!aligned(w->cand_id, 4) || !aligned(w->path_tok, 4) || !aligned(w->path_slot, 4) ||
        !aligned(w->path_s, 4) || !aligned(w->q, 4) || !aligned(w->uniforms, 4))
        return DSEL_E_ALIGN;
    out->mode = w->mode;
    out->temperature = w->mode == DSEL_SAMPLED ? w->temperature : 1.0f;
    out->uniforms = w->uniforms;
    out->cand_id = w->cand_id;
    out->path_tok = w->path_tok;
    out->path_slot = w->path_slot;
    out->path_s = w->path_s;
    out->q = w->q;
    return DSEL_OK;
}

}  // namespace

DSEL_API size_t dsel_topk_workspace_bytes(int64_t rows, int64_t vocab, dsel_dtype dt) {
    if (rows <= 0 || vocab < kK || vocab >= (int64_t)INT_MAX || (dt != DSEL_F32 && dt != DSEL_BF16))
        return 0;
    int ns = topk_nsplit(rows, vocab);
    return ns > 1 ? (size_t)rows * (size_t)ns * kK * sizeof(uint64_t) : 0;
}

namespace {

// Validation and launch geometry of each step, shared by its own entry point
// and by dsel_select_path.  A plan with `empty` set has nothing to launch.
struct TopkPlan {
    TopkParams p;
    bool bf16 = false, empty = false;
};

dsel_status plan_topk(const void *logits, dsel_dtype dt, int64_t batch, int64_t block, const int32_t *block_len,
                      int64_t vocab, int64_t ld, int32_t *cand_id, float *cand_u, void *workspace,
                      size_t workspace_bytes, TopkPlan *t) {
    if (dt != DSEL_F32 && dt != DSEL_BF16) return DSEL_E_DTYPE;
    if (batch < 0 || block < 0 || vocab < kK || vocab >= (int64_t)INT_MAX || ld < vocab) return DSEL_E_ARG;
    const int64_t rows = batch * block;
    if (block != 0 && rows / block != batch) return DSEL_E_ARG;
    t->empty = rows == 0;
    if (t->empty) return DSEL_OK;  // nothing to read or write; pointers may be NULL
    if (!logits || !cand_id || !cand_u) return DSEL_E_ARG;
    const size_t es = dt == DSEL_BF16 ? 2 : 4;
    if (!aligned(logits, es) || !aligned(cand_id, 4) || !aligned(cand_u, 4) || !aligned(block_len, 4))
        return DSEL_E_ALIGN;
    if (ld > INT64_MAX / (int64_t)es / rows) return DSEL_E_ARG;
    const int ns = topk_nsplit(rows, vocab);
    if ((int64_t)ns * rows >= (int64_t)INT_MAX) return DSEL_E_ARG;
    const size_t need = dsel_topk_workspace_bytes(rows, vocab, dt);
    if (need && (!workspace || workspace_bytes < need)) return DSEL_E_WORKSPACE;
    if (need && !aligned(workspace, 8)) return DSEL_E_ALIGN;
    TopkParams &p = t->p;
    p.logits = (const char *)logits;
    p.rows = rows;
    p.V = vocab;
    p.ld = ld;
    p.nsplit = ns;
    p.L = (int)block;
    p.len = block_len;
    p.cand_id = cand_id;
    p.cand_u = cand_u;
    p.partial = (uint64_t *)workspace;
    t->bf16 = dt == DSEL_BF16;
    return DSEL_OK;
}

// The top-16 launch; with `gate` (a split gate job) its reduction rides along
// as extra workgroups (path.h).
dsel_status launch_topk(const TopkPlan &t, const GateParams *gate, int64_t gate_units, dsel_stream_t stream) {
    TopkParams p = t.p;
    const int64_t wgs = p.rows * p.nsplit;
    dsel_status s;
    if (gate) {
        GateParams gp = *gate;
        int64_t tw = wgs;
        constexpr int TT = 64 * kTopkWaves;
        const int64_t grid = wgs + (gate_units + TT - 1) / TT;
        if (grid >= (int64_t)INT_MAX) return DSEL_E_ARG;
        const void *k = t.bf16 ? (const void *)topk16_gate_kernel<true, kTopkUnroll<true>>
                               : (const void *)topk16_gate_kernel<false, kTopkUnroll<false>>;
        void *args[] = {&p, &gp, &tw};
        s = hipLaunchKernel(k, dim3((unsigned)grid), dim3(64 * kTopkWaves), args, 0, (hipStream_t)stream) == hipSuccess
                ? DSEL_OK : DSEL_E_HIP;
    } else {
        const void *k = t.bf16 ? (const void *)topk16_kernel<true, kTopkUnroll<true>>
                               : (const void *)topk16_kernel<false, kTopkUnroll<false>>;
        s = launch(k, dim3((unsigned)wgs), dim3(64 * kTopkWaves), &p, 0, stream);
    }
    if (s != DSEL_OK || p.nsplit == 1) return s;
    const void *k2 = t.bf16 ? (const void *)topk16_merge_kernel<true> : (const void *)topk16_merge_kernel<false>;
    return launch(k2, dim3((unsigned)p.rows), dim3(256), &p, 0, stream);
}

}  // namespace

DSEL_API dsel_status dsel_select_topk(const void *logits, dsel_dtype dt, int64_t batch,
                                      int64_t block, const int32_t *block_len, int64_t vocab, int64_t ld,
                                      int32_t *cand_id, float *cand_u, void *workspace, size_t workspace_bytes,
                                      dsel_stream_t stream) {
    TopkPlan t;
    dsel_status st = plan_topk(logits, dt, batch, block, block_len, vocab, ld, cand_id, cand_u, workspace,
                               workspace_bytes, &t);
    if (st != DSEL_OK || t.empty) return st;
    return launch_topk(t, nullptr, 0, stream);
}

namespace {

dsel_status check_project_common(const uint16_t *E, int64_t vocab, int64_t d, int64_t r,
                                 int64_t batch, int64_t block) {
    if (vocab < 1 || vocab >= (int64_t)INT_MAX || d < 64 || d % 64 != 0 || d > (1 << 20)) return DSEL_E_ARG;
    if (r < 32 || r > DSEL_MAX_RANK || r % 32 != 0) return DSEL_E_ARG;
    if (batch < 0 || block < 1 || batch > (1 << 24) || block > (1 << 16)) return DSEL_E_ARG;
    if (batch > 0 && !E) return DSEL_E_ARG;
    if (!aligned(E, 16)) return DSEL_E_ALIGN;
    return DSEL_OK;
}

// Workspace layout shared by dsel_project, dsel_project_gate and
// dsel_project_cand: the gate's partial tiles first, then (256-byte aligned)
// the candidate job's, so the two halves never touch each other's part.
size_t cand_workspace_offset(int64_t batch, int64_t block, int64_t d, int64_t r) {
    return (gate_workspace_bytes(batch, block, d, r) + 255) / 256 * 256;
}

}  // namespace

DSEL_API size_t dsel_project_workspace_bytes(int64_t batch, int64_t block, int64_t d, int64_t r) {
    if (batch <= 0 || block < 1 || d < 64 || d % 64 != 0 || r < 32 || r > DSEL_MAX_RANK || r % 32 != 0)
        return 0;
    const size_t c = cand_workspace_bytes(batch, block, d, r);
    return c ? cand_workspace_offset(batch, block, d, r) + c : gate_workspace_bytes(batch, block, d, r);
}

namespace {

struct GatePlan {
    GateParams p;
    int BN = 0;
    bool empty = false;
};

// The gate job; `split` = false runs one workgroup per output tile with no
// K split and no workspace.
dsel_status plan_gate(const uint16_t *E, int64_t vocab, int64_t d, const uint16_t *W_A, const uint16_t *W_H,
                      int64_t r, const uint16_t *h, const int32_t *verified, int64_t batch, int64_t block,
                      const int32_t *block_len, float *A_prev, float *G, void *workspace, size_t workspace_bytes,
                      bool split, GatePlan *g) {
    dsel_status st = check_project_common(E, vocab, d, r, batch, block);
    g->empty = batch == 0;
    if (st != DSEL_OK || g->empty) return st;
    if (!W_A || !W_H || !h || !verified || !A_prev || !G) return DSEL_E_ARG;
    if (!aligned(W_A, 16) || !aligned(W_H, 16) || !aligned(h, 16) || !aligned(verified, 4) ||
        !aligned(A_prev, 16) || !aligned(G, 16) || !aligned(block_len, 4))
        return DSEL_E_ALIGN;
    const size_t need = split ? gate_workspace_bytes(batch, block, d, r) : 0;
    if (need && (!workspace || workspace_bytes < need)) return DSEL_E_WORKSPACE;
    if (need && !aligned(workspace, 16)) return DSEL_E_ALIGN;
    GateParams &p = g->p;
    p.E = E;
    p.V = vocab;
    p.d = (int)d;
    p.r = (int)r;
    p.WA = W_A;
    p.WH = W_H;
    p.h = h;
    p.ver = verified;
    p.B = (int)batch;
    p.L = (int)block;
    p.len = block_len;
    p.A_prev = A_prev;
    p.G = G;
    p.A_ver = A_prev;
    p.ver_stride = block * kK * r;
    p.ver_zero = true;
    p.part = (float *)workspace;
    g->BN = gate_bn(batch, block, r);
    p.nside = (int)(r / g->BN);
    p.mt_gate = (int)((batch * block + 127) / 128);
    p.mt_ver = (int)((batch + 127) / 128);
    p.nsplit = split ? gate_nsplit(batch, block, d, r) : 1;
    const int64_t grid = (int64_t)(p.mt_gate + p.mt_ver) * p.nside * p.nsplit;
    if (grid >= (int64_t)INT_MAX) return DSEL_E_ARG;
    return DSEL_OK;
}

// Output elements of the gate's reduction (0 when it is not split).
// Work units (four output elements each) of the gate reduction; 0 when unsplit.
int64_t gate_reduce_units(const GatePlan &g) {
    return g.p.nsplit > 1 ? ((int64_t)g.p.B * g.p.L + g.p.B) * g.p.r / 4 : 0;
}

dsel_status launch_gate_gemm(const GatePlan &g, dsel_stream_t stream) {
    GateParams p = g.p;
    const int64_t grid = (int64_t)(p.mt_gate + p.mt_ver) * p.nside * p.nsplit;
    const void *k = g.BN == 256 ? (const void *)project_gate_kernel<256>
                  : g.BN == 128 ? (const void *)project_gate_kernel<128>
                  : g.BN == 64  ? (const void *)project_gate_kernel<64>
                                : (const void *)project_gate_kernel<32>;
    return launch(k, dim3((unsigned)grid), dim3(tile_threads(g.BN)), &p, 0, stream);
}

dsel_status launch_gate_reduce(const GatePlan &g, dsel_stream_t stream) {
    GateParams p = g.p;
    const int64_t elems = gate_reduce_units(g);
    if (elems == 0) return DSEL_OK;
    return launch((const void *)project_gate_reduce_kernel, dim3((unsigned)((elems + 255) / 256)), dim3(256), &p,
                  0, stream);
}

// The gate's split-K reduction and the top-16 (the reduction is needed only
// after the top-16).  Where the top-16 is one round of workgroups (at most
// DSEL_FOLD_MAX_TOPK_WG: four rows per CU), the reduction rides in its
// launch as extra workgroups, beside it; beyond, those workgroups would land
// on the last round, so the reduction is a launch of its own before it
// (MI355X: 1,024 bf16 rows, folded 120.8 / 160.8 us per step against
// 124.6 / 164.1 at the two shapes of 1,024 rows; 4,096 fp32 rows, 912.1 us
// separate against 921.0 folded).
#ifndef DSEL_FOLD_MAX_TOPK_WG
#define DSEL_FOLD_MAX_TOPK_WG 1024
#endif
dsel_status launch_topk_and_gate_reduce(const TopkPlan &t, const GatePlan &g, dsel_stream_t stream) {
    const int64_t ge = gate_reduce_units(g);
    if (ge == 0 || t.p.rows * t.p.nsplit <= DSEL_FOLD_MAX_TOPK_WG)
        return launch_topk(t, ge ? &g.p : nullptr, ge, stream);
    dsel_status st = launch_gate_reduce(g, stream);
    return st == DSEL_OK ? launch_topk(t, nullptr, 0, stream) : st;
}

dsel_status project_gate_impl(const uint16_t *E, int64_t vocab, int64_t d, const uint16_t *W_A,
                              const uint16_t *W_H, int64_t r, const uint16_t *h, const int32_t *verified,
                              int64_t batch, int64_t block, const int32_t *block_len, float *A_prev, float *G,
                              void *workspace, size_t workspace_bytes, bool split, dsel_stream_t stream) {
    GatePlan g;
    dsel_status st = plan_gate(E, vocab, d, W_A, W_H, r, h, verified, batch, block, block_len, A_prev, G, workspace,
                               workspace_bytes, split, &g);
    if (st != DSEL_OK || g.empty) return st;
    st = launch_gate_gemm(g, stream);
    if (st != DSEL_OK) return st;
    return launch_gate_reduce(g, stream);
}

}  // namespace

DSEL_API dsel_status dsel_project_gate(const uint16_t *E, int64_t vocab, int64_t d,
                                       const uint16_t *W_A, const uint16_t *W_H, int64_t r,
                                       const uint16_t *h, const int32_t *verified, int64_t batch,
                                       int64_t block, const int32_t *block_len, float *A_prev, float *G,
                                       void *workspace, size_t workspace_bytes, dsel_stream_t stream) {
    return project_gate_impl(E, vocab, d, W_A, W_H, r, h, verified, batch, block, block_len, A_prev, G,
                             workspace, workspace_bytes, true, stream);
}

DSEL_API dsel_status dsel_project_gate_overlap(const uint16_t *E, int64_t vocab, int64_t d,
                                               const uint16_t *W_A, const uint16_t *W_H, int64_t r,
                                               const uint16_t *h, const int32_t *verified, int64_t batch,
                                               int64_t block, const int32_t *block_len, float *A_prev,
                                               float *G, dsel_stream_t stream) {
    return project_gate_impl(E, vocab, d, W_A, W_H, r, h, verified, batch, block, block_len, A_prev, G, nullptr,
                             0, false, stream);
}

namespace {

struct CandPlan {
    CandParams p;
    int BN = 0;
    bool empty = false;
};

dsel_status plan_cand(const uint16_t *E, int64_t vocab, int64_t d, const uint16_t *W_A, const uint16_t *W_B,
                      int64_t r, const int32_t *cand_id, int64_t batch, int64_t block, const int32_t *block_len,
                      float *A_prev, float *B_cur, void *workspace, size_t workspace_bytes, CandPlan *c) {
    dsel_status st = check_project_common(E, vocab, d, r, batch, block);
    c->empty = batch == 0;
    if (st != DSEL_OK || c->empty) return st;
    if (!W_A || !W_B || !cand_id || !A_prev || !B_cur) return DSEL_E_ARG;
    if (!aligned(W_A, 16) || !aligned(W_B, 16) || !aligned(cand_id, 4) || !aligned(A_prev, 16) ||
        !aligned(B_cur, 16) || !aligned(block_len, 4))
        return DSEL_E_ALIGN;
    const size_t cneed = cand_workspace_bytes(batch, block, d, r);
    const size_t coff = cand_workspace_offset(batch, block, d, r);
    if (cneed && (!workspace || workspace_bytes < coff + cneed)) return DSEL_E_WORKSPACE;
    if (cneed && !aligned(workspace, 16)) return DSEL_E_ALIGN;
    CandParams &p = c->p;
    p.E = E;
    p.V = vocab;
    p.d = (int)d;
    p.r = (int)r;
    p.WA = W_A;
    p.WB = W_B;
    p.cand = cand_id;
    p.L = (int)block;
    p.len = block_len;
    p.M = batch * block * kK;
    p.A_prev = A_prev;
    p.B_cur = B_cur;
    p.tk_part = nullptr;
    p.tk_nsplit = 0;
    p.cand_id = nullptr;
    p.cand_u = nullptr;
    p.logits = nullptr;
    p.ld = p.V_logits = 0;
    p.logits_bf16 = false;
    constexpr int BM = 128;
    c->BN = cand_bn(batch, block, r);
    p.nside = (int)(r / c->BN);
    p.mt = (int)((p.M + BM - 1) / BM);
    p.mt_pad = (p.mt + 7) / 8 * 8;
    p.nsplit = cand_nsplit(batch, block, d, r);
    p.part = cneed ? (float *)((char *)workspace + coff) : nullptr;
    const int64_t grid = (int64_t)p.mt_pad * 2 * p.nside * p.nsplit;
    if (grid >= (int64_t)INT_MAX || p.M * 2 * r >= (int64_t)INT_MAX * 256) return DSEL_E_ARG;
    return DSEL_OK;
}

dsel_status launch_cand_gemm(const CandPlan &c, dsel_stream_t stream) {
    CandParams p = c.p;
    const int BN = c.BN;
    const int64_t grid = (int64_t)p.mt_pad * 2 * p.nside * p.nsplit;
    const void *k = BN == 256 ? (const void *)project_cand_kernel<256>
                  : BN == 128 ? (const void *)project_cand_kernel<128>
                  : BN == 64  ? (const void *)project_cand_kernel<64>
                              : (const void *)project_cand_kernel<32>;
    return launch(k, dim3((unsigned)grid), dim3(tile_threads(BN)), &p, 0, stream);
}

dsel_status launch_cand(const CandPlan &c, dsel_stream_t stream) {
    CandParams p = c.p;
    const int BN = c.BN;
    dsel_status st = launch_cand_gemm(c, stream);
    if (st != DSEL_OK || p.nsplit == 1) return st;
    const int64_t elems = p.M * 2 * p.r;
    const void *kr = BN == 256 ? (const void *)project_cand_reduce_kernel<256>
                   : BN == 128 ? (const void *)project_cand_reduce_kernel<128>
                   : BN == 64  ? (const void *)project_cand_reduce_kernel<64>
                               : (const void *)project_cand_reduce_kernel<32>;
    return launch(kr, dim3((unsigned)((elems + 255) / 256)), dim3(256), &p, 0, stream);
}

}  // namespace

DSEL_API dsel_status dsel_project_cand(const uint16_t *E, int64_t vocab, int64_t d,
                                       const uint16_t *W_A, const uint16_t *W_B, int64_t r,
                                       const int32_t *cand_id, int64_t batch, int64_t block,
                                       const int32_t *block_len, float *A_prev, float *B_cur,
                                       void *workspace, size_t workspace_bytes, dsel_stream_t stream) {
    CandPlan c;
    dsel_status st = plan_cand(E, vocab, d, W_A, W_B, r, cand_id, batch, block, block_len, A_prev, B_cur,
                               workspace, workspace_bytes, &c);
    if (st != DSEL_OK || c.empty) return st;
    return launch_cand(c, stream);
}

DSEL_API dsel_status dsel_project(const uint16_t *E, int64_t vocab, int64_t d, const uint16_t *W_A,
                                  const uint16_t *W_B, const uint16_t *W_H, int64_t r,
                                  const uint16_t *h, const int32_t *cand_id,
                                  const int32_t *verified, int64_t batch, int64_t block,
                                  const int32_t *block_len, float *A_prev, float *B_cur, float *G,
                                  void *workspace, size_t workspace_bytes, dsel_stream_t stream) {
    dsel_status st = check_project_common(E, vocab, d, r, batch, block);
    if (st != DSEL_OK || batch == 0) return st;
    if (!W_A || !W_B || !W_H || !h || !cand_id || !verified || !A_prev || !B_cur || !G)
        return DSEL_E_ARG;
    const size_t need = dsel_project_workspace_bytes(batch, block, d, r);
    if (need && (!workspace || workspace_bytes < need)) return DSEL_E_WORKSPACE;
    st = dsel_project_gate(E, vocab, d, W_A, W_H, r, h, verified, batch, block, block_len, A_prev, G,
                           workspace, workspace_bytes, stream);
    if (st != DSEL_OK) return st;
    return dsel_project_cand(E, vocab, d, W_A, W_B, r, cand_id, batch, block, block_len, A_prev, B_cur,
                             workspace, workspace_bytes, stream);
}

namespace {

const void *pair_kernel_for(int64_t r) {
    switch (r) {
        case 32: return (const void *)pair_kernel<32>;
        case 64: return (const void *)pair_kernel<64>;
        case 96: return (const void *)pair_kernel<96>;
        case 128: return (const void *)pair_kernel<128>;
        case 160: return (const void *)pair_kernel<160>;
        case 192: return (const void *)pair_kernel<192>;
        case 224: return (const void *)pair_kernel<224>;
        case 256: return (const void *)pair_kernel<256>;
    }
    return nullptr;
}

dsel_status launch_walk(PairParams &p, dsel_stream_t stream) {
    const int waves = p.L < 16 ? p.L : 16;
    const size_t shmem = pair_walk_shmem(p.L, p.w.q != nullptr);
    return launch((const void *)walk_kernel, dim3((unsigned)p.B), dim3(waves * kWave), &p, shmem, stream);
}

}  // namespace

namespace {

struct PairPlan {
    PairParams p = {};
    bool walk = false, empty = false;
};

dsel_status plan_pairs(const float *cand_u, const float *A_prev, const float *B_cur, const float *G, int64_t batch,
                       int64_t block, const int32_t *block_len, int64_t r, float *S, const dsel_walk_args *walk,
                       PairPlan *q) {
    if (batch < 0 || batch >= (int64_t)INT_MAX / DSEL_MAX_BLOCK || block < 1 || block > DSEL_MAX_BLOCK)
        return DSEL_E_ARG;
    if (r < 32 || r > DSEL_MAX_RANK || r % 32 != 0) return DSEL_E_ARG;
    if (walk && walk->mode != DSEL_GREEDY && walk->mode != DSEL_SAMPLED) return DSEL_E_DTYPE;
    q->empty = batch == 0;
    if (q->empty) return DSEL_OK;  // nothing to read or write; pointers may be NULL
    if (!cand_u || !A_prev || !B_cur || !G || !S) return DSEL_E_ARG;
    if (!aligned(A_prev, 16) || !aligned(B_cur, 16) || !aligned(G, 16) || !aligned(cand_u, 4) ||
        !aligned(S, 4) || !aligned(block_len, 4))
        return DSEL_E_ALIGN;
    PairParams &p = q->p;
    if (walk) {
        dsel_status s = check_walk(walk, &p.w);
        if (s != DSEL_OK) return s;
    }
    q->walk = walk != nullptr;
    p.cand_u = cand_u;
    p.A_prev = A_prev;
    p.B_cur = B_cur;
    p.G = G;
    p.B = (int)batch;
    p.L = (int)block;
    p.len = block_len;
    p.r = (int)r;
    p.S = S;
    p.S_in = S;
    return DSEL_OK;
}

dsel_status launch_pairs(const PairPlan &q, dsel_stream_t stream) {
    PairParams p = q.p;
    const int64_t positions = (int64_t)p.B * p.L;
    dsel_status st = launch(pair_kernel_for(p.r), dim3((unsigned)positions), dim3(256), &p, 0, stream);
    if (st != DSEL_OK || !q.walk) return st;
    return launch_walk(p, stream);
}

}  // namespace

DSEL_API dsel_status dsel_score_pairs(const float *cand_u, const float *A_prev, const float *B_cur,
                                      const float *G, int64_t batch, int64_t block,
                                      const int32_t *block_len, int64_t r, float *S,
                                      const dsel_walk_args *walk, dsel_stream_t stream) {
    PairPlan q;
    dsel_status st = plan_pairs(cand_u, A_prev, B_cur, G, batch, block, block_len, r, S, walk, &q);
    if (st != DSEL_OK || q.empty) return st;
    return launch_pairs(q, stream);
}

DSEL_API dsel_status dsel_walk(const float *S, int64_t batch, int64_t block, const int32_t *block_len,
                               const dsel_walk_args *walk, dsel_stream_t stream) {
    if (!walk) return DSEL_E_ARG;
    if (batch < 0 || batch >= (int64_t)INT_MAX || block < 1 || block > DSEL_MAX_BLOCK) return DSEL_E_ARG;
    if (walk->mode != DSEL_GREEDY && walk->mode != DSEL_SAMPLED) return DSEL_E_DTYPE;
    if (batch == 0) return DSEL_OK;  // nothing to read or write; pointers may be NULL
    if (!S) return DSEL_E_ARG;
    if (!aligned(S, 4) || !aligned(block_len, 4)) return DSEL_E_ALIGN;
    PairParams p = {};
    dsel_status s = check_walk(walk, &p.w);
    if (s != DSEL_OK) return s;
    p.S_in = S;
    p.B = (int)batch;
    p.L = (int)block;
    p.len = block_len;
    return launch_walk(p, stream);
}

// ---- measurement aid: the candidate gather alone -----------------------------

DSEL_API dsel_status dsel_gather_probe(const uint16_t *E, int64_t vocab, int64_t d, const int32_t *cand_id,
                                       int64_t batch, int64_t block, uint32_t *out, size_t out_words,
                                       dsel_stream_t stream) {
    dsel_status st = check_project_common(E, vocab, d, 32, batch, block);
    if (st != DSEL_OK || batch == 0) return st;
    if (!cand_id || !out) return DSEL_E_ARG;
    if (!aligned(cand_id, 4) || !aligned(out, 4)) return DSEL_E_ALIGN;
    GatherProbeParams p;
    p.E = E;
    p.V = vocab;
    p.d = (int)d;
    p.cand = cand_id;
    p.M = batch * block * kK;
    const int64_t mt = (p.M + 127) / 128;
    p.nsplit = gather_probe_nsplit(p.M, d);
    const int64_t grid = mt * p.nsplit;
    if (grid >= (int64_t)INT_MAX / 256 || out_words < (size_t)grid * 256) return DSEL_E_ARG;
    p.mt = (int)mt;
    p.out = out;
    return launch((const void *)gather_probe_kernel, dim3((unsigned)grid), dim3(256), &p, 0, stream);
}

DSEL_API size_t dsel_gather_probe_words(int64_t batch, int64_t block, int64_t d) {
    if (batch <= 0 || block < 1 || d < 64 || d % 64 != 0) return 0;
    const int64_t M = batch * block * kK;
    return (size_t)((M + 127) / 128) * (size_t)gather_probe_nsplit(M, d) * 256;
}

// ---- the whole selector ----------------------------------------------------

namespace {

inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of dsel_select_path, in this order (each part 256-byte aligned):
// the top-16's partial lists; the projections' split-K partials; G; then, on
// the fused route, A(verified) [B][r] and the pair partials, else A_prev,
// B_cur [B, L, 16, r] and S [B, L, 16, 16].  The parts for outputs the caller
// supplies are reserved but unused.
struct PathLayout {
    size_t topk = 0, proj = 0, g = 0, aver = 0, part = 0, a = 0, b = 0, s = 0, lat = 0, cnt = 0, total = 0;
    bool fused = false;
};

bool path_layout(int64_t batch, int64_t block, int64_t vocab, dsel_dtype dt, int64_t d, int64_t r,
                 PathLayout *l) {
    if (batch <= 0 || block < 1 || block > DSEL_MAX_BLOCK || batch > (int64_t)INT_MAX / block) return false;
    if (d < 64 || d % 64 != 0 || r < 32 || r > DSEL_MAX_RANK || r % 32 != 0) return false;
    const int64_t pos = batch * block;
    size_t off = align256(dsel_topk_workspace_bytes(pos, vocab, dt));
    l->topk = 0;
    l->proj = off;
    off += align256(dsel_project_workspace_bytes(batch, block, d, r));
    l->g = off;
    off += align256((size_t)pos * r * sizeof(float));
    l->fused = use_fused(batch, block, r);
    if (l->fused) {
        l->aver = off;
        off += align256((size_t)batch * r * sizeof(float));
        l->part = off;
        off += align256(fused_partial_bytes(batch, block, r));
    } else {
        const size_t ab = align256((size_t)pos * kK * r * sizeof(float));
        l->a = off;
        off += ab;
        l->b = off;
        off += ab;
        l->s = off;
        off += align256((size_t)pos * kK * kK * sizeof(float));
        // the small-batch route's decision tables (slot, score, distribution
        // per predecessor row), group tables and arrival counters (per
        // position, then per block)
        l->lat = off;
        off += align256((size_t)pos * kK) + align256((size_t)pos * kK * sizeof(float)) +
               align256((size_t)pos * kK * kK * sizeof(float)) +
               align256((size_t)pos * (r / pair_cw((int)r)) * kK * kK * sizeof(float));
        l->cnt = off;
        off += align256((size_t)(pos + batch) * sizeof(int));
    }
    l->total = off;
    return true;
}

struct FusedPlan {
    FusedParams p;
    int CW = 64;
    int NG = 1;  // rank groups per workgroup
};

dsel_status plan_fused(const uint16_t *E, int64_t vocab, int64_t d, const uint16_t *W_A, const uint16_t *W_B,
                       int64_t r, const int32_t *cand_id, const float *G, const float *A_ver, int64_t ver_stride,
                       int64_t batch, int64_t block, const int32_t *block_len, float *P, float *A_prev,
                       float *B_cur, FusedPlan *f) {
    dsel_status st = check_project_common(E, vocab, d, r, batch, block);
    if (st != DSEL_OK) return st;
    if (fused_blocks_per_tile(block) == 0 || batch > (int64_t)INT_MAX / 16) return DSEL_E_ARG;
    if (!W_A || !W_B || !cand_id || !G || !A_ver || !P || ver_stride < r) return DSEL_E_ARG;
    if ((A_prev == nullptr) != (B_cur == nullptr)) return DSEL_E_ARG;
    if (!aligned(W_A, 16) || !aligned(W_B, 16) || !aligned(cand_id, 4) || !aligned(G, 16) || !aligned(A_ver, 16) ||
        ver_stride % 4 != 0 || !aligned(P, 16) || !aligned(A_prev, 16) || !aligned(B_cur, 16) ||
        !aligned(block_len, 4))
        return DSEL_E_ALIGN;
    FusedParams &p = f->p;
    p.E = E;
    p.V = vocab;
    p.d = (int)d;
    p.r = (int)r;
    p.WA = W_A;
    p.WB = W_B;
    p.cand = cand_id;
    p.G = G;
    p.A_ver = A_ver;
    p.ver_stride = ver_stride;
    p.B = (int)batch;
    p.L = (int)block;
    p.len = block_len;
    p.nb = fused_blocks_per_tile(block);
    p.ntile = (int)fused_grid_tiles(batch, block, block_len != nullptr);
    f->CW = pair_group_width((int)r);
    f->NG = fused_groups(batch, block, r, block_len != nullptr);
    p.nq = (int)(r / f->CW);
    p.P = P;
    p.A_prev = A_prev;
    p.B_cur = B_cur;
    if (fused_grid(batch, block, r, block_len != nullptr) >= (int64_t)INT_MAX) return DSEL_E_ARG;
    return DSEL_OK;
}

dsel_status launch_fused(const FusedPlan &f, dsel_stream_t stream) {
    FusedParams p = f.p;
    const int64_t grid = fused_grid(p.B, p.L, p.r, p.len != nullptr);
    const void *k = f.CW == 32 ? (const void *)project_pair_kernel<32, 1>
                    : f.NG == 2 ? (const void *)project_pair_kernel<64, 2>
                                : (const void *)project_pair_kernel<64, 1>;
    const int nt = f.CW == 32 ? FusedTile<32, 1>::NT : f.NG == 2 ? FusedTile<64, 2>::NT : FusedTile<64, 1>::NT;
    return launch(k, dim3((unsigned)grid), dim3(nt), &p, 0, stream);
}

}  // namespace

DSEL_API size_t dsel_select_path_workspace_bytes(int64_t batch, int64_t block, int64_t vocab, dsel_dtype dt,
                                                 int64_t d, int64_t r) {
    PathLayout l;
    return path_layout(batch, block, vocab, dt, d, r, &l) ? l.total : 0;
}

DSEL_API int64_t dsel_pair_groups(int64_t r) {
    if (r < 32 || r > DSEL_MAX_RANK || r % 32 != 0) return 0;
    return r / pair_group_width((int)r);
}

DSEL_API dsel_status dsel_project_pairs(const uint16_t *E, int64_t vocab, int64_t d, const uint16_t *W_A,
                                        const uint16_t *W_B, int64_t r, const int32_t *cand_id, const float *G,
                                        const float *A_ver, int64_t ver_stride, int64_t batch, int64_t block,
                                        const int32_t *block_len, float *partials, float *A_prev, float *B_cur,
                                        dsel_stream_t stream) {
    if (batch == 0 && block >= 1 && block <= 16) {
        dsel_status st = check_project_common(E, vocab, d, r, batch, block);
        return st;  // nothing to do; pointers may be NULL
    }
    FusedPlan f;
    dsel_status st = plan_fused(E, vocab, d, W_A, W_B, r, cand_id, G, A_ver, ver_stride, batch, block, block_len,
                                partials, A_prev, B_cur, &f);
    if (st != DSEL_OK) return st;
    return launch_fused(f, stream);
}

DSEL_API dsel_status dsel_walk_pairs(const float *cand_u, const float *partials, int64_t batch, int64_t block,
                                     const int32_t *block_len, int64_t nq, float *S, const dsel_walk_args *walk,
                                     dsel_stream_t stream) {
    if (!walk) return DSEL_E_ARG;
    if (batch < 0 || batch >= (int64_t)INT_MAX / DSEL_MAX_BLOCK || block < 1 || block > DSEL_MAX_BLOCK) return DSEL_E_ARG;
    if (nq < 1 || nq > DSEL_MAX_RANK / 32) return DSEL_E_ARG;
    if (walk->mode != DSEL_GREEDY && walk->mode != DSEL_SAMPLED) return DSEL_E_DTYPE;
    if (batch == 0) return DSEL_OK;
    if (!cand_u || !partials) return DSEL_E_ARG;
    if (!aligned(cand_u, 4) || !aligned(partials, 16) || !aligned(S, 4) || !aligned(block_len, 4)) return DSEL_E_ALIGN;
    PairParams p = {};
    dsel_status st = check_walk(walk, &p.w);
    if (st != DSEL_OK) return st;
    p.cand_u = cand_u;
    p.P = partials;
    p.nq = (int)nq;
    p.B = (int)batch;
    p.L = (int)block;
    p.len = block_len;
    p.S = S;
    return launch_walk(p, stream);
}

// ---- the small-batch route (latency.h) ----------------------------------------

// Top-16 workgroups beside the gate GEMM's in the first launch: the gate's LDS
// ring leaves room for two workgroups per CU, 512 in all.
#ifndef DSEL_LAT_TOPK_WG
#define DSEL_LAT_TOPK_WG 448
#endif
// Partial lists per top-16 row at most (measured at one block of 16, bf16 rows
// of 151,936: 8, 16 and 24 lists within 1 us of each other, 24 ahead; 4
// lists 8 us slower).
#ifndef DSEL_LAT_TOPK_LISTS
#define DSEL_LAT_TOPK_LISTS 24
#endif
// Partial lists per row that the candidate GEMM's merge can stage in its LDS
// ring (8 positions per tile, 16 keys of 8 bytes per list).
constexpr int kLatMaxLists = (int)(3 * 128 * kBK * sizeof(uint16_t) / (8 * kK * sizeof(uint64_t)));

struct LatPlan {
    TopkPlan t;
    GatePlan g;
    CandPlan c;
    LatParams k;
    int64_t topk_wgs = 0, gate_wgs = 0;
    bool use = false;
};

// The small-batch route serves a call of at most DSEL_LAT_MAX_ROWS positions
// that is not on the fused route and asks for no intermediates (A_prev,
// B_cur, G), when the gate GEMM is split with column tiles of at most 64 (its
// LDS ring then leaves room for the top-16 beside it); otherwise lp->use stays
// false.
// Workspace: the top-16 lists, the gate and candidate partials (or, from an
// unsplit candidate GEMM, A_prev and B_cur) where the separate route keeps
// them; the decision tables and the arrival counters in regions of their own.
// Positions up to which the small-batch route runs.  Beyond, the separate
// kernels are faster: the top-16 rows split fewer ways in the shared launch,
// and the last-arrival hand-offs grow with the positions (MI355X, blocks of 16
// at d 2560: 1 and 2 blocks 48.5 / 53.2 us against 52.6 / 54.1 separate; 4 and
// 8 blocks 65.4 / 87.7 us against 59.8 / 64.7).
#ifndef DSEL_LAT_MAX_ROWS
#define DSEL_LAT_MAX_ROWS 32
#endif

bool latency_route(int64_t batch, int64_t block, int64_t d, int64_t r, bool fused, bool intermediates) {
    return !fused && !intermediates && batch * block <= DSEL_LAT_MAX_ROWS && gate_bn(batch, block, r) <= 64 &&
           gate_nsplit(batch, block, d, r) > 1;
}

dsel_status plan_latency(const dsel_path_args *a, const dsel_walk_args *walk, char *ws, const PathLayout &l,
                         LatPlan *lp) {
    lp->use = false;
    if (!latency_route(a->batch, a->block, a->d, a->r, l.fused, a->A_prev || a->G)) return DSEL_OK;
    const int64_t rows = a->batch * a->block;
    float *A_buf = (float *)(ws + l.a), *B_buf = (float *)(ws + l.b);  // written by an unsplit candidate GEMM
    dsel_status st = plan_topk(a->logits, a->dt, a->batch, a->block, a->block_len, a->vocab, a->ld, a->cand_id,
                               a->cand_u, ws, l.proj, &lp->t);
    if (st != DSEL_OK) return st;
    st = plan_gate(a->E, a->vocab, a->d, a->W_A, a->W_H, a->r, a->h, a->verified, a->batch, a->block,
                   a->block_len, A_buf, A_buf, ws + l.proj, l.g - l.proj, true, &lp->g);
    if (st != DSEL_OK) return st;
    st = plan_cand(a->E, a->vocab, a->d, a->W_A, a->W_B, a->r, a->cand_id, a->batch, a->block, a->block_len,
                   A_buf, B_buf, ws + l.proj, l.g - l.proj, &lp->c);
    if (st != DSEL_OK) return st;
    if (lp->g.BN > 64 || lp->g.p.nsplit < 2) return DSEL_OK;
    if (!a->cand_u || !aligned(a->S, 4)) return !a->cand_u ? DSEL_E_ARG : DSEL_E_ALIGN;
    const GateParams &gp = lp->g.p;
    lp->gate_wgs = (int64_t)(gp.mt_gate + gp.mt_ver) * gp.nside * gp.nsplit;
    TopkParams &tp = lp->t.p;
    if (tp.nsplit > 1) {
        int64_t ns = (DSEL_LAT_TOPK_WG - lp->gate_wgs) / rows;
        if (ns > tp.nsplit) ns = tp.nsplit;
        if (ns > DSEL_LAT_TOPK_LISTS) ns = DSEL_LAT_TOPK_LISTS;
        if (ns > kLatMaxLists) ns = kLatMaxLists;
        tp.nsplit = (int)(ns < 1 ? 1 : ns);
    }
    lp->topk_wgs = rows * tp.nsplit;
    CandParams &cp = lp->c.p;
    if (tp.nsplit > 1) {  // the candidate GEMM merges the lists itself
        cp.tk_part = tp.partial;
        cp.tk_nsplit = tp.nsplit;
        cp.cand_id = a->cand_id;
        cp.cand_u = a->cand_u;
        cp.logits = (const char *)a->logits;
        cp.ld = a->ld;
        cp.V_logits = a->vocab;
        cp.logits_bf16 = a->dt == DSEL_BF16;
    }
    LatParams &k = lp->k;
    k = LatParams{};
    st = check_walk(walk, &k.pw.w);
    if (st != DSEL_OK) return st;
    k.pw.cand_u = a->cand_u;
    k.pw.B = (int)a->batch;
    k.pw.L = (int)a->block;
    k.pw.r = (int)a->r;
    k.pw.len = a->block_len;
    k.pw.S = a->S;
    k.pw.A_prev = A_buf;
    k.pw.B_cur = B_buf;
    k.ch = (uint8_t *)(ws + l.lat);
    k.sc = (float *)(ws + l.lat + align256((size_t)rows * kK));
    const size_t qoff = l.lat + align256((size_t)rows * kK) + align256((size_t)rows * kK * sizeof(float));
    k.Q = walk->q ? (float *)(ws + qoff) : nullptr;
    k.P = (float *)(ws + qoff + align256((size_t)rows * kK * kK * sizeof(float)));
    k.pw.nq = (int)(a->r / pair_cw((int)a->r));
    k.cpart = cp.part;
    k.c_nsplit = cp.nsplit;
    k.c_mt = cp.mt;
    k.c_nside = cp.nside;
    k.c_BN = lp->c.BN;
    k.gpart = gp.part;
    k.g_nsplit = gp.nsplit;
    k.cand = a->cand_id;
    k.V = a->vocab;
    k.pos_count = (int *)(ws + l.cnt);
    k.count = k.pos_count + rows;
    if (lp->topk_wgs + lp->gate_wgs >= (int64_t)INT_MAX) return DSEL_OK;
    lp->use = true;
    return DSEL_OK;
}

dsel_status launch_latency(LatPlan &lp, dsel_stream_t stream) {
    TopkParams tp = lp.t.p;
    GateParams gp = lp.g.p;
    int64_t tw = lp.topk_wgs;
    int *count = lp.k.pos_count;  // then the block counters
    int ncount = lp.k.pw.B * lp.k.pw.L + lp.k.pw.B;
    const int BN = lp.g.BN;
    const void *k1 = lp.t.bf16 ? (BN == 64 ? (const void *)topk16_gate_gemm_kernel<true, kTopkUnroll<true>, 64>
                                           : (const void *)topk16_gate_gemm_kernel<true, kTopkUnroll<true>, 32>)
                               : (BN == 64 ? (const void *)topk16_gate_gemm_kernel<false, kTopkUnroll<false>, 64>
                                           : (const void *)topk16_gate_gemm_kernel<false, kTopkUnroll<false>, 32>);
    void *args[] = {&tp, &gp, &tw, &count, &ncount};
    if (hipLaunchKernel(k1, dim3((unsigned)(lp.topk_wgs + lp.gate_wgs)), dim3(64 * kTopkWaves), args, 0,
                        (hipStream_t)stream) != hipSuccess)
        return DSEL_E_HIP;
    dsel_status st = launch_cand_gemm(lp.c, stream);
    if (st != DSEL_OK) return st;
    LatParams k = lp.k;
    const int CW = pair_cw(k.pw.r);
    const void *k3 = CW == 64 ? (const void *)pair_walk_lat_kernel<64> : (const void *)pair_walk_lat_kernel<32>;
    return launch(k3, dim3((unsigned)((int64_t)k.pw.B * k.pw.L * k.pw.nq)), dim3(CW / 16 * kWave), &k, 0, stream);
}

DSEL_API int dsel_select_path_route(const dsel_path_args *a) {
    if (!a) return -1;
    PathLayout l;
    if (a->batch <= 0 || !path_layout(a->batch, a->block, a->vocab, a->dt, a->d, a->r, &l)) return -1;
    if (l.fused) return DSEL_ROUTE_FUSED;
    return latency_route(a->batch, a->block, a->d, a->r, false, a->A_prev || a->G) ? DSEL_ROUTE_SMALL
                                                                                      : DSEL_ROUTE_SEPARATE;
}

DSEL_API dsel_status dsel_select_path(const dsel_path_args *a, const dsel_walk_args *walk, void *workspace,
                                      size_t workspace_bytes, dsel_stream_t stream) {
    if (!a || !walk) return DSEL_E_ARG;
    if (a->batch < 0 || a->block < 1 || a->block > DSEL_MAX_BLOCK || a->batch > (int64_t)INT_MAX / a->block)
        return DSEL_E_ARG;
    if ((a->A_prev == nullptr) != (a->B_cur == nullptr)) return DSEL_E_ARG;  // both or neither
    PathLayout l;
    if (a->batch > 0) {
        if (!path_layout(a->batch, a->block, a->vocab, a->dt, a->d, a->r, &l)) return DSEL_E_ARG;
        if (!workspace || workspace_bytes < l.total) return DSEL_E_WORKSPACE;
        if (!aligned(workspace, 256)) return DSEL_E_ALIGN;
    }
    char *ws = (char *)workspace;
    float *G = a->G ? a->G : (float *)(ws + l.g);
    // every step is validated before anything is launched
    TopkPlan t;
    GatePlan g;
    dsel_status st = plan_topk(a->logits, a->dt, a->batch, a->block, a->block_len, a->vocab, a->ld, a->cand_id,
                               a->cand_u, ws, l.proj, &t);
    if (st != DSEL_OK || a->batch == 0) return st;
    if (l.fused) {
        // gate GEMM; top-16 with the gate's reduction beside it; the fused
        // candidate projection + pair partials; the walk, which also forms S
        const bool ab = a->A_prev != nullptr;
        float *A_ver = ab ? a->A_prev : (float *)(ws + l.aver);
        st = plan_gate(a->E, a->vocab, a->d, a->W_A, a->W_H, a->r, a->h, a->verified, a->batch, a->block,
                       a->block_len, ab ? a->A_prev : A_ver, G, ws + l.proj, l.g - l.proj, true, &g);
        if (st != DSEL_OK) return st;
        if (!ab) {  // A(verified) to the compact buffer
            g.p.A_ver = A_ver;
            g.p.ver_stride = a->r;
            g.p.ver_zero = false;
        }
        FusedPlan f;
        st = plan_fused(a->E, a->vocab, a->d, a->W_A, a->W_B, a->r, a->cand_id, G, A_ver,
                        ab ? a->block * kK * a->r : a->r, a->batch, a->block, a->block_len, (float *)(ws + l.part),
                        a->A_prev, a->B_cur, &f);
        if (st != DSEL_OK) return st;
        PairPlan q;
        if (!a->cand_u || !aligned(a->S, 4)) return !a->cand_u ? DSEL_E_ARG : DSEL_E_ALIGN;
        st = check_walk(walk, &q.p.w);
        if (st != DSEL_OK) return st;
        q.p.cand_u = a->cand_u;
        q.p.P = f.p.P;
        q.p.nq = f.p.nq;
        q.p.B = (int)a->batch;
        q.p.L = (int)a->block;
        q.p.len = a->block_len;
        q.p.r = (int)a->r;
        q.p.S = a->S;
        st = launch_gate_gemm(g, stream);
        if (st == DSEL_OK) st = launch_topk_and_gate_reduce(t, g, stream);
        if (st == DSEL_OK) st = launch_fused(f, stream);
        if (st == DSEL_OK) st = launch_walk(q.p, stream);
        return st;
    }
    {
        LatPlan lp;
        st = plan_latency(a, walk, ws, l, &lp);
        if (st != DSEL_OK) return st;
        if (lp.use) return launch_latency(lp, stream);
    }
    // the separate kernels: gate GEMM; top-16 with the gate's reduction beside
    // it; candidate GEMM; pair scores and the walk (intermediates the caller
    // does not want live in the workspace)
    float *A_prev = a->A_prev ? a->A_prev : (float *)(ws + l.a);
    float *B_cur = a->B_cur ? a->B_cur : (float *)(ws + l.b);
    float *S = a->S ? a->S : (float *)(ws + l.s);
    CandPlan c;
    PairPlan q;
    st = plan_gate(a->E, a->vocab, a->d, a->W_A, a->W_H, a->r, a->h, a->verified, a->batch, a->block,
                   a->block_len, A_prev, G, ws + l.proj, l.g - l.proj, true, &g);
    if (st == DSEL_OK)
        st = plan_cand(a->E, a->vocab, a->d, a->W_A, a->W_B, a->r, a->cand_id, a->batch, a->block, a->block_len,
                       A_prev, B_cur, ws + l.proj, l.g - l.proj, &c);
    if (st == DSEL_OK)
        st = plan_pairs(a->cand_u, A_prev, B_cur, G, a->batch, a->block, a->block_len, a->r, S, walk, &q);
    if (st != DSEL_OK) return st;
    st = launch_gate_gemm(g, stream);
    if (st == DSEL_OK) st = launch_topk_and_gate_reduce(t, g, stream);
    if (st == DSEL_OK) st = launch_cand(c, stream);
    if (st == DSEL_OK) st = launch_pairs(q, stream);
    return st;
}

// ---- the whole selector without a caller workspace ---------------------------

namespace {

// The workspace of dsel_select_path_noalloc: one array per device, which the
// HIP runtime places when the library's code is loaded on that device and
// keeps until the process ends.  Host code never passes `scratch` itself to a
// kernel (its name is a host-side stand-in, not the device address); it uses
// the address hipGetSymbolAddress returns, looked up once per device.
constexpr size_t kScratchBytes = (size_t)DSEL_NOALLOC_MAX_WORKSPACE;
static __device__ __align__(256) unsigned char scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices] = {};

dsel_status scratch_for_current_device(void **out) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return DSEL_E_HIP;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void *ptr = nullptr;
        if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || !ptr) return DSEL_E_HIP;
        g_scratch_ptr[dev] = ptr;
    }
    *out = g_scratch_ptr[dev];
    return DSEL_OK;
}

}  // namespace

DSEL_API dsel_status dsel_select_path_noalloc(const dsel_path_args *a, const dsel_walk_args *walk,
                                              dsel_stream_t stream) {
    if (!a || !walk) return DSEL_E_ARG;
    if (a->batch < 0 || a->block < 1 || a->block > DSEL_MAX_BLOCK || a->batch > (int64_t)INT_MAX / a->block)
        return DSEL_E_ARG;
    size_t need = 0;
    if (a->batch > 0) {
        PathLayout l;
        if (!path_layout(a->batch, a->block, a->vocab, a->dt, a->d, a->r, &l)) return DSEL_E_ARG;
        need = l.total;
        if (need > kScratchBytes) return DSEL_E_WORKSPACE;  // beyond the fixed scratch array
    }
    void *ws = nullptr;
    if (need) {
        dsel_status st = scratch_for_current_device(&ws);
        if (st != DSEL_OK) return st;
    }
    return dsel_select_path(a, walk, ws, need ? kScratchBytes : 0, stream);
}

DSEL_API dsel_status dsel_device_error(int32_t *out_code, dsel_stream_t stream) {
    if (!out_code) return DSEL_E_ARG;
    if (hipStreamSynchronize((hipStream_t)stream) != hipSuccess) return DSEL_E_HIP;
    int v = 0, zero = 0;
    if (hipMemcpyFromSymbol(&v, HIP_SYMBOL(dsel::g_device_error), sizeof(int), 0,
                            hipMemcpyDeviceToHost) != hipSuccess)
        return DSEL_E_HIP;
    if (hipMemcpyToSymbol(HIP_SYMBOL(dsel::g_device_error), &zero, sizeof(int), 0,
                          hipMemcpyHostToDevice) != hipSuccess)
        return DSEL_E_HIP;
    *out_code = v;
    return DSEL_OK;
}

DSEL_API const char *dsel_status_string(dsel_status s) {
    switch (s) {
        case DSEL_OK: return "DSEL_OK";
        case DSEL_E_ARG: return "DSEL_E_ARG: invalid argument";
        case DSEL_E_DTYPE: return "DSEL_E_DTYPE: unknown dtype or walk mode";
        case DSEL_E_ALIGN: return "DSEL_E_ALIGN: misaligned pointer or leading dimension";
        case DSEL_E_WORKSPACE: return "DSEL_E_WORKSPACE: workspace missing or too small";
        case DSEL_E_HIP: return "DSEL_E_HIP: HIP runtime or launch failure";
    }
    return "unknown dsel status";
}

DSEL_API int32_t dsel_version(void) { return DSEL_VERSION; }

// ---- LM head with the top-16 ------------------------------------------------

DSEL_API size_t dsel_lmhead_topk_workspace_bytes(int64_t rows, int64_t vocab) {
    if (rows <= 0 || vocab < kK || vocab >= (int64_t)INT_MAX) return 0;
    return lmhead_workspace_bytes(rows, vocab);
}

DSEL_API dsel_status dsel_lmhead_topk(const uint16_t *h, const uint16_t *W, int64_t rows, int64_t vocab,
                                      int64_t d, int32_t *cand_id, float *cand_u, void *workspace,
                                      size_t workspace_bytes, dsel_stream_t stream) {
    if (rows < 0 || rows > (1 << 24) || vocab < kK || vocab >= (int64_t)INT_MAX || d < 64 || d % 64 != 0 ||
        d > (1 << 20))
        return DSEL_E_ARG;
    if (rows == 0) return DSEL_OK;
    if (!h || !W || !cand_id || !cand_u) return DSEL_E_ARG;
    if (!aligned(h, 16) || !aligned(W, 16) || !aligned(cand_id, 4) || !aligned(cand_u, 4)) return DSEL_E_ALIGN;
    const size_t need = lmhead_workspace_bytes(rows, vocab);
    if (!workspace || workspace_bytes < need) return DSEL_E_WORKSPACE;
    if (!aligned(workspace, 16)) return DSEL_E_ALIGN;
    LmheadParams p;
    p.h = h;
    p.W = W;
    p.R = rows;
    p.V = vocab;
    p.d = (int)d;
    p.mt = (int)((rows + 127) / 128);
    p.nct = (int)((vocab + kLmBN - 1) / kLmBN);
    p.nvs = lmhead_nvs(rows, vocab);
    p.cpw = (p.nct + p.nvs - 1) / p.nvs;
    p.partial = (uint64_t *)workspace;
    const int64_t grid = (int64_t)p.mt * p.nvs;
    if (grid >= (int64_t)INT_MAX) return DSEL_E_ARG;
    dsel_status st = launch((const void *)lmhead_topk_kernel, dim3((unsigned)grid), dim3(LmTile::NT), &p, 0, stream);
    if (st != DSEL_OK) return st;
    TopkParams tp;
    tp.logits = nullptr;
    tp.rows = rows;
    tp.V = vocab;
    tp.ld = vocab;
    tp.nsplit = p.nvs;
    tp.L = 1;
    tp.len = nullptr;
    tp.cand_id = cand_id;
    tp.cand_u = cand_u;
    tp.partial = p.partial;
    return launch((const void *)topk16_merge_kernel<true>, dim3((unsigned)rows), dim3(256), &tp, 0, stream);
}

// ---- dynamic short convolution ---------------------------------------------

DSEL_API size_t dsel_dyn_conv_workspace_bytes(int64_t batch, int64_t block, int64_t d) {
    if (batch <= 0 || block < 1 || d < 512 || d % 512 != 0 || d > (1 << 16)) return 0;
    return conv_workspace_bytes(batch, block, d);
}

DSEL_API dsel_status dsel_dyn_conv(const uint16_t *x, const uint16_t *x_prev, const uint16_t *base,
                                   const uint16_t *W_c, int64_t batch, int64_t block,
                                   const int32_t *block_len, int64_t d, uint16_t *y, void *workspace,
                                   size_t workspace_bytes, dsel_stream_t stream) {
    if (batch < 0 || block < 1 || d < 512 || d % 512 != 0 || d > (1 << 16)) return DSEL_E_ARG;
    if (batch > (int64_t)INT_MAX / block) return DSEL_E_ARG;
    if (batch == 0) return DSEL_OK;
    if (!x || !x_prev || !base || !W_c || !y) return DSEL_E_ARG;
    if (!aligned(x, 16) || !aligned(x_prev, 16) || !aligned(base, 16) || !aligned(W_c, 16) || !aligned(y, 16) ||
        !aligned(block_len, 4))
        return DSEL_E_ALIGN;
    const size_t need = conv_workspace_bytes(batch, block, d);
    if (!workspace || workspace_bytes < need) return DSEL_E_WORKSPACE;
    if (!aligned(workspace, 16)) return DSEL_E_ALIGN;
    ConvParams p;
    p.x = x;
    p.x_prev = x_prev;
    p.base = base;
    p.W_c = W_c;
    p.y = y;
    p.B = (int)batch;
    p.L = (int)block;
    p.len = block_len;
    p.d = (int)d;
    p.M = batch * block;
    p.N = (int)(d / 8);
    p.mt = (int)((p.M + 127) / 128);
    const int BN = conv_bn(p.M, p.N);
    p.nt = p.N / BN;
    p.nsplit = conv_nsplit(batch, block, d);
    p.part = (float *)workspace;
    const int64_t grid = (int64_t)p.mt * p.nt * p.nsplit;
    if (grid >= (int64_t)INT_MAX) return DSEL_E_ARG;
    const void *kc = BN == 256 ? (const void *)conv_corr_kernel<256> : (const void *)conv_corr_kernel<64>;
    dsel_status st = launch(kc, dim3((unsigned)grid), dim3(tile_threads(BN)), &p, 0, stream);
    if (st != DSEL_OK) return st;
    return launch((const void *)conv_apply_kernel, dim3((unsigned)p.M), dim3(256), &p,
                  (size_t)p.N * sizeof(float), stream);
}

// ---- the cache side of verifying a tree ---------------------------------------

namespace {

bool is_cache_type(dsel_dtype dt) { return dt == DSEL_BF16 || dt == DSEL_E4M3 || dt == DSEL_MXFP4; }

// Checks a cache and lays its strides out in 16-byte vectors.  A stride of an
// extent of one is never used and may be anything; so may the pointers of a call
// with no work.
dsel_status check_cache(const dsel_cache *c, bool work, CacheView *v) {
    if (!c) return DSEL_E_ARG;
    if (!is_cache_type(c->dt)) return DSEL_E_DTYPE;
    const bool fp4 = c->dt == DSEL_MXFP4;
    const int64_t per = c->dt == DSEL_BF16 ? 8 : fp4 ? 32 : 16;
    if (c->layers < 1 || c->layers > DSEL_MAX_LAYERS || c->heads < 1 || c->heads > DSEL_MAX_HEADS || c->dim < 1 ||
        c->dim > DSEL_MAX_HEAD_DIM || c->num_pages < 1 || c->num_pages > INT_MAX || c->page_size < 1 ||
        c->page_size > DSEL_MAX_PAGE)
        return DSEL_E_ARG;
    if (work && (!c->k || !c->v)) return DSEL_E_ARG;
    if (c->dt == DSEL_BF16 && (c->k_scale || c->v_scale)) return DSEL_E_ARG;
    if (work && fp4 && (!c->k_block || !c->v_block)) return DSEL_E_ARG;
    if (c->dim % per) return DSEL_E_ALIGN;
    if (work && (!aligned(c->k, 16) || !aligned(c->v, 16))) return DSEL_E_ALIGN;
    if (work && !fp4 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))) return DSEL_E_ALIGN;
    const int64_t extent[4] = {c->layers, c->num_pages, c->page_size, c->heads};
    const int64_t stride[4] = {c->layer_stride, c->page_stride, c->slot_stride, c->head_stride};
    int64_t st[4], reach = 0;
    for (int i = 0; i < 4; ++i) {
        st[i] = 0;
        if (extent[i] == 1) continue;
        if (stride[i] < c->dim || stride[i] > (INT64_MAX / 4 - reach) / extent[i]) return DSEL_E_ARG;
        if (stride[i] % per) return DSEL_E_ALIGN;
        st[i] = stride[i] / per;
        reach += stride[i] * (extent[i] - 1);
    }
    v->k = (char *)c->k;
    v->v = (char *)c->v;
    v->layers = (int)c->layers;
    v->heads = (int)c->heads;
    v->vecs = (int)(c->dim / per);
    v->layer_stride = st[0];
    v->page_stride = st[1];
    v->slot_stride = st[2];
    v->head_stride = st[3];
    v->num_pages = c->num_pages;
    v->page_size = (int)c->page_size;
    v->k_scale = fp4 ? nullptr : c->k_scale;
    v->v_scale = fp4 ? nullptr : c->v_scale;
    v->k_block = fp4 ? c->k_block : nullptr;
    v->v_block = fp4 ? c->v_block : nullptr;
    return DSEL_OK;
}

// K and V of a cache that is written, whose K and V go to different workgroups:
// two arrays, or one as both (`tied`) whose rows are then the same for both.  The
// scale bytes of 4-bit caches go with them.
dsel_status check_kv(const dsel_cache *c, bool tied) {
    const bool fp4 = c->dt == DSEL_MXFP4, one = tied && c->k == c->v;
    const int64_t row = fp4 ? c->dim / 2 : c->dim * (c->dt == DSEL_BF16 ? 2 : 1);
    if (fp4 && (one ? c->k_block != c->v_block : overlap(c->k_block, c->dim / 32, c->v_block, c->dim / 32)))
        return DSEL_E_ARG;
    return overlap(c->k, row, c->v, row) && !one ? DSEL_E_ARG : DSEL_OK;
}

// The batch that reads or writes a cache through its page table
dsel_status check_table(const int32_t *table, int64_t ld, int64_t max_pages, int64_t page_size,
                        const int32_t *seq_len, int64_t batch, int64_t block, const int32_t *block_len,
                        TableView *t) {
    if (max_pages < 1 || ld < max_pages || max_pages > (INT_MAX - DSEL_MAX_PAGE) / page_size ||
        ld > INT64_MAX / 8 / (batch + 1))
        return DSEL_E_ARG;
    if (batch == 0 || block == 0) return DSEL_OK;
    if (!table || !seq_len) return DSEL_E_ARG;
    if (!aligned(table, 4) || !aligned(seq_len, 4) || !aligned(block_len, 4)) return DSEL_E_ALIGN;
    t->table = table;
    t->ld = ld;
    t->max_pages = (int)max_pages;
    t->seq_len = seq_len;
    return DSEL_OK;
}

dsel_status check_tree(int64_t batch, int64_t block) {
    return batch < 0 || batch > DSEL_MAX_TREE_BATCH || block < 1 || block > DSEL_MAX_TREE ? DSEL_E_ARG : DSEL_OK;
}

}  // namespace

DSEL_API dsel_status dsel_tree_mask(const int32_t *parent, int64_t batch, int64_t block, const int32_t *block_len,
                                    int32_t *mask, int32_t *depth, dsel_stream_t stream) {
    dsel_status st = check_tree(batch, block);
    if (st != DSEL_OK) return st;
    if (batch == 0) return DSEL_OK;
    if (!parent || !mask) return DSEL_E_ARG;
    if (!aligned(parent, 4) || !aligned(mask, 4) || !aligned(depth, 4) || !aligned(block_len, 4)) return DSEL_E_ALIGN;
    TreeParams p{};
    p.parent = parent;
    p.T = (int)block;
    p.len = block_len;
    p.mask = mask;
    p.depth = depth;
    return launch((const void *)tree_mask_kernel, dim3((unsigned)batch), dim3((unsigned)(block + 63) / 64 * 64), &p, 0,
                  stream);
}

DSEL_API dsel_status dsel_tree_accept(const int32_t *parent, const int32_t *tok, const int32_t *target_tok,
                                      int64_t target_stride, int64_t batch, int64_t block, const int32_t *block_len,
                                      int32_t *n_keep, int32_t *path, int32_t *out_tok, dsel_stream_t stream) {
    dsel_status st = check_tree(batch, block);
    if (st != DSEL_OK) return st;
    if (target_stride < 1 || target_stride > (1 << 30)) return DSEL_E_ARG;
    if (batch == 0) return DSEL_OK;
    if (!parent || !tok || !target_tok || !n_keep || !path || !out_tok) return DSEL_E_ARG;
    if (!aligned(parent, 4) || !aligned(tok, 4) || !aligned(target_tok, 4) || !aligned(n_keep, 4) ||
        !aligned(path, 4) || !aligned(out_tok, 4) || !aligned(block_len, 4))
        return DSEL_E_ALIGN;
    TreeParams p{};
    p.parent = parent;
    p.tok = tok;
    p.target = target_tok;
    p.target_stride = target_stride;
    p.T = (int)block;
    p.len = block_len;
    p.n_keep = n_keep;
    p.path = path;
    p.out_tok = out_tok;
    return launch((const void *)tree_accept_kernel, dim3((unsigned)batch), dim3(64), &p, 0, stream);
}

namespace {

// The kernels of one shape: row waves by how many rows (nodes x query heads of
// a K/V head) there are, padded head dim by the head dim.
struct AttnKernels {
    const void *attn, *join;
    int threads, wgs, part, join_y;
};
template <class C>
AttnKernels attn_kernels(const void *attn) {
    using J = AttnJoin<C::E4M3, C::DP, C::ROWS>;
    return {attn, (const void *)tree_attn_join_kernel<J>, C::NT, kAttnCUs * C::WGS, C::PART, J::Y};
}
template <bool E4M3, bool WIN, int... X>
AttnKernels attn_of() {
    using C = AttnCfg<E4M3, WIN, X...>;
    return attn_kernels<C>((const void *)tree_attn_kernel<C>);
}
template <bool WIN, int... X>
AttnKernels attn4_of() {
    using C = Attn4Cfg<WIN, X...>;
    return attn_kernels<C>((const void *)tree_attn4_kernel<C>);
}
template <bool WIN, int... X>
AttnKernels attn4_few_of() {
    using C = Attn4FewCfg<WIN, X...>;
    return attn_kernels<C>((const void *)tree_attn4_few_kernel<C>);
}
template <bool E4M3, bool WIN>
AttnKernels attn_pick(int64_t rows, int64_t dim) {
    // an 8-bit tile of 64 keys and 64 columns is one LDS-DMA load for each of four waves
    constexpr int S = E4M3 ? 64 : 32, R = E4M3 ? 4 : 8;
    if (dim <= 64)
        return rows <= 32    ? attn_of<E4M3, WIN, 64, 1, 1, 4, 32, 2>()
               : rows <= 64  ? attn_of<E4M3, WIN, 64, 2, 1, 2, S, 2>()
               : rows <= 128 ? attn_of<E4M3, WIN, 64, 4, 1, 1, 64, 2>()
                             : attn_of<E4M3, WIN, 64, R, 1, 1, 64, 2>();
    if (dim <= 128)
        return rows <= 32    ? attn_of<E4M3, WIN, 128, 1, 1, 4, 32, 2>()
               : rows <= 64  ? attn_of<E4M3, WIN, 128, 2, 1, 2, S, 2>()
               : rows <= 128 ? attn_of<E4M3, WIN, 128, 4, 1, 1, 64, 2>()
                             : attn_of<E4M3, WIN, 128, 8, 1, 1, 64, 3>();
    return rows <= 32   ? attn_of<E4M3, WIN, 256, 1, 2, 2, 32, 2>()
           : rows <= 64 ? attn_of<E4M3, WIN, 256, 2, 2, 1, 32, 2>()
                        : attn_of<E4M3, WIN, 256, 4, 2, 1, 32, 3>();
}
template <bool WIN>
AttnKernels attn4_pick(int64_t rows, int64_t dim) {
    if (dim <= 64)
        return rows <= 16   ? attn4_few_of<WIN, 64, 1, 4>()
               : rows <= 32 ? attn4_few_of<WIN, 64, 2, 4>()
               : rows <= 64 ? attn4_of<WIN, 64, 2, 1, 2, 32>()
                            : attn4_of<WIN, 64, 4, 1, 1, 64>();
    if (dim <= 128)
        return rows <= 16   ? attn4_few_of<WIN, 128, 1, 4>()
               : rows <= 32 ? attn4_few_of<WIN, 128, 2, 4>()
               : rows <= 64 ? attn4_of<WIN, 128, 2, 1, 2, 32>()
                            : attn4_of<WIN, 128, 4, 1, 1, 64>();
    // (Two row tiles of 256 columns do not fit the registers: a kilobyte of a lane's were
    // kept in scratch, in the loop, and 8 tokens for each of 32 rows took 869 us, not 426.)
    return rows <= 16   ? attn4_few_of<WIN, 256, 1, 4>()
           : rows <= 64 ? attn4_of<WIN, 256, 2, 2, 1, 32>()
                        : attn4_of<WIN, 256, 4, 2, 1, 32>();
}
template <bool WIN>
AttnKernels attn_pick(dsel_dtype dt, int64_t rows, int64_t dim) {
    return dt == DSEL_MXFP4  ? attn4_pick<WIN>(rows, dim)
           : dt == DSEL_E4M3 ? attn_pick<true, WIN>(rows, dim)
                             : attn_pick<false, WIN>(rows, dim);
}

// Workspace of an attention whose rows see `keys` positions at most, and of which
// rows of up to `whole` are not split
size_t attn_workspace(const AttnKernels &k, int64_t keys, int64_t whole) {
    return keys <= whole ? 0 : (size_t)k.wgs * (2 * k.part + kJoinWords) * sizeof(float);
}
bool attn_sizes(int64_t batch, int64_t block, int64_t q_heads, int64_t kv_heads, int64_t dim, dsel_dtype dt) {
    return check_tree(batch, block) == DSEL_OK && batch > 0 && kv_heads >= 1 && q_heads >= 1 && q_heads <= DSEL_MAX_HEADS &&
           q_heads % kv_heads == 0 && dim >= 1 && dim <= DSEL_MAX_HEAD_DIM && is_cache_type(dt);
}
// What the nodes of a row see under a window, at most
int64_t window_keys(int64_t max_len, int64_t window, int64_t sinks, int64_t block) {
    return window >= max_len || sinks >= max_len ? max_len : max_len < window + sinks + block ? max_len : window + sinks + block;
}

// q's strides, those of extents of one as 0
dsel_status check_q(const dsel_tree_attn_args *a, int64_t sq[3]) {
    const int64_t extent[3] = {a->batch, a->block, a->q_heads}, stride[3] = {a->q_batch, a->q_token, a->q_head};
    for (int i = 0; i < 3; ++i) {
        sq[i] = 0;
        if (extent[i] == 1) continue;
        if (stride[i] < 0 || stride[i] > INT64_MAX / 16 / extent[i]) return DSEL_E_ARG;
        if (stride[i] % 8) return DSEL_E_ALIGN;
        sq[i] = stride[i];
    }
    return DSEL_OK;
}

int page_shift_of(int page_size) {
    return (page_size & (page_size - 1)) == 0 ? __builtin_ctz((unsigned)page_size) : -1;
}

template <bool WIN>
dsel_status tree_attn(const dsel_tree_attn_args *a, const dsel_cache *cache, int64_t window, int64_t sinks,
                      const int32_t *depth, void *workspace, size_t workspace_bytes, dsel_stream_t stream) {
    if (!a) return DSEL_E_ARG;
    dsel_status st = check_tree(a->batch, a->block);
    if (st != DSEL_OK) return st;
    TreeAttnParams p{};
    if ((st = check_cache(cache, a->batch > 0, &p.c)) != DSEL_OK) return st;
    if (cache->layers != 1 || a->q_heads < 1 || a->q_heads > DSEL_MAX_HEADS || a->q_heads % cache->heads)
        return DSEL_E_ARG;
    if (!(a->scale > 0.0f && a->scale <= 0x1p127f)) return DSEL_E_ARG;  // times log2(e) it is finite
    if (WIN && (window < 1 || sinks < 0)) return DSEL_E_ARG;
    if ((st = check_table(a->page_table, a->table_ld, a->max_pages, cache->page_size, a->seq_len, a->batch, a->block,
                          a->block_len, &p.t)) != DSEL_OK)
        return st;
    if (a->batch == 0) return DSEL_OK;
    if (!a->q || !a->out) return DSEL_E_ARG;
    if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->lse, 4) || !aligned(a->mask, 4) || !aligned(depth, 4))
        return DSEL_E_ALIGN;
    int64_t sq[3];
    if ((st = check_q(a, sq)) != DSEL_OK) return st;
    const int64_t rows = a->block * (a->q_heads / cache->heads), max_len = a->max_pages * cache->page_size;
    const AttnKernels k = attn_pick<WIN>(cache->dt, rows, cache->dim);
    const size_t need = WIN ? attn_workspace(k, window_keys(max_len, window, sinks, a->block), kWindowWholeKeys)
                            : attn_workspace(k, max_len, kAttnWholeKeys);
    if (need && (!workspace || workspace_bytes < need)) return DSEL_E_WORKSPACE;
    if (need && !aligned(workspace, 16)) return DSEL_E_ALIGN;
    p.q = (const char *)a->q;
    p.sqb = sq[0];
    p.sqt = sq[1];
    p.sqh = sq[2];
    p.out = a->out;
    p.lse = a->lse;
    p.mask = a->mask;
    p.len = a->block_len;
    p.B = (int)a->batch;
    p.T = (int)a->block;
    p.Hq = (int)a->q_heads;
    p.D = (int)cache->dim;
    p.group = (int)(a->q_heads / cache->heads);
    p.words = (int)(a->block + 31) / 32;
    p.scale = (float)((double)a->scale * 1.4426950408889634);
    p.window = (int)(window < INT_MAX ? window : INT_MAX);
    p.sinks = (int)(sinks < INT_MAX ? sinks : INT_MAX);
    p.depth = depth;
    p.page_shift = page_shift_of(p.c.page_size);
    p.part = (float *)workspace;
    p.wgs = k.wgs;
    p.whole = need == 0;
    p.join = (int32_t *)(p.part + (int64_t)k.wgs * 2 * k.part);
    st = launch(k.attn, dim3((unsigned)k.wgs), dim3((unsigned)k.threads), &p, 0, stream);
    if (st != DSEL_OK || p.whole) return st;
    return launch(k.join, dim3((unsigned)k.wgs, (unsigned)k.join_y), dim3(256), &p, 0, stream);
}

}  // namespace

DSEL_API size_t dsel_tree_attn_workspace_bytes(int64_t batch, int64_t block, int64_t q_heads, int64_t kv_heads,
                                               int64_t dim, dsel_dtype dt, int64_t max_len) {
    if (!attn_sizes(batch, block, q_heads, kv_heads, dim, dt)) return 0;
    return attn_workspace(attn_pick<false>(dt, block * (q_heads / kv_heads), dim), max_len, kAttnWholeKeys);
}

DSEL_API dsel_status dsel_tree_attn(const dsel_tree_attn_args *a, const dsel_cache *cache, void *workspace,
                                    size_t workspace_bytes, dsel_stream_t stream) {
    return tree_attn<false>(a, cache, 1, 0, nullptr, workspace, workspace_bytes, stream);
}

DSEL_API size_t dsel_tree_attn_window_workspace_bytes(int64_t batch, int64_t block, int64_t q_heads, int64_t kv_heads,
                                                      int64_t dim, dsel_dtype dt, int64_t max_len, int64_t window,
                                                      int64_t sinks) {
    if (!attn_sizes(batch, block, q_heads, kv_heads, dim, dt) || window < 1 || sinks < 0) return 0;
    return attn_workspace(attn_pick<true>(dt, block * (q_heads / kv_heads), dim), window_keys(max_len, window, sinks, block),
                          kWindowWholeKeys);
}

DSEL_API dsel_status dsel_tree_attn_window(const dsel_tree_attn_args *a, const dsel_cache *cache, int64_t window,
                                           int64_t sinks, const int32_t *depth, void *workspace, size_t workspace_bytes,
                                           dsel_stream_t stream) {
    return tree_attn<true>(a, cache, window, sinks, depth, workspace, workspace_bytes, stream);
}

DSEL_API dsel_status dsel_cache_append(const uint16_t *k_new, const uint16_t *v_new, const int64_t strides[4],
                                       const dsel_cache *cache, const int32_t *page_table, int64_t table_ld,
                                       int64_t max_pages, const int32_t *seq_len, int64_t batch, int64_t block,
                                       const int32_t *block_len, dsel_stream_t stream) {
    if (batch < 0 || batch > DSEL_MAX_TREE_BATCH || block < 0 || block > DSEL_MAX_APPEND) return DSEL_E_ARG;
    AppendParams p{};
    dsel_status st = check_cache(cache, batch > 0 && block > 0, &p.c);
    if (st != DSEL_OK) return st;
    if ((st = check_table(page_table, table_ld, max_pages, cache->page_size, seq_len, batch, block, block_len, &p.t)) !=
        DSEL_OK)
        return st;
    if (batch == 0 || block == 0) return DSEL_OK;
    if (!k_new || !v_new || !strides) return DSEL_E_ARG;
    if (!aligned(k_new, 16) || !aligned(v_new, 16)) return DSEL_E_ALIGN;
    const int64_t extent[4] = {cache->layers, batch, block, cache->heads};
    int64_t sn[4];
    for (int i = 0; i < 4; ++i) {
        sn[i] = 0;
        if (extent[i] == 1) continue;
        if (strides[i] < 0 || strides[i] > INT64_MAX / 16 / extent[i]) return DSEL_E_ARG;
        if (strides[i] % 8) return DSEL_E_ALIGN;
        sn[i] = strides[i] / 8;
    }
    p.k = (const char *)k_new;
    p.v = (const char *)v_new;
    p.sl = sn[0];
    p.sb = sn[1];
    p.st = sn[2];
    p.sh = sn[3];
    p.T = (int)block;
    p.len = block_len;
    if ((st = check_kv(cache, k_new == v_new && cache->k_scale == cache->v_scale)) != DSEL_OK) return st;
    const void *k = cache->dt == DSEL_MXFP4  ? (const void *)cache_append_kernel<kMxfp4>
                    : cache->dt == DSEL_E4M3 ? (const void *)cache_append_kernel<kE4m3>
                                             : (const void *)cache_append_kernel<kBf16>;
    return launch(k, dim3((unsigned)((block + kAppendTokens - 1) / kAppendTokens), (unsigned)cache->layers * 2,
                          (unsigned)batch), dim3(256), &p, 0, stream);
}

DSEL_API dsel_status dsel_cache_compact(const dsel_cache *cache, const int32_t *page_table, int64_t table_ld,
                                        int64_t max_pages, const int32_t *seq_len, const int32_t *path,
                                        const int32_t *n_keep, int64_t batch, int64_t block, int32_t *new_len,
                                        dsel_stream_t stream) {
    dsel_status st = check_tree(batch, block);
    if (st != DSEL_OK) return st;
    CompactParams p{};
    if ((st = check_cache(cache, batch > 0, &p.c)) != DSEL_OK) return st;
    if ((st = check_table(page_table, table_ld, max_pages, cache->page_size, seq_len, batch, block, nullptr, &p.t)) !=
        DSEL_OK)
        return st;
    if (batch == 0) return DSEL_OK;
    if (!path || !n_keep || !new_len) return DSEL_E_ARG;
    if (!aligned(path, 4) || !aligned(n_keep, 4) || !aligned(new_len, 4)) return DSEL_E_ALIGN;
    // a row's first workgroup writes new_len while its others still read these
    const int64_t nb = batch * (int64_t)sizeof(int32_t);
    if (overlap(new_len, nb, seq_len, nb) || overlap(new_len, nb, n_keep, nb) || overlap(new_len, nb, path, nb * block) ||
        overlap(new_len, nb, page_table, ((batch - 1) * table_ld + max_pages) * (int64_t)sizeof(int32_t)))
        return DSEL_E_ARG;
    if ((st = check_kv(cache, true)) != DSEL_OK) return st;
    p.kinds = cache->k == cache->v ? 1 : 2;
    p.path = path;
    p.n_keep = n_keep;
    p.new_len = new_len;
    p.T = (int)block;
    const int64_t vecs = (int64_t)p.kinds * p.c.layers * p.c.heads * p.c.vecs;
    return launch((const void *)cache_compact_kernel, dim3((unsigned)((vecs + 255) / 256), (unsigned)batch), dim3(256),
                  &p, 0, stream);
}

namespace {

dsel_status check_pages(const dsel_pages *g, const int32_t *arg, PoolParams *p) {
    if (!g) return DSEL_E_ARG;
    if (g->rows < 0 || g->rows > DSEL_MAX_ROWS || g->max_pages < 1 || g->table_ld < g->max_pages ||
        g->num_pages < 1 || g->num_pages > INT_MAX - 32768 || g->page_size < 1 || g->page_size > DSEL_MAX_PAGE ||
        g->max_pages > (INT_MAX - DSEL_MAX_PAGE) / g->page_size || g->table_ld > INT64_MAX / 8 / DSEL_MAX_ROWS)
        return DSEL_E_ARG;
    if (g->rows == 0) return DSEL_OK;
    if (!g->table || !g->row_pages || !g->seq_len || !g->refcount || !arg) return DSEL_E_ARG;
    if (!aligned(g->table, 4) || !aligned(g->row_pages, 4) || !aligned(g->seq_len, 4) || !aligned(g->refcount, 4) ||
        !aligned(arg, 4))
        return DSEL_E_ALIGN;
    p->table = g->table;
    p->ld = g->table_ld;
    p->rows = (int)g->rows;
    p->max_pages = (int)g->max_pages;
    p->row_pages = g->row_pages;
    p->seq_len = g->seq_len;
    p->refcount = g->refcount;
    p->num_pages = g->num_pages;
    p->page_size = (int)g->page_size;
    p->arg = arg;
    return DSEL_OK;
}

}  // namespace

DSEL_API dsel_status dsel_pages_reserve(const dsel_pages *pages, const int32_t *extra, int32_t *granted,
                                        dsel_stream_t stream) {
    PoolParams p{};
    dsel_status st = check_pages(pages, extra, &p);
    if (st != DSEL_OK || pages->rows == 0) return st;
    if (!granted) return DSEL_E_ARG;
    if (!aligned(granted, 4)) return DSEL_E_ALIGN;
    p.granted = granted;
    return launch((const void *)pool_give_kernel<kMore>, dim3(1), dim3(1024), &p, 0, stream);
}

DSEL_API size_t dsel_pages_fork_workspace_bytes(int64_t rows) {
    return rows <= 0 || rows > DSEL_MAX_ROWS ? 0 : (size_t)rows * sizeof(int32_t);
}

DSEL_API dsel_status dsel_pages_fork(const dsel_pages *pages, const int32_t *src, const dsel_cache *cache,
                                     int32_t *granted, void *workspace, size_t workspace_bytes, dsel_stream_t stream) {
    PoolParams p{};
    CacheView c{};
    dsel_status st = check_pages(pages, src, &p);
    if (st != DSEL_OK) return st;
    if ((st = check_cache(cache, pages->rows > 0, &c)) != DSEL_OK) return st;
    if (cache->num_pages != pages->num_pages || cache->page_size != pages->page_size) return DSEL_E_ARG;
    if (pages->rows == 0) return DSEL_OK;
    if (!granted) return DSEL_E_ARG;
    if (!aligned(granted, 4)) return DSEL_E_ALIGN;
    if (!workspace || workspace_bytes < dsel_pages_fork_workspace_bytes(pages->rows)) return DSEL_E_WORKSPACE;
    if (!aligned(workspace, 4)) return DSEL_E_ALIGN;
    if ((st = check_kv(cache, true)) != DSEL_OK) return st;
    p.granted = granted;
    p.plan = (int32_t *)workspace;
    st = launch((const void *)pool_give_kernel<kFork>, dim3(1), dim3(1024), &p, 0, stream);
    if (st != DSEL_OK) return st;
    const int chunks = (c.page_size + kForkSlots - 1) / kForkSlots;
    void *args[] = {&p, &c};
    return hipLaunchKernel((const void *)pages_fork_kernel, dim3((unsigned)(1 + 2 * c.layers * chunks), (unsigned)p.rows),
                           dim3(256), args, 0, (hipStream_t)stream) == hipSuccess ? DSEL_OK : DSEL_E_HIP;
}

DSEL_API dsel_status dsel_pages_free(const dsel_pages *pages, const int32_t *which, dsel_stream_t stream) {
    PoolParams p{};
    dsel_status st = check_pages(pages, which, &p);
    if (st != DSEL_OK || pages->rows == 0) return st;
    return launch((const void *)pages_free_kernel, dim3((unsigned)p.rows), dim3(256), &p, 0, stream);
}

// ---- key weights and eviction -------------------------------------------------

namespace {

template <CacheType F, int NK>
const void *key_weights_of(int64_t dim) {
    return dim <= 64    ? (const void *)key_weights_kernel<KeyWeightsCfg<F, 64, NK>>
           : dim <= 128 ? (const void *)key_weights_kernel<KeyWeightsCfg<F, 128, NK>>
                        : (const void *)key_weights_kernel<KeyWeightsCfg<F, 256, NK>>;
}
template <CacheType F>
const void *key_weights_pick(int64_t dim, bool many) {
    return many ? key_weights_of<F, 4>(dim) : key_weights_of<F, 1>(dim);
}

int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }

// Workgroups for each of `rows` rows that a table gives `most` pieces of work at
// most: one each, up to 2^16 in all (a piece may be as little as a few hundred
// cycles, and most of a wide table's are none), beyond which they take several.
int64_t wgs_for(int64_t most, int64_t rows) {
    const int64_t cap = rows < 65536 ? 65536 / rows : 1;
    return most < cap ? most : cap;
}

}  // namespace

DSEL_API dsel_status dsel_key_weights(const dsel_tree_attn_args *a, const dsel_cache *cache, const float *count,
                                      float decay, float *weights, int64_t weights_ld, dsel_stream_t stream) {
    if (!a) return DSEL_E_ARG;
    dsel_status st = check_tree(a->batch, a->block);
    if (st != DSEL_OK) return st;
    KeyWeightsParams p{};
    if (!cache) return DSEL_E_ARG;
    dsel_cache c = *cache;  // V is not looked at
    c.v = c.k;
    c.v_scale = c.k_scale;
    if ((st = check_cache(&c, a->batch > 0, &p.c)) != DSEL_OK) return st;
    if (c.layers != 1 || a->q_heads < 1 || a->q_heads > DSEL_MAX_HEADS || a->q_heads % c.heads) return DSEL_E_ARG;
    if (!(a->scale > 0.0f && a->scale <= 0x1p127f)) return DSEL_E_ARG;
    if (!(decay >= 0.0f && decay <= 1.0f)) return DSEL_E_ARG;
    if ((st = check_table(a->page_table, a->table_ld, a->max_pages, c.page_size, a->seq_len, a->batch, a->block,
                          a->block_len, &p.t)) != DSEL_OK)
        return st;
    const int64_t max_len = a->max_pages * c.page_size;
    if (weights_ld < max_len || weights_ld > INT64_MAX / 8 / (a->batch + 1)) return DSEL_E_ARG;
    if (a->batch == 0) return DSEL_OK;
    if (!a->q || !a->lse || !weights) return DSEL_E_ARG;
    if (!aligned(a->q, 16) || !aligned(a->lse, 4) || !aligned(count, 4) || !aligned(weights, 4)) return DSEL_E_ALIGN;
    int64_t sq[3];
    if ((st = check_q(a, sq)) != DSEL_OK) return st;
    const int64_t tokens = a->batch * a->block * 4, col = a->batch * 4;
    const Span out = {weights, max_len * 4, a->batch, weights_ld * 4};
    for (const Span &in : {Span{a->lse, tokens * a->q_heads}, Span{count, tokens}, Span{a->seq_len, col}, Span{a->block_len, col},
                           Span{a->page_table, a->max_pages * 4, a->batch, a->table_ld * 4}})
        if (overlap(out, in)) return DSEL_E_ARG;
    p.q = (const char *)a->q;
    p.sqb = sq[0];
    p.sqt = sq[1];
    p.sqh = sq[2];
    p.lse = a->lse;
    p.count = count;
    p.w = weights;
    p.ld = weights_ld;
    p.len = a->block_len;
    p.B = (int)a->batch;
    p.T = (int)a->block;
    p.Hq = (int)a->q_heads;
    p.D = (int)c.dim;
    p.group = (int)(a->q_heads / c.heads);
    p.scale = a->scale;
    p.decay = decay;
    p.page_shift = page_shift_of(p.c.page_size);
    // 64 keys a wave, two waves to a head's keys, where that makes two workgroups a CU.
    // (By what the table holds: lengths are on the device.  One token over 700 positions
    // takes 14.5 us instead of 6.2 where the table has room for 65,536 or more.)
    const bool many = a->batch * ((max_len + 127) / 128) >= 2 * kAttnCUs;
    p.hs = c.heads >= 4 && !many ? 4 : c.heads >= 2 ? 2 : 1;
    const void *k = c.dt == DSEL_MXFP4  ? key_weights_pick<kMxfp4>(c.dim, many)
                    : c.dt == DSEL_E4M3 ? key_weights_pick<kE4m3>(c.dim, many)
                                        : key_weights_pick<kBf16>(c.dim, many);
    const int64_t keys = 4 / p.hs * (many ? 64 : 16), wgs = wgs_for((max_len + keys - 1) / keys, a->batch);
    return launch(k, dim3((unsigned)wgs, (unsigned)a->batch), dim3(256), &p, 0, stream);
}

// The workspace: pages wanted and lengths [rows], the pages handed out [rows]
// [max_pages], the positions kept and their weights [rows][max_len], each rounded up
// to 16 bytes.
DSEL_API size_t dsel_cache_evict_workspace_bytes(int64_t rows, int64_t max_len, int64_t page_size) {
    if (rows <= 0 || rows > DSEL_MAX_ROWS || page_size < 1 || page_size > DSEL_MAX_PAGE || max_len < page_size ||
        max_len % page_size || max_len > INT_MAX - DSEL_MAX_PAGE)
        return 0;
    return (size_t)(2 * up16(rows * 4) + up16(rows * (max_len / page_size) * 4) + 2 * up16(rows * max_len * 4));
}

DSEL_API dsel_status dsel_cache_evict(const dsel_pages *pages, const int32_t *budget, float *weights, int64_t weights_ld,
                                      int64_t sinks, int64_t recent, const dsel_cache *cache, int32_t *kept,
                                      int32_t *granted, void *workspace, size_t workspace_bytes, dsel_stream_t stream) {
    EvictParams p{};
    dsel_status st = check_pages(pages, budget, &p.g);
    if (st != DSEL_OK) return st;
    if ((st = check_cache(cache, pages->rows > 0, &p.c)) != DSEL_OK) return st;
    if (cache->num_pages != pages->num_pages || cache->page_size != pages->page_size) return DSEL_E_ARG;
    const int64_t max_len = pages->max_pages * pages->page_size;
    if (sinks < 0 || recent < 0 || weights_ld < max_len || weights_ld > INT64_MAX / 8 / DSEL_MAX_ROWS) return DSEL_E_ARG;
    if (pages->rows == 0) return DSEL_OK;
    if (!weights || !granted) return DSEL_E_ARG;
    if (!aligned(weights, 4) || !aligned(kept, 4) || !aligned(granted, 4)) return DSEL_E_ALIGN;
    const size_t need = dsel_cache_evict_workspace_bytes(pages->rows, max_len, pages->page_size);
    if (!workspace || workspace_bytes < need) return DSEL_E_WORKSPACE;
    if (!aligned(workspace, 16)) return DSEL_E_ALIGN;
    if ((st = check_kv(cache, true)) != DSEL_OK) return st;
    // one launch writes what others still read
    const int64_t col = pages->rows * 4, ld = weights_ld * 4;
    const Span all[] = {{weights, max_len * 4, pages->rows, ld}, {kept, max_len * 4, pages->rows, ld},
                        {budget, col}, {granted, 4}, {workspace, (int64_t)need},
                        {pages->table, pages->max_pages * 4, pages->rows, pages->table_ld * 4},
                        {pages->row_pages, col}, {pages->seq_len, col}, {pages->refcount, pages->num_pages * 4}};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 9; ++j)
            if (overlap(all[i], all[j])) return DSEL_E_ARG;
    p.budget = budget;
    p.weights = weights;
    p.ld = weights_ld;
    p.sinks = (int)(sinks < INT_MAX ? sinks : INT_MAX);
    p.recent = (int)(recent < INT_MAX ? recent : INT_MAX);
    char *at = (char *)workspace;
    auto part = [&](int64_t bytes) {
        char *const x = at;
        at += up16(bytes);
        return x;
    };
    p.need = (int32_t *)part(pages->rows * 4);
    p.len = (int32_t *)part(pages->rows * 4);
    p.g.plan = (int32_t *)part(pages->rows * pages->max_pages * 4);
    p.moved = (float *)part(pages->rows * max_len * 4);
    p.moved_ld = max_len;
    p.list = kept ? kept : (int32_t *)part(pages->rows * max_len * 4);
    p.list_ld = kept ? weights_ld : max_len;
    p.kinds = cache->k == cache->v ? 1 : 2;
    p.g.granted = granted;
    if ((st = launch((const void *)evict_plan_kernel, dim3((unsigned)pages->rows), dim3(1024), &p, 0, stream)) != DSEL_OK)
        return st;
    PoolParams g = p.g;
    g.arg = p.need;
    if ((st = launch((const void *)pool_give_kernel<kCut>, dim3(1), dim3(1024), &g, 0, stream)) != DSEL_OK) return st;
    const int64_t parts = p.kinds * cache->layers, runs = wgs_for((max_len + kEvictRows - 1) / kEvictRows, parts * pages->rows);
    st = launch((const void *)evict_copy_kernel, dim3((unsigned)runs, (unsigned)parts + 1, (unsigned)pages->rows), dim3(256),
                &p, 0, stream);
    if (st != DSEL_OK) return st;
    return launch((const void *)evict_finish_kernel, dim3(1 + kEvictParts, (unsigned)pages->rows), dim3(1024), &p, 0, stream);
}

// ---- verify ----------------------------------------------------------------

DSEL_API size_t dsel_verify_workspace_bytes(int64_t batch, int64_t block, int64_t vocab) {
    if (batch <= 0 || block < 1 || block > DSEL_MAX_BLOCK || vocab < kK ||
        vocab > kVMaxVocab)
        return 0;
    return verify_workspace_bytes(batch, block, vocab);
}

DSEL_API dsel_status dsel_verify(const void *target_logits, dsel_dtype dt, int64_t batch,
                                 int64_t block, const int32_t *block_len, int64_t vocab, int64_t ld,
                                 const int32_t *cand_id,
                                 const int32_t *path_slot, const float *q, dsel_walk_mode mode,
                                 float temperature, const float *u_acc, const float *u_res,
                                 int32_t *n_accepted, int32_t *out_tok, void *workspace,
                                 size_t workspace_bytes, dsel_stream_t stream) {
    if (dt != DSEL_F32 && dt != DSEL_BF16) return DSEL_E_DTYPE;
    if (mode != DSEL_GREEDY && mode != DSEL_SAMPLED) return DSEL_E_DTYPE;
    if (batch < 0 || batch >= (int64_t)INT_MAX / (DSEL_MAX_BLOCK + 1) || block < 1 || block > DSEL_MAX_BLOCK)
        return DSEL_E_ARG;
    if (vocab < kK || vocab > kVMaxVocab || ld < vocab) return DSEL_E_ARG;
    if (mode == DSEL_SAMPLED && !(temperature > 0.0f && temperature < __builtin_inff())) return DSEL_E_ARG;
    if (batch == 0) return DSEL_OK;
    if (!target_logits || !cand_id || !path_slot || !n_accepted || !out_tok) return DSEL_E_ARG;
    if (mode == DSEL_SAMPLED && (!q || !u_acc || !u_res)) return DSEL_E_ARG;
    const int64_t es = dt == DSEL_BF16 ? 2 : 4;
    const int64_t rows = batch * (block + 1);
    if (ld > INT64_MAX / es / rows) return DSEL_E_ARG;
    if (!aligned(target_logits, 16) || (ld * es) % 16 != 0) return DSEL_E_ALIGN;
    if (!aligned(cand_id, 4) || !aligned(path_slot, 4) || !aligned(n_accepted, 4) || !aligned(out_tok, 4) ||
        (q && !aligned(q, 4)) || (u_acc && !aligned(u_acc, 4)) || (u_res && !aligned(u_res, 4)) ||
        !aligned(block_len, 4))
        return DSEL_E_ALIGN;
    const size_t need = verify_workspace_bytes(batch, block, vocab);
    if (!workspace || workspace_bytes < need) return DSEL_E_WORKSPACE;
    if (!aligned(workspace, 16)) return DSEL_E_ALIGN;

    VerifyParams p;
    p.logits = (const char *)target_logits;
    p.V = vocab;
    p.ld = ld;
    p.B = (int)batch;
    p.L = (int)block;
    p.len = block_len;
    p.scale = mode == DSEL_SAMPLED ? (float)(1.4426950408889634 / (double)temperature) : 0.0f;
    p.cand_id = cand_id;
    p.path_slot = path_slot;
    p.q = q;
    p.u_acc = u_acc;
    p.u_res = u_res;
    p.n_acc = n_accepted;
    p.out_tok = out_tok;
    const bool bf = dt == DSEL_BF16, sm = mode == DSEL_SAMPLED;
    // chunks of 256 16-byte vectors; enough workgroups per row for about 2048
    // in all (8 per CU), at most kVMaxSplit, none of them empty
    const int64_t chunk_tokens = (int64_t)kVChunkVecs * (bf ? 8 : 4);
    p.nchunk = (int)((vocab + chunk_tokens - 1) / chunk_tokens);
    int64_t ns = (DSEL_VERIFY_WGS + rows - 1) / rows;
    ns = ns < 1 ? 1 : ns > kVMaxSplit ? kVMaxSplit : ns;
    ns = ns < p.nchunk ? ns : p.nchunk;
    p.cps = (int)((p.nchunk + ns - 1) / ns);
    p.nsplit = (p.nchunk + p.cps - 1) / p.cps;
    if (rows * p.nsplit > (int64_t)INT_MAX) return DSEL_E_ARG;
    p.part = (VerifyPart *)workspace;
    p.chunk = (float2 *)((char *)workspace + verify_part_bytes(batch, block));
    const void *k1 = bf ? (sm ? (const void *)verify_stats_kernel<true, true> : (const void *)verify_stats_kernel<true, false>)
                        : (sm ? (const void *)verify_stats_kernel<false, true> : (const void *)verify_stats_kernel<false, false>);
    const void *k2 = bf ? (sm ? (const void *)verify_draw_kernel<true, true> : (const void *)verify_draw_kernel<true, false>)
                        : (sm ? (const void *)verify_draw_kernel<false, true> : (const void *)verify_draw_kernel<false, false>);
    dsel_status st = launch(k1, dim3((unsigned)(rows * p.nsplit)), dim3(256), &p, 0, stream);
    if (st != DSEL_OK) return st;
    return launch(k2, dim3((unsigned)batch), dim3(256), &p, 0, stream);
}
