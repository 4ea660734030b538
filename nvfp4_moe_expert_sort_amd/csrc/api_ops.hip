// api_ops.hip -- host side of the entry points beside the expert forward:
// router logits, expert selection and its gradient, the balance loss and its
// gradient, the MXFP4 quantizer and products, low-rank adapters and their
// gradients, and gradient clipping.  Argument checks (before any launch),
// workspace carving and launches; include/nvfp4moe.h documents each.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "../../include/nvfp4moe.h"
#include "nvfp4_kernels.h"

using namespace nvfp4;

namespace {

static_assert(kBalanceOneLaunch == NVFP4MOE_BALANCE_ONE_LAUNCH && kBalanceOneLogits == NVFP4MOE_BALANCE_ONE_LAUNCH_LOGITS &&
                  kBalanceOneSequences == NVFP4MOE_BALANCE_ONE_LAUNCH_SEQUENCES,
              "the header's constants");

constexpr size_t kAlign = 256;
size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_E_HIP; }

int select_params(const nvfp4moe_select_config* c, const void* logits, int64_t ld, int64_t T, const float* bias,
                  SelectParams* P) {
    if (!c) return NVFP4_E_NULL;
    if (c->score != NVFP4MOE_SCORE_SOFTMAX && c->score != NVFP4MOE_SCORE_SIGMOID) return NVFP4_E_ARG;
    if (c->renormalize != 0 && c->renormalize != 1) return NVFP4_E_ARG;
    if (c->group_score != NVFP4MOE_GROUP_MAX && c->group_score != NVFP4MOE_GROUP_TOP2) return NVFP4_E_ARG;
    if (c->logits_type != NVFP4MOE_F32 && c->logits_type != NVFP4MOE_BF16) return NVFP4_E_ARG;
    if (!std::isfinite(c->scale)) return NVFP4_E_ARG;
    if (c->n_experts < 1 || c->n_experts > kMaxExperts) return NVFP4_E_SHAPE;
    if (c->n_groups < 1 || c->n_groups > kMaxGroups || c->n_experts % c->n_groups != 0) return NVFP4_E_SHAPE;
    if (c->top_groups < 1 || c->top_groups > c->n_groups) return NVFP4_E_SHAPE;
    const int32_t size = c->n_experts / c->n_groups;
    if (c->top_k < 1 || c->top_k > kMaxTopK || c->top_k > c->top_groups * size) return NVFP4_E_SHAPE;
    if (T < 0 || T >= ((int64_t)1 << 31) || ld < c->n_experts) return NVFP4_E_SHAPE;
    const size_t elem = c->logits_type == NVFP4MOE_BF16 ? 2 : 4;
    if (!aligned(logits, elem) || !aligned(bias, 4)) return NVFP4_E_ALIGN;
    *P = SelectParams{};
    P->logits = logits;
    P->ld = ld;
    P->T = T;
    P->E = c->n_experts;
    P->K = c->top_k;
    P->bias = bias;
    P->sigmoid = c->score == NVFP4MOE_SCORE_SIGMOID;
    P->renorm = c->renormalize != 0;
    P->top2 = c->group_score == NVFP4MOE_GROUP_TOP2;
    P->vec = ld % 4 == 0 && aligned(logits, 4 * elem);
    P->vec_bias = aligned(bias, 16);
    P->scale = c->scale;
    P->n_groups = c->n_groups;
    P->group_size = size;
    P->top_groups = c->top_groups;
    P->group_magic = ((1u << 22) + (uint32_t)size - 1) / (uint32_t)size;
    return NVFP4_OK;
}

int balance_params(const nvfp4moe_balance_config* c, const void* logits, int64_t ld, int64_t T, const int32_t* offsets,
                   int32_t S, BalanceParams* P) {
    if (!c) return NVFP4_E_NULL;
    if (c->score != NVFP4MOE_SCORE_SOFTMAX && c->score != NVFP4MOE_SCORE_SIGMOID) return NVFP4_E_ARG;
    if (c->logits_type != NVFP4MOE_F32 && c->logits_type != NVFP4MOE_BF16) return NVFP4_E_ARG;
    if (!std::isfinite(c->coef)) return NVFP4_E_ARG;
    if (c->n_experts < 1 || c->n_experts > kMaxExperts || c->top_k < 1 || c->top_k > kMaxTopK) return NVFP4_E_SHAPE;
    if (S < 1 || S > kMaxSequences || (!offsets && S != 1)) return NVFP4_E_SHAPE;
    if (T < 0 || T >= ((int64_t)1 << 31) || ld < c->n_experts) return NVFP4_E_SHAPE;
    const size_t elem = c->logits_type == NVFP4MOE_BF16 ? 2 : 4;
    if (!aligned(logits, elem) || !aligned(offsets, 4)) return NVFP4_E_ALIGN;
    *P = BalanceParams{};
    P->logits = logits;
    P->ld = ld;
    P->T = T;
    P->E = c->n_experts;
    P->K = c->top_k;
    P->S = S;
    P->offsets = offsets;
    P->coef = c->coef;
    P->sigmoid = c->score == NVFP4MOE_SCORE_SIGMOID;
    P->vec = ld % 4 == 0 && aligned(logits, 4 * elem);
    return NVFP4_OK;
}
// Workspace of the loss: the chunks' sums and counts, the shares of the loss, a counter.
struct BalanceWork {
    size_t csum, part, done, total;
};
bool balance_work(int64_t T, int64_t E, int64_t S, BalanceWork* w) {
    if (T < 0 || T >= ((int64_t)1 << 31) || E < 1 || E > kMaxExperts || S < 1 || S > kMaxSequences) return false;
    // the most chunks that T rows or fewer have (balance_chunk)
    const int64_t slots = std::max({std::min<int64_t>((T + 15) / 16, 512), (T + 255) / 256, std::min<int64_t>((T + 15) / 16, S / 2 + 1)}) + S;
    w->csum = up(slots * E * 4, kAlign);
    w->part = 2 * w->csum;
    w->done = w->part + up(S * ((E + 63) / 64) * 8, kAlign);
    w->total = w->done + kAlign;
    return true;
}

struct MxShape {
    int64_t row_tiles, chunks, quads;
};
MxShape mx_shape(const nvfp4moe_mxfp4_tensor* q) {
    const int64_t chunks = ((int64_t)q->cols + 127) / 128;
    return {((int64_t)q->rows + 15) / 16, chunks, (chunks + 3) / 4};
}
// Shape, size and layout of a tensor (its pointers are checked where they are used).
int mx_tensor(const nvfp4moe_mxfp4_tensor* q) {
    if (!q) return NVFP4_E_NULL;
    if (q->layout != NVFP4_LAYOUT_LOGICAL && q->layout != NVFP4_LAYOUT_GEMM) return NVFP4_E_ARG;
    if (q->n_mats < 0 || q->rows < 0 || q->cols <= 0 || q->cols % 32 != 0) return NVFP4_E_SHAPE;
    // the padded matrices too, so that every index of the kernels stays in its type
    const int64_t rows = (int64_t)q->n_mats * (((int64_t)q->rows + 15) / 16 * 16), cols = ((int64_t)q->cols + 511) / 512 * 512;
    if (rows >= ((int64_t)1 << 31) || (rows > 0 && cols > ((int64_t)1 << 36) / rows)) return NVFP4_E_SHAPE;
    if ((int64_t)q->n_mats * q->rows > 0 && q->cols >= ((int64_t)1 << 34) / ((int64_t)q->n_mats * q->rows) + 1)
        return NVFP4_E_SHAPE;
    return NVFP4_OK;
}
int mx_planes(const nvfp4moe_mxfp4_tensor* q) {
    if (!q->codes || !q->scales) return NVFP4_E_NULL;
    if (!aligned(q->codes, 16) || !aligned(q->scales, q->layout == NVFP4_LAYOUT_GEMM ? 4 : 1)) return NVFP4_E_ALIGN;
    return NVFP4_OK;
}

// Workspace of a product: the quantized operand rows, and the row tiles of a
// grouped one.
struct MxWork {
    size_t codes, scales, n_tiles, tiles, total;
    int64_t ld_codes, ld_scales;
};
bool mx_work(int64_t M, int64_t K, int64_t E, MxWork* w) {
    if (M < 0 || M >= ((int64_t)1 << 31) || K <= 0 || K % 32 != 0 || K >= ((int64_t)1 << 24) || E < 1 || E > kMaxExperts)
        return false;
    if (M > 0 && (K + 255) / 256 * 256 >= ((int64_t)1 << 34) / M) return false;
    w->ld_codes = (K + 255) / 256 * 128;
    w->ld_scales = (K + 511) / 512 * 16;
    w->codes = 0;
    w->scales = up(M * w->ld_codes, kAlign);
    w->n_tiles = w->scales + up(M * w->ld_scales, kAlign);
    w->tiles = w->n_tiles + kAlign;
    w->total = w->tiles + up((M / mx_tile_rows() + std::min(M, E) + 1) * 16, kAlign);
    return true;
}

int mx_product(const uint16_t* x, int64_t M, int64_t ldx, const int32_t* offsets, bool grouped,
               const nvfp4moe_mxfp4_tensor* Wq, uint16_t* out, int64_t ld_out, int32_t scale_round, void* workspace,
               size_t workspace_bytes, void* stream) {
    if (scale_round != NVFP4MOE_MXFP4_SCALE_FLOOR && scale_round != NVFP4MOE_MXFP4_SCALE_RU) return NVFP4_E_ARG;
    int st = mx_tensor(Wq);
    if (st != NVFP4_OK) return st;
    if (Wq->layout != NVFP4_LAYOUT_GEMM || Wq->rows < 1 || Wq->n_mats < 1) return NVFP4_E_SHAPE;
    if (!grouped && Wq->n_mats != 1) return NVFP4_E_SHAPE;
    const int64_t K = Wq->cols, N = Wq->rows, E = Wq->n_mats;
    MxWork w;
    if (!mx_work(M, K, E, &w)) return NVFP4_E_SHAPE;
    if (ldx < K || ld_out < N) return NVFP4_E_SHAPE;
    if ((st = mx_planes(Wq)) != NVFP4_OK) return st;
    if (!workspace) return NVFP4_E_NULL;
    if (workspace_bytes < w.total) return NVFP4_E_WORKSPACE;
    if (!aligned(workspace, kAlign)) return NVFP4_E_ALIGN;
    if (M == 0) return NVFP4_OK;
    if (!x || !out || (grouped && !offsets)) return NVFP4_E_NULL;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(out, 2) || !aligned(offsets, 4)) return NVFP4_E_ALIGN;
    const int bm = mx_tile_rows();
    const int64_t tiles = grouped ? M / bm + std::min(M, E) : (M + bm - 1) / bm;
    // One workgroup of 256 threads a tile, and a dispatch holds fewer than 2^32
    // work-items.  (Tiles of 64 columns are taken for a few hundred at most.)
    if (tiles * ((N + 255) / 256) >= ((int64_t)1 << 24) - 8) return NVFP4_E_SHAPE;
    uint8_t* ws = (uint8_t*)workspace;
    hipStream_t s = (hipStream_t)stream;
    const MxShape sh = mx_shape(Wq);
    MxGemmParams p{};
    p.w_codes = Wq->codes;
    p.w_scales = Wq->scales;
    p.row_tiles = (int32_t)sh.row_tiles;
    p.chunks = (int32_t)sh.chunks;
    p.quads = (int32_t)sh.quads;
    p.N = (int32_t)N;
    p.vec_out = ld_out % 4 == 0 && aligned(out, 8);
    p.vec_out8 = ld_out % 8 == 0 && aligned(out, 16);
    p.M = M;
    p.out = out;
    p.ld_out = ld_out;
    const bool up = scale_round == NVFP4MOE_MXFP4_SCALE_RU;
    if (mx_small(M, E, K)) {
        p.x = x;
        p.ldx = ldx;
        p.cols = (uint32_t)K;
        p.up = up;
        p.offsets = offsets;
        return hip_status(launch_mx_gemm_small(p, E, s));
    }
    MxRowsParams q{};
    q.x = x;
    q.rows = M;
    q.ld = ldx;
    q.cols = (uint32_t)K;
    q.up = up;
    q.operand = true;
    q.codes = ws + w.codes;
    q.scales = ws + w.scales;
    q.ld_codes = w.ld_codes;
    q.ld_scales = w.ld_scales;
    if (grouped) {
        q.tiles = (int4*)(ws + w.tiles);
        q.n_tiles = (int32_t*)(ws + w.n_tiles);
        q.offsets = offsets;
        q.E = (int32_t)E;
        q.bm = bm;
    }
    if (launch_mx_quant_rows(q, s) != hipSuccess) return NVFP4_E_HIP;
    p.a_codes = q.codes;
    p.a_scales = q.scales;
    p.ld_a = w.ld_codes;
    p.ld_as = w.ld_scales;
    p.tiles = q.tiles;
    p.n_tiles = q.n_tiles;
    return hip_status(launch_mx_gemm(p, tiles, s));
}

// Sizes and pointers of a set of adapters.
int adapter_shape(const nvfp4moe_adapters* ad, int64_t M) {
    if (!ad) return NVFP4_E_NULL;
    if (ad->n < 1 || ad->n > kMaxExperts || ad->rank < 8 || ad->rank > kMaxRank || ad->rank % 8 != 0) return NVFP4_E_SHAPE;
    for (const int32_t w : {ad->in_features, ad->out_features})
        if (w < 8 || w % 8 != 0 || w >= (1 << 24)) return NVFP4_E_SHAPE;
    if (M < 0 || M >= ((int64_t)1 << 26)) return NVFP4_E_SHAPE;
    // (of A and B together; more than any memory holds, and what the launches' sizes allow)
    if ((int64_t)ad->n * ad->rank * ((int64_t)ad->in_features + ad->out_features) >= ((int64_t)1 << 37)) return NVFP4_E_SHAPE;
    return NVFP4_OK;
}
int adapter_planes(const nvfp4moe_adapters* ad) {
    if (!ad->A || !ad->B) return NVFP4_E_NULL;
    if (!aligned(ad->A, 16) || !aligned(ad->B, 16) || !aligned(ad->scale, 4)) return NVFP4_E_ALIGN;
    return NVFP4_OK;
}
// Workspace: the plan (rows by adapter, its tables) and, for the gradients, the
// transposed adapters, w and v as operands and partial sums.  A size for M rows
// is enough for fewer: no part of it falls as M grows.
struct AdapterWork {
    size_t order, tiles, chunks, steps, info, first, second, v_pack, w_pack, slots, total;
    int64_t n_tiles, n_chunks;
    AdapterSplit split;
};
AdapterWork adapter_work(const nvfp4moe_adapters* ad, int64_t M, bool backward) {
    AdapterWork w{};
    const int64_t n = ad->n, R = ad->rank, K = ad->in_features, N = ad->out_features;
    w.n_tiles = M / (backward ? kAdTile : 16) + std::min(M, n + 1);
    w.order = kAlign;
    w.tiles = w.order + up(M * 4, kAlign);
    w.total = w.tiles + up(w.n_tiles * 16, kAlign);
    if (!backward) return w;
    w.info = w.total;
    w.first = w.info + up(n * 8, kAlign);
    w.second = w.first + up(n * adapter_units(N, ad->rank) * 16, kAlign);
    w.total = w.second + up(n * adapter_units(K, ad->rank) * 16, kAlign);
    w.split = adapter_split(M, ad->rank, K, N, n);
    w.n_chunks = w.split.most + n;
    w.chunks = w.total;
    w.steps = w.chunks + up(w.n_chunks * 16, kAlign);
    w.v_pack = w.steps + up(w.n_chunks * 4, kAlign);
    w.w_pack = w.v_pack + (size_t)w.n_tiles * adapter_rank_blocks(ad->rank) * 3 * 1024;
    w.slots = 2 * w.w_pack - w.v_pack;
    // chunks of adapters that have more than one: at most floor(rows / chunk) + 1
    // each, which is at most twice the first term
    w.total = w.slots + (w.split.join ? up(2 * w.split.most * R * (K + N) * 4, kAlign) : 0);
    return w;
}
int adapter_rows(const uint16_t* p, int64_t ld, int64_t cols) {
    if (ld < cols) return NVFP4_E_SHAPE;
    return aligned(p, 16) && ld % 8 == 0 ? NVFP4_OK : NVFP4_E_ALIGN;
}

struct Range {
    uintptr_t lo, hi;
    bool write;
};

// Checks the tensors; the elements per chunk and the number of chunks.  A chunk
// is one workgroup's turn: kGradChunk elements, and fewer (down to 2048) while
// that would give the grid less than one chunk for each workgroup.
int grad_chunks(const nvfp4moe_grad* g, int32_t n, int64_t* chunk, int64_t* chunks) {
    if (n < 0) return NVFP4_E_SHAPE;
    if (n > 0 && !g) return NVFP4_E_NULL;
    int64_t total = 0;
    for (int32_t i = 0; i < n; i++) {
        if (g[i].type != NVFP4MOE_F32 && g[i].type != NVFP4MOE_BF16) return NVFP4_E_ARG;
        if (g[i].n < 0 || g[i].n >= ((int64_t)1 << 40)) return NVFP4_E_SHAPE;
        if (g[i].n == 0) continue;
        if (!g[i].in || !g[i].out) return NVFP4_E_NULL;
        const size_t elem = g[i].type == NVFP4MOE_BF16 ? 2 : 4;
        if (!aligned(g[i].in, elem) || !aligned(g[i].out, elem)) return NVFP4_E_ALIGN;
        total += g[i].n;
    }
    *chunk = kGradChunk;
    while (*chunk > 2048 && total < *chunk * kGradBlocks) *chunk /= 2;
    *chunks = 0;
    for (int32_t i = 0; i < n; i++) *chunks += (g[i].n + *chunk - 1) / *chunk;
    return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4moe_router_logits(const uint16_t* x, int32_t T, int32_t H, const uint16_t* w_router, int32_t E, float* logits,
                           void* stream) {
    if (T < 0 || H <= 0 || H % 16 != 0 || E < 1 || E > kMaxExperts) return NVFP4_E_SHAPE;
    if ((int64_t)T * std::max(H, E) >= ((int64_t)1 << 31)) return NVFP4_E_SHAPE;
    if (T == 0) return NVFP4_OK;
    if (!x || !w_router || !logits) return NVFP4_E_NULL;
    if (!aligned(x, 16) || !aligned(w_router, 16) || !aligned(logits, 4)) return NVFP4_E_ALIGN;
    return hip_status(launch_router_scores(x, T, H, w_router, E, logits, (hipStream_t)stream));
}

int nvfp4moe_router_select(const nvfp4moe_select_config* cfg, const void* logits, int64_t ld, int64_t T, const float* bias,
                           int32_t* ids, float* probs, void* stream) {
    SelectParams P;
    const int st = select_params(cfg, logits, ld, T, bias, &P);
    if (st != NVFP4_OK) return st;
    if (T == 0) return NVFP4_OK;
    if (!logits || !ids || !probs) return NVFP4_E_NULL;
    if (!aligned(ids, 4) || !aligned(probs, 4)) return NVFP4_E_ALIGN;
    P.ids = ids;
    P.probs = probs;
    return hip_status(launch_router_select(P, cfg->logits_type == NVFP4MOE_BF16, (hipStream_t)stream));
}

int nvfp4moe_router_select_backward(const nvfp4moe_select_config* cfg, const void* logits, int64_t ld, int64_t T,
                                    const float* bias, const int32_t* ids, const float* dprobs, void* dlogits,
                                    int64_t ld_out, void* stream) {
    SelectParams P;
    const int st = select_params(cfg, logits, ld, T, bias, &P);
    if (st != NVFP4_OK) return st;
    if (ld_out < cfg->n_experts) return NVFP4_E_SHAPE;
    if (T == 0) return NVFP4_OK;
    if (!logits || !ids || !dprobs || !dlogits) return NVFP4_E_NULL;
    const size_t elem = cfg->logits_type == NVFP4MOE_BF16 ? 2 : 4;
    if (!aligned(ids, 4) || !aligned(dprobs, 4) || !aligned(dlogits, elem)) return NVFP4_E_ALIGN;
    P.ids_in = ids;
    P.dprobs = dprobs;
    P.dlogits = dlogits;
    P.ld_out = ld_out;
    P.vec_out = ld_out % 4 == 0 && aligned(dlogits, 4 * elem);
    return hip_status(launch_router_select_backward(P, cfg->logits_type == NVFP4MOE_BF16, (hipStream_t)stream));
}

size_t nvfp4moe_balance_workspace_bytes(int64_t T, int32_t n_experts, int32_t n_sequences) {
    BalanceWork w;
    return balance_work(T, n_experts, n_sequences, &w) ? w.total : 0;
}

int nvfp4moe_router_balance_loss(const nvfp4moe_balance_config* cfg, const void* logits, int64_t ld, int64_t T,
                                 const int32_t* ids, const int32_t* seq_offsets, int32_t n_sequences, float* loss,
                                 int32_t* counts, void* workspace, size_t workspace_bytes, void* stream) {
    BalanceParams P;
    const int st = balance_params(cfg, logits, ld, T, seq_offsets, n_sequences, &P);
    if (st != NVFP4_OK) return st;
    BalanceWork w;
    if (!balance_work(T, P.E, P.S, &w)) return NVFP4_E_SHAPE;
    P.chunk = balance_chunk(T, P.E, P.S);
    if (!loss || !counts || (T > P.chunk && !workspace) || (T > 0 && (!logits || !ids))) return NVFP4_E_NULL;
    if (T > P.chunk && workspace_bytes < w.total) return NVFP4_E_WORKSPACE;
    if (!aligned(ids, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(workspace, kAlign)) return NVFP4_E_ALIGN;
    uint8_t* ws = (uint8_t*)workspace;
    P.ids = ids;
    P.psum = (float*)ws;
    P.csum = (int32_t*)(ws + w.csum);
    P.part = (double*)(ws + w.part);
    P.done = (uint32_t*)(ws + w.done);
    P.loss = loss;
    P.counts = counts;
    return hip_status(launch_balance(P, cfg->logits_type == NVFP4MOE_BF16, (hipStream_t)stream));
}

int nvfp4moe_router_balance_backward(const nvfp4moe_balance_config* cfg, const void* logits, int64_t ld, int64_t T,
                                     const int32_t* counts, const int32_t* seq_offsets, int32_t n_sequences,
                                     const float* dloss, const void* add, int64_t ld_add, void* dlogits, int64_t ld_out,
                                     void* stream) {
    BalanceParams P;
    const int st = balance_params(cfg, logits, ld, T, seq_offsets, n_sequences, &P);
    if (st != NVFP4_OK) return st;
    if (ld_out < P.E || (add && ld_add < P.E)) return NVFP4_E_SHAPE;
    if (T == 0) return NVFP4_OK;
    if (!logits || !counts || !dlogits) return NVFP4_E_NULL;
    const size_t elem = cfg->logits_type == NVFP4MOE_BF16 ? 2 : 4;
    if (add == dlogits && ld_add != ld_out) return NVFP4_E_ARG;
    if (!aligned(counts, 4) || !aligned(dloss, 4) || !aligned(add, elem) || !aligned(dlogits, elem)) return NVFP4_E_ALIGN;
    P.counts_in = counts;
    P.dloss = dloss;
    P.add = add;
    P.ld_add = ld_add;
    P.dlogits = dlogits;
    P.ld_out = ld_out;
    P.vec_add = ld_add % 4 == 0 && aligned(add, 4 * elem);
    P.vec_out = ld_out % 4 == 0 && aligned(dlogits, 4 * elem);
    P.vec_counts = P.E % 4 == 0 && aligned(counts, 16);
    return hip_status(launch_balance(P, cfg->logits_type == NVFP4MOE_BF16, (hipStream_t)stream));
}

int nvfp4moe_mxfp4_bytes(const nvfp4moe_mxfp4_tensor* q, size_t* codes_bytes, size_t* scales_bytes) {
    const int st = mx_tensor(q);
    if (st != NVFP4_OK) return st;
    if (!codes_bytes || !scales_bytes) return NVFP4_E_NULL;
    const size_t n = (size_t)q->n_mats;
    if (q->layout == NVFP4_LAYOUT_GEMM) {
        const MxShape s = mx_shape(q);
        *codes_bytes = n * s.row_tiles * s.chunks * 1024;
        *scales_bytes = n * s.row_tiles * s.quads * 256;
    } else {
        *codes_bytes = n * q->rows * ((size_t)q->cols / 2);
        *scales_bytes = n * q->rows * ((size_t)q->cols / 32);
    }
    return NVFP4_OK;
}

int nvfp4moe_mxfp4_quantize(const uint16_t* x, int64_t ld, const nvfp4moe_mxfp4_tensor* q, int32_t scale_round, void* stream) {
    if (scale_round != NVFP4MOE_MXFP4_SCALE_FLOOR && scale_round != NVFP4MOE_MXFP4_SCALE_RU) return NVFP4_E_ARG;
    int st = mx_tensor(q);
    if (st != NVFP4_OK) return st;
    if (ld < q->cols) return NVFP4_E_SHAPE;
    const int64_t rows = (int64_t)q->n_mats * q->rows;
    if (rows == 0) return NVFP4_OK;
    if (!x) return NVFP4_E_NULL;
    if ((st = mx_planes(q)) != NVFP4_OK) return st;
    if (!aligned(x, 16) || ld % 8 != 0) return NVFP4_E_ALIGN;
    const bool ru = scale_round == NVFP4MOE_MXFP4_SCALE_RU;
    if (q->layout == NVFP4_LAYOUT_GEMM)
        return hip_status(launch_mx_quant_tiles(x, q->n_mats, q->rows, q->cols, ld, q->codes, q->scales, ru,
                                                (hipStream_t)stream));
    MxRowsParams p{};
    p.x = x;
    p.rows = rows;
    p.ld = ld;
    p.cols = (uint32_t)q->cols;
    p.up = ru;
    p.codes = q->codes;
    p.scales = q->scales;
    p.ld_codes = q->cols / 2;
    p.ld_scales = q->cols / 32;
    return hip_status(launch_mx_quant_rows(p, (hipStream_t)stream));
}

int nvfp4moe_mxfp4_dequantize(const nvfp4moe_mxfp4_tensor* q, uint16_t* out, int64_t ld, void* stream) {
    int st = mx_tensor(q);
    if (st != NVFP4_OK) return st;
    if (ld < q->cols) return NVFP4_E_SHAPE;
    const int64_t rows = (int64_t)q->n_mats * q->rows;
    if (rows == 0) return NVFP4_OK;
    if (!out) return NVFP4_E_NULL;
    if ((st = mx_planes(q)) != NVFP4_OK) return st;
    if (!aligned(out, 16) || ld % 8 != 0) return NVFP4_E_ALIGN;
    MxDequantParams p{};
    p.codes = q->codes;
    p.scales = q->scales;
    p.out = out;
    p.rows = rows;
    p.ld = ld;
    p.cols = (uint32_t)q->cols;
    p.mat_rows = (uint32_t)q->rows;
    p.tiled = q->layout == NVFP4_LAYOUT_GEMM;
    return hip_status(launch_mx_dequant(p, (hipStream_t)stream));
}

size_t nvfp4moe_mxfp4_workspace_bytes(int64_t M, int64_t K, int64_t n_mats) {
    MxWork w;
    return mx_work(M, K, n_mats, &w) ? w.total : 0;
}

int nvfp4moe_mxfp4_linear(const uint16_t* x, int64_t M, int64_t ldx, const nvfp4moe_mxfp4_tensor* Wq, uint16_t* out,
                          int64_t ld_out, int32_t scale_round, void* workspace, size_t workspace_bytes, void* stream) {
    return mx_product(x, M, ldx, nullptr, false, Wq, out, ld_out, scale_round, workspace, workspace_bytes, stream);
}

int nvfp4moe_mxfp4_grouped_linear(const uint16_t* x, int64_t R, int64_t ldx, const int32_t* offsets,
                                  const nvfp4moe_mxfp4_tensor* Wq, uint16_t* out, int64_t ld_out, int32_t scale_round,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    return mx_product(x, R, ldx, offsets, true, Wq, out, ld_out, scale_round, workspace, workspace_bytes, stream);
}

size_t nvfp4moe_adapter_workspace_bytes(const nvfp4moe_adapters* ad, int64_t M, int32_t backward) {
    return adapter_shape(ad, M) == NVFP4_OK ? adapter_work(ad, M, backward != 0).total : 0;
}

int nvfp4moe_adapter_linear(const nvfp4moe_adapters* ad, const uint16_t* x, int64_t M, int64_t ldx, const int32_t* ids,
                            const uint16_t* base, int64_t ld_base, uint16_t* out, int64_t ld_out, float* v,
                            void* workspace, size_t workspace_bytes, void* stream) {
    int st = adapter_shape(ad, M);
    if (st != NVFP4_OK) return st;
    const int32_t K = ad->in_features, N = ad->out_features;
    if (M == 0) return NVFP4_OK;
    if (!x || !ids || !out || !workspace) return NVFP4_E_NULL;
    if ((st = adapter_planes(ad)) != NVFP4_OK || (st = adapter_rows(x, ldx, K)) != NVFP4_OK ||
        (st = adapter_rows(out, ld_out, N)) != NVFP4_OK || (base && (st = adapter_rows(base, ld_base, N)) != NVFP4_OK))
        return st;
    if (base == out && ld_base != ld_out) return NVFP4_E_ARG;
    const AdapterWork w = adapter_work(ad, M, false);
    if (workspace_bytes < w.total) return NVFP4_E_WORKSPACE;
    if (!aligned(ids, 4) || !aligned(v, 16) || !aligned(workspace, kAlign)) return NVFP4_E_ALIGN;
    uint8_t* ws = (uint8_t*)workspace;
    AdapterParams p{};
    p.x = x;
    p.ldx = ldx;
    p.A = ad->A;
    p.B = ad->B;
    p.scale = ad->scale;
    p.R = ad->rank;
    p.K = K;
    p.N = N;
    p.base = base;
    p.ld_base = ld_base;
    p.out = out;
    p.ld_out = ld_out;
    p.v = v;
    p.M = M;
    p.n = ad->n;
    p.rest = base != out || v;
    if (adapter_small(M)) {
        p.ids = ids;
        return hip_status(launch_adapter(p, M, (hipStream_t)stream));
    }
    AdapterPlan plan{};
    plan.ids = ids;
    plan.M = M;
    plan.n = ad->n;
    plan.tile = adapter_tile(ad->rank, M, ad->n);
    plan.rest = p.rest;
    plan.n_tables = (int32_t*)ws;
    plan.order = (int32_t*)(ws + w.order);
    plan.tiles = (int4*)(ws + w.tiles);
    if (launch_adapter_plan(plan, nullptr, (hipStream_t)stream) != hipSuccess) return NVFP4_E_HIP;
    p.order = plan.order;
    p.tiles = plan.tiles;
    p.n_tiles = plan.n_tables;
    return hip_status(launch_adapter(p, w.n_tiles, (hipStream_t)stream));
}

int nvfp4moe_adapter_backward(const nvfp4moe_adapters* ad, const uint16_t* x, int64_t M, int64_t ldx, const int32_t* ids,
                              const float* v, const uint16_t* dy, int64_t ld_dy, const uint16_t* base, int64_t ld_base,
                              uint16_t* dx, int64_t ld_dx, float* dA, float* dB, void* workspace, size_t workspace_bytes,
                              void* stream) {
    int st = adapter_shape(ad, M);
    if (st != NVFP4_OK) return st;
    const int32_t K = ad->in_features, N = ad->out_features;
    if (!dA || !dB || !workspace || (M > 0 && (!x || !ids || !v || !dy || !dx))) return NVFP4_E_NULL;
    if ((st = adapter_planes(ad)) != NVFP4_OK || (st = adapter_rows(x, ldx, K)) != NVFP4_OK ||
        (st = adapter_rows(dy, ld_dy, N)) != NVFP4_OK || (st = adapter_rows(dx, ld_dx, K)) != NVFP4_OK ||
        (base && (st = adapter_rows(base, ld_base, K)) != NVFP4_OK))
        return st;
    if (base && base == dx && ld_base != ld_dx) return NVFP4_E_ARG;
    const AdapterWork w = adapter_work(ad, M, true);
    if (workspace_bytes < w.total) return NVFP4_E_WORKSPACE;
    if (!aligned(ids, 4) || !aligned(v, 4) || !aligned(dA, 16) || !aligned(dB, 16) || !aligned(workspace, kAlign))
        return NVFP4_E_ALIGN;
    uint8_t* ws = (uint8_t*)workspace;
    hipStream_t s = (hipStream_t)stream;
    AdapterPlan plan{};
    plan.ids = ids;
    plan.M = M;
    plan.n = ad->n;
    plan.tile = kAdTile;
    plan.chunk = w.split.chunk;
    plan.rest = base != dx;
    plan.n_tables = (int32_t*)ws;
    plan.order = (int32_t*)(ws + w.order);
    plan.tiles = (int4*)(ws + w.tiles);
    plan.chunks = (int4*)(ws + w.chunks);
    plan.chunk_step = (int32_t*)(ws + w.steps);
    plan.info = (int2*)(ws + w.info);
    AdapterPack k{};
    k.A = ad->A;
    k.B = ad->B;
    k.info = plan.info;
    k.n = ad->n;
    k.R = ad->rank;
    k.K = K;
    k.N = N;
    k.first = (u32x4*)(ws + w.first);
    k.second = (u32x4*)(ws + w.second);
    k.units_first = adapter_units(N, ad->rank);
    k.units_second = adapter_units(K, ad->rank);
    if (launch_adapter_plan(plan, M > 0 ? &k : nullptr, s) != hipSuccess) return NVFP4_E_HIP;
    AdapterGrad g{};
    g.scale = ad->scale;
    g.n = ad->n;
    g.R = ad->rank;
    g.K = K;
    g.N = N;
    g.x = x;
    g.dy = dy;
    g.ldx = ldx;
    g.ld_dy = ld_dy;
    g.v_pack = (u32x4*)(ws + w.v_pack);
    g.w_pack = (u32x4*)(ws + w.w_pack);
    g.rank_blocks = adapter_rank_blocks(ad->rank);
    g.order = plan.order;
    g.chunks = plan.chunks;
    g.chunk_step = plan.chunk_step;
    g.n_tables = plan.n_tables;
    g.info = plan.info;
    g.slots = (float*)(ws + w.slots);
    g.dA = dA;
    g.dB = dB;
    if (M > 0) {
        AdapterParams p{};
        p.A = (const uint16_t*)k.first;
        p.B = (const uint16_t*)k.second;
        p.units_a = k.units_first;
        p.units_b = k.units_second;
        p.x = dy;
        p.ldx = ld_dy;
        p.scale = ad->scale;
        p.R = ad->rank;
        p.K = N;
        p.N = K;
        p.base = base;
        p.ld_base = ld_base;
        p.out = dx;
        p.ld_out = ld_dx;
        p.v_in = v;
        p.v_pack = (u32x4*)(ws + w.v_pack);
        p.w_pack = (u32x4*)(ws + w.w_pack);
        p.M = M;
        p.order = plan.order;
        p.tiles = plan.tiles;
        p.n_tiles = plan.n_tables;
        if (launch_adapter(p, w.n_tiles, s) != hipSuccess) return NVFP4_E_HIP;
    }
    return hip_status(launch_adapter_wgrad(g, w.split, w.n_chunks, s));
}

int nvfp4moe_grad_plan_bytes(const nvfp4moe_grad* grads, int32_t n_grads, size_t* bytes, int64_t* n_chunks) {
    if (!bytes || !n_chunks) return NVFP4_E_NULL;
    int64_t chunk = 0;
    const int st = grad_chunks(grads, n_grads, &chunk, n_chunks);
    if (st != NVFP4_OK) return st;
    *bytes = (size_t)*n_chunks * sizeof(GradChunk);
    return NVFP4_OK;
}

int nvfp4moe_grad_plan(const nvfp4moe_grad* grads, int32_t n_grads, void* plan_host, size_t plan_bytes) {
    int64_t chunk = 0, n_chunks = 0;
    const int st = grad_chunks(grads, n_grads, &chunk, &n_chunks);
    if (st != NVFP4_OK) return st;
    if (plan_bytes < (size_t)n_chunks * sizeof(GradChunk)) return NVFP4_E_WORKSPACE;
    if (n_chunks == 0) return NVFP4_OK;
    if (!plan_host) return NVFP4_E_NULL;
    if (!aligned(plan_host, 8)) return NVFP4_E_ALIGN;
    // No output may overlap another range: sorted by start, every range must
    // begin at or after the end of all earlier ones if either of them is
    // written (a tensor's own identical in and out are one range).
    std::vector<Range> ranges;
    try {
        ranges.reserve(2 * (size_t)n_grads);
    } catch (...) {  // no exception crosses the ABI
        return NVFP4_E_WORKSPACE;
    }
    for (int32_t i = 0; i < n_grads; i++) {
        const nvfp4moe_grad& g = grads[i];
        if (g.n == 0) continue;
        const size_t len = (size_t)g.n * (g.type == NVFP4MOE_BF16 ? 2 : 4);
        ranges.push_back({(uintptr_t)g.out, (uintptr_t)g.out + len, true});
        if (g.in != g.out) ranges.push_back({(uintptr_t)g.in, (uintptr_t)g.in + len, false});
    }
    std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t end_any = 0, end_write = 0;
    for (const Range& r : ranges) {
        if (r.lo < end_write || (r.write && r.lo < end_any)) return NVFP4_E_ARG;
        end_any = std::max(end_any, r.hi);
        if (r.write) end_write = std::max(end_write, r.hi);
    }
    GradChunk* c = (GradChunk*)plan_host;
    for (int32_t i = 0; i < n_grads; i++) {
        const nvfp4moe_grad& g = grads[i];
        const size_t elem = g.type == NVFP4MOE_BF16 ? 2 : 4;
        for (int64_t at = 0; at < g.n; at += chunk, c++) {
            *c = GradChunk{};
            c->in = (const uint8_t*)g.in + at * elem;
            c->out = (uint8_t*)g.out + at * elem;
            c->n = (uint32_t)std::min<int64_t>(chunk, g.n - at);
            const size_t off = (uintptr_t)c->in % 16;
            c->head = (uint16_t)std::min<size_t>(c->n, off ? (16 - off) / elem : 0);
            c->bf16 = g.type == NVFP4MOE_BF16;
            c->out_vec = (uintptr_t)c->out % 16 == off;
        }
    }
    return NVFP4_OK;
}

size_t nvfp4moe_clip_workspace_bytes(void) { return kGradBlocks * sizeof(double); }

int nvfp4moe_clip_grad_norm(const void* plan, int64_t n_chunks, double max_norm, double* norm_out, void* workspace,
                            size_t workspace_bytes, void* stream) {
    if (n_chunks < 0) return NVFP4_E_SHAPE;
    if (!(max_norm >= 0.0)) return NVFP4_E_ARG;
    if ((n_chunks > 0 && !plan) || !norm_out || !workspace) return NVFP4_E_NULL;
    if (workspace_bytes < nvfp4moe_clip_workspace_bytes()) return NVFP4_E_WORKSPACE;
    if (!aligned(plan, 8) || !aligned(norm_out, 8) || !aligned(workspace, 8)) return NVFP4_E_ALIGN;
    return hip_status(launch_clip_grad_norm((const GradChunk*)plan, n_chunks, max_norm, (double*)workspace, norm_out,
                                            (hipStream_t)stream));
}

}  // extern "C"
