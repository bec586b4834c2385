// dsa_api.cu -- the extern "C" entry points of libdsa: host-side validation,
// workspace layout, and the order in which the kernels are enqueued.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "dsa.h"
#include "dsa_kernels.cuh"
#include "extents.h"

namespace dsa {
namespace {

constexpr size_t kAlign = 256;
constexpr uint32_t kKnownFlags = DSA_FLAG_TWO_LAUNCH | DSA_FLAG_DESC_ORDER | DSA_FLAG_DENSE;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

}  // namespace

size_t ws_zero_bytes() { return kWsHeaderBytes + index_select_fused_state_bytes(); }

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The address at which the current device reaches a caller's buffer: the
// pointer itself for device or managed memory, the mapped address for
// page-locked host memory; nullptr for memory the device cannot address
// (pageable host memory) or a pointer the runtime cannot classify.
const void* device_address(const void* p) {
    if (p == nullptr) return nullptr;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();                       // leave no error behind for the caller
        return nullptr;
    }
    switch (a.type) {
        case cudaMemoryTypeDevice:
        case cudaMemoryTypeManaged: return p;
        case cudaMemoryTypeHost: return a.devicePointer;
        default: return nullptr;
    }
}

bool trace_on() {
    static const bool on = [] {
        const char* e = getenv("DSA_TRACE");
        return e != nullptr && e[0] != '\0' && e[0] != '0';
    }();
    return on;
}

dsa_status check_shape(const dsa_shape* s, Shape* out) {
    if (s == nullptr) return DSA_ERR_INVALID_ARG;
    if (s->idx_heads <= 0 || s->idx_dim <= 0 || s->heads <= 0 || s->kv_lora <= 0 ||
        s->rope_dim < 0 || s->top_k <= 0 || s->kpool <= 0)
        return DSA_ERR_INVALID_ARG;
    if (s->top_k % s->kpool != 0) return DSA_ERR_INVALID_ARG;
    if (!isfinite(s->scale) || !(s->scale > 0.f)) return DSA_ERR_INVALID_ARG;
    if (s->dtype != DSA_F32 && s->dtype != DSA_BF16) return DSA_ERR_INVALID_ARG;
    // What this build implements: the layer geometry of the pages.
    if (s->idx_heads > 64 || s->idx_dim != 128 || s->heads != 64 || s->kv_lora != 512 ||
        (s->rope_dim != 0 && s->rope_dim != 64) || s->kpool > 16 || s->top_k > 65536)
        return DSA_ERR_UNSUPPORTED;
    *out = Shape{s->idx_heads, s->idx_dim, s->heads, s->kv_lora, s->rope_dim,
                 s->top_k, s->kpool, s->scale, s->dtype};
    return DSA_OK;
}

// max_n_q: the query count this entry point's grids take (the queries of the
// pool compression are the new tokens, which a prompt may have millions of).
dsa_status check_batch(const dsa_batch* b, const Shape& sh, BatchDev* out,
                       int64_t max_n_q = 65535) {
    if (b == nullptr) return DSA_ERR_INVALID_ARG;
    if (b->n_seq < 0 || b->n_q < 0 || b->max_q_len < 0 || b->max_kv_len < 0 ||
        (b->flags & ~kKnownFlags) != 0 || b->total_rows < 0 || b->total_keys < 0)
        return DSA_ERR_INVALID_ARG;
    if (b->n_q > 0) {
        if (b->n_seq < 1 || b->row_off == nullptr || b->key_off == nullptr || b->q_off == nullptr)
            return DSA_ERR_INVALID_ARG;
        if (b->max_q_len < 1 || b->max_kv_len < b->max_q_len) return DSA_ERR_INVALID_ARG;
        if ((int64_t)b->max_q_len > (int64_t)b->n_q) return DSA_ERR_INVALID_ARG;
        if (b->total_rows < 1) return DSA_ERR_INVALID_ARG;
    }
    if (b->max_kv_len >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
    if (b->n_q > max_n_q) return DSA_ERR_UNSUPPORTED;
    // descending order sorts a query's selected units in shared memory
    if ((b->flags & DSA_FLAG_DESC_ORDER) && sh.top_k / sh.kpool > 16384) return DSA_ERR_UNSUPPORTED;
    *out = BatchDev{b->row_off,    b->key_off,    b->q_off,      b->n_seq,      b->n_q,
                    b->max_q_len,  b->max_kv_len, b->total_rows, b->total_keys, sh.kpool,
                    b->flags};
    return DSA_OK;
}

// The host scalars of a batch, for sizing and planning (no device pointers).
BatchDev host_batch(const dsa_batch* batch, const Shape& sh) {
    return BatchDev{nullptr,           nullptr,           nullptr,           batch->n_seq,
                    batch->n_q,        batch->max_q_len,  batch->max_kv_len, batch->total_rows,
                    batch->total_keys, sh.kpool,          batch->flags};
}

// Keys a query may score at most, and the default score row stride.
int64_t max_keys(const Shape& sh, const BatchDev& b) { return b.max_kv_len / sh.kpool; }
int64_t default_ld(const Shape& sh, const BatchDev& b) {
    const int64_t k = max_keys(sh, b);
    return k < 4 ? 4 : (k + 3) / 4 * 4;
}

struct StepLayout {
    size_t sel, idx_plan, scores, idx, n_sel, attn, total;
};

// Decode-step workspace: header | fused selection state (fixed size, kept zero
// between launches) | indexer plan | scores | selections | counts | attention.
StepLayout step_layout(const Shape& sh, const BatchDev& b) {
    StepLayout L{};
    size_t off = kWsHeaderBytes;
    L.sel = off;
    off = align_up(off + index_select_fused_state_bytes());
    L.idx_plan = off;
    off = align_up(off + index_scores_scratch_bytes(sh, b));
    L.scores = off;
    off = align_up(off + (size_t)b.n_q * default_ld(sh, b) * sizeof(float));
    L.idx = off;
    off = align_up(off + (size_t)b.n_q * sh.index_row_width() * sizeof(int32_t));
    L.n_sel = off;
    off = align_up(off + (size_t)b.n_q * sizeof(int32_t));
    L.attn = off;
    off = align_up(off + sparse_mla_scratch_bytes(sh, b));
    L.total = off;
    return L;
}

// Host-fed decode step: the step's workspace, then the staged query-side
// inputs (indexer queries, head weights, absorbed queries).
struct StageLayout {
    size_t q_idx, w, q_abs, total;
};
StageLayout stage_layout(const Shape& sh, const BatchDev& b) {
    StageLayout L{};
    size_t off = step_layout(sh, b).total;
    L.q_idx = off;
    off = align_up(off + (size_t)b.n_q * sh.idx_heads * sh.idx_dim * sh.elem_bytes());
    L.w = off;
    off = align_up(off + (size_t)b.n_q * sh.idx_heads * sizeof(float));
    L.q_abs = off;
    off = align_up(off + (size_t)b.n_q * sh.heads * sh.width() * sh.elem_bytes());
    L.total = off;
    return L;
}

// Where the scratch of the single-step entry points begins: after the prefix
// the fused decode launch keeps zero, so that one workspace can serve every
// entry point in turn.
size_t scratch_off() { return align_up(ws_zero_bytes()); }

size_t op_bytes(const Shape& sh, const BatchDev& b, int32_t op) {
    switch (op) {
        case DSA_OP_INDEX_SCORES:
            return align_up(scratch_off() + index_scores_scratch_bytes(sh, b));
        case DSA_OP_TOPK_SELECT: return kWsHeaderBytes;
        case DSA_OP_SPARSE_MLA:
            return align_up(scratch_off() + sparse_mla_scratch_bytes(sh, b));
        case DSA_OP_DECODE_STEP: return step_layout(sh, b).total;
        case DSA_OP_DECODE_STEP_HOST: return stage_layout(sh, b).total;
        case DSA_OP_INDEX_SELECT: return step_layout(sh, b).attn;
        case DSA_OP_POOL_COMPRESS: return kWsHeaderBytes;
        case DSA_OP_PROJECT: return kWsHeaderBytes;
        case DSA_OP_PAGE_PLAN: return align_up(scratch_off() + page_plan_scratch_bytes(b.n_seq));
        case DSA_OP_CACHE_APPEND: return kWsHeaderBytes;
        case DSA_OP_PAGED_MLA: return align_up(scratch_off() + paged_mla_scratch_bytes(sh, b));
        case DSA_OP_EXPANDED_MLA: return align_up(scratch_off() + expanded_mla_scratch_bytes(sh, b));
        default: return 0;
    }
}

dsa_status check_ws(void* ws, size_t ws_bytes, size_t need) {
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0 || ws_bytes < need)
        return DSA_ERR_WORKSPACE;
    return DSA_OK;
}

dsa_status cuda_status(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return DSA_OK;
    if (trace_on()) fprintf(stderr, "[dsa] %s: %s\n", what, cudaGetErrorString(e));
    return DSA_ERR_CUDA;
}

unsigned char* bytes(void* p) { return static_cast<unsigned char*>(p); }

// Steps 1 and 2 into idx / n_sel: the fused launch where it applies, else the
// indexer and the selection; with DSA_FLAG_DESC_ORDER each row is then put in
// descending score order.
cudaError_t enqueue_index_select(const Shape& sh, const BatchDev& b, const StepLayout& lay,
                                 void* ws, const void* q_idx, const float* w, const void* k_idx,
                                 int32_t* idx, int32_t* n_sel, const void* cache,
                                 cudaStream_t st, const char** what) {
    int32_t* err = static_cast<int32_t*>(ws);
    float* scores = reinterpret_cast<float*>(bytes(ws) + lay.scores);
    const int64_t ld = default_ld(sh, b);
    if (index_select_fused_eligible(sh, b)) {
        *what = "index_select_fused";
        return launch_index_select_fused(sh, b, q_idx, w, k_idx, scores, ld, idx, n_sel,
                                         bytes(ws) + lay.sel,
                                         reinterpret_cast<uint32_t*>(bytes(ws) + kWsGridBarOffset),
                                         cache, (int64_t)sh.width() * (int64_t)sh.elem_bytes(),
                                         err, st);
    }
    *what = "index_scores";
    cudaError_t e = launch_index_scores(sh, b, max_keys(sh, b), q_idx, w, k_idx, scores, ld,
                                        bytes(ws) + lay.idx_plan, err, st);
    if (e != cudaSuccess) return e;
    *what = "topk_select";
    e = launch_topk_select(sh, b, scores, ld, idx, n_sel, err, st);
    if (e != cudaSuccess || !(b.flags & DSA_FLAG_DESC_ORDER)) return e;
    *what = "select_order";
    return launch_select_order_desc(sh, b, scores, ld, idx, n_sel, err, st);
}

// The operations of the paged 8-bit cache, numbered apart from the others.
bool paged_op(int32_t op) { return op >= DSA_OP_PAGE_PLAN && op <= DSA_OP_PAGED_MLA; }
bool known_op(int32_t op) {
    return (op >= DSA_OP_INDEX_SCORES && op <= DSA_OP_DECODE_STEP_HOST) || paged_op(op) ||
           op == DSA_OP_EXPANDED_MLA;
}
// Operations whose queries are new tokens, of which a batch may have millions.
bool any_n_q(int32_t op) {
    return op == DSA_OP_POOL_COMPRESS || op == DSA_OP_PAGE_PLAN || op == DSA_OP_CACHE_APPEND ||
           op == DSA_OP_EXPANDED_MLA;
}

dsa_status check_pages(const dsa_pages* p, PagesDev* out) {
    if (p == nullptr || p->n_pages < 1 || p->table_ld < 1) return DSA_ERR_INVALID_ARG;
    if (p->format != DSA_CACHE_E4M3 && p->format != DSA_CACHE_S8) return DSA_ERR_INVALID_ARG;
    if (p->page_rows < 1) return DSA_ERR_INVALID_ARG;
    int32_t shift = 4;
    while (shift < 7 && (1 << shift) != p->page_rows) ++shift;
    if ((1 << shift) != p->page_rows || p->n_pages >= ((int64_t)1 << 31) ||
        p->table_ld >= ((int64_t)1 << 27))
        return DSA_ERR_UNSUPPORTED;
    *out = PagesDev{p->page_rows, shift, p->format, p->n_pages, p->table_ld};
    return DSA_OK;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Kernels one call of `op` enqueues for this shape and batch bound.
int32_t plan_launches(const Shape& sh, const BatchDev& bh, int32_t op, int32_t splits) {
    if (op == DSA_OP_PAGE_PLAN) return page_plan_launches(bh.n_seq);
    if (bh.n_q <= 0) return 0;
    // attention, then the split merge -- except for two tensor-core splits,
    // which merge inside the attention launch (a CTA pair)
    const int32_t attn = splits > 2 || (splits == 2 && !sparse_mla_tc_eligible(sh, bh)) ? 2 : 1;
    const int32_t idx = bh.max_kv_len / sh.kpool > 0
                            ? (index_scores_tc_eligible(sh, bh) ? index_scores_tc_launches(sh, bh) : 1)
                            : 0;
    const int32_t order = (bh.flags & DSA_FLAG_DESC_ORDER) ? 1 : 0;
    const int32_t sel = index_select_fused_eligible(sh, bh) ? 1 : idx + 1 + order;
    switch (op) {
        case DSA_OP_INDEX_SCORES: return idx;
        case DSA_OP_TOPK_SELECT: return 1 + order;
        case DSA_OP_SPARSE_MLA: return attn;
        case DSA_OP_INDEX_SELECT: return sel;
        case DSA_OP_POOL_COMPRESS: return sh.kpool > 1 ? 1 : 0;
        case DSA_OP_PROJECT: return 1;
        case DSA_OP_CACHE_APPEND: return 1;
        case DSA_OP_PAGED_MLA: return paged_mla_launches(sh, bh);
        case DSA_OP_EXPANDED_MLA: return splits > 1 ? 2 : 1;
        case DSA_OP_DECODE_STEP_HOST:                      // the input copy, then the step
            return 1 + ((bh.flags & DSA_FLAG_DENSE) ? attn : sel + attn);
        default: return (bh.flags & DSA_FLAG_DENSE) ? attn : sel + attn;
    }
}

}  // namespace

// Host validation of dsa_decode_step's arguments, everything but the
// workspace: shapes, pointers, alignment, flags.  *ws_need receives the bytes
// of workspace the step needs and *n_q its query count.
dsa_status decode_step_check(const dsa_shape* shape, const dsa_batch* batch, const void* q_idx,
                             const float* w, const void* k_idx, const void* q_abs,
                             const void* cache, const float* out, const float* lse,
                             const int32_t* idx_out, const int32_t* n_sel_out, size_t* ws_need,
                             int32_t* n_q) {
    Shape sh;
    BatchDev b;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if ((s = check_batch(batch, sh, &b)) != DSA_OK) return s;
    const bool dense = (b.flags & DSA_FLAG_DENSE) != 0;
    if (dense && (idx_out != nullptr || n_sel_out != nullptr)) return DSA_ERR_INVALID_ARG;
    if (b.n_q > 0 && (q_abs == nullptr || cache == nullptr || out == nullptr ||
                      (!dense && (q_idx == nullptr || w == nullptr || k_idx == nullptr))))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_idx) || !aligned16(w) || !aligned16(k_idx) || !aligned16(q_abs) ||
        !aligned16(cache) || !aligned16(out) || !aligned16(idx_out) || !aligned16(n_sel_out) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
        return DSA_ERR_INVALID_ARG;
    if (ws_need != nullptr) *ws_need = step_layout(sh, b).total;
    if (n_q != nullptr) *n_q = b.n_q;
    return DSA_OK;
}

}  // namespace dsa

using namespace dsa;

extern "C" {

int dsa_version(void) { return DSA_ABI_VERSION; }

const char* dsa_status_string(int32_t status) {
    switch (status) {
        case DSA_OK: return "ok";
        case DSA_ERR_INVALID_ARG: return "invalid argument";
        case DSA_ERR_UNSUPPORTED: return "unsupported shape or size";
        case DSA_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
        case DSA_ERR_CUDA: return "CUDA runtime or launch error";
        case DSA_ERR_DEVICE: return "a kernel reported invalid data";
        case DSA_ERR_TIMEOUT: return "a bounded device wait timed out";
        default: return "unknown status";
    }
}

int64_t dsa_index_row_width(const dsa_shape* shape) {
    Shape sh;
    if (check_shape(shape, &sh) != DSA_OK) return -1;
    return sh.index_row_width();
}

dsa_status dsa_workspace_size(const dsa_shape* shape, const dsa_batch* batch, int32_t op,
                              size_t* out_bytes) {
    Shape sh;
    if (out_bytes == nullptr) return DSA_ERR_INVALID_ARG;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    // Sizing needs only the host scalars of the batch.
    if (batch == nullptr || batch->n_q < 0 || batch->max_kv_len < 0 ||
        (batch->flags & ~kKnownFlags) != 0)
        return DSA_ERR_INVALID_ARG;
    if (batch->max_kv_len >= ((int64_t)1 << 31) || (batch->n_q > 65535 && !any_n_q(op)))
        return DSA_ERR_UNSUPPORTED;
    if (!known_op(op) || (paged_op(op) && batch->n_seq < 0)) return DSA_ERR_INVALID_ARG;
    *out_bytes = op_bytes(sh, host_batch(batch, sh), op);
    return DSA_OK;
}

dsa_status dsa_plan(const dsa_shape* shape, const dsa_batch* batch, int32_t op,
                    dsa_plan_info* info) {
    Shape sh;
    if (info == nullptr || batch == nullptr) return DSA_ERR_INVALID_ARG;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if (batch->n_q < 0 || batch->max_kv_len < 0 || (batch->flags & ~kKnownFlags) != 0)
        return DSA_ERR_INVALID_ARG;
    if (!known_op(op)) return DSA_ERR_INVALID_ARG;
    const BatchDev bh = host_batch(batch, sh);
    int32_t rps = 0, splits = 0;
    if (op == DSA_OP_PAGED_MLA) plan_paged_splits(sh, bh, &rps, &splits);
    else if (op == DSA_OP_EXPANDED_MLA) splits = plan_expanded_splits(sh, bh);
    else plan_attention_splits(sh, bh, &rps, &splits);
    *info = dsa_plan_info{plan_launches(sh, bh, op, splits), splits, rps, 0};
    return DSA_OK;
}

dsa_status dsa_index_scores(const dsa_shape* shape, const dsa_batch* batch, const void* q_idx,
                            const float* w, const void* k_idx, float* scores, int64_t ld,
                            void* ws, size_t ws_bytes, void* stream) {
    Shape sh;
    BatchDev b;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if ((s = check_batch(batch, sh, &b)) != DSA_OK) return s;
    if (b.n_q > 0 && (q_idx == nullptr || w == nullptr || k_idx == nullptr || scores == nullptr))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_idx) || !aligned16(k_idx) || !aligned16(w) || !aligned16(scores))
        return DSA_ERR_INVALID_ARG;
    if (ld < max_keys(sh, b) || ld < 1) return DSA_ERR_INVALID_ARG;
    if ((s = check_ws(ws, ws_bytes, op_bytes(sh, b, DSA_OP_INDEX_SCORES))) != DSA_OK) return s;
    int32_t* err = static_cast<int32_t*>(ws);
    return cuda_status(launch_index_scores(sh, b, max_keys(sh, b), q_idx, w, k_idx, scores, ld,
                                           bytes(ws) + scratch_off(), err,
                                           static_cast<cudaStream_t>(stream)),
                       "index_scores");
}

dsa_status dsa_topk_select(const dsa_shape* shape, const dsa_batch* batch, const float* scores,
                           int64_t ld, int32_t* idx, int32_t* n_sel, void* ws, size_t ws_bytes,
                           void* stream) {
    Shape sh;
    BatchDev b;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if ((s = check_batch(batch, sh, &b)) != DSA_OK) return s;
    if (b.flags & DSA_FLAG_DENSE) return DSA_ERR_INVALID_ARG;   // no selection to make
    if (b.n_q > 0 && (scores == nullptr || idx == nullptr || n_sel == nullptr))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(scores) || !aligned16(idx) || !aligned16(n_sel)) return DSA_ERR_INVALID_ARG;
    if (ld < max_keys(sh, b) || ld < 1) return DSA_ERR_INVALID_ARG;
    if ((s = check_ws(ws, ws_bytes, op_bytes(sh, b, DSA_OP_TOPK_SELECT))) != DSA_OK) return s;
    int32_t* err = static_cast<int32_t*>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_topk_select(sh, b, scores, ld, idx, n_sel, err, st);
    if (e == cudaSuccess && (b.flags & DSA_FLAG_DESC_ORDER))
        e = launch_select_order_desc(sh, b, scores, ld, idx, n_sel, err, st);
    return cuda_status(e, "topk_select");
}

dsa_status dsa_sparse_mla_attn(const dsa_shape* shape, const dsa_batch* batch, const void* q_abs,
                               const void* cache, const int32_t* idx, const int32_t* n_sel,
                               float* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    Shape sh;
    BatchDev b;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if ((s = check_batch(batch, sh, &b)) != DSA_OK) return s;
    const bool dense = (b.flags & DSA_FLAG_DENSE) != 0;
    if (b.n_q > 0 && (q_abs == nullptr || cache == nullptr || out == nullptr ||
                      (!dense && (idx == nullptr || n_sel == nullptr))))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_abs) || !aligned16(cache) || !aligned16(out) || !aligned16(idx))
        return DSA_ERR_INVALID_ARG;
    const size_t need = op_bytes(sh, b, DSA_OP_SPARSE_MLA);
    if ((s = check_ws(ws, ws_bytes, need)) != DSA_OK) return s;
    int32_t* err = static_cast<int32_t*>(ws);
    // The previous kernel in the stream is the caller's: the query is read
    // only after it has completed.
    return cuda_status(launch_sparse_mla(sh, b, q_abs, cache, dense ? nullptr : idx,
                                         dense ? nullptr : n_sel, out, lse,
                                         bytes(ws) + scratch_off(), need - scratch_off(), err,
                                         /*q_early=*/false, static_cast<cudaStream_t>(stream)),
                       "sparse_mla_attn");
}

dsa_status dsa_index_prepare(const dsa_shape* shape, int64_t n_vec, const float* x,
                             const int64_t* pos, int32_t rope_dims, double rope_base, void* out,
                             void* stream) {
    Shape sh;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if (n_vec < 0 || rope_dims < 0 || rope_dims > sh.idx_dim || (rope_dims & 1) ||
        !isfinite(rope_base) || !(rope_base > 0.0))
        return DSA_ERR_INVALID_ARG;
    if (n_vec > 0 && (x == nullptr || out == nullptr || (rope_dims > 0 && pos == nullptr)))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(out) || (reinterpret_cast<uintptr_t>(pos) & 7) != 0)
        return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_index_prepare(sh, n_vec, x, pos, rope_dims, rope_base, out,
                                            static_cast<cudaStream_t>(stream)),
                       "index_prepare");
}

dsa_status dsa_pool_compress(const dsa_shape* shape, const dsa_batch* batch, const void* cells,
                             const float* pos, void* pool_keys, void* ws, size_t ws_bytes,
                             void* stream) {
    Shape sh;
    BatchDev b;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if (sh.kpool < 2) return DSA_ERR_INVALID_ARG;          // token mode has no pools
    if ((s = check_batch(batch, sh, &b, 0x7fffffff)) != DSA_OK) return s;
    if (b.n_seq > 65535) return DSA_ERR_UNSUPPORTED;
    if (b.n_q > 0 && (cells == nullptr || pos == nullptr || pool_keys == nullptr))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(cells) || !aligned16(pos) || !aligned16(pool_keys)) return DSA_ERR_INVALID_ARG;
    if ((s = check_ws(ws, ws_bytes, op_bytes(sh, b, DSA_OP_POOL_COMPRESS))) != DSA_OK) return s;
    if (b.n_q == 0) return DSA_OK;
    int32_t* err = static_cast<int32_t*>(ws);
    return cuda_status(launch_pool_compress(sh, b, cells, pos, pool_keys, err,
                                            static_cast<cudaStream_t>(stream)),
                       "pool_compress");
}

// The projections' common checks: sizes, pointers (16-byte aligned), workspace.
static dsa_status check_projection(const dsa_shape* shape, int32_t n_q, int32_t k_dim, int32_t k_unit,
                            const void* in, const void* w, const void* out, void* ws,
                            size_t ws_bytes, Shape* sh) {
    dsa_status s = check_shape(shape, sh);
    if (s != DSA_OK) return s;
    if (n_q < 0 || k_dim < k_unit || k_dim % k_unit != 0) return DSA_ERR_INVALID_ARG;
    if (k_dim > 512 || n_q > (1 << 24)) return DSA_ERR_UNSUPPORTED;
    if (n_q > 0 && (in == nullptr || w == nullptr || out == nullptr)) return DSA_ERR_INVALID_ARG;
    if (!aligned16(in) || !aligned16(w) || !aligned16(out)) return DSA_ERR_INVALID_ARG;
    return check_ws(ws, ws_bytes, kWsHeaderBytes);
}

dsa_status dsa_absorb_q(const dsa_shape* shape, int32_t n_q, int32_t nope_dim, const void* q,
                        const void* w_uk, void* q_abs, void* ws, size_t ws_bytes, void* stream) {
    Shape sh;
    dsa_status s = check_projection(shape, n_q, nope_dim, 64, q, w_uk, q_abs, ws, ws_bytes, &sh);
    if (s != DSA_OK) return s;
    return cuda_status(launch_absorb_q(sh, n_q, nope_dim, q, w_uk, q_abs,
                                       static_cast<int32_t*>(ws),
                                       static_cast<cudaStream_t>(stream)),
                       "absorb_q");
}

dsa_status dsa_up_project(const dsa_shape* shape, int32_t n_q, int32_t v_dim, const float* o,
                          const void* w_uv, float* out, void* ws, size_t ws_bytes, void* stream) {
    Shape sh;
    dsa_status s = check_projection(shape, n_q, v_dim, 128, o, w_uv, out, ws, ws_bytes, &sh);
    if (s != DSA_OK) return s;
    return cuda_status(launch_up_project(sh, n_q, v_dim, o, w_uv, out, static_cast<int32_t*>(ws),
                                         static_cast<cudaStream_t>(stream)),
                       "up_project");
}

dsa_status dsa_page_plan(const dsa_pages* pages, int32_t n_seq, int64_t max_new,
                         const int64_t* held_len, const int64_t* kv_len, const int64_t* q_len,
                         int32_t* free_pages, const int32_t* n_free_in, int32_t* n_free_out,
                         int32_t* block_table, int64_t* row_off, int64_t* q_off, int64_t* slots,
                         void* ws, size_t ws_bytes, void* stream) {
    PagesDev pg;
    dsa_status s = check_pages(pages, &pg);
    if (s != DSA_OK) return s;
    if (n_seq < 0 || max_new < 0) return DSA_ERR_INVALID_ARG;
    if (n_seq > (1 << 20) || max_new >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
    if (row_off == nullptr || q_off == nullptr || free_pages == nullptr || n_free_in == nullptr ||
        n_free_out == nullptr || (max_new > 0 && slots == nullptr) ||
        (n_seq > 0 && (held_len == nullptr || kv_len == nullptr || q_len == nullptr ||
                       block_table == nullptr)))
        return DSA_ERR_INVALID_ARG;
    if (!aligned(held_len, 8) || !aligned(kv_len, 8) || !aligned(q_len, 8) ||
        !aligned(row_off, 8) || !aligned(q_off, 8) || !aligned(slots, 8) ||
        !aligned(free_pages, 4) || !aligned(n_free_in, 4) || !aligned(n_free_out, 4) ||
        !aligned(block_table, 4))
        return DSA_ERR_INVALID_ARG;
    if ((s = check_ws(ws, ws_bytes, align_up(scratch_off() + page_plan_scratch_bytes(n_seq)))) != DSA_OK)
        return s;
    const PagePlanArgs a{pg,         n_seq,       max_new,   held_len, kv_len, q_len, free_pages,
                         n_free_in,  n_free_out,  block_table, row_off, q_off, slots};
    return cuda_status(launch_page_plan(a, bytes(ws) + scratch_off(),
                                        reinterpret_cast<uint32_t*>(bytes(ws) + kWsPlanTicketOffset),
                                        static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)),
                       "page_plan");
}

dsa_status dsa_cache_append(const dsa_shape* shape, const dsa_batch* batch, const dsa_pages* pages,
                            const void* rows, const int64_t* slots, void* codes, void* scales,
                            void* ws, size_t ws_bytes, void* stream) {
    Shape sh;
    BatchDev b;
    PagesDev pg;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if ((s = check_batch(batch, sh, &b, 0x7fffffff)) != DSA_OK) return s;
    if ((s = check_pages(pages, &pg)) != DSA_OK) return s;
    if (b.n_seq > 65535) return DSA_ERR_UNSUPPORTED;
    if (b.n_q > 0 && (rows == nullptr || slots == nullptr || codes == nullptr || scales == nullptr))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(rows) || !aligned(slots, 8) || !aligned(codes, 32)) return DSA_ERR_INVALID_ARG;
    if ((s = check_ws(ws, ws_bytes, op_bytes(sh, b, DSA_OP_CACHE_APPEND))) != DSA_OK) return s;
    if (b.n_q == 0) return DSA_OK;
    return cuda_status(launch_cache_append(sh, b, pg, rows, slots, static_cast<uint8_t*>(codes),
                                           static_cast<uint8_t*>(scales), static_cast<int32_t*>(ws),
                                           static_cast<cudaStream_t>(stream)),
                       "cache_append");
}

dsa_status dsa_paged_mla_attn(const dsa_shape* shape, const dsa_batch* batch,
                              const dsa_pages* pages, const void* q_abs, const void* codes,
                              const void* scales, const int32_t* block_table, const int32_t* idx,
                              const int32_t* n_sel, float* out, float* lse, void* ws,
                              size_t ws_bytes, void* stream) {
    Shape sh;
    BatchDev b;
    PagedCache pc;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if ((s = check_batch(batch, sh, &b)) != DSA_OK) return s;
    if ((s = check_pages(pages, &pc.pg)) != DSA_OK) return s;
    const bool dense = (b.flags & DSA_FLAG_DENSE) != 0;
    if (b.n_q > 0 && (q_abs == nullptr || codes == nullptr || scales == nullptr ||
                      block_table == nullptr || out == nullptr ||
                      (!dense && (idx == nullptr || n_sel == nullptr))))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_abs) || !aligned(codes, 32) || !aligned16(out) || !aligned16(idx) ||
        !aligned(lse, 4) || !aligned(n_sel, 4) || !aligned(block_table, 4))
        return DSA_ERR_INVALID_ARG;
    const size_t need = op_bytes(sh, b, DSA_OP_PAGED_MLA);
    if ((s = check_ws(ws, ws_bytes, need)) != DSA_OK) return s;
    pc.codes = static_cast<const uint8_t*>(codes);
    pc.scales = static_cast<const uint8_t*>(scales);
    pc.block_table = block_table;
    return cuda_status(launch_paged_mla(sh, b, pc, q_abs, dense ? nullptr : idx,
                                        dense ? nullptr : n_sel, out, lse,
                                        bytes(ws) + scratch_off(), need - scratch_off(),
                                        static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)),
                       "paged_mla_attn");
}

dsa_status dsa_rms_norm(int64_t n_rows, int32_t width, int32_t dtype, const void* x, int64_t x_ld,
                        const void* add, int64_t add_ld, const float* weight, float eps, void* total,
                        int64_t total_ld, void* out, int64_t out_ld, int32_t out_format, float* scales,
                        int32_t group, void* stream) {
    const bool e4m3 = out_format == DSA_NORM_E4M3;
    if (n_rows < 0 || width < 1 || (dtype != DSA_F32 && dtype != DSA_BF16) ||
        (out_format != DSA_NORM_SAME && !e4m3) || !isfinite(eps) || !(eps > 0.f))
        return DSA_ERR_INVALID_ARG;
    if (e4m3 ? group != 0 && group != 32 && group != 64 && group != 128 : group != 0)
        return DSA_ERR_INVALID_ARG;
    if (x_ld < width || (add != nullptr && add_ld < width) || (total != nullptr && total_ld < width) ||
        out_ld < width)
        return DSA_ERR_INVALID_ARG;
    if (n_rows > 0 && (x == nullptr || out == nullptr || (e4m3 && scales == nullptr)))
        return DSA_ERR_INVALID_ARG;
    const uintptr_t e = dtype == DSA_BF16 ? 2 : 4;
    if (!aligned(x, e) || !aligned(add, e) || !aligned(total, e) || (!e4m3 && !aligned(out, e)) ||
        !aligned(weight, 4) || !aligned(scales, 4))
        return DSA_ERR_INVALID_ARG;
    if (width > 16384 || n_rows >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
    // an output in an input's place has its rows where they are, and its type; else they are apart
    if (n_rows > 0) {
        struct Tensor { const void* p; Rows rows; wide size; };
        auto rows = [&](const void* p, wide ld, wide size) { return Tensor{p, make_rows(p, n_rows, ld * size, width * size), size}; };
        const wide n_scales = (wide)n_rows * (group == 0 ? 1 : (width + group - 1) / group);
        const Tensor in[] = {rows(x, x_ld, e), rows(add, add_ld, e), {weight, make_rows(weight, 1, 0, (wide)width * 4), 0}};
        const Tensor to[] = {rows(out, out_ld, e4m3 ? 1 : e), rows(total, total_ld, e),
                             {e4m3 ? scales : nullptr, make_rows(scales, 1, 0, n_scales * 4), 0}};
        for (int i = 0; i < 3; ++i) {
            if (to[i].p == nullptr) continue;
            for (int j = 0; j < i; ++j)
                if (to[j].p != nullptr && rows_meet(to[i].rows, to[j].rows)) return DSA_ERR_INVALID_ARG;
            for (int j = 0; j < 3; ++j) {
                if (in[j].p == nullptr || !rows_meet(to[i].rows, in[j].rows)) continue;
                if (j == 2 || to[i].p != in[j].p || to[i].size != in[j].size || to[i].rows.stride != in[j].rows.stride)
                    return DSA_ERR_INVALID_ARG;
            }
        }
    }
    const NormArgs a{n_rows, x_ld, add_ld, total_ld, out_ld, x,     add, weight,
                     total,  out,  scales, width,    group,  eps,   (float)(1.0 / width)};
    return cuda_status(launch_rms_norm(a, dtype, e4m3, static_cast<cudaStream_t>(stream)), "rms_norm");
}

dsa_status dsa_rope_init(dsa_rope_plan* plan, int32_t dims, int32_t layout, int32_t inverse,
                         double base, double factor, double original_len, double beta_fast,
                         double beta_slow, double magnitude) {
    if (plan == nullptr || dims < 2 || (dims & 1) || (layout != DSA_ROPE_PAIRS && layout != DSA_ROPE_HALVES) ||
        (inverse != 0 && inverse != 1) || !isfinite(base) || !(base > 1.0) || !isfinite(factor) ||
        !(factor >= 1.0) || !isfinite((float)magnitude))
        return DSA_ERR_INVALID_ARG;
    if (factor != 1.0 && !(beta_fast == 0.0 && beta_slow == 0.0) &&
        (!isfinite(original_len) || !(original_len > 0.0) || !isfinite(beta_fast) || !(beta_slow > 0.0) ||
         !(beta_fast >= beta_slow)))
        return DSA_ERR_INVALID_ARG;
    if (dims > 2 * DSA_ROPE_MAX_PAIRS) return DSA_ERR_UNSUPPORTED;
    memset(plan, 0, sizeof(*plan));
    plan->dims = dims;
    plan->layout = layout;
    plan->inverse = inverse;
    plan->magnitude = (float)magnitude;
    init_rope_plan(dims, base, factor, original_len, beta_fast, beta_slow, plan->turns);
    return DSA_OK;
}

dsa_status dsa_rope(const dsa_rope_plan* plan, int32_t dtype, int64_t n_tok, int32_t heads,
                    const void* x, int64_t x_tok, int64_t x_head, const int64_t* pos, void* out,
                    int64_t out_tok, int64_t out_head, void* stream) {
    if (plan == nullptr || plan->dims < 2 || (plan->dims & 1) || plan->dims > 2 * DSA_ROPE_MAX_PAIRS ||
        (plan->layout != DSA_ROPE_PAIRS && plan->layout != DSA_ROPE_HALVES) ||
        (dtype != DSA_F32 && dtype != DSA_BF16) || n_tok < 0 || heads < 0)
        return DSA_ERR_INVALID_ARG;
    if (x_tok < 0 || x_head < 0 || out_tok < 0 || out_head < 0) return DSA_ERR_INVALID_ARG;
    // no two of the output's heads, or tokens, share a column
    if (n_tok > 0 && heads > 0) {
        if (x == nullptr || out == nullptr || pos == nullptr) return DSA_ERR_INVALID_ARG;
        const int64_t d = plan->dims;
        const bool inner = heads == 1 || out_head >= d, outer = n_tok == 1 || out_tok >= d;
        if (!inner || !outer) return DSA_ERR_INVALID_ARG;
        if (heads > 1 && n_tok > 1) {
            const bool tok_outer = (__int128)out_tok >= (__int128)(heads - 1) * out_head + d;
            const bool head_outer = (__int128)out_head >= (__int128)(n_tok - 1) * out_tok + d;
            if (!tok_outer && !head_outer) return DSA_ERR_INVALID_ARG;
        }
        if (x == out && ((n_tok > 1 && x_tok != out_tok) || (heads > 1 && x_head != out_head)))
            return DSA_ERR_INVALID_ARG;
    }
    const uintptr_t e = dtype == DSA_BF16 ? 2 : 4;
    if (!aligned(x, e) || !aligned(out, e) || !aligned(pos, 8)) return DSA_ERR_INVALID_ARG;
    if (n_tok >= ((int64_t)1 << 31) || heads > 65536) return DSA_ERR_UNSUPPORTED;
    if (n_tok > 0 && heads > 0) {
        const wide size = (wide)e, d = plan->dims * size;
        const Heads to = make_heads(out, out_tok * size, n_tok, out_head * size, heads, d);
        if (x != out && heads_meet(make_heads(x, x_tok * size, n_tok, x_head * size, heads, d), to))
            return DSA_ERR_INVALID_ARG;
        if (rows_meet(to.rows(), make_rows(pos, 1, 0, (wide)n_tok * 8))) return DSA_ERR_INVALID_ARG;
    }
    return cuda_status(launch_rope(*plan, dtype, n_tok, heads, x, x_tok, x_head, pos, out, out_tok,
                                   out_head, static_cast<cudaStream_t>(stream)),
                       "rope");
}

// The head widths of the expanded form: nope_dim and v_dim.
static dsa_status check_expanded(const Shape& sh, int32_t nope_dim, int32_t v_dim) {
    if (nope_dim < 64 || nope_dim % 64 != 0 || v_dim < 128 || v_dim % 128 != 0) return DSA_ERR_INVALID_ARG;
    if (nope_dim + sh.rope > 256 || v_dim > 256) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

dsa_status dsa_expand_kv(const dsa_shape* shape, int64_t n_rows, int32_t nope_dim, int32_t v_dim,
                         const void* cache, const void* w_uk, const void* w_uv, void* k_nope, void* v,
                         void* ws, size_t ws_bytes, void* stream) {
    Shape sh;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if (n_rows < 0) return DSA_ERR_INVALID_ARG;
    if ((s = check_expanded(sh, nope_dim, v_dim)) != DSA_OK) return s;
    if (n_rows > (1 << 24)) return DSA_ERR_UNSUPPORTED;
    if (n_rows > 0 && (cache == nullptr || w_uk == nullptr || w_uv == nullptr || k_nope == nullptr || v == nullptr))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(cache) || !aligned16(w_uk) || !aligned16(w_uv) || !aligned(k_nope, 32) || !aligned(v, 32))
        return DSA_ERR_INVALID_ARG;
    if ((s = check_ws(ws, ws_bytes, kWsHeaderBytes)) != DSA_OK) return s;
    return cuda_status(launch_expand_kv(sh, n_rows, nope_dim, v_dim, cache, w_uk, w_uv, k_nope, v,
                                        static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)),
                       "expand_kv");
}

dsa_status dsa_expanded_mla_attn(const dsa_shape* shape, const dsa_batch* batch, int32_t nope_dim,
                                 int32_t v_dim, const void* q, const void* k_nope, const void* cache,
                                 const void* v, void* out, float* lse, void* ws, size_t ws_bytes,
                                 void* stream) {
    Shape sh;
    BatchDev b;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if ((s = check_batch(batch, sh, &b, 1 << 24)) != DSA_OK) return s;
    if ((s = check_expanded(sh, nope_dim, v_dim)) != DSA_OK) return s;
    if (b.n_seq > (1 << 20) || b.total_rows >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
    if (b.n_q > 0 && (q == nullptr || k_nope == nullptr || v == nullptr || out == nullptr ||
                      (sh.rope > 0 && cache == nullptr)))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_nope) || !aligned16(cache) || !aligned16(v) || !aligned(out, 32) ||
        !aligned(lse, 4))
        return DSA_ERR_INVALID_ARG;
    if ((s = check_ws(ws, ws_bytes, op_bytes(sh, b, DSA_OP_EXPANDED_MLA))) != DSA_OK) return s;
    return cuda_status(launch_expanded_mla(sh, b, nope_dim, v_dim, q, k_nope, cache, v, out, lse,
                                           bytes(ws) + scratch_off(), static_cast<int32_t*>(ws),
                                           static_cast<cudaStream_t>(stream)),
                       "expanded_mla_attn");
}

dsa_status dsa_decode_step(const dsa_shape* shape, const dsa_batch* batch, const void* q_idx,
                           const float* w, const void* k_idx, const void* q_abs,
                           const void* cache, float* out, float* lse, int32_t* idx_out,
                           int32_t* n_sel_out, void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    int32_t n_q = 0;
    dsa_status s = decode_step_check(shape, batch, q_idx, w, k_idx, q_abs, cache, out, lse,
                                     idx_out, n_sel_out, &need, &n_q);
    if (s != DSA_OK) return s;
    if ((s = check_ws(ws, ws_bytes, need)) != DSA_OK) return s;
    if (n_q == 0) return DSA_OK;
    Shape sh;
    BatchDev b;
    check_shape(shape, &sh);
    check_batch(batch, sh, &b);
    const StepLayout lay = step_layout(sh, b);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int32_t* err = static_cast<int32_t*>(ws);
    if (trace_on())
        fprintf(stderr, "[dsa] decode_step n_q=%d max_kv=%lld flags=%u ws=%zu\n", b.n_q,
                (long long)b.max_kv_len, b.flags, lay.total);
    if (b.flags & DSA_FLAG_DENSE) {
        // the indexer's A/B switch: every visible row, no scoring or selection
        return cuda_status(launch_sparse_mla(sh, b, q_abs, cache, nullptr, nullptr, out, lse,
                                             bytes(ws) + lay.attn, lay.total - lay.attn, err,
                                             /*q_early=*/false, st),
                           "decode_step/dense attention");
    }
    int32_t* idx = idx_out ? idx_out : reinterpret_cast<int32_t*>(bytes(ws) + lay.idx);
    int32_t* n_sel = n_sel_out ? n_sel_out : reinterpret_cast<int32_t*>(bytes(ws) + lay.n_sel);
    const char* what = "";
    cudaError_t e = enqueue_index_select(sh, b, lay, ws, q_idx, w, k_idx, idx, n_sel, cache, st,
                                         &what);
    if (e != cudaSuccess) return cuda_status(e, what);
    // The kernel before the attention is this step's selection, which released
    // its dependents only after waiting for the caller's kernels: the query
    // may be loaded before the attention waits for the selection.
    e = launch_sparse_mla(sh, b, q_abs, cache, idx, n_sel, out, lse, bytes(ws) + lay.attn,
                          lay.total - lay.attn, err, /*q_early=*/true, st);
    return cuda_status(e, "decode_step/sparse_mla_attn");
}

dsa_status dsa_decode_step_host(const dsa_shape* shape, const dsa_batch* batch,
                                const void* h_q_idx, const float* h_w, const void* k_idx,
                                const void* h_q_abs, const void* cache, float* h_out,
                                float* h_lse, int32_t* idx_out, int32_t* n_sel_out, void* ws,
                                size_t ws_bytes, void* stream) {
    Shape sh;
    BatchDev b;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if ((s = check_batch(batch, sh, &b)) != DSA_OK) return s;
    const bool dense = (b.flags & DSA_FLAG_DENSE) != 0;
    // the device's view of the caller's per-step buffers
    const void *q_idx = nullptr, *w = nullptr, *q_abs = nullptr;
    float *out = nullptr, *lse = nullptr;
    if (b.n_q > 0) {
        if (h_q_abs == nullptr || h_out == nullptr || (!dense && (h_q_idx == nullptr || h_w == nullptr)))
            return DSA_ERR_INVALID_ARG;
        q_abs = device_address(h_q_abs);
        out = static_cast<float*>(const_cast<void*>(device_address(h_out)));
        if (q_abs == nullptr || out == nullptr) return DSA_ERR_INVALID_ARG;
        if (!dense) {
            q_idx = device_address(h_q_idx);
            w = device_address(h_w);
            if (q_idx == nullptr || w == nullptr) return DSA_ERR_INVALID_ARG;
        }
        if (h_lse != nullptr) {
            lse = static_cast<float*>(const_cast<void*>(device_address(h_lse)));
            if (lse == nullptr) return DSA_ERR_INVALID_ARG;
        }
    }
    if (!aligned16(q_idx) || !aligned16(w) || !aligned16(q_abs)) return DSA_ERR_INVALID_ARG;
    const StageLayout sl = stage_layout(sh, b);
    void* s_q_idx = dense ? nullptr : bytes(ws) + sl.q_idx;
    float* s_w = dense ? nullptr : reinterpret_cast<float*>(bytes(ws) + sl.w);
    void* s_q_abs = bytes(ws) + sl.q_abs;
    int32_t n_q = 0;
    s = decode_step_check(shape, batch, s_q_idx, s_w, k_idx, s_q_abs, cache, out, lse, idx_out,
                          n_sel_out, nullptr, &n_q);
    if (s != DSA_OK) return s;
    if ((s = check_ws(ws, ws_bytes, sl.total)) != DSA_OK) return s;
    if (n_q == 0) return DSA_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t q_idx_vecs =
        dense ? 0 : (int64_t)b.n_q * sh.idx_heads * sh.idx_dim * (int64_t)sh.elem_bytes() / 16;
    const int64_t q_abs_vecs = (int64_t)b.n_q * sh.heads * sh.width() * (int64_t)sh.elem_bytes() / 16;
    const StageSeg a{static_cast<const uint4*>(q_idx), static_cast<uint4*>(s_q_idx), q_idx_vecs};
    const StageSeg c{static_cast<const uint4*>(q_abs), static_cast<uint4*>(s_q_abs), q_abs_vecs};
    const int64_t w_words = dense ? 0 : (int64_t)b.n_q * sh.idx_heads;
    cudaError_t e = launch_stage_inputs(a, c, static_cast<const uint32_t*>(w),
                                        reinterpret_cast<uint32_t*>(s_w), w_words, st);
    if (e != cudaSuccess) return cuda_status(e, "decode_step_host/stage_inputs");
    return dsa_decode_step(shape, batch, s_q_idx, s_w, k_idx, s_q_abs, cache, out, lse, idx_out,
                           n_sel_out, ws, ws_bytes, stream);
}

dsa_status dsa_index_select(const dsa_shape* shape, const dsa_batch* batch, const void* q_idx,
                            const float* w, const void* k_idx, int32_t* idx, int32_t* n_sel,
                            void* ws, size_t ws_bytes, void* stream) {
    Shape sh;
    BatchDev b;
    dsa_status s = check_shape(shape, &sh);
    if (s != DSA_OK) return s;
    if ((s = check_batch(batch, sh, &b)) != DSA_OK) return s;
    if (b.flags & DSA_FLAG_DENSE) return DSA_ERR_INVALID_ARG;   // no selection to make
    if (b.n_q > 0 && (q_idx == nullptr || w == nullptr || k_idx == nullptr || idx == nullptr ||
                      n_sel == nullptr))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_idx) || !aligned16(w) || !aligned16(k_idx) || !aligned16(idx) ||
        !aligned16(n_sel))
        return DSA_ERR_INVALID_ARG;
    const StepLayout lay = step_layout(sh, b);
    if ((s = check_ws(ws, ws_bytes, lay.attn)) != DSA_OK) return s;
    if (b.n_q == 0) return DSA_OK;
    const char* what = "";
    const cudaError_t e = enqueue_index_select(sh, b, lay, ws, q_idx, w, k_idx, idx, n_sel,
                                               nullptr, static_cast<cudaStream_t>(stream), &what);
    return cuda_status(e, what);
}

dsa_status dsa_check_device_error(void* ws, size_t ws_bytes, void* stream, int32_t* code) {
    if (ws == nullptr) {
        // the no-allocation entry point's scratch array on the current device
        dsa_status s = noalloc_scratch(&ws);
        if (s != DSA_OK) return s;
        ws_bytes = DSA_NOALLOC_SCRATCH_BYTES;
    }
    if (ws_bytes < kWsHeaderBytes) return DSA_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_status(e, "check_device_error/sync");
    int32_t words[3] = {0, 0, 0};
    e = cudaMemcpy(words, ws, sizeof(words), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_status(e, "check_device_error/read");
    if (code != nullptr) *code = words[0];
    if (words[0] == 0) return DSA_OK;
    if (trace_on())
        fprintf(stderr, "[dsa] device error %d (detail %d, kernel %d)\n", words[0], words[1],
                words[2]);
    // an interrupted launch may leave the selection state and the grid
    // barrier dirty: start them from zero again
    e = cudaMemset(ws, 0, ws_bytes < ws_zero_bytes() ? ws_bytes : ws_zero_bytes());
    if (e != cudaSuccess) return cuda_status(e, "check_device_error/clear");
    return words[0] == kDevTimeout ? DSA_ERR_TIMEOUT : DSA_ERR_DEVICE;
}

dsa_status dsa_workspace_init(void* ws, size_t ws_bytes, void* stream) {
    if (ws == nullptr || ws_bytes < kWsHeaderBytes ||
        (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0)
        return DSA_ERR_WORKSPACE;
    const size_t n = ws_bytes < ws_zero_bytes() ? ws_bytes : ws_zero_bytes();
    return cuda_status(cudaMemsetAsync(ws, 0, n, static_cast<cudaStream_t>(stream)),
                       "workspace_init");
}

dsa_status dsa_workspace_set_wait_budget(void* ws, size_t ws_bytes, uint64_t ns, void* stream) {
    if (ws == nullptr || ws_bytes < kWsHeaderBytes ||
        (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0)
        return DSA_ERR_WORKSPACE;
    // from pageable host memory: staged before the call returns
    const uint64_t v = ns;
    return cuda_status(cudaMemcpyAsync(bytes(ws) + kWsWaitBudgetOffset, &v, sizeof(v),
                                       cudaMemcpyHostToDevice, static_cast<cudaStream_t>(stream)),
                       "workspace_set_wait_budget");
}

}  // extern "C"
