// C-ABI entry points of qmv_serve.h: argument checks on the host, then the
// launch of the kernels on the caller's stream.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "qmv_serve.h"
#include "serve_kernels.h"

namespace {

constexpr uint32_t kDimLimit = 1u << 24;
// Workgroups (of up to 512 threads) along a grid's first axis: a launch holds
// fewer than 2^32 threads there.
constexpr uint32_t kGridLimit = 1u << 22;

bool aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// As in the product calls: an error that an earlier call of this thread left
// is cleared, so that the launch's own is reported.
int enqueue(hipError_t e) {
    if (e == hipSuccess) return QMV_OK;
    return e == hipErrorOutOfMemory ? QMV_E_NOMEM : QMV_E_DEVICE;
}

int check_kv(const qmv_kv_cache* c, const qmv_kv_seqs* s, uint32_t dtype) {
    if (c == nullptr || s == nullptr || dtype > QMV_BF16) return QMV_E_ARG;
    if (c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr) return QMV_E_ARG;
    if (s->table == nullptr || s->len == nullptr || s->start == nullptr) return QMV_E_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
        return QMV_E_ARG;
    if (!aligned(s->table, 4) || !aligned(s->len, 4) || !aligned(s->start, 4)) return QMV_E_ARG;
    if (c->pages == 0 || c->kv_heads == 0 || s->seqs == 0 || s->table_stride == 0 || s->rows == 0)
        return QMV_E_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QMV_E_SHAPE;
    if (c->kv_heads > 65535 || c->pages > 0x7FFFFFFFu || s->rows > 0x7FFF0000u ||
        uint64_t{s->seqs} * c->kv_heads > kGridLimit || uint64_t{c->pages} * c->kv_heads > 0x7FFFFFFFu ||
        uint64_t{s->seqs} * s->table_stride > 0x7FFFFFFFu)
        return QMV_E_SHAPE;
    return QMV_OK;
}

int check_heads(const qmv_kv_cache* c, const qmv_kv_seqs* s, uint32_t heads) {
    if (heads == 0 || heads % c->kv_heads != 0 || heads > kDimLimit) return QMV_E_SHAPE;
    return uint64_t{s->rows} * heads > 0x7FFF0000u ? QMV_E_SHAPE : QMV_OK;
}

}  // namespace

extern "C" {

int qmv_rms_norm(const float* x, const float* res, const float* w, float eps, uint32_t rows,
                 uint32_t cols, float* sum, float* y, uint16_t* y_bf16, int8_t* q, float* d,
                 void* stream) {
    if (x == nullptr || w == nullptr || rows == 0) return QMV_E_ARG;
    if (sum == nullptr && y == nullptr && y_bf16 == nullptr && q == nullptr) return QMV_E_ARG;
    if ((q == nullptr) != (d == nullptr)) return QMV_E_ARG;
    if (!(eps >= 0.f) || std::isinf(eps)) return QMV_E_ARG;
    for (const void* p : {static_cast<const void*>(x), static_cast<const void*>(res),
                          static_cast<const void*>(w), static_cast<const void*>(sum),
                          static_cast<const void*>(y), static_cast<const void*>(y_bf16),
                          static_cast<const void*>(q), static_cast<const void*>(d)})
        if (!aligned(p, 16)) return QMV_E_ARG;
    if (cols == 0 || cols % 32 != 0 || cols > kDimLimit) return QMV_E_SHAPE;
    (void)hipGetLastError();
    const qmv::NormArgs a{x, res, w, sum, y, y_bf16, q, d, rows, cols, eps, 1.0 / cols};
    return enqueue(qmv::launch_rms_norm(a, static_cast<hipStream_t>(stream)));
}

int qmv_kv_write(const qmv_kv_cache* cache, const qmv_kv_seqs* seqs, uint32_t dtype, const void* k,
                 const void* v, void* stream) {
    const int st = check_kv(cache, seqs, dtype);
    if (st != QMV_OK) return st;
    if (k == nullptr || v == nullptr || !aligned(k, 16) || !aligned(v, 16)) return QMV_E_ARG;
    (void)hipGetLastError();
    return enqueue(qmv::launch_kv_write(*cache, *seqs, dtype, k, v, static_cast<hipStream_t>(stream)));
}

int qmv_kv_read(const qmv_kv_cache* cache, const qmv_kv_seqs* seqs, uint32_t dtype, void* k,
                void* v, void* stream) {
    const int st = check_kv(cache, seqs, dtype);
    if (st != QMV_OK) return st;
    if ((k == nullptr && v == nullptr) || !aligned(k, 16) || !aligned(v, 16)) return QMV_E_ARG;
    (void)hipGetLastError();
    return enqueue(qmv::launch_kv_read(*cache, *seqs, dtype, k, v, static_cast<hipStream_t>(stream)));
}

int qmv_kv_attend_workspace(const qmv_kv_cache* cache, const qmv_kv_seqs* seqs, uint32_t dtype,
                            uint32_t heads, uint32_t window, uint64_t* bytes) {
    if (bytes == nullptr) return QMV_E_ARG;
    *bytes = 0;
    int st = check_kv(cache, seqs, dtype);
    if (st == QMV_OK) st = check_heads(cache, seqs, heads);
    if (st != QMV_OK) return st;
    *bytes = qmv::kv_attend_workspace_bytes(*cache, *seqs, dtype, heads, window);
    return QMV_OK;
}

int qmv_kv_attend(const qmv_kv_cache* cache, const qmv_kv_seqs* seqs, uint32_t dtype,
                  uint32_t heads, float scale, uint32_t window, const void* q, void* out,
                  void* workspace, uint64_t workspace_bytes, void* stream) {
    int st = check_kv(cache, seqs, dtype);
    if (st == QMV_OK) st = check_heads(cache, seqs, heads);
    if (st != QMV_OK) return st;
    if (q == nullptr || out == nullptr || !std::isfinite(scale)) return QMV_E_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16)) return QMV_E_ARG;
    const uint64_t need = qmv::kv_attend_workspace_bytes(*cache, *seqs, dtype, heads, window);
    if (need != 0 && (workspace == nullptr || workspace_bytes < need)) return QMV_E_ARG;
    (void)hipGetLastError();
    return enqueue(qmv::launch_kv_attend(*cache, *seqs, dtype, heads, scale, window, q, out, workspace,
                                         static_cast<hipStream_t>(stream)));
}

int qmv_logprobs_workspace(uint32_t rows, uint32_t vocab, uint32_t top, uint64_t* bytes) {
    if (bytes == nullptr) return QMV_E_ARG;
    *bytes = 0;
    if (rows == 0 || vocab == 0) return QMV_E_ARG;
    if (vocab > kDimLimit || top > 32 || top > vocab || rows > (1u << 22)) return QMV_E_SHAPE;
    *bytes = qmv::logprobs_workspace_bytes(rows, vocab, top);
    return QMV_OK;
}

int qmv_logprobs(const float* logits, uint32_t rows, uint32_t vocab, const int32_t* ids,
                 uint32_t n_ids, uint32_t top, float* lp, float* entropy, int32_t* top_ids,
                 float* top_lp, void* workspace, uint64_t workspace_bytes, void* stream) {
    uint64_t need = 0;
    const int st = qmv_logprobs_workspace(rows, vocab, top, &need);
    if (st != QMV_OK) return st;
    if (logits == nullptr || (lp == nullptr && entropy == nullptr && top_ids == nullptr)) return QMV_E_ARG;
    if (lp != nullptr && (ids == nullptr || n_ids == 0)) return QMV_E_ARG;
    if ((top_ids == nullptr) != (top_lp == nullptr) || (top == 0) != (top_ids == nullptr)) return QMV_E_ARG;
    for (const void* p : {static_cast<const void*>(logits), static_cast<const void*>(ids),
                          static_cast<const void*>(lp), static_cast<const void*>(entropy),
                          static_cast<const void*>(top_ids), static_cast<const void*>(top_lp)})
        if (!aligned(p, 4)) return QMV_E_ARG;
    if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need) return QMV_E_ARG;
    (void)hipGetLastError();
    const qmv::LogprobArgs a{logits, lp != nullptr ? ids : nullptr, lp, entropy, top_ids, top_lp,
                             rows, vocab, lp != nullptr ? n_ids : 0u, top};
    return enqueue(qmv::launch_logprobs(a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
