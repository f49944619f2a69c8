// Launchers of the kernels behind qmv_serve.h (internal to libqmv).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "qmv_serve.h"

namespace qmv {

struct NormArgs {
    const float* x;
    const float* res;   // may be null
    const float* w;
    float* sum;         // outputs: each may be null
    float* y;
    uint16_t* y_bf16;
    int8_t* q;
    float* d;
    uint32_t rows, cols;
    float eps;
    double inv_cols;    // 1 / cols
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream);

hipError_t launch_kv_write(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype,
                           const void* k, const void* v, hipStream_t stream);
hipError_t launch_kv_read(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype, void* k,
                          void* v, hipStream_t stream);

uint64_t kv_attend_workspace_bytes(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype,
                                   uint32_t heads, uint32_t window);
hipError_t launch_kv_attend(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype,
                            uint32_t heads, float scale, uint32_t window, const void* q, void* out,
                            void* workspace, hipStream_t stream);

struct LogprobArgs {
    const float* logits;
    const int32_t* ids;  // may be null (n_ids 0)
    float* lp;           // outputs: each may be null
    float* entropy;
    int32_t* top_ids;
    float* top_lp;
    uint32_t rows, vocab, n_ids, top;
};
uint64_t logprobs_workspace_bytes(uint32_t rows, uint32_t vocab, uint32_t top);
hipError_t launch_logprobs(const LogprobArgs& a, void* workspace, hipStream_t stream);

}  // namespace qmv
