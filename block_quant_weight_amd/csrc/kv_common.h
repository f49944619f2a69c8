// What the cache's kernels share: which rows a sequence has, where a token
// lives, and bfloat16 / float32 loads and stores.
#pragma once
#include "device_common.h"
#include "serve_kernels.h"

namespace qmv {

constexpr int kPage = QMV_KV_PAGE;

// Rows [first, first + count) of sequence i, at positions base + 0 ..
// count - 1 (base may be negative), of `len` tokens.  All below 2^31; base
// >= -2^31 + 1 as count <= rows < 2^31.
struct SeqRows {
    int32_t first, count, base, len;
};
__device__ __forceinline__ SeqRows seq_rows(const qmv_kv_seqs& s, uint32_t i) {
    const int32_t rows = static_cast<int32_t>(s.rows);
    const int32_t a = min(max(s.start[i], 0), rows);
    const int32_t b = min(max(s.start[i + 1], a), rows);
    // (lengths end 2^31 - 2^16 early, so that a page past one is counted without overflow)
    const int32_t len = min(max(s.len[i], 0), 0x7FFF0000);
    return SeqRows{a, b - a, len - (b - a), len};
}

// Page id of a sequence's page number p, or -1 where there is none.
__device__ __forceinline__ int32_t page_id(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t seq, int32_t p) {
    if (p < 0 || static_cast<uint32_t>(p) >= s.table_stride) return -1;
    const int32_t id = s.table[static_cast<uint64_t>(seq) * s.table_stride + p];
    return id >= 0 && static_cast<uint32_t>(id) < c.pages ? id : -1;
}

template <uint32_t DT>
struct Elem;
template <>
struct Elem<QMV_F32> {
    typedef float type;
};
template <>
struct Elem<QMV_BF16> {
    typedef uint16_t type;
};

// Eight consecutive values at p (16-byte aligned).
template <uint32_t DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::type* p, float v[8]) {
    if constexpr (DT == QMV_F32) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
            v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
        }
    }
}
template <uint32_t DT>
__device__ __forceinline__ void store8(typename Elem<DT>::type* p, const float v[8]) {
    if constexpr (DT == QMV_F32) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        bf16x8 b;
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = static_cast<__bf16>(v[i]);
        *reinterpret_cast<bf16x8*>(p) = b;
    }
}

}  // namespace qmv
