// Keys by which logits are ordered: the value's place in the order of the
// floats above the lower index.  Nothing but arithmetic, so that a host
// program can list what the kernels list.
#pragma once
#include <cstdint>

namespace qmv {

// A float's place in the order of the floats (-0 and 0 alike, a NaN at the
// place of -infinity), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x == x ? x + 0.f : -__builtin_inff());
    return (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t u) {
    return __builtin_bit_cast(float, (u & 0x80000000u) != 0 ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
    return (static_cast<uint64_t>(order_of(x)) << 32) | (0xFFFFFFFFu - index);
}

// Row index of a thread's element e, of those from `first` on.
__device__ __forceinline__ uint32_t index_of(int e, uint32_t tid, uint32_t first) {
    return first + (static_cast<uint32_t>(e >> 2) * 256 + tid) * 4 + static_cast<uint32_t>(e & 3);
}

// The largest key of a thread's elements, whose maximum is m: of the first that
// has it, or, where there are only NaN and -infinity, which are of one place,
// of the first; 0 of a thread without elements.
template <int E>
__device__ __forceinline__ uint64_t best_key(const float (&v)[E], float m, uint32_t tid, uint32_t first, uint32_t vocab) {
    int at = 0;
#pragma unroll
    for (int e = E - 1; e >= 0; --e) at = v[e] == m ? e : at;
    if (!(m > -__builtin_inff())) at = 0;
    const uint32_t i = index_of(at, tid, first);
    return i < vocab ? key_of(m, i) : 0;
}

}  // namespace qmv
