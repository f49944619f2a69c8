// What the 4-bit cache's kernels share: the format of a page and its
// conversions.
#pragma once
#include "kv_common.h"

namespace qmv {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// A block is 32 channels of one token and head: codes of a sign and an index
// into 0, .5, 1, 1.5, 2, 3, 4, 6 (two exponent bits and one of fraction, what
// gfx950 converts in one instruction a pair), times 2^(byte - 127).
constexpr int kBlock = 32;
constexpr uint32_t kByteMin = 2, kByteMax = 252;   // scales 2^-125 to 2^125: stored values are normal and finite
constexpr uint32_t kByteNan = 255;                 // of a key: the token is no number

// Byte offsets in one page and head of D channels: where token t has the
// codes of channels 8 c .. 8 c + 7, and the scale of block b.  Keys lie token
// by token.  Values lie in groups of four tokens, and in a group by
// sixteenths of the head: the bytes of four tokens and one sixteenth are
// neighbours, which is what a lane of the output's product takes.
template <int D>
__host__ __device__ constexpr uint32_t k_at(uint32_t t, uint32_t c) { return t * (D / 2) + 4 * c; }
template <int D>
__host__ __device__ constexpr uint32_t v_at(uint32_t t, uint32_t channel) {
    constexpr uint32_t each = D / 16;             // channels of a sixteenth
    return ((t / 4 * 16 + channel / each) * 4 + t % 4) * (each / 2) + channel % each / 2;
}
template <int D>
__host__ __device__ constexpr uint32_t k_scale_at(uint32_t t, uint32_t b) { return (t % 16 * (D / kBlock) + b) * 4 + t / 16; }
template <int D>
__host__ __device__ constexpr uint32_t v_scale_at(uint32_t t, uint32_t b) {
    return ((t % 16 / 4 * (D / kBlock) + b) * 4 + t / 16) * 4 + t % 4;
}
// Bytes of a page and head: codes, and scales.
template <int D>
constexpr uint32_t kCodeBytes = kPage * D / 2;
template <int D>
constexpr uint32_t kScaleBytes = kPage * D / kBlock;

// Scale byte of a block from the bits of its largest magnitude, a number: the
// least d = 2^e with amax <= 7 d.  (6 is the largest value; between 6 d and 7 d
// its error is at most d, as between 4 d and 6 d.)
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    // amax = 1.f 2^X, 7 = 1.75 2^2: e = X - 2, one more if 1.f > 1.75
    const int e = static_cast<int>(amax_bits >> 23) - 2 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(min(max(e, static_cast<int>(kByteMin)), static_cast<int>(kByteMax)));
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// Eight values as codes, the first in the lowest bits: x / d to the nearest
// value, halves to the even code, at most 6.
__device__ __forceinline__ uint32_t codes8(const float x[8], float d) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], d, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], d, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], d, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], d, 3);
    return w;
}

// The two codes of byte B of a word as what they stand for, exactly.
template <int B>
__device__ __forceinline__ uint32_t pair_bf16(uint32_t w, float d) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, d, B));
}
// As float16 (rounded below 2^-24, infinite past 65504).
template <int B>
__device__ __forceinline__ uint32_t pair_f16(uint32_t w, float d) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, d, B));
}
// Eight codes as bfloat16 values.
__device__ __forceinline__ bf16x8 values8(uint32_t w, float d) {
    const uint4 u = make_uint4(pair_bf16<0>(w, d), pair_bf16<1>(w, d), pair_bf16<2>(w, d), pair_bf16<3>(w, d));
    return __builtin_bit_cast(bf16x8, u);
}

}  // namespace qmv
