// The 4-bit key/value cache: quantizing tokens as they are written into their
// pages, and reading them back.
//
// A block of 32 channels of one token and head has its own scale, so what is
// stored of a token depends on that token alone: no call changes an earlier
// token, and a page needs no first write.  A thread has 8 channels of keys and
// of values; a block is four neighbouring lanes, a token's head D / 8.
//
// A workgroup has 256 / (D / 8) neighbouring tokens of a head at a time, whose
// bytes in a page are neighbours too; the next one has the next head of the
// same tokens, which is the neighbour in the rows.  Bound by memory: four prompts
// of up to 4096 tokens (8 heads of 128, bfloat16, 56 MB a call) are written and
// read back in 30 us, 3.8 TB/s (heads one after the other, each with all its
// tokens: 32.7; a workgroup with 64 tokens: 32.3 to 35); 64 sequences of one
// token, with 100 read back as float32, in 16.6.
#include "kv4_common.h"

namespace qmv {
namespace {

constexpr int kThreads = 256;

// Largest over four neighbouring lanes, in each.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, dpp_u32<0xB1>(v));
    return max(v, dpp_u32<0x4E>(v));
}

// Where a thread's token lies: its place in the codes' and scales' arrays (in
// pages and heads) and in its page; false: nowhere.
struct Place {
    uint64_t at;
    uint32_t t;
};
__device__ __forceinline__ bool find(const qmv_kv4_cache& c, const qmv_kv_seqs& s, uint32_t seq, uint32_t head, int32_t pos, Place* o) {
    const int32_t id = pos < 0 ? -1 : page_id(c, s, seq, pos / kPage);
    if (id < 0) return false;
    o->at = static_cast<uint64_t>(id) * c.kv_heads + head;
    o->t = static_cast<uint32_t>(pos % kPage);
    return true;
}

// Writes 4 bytes of values' codes, channels 8 c .. 8 c + 7.
template <int D>
__device__ __forceinline__ void put_v(uint8_t* p, uint32_t t, uint32_t c, uint32_t w) {
    if constexpr (D == 64) {     // two sixteenths of 4 channels
        *reinterpret_cast<uint16_t*>(p + v_at<D>(t, 8 * c)) = static_cast<uint16_t>(w);
        *reinterpret_cast<uint16_t*>(p + v_at<D>(t, 8 * c + 4)) = static_cast<uint16_t>(w >> 16);
    } else {
        *reinterpret_cast<uint32_t*>(p + v_at<D>(t, 8 * c)) = w;
    }
}
template <int D>
__device__ __forceinline__ uint32_t get_v(const uint8_t* p, uint32_t t, uint32_t c) {
    if constexpr (D == 64) {
        return *reinterpret_cast<const uint16_t*>(p + v_at<D>(t, 8 * c)) |
               static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + v_at<D>(t, 8 * c + 4))) << 16;
    } else {
        return *reinterpret_cast<const uint32_t*>(p + v_at<D>(t, 8 * c));
    }
}

template <uint32_t DT, int D>
__global__ __launch_bounds__(kThreads) void write4_kernel(Kv4Args a) {
    typedef typename Elem<DT>::type T;
    constexpr uint32_t L = D / 8, kTokens = kThreads / L;   // lanes of a token and head
    const uint32_t seq = blockIdx.x, lane = threadIdx.x & 63, c = threadIdx.x % L;
    const SeqRows r = seq_rows(a.s, seq);
    const uint64_t blocks = (static_cast<uint64_t>(r.count) + kTokens - 1) / kTokens * a.c.kv_heads;
    for (uint64_t n = blockIdx.y; n < blocks; n += gridDim.y) {
        const uint32_t head = static_cast<uint32_t>(n % a.c.kv_heads);
        const uint32_t tok = static_cast<uint32_t>(n / a.c.kv_heads) * kTokens + threadIdx.x / L;
        if (tok >= static_cast<uint32_t>(r.count)) continue;
        const int32_t t = static_cast<int32_t>(tok);
        const uint64_t from = (static_cast<uint64_t>(r.first + t) * a.c.kv_heads + head) * D + 8 * c;
        float k[8], v[8];
        load8<DT>(static_cast<const T*>(a.k_in) + from, k);
        load8<DT>(static_cast<const T*>(a.v_in) + from, v);
        Place at;
        const bool there = find(a.c, a.s, seq, head, r.base + t, &at);
        uint32_t km = 0, vm = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            km = max(km, __builtin_bit_cast(uint32_t, k[j]) & 0x7FFFFFFFu);
            vm = max(vm, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
        }
        // whether any lane of the token's head holds what is no number
        const uint64_t bad = __ballot(max(km, vm) >= 0x7F800000u);
        const bool none = (bad >> (lane / L * L) & ((2ull << (L - 1)) - 1)) != 0;
        const uint32_t kb = scale_byte(quad_max(km)), vb = scale_byte(quad_max(vm));
        if (!there) continue;
        uint8_t* ks = a.c.k_scale + at.at * kScaleBytes<D> + k_scale_at<D>(at.t, c / 4);
        uint8_t* vs = a.c.v_scale + at.at * kScaleBytes<D> + v_scale_at<D>(at.t, c / 4);
        *reinterpret_cast<uint32_t*>(a.c.k + at.at * kCodeBytes<D> + k_at<D>(at.t, c)) = none ? 0u : codes8(k, scale_of(kb));
        put_v<D>(a.c.v + at.at * kCodeBytes<D>, at.t, c, none ? 0u : codes8(v, scale_of(vb)));
        if (c % 4 == 0) {
            *ks = static_cast<uint8_t>(none ? kByteNan : kb);
            *vs = static_cast<uint8_t>(none ? kByteMin : vb);
        }
    }
}

template <uint32_t DT, int D>
__global__ __launch_bounds__(kThreads) void read4_kernel(Kv4Args a) {
    typedef typename Elem<DT>::type T;
    constexpr uint32_t L = D / 8, kTokens = kThreads / L;
    const uint32_t seq = blockIdx.x, c = threadIdx.x % L;
    const SeqRows r = seq_rows(a.s, seq);
    const uint64_t blocks = (static_cast<uint64_t>(r.count) + kTokens - 1) / kTokens * a.c.kv_heads;
    for (uint64_t n = blockIdx.y; n < blocks; n += gridDim.y) {
        const uint32_t head = static_cast<uint32_t>(n % a.c.kv_heads);
        const uint32_t tok = static_cast<uint32_t>(n / a.c.kv_heads) * kTokens + threadIdx.x / L;
        if (tok >= static_cast<uint32_t>(r.count)) continue;
        const int32_t t = static_cast<int32_t>(tok);
        const uint64_t to = (static_cast<uint64_t>(r.first + t) * a.c.kv_heads + head) * D + 8 * c;
        Place at;
        const bool there = find(a.c, a.s, seq, head, r.base + t, &at);
        uint32_t kw = 0, vw = 0, kb = kByteMin, vb = kByteMin;
        if (there) {
            kw = *reinterpret_cast<const uint32_t*>(a.c.k + at.at * kCodeBytes<D> + k_at<D>(at.t, c));
            vw = get_v<D>(a.c.v + at.at * kCodeBytes<D>, at.t, c);
            kb = a.c.k_scale[at.at * kScaleBytes<D> + k_scale_at<D>(at.t, c / 4)];
            vb = a.c.v_scale[at.at * kScaleBytes<D> + v_scale_at<D>(at.t, c / 4)];
        }
        auto give = [&](void* out, uint32_t w, uint32_t byte) {
            const bf16x8 v = values8(w, scale_of(byte));
            if constexpr (DT == QMV_BF16) {
                *reinterpret_cast<bf16x8*>(static_cast<T*>(out) + to) = v;
            } else {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = static_cast<float>(v[j]);
                store8<DT>(static_cast<T*>(out) + to, x);
            }
        };
        if (a.k_out != nullptr) give(a.k_out, kw, kb);
        if (a.v_out != nullptr) give(a.v_out, vw, kb == kByteNan ? kByteNan : vb);
    }
}

template <uint32_t DT, int D>
hipError_t go(const Kv4Args& a, bool write, hipStream_t s) {
    const uint64_t most = a.s.max_new < a.s.rows ? a.s.max_new : a.s.rows;
    constexpr uint32_t kTokens = kThreads / (D / 8);
    uint64_t y = (most + kTokens - 1) / kTokens * a.c.kv_heads;
    if (y < 1) y = 1;
    if (y > 65535) y = 65535;
    const dim3 grid(a.s.seqs, static_cast<uint32_t>(y)), block(kThreads);
    if (write) hipLaunchKernelGGL((write4_kernel<DT, D>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((read4_kernel<DT, D>), grid, block, 0, s, a);
    return hipGetLastError();
}
template <uint32_t DT>
hipError_t go(const Kv4Args& a, bool write, hipStream_t s) {
    if (a.c.head_dim == 64) return go<DT, 64>(a, write, s);
    if (a.c.head_dim == 128) return go<DT, 128>(a, write, s);
    return go<DT, 256>(a, write, s);
}

}  // namespace

hipError_t launch_kv4_write(const qmv_kv4_cache& c, const qmv_kv_seqs& s, uint32_t dtype, const void* k, const void* v, hipStream_t stream) {
    const Kv4Args a{c, s, k, v, nullptr, nullptr};
    return dtype == QMV_F32 ? go<QMV_F32>(a, true, stream) : go<QMV_BF16>(a, true, stream);
}
hipError_t launch_kv4_read(const qmv_kv4_cache& c, const qmv_kv_seqs& s, uint32_t dtype, void* k, void* v, hipStream_t stream) {
    const Kv4Args a{c, s, nullptr, nullptr, k, v};
    return dtype == QMV_F32 ? go<QMV_F32>(a, false, stream) : go<QMV_BF16>(a, false, stream);
}

}  // namespace qmv
