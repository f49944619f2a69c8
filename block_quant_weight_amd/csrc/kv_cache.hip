// The 8-bit key/value cache: quantizing tokens as they are written into their
// pages, and reading them back.
//
// A page of 64 tokens holds, per key/value head, 64 x D codes of keys
// ([token][dim]) and of values ([dim][token]) and one scale of each.  A scale
// is a power of two, d = 2^e with the least e such that the largest magnitude
// amax of what is written is at most 127 d; codes are x / d to the nearest
// whole number.  Powers of two because a page fills over many calls: when a
// larger value arrives, the earlier codes are rescaled, and as each growth at
// least doubles d the roundings of all of them sum to less than one d
// (d0/2 + d1/2 + ... + dn/2 < dn), where scales of amax / 127 could lose half
// a step at each of 64 writes.  It also makes a stored value exact in
// bfloat16 and the quotient x / d exact.
//
// One workgroup owns (page, head, keys or values): it finds amax of the new
// tokens, settles the scale, rescales the earlier tokens where the scale
// grew, and writes the new codes, so nothing is shared between workgroups
// and the result does not depend on their order.  Values are turned through
// shared memory, whose rows of 64 tokens are 68 bytes apart (17 words: odd,
// so that neighbouring dims fall into different banks).
#include "kv_common.h"

namespace qmv {
namespace {

#pragma clang fp contract(off)

constexpr int kPitch = kPage + 4;

// Least power of two d from 2^-126 with amax <= 127 d, at most 2^121 (a code
// of 64 times 2^122 would be infinite); 0 for 0; NaN for an infinity or NaN
// (bits of a magnitude).
__device__ __forceinline__ float scale_for(uint32_t amax_bits) {
    if (amax_bits == 0) return 0.f;
    if (amax_bits >= 0x7F800000u) return __builtin_nanf("");
    // amax = 1.f 2^X, 127 = 1.984375 2^6: e = X - 6, one more if 1.f > 1.984375
    int e = static_cast<int>(amax_bits >> 23) - 127 - 6 + ((amax_bits & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
    e = min(max(e, -126), 121);
    return __builtin_bit_cast(float, static_cast<uint32_t>(e + 127) << 23);
}

// x / d to the nearest whole number, in -127 .. 127; 0 where d is 0 or NaN.
__device__ __forceinline__ uint32_t code(float x, float inv, bool none) {
    if (none) return 0;
    const float r = fminf(fmaxf(rintf(x * inv), -127.f), 127.f);
    return static_cast<uint32_t>(static_cast<int>(r)) & 0xFFu;
}

// Four codes rescaled by old / new.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    uint32_t o = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const float v = static_cast<float>(static_cast<int8_t>(w >> (8 * b)));
        const float r = fminf(fmaxf(rintf(v * ratio), -127.f), 127.f);
        o |= (static_cast<uint32_t>(static_cast<int>(r)) & 0xFFu) << (8 * b);
    }
    return o;
}

__device__ __forceinline__ uint32_t wg_max(uint32_t v, uint32_t* lds) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), m)));
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return max(max(lds[0], lds[1]), max(lds[2], lds[3]));
}

// grid: x = sequence * kv_heads + head, y = the sequence's touched pages
// (strided), z = 0 keys, 1 values.
template <uint32_t DT, int D>
__global__ __launch_bounds__(256) void kv_write_kernel(qmv_kv_cache c, qmv_kv_seqs s,
                                                       const typename Elem<DT>::type* __restrict__ k,
                                                       const typename Elem<DT>::type* __restrict__ v) {
    constexpr int CPT = D / 8;                    // chunks of 8 values a token
    constexpr int PER = kPage * CPT / 256;        // chunks a thread
    __shared__ uint32_t red[4];
    __shared__ __attribute__((aligned(16))) uint8_t turn[D * kPitch];
    const uint32_t seq = blockIdx.x / c.kv_heads, head = blockIdx.x % c.kv_heads;
    const bool values = blockIdx.z != 0;
    const int tid = threadIdx.x;
    const SeqRows r = seq_rows(s, seq);
    if (r.count == 0 || r.len == 0) return;
    const int32_t from = max(r.base, 0);               // first new position
    const int32_t last = (r.len - 1) / kPage;
    const typename Elem<DT>::type* src = values ? v : k;
    for (int32_t p = from / kPage + blockIdx.y; p <= last; p += gridDim.y) {
        const int32_t id = page_id(c, s, seq, p);
        if (id < 0) continue;
        const int lo = max(from - p * kPage, 0);
        const int hi = min(r.len - p * kPage, kPage);
        const int32_t row0 = r.first + (p * kPage - r.base);      // row of the page's token 0
        float x[PER][8];
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int ch = tid + 256 * u, t = ch / CPT, dim = (ch % CPT) * 8;
            if (t >= lo && t < hi) {
                load8<DT>(src + (static_cast<uint64_t>(row0 + t) * c.kv_heads + head) * D + dim, x[u]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[u][j] = 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < PER; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(uint32_t, x[u][j]) & 0x7FFFFFFFu);
        m = wg_max(m, red);
        const uint64_t at = static_cast<uint64_t>(id) * c.kv_heads + head;
        float* sp = (values ? c.v_scale : c.k_scale) + at;
        const float old = lo == 0 ? 0.f : *sp;
        const float need = scale_for(m);
        // a NaN, of now or of before, stays
        const float d = need != need ? need : (old != old ? old : fmaxf(old, need));
        const bool none = !(d > 0.f);
        const bool grew = lo > 0 && !none && old < d;
        const float ratio = grew ? old / d : 1.f;
        const float inv = none ? 0.f : 1.f / d;
        __syncthreads();                          // every thread has read the old scale and `red`
        if (tid == 0) *sp = d;
        uint8_t* page = reinterpret_cast<uint8_t*>(values ? c.v : c.k) + at * (kPage * D);
        if (!values) {
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int ch = tid + 256 * u, t = ch / CPT, dim = (ch % CPT) * 8;
                uint2* q = reinterpret_cast<uint2*>(page + t * D + dim);
                if (t >= lo && t < hi) {
                    uint32_t w[2] = {0, 0};
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j >> 2] |= code(x[u][j], inv, none) << (8 * (j & 3));
                    *q = make_uint2(w[0], w[1]);
                } else if (grew && t < lo) {
                    const uint2 w = *q;
                    *q = make_uint2(rescale4(w.x, ratio), rescale4(w.y, ratio));
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int ch = tid + 256 * u, t = ch / CPT, dim = (ch % CPT) * 8;
                if (t >= lo && t < hi) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        turn[(dim + j) * kPitch + t] = static_cast<uint8_t>(code(x[u][j], inv, none));
                }
            }
            __syncthreads();
            for (int i = tid; i < D * (kPage / 4); i += 256) {
                const int dim = i / (kPage / 4), t = (i % (kPage / 4)) * 4;  // tokens t .. t + 3
                if (t >= hi || (t + 4 <= lo && !grew)) continue;
                uint32_t* q = reinterpret_cast<uint32_t*>(page + dim * kPage + t);
                uint32_t fresh = *reinterpret_cast<const uint32_t*>(&turn[dim * kPitch + t]);
                if (t < lo || t + 4 > hi) {
                    // bytes of earlier tokens (rescaled) and of later places (kept)
                    const uint32_t was = *q;
                    const uint32_t early = grew ? rescale4(was, ratio) : was;
                    uint32_t w = 0;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint32_t pick = t + b < lo ? early : (t + b < hi ? fresh : was);
                        w |= pick & (0xFFu << (8 * b));
                    }
                    fresh = w;
                }
                *q = fresh;
            }
            __syncthreads();                      // `turn` is used again
        }
    }
}

template <uint32_t DT, int D>
__global__ __launch_bounds__(256) void kv_read_kernel(qmv_kv_cache c, qmv_kv_seqs s,
                                                      typename Elem<DT>::type* __restrict__ k,
                                                      typename Elem<DT>::type* __restrict__ v) {
    constexpr int CPT = D / 8;
    constexpr int PER = kPage * CPT / 256;
    __shared__ __attribute__((aligned(16))) uint8_t turn[D * kPitch];
    const uint32_t seq = blockIdx.x / c.kv_heads, head = blockIdx.x % c.kv_heads;
    const bool values = blockIdx.z != 0;
    typename Elem<DT>::type* dst = values ? v : k;
    if (dst == nullptr) return;
    const int tid = threadIdx.x;
    const SeqRows r = seq_rows(s, seq);
    if (r.count == 0) return;
    // pages that hold the rows, from the one below position 0 that rows
    // without a place count as (floor division)
    const int32_t first = (r.base >= 0 ? r.base : r.base - (kPage - 1)) / kPage;
    const int32_t last = (r.len + kPage - 1) / kPage - 1;
    for (int32_t p = first + blockIdx.y; p <= last; p += gridDim.y) {
        const int32_t id = page_id(c, s, seq, p);
        const int lo = max(r.base - p * kPage, 0);
        const int hi = min(r.len - p * kPage, kPage);
        const int32_t row0 = r.first + (p * kPage - r.base);
        const uint64_t at = static_cast<uint64_t>(id < 0 ? 0 : id) * c.kv_heads + head;
        const float d = id < 0 ? 0.f : (values ? c.v_scale : c.k_scale)[at];
        const uint8_t* page = reinterpret_cast<const uint8_t*>(values ? c.v : c.k) + at * (kPage * D);
        if (values && id >= 0) {
            for (int i = tid; i < D * (kPage / 4); i += 256) {
                const int dim = i / (kPage / 4), t = (i % (kPage / 4)) * 4;
                *reinterpret_cast<uint32_t*>(&turn[dim * kPitch + t]) =
                    *reinterpret_cast<const uint32_t*>(page + dim * kPage + t);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int ch = tid + 256 * u, t = ch / CPT, dim = (ch % CPT) * 8;
            if (t < lo || t >= hi) continue;
            float o[8];
            if (id < 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = 0.f;
            } else if (!values) {
                const uint2 w = *reinterpret_cast<const uint2*>(page + t * D + dim);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] = static_cast<float>(static_cast<int8_t>((j < 4 ? w.x : w.y) >> (8 * (j & 3)))) * d;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] = static_cast<float>(static_cast<int8_t>(turn[(dim + j) * kPitch + t])) * d;
            }
            store8<DT>(dst + (static_cast<uint64_t>(row0 + t) * c.kv_heads + head) * D + dim, o);
        }
        if (values) __syncthreads();
    }
}

// Touched pages of a sequence, as far as the host knows, up to the grid's limit.
uint32_t pages_hint(const qmv_kv_seqs& s) {
    const uint64_t n = s.max_new < s.rows ? s.max_new : s.rows;
    const uint64_t p = n <= 1 ? 1 : (n + kPage - 2) / kPage + 1;
    return static_cast<uint32_t>(p < 4096 ? p : 4096);
}

}  // namespace

hipError_t launch_kv_write(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype, const void* k,
                           const void* v, hipStream_t stream) {
    const dim3 grid(s.seqs * c.kv_heads, pages_hint(s), 2), block(256);
#define QMV_KV_GO(DT, D)                                                                             \
    hipLaunchKernelGGL((kv_write_kernel<DT, D>), grid, block, 0, stream, c, s,                       \
                       static_cast<const Elem<DT>::type*>(k), static_cast<const Elem<DT>::type*>(v))
    if (dtype == QMV_F32) {
        if (c.head_dim == 64) QMV_KV_GO(QMV_F32, 64);
        else if (c.head_dim == 128) QMV_KV_GO(QMV_F32, 128);
        else QMV_KV_GO(QMV_F32, 256);
    } else {
        if (c.head_dim == 64) QMV_KV_GO(QMV_BF16, 64);
        else if (c.head_dim == 128) QMV_KV_GO(QMV_BF16, 128);
        else QMV_KV_GO(QMV_BF16, 256);
    }
#undef QMV_KV_GO
    return hipGetLastError();
}

hipError_t launch_kv_read(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype, void* k, void* v,
                          hipStream_t stream) {
    const dim3 grid(s.seqs * c.kv_heads, pages_hint(s), 2), block(256);
#define QMV_KV_GO(DT, D)                                                                             \
    hipLaunchKernelGGL((kv_read_kernel<DT, D>), grid, block, 0, stream, c, s,                        \
                       static_cast<Elem<DT>::type*>(k), static_cast<Elem<DT>::type*>(v))
    if (dtype == QMV_F32) {
        if (c.head_dim == 64) QMV_KV_GO(QMV_F32, 64);
        else if (c.head_dim == 128) QMV_KV_GO(QMV_F32, 128);
        else QMV_KV_GO(QMV_F32, 256);
    } else {
        if (c.head_dim == 64) QMV_KV_GO(QMV_BF16, 64);
        else if (c.head_dim == 128) QMV_KV_GO(QMV_BF16, 128);
        else QMV_KV_GO(QMV_BF16, 256);
    }
#undef QMV_KV_GO
    return hipGetLastError();
}

}  // namespace qmv
