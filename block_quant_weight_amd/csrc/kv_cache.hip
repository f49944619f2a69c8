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
// and the result does not depend on their order.  A thread has 4 tokens x 8
// dims: rows are read and written in whole lines, and the values' codes are
// turned 4 x 4 in registers (two byte permutations a word) on their way
// through shared memory, whose rows of 64 tokens are 68 bytes apart (17
// words: odd, so that neighbouring dims fall into different banks).
//
// Bound by memory.  8 heads of 128: prompts of up to 4096 bfloat16 tokens (4
// sequences) written in 18.6 us and read back in 15.9, 4.0 TB/s over both; one
// float32 token for each of 64 sequences written in 6.3 us (a launch and two
// dependent trips to memory, the page's id and the page), their last 100 read
// back in 15.8 us, 4.1 TB/s.
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

// Codes of four values: x / d to the nearest whole number, in -127 .. 127.
// Added to 1.5 2^23, the whole number is the sum's low bits (the quotient
// by a power of two is exact, so the sum rounds once).
__device__ __forceinline__ uint32_t code4(const float* x, float inv) {
    constexpr float kMagic = 12582912.f;
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        u[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(fmaf(x[j], inv, kMagic), kMagic - 127.f, kMagic + 127.f));
    const uint32_t a = __builtin_amdgcn_perm(u[1], u[0], 0x00000400u);
    const uint32_t b = __builtin_amdgcn_perm(u[3], u[2], 0x04000000u);
    return __builtin_amdgcn_perm(b, a, 0x07060100u);
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

// Four words of four bytes turned: byte i of out[b] is byte b of in[i].
__device__ __forceinline__ void turn4(const uint32_t in[4], uint32_t out[4]) {
    const uint32_t a = __builtin_amdgcn_perm(in[1], in[0], 0x05010400u);
    const uint32_t b = __builtin_amdgcn_perm(in[3], in[2], 0x05010400u);
    const uint32_t c = __builtin_amdgcn_perm(in[1], in[0], 0x07030602u);
    const uint32_t d = __builtin_amdgcn_perm(in[3], in[2], 0x07030602u);
    out[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    out[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    out[2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
    out[3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
}

// Threads of a workgroup, and pieces of 4 tokens x 8 dims each has.
template <int D>
struct Shape {
    static constexpr int NT = D == 64 ? 128 : 256;
    static constexpr int PER = 2 * D / NT;
};

template <int NT>
__device__ __forceinline__ uint32_t wg_max(uint32_t v, uint32_t* lds) {
    v = wave_max_u32(v);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) v = max(v, lds[w]);
    return v;
}

// Eight values as they come: their largest magnitude (as float bits), and
// their codes.  bfloat16 stays packed until its codes are made.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <uint32_t DT>
struct Eight;
template <>
struct Eight<QMV_F32> {
    float v[8];
    __device__ __forceinline__ void load(const float* p) { load8<QMV_F32>(p, v); }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
    typedef uint32_t Max;
    __device__ __forceinline__ void most(Max& m) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
    }
    static __device__ __forceinline__ uint32_t bits(Max m) { return m; }
    __device__ __forceinline__ uint32_t codes(int h, float inv) const { return code4(v + 4 * h, inv); }
};
template <>
struct Eight<QMV_BF16> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const uint16_t* p) {
        const uint4 t = *reinterpret_cast<const uint4*>(p);
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
    }
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
    typedef u16x2 Max;
    __device__ __forceinline__ void most(Max& m) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[j] & 0x7FFF7FFFu));
    }
    static __device__ __forceinline__ uint32_t bits(Max m) {
        const uint32_t a = m[0], b = m[1];
        return max(a, b) << 16;
    }
    __device__ __forceinline__ uint32_t codes(int h, float inv) const {
        float v[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            v[2 * j] = __builtin_bit_cast(float, w[2 * h + j] << 16);
            v[2 * j + 1] = __builtin_bit_cast(float, w[2 * h + j] & 0xFFFF0000u);
        }
        return code4(v, inv);
    }
};

// grid: x = sequence * kv_heads + head, y = the sequence's touched pages
// (strided), z = 0 keys, 1 values.
template <uint32_t DT, int D>
__global__ __launch_bounds__(Shape<D>::NT) void kv_write_kernel(qmv_kv_cache c, qmv_kv_seqs s,
                                                                const typename Elem<DT>::type* __restrict__ k,
                                                                const typename Elem<DT>::type* __restrict__ v) {
    constexpr int NT = Shape<D>::NT, PER = Shape<D>::PER, CPT = D / 8;
    __shared__ uint32_t red[NT / 64];
    __shared__ __attribute__((aligned(16))) uint8_t turn[D * kPitch];
    const uint32_t seq = blockIdx.x / c.kv_heads, head = blockIdx.x % c.kv_heads;
    const bool values = blockIdx.z != 0;
    const int tid = threadIdx.x;
    const SeqRows r = seq_rows(s, seq);
    if (r.count == 0 || r.len == 0) return;
    const int32_t from = max(r.base, 0);                        // first new position
    const int32_t last = (r.len - 1) / kPage;
    const typename Elem<DT>::type* src = values ? v : k;
    for (int32_t p = from / kPage + blockIdx.y; p <= last; p += gridDim.y) {
        const int lo = max(from - p * kPage, 0);
        const int hi = min(r.len - p * kPage, kPage);
        const int32_t row0 = r.first + (p * kPage - r.base);      // row of the page's token 0
        // the rows and the page's id are on the way together
        Eight<DT> x[PER][4];
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int ch = tid + NT * u, t = ch / CPT * 4, dim = ch % CPT * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[u][i].clear();
                if (t + i >= lo && t + i < hi)
                    x[u][i].load(src + (static_cast<uint64_t>(row0 + t + i) * c.kv_heads + head) * D + dim);
            }
        }
        const int32_t id = page_id(c, s, seq, p);
        if (id < 0) continue;
        const uint64_t at = static_cast<uint64_t>(id) * c.kv_heads + head;
        float* sp = (values ? c.v_scale : c.k_scale) + at;
        const float old = lo == 0 ? 0.f : *sp;
        uint8_t* page = reinterpret_cast<uint8_t*>(values ? c.v : c.k) + at * (kPage * D);
        // values: words of four tokens that hold earlier tokens or later
        // places beside new ones, the first and the last that are written
        uint32_t was[2] = {0, 0};
        if (values && tid < D) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(page + tid * kPage);
            if ((lo & 3) != 0) was[0] = q[lo >> 2];
            if ((hi & 3) != 0) was[1] = q[hi >> 2];
        }
        typename Eight<DT>::Max most = {};
#pragma unroll
        for (int u = 0; u < PER; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i].most(most);
        const uint32_t m = wg_max<NT>(Eight<DT>::bits(most), red);
        const float need = scale_for(m);
        // a NaN, of now or of before, stays
        const float d = need != need ? need : (old != old ? old : fmaxf(old, need));
        const bool none = !(d > 0.f);
        const bool grew = lo > 0 && !none && old < d;
        const float ratio = grew ? old / d : 1.f;
        const float inv = none ? 0.f : 1.f / d;
        __syncthreads();                          // every thread has read the old scale and `red`
        if (tid == 0) *sp = d;
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int ch = tid + NT * u, t = ch / CPT * 4, dim = ch % CPT * 8;
            uint32_t w[2][4];                     // codes of dims 0 .. 3, 4 .. 7 of each token
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    w[h][i] = none ? 0u : x[u][i].codes(h, inv);
                }
            if (!values) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint2* q = reinterpret_cast<uint2*>(page + (t + i) * D + dim);
                    if (t + i >= lo && t + i < hi) {
                        *q = make_uint2(w[0][i], w[1][i]);
                    } else if (grew && t + i < lo) {
                        const uint2 o = *q;
                        *q = make_uint2(rescale4(o.x, ratio), rescale4(o.y, ratio));
                    }
                }
            } else if (t < hi && t + 4 > lo) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[4];
                    turn4(w[h], o);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint32_t*>(&turn[(dim + 4 * h + j) * kPitch + t]) = o[j];
                }
            }
        }
        if (values) {
            __syncthreads();
            // whole words of new tokens, and of earlier ones if they change
            const int w_lo = (lo + 3) >> 2, w_hi = hi >> 2, w_from = grew ? 0 : w_lo;
            for (int i = tid; i < D * (kPage / 4); i += NT) {
                const int dim = i / (kPage / 4), w = i % (kPage / 4);
                uint32_t* q = reinterpret_cast<uint32_t*>(page + dim * kPage) + w;
                if (w >= w_lo && w < w_hi) *q = *reinterpret_cast<const uint32_t*>(&turn[dim * kPitch + 4 * w]);
                else if (w >= w_from && w < lo >> 2) *q = rescale4(*q, ratio);
            }
            // words that hold both, and later places, which stay
            if (tid < D) {
                uint32_t* q = reinterpret_cast<uint32_t*>(page + tid * kPage);
                const uint32_t* n = reinterpret_cast<const uint32_t*>(&turn[tid * kPitch]);
                const uint32_t early = grew ? rescale4(was[0], ratio) : was[0];
                // bytes below lo, and from hi on
                const uint32_t below = (1u << (8 * (lo & 3))) - 1, above = ~((1u << (8 * (hi & 3))) - 1);
                if ((lo & 3) != 0 && lo >> 2 == hi >> 2) {   // (hi is then no multiple of 4)
                    q[lo >> 2] = (early & below) | (n[lo >> 2] & ~below & ~above) | (was[1] & above);
                } else {
                    if ((lo & 3) != 0) q[lo >> 2] = (early & below) | (n[lo >> 2] & ~below);
                    if ((hi & 3) != 0) q[hi >> 2] = (n[hi >> 2] & ~above) | (was[1] & above);
                }
            }
            __syncthreads();                      // `turn` is used again
        }
    }
}

template <uint32_t DT, int D>
__global__ __launch_bounds__(Shape<D>::NT) void kv_read_kernel(qmv_kv_cache c, qmv_kv_seqs s,
                                                               typename Elem<DT>::type* __restrict__ k,
                                                               typename Elem<DT>::type* __restrict__ v) {
    constexpr int NT = Shape<D>::NT, PER = Shape<D>::PER, CPT = D / 8;
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
        // (without a page: page 0 times 0)
        const uint64_t at = static_cast<uint64_t>(max(id, 0)) * c.kv_heads + head;
        const float d = id < 0 ? 0.f : (values ? c.v_scale : c.k_scale)[at];
        const uint8_t* page = reinterpret_cast<const uint8_t*>(values ? c.v : c.k) + at * (kPage * D);
        if (values) {
            for (int i = tid; i < D * (kPage / 16); i += NT) {
                const int dim = i / (kPage / 16), t = (i % (kPage / 16)) * 16;
                const uint4 w = *reinterpret_cast<const uint4*>(page + dim * kPage + t);
                uint32_t* o = reinterpret_cast<uint32_t*>(&turn[dim * kPitch + t]);
                o[0] = w.x; o[1] = w.y; o[2] = w.z; o[3] = w.w;
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int ch = tid + NT * u, t = ch / CPT * 4, dim = ch % CPT * 8;
            if (t >= hi || t + 4 <= lo) continue;
            uint32_t w[2][4];
            if (!values) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint2 o = *reinterpret_cast<const uint2*>(page + (t + i) * D + dim);
                    w[0][i] = o.x;
                    w[1][i] = o.y;
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[j] = *reinterpret_cast<const uint32_t*>(&turn[(dim + 4 * h + j) * kPitch + t]);
                    turn4(o, w[h]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (t + i < lo || t + i >= hi) continue;
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] = id < 0 ? 0.f : static_cast<float>(static_cast<int8_t>(w[j >> 2][i] >> (8 * (j & 3)))) * d;
                store8<DT>(dst + (static_cast<uint64_t>(row0 + t + i) * c.kv_heads + head) * D + dim, o);
            }
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
    const dim3 grid(s.seqs * c.kv_heads, pages_hint(s), 2), block(c.head_dim == 64 ? 128 : 256);
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
    const dim3 grid(s.seqs * c.kv_heads, pages_hint(s), 2), block(c.head_dim == 64 ? 128 : 256);
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
