// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits.
//
// With m the row's maximum, S0 = sum e^(x - m) and S1 = sum e^(x - m) (x - m):
//   ln p(i) = (x_i - m) - ln S0,   entropy = ln S0 - S1 / S0
// (S1 <= 0, so nothing cancels).
//
// One pass over the logits, bound by their reading: a workgroup holds a
// piece of the row in registers and leaves its maximum, S0 and S1 relative
// to it, and for every group of four lanes the group's best element as one
// 64-bit key (the value's order, then the lower index).  A second kernel, one
// workgroup a row, joins the pieces and finds the top n: the n groups with
// the best keys hold the n best elements (an element outside them has n
// better ones, the groups' own bests), so only their elements are read again.
#include "device_common.h"
#include "serve_kernels.h"

namespace qmv {
namespace {

constexpr int kGroupLanes = 4;
constexpr int kMaxTop = 32;
constexpr float kInf = __builtin_inff();

// A float's place in the order of the floats (-0 and 0 alike, a NaN at the
// place of -infinity), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x == x ? x + 0.f : -kInf);
    return (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t u) {
    return __builtin_bit_cast(float, (u & 0x80000000u) != 0 ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
    return (static_cast<uint64_t>(order_of(x)) << 32) | (0xFFFFFFFFu - index);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
    return (static_cast<uint64_t>(dpp_u32<CTRL>(static_cast<uint32_t>(v >> 32))) << 32) |
           dpp_u32<CTRL>(static_cast<uint32_t>(v));
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, dpp_u32<0xB1>(v));   // lanes 1 apart
    v = max(v, dpp_u32<0x4E>(v));   // 2 apart
    v = max(v, dpp_u32<0x141>(v));  // the other half of eight
    v = max(v, dpp_u32<0x140>(v));  // the other half of sixteen
    const uint32_t a = max(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 0)),
                           static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 16)));
    const uint32_t b = max(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 32)),
                           static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 48)));
    return max(a, b);
}
// The largest of the 64 lanes' keys, in every lane.
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t k) {
    const uint32_t hi = static_cast<uint32_t>(k >> 32);
    const uint32_t mh = wave_max_u32(hi);
    return (static_cast<uint64_t>(mh) << 32) | wave_max_u32(hi == mh ? static_cast<uint32_t>(k) : 0u);
}
__device__ __forceinline__ float wave_max_f32(float v) {
    v = fmaxf(v, dpp_mov<0xB1>(v));
    v = fmaxf(v, dpp_mov<0x4E>(v));
    v = fmaxf(v, dpp_mov<0x141>(v));
    v = fmaxf(v, dpp_mov<0x140>(v));
    return fmaxf(fmaxf(read_lane(v, 0), read_lane(v, 16)), fmaxf(read_lane(v, 32), read_lane(v, 48)));
}

// Four floats at any 4-byte aligned place.
struct __attribute__((packed, aligned(4))) Float4u {
    float x, y, z, w;
};

struct Piece {
    float m, s0, s1, pad;
};

// E values a thread: element (u * 256 + tid) * 4 + c of the piece.
template <int E>
__global__ __launch_bounds__(256) void logits_kernel(const float* __restrict__ x, uint32_t rows, uint32_t vocab,
                                                     uint32_t pieces, Piece* __restrict__ stat,
                                                     uint64_t* __restrict__ keys) {
    __shared__ float red[3][4];
    const uint64_t total = static_cast<uint64_t>(rows) * pieces;
    const int tid = threadIdx.x, wave = tid >> 6;
    for (uint64_t g = blockIdx.x; g < total; g += gridDim.x) {
        const uint64_t row = g / pieces;
        const uint32_t first = static_cast<uint32_t>(g % pieces) * (256 * E);
        const float* p = x + row * vocab;
        float v[E];
#pragma unroll
        for (int u = 0; u < E / 4; ++u) {
            const uint32_t i = first + (u * 256 + tid) * 4;
            if (i + 4 <= vocab) {
                const Float4u t = *reinterpret_cast<const Float4u*>(p + i);
                v[4 * u] = t.x; v[4 * u + 1] = t.y; v[4 * u + 2] = t.z; v[4 * u + 3] = t.w;
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[4 * u + c] = i + c < vocab ? p[i + c] : -kInf;
            }
        }
        float m = -kInf;
#pragma unroll
        for (int e = 0; e < E; ++e) m = fmaxf(m, v[e]);
        if (keys != nullptr) {
            // the first element that has the thread's maximum (one of only
            // NaN and -infinity: its first)
            int at = 0;
#pragma unroll
            for (int e = E - 1; e >= 0; --e) at = v[e] == m ? e : at;
            const uint32_t i = first + ((at >> 2) * 256 + tid) * 4 + (at & 3);
            uint64_t k = i < vocab ? key_of(m, i) : 0;
            k = max64(k, dpp_u64<0xB1>(k));
            k = max64(k, dpp_u64<0x4E>(k));
            if ((tid & 3) == 0) keys[g * (256 / kGroupLanes) + (tid >> 2)] = k;
        }
        m = wave_max_f32(m);
        if ((tid & 63) == 0) red[0][wave] = m;
        __syncthreads();
        m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
        const float ref = m > -kInf ? m : 0.f;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float d = v[e] - ref, t = __expf(d);
            s0 += t;
            s1 += d > -kInf ? t * d : 0.f;
        }
        s0 = wave_reduce(s0);
        s1 = wave_reduce(s1);
        if ((tid & 63) == 0) {
            red[1][wave] = s0;
            red[2][wave] = s1;
        }
        __syncthreads();
        if (tid == 0)
            stat[g] = Piece{m, (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]),
                            (red[2][0] + red[2][1]) + (red[2][2] + red[2][3]), 0.f};
    }
}

// The wave's n largest of its lanes' R keys each, in order, to list.
template <int R>
__device__ __forceinline__ void wave_top(uint64_t (&k)[R], uint32_t n, uint64_t* list) {
    for (uint32_t i = 0; i < n; ++i) {
        uint64_t b = k[0];
#pragma unroll
        for (int r = 1; r < R; ++r) b = max64(b, k[r]);
        b = wave_max_u64(b);
#pragma unroll
        for (int r = 0; r < R; ++r) k[r] = k[r] == b ? 0 : k[r];
        if ((threadIdx.x & 63) == 0) list[i] = b;
    }
}

// The n largest of the four waves' lists (n in each, keys distinct but for
// 0), in order, to best.  Ends with a barrier.
__device__ __forceinline__ void join_top(const uint64_t (&lists)[4][kMaxTop], uint32_t n, uint64_t* best) {
    __syncthreads();
    const uint32_t tid = threadIdx.x;
    if (tid < 4 * n) {
        const uint64_t k = lists[tid / n][tid % n];
        uint32_t rank = 0;
        for (uint32_t w = 0; w < 4; ++w)
            for (uint32_t i = 0; i < n; ++i) rank += lists[w][i] > k ? 1 : 0;
        if (k != 0 && rank < n) best[rank] = k;
    }
    __syncthreads();
}

template <int E>
__global__ __launch_bounds__(256) void logprobs_kernel(LogprobArgs a, uint32_t pieces,
                                                       const Piece* __restrict__ stat,
                                                       const uint64_t* __restrict__ keys) {
    constexpr int R = 16;                       // keys a thread takes at once
    constexpr uint32_t kElems = kGroupLanes * E;  // elements of a group
    __shared__ float red[3][4];
    __shared__ uint64_t lists[4][kMaxTop];
    __shared__ uint64_t groups[kMaxTop], best[kMaxTop];
    const uint64_t row = blockIdx.x;
    const uint32_t tid = threadIdx.x, wave = tid >> 6;
    const float* x = a.logits + row * a.vocab;
    // the row's maximum and sums
    const Piece* st = stat + row * pieces;
    float m = -kInf;
    for (uint32_t i = tid; i < pieces; i += 256) m = fmaxf(m, st[i].m);
    m = wave_max_f32(m);
    if ((tid & 63) == 0) red[0][wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    float s0 = 0.f, s1 = 0.f;
    for (uint32_t i = tid; i < pieces; i += 256) {
        const Piece p = st[i];
        // a piece of nothing but -infinity (and NaN) has its sums relative to 0
        const float d = p.m > -kInf ? p.m - m : (p.s0 == 0.f ? -kInf : 0.f);
        const float f = expf(d);
        s0 += f * p.s0;
        s1 += f != 0.f ? f * (p.s1 + d * p.s0) : 0.f;  // d may be a type's lowest value; a NaN f stays
    }
    s0 = wave_reduce(s0);
    s1 = wave_reduce(s1);
    if ((tid & 63) == 0) {
        red[1][wave] = s0;
        red[2][wave] = s1;
    }
    __syncthreads();
    s0 = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    s1 = (red[2][0] + red[2][1]) + (red[2][2] + red[2][3]);
    // nothing but -infinity: no distribution
    const float ln = s0 > 0.f ? logf(s0) : __builtin_nanf("");
    if (a.entropy != nullptr && tid == 0) a.entropy[row] = ln - s1 / s0;
    for (uint32_t i = tid; i < a.n_ids; i += 256) {
        const int32_t id = a.ids[row * a.n_ids + i];
        const bool in = id >= 0 && static_cast<uint32_t>(id) < a.vocab;
        a.lp[row * a.n_ids + i] = in ? (x[id] - m) - ln : 0.f;
    }
    if (a.top == 0) return;

    // the n best groups, then the n best of their elements
    const uint64_t* gk = keys + row * pieces * (256 / kGroupLanes);
    const uint32_t n_groups = pieces * (256 / kGroupLanes);
    if (tid < kMaxTop) {
        groups[tid] = 0;
        best[tid] = 0;
    }
    __syncthreads();
    for (uint32_t base = 0; base < n_groups; base += 256 * R - kMaxTop) {
        uint64_t k[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t i = r * 256 + tid;    // the best so far come first
            k[r] = i < kMaxTop ? groups[i] : (base + i - kMaxTop < n_groups ? gk[base + i - kMaxTop] : 0);
        }
        wave_top<R>(k, a.top, lists[wave]);
        join_top(lists, a.top, groups);
    }
    const uint32_t all = a.top * kElems;
    for (uint32_t base = 0; base < all; base += 256 * R - kMaxTop) {
        uint64_t k[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t i = r * 256 + tid, j = base + i - kMaxTop;
            k[r] = 0;
            if (i < kMaxTop) {
                k[r] = best[i];
            } else if (j < all && groups[j / kElems] != 0) {
                // the group of a best element: its piece and four lanes
                const uint32_t e = 0xFFFFFFFFu - static_cast<uint32_t>(groups[j / kElems]);
                const uint32_t piece = e / (256 * E), lane4 = (e % 1024) / (4 * kGroupLanes);
                const uint32_t o = j % kElems;
                const uint32_t index = piece * (256 * E) + (o / 16) * 1024 + lane4 * 16 + (o % 16);
                if (index < a.vocab) k[r] = key_of(x[index], index);
            }
        }
        wave_top<R>(k, a.top, lists[wave]);
        join_top(lists, a.top, best);
    }
    if (tid < a.top) {
        const uint64_t k = best[tid];
        a.top_ids[row * a.top + tid] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(k));
        a.top_lp[row * a.top + tid] = (of_order(static_cast<uint32_t>(k >> 32)) - m) - ln;
    }
}

// Values a thread of the first kernel holds: 32, or 8 where that would leave
// compute units idle.
int values(uint64_t rows, uint32_t vocab) {
    return rows * ((vocab + 8191) / 8192) >= 512 ? 32 : 8;
}

}  // namespace

uint64_t logprobs_workspace_bytes(uint32_t rows, uint32_t vocab, uint32_t top) {
    const uint64_t per = 256ull * values(rows, vocab);
    const uint64_t pieces = (vocab + per - 1) / per * rows;
    return pieces * sizeof(Piece) + (top != 0 ? pieces * (256 / kGroupLanes) * 8 : 0);
}

hipError_t launch_logprobs(const LogprobArgs& a, void* workspace, hipStream_t s) {
    const int e = values(a.rows, a.vocab);
    const uint32_t per = 256u * e;
    const uint32_t pieces = (a.vocab + per - 1) / per;
    const uint64_t total = uint64_t{pieces} * a.rows;
    Piece* stat = static_cast<Piece*>(workspace);
    uint64_t* keys = a.top != 0 ? reinterpret_cast<uint64_t*>(stat + total) : nullptr;
    const dim3 grid(static_cast<uint32_t>(total < 0x7FFFFFFFull ? total : 0x7FFFFFFFull)), block(256);
    if (e == 32)
        hipLaunchKernelGGL(logits_kernel<32>, grid, block, 0, s, a.logits, a.rows, a.vocab, pieces, stat, keys);
    else
        hipLaunchKernelGGL(logits_kernel<8>, grid, block, 0, s, a.logits, a.rows, a.vocab, pieces, stat, keys);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (e == 32)
        hipLaunchKernelGGL(logprobs_kernel<32>, dim3(a.rows), block, 0, s, a, pieces, stat, keys);
    else
        hipLaunchKernelGGL(logprobs_kernel<8>, dim3(a.rows), block, 0, s, a, pieces, stat, keys);
    return hipGetLastError();
}

}  // namespace qmv
