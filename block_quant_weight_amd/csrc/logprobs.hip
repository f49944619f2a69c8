// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits.
//
// With m the row's maximum, S0 = sum e^(x - m) and S1 = sum e^(x - m) (x - m):
//   ln p(i) = (x_i - m) - ln S0,   entropy = ln S0 - S1 / S0
// (S1 <= 0, so nothing cancels).
//
// One pass over the logits, bound by their reading: a workgroup holds a
// piece of the row in registers and leaves its maximum, S0 and S1 relative
// to it, and for every group of 128 elements (of 8 or 16 lanes) its best
// element as one 64-bit key (the value's order, then the lower index).  A
// second kernel, one workgroup a row, joins the pieces and finds the top n: the n groups with
// the best keys hold the n best elements (an element outside them has n
// better ones, the groups' own bests), so only their elements are read again.
// Both searches list what reaches a bound that few pass, and place each listed
// key by counting the larger ones.  Rows of up to 8192 are done by one kernel.
//
// 64 rows of 248320: 12.6 us for the first kernel, 5.0 TB/s, and 7.2 for the
// second, a chain of six trips to memory or barriers; one row: 3.1 and 7.0.
#include "device_common.h"
#include "logprob_keys.h"
#include "serve_kernels.h"

namespace qmv {
namespace {

constexpr uint32_t kGroup = 128;   // elements of a group: 8 lanes' of 16, or 16 lanes' of 8
constexpr int kMaxTop = 32;
constexpr float kInf = __builtin_inff();

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
    return (static_cast<uint64_t>(dpp_u32<CTRL>(static_cast<uint32_t>(v >> 32))) << 32) |
           dpp_u32<CTRL>(static_cast<uint32_t>(v));
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

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

// E values a thread: element first + (u * 256 + thread) * 4 + c of the row,
// -infinity past its end.
template <int E>
__device__ __forceinline__ void load_piece(const float* p, uint32_t first, uint32_t vocab, float (&v)[E]) {
#pragma unroll
    for (int u = 0; u < E / 4; ++u) {
        const uint32_t i = index_of(4 * u, threadIdx.x, first);
        if (i + 4 <= vocab) {
            const Float4u t = *reinterpret_cast<const Float4u*>(p + i);
            v[4 * u] = t.x; v[4 * u + 1] = t.y; v[4 * u + 2] = t.z; v[4 * u + 3] = t.w;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) v[4 * u + c] = i + c < vocab ? p[i + c] : -kInf;
        }
    }
}

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
        load_piece<E>(p, first, vocab, v);
        float m = -kInf;
#pragma unroll
        for (int e = 0; e < E; ++e) m = fmaxf(m, v[e]);
        if (keys != nullptr) {
            uint64_t k = best_key<E>(v, m, tid, first, vocab);
            k = max64(k, dpp_u64<0xB1>(k));
            k = max64(k, dpp_u64<0x4E>(k));
            k = max64(k, dpp_u64<0x141>(k));
            if constexpr (E == 8) k = max64(k, dpp_u64<0x140>(k));
            constexpr int kLanes = kGroup / E;
            if (tid % kLanes == 0) keys[g * (256 / kLanes) + tid / kLanes] = k;
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

// The n-th largest of the wave's 64 keys (distinct where not 0), 0 if fewer
// than n are not 0: each lane counts the keys above its own.
__device__ __forceinline__ uint64_t wave_nth(uint64_t k, uint32_t n) {
    const int lo = static_cast<int>(k), hi = static_cast<int>(k >> 32);
    uint32_t above = 0;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
        const uint64_t o = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, i))) << 32 |
                           static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, i));
        above += o > k ? 1u : 0u;
    }
    const uint64_t at = __ballot(above == n - 1 && k != 0);
    if (at == 0) return 0;
    const int lane = __builtin_ctzll(at);
    return static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, lane))) << 32 |
           static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, lane));
}

constexpr uint32_t kList = 4096;   // candidates that a workgroup holds

// Appends the wave's keys that are at least `from` (and not 0) to the list, which
// holds CAP.  The callers' bounds keep the count below that; it is held to CAP here
// and where it is read all the same, so that no row can write past the list's end.
template <int R, uint32_t CAP>
__device__ __forceinline__ void collect(const uint64_t (&k)[R], uint64_t from, uint64_t* list, uint32_t* count) {
    uint64_t take[R];
    uint32_t all = 0;
    if (from == 0) from = 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        take[r] = __ballot(k[r] >= from);
        all += __builtin_popcountll(take[r]);
    }
    if (all == 0) return;
    uint32_t at = 0;
    if ((threadIdx.x & 63) == 0) at = atomicAdd(count, all);
    at = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(at)));
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (take[r] == 0) continue;
        const uint32_t before = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(take[r] >> 32),
                                                          __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(take[r]), 0));
        if ((take[r] >> (threadIdx.x & 63) & 1) != 0 && at + before < CAP) list[at + before] = k[r];
        at += __builtin_popcountll(take[r]);
    }
}

// The n largest of the list's keys (all distinct), in order, to best: every
// key's place is the number of larger ones, whatever the list's order.  Four
// threads count for two keys, each a quarter of the list eight keys at a time,
// with zeros after its end.
__device__ __forceinline__ void place(uint64_t* list, uint32_t count, uint32_t n, uint64_t* best) {
    const uint32_t end = (count + 31) & ~31u, tid = threadIdx.x;
    if (tid < end - count) list[count + tid] = 0;
    __syncthreads();
    for (uint32_t base = 0; base < count; base += 128) {
        const uint32_t i = base + (tid >> 2);
        const uint64_t k0 = i < count ? list[i] : 0, k1 = i + 64 < count ? list[i + 64] : 0;
        uint32_t r0 = 0, r1 = 0;
        for (uint32_t j = 8 * (tid & 3); j < end; j += 32) {
            uint64_t o[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) o[u] = list[j + u];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                r0 += o[u] > k0 ? 1 : 0;
                r1 += o[u] > k1 ? 1 : 0;
            }
        }
        r0 += dpp_u32<0xB1>(r0);
        r1 += dpp_u32<0xB1>(r1);
        r0 += dpp_u32<0x4E>(r0);
        r1 += dpp_u32<0x4E>(r1);
        if ((tid & 3) == 0) {
            if (k0 != 0 && r0 < n) best[r0] = k0;
            if (k1 != 0 && r1 < n) best[r1] = k1;
        }
    }
    __syncthreads();
}

// A group's elements, from one of them: the first, and how far element o is from it.
template <int E>
__device__ __forceinline__ uint32_t group_first(uint32_t e) {
    constexpr uint32_t kStrip = 4 * (kGroup / E);   // elements side by side
    return e / (256 * E) * (256 * E) + e % 1024 / kStrip * kStrip;
}
template <int E>
__device__ __forceinline__ uint32_t in_group(uint32_t o) {
    constexpr uint32_t kStrip = 4 * (kGroup / E);
    return o / kStrip * 1024 + o % kStrip;
}

template <int E>
__global__ __launch_bounds__(256) void logprobs_kernel(LogprobArgs a, uint32_t pieces,
                                                       const Piece* __restrict__ stat,
                                                       const uint64_t* __restrict__ keys) {
    constexpr int R = 8, RE = 10;                 // keys, elements a thread takes at once (20 groups' in one turn)
    constexpr uint32_t kLanes = kGroup / E;       // lanes of a group
    static_assert(4 * kMaxTop * R + kMaxTop <= kList && kMaxTop * kGroup <= kList, "candidates fit the list");
    __shared__ float red[3][4];
    __shared__ __attribute__((aligned(16))) uint64_t list[kList + 32];
    __shared__ uint64_t groups[kMaxTop], best[kMaxTop], bound[4];
    __shared__ uint32_t count;
    const uint64_t row = blockIdx.x;
    const uint32_t tid = threadIdx.x;
    const uint32_t wave = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(tid >> 6)));
    const float* x = a.logits + row * a.vocab;
    // the first pieces and the groups' keys are on the way together
    const Piece* st = stat + row * pieces;
    const Piece none = {-kInf, 0.f, 0.f, 0.f}, own = tid < pieces ? st[tid] : none;
    int32_t id = -1;
    if (tid < a.n_ids) id = a.ids[row * a.n_ids + tid];
    const uint64_t* gk = keys + row * pieces * (256 / kLanes);
    const uint32_t n_groups = pieces * (256 / kLanes);
    uint64_t k[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t i = r * 256 + tid;
        k[r] = a.top != 0 && i < n_groups ? gk[i] : 0;
    }
    // the row's maximum and sums
    float m = own.m;
    for (uint32_t i = tid + 256; i < pieces; i += 256) m = fmaxf(m, st[i].m);
    m = wave_max_f32(m);
    if ((tid & 63) == 0) red[0][wave] = m;
    float xid = 0.f;
    if (id >= 0 && static_cast<uint32_t>(id) < a.vocab) xid = x[id];
    __syncthreads();
    m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    float s0 = 0.f, s1 = 0.f;
    for (uint32_t i = tid; i < pieces; i += 256) {
        const Piece p = i == tid ? own : st[i];
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
        if (i >= 256) {
            id = a.ids[row * a.n_ids + i];
            if (id >= 0 && static_cast<uint32_t>(id) < a.vocab) xid = x[id];
        }
        a.lp[row * a.n_ids + i] = id >= 0 && static_cast<uint32_t>(id) < a.vocab ? (xid - m) - ln : 0.f;
    }
    if (a.top == 0) return;

    // The n best groups.  Of each wave's lanes, the n with the best keys hold
    // its n best, so the n-th of them is a bound that at least n keys reach
    // and few others; the largest of the four waves' bounds is taken.  At most
    // n lanes of a wave reach it, so at most 4 n R keys are listed.
    if (tid < kMaxTop) {
        groups[tid] = 0;
        best[tid] = 0;
    }
    for (uint32_t base = 0; base < n_groups; base += 256 * R) {
        uint64_t b = 0;
        if (base != 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t i = base + r * 256 + tid;
                k[r] = i < n_groups ? gk[i] : 0;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) b = max64(b, k[r]);
        b = wave_nth(b, a.top);
        if ((tid & 63) == 0) bound[wave] = b;
        if (tid == 0) count = 0;
        __syncthreads();
        b = max64(max64(bound[0], bound[1]), max64(bound[2], bound[3]));
        collect<R, kList>(k, b, list, &count);
        // the best of the batches before
        if (base != 0 && tid < a.top && groups[tid] != 0) {
            const uint32_t at = atomicAdd(&count, 1);
            if (at < kList) list[at] = groups[tid];
        }
        __syncthreads();
        // The elements of the first listed groups (there are about four to
        // each of the n) are fetched while these are placed: a line of 128
        // bytes a thread.
        float ahead[2];
#pragma unroll
        for (uint32_t u = 0; u < 2; ++u) {
            const uint32_t i = u * 64 + tid / 4;
            const uint64_t g = i < min(count, kList) ? list[i] : 0;
            const uint32_t at = group_first<E>(0xFFFFFFFFu - static_cast<uint32_t>(g)) + in_group<E>(tid % 4 * 32);
            ahead[u] = x[g != 0 && at < a.vocab ? at : 0];
        }
        place(list, min(count, kList), a.top, groups);
        asm volatile("" ::"v"(ahead[0]), "v"(ahead[1]));
    }
    // Their elements that reach the last of them (its value is looked at
    // first: most are below it).
    const uint64_t last = groups[a.top - 1];
    const float least = last != 0 ? of_order(static_cast<uint32_t>(last >> 32)) : -kInf;
    if (tid == 0) count = 0;
    __syncthreads();
    // (half of the workgroup has a group at a time; lane i knows group i)
    const uint32_t mine = static_cast<uint32_t>(groups[tid % kMaxTop]), off = in_group<E>(tid % kGroup);
    for (uint32_t base = 0; base < a.top; base += 2 * RE) {
        uint64_t k[RE];
        float v[RE];
        uint32_t index[RE];
#pragma unroll
        for (int r = 0; r < RE; ++r) {
            const uint32_t i = base + 2 * r + wave / 2;
            const uint32_t g = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(mine), static_cast<int>(i % kMaxTop)));
            const uint32_t at = group_first<E>(0xFFFFFFFFu - g) + off;
            // (the rest of a key is never 0)
            index[r] = i < a.top && g != 0 && at < a.vocab ? at : a.vocab;
            v[r] = x[index[r] < a.vocab ? index[r] : 0];
        }
#pragma unroll
        for (int r = 0; r < RE; ++r) {
            const bool may = index[r] < a.vocab && !(v[r] < least);
            k[r] = 0;
            if (__any(may) && may) k[r] = key_of(v[r], index[r]);
        }
        collect<RE, kList>(k, last, list, &count);
    }
    __syncthreads();
    place(list, min(count, kList), a.top, best);
    if (tid < a.top) {
        const uint64_t k = best[tid];
        a.top_ids[row * a.top + tid] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(k));
        a.top_lp[row * a.top + tid] = (of_order(static_cast<uint32_t>(k >> 32)) - m) - ln;
    }
}

// Rows of at most 256 E elements, in one kernel: a workgroup has its row in
// registers, and the bound of the best elements is that of the threads' bests.
// (One row, this / the two kernels, us: 500 elements 4.3 / 17, 1500 4.9 / 81, as
// few groups mean many candidates; 4000 6.1 / 8.9, 8000 8.3 / 9.2; 2000 rows of
// 8000 28 / 30.  Rows longer than 8192 would need more registers than a thread
// may have for four workgroups a compute unit.)
template <int E>
__global__ __launch_bounds__(256) void logprobs_row_kernel(LogprobArgs a) {
    // at most n threads of a wave have a key that reaches the bound
    constexpr uint32_t kRowList = 4 * kMaxTop * E;
    __shared__ __attribute__((aligned(16))) uint64_t list[kRowList + 32];
    __shared__ float red[3][4];
    __shared__ uint64_t best[kMaxTop], bound[4];
    __shared__ uint32_t count;
    const uint64_t row = blockIdx.x;
    const uint32_t tid = threadIdx.x, wave = tid >> 6;
    const float* x = a.logits + row * a.vocab;
    int32_t id = -1;
    if (tid < a.n_ids) id = a.ids[row * a.n_ids + tid];
    float v[E];
    load_piece<E>(x, 0, a.vocab, v);
    float m = -kInf;
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, v[e]);
    if (a.top != 0) {
        const uint64_t b = wave_nth(best_key<E>(v, m, tid, 0, a.vocab), a.top);
        if ((tid & 63) == 0) bound[wave] = b;
        if (tid == 0) count = 0;
        if (tid < kMaxTop) best[tid] = 0;
    }
    m = wave_max_f32(m);
    if ((tid & 63) == 0) red[0][wave] = m;
    float xid = 0.f;
    if (id >= 0 && static_cast<uint32_t>(id) < a.vocab) xid = x[id];
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
    if (a.top != 0) {
        const uint64_t from = max64(max64(bound[0], bound[1]), max64(bound[2], bound[3]));
        const float least = from != 0 ? of_order(static_cast<uint32_t>(from >> 32)) : -kInf;
        uint64_t k[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t i = index_of(e, tid, 0);
            const bool may = i < a.vocab && !(v[e] < least);
            k[e] = 0;
            if (__any(may) && may) k[e] = key_of(v[e], i);
        }
        collect<E, kRowList>(k, from, list, &count);
    }
    __syncthreads();
    s0 = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    s1 = (red[2][0] + red[2][1]) + (red[2][2] + red[2][3]);
    const float ln = s0 > 0.f ? logf(s0) : __builtin_nanf("");
    if (a.entropy != nullptr && tid == 0) a.entropy[row] = ln - s1 / s0;
    for (uint32_t i = tid; i < a.n_ids; i += 256) {
        if (i >= 256) {
            id = a.ids[row * a.n_ids + i];
            if (id >= 0 && static_cast<uint32_t>(id) < a.vocab) xid = x[id];
        }
        a.lp[row * a.n_ids + i] = id >= 0 && static_cast<uint32_t>(id) < a.vocab ? (xid - m) - ln : 0.f;
    }
    if (a.top == 0) return;
    place(list, min(count, kRowList), a.top, best);
    if (tid < a.top) {
        const uint64_t k = best[tid];
        a.top_ids[row * a.top + tid] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(k));
        a.top_lp[row * a.top + tid] = (of_order(static_cast<uint32_t>(k >> 32)) - m) - ln;
    }
}

// Values a thread of the first kernel holds: 16 (64 x 248320: 13.4 us, 32
// 13.8, 8 14.9), or 8 where that would leave compute units idle.
int values(uint64_t rows, uint32_t vocab) {
    return rows * ((vocab + 4095) / 4096) >= 512 ? 16 : 8;
}

}  // namespace

uint64_t logprobs_workspace_bytes(uint32_t rows, uint32_t vocab, uint32_t top) {
    const uint64_t per = 256ull * values(rows, vocab);
    const uint64_t pieces = (vocab + per - 1) / per * rows;
    return pieces * sizeof(Piece) + (top != 0 ? pieces * per / kGroup * 8 : 0);
}

hipError_t launch_logprobs(const LogprobArgs& a, void* workspace, hipStream_t s) {
    if (a.vocab <= 8192) {
        if (a.vocab <= 1024) hipLaunchKernelGGL(logprobs_row_kernel<4>, dim3(a.rows), dim3(256), 0, s, a);
        else if (a.vocab <= 2048) hipLaunchKernelGGL(logprobs_row_kernel<8>, dim3(a.rows), dim3(256), 0, s, a);
        else if (a.vocab <= 4096) hipLaunchKernelGGL(logprobs_row_kernel<16>, dim3(a.rows), dim3(256), 0, s, a);
        else hipLaunchKernelGGL(logprobs_row_kernel<32>, dim3(a.rows), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const int e = values(a.rows, a.vocab);
    const uint32_t per = 256u * e;
    const uint32_t pieces = (a.vocab + per - 1) / per;
    const uint64_t total = uint64_t{pieces} * a.rows;
    Piece* stat = static_cast<Piece*>(workspace);
    uint64_t* keys = a.top != 0 ? reinterpret_cast<uint64_t*>(stat + total) : nullptr;
    // (a launch holds fewer than 2^32 threads)
    const dim3 grid(static_cast<uint32_t>(total < (1u << 18) ? total : 1u << 18)), block(256);
    if (e == 16)
        hipLaunchKernelGGL(logits_kernel<16>, grid, block, 0, s, a.logits, a.rows, a.vocab, pieces, stat, keys);
    else
        hipLaunchKernelGGL(logits_kernel<8>, grid, block, 0, s, a.logits, a.rows, a.vocab, pieces, stat, keys);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (e == 16)
        hipLaunchKernelGGL(logprobs_kernel<16>, dim3(a.rows), block, 0, s, a, pieces, stat, keys);
    else
        hipLaunchKernelGGL(logprobs_kernel<8>, dim3(a.rows), block, 0, s, a, pieces, stat, keys);
    return hipGetLastError();
}

}  // namespace qmv
