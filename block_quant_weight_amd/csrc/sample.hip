// The next token, drawn from an LM head's logits with a given random number.
//
// For a row of logits x with its maximum M and temperature T a token's weight
// is w = e^{(x - M) / T}, held as a whole number of 2^-39: sums of whole
// numbers do not depend on their order, and a running sum meets a border the
// same way whoever adds it up.  The exponent is formed in two float32 parts,
// so that a weight is right to about one rounding also far below the largest.
//
// The tokens that stay are a prefix in the order of the logits, so they are
// given by a threshold: the key (a logit's bits in the order of its value) of
// the last of them, and where several share it the index of the last.  top-k
// counts to it, top-p sums to it, each by three histograms over 11, 11 and 10
// bits of the key; the draw is a running sum over the indexes, found by sums
// of sixteenths, of a sixteenth's sixteenths, and one by one.
#include "device_common.h"
#include "serve_kernels.h"

namespace qmv {
namespace {

#pragma clang fp contract(off)

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr float kUnit = 0x1p39f;            // the largest weight as a whole number

// Bits in the order of the value; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint64_t shfl_u64(uint64_t v, int from) {
    const uint32_t lo = static_cast<uint32_t>(__shfl(static_cast<int>(static_cast<uint32_t>(v)), from));
    const uint32_t hi = static_cast<uint32_t>(__shfl(static_cast<int>(static_cast<uint32_t>(v >> 32)), from));
    return static_cast<uint64_t>(hi) << 32 | lo;
}
// Sum over a wave, in every lane; and over the lanes up to this one.
__device__ __forceinline__ uint64_t wave_sum(uint64_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += shfl_u64(v, lane ^ m);
    return v;
}
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint64_t u = shfl_u64(v, lane >= m ? lane - m : lane);
        if (lane >= m) v += u;
    }
    return v;
}

// How a row's weights are formed.
struct Weigher {
    float max, c, c_low;     // c + c_low = log2(e) / T

    // log2 of a weight in two parts.
    __device__ __forceinline__ float2 log2_of(float x) const {
        const float d = x - max;
        if (d == 0.f) return make_float2(0.f, 0.f);
        // x - max = d + e exactly
        const float z = d - x, e = (x - (d - z)) - (max + z);
        const float hi = d * c;
        return make_float2(hi, fmaf(e, c, fmaf(d, c_low, fmaf(d, c, -hi))));
    }
    __device__ __forceinline__ uint64_t operator()(float x) const {
        const float2 t = log2_of(x);
        if (!(t.x > -42.f)) return 0;        // (below half a unit; also where the low part is no number)
        const float w = __builtin_amdgcn_exp2f(t.x);
        const float v = fminf(fmaf(w, t.y * 0.6931471805599453f, w), 1.f) * 0x1p15f;
        const float whole = truncf(v);
        return (static_cast<uint64_t>(static_cast<uint32_t>(whole)) << 24) + static_cast<uint32_t>(rintf((v - whole) * 0x1p24f));
    }
};

// What is asked of a row.
struct Wish {
    float t;
    uint32_t k;              // 0: all
    float p;                 // 1: all
    float m;                 // 0: all
    float u;
};
__device__ __forceinline__ Wish wish_of(const SampleArgs& a, uint64_t row) {
    Wish w;
    w.t = a.temperature != nullptr ? a.temperature[row] : 1.f;
    const int32_t k = a.top_k != nullptr ? a.top_k[row] : 0;
    w.k = k > 0 && static_cast<uint32_t>(k) < a.vocab ? static_cast<uint32_t>(k) : 0u;
    const float p = a.top_p != nullptr ? a.top_p[row] : 1.f;
    w.p = p < 1.f ? fmaxf(p, 0.f) : 1.f;
    const float m = a.min_p != nullptr ? a.min_p[row] : 0.f;
    w.m = m > 0.f ? fminf(m, 1.f) : 0.f;
    const float u = a.u[row];
    w.u = u > 0.f ? fminf(u, 1.f) : 0.f;
    return w;
}

// A workgroup's shared memory.
struct Shared {
    uint64_t weight[kBins];
    uint32_t count[kBins];
    uint64_t sums[kWaves];
    uint32_t bins[2];
    float maxes[kWaves];
    uint32_t found;
    uint64_t left;
};

// Of `bins` bins with sums f(0), f(1), .. (from the best on) the first at
// which the running sum exceeds `target`, and what is before it.
template <typename F>
__device__ __forceinline__ void first_bin(Shared& s, F f, uint64_t target, uint32_t* bin, uint64_t* before) {
    constexpr int kEach = kBins / kThreads;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint64_t v[kEach], own = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        v[i] = f(kEach * tid + i);
        own += v[i];
    }
    const uint64_t upto = wave_scan(own);
    if (lane == 63) s.sums[wave] = upto;
    if (tid == 0) s.found = kBins - 1;
    __syncthreads();
    uint64_t at = upto - own;
    for (int i = 0; i < wave; ++i) at += s.sums[i];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (at <= target && at + v[i] > target) {
            s.found = kEach * tid + i;
            s.left = at;
        }
        at += v[i];
    }
    __syncthreads();
    *bin = s.found;
    *before = s.left;
    __syncthreads();
}

// The first place i in [0, n) at which the running sum of f(i) exceeds
// pick(sum of all); all sums below 2^64.  n > 0.
template <typename F, typename P>
__device__ __forceinline__ uint32_t locate(Shared& s, uint32_t n, F f, P pick, uint64_t* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t from = 0, size = n;
    uint64_t target = 0;
    bool first = true;
    while (first || size > 64) {
        const uint32_t each = ((size + kWaves - 1) / kWaves + 63) & ~63u;   // a wave's places
        const uint32_t b = min(wave * each, size), e = min(b + each, size);
        uint64_t v = 0;
#pragma unroll 4
        for (uint32_t i = b + lane; i < e; i += 64) v += f(from + i);
        v = wave_sum(v);
        if (lane == 0) s.sums[wave] = v;
        __syncthreads();
        if (first) {
            uint64_t all = 0;
            for (int i = 0; i < kWaves; ++i) all += s.sums[i];
            *total = all;
            target = pick(all);
            first = false;
        }
        int w = 0;
        uint64_t at = 0;
        while (w < kWaves - 1 && at + s.sums[w] <= target) at += s.sums[w++];
        target -= at;
        const uint32_t begin = min(w * each, size);
        from += begin;
        size = min(each, size - begin);
        __syncthreads();
    }
    // (every wave finds the same)
    const uint64_t v = wave_scan(static_cast<uint32_t>(lane) < size ? f(from + lane) : 0);
    const uint64_t past = __ballot(v > target);
    return from + (past != 0 ? static_cast<uint32_t>(__builtin_ctzll(past)) : size - 1);
}

// The tokens of a row as they lie in memory.
struct RowSource {
    const float* x;
    uint32_t n;
    __device__ __forceinline__ float value(uint32_t i) const { return x[i]; }
    __device__ __forceinline__ uint32_t index(uint32_t i) const { return i; }
};

// The threshold at which the running sum, in the order of the keys, of what
// `mass` says exceeds `target`: the key, the number of its tokens that come
// before that, and the mass before the key.
struct Cut {
    uint32_t key;
    uint64_t before;         // mass of larger keys
};
template <typename S, typename M>
__device__ __forceinline__ Cut cut_at(Shared& s, const S& src, M mass, uint64_t target) {
    uint32_t fixed = 0, mask = 0;
    uint64_t before = 0;
#pragma unroll
    for (int step = 0; step < 3; ++step) {
        const int shift = step == 0 ? 21 : (step == 1 ? 10 : 0), bits = step == 2 ? 10 : 11;
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.weight[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (uint32_t i = threadIdx.x; i < src.n; i += kThreads) {
            const float x = src.value(i);
            const uint32_t key = key_of(x);
            if ((key & mask) == fixed) {
                const uint64_t v = mass(x, key);
                if (v != 0) atomicAdd(reinterpret_cast<unsigned long long*>(&s.weight[key >> shift & ((1u << bits) - 1)]), static_cast<unsigned long long>(v));
            }
        }
        __syncthreads();
        uint32_t bin;
        uint64_t at;
        first_bin(s, [&](int i) { return s.weight[kBins - 1 - i]; }, target - before, &bin, &at);
        before += at;
        fixed |= (kBins - 1 - bin) << shift;
        mask |= ((1u << bits) - 1) << shift;
    }
    return Cut{fixed, before};
}

__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleArgs a) {
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const RowSource src{a.logits + row * a.vocab, a.vocab};
        const Wish w = wish_of(a, row);
        // the maximum, and whether the row can be drawn from
        float m = -__builtin_inff();
        bool bad = false;
#pragma unroll 4
        for (uint32_t i = tid; i < src.n; i += kThreads) {
            const float x = src.value(i);
            bad |= !(x < __builtin_inff());
            m = fmaxf(m, x);
        }
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k));
        if (__any(bad)) m = __builtin_inff();
        if (lane == 0) s.maxes[wave] = m;
        __syncthreads();
        m = s.maxes[0];
        for (int i = 1; i < kWaves; ++i) m = fmaxf(m, s.maxes[i]);
        __syncthreads();
        if (!(m > -__builtin_inff() && m < __builtin_inff()) || !(w.t >= 0.f && w.t < __builtin_inff())) {
            if (tid == 0) {
                a.ids[row] = -1;
                if (a.lp != nullptr) a.lp[row] = __builtin_nanf("");
            }
            continue;
        }
        uint64_t total;
        if (w.t == 0.f) {
            const uint32_t at = locate(s, src.n, [&](uint32_t i) { return static_cast<uint64_t>(src.value(i) == m); },
                                       [](uint64_t) { return uint64_t{0}; }, &total);
            if (tid == 0) {
                a.ids[row] = static_cast<int32_t>(at);
                if (a.lp != nullptr) a.lp[row] = 0.f;
            }
            continue;
        }
        const double c = 1.4426950408889634 / static_cast<double>(w.t);
        Weigher g;
        g.max = m;
        g.c = static_cast<float>(fmin(c, 3e38));
        g.c_low = static_cast<float>(c - static_cast<double>(g.c));
        if (c > 3e38) g.c_low = 0.f;

        // threshold: keys above `key` stay, and of those equal to it the ones up to index `last`
        uint32_t key = 0, last = 0xFFFFFFFFu;
        auto keep_equal = [&](uint32_t at_key, uint64_t count) {   // the first `count` of a key
            key = at_key;
            last = 0xFFFFFFFFu;
            uint64_t there;
            const uint32_t i = locate(s, src.n, [&](uint32_t j) { return static_cast<uint64_t>(key_of(src.value(j)) == at_key); },
                                      [&](uint64_t all) { return min(all, count) - 1; }, &there);
            if (there > count) last = src.index(i);
        };
        auto stays = [&](uint32_t k, uint32_t i) { return k > key || (k == key && src.index(i) <= last); };
        if (w.k != 0) {
            const Cut cut = cut_at(s, src, [](float, uint32_t) { return uint64_t{1}; }, w.k - 1);
            keep_equal(cut.key, w.k - cut.before);
        }
        if (w.p < 1.f) {
            // a token stays if the weight before it is below p times the total: up to the first at
            // which the running sum reaches it
            locate(s, src.n, [&](uint32_t i) {
                const float x = src.value(i);
                return stays(key_of(x), i) ? g(x) : uint64_t{0};
            }, [](uint64_t) { return uint64_t{0}; }, &total);
            const double want = ceil(static_cast<double>(w.p) * static_cast<double>(total));
            const uint64_t target = want < 1.0 ? 0 : min(static_cast<uint64_t>(want), total) - 1;
            const uint32_t old_key = key;
            const Cut cut = cut_at(s, src, [&](float x, uint32_t k) { return k >= old_key ? g(x) : uint64_t{0}; }, target);
            // of the key's tokens, all of one weight, as many as reach the target
            const uint32_t bits = cut.key & 0x80000000u ? cut.key & 0x7FFFFFFFu : ~cut.key;
            const uint64_t one = max(g(__builtin_bit_cast(float, bits)), uint64_t{1});
            const uint64_t count = (target - cut.before) / one + 1;
            if (cut.key > key) {
                keep_equal(cut.key, count);
            } else if (cut.key == key) {
                const uint32_t before_last = last;
                keep_equal(cut.key, count);
                last = min(last, before_last);
            }
        }
        const float floor_hi = w.m > 0.f ? static_cast<float>(log2(static_cast<double>(w.m))) : 0.f;
        const float floor_lo = w.m > 0.f ? static_cast<float>(log2(static_cast<double>(w.m)) - static_cast<double>(floor_hi)) : 0.f;
        const uint32_t at = locate(s, src.n, [&](uint32_t i) {
            const float x = src.value(i);
            if (!stays(key_of(x), i)) return uint64_t{0};
            if (w.m > 0.f && x != m) {
                const float2 t = g.log2_of(x);
                if (!((t.x - floor_hi) + (t.y - floor_lo) >= 0.f)) return uint64_t{0};
            }
            return g(x);
        }, [&](uint64_t all) {
            const double want = floor(static_cast<double>(w.u) * static_cast<double>(all));
            return min(static_cast<uint64_t>(want), all - 1);
        }, &total);
        if (tid == 0) {
            a.ids[row] = static_cast<int32_t>(src.index(at));
            if (a.lp != nullptr)
                a.lp[row] = static_cast<float>((static_cast<double>(src.value(at)) - static_cast<double>(m)) / static_cast<double>(w.t) -
                                               log(static_cast<double>(total) * 0x1p-39));
        }
    }
}

}  // namespace

uint64_t sample_workspace_bytes(uint32_t, uint32_t) { return 16; }

hipError_t launch_sample(const SampleArgs& a, void*, hipStream_t stream) {
    const uint32_t grid = a.rows < (1u << 20) ? a.rows : (1u << 20);
    hipLaunchKernelGGL(sample_row_kernel, dim3(grid), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace qmv
