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

// The double-precision parts of a row's weights.
__device__ __forceinline__ Weigher weigher_of(float max, float t) {
    const double c = 1.4426950408889634 / static_cast<double>(t);
    Weigher g;
    g.max = max;
    g.c = static_cast<float>(fmin(c, 3e38));
    g.c_low = c > 3e38 ? 0.f : static_cast<float>(c - static_cast<double>(g.c));
    return g;
}
// log2(min_p) in two parts, and whether a token of log2 weight t passes.
struct Floor {
    bool on;
    float hi, lo;
    __device__ __forceinline__ bool passes(float2 t) const { return !on || (t.x - hi) + (t.y - lo) >= 0.f; }
};
__device__ __forceinline__ Floor floor_of(float m) {
    if (!(m > 0.f)) return Floor{false, 0.f, 0.f};
    const double l = log2(static_cast<double>(m));
    const float hi = static_cast<float>(l);
    return Floor{true, hi, static_cast<float>(l - static_cast<double>(hi))};
}
// A token's place in a running sum to `total`: the sum's whole part below u of it.
__device__ __forceinline__ uint64_t aim(float u, uint64_t total) {
    return min(static_cast<uint64_t>(floor(static_cast<double>(u) * static_cast<double>(total))), total - 1);
}
__device__ __forceinline__ void answer(const SampleArgs& a, uint64_t row, uint32_t index, float x, float max, float t, double total) {
    a.ids[row] = static_cast<int32_t>(index);
    if (a.lp != nullptr)
        a.lp[row] = t == 0.f ? 0.f : static_cast<float>((static_cast<double>(x) - static_cast<double>(max)) / static_cast<double>(t) - log(total * 0x1p-39));
}
__device__ __forceinline__ void no_answer(const SampleArgs& a, uint64_t row) {
    a.ids[row] = -1;
    if (a.lp != nullptr) a.lp[row] = __builtin_nanf("");
}

// A whole row by one workgroup, whatever its values and wishes: the maximum m
// and T > 0 are numbers.
__device__ __noinline__ void draw_from_row(const SampleArgs& a, uint64_t row, const Wish& w, float m, Shared& s) {
    const int tid = threadIdx.x;
    const RowSource src{a.logits + row * a.vocab, a.vocab};
    const Weigher g = weigher_of(m, w.t);
    uint64_t total;
    // threshold: keys above `key` stay, and of those equal to it the ones up to index `last`
    uint32_t key = 0, last = 0xFFFFFFFFu;
    auto keep_equal = [&](uint32_t at_key, uint64_t count) {   // the first `count` of a key
        key = at_key;
        last = 0xFFFFFFFFu;
        uint64_t there;
        const uint32_t i = locate(s, src.n, [&](uint32_t j) { return static_cast<uint64_t>(key_of(src.value(j)) == at_key); },
                                  [&](uint64_t all) { return min(all, count) - 1; }, &there);
        if (there > count) last = i;
    };
    auto stays = [&](uint32_t k, uint32_t i) { return k > key || (k == key && i <= last); };
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
    const Floor f = floor_of(w.m);
    const uint32_t at = locate(s, src.n, [&](uint32_t i) {
        const float x = src.value(i);
        return stays(key_of(x), i) && (x == m || f.passes(g.log2_of(x))) ? g(x) : uint64_t{0};
    }, [&](uint64_t all) { return aim(w.u, all); }, &total);
    if (tid == 0) answer(a, row, at, src.value(at), m, w.t, static_cast<double>(total));
    __syncthreads();
}

// ---- rows of up to 2^20: a list of the likely tokens -------------------------

constexpr uint32_t kChunk = 1024;          // tokens of a wave of the scan
constexpr uint32_t kKept = 256;            // likely ones that it can hand on
constexpr uint32_t kList = 8192;           // of a row
constexpr uint32_t kGather = 512;          // of a histogram's bin
constexpr uint32_t kSlots = kList / kThreads;
constexpr uint32_t kSamples = 512;
constexpr uint32_t kOver = 0x80000000u;    // more likely tokens than kKept

// What a wave of the scan says of its tokens: the largest, the sum of their
// weights relative to that, and how many are in its list.
struct Record {
    float max, sum;
    uint32_t count, pad;
};
struct Work {
    Record* records;       // [rows][chunks]
    float2* lists;         // [rows][chunks][kKept]: logit, index
    float* bounds;         // [rows]
    uint32_t chunks;
};

__device__ __forceinline__ bool wants_list(const Wish& w) { return w.t == 0.f || w.k != 0 || w.p < 1.f || w.m > 0.f; }
__device__ __forceinline__ bool wants_sum(const Wish& w) { return w.t > 0.f && w.k == 0 && (w.p < 1.f || !(w.m > 0.f)); }
__device__ __forceinline__ bool drawable(const Wish& w) { return w.t >= 0.f && w.t < __builtin_inff(); }

// A bound above which a row has some thousands of its tokens, from 512 of them
// evenly apart: the r-th largest (its upper 16 bits, rounded down).
__global__ __launch_bounds__(64) void sample_bound_kernel(SampleArgs a, Work k) {
    constexpr int kEach = kSamples / 64;
    const int lane = threadIdx.x;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const Wish w = wish_of(a, row);
        const float* x = a.logits + row * a.vocab;
        uint32_t key[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) key[i] = key_of(x[(static_cast<uint64_t>(64 * i + lane) * a.vocab) / kSamples]) >> 16;
        const uint64_t some = w.t == 0.f ? 1 : (w.k != 0 ? 3ull * w.k + 1000 : 2500);
        const uint32_t least = w.t == 0.f ? 1 : 5;
        const uint32_t r = min(max(static_cast<uint32_t>(some * kSamples / a.vocab), least), kSamples);
        uint32_t bound = 0;
#pragma unroll
        for (int b = 15; b >= 0; --b) {
            const uint32_t at = bound | 1u << b;
            uint32_t n = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) n += static_cast<uint32_t>(__popcll(__ballot(key[i] >= at)));
            if (n >= r) bound = at;
        }
        const uint32_t bits = bound << 16;
        // (rounded down, -infinity is no number: all that is finite is listed then)
        float v = __builtin_bit_cast(float, bits & 0x80000000u ? bits & 0x7FFFFFFFu : ~bits);
        if (!(v > -3.4028235e38f)) v = -3.4028235e38f;
        if (lane == 0) k.bounds[row] = wants_list(w) && drawable(w) ? v : __builtin_inff();
    }
}

// Reads every logit once: a wave has 1024, 16 a lane.
__global__ __launch_bounds__(256) void sample_scan_kernel(SampleArgs a, Work k) {
    struct __attribute__((packed, aligned(4))) Four {
        float v[4];
    };
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t chunk = blockIdx.x * 4 + static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)));
    if (chunk >= k.chunks) return;
    const uint32_t from = chunk * kChunk;
    for (uint64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float* p = a.logits + row * a.vocab + from;
        float x[4][4];
        if (from + kChunk <= a.vocab) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Four f = reinterpret_cast<const Four*>(p)[64 * i + lane];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = f.v[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t at = 256 * i + 4 * lane + j;
                    x[i][j] = from + at < a.vocab ? p[at] : -__builtin_inff();
                }
        }
        const Wish w = wish_of(a, row);
        const float bound = k.bounds[row];
        float m = -__builtin_inff();
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bad |= !(x[i][j] < __builtin_inff());
                m = fmaxf(m, x[i][j]);
            }
#pragma unroll
        for (int b = 1; b < 64; b <<= 1) m = fmaxf(m, __shfl_xor(m, b));
        if (__any(bad)) m = __builtin_inff();
        float sum = 0.f;
        if (wants_sum(w) && m > -__builtin_inff() && m < __builtin_inff()) {
            const Weigher g = weigher_of(m, w.t);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float d = x[i][j] - m;
                    // (-infinity times the low part may be no number)
                    const float t = fmaxf(fmaf(d, g.c, d * g.c_low), d * g.c - 1.f);
                    sum += d == 0.f ? 1.f : __builtin_amdgcn_exp2f(t);
                }
#pragma unroll
            for (int b = 1; b < 64; b <<= 1) sum += __shfl_xor(sum, b);
        }
        // the list, in the order of the indexes
        const uint64_t slot = row * k.chunks + chunk;
        float2* list = k.lists + slot * kKept;
        uint32_t n = 0;
        const uint64_t below = (1ull << lane) - 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t who[4];
            uint32_t mine = 0, all = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                who[j] = __ballot(x[i][j] >= bound);
                mine += static_cast<uint32_t>(__popcll(who[j] & below));
                all += static_cast<uint32_t>(__popcll(who[j]));
            }
            if (all != 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (x[i][j] >= bound) {
                        if (n + mine < kKept) list[n + mine] = make_float2(x[i][j], __builtin_bit_cast(float, from + 256 * i + 4 * lane + j));
                        ++mine;
                    }
                }
                n += all;
            }
        }
        if (lane == 0) k.records[slot] = Record{m, sum, n <= kKept ? n : kOver, 0};
    }
}

// Shared memory of the kernel that picks.
struct Picks {
    union {
        struct {
            float x[kList];
            uint32_t index[kList];
        };
        Shared row;
    };
    uint64_t weight[kThreads];
    uint32_t count[kThreads];
    uint64_t g_weight[kGather];
    uint32_t g_key[kGather], g_at[kGather];
    uint64_t sums[kWaves], sums2[kWaves];
    float maxes[kWaves], mins[kWaves];
    uint32_t flags[kWaves];
    uint32_t bin, gathered, key, at;
    uint64_t before, inside;
};

// Exclusive sums of a and b over the workgroup's threads, and their totals.
__device__ __forceinline__ void scan2(Picks& s, uint64_t a, uint64_t b, uint64_t* a_before, uint64_t* b_before, uint64_t* a_all, uint64_t* b_all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t ua = wave_scan(a), ub = wave_scan(b);
    if (lane == 63) {
        s.sums[wave] = ua;
        s.sums2[wave] = ub;
    }
    __syncthreads();
    uint64_t pa = ua - a, pb = ub - b, ta = 0, tb = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i == wave) {
            pa += ta;
            pb += tb;
        }
        ta += s.sums[i];
        tb += s.sums2[i];
    }
    *a_before = pa;
    *b_before = pb;
    *a_all = ta;
    *b_all = tb;
    __syncthreads();
}

// The tokens of bin `bin` into the gather list; how many they are (past kGather they are not all there).
template <typename X, typename Q, typename B>
__device__ __forceinline__ uint32_t gather(Picks& s, uint32_t bin, uint32_t first, const X& x, const Q& q, const B& bins) {
    if (threadIdx.x == 0) s.gathered = 0;
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < kSlots; ++i) {
        if (bins[i] == bin) {
            const uint32_t at = atomicAdd(&s.gathered, 1u);
            if (at < kGather) {
                s.g_key[at] = key_of(x[i]);
                s.g_at[at] = first + 64 * i;
                s.g_weight[at] = q[i];
            }
        }
    }
    __syncthreads();
    return s.gathered;
}

// DIRECT: rows of at most kList, read here; else the row's list is.
template <bool DIRECT>
__global__ __launch_bounds__(kThreads) void sample_pick_kernel(SampleArgs a, Work k) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    Picks& s = *reinterpret_cast<Picks*>(lds);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const Wish w = wish_of(a, row);
        __syncthreads();
        s.weight[tid] = 0;
        s.count[tid] = 0;
        // the row's largest logit, its number of listed tokens, the sum of its weights
        float x[kSlots], m = -__builtin_inff(), low = __builtin_inff();
        uint32_t n, first, flag = 0;
        Record r{-__builtin_inff(), 0.f, 0, 0};
        const float bound = DIRECT ? -__builtin_inff() : k.bounds[row];
        if constexpr (DIRECT) {
            n = a.vocab;
            first = wave * (((n + kThreads - 1) / kThreads) * 64) + lane;
            const uint32_t end = min((wave + 1) * (((n + kThreads - 1) / kThreads) * 64), n);
#pragma unroll
            for (uint32_t i = 0; i < kSlots; ++i) {
                x[i] = first + 64 * i < end ? a.logits[row * a.vocab + first + 64 * i] : -__builtin_inff();
                if (!(x[i] < __builtin_inff())) flag = kOver;
                m = fmaxf(m, x[i]);
                if (x[i] > -__builtin_inff()) low = fminf(low, x[i]);
            }
            if (flag != 0) m = __builtin_inff();
            flag = 0;
        } else {
            if (static_cast<uint32_t>(tid) < k.chunks) r = k.records[row * k.chunks + tid];
            m = r.max;
            flag = r.count & kOver;
        }
#pragma unroll
        for (int b = 1; b < 64; b <<= 1) {
            m = fmaxf(m, __shfl_xor(m, b));
            if constexpr (DIRECT) low = fminf(low, __shfl_xor(low, b));
        }
        flag = __any(flag != 0) ? 1u : 0u;
        if (lane == 0) {
            s.maxes[wave] = m;
            s.mins[wave] = low;
            s.flags[wave] = flag;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            m = fmaxf(m, s.maxes[i]);
            low = fminf(low, s.mins[i]);
            flag |= s.flags[i];
        }
        if (!(m > -__builtin_inff() && m < __builtin_inff()) || !drawable(w)) {
            if (tid == 0) no_answer(a, row);
            continue;
        }
        const bool greedy = w.t == 0.f;
        const Weigher g = weigher_of(m, greedy ? 1.f : w.t);
        uint64_t all = 0;                        // the weights of the whole row
        if constexpr (!DIRECT) {
            // records' weights as whole numbers, and the places of their lists
            uint64_t mine = 0, before, n_before, n_all;
            if (r.max > -__builtin_inff()) {
                const float2 t = g.log2_of(r.max);
                if (t.x > -60.f) mine = static_cast<uint64_t>(static_cast<double>(r.sum) * exp2(static_cast<double>(t.x) + static_cast<double>(t.y)) * 0x1p39);
            }
            scan2(s, mine, r.count & ~kOver, &before, &n_before, &all, &n_all);
            if (!wants_list(w)) {
                // drawn from all: the record, then its tokens one a thread
                const uint64_t target = aim(w.u, max(all, uint64_t{1}));
                if (mine != 0 && before <= target && target - before < mine) {
                    s.bin = tid;
                    s.before = target - before;
                }
                __syncthreads();
                const uint32_t at = s.bin * kChunk + tid;
                const float v = at < a.vocab ? a.logits[row * a.vocab + at] : -__builtin_inff();
                const uint64_t q = g(v);
                uint64_t q_before, unused, q_all, unused_all;
                const uint64_t want = s.before;
                scan2(s, q, 0, &q_before, &unused, &q_all, &unused_all);
                const uint64_t place = q_all == 0 ? 0 : min(want, q_all - 1);
                if (q_all == 0 ? tid == 0 : (q_before <= place && place - q_before < q)) answer(a, row, at, v, m, w.t, static_cast<double>(all));
                continue;
            }
            n = static_cast<uint32_t>(min(n_all, static_cast<uint64_t>(kList)));
            flag |= n_all > kList ? 1u : 0u;
            if (flag == 0) {
                // lists into shared memory, 16 lanes a list
                if (static_cast<uint32_t>(tid) < k.chunks) {
                    s.weight[tid] = n_before << 32 | r.count;   // (the histogram's memory, cleared again below)
                }
                __syncthreads();
                const uint32_t part = tid & 15;
                for (uint32_t c = tid >> 4; c < k.chunks; c += kThreads / 16) {
                    const uint32_t to = static_cast<uint32_t>(s.weight[c] >> 32), count = static_cast<uint32_t>(s.weight[c]);
                    const float2* list = k.lists + (row * k.chunks + c) * kKept;
                    for (uint32_t j = part; j < count; j += 16) {
                        const float2 v = list[j];
                        s.x[to + j] = v.x;
                        s.index[to + j] = __builtin_bit_cast(uint32_t, v.y);
                    }
                }
                __syncthreads();
                s.weight[tid] = 0;
            }
            const uint32_t each = ((n + kThreads - 1) / kThreads) * 64;
            first = wave * each + lane;
            const uint32_t end = min((wave + 1) * each, n);
#pragma unroll
            for (uint32_t i = 0; i < kSlots; ++i) x[i] = flag == 0 && first + 64 * i < end ? s.x[first + 64 * i] : -__builtin_inff();
        }
        const auto index_of = [&](uint32_t at) { return DIRECT ? at : s.index[at]; };
        // tokens below `low` weigh nothing, or are in no list
        const float nothing = m - 29.2f * w.t;
        const bool complete = DIRECT || bound <= nothing;
        low = greedy ? m : fmaxf(DIRECT ? low : bound, nothing);
        const float per = m > low ? (kThreads - 0.01f) / (m - low) : 0.f;
        uint64_t q[kSlots];
        uint32_t bins[kSlots];
        __syncthreads();
#pragma unroll
        for (uint32_t i = 0; i < kSlots; ++i) {
            const bool in = x[i] >= low;
            q[i] = in ? g(x[i]) : 0;
            bins[i] = in ? static_cast<uint32_t>(fminf((m - x[i]) * per, kThreads - 1.f)) : 0xFFFFFFFFu;
            if (in) {
                atomicAdd(&s.count[bins[i]], 1u);
                if (!greedy && q[i] != 0) atomicAdd(reinterpret_cast<unsigned long long*>(&s.weight[bins[i]]), static_cast<unsigned long long>(q[i]));
            }
        }
        __syncthreads();
        uint64_t c_before, w_before, c_all, w_all;
        scan2(s, s.count[tid], s.weight[tid], &c_before, &w_before, &c_all, &w_all);
        // (w.k etc. are the row's, so the workgroup goes one way)
        bool cut = false, lost = flag != 0;
        uint32_t key = 0, last = 0xFFFFFFFFu;
        uint64_t among = complete ? w_all : all;
        const uint32_t want_k = greedy ? 1u : w.k;
        if (!lost && want_k != 0) {
            if (c_all >= want_k) {
                if (c_before < want_k && c_before + s.count[tid] >= want_k) {
                    s.bin = tid;
                    s.before = w_before;
                    s.at = want_k - static_cast<uint32_t>(c_before);
                }
                if (tid == 0) s.inside = 0;
                __syncthreads();
                const uint32_t need = s.at, got = gather(s, s.bin, first, x, q, bins);
                if (got > kGather) {
                    lost = true;
                } else {
                    if (static_cast<uint32_t>(tid) < got) {
                        const uint32_t ka = s.g_key[tid], pa = s.g_at[tid];
                        uint32_t rank = 0;
                        for (uint32_t j = 0; j < got; ++j) rank += s.g_key[j] > ka || (s.g_key[j] == ka && s.g_at[j] < pa) ? 1u : 0u;
                        if (rank < need) atomicAdd(reinterpret_cast<unsigned long long*>(&s.inside), static_cast<unsigned long long>(s.g_weight[tid]));
                        if (rank == need - 1) {
                            s.key = ka;
                            s.at = pa;
                        }
                    }
                    __syncthreads();
                    key = s.key;
                    last = s.at;
                    among = s.before + s.inside;
                    cut = true;
                }
            } else if (complete) {
                cut = true;                      // all that weigh anything stay
            } else {
                lost = true;
            }
        }
        __syncthreads();
        if (!lost && !greedy && w.p < 1.f && (w.k != 0 || complete || all != 0)) {
            const double want = ceil(static_cast<double>(w.p) * static_cast<double>(among));
            const uint64_t target = want < 1.0 ? 0 : min(static_cast<uint64_t>(want), among) - 1;
            if (target < w_all) {
                const uint64_t mine = s.weight[tid];
                if (mine != 0 && w_before <= target && target - w_before < mine) {
                    s.bin = tid;
                    s.before = w_before;
                }
                __syncthreads();
                const uint32_t got = gather(s, s.bin, first, x, q, bins);
                if (got > kGather) {
                    lost = true;
                } else {
                    if (static_cast<uint32_t>(tid) < got) {
                        const uint32_t ka = s.g_key[tid], pa = s.g_at[tid];
                        uint64_t sum = s.before;
                        for (uint32_t j = 0; j < got; ++j) sum += s.g_key[j] > ka || (s.g_key[j] == ka && s.g_at[j] < pa) ? s.g_weight[j] : uint64_t{0};
                        if (sum <= target && target - sum < s.g_weight[tid]) {
                            s.key = ka;
                            s.at = pa;
                        }
                    }
                    __syncthreads();
                    key = s.key;
                    last = s.at;
                    cut = true;
                }
            } else if (!cut) {
                lost = true;
            }
        }
        const Floor f = floor_of(greedy ? 0.f : w.m);
        // (without another cut, a list that ends above what min_p lets pass is none)
        if (!cut && !complete && !(f.on && !f.passes(g.log2_of(bound)))) lost = true;
        if (lost) {
            __syncthreads();
            if (greedy) {
                uint64_t total;
                const float* p = a.logits + row * a.vocab;
                const uint32_t at = locate(s.row, a.vocab, [&](uint32_t i) { return static_cast<uint64_t>(p[i] == m); }, [](uint64_t) { return uint64_t{0}; }, &total);
                if (tid == 0) answer(a, row, at, m, m, 0.f, 1.0);
                __syncthreads();
            } else {
                draw_from_row(a, row, w, m, s.row);
            }
            continue;
        }
        // the draw: a wave's tokens are consecutive, 64 a step
        uint64_t sum = 0;
#pragma unroll
        for (uint32_t i = 0; i < kSlots; ++i) {
            const uint32_t ka = key_of(x[i]);
            const bool stays = bins[i] != 0xFFFFFFFFu && (ka > key || (ka == key && first + 64 * i <= last)) && (x[i] == m || f.passes(g.log2_of(x[i])));
            q[i] = stays ? (greedy ? uint64_t{1} : q[i]) : uint64_t{0};
            sum += q[i];
        }
        sum = wave_sum(sum);
        __syncthreads();
        if (lane == 0) s.sums[wave] = sum;
        __syncthreads();
        uint64_t total = 0, before = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            before += i < wave ? s.sums[i] : 0;
            total += s.sums[i];
        }
        const uint64_t target = aim(greedy ? 0.f : w.u, total);
        if (before <= target && target - before < sum) {      // (one wave)
#pragma unroll
            for (uint32_t i = 0; i < kSlots; ++i) {
                const uint64_t upto = wave_scan(q[i]) + before;
                if (upto > target && upto - q[i] <= target) answer(a, row, index_of(first + 64 * i), x[i], m, w.t, static_cast<double>(total));
                before = shfl_u64(upto, 63);
            }
        }
    }
}

// Rows past 2^20: a workgroup a row.
__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleArgs a) {
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float* p = a.logits + row * a.vocab;
        const Wish w = wish_of(a, row);
        float m = -__builtin_inff();
        bool bad = false;
#pragma unroll 4
        for (uint32_t i = tid; i < a.vocab; i += kThreads) {
            const float x = p[i];
            bad |= !(x < __builtin_inff());
            m = fmaxf(m, x);
        }
#pragma unroll
        for (int b = 1; b < 64; b <<= 1) m = fmaxf(m, __shfl_xor(m, b));
        if (__any(bad)) m = __builtin_inff();
        if (lane == 0) s.maxes[wave] = m;
        __syncthreads();
        for (int i = 0; i < kWaves; ++i) m = fmaxf(m, s.maxes[i]);
        __syncthreads();
        if (!(m > -__builtin_inff() && m < __builtin_inff()) || !drawable(w)) {
            if (tid == 0) no_answer(a, row);
        } else if (w.t == 0.f) {
            uint64_t total;
            const uint32_t at = locate(s, a.vocab, [&](uint32_t i) { return static_cast<uint64_t>(p[i] == m); }, [](uint64_t) { return uint64_t{0}; }, &total);
            if (tid == 0) answer(a, row, at, m, m, 0.f, 1.0);
            __syncthreads();
        } else {
            draw_from_row(a, row, w, m, s);
        }
    }
}

uint32_t chunks_of(uint32_t vocab) { return (vocab + kChunk - 1) / kChunk; }
bool listed(uint32_t vocab) { return vocab > kList && vocab <= kThreads * kChunk; }

template <bool DIRECT>
hipError_t pick(const SampleArgs& a, const Work& k, uint32_t grid, hipStream_t s) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(sample_pick_kernel<DIRECT>), hipFuncAttributeMaxDynamicSharedMemorySize, sizeof(Picks));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((sample_pick_kernel<DIRECT>), dim3(grid), dim3(kThreads), sizeof(Picks), s, a, k);
    return hipGetLastError();
}

}  // namespace

uint64_t sample_workspace_bytes(uint32_t rows, uint32_t vocab) {
    if (!listed(vocab)) return 16;
    const uint64_t slots = uint64_t{rows} * chunks_of(vocab);
    return slots * (sizeof(Record) + kKept * sizeof(float2)) + (uint64_t{rows} * 4 + 15) / 16 * 16;
}

hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t stream) {
    const uint32_t grid = a.rows < (1u << 20) ? a.rows : (1u << 20);
    Work k{};
    if (a.vocab <= kList) return pick<true>(a, k, grid, stream);
    if (!listed(a.vocab)) {
        hipLaunchKernelGGL(sample_row_kernel, dim3(grid), dim3(kThreads), 0, stream, a);
        return hipGetLastError();
    }
    k.chunks = chunks_of(a.vocab);
    const uint64_t slots = uint64_t{a.rows} * k.chunks;
    k.records = static_cast<Record*>(workspace);
    k.lists = reinterpret_cast<float2*>(k.records + slots);
    k.bounds = reinterpret_cast<float*>(k.lists + slots * kKept);
    hipLaunchKernelGGL(sample_bound_kernel, dim3(grid), dim3(64), 0, stream, a, k);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sample_scan_kernel, dim3((k.chunks + 3) / 4, a.rows < 65535 ? a.rows : 65535), dim3(256), 0, stream, a, k);
    e = hipGetLastError();
    return e != hipSuccess ? e : pick<false>(a, k, grid, stream);
}

}  // namespace qmv
