// The next token, drawn from an LM head's logits with a given random number.
//
// For a row of logits x with its maximum M and temperature T a token's weight
// is w = e^{(x - M) / T}, held as a whole number of 2^-39: sums of whole
// numbers do not depend on their order, and a running sum meets a border the
// same way whoever adds it up.  The exponent is formed in two float32 parts,
// so that a weight is right to about one rounding also far below the largest.
//
// The tokens that stay are a prefix in the order of the logits, and nearly
// always a short one.  Three kernels (of few rows the first is part of the second):
//   bound  reads 2048 logits of a row and sets a bound above which some hundreds
//          or thousands of its tokens lie;
//   scan   reads every logit once: a wave has 1024, of which it hands on the
//          largest, the sum of the weights relative to that (float32; each wave's
//          sum is then a whole number), and the list of those above the bound;
//   pick   a workgroup a row: the lists into shared memory, their weights, a
//          histogram by value of counts and weights, in which top-k, top-p and
//          the draw each find their bin by one scan and their place in it by
//          comparing its tokens with each other.
// Rows of up to 8192 are picked from directly.  Where the list cannot show what
// stays (a nucleus that goes below the bound, more listed tokens than there is
// room for, a bin too full), one workgroup goes over the whole row: a threshold
// is the key (a logit's bits in the order of its value) of the last token that
// stays, and where several share it the index of the last; top-k counts to it,
// top-p sums to it, each by three histograms over 11, 11 and 10 bits of the key,
// and the draw is a running sum over the indexes.
//
// One row of 248320 takes 15.4 us (6 in a scan that finds the bound itself, 9 in the
// last kernel: launches and trips to memory, and the fetching of its instructions),
// 64 rows (64 MB)
// 34.6 to 35.4 (scan 14 to 16, 4.5 TB/s; the last 14, a workgroup a row on 64 of
// 256 compute units).  A row over the whole of which one workgroup goes 0.42 ms
// for top-k, 0.70 for top-p (64 rows 0.8 and 1.2).
#include "device_common.h"
#include "serve_kernels.h"

namespace qmv {
namespace {

#pragma clang fp contract(off)

// An address in shared memory, as a function that is called takes it: through a
// plain pointer its reads and writes would not be known to go there.
typedef __attribute__((address_space(3))) uint8_t* Lds;

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr float kUnit = 0x1p39f;            // the largest weight as a whole number

// Bits in the order of the value; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A value from the lanes that CTRL names, 0 where there is none (or in rows of
// 16 lanes that ROWS leaves out).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
    const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(static_cast<uint32_t>(v)), CTRL, ROWS, 0xF, true);
    const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(static_cast<uint32_t>(v >> 32)), CTRL, ROWS, 0xF, true);
    return static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 | static_cast<uint32_t>(lo);
}
__device__ __forceinline__ uint64_t read_lane_u64(uint64_t v, int lane) {
    return static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(v >> 32)), lane))) << 32 |
           static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(v)), lane));
}
// Sums over the lanes of a row of 16 up to this one.
__device__ __forceinline__ uint64_t row_scan(uint64_t v) {
    v += dpp_u64<0x111, 0xF>(v);   // lanes 1, 2, 4, 8 before
    v += dpp_u64<0x112, 0xF>(v);
    v += dpp_u64<0x114, 0xF>(v);
    return v + dpp_u64<0x118, 0xF>(v);
}
// Sums over the lanes of a wave up to this one; over all.
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
    v = row_scan(v);
    v += dpp_u64<0x142, 0xA>(v);   // a row's last lane to the next row
    return v + dpp_u64<0x143, 0xC>(v);   // the first half's last lane to the second half
}
__device__ __forceinline__ uint64_t wave_sum(uint64_t v) { return read_lane_u64(wave_scan(v), 63); }
// Largest over a row of 16 lanes, in each.
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, dpp_mov<0xB1>(v));    // lanes 1 apart
    v = fmaxf(v, dpp_mov<0x4E>(v));    // 2 apart
    v = fmaxf(v, dpp_mov<0x141>(v));   // half rows mirrored
    return fmaxf(v, dpp_mov<0x140>(v));
}
__device__ __forceinline__ float wave_max(float v) {
    v = row_max(v);
    return fmaxf(fmaxf(read_lane(v, 0), read_lane(v, 16)), fmaxf(read_lane(v, 32), read_lane(v, 48)));
}
__device__ __forceinline__ int this_wave() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)); }

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
    __device__ __forceinline__ uint64_t operator()(float x) const { return weight_of(log2_of(x)); }
    __device__ __forceinline__ uint64_t weight_of(float2 t) const {
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
    const int lane = threadIdx.x & 63, wave = this_wave();
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
// ln of the token's weight over the total, a number of 2^-39 of the largest;
// what the total has above the largest is exact.  (ln 2 in two parts: float32's
// is above it.)
__device__ __forceinline__ void answer(const SampleArgs& a, uint64_t row, uint32_t index, float x, const Weigher& g, bool greedy, uint64_t total) {
    a.ids[row] = static_cast<int32_t>(index);
    if (a.lp == nullptr) return;
    const float2 t = g.log2_of(x);
    // (up to 2^24 times the unit: past what a signed number holds)
    constexpr uint64_t one = static_cast<uint64_t>(kUnit);
    const float above = static_cast<float>(total > one ? total - one : 0) * (1.f / kUnit);
    a.lp[row] = greedy ? 0.f : fmaf(t.x, 0.6931471805599453f, fmaf(t.x, -1.9046542e-9f, t.y * 0.6931471805599453f)) - log1pf(above);
}
__device__ __forceinline__ void no_answer(const SampleArgs& a, uint64_t row) {
    a.ids[row] = -1;
    if (a.lp != nullptr) a.lp[row] = __builtin_nanf("");
}

// A whole row by one workgroup, whatever its values and wishes: the maximum m
// and T > 0 are numbers.
__device__ __noinline__ void draw_from_row(SampleArgs a, uint64_t row, Wish w, float m, Lds at_s) {
    Shared& s = *(Shared*)at_s;
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
    if (tid == 0) answer(a, row, at, src.value(at), g, false, total);
    __syncthreads();
}

// The first of the largest logits of a row, by one workgroup.
__device__ __noinline__ void take_first(SampleArgs a, uint64_t row, float m, Lds at_s) {
    Shared& s = *(Shared*)at_s;
    const float* p = a.logits + row * a.vocab;
    uint64_t total;
    const uint32_t at = locate(s, a.vocab, [&](uint32_t i) { return static_cast<uint64_t>(p[i] == m); }, [](uint64_t) { return uint64_t{0}; }, &total);
    if (threadIdx.x == 0) answer(a, row, at, m, Weigher{m, 1.f, 0.f}, true, 0);
    __syncthreads();
}

// ---- rows of up to 2^19: a list of the likely tokens -------------------------

constexpr uint32_t kChunk = 1024;          // tokens of a wave of the scan
constexpr uint32_t kKept = 256;            // likely ones that it can hand on
// Tokens of a row that shared memory holds beside their weights; rows up to it
// need no list (us, direct / by a list: 1 row of 8000 21 / 23, 64 22 / 46, 512 40 /
// 81).  With room for 2048 alone, several workgroups share a compute unit (512 rows
// of 2000: 14 us, else 21).
constexpr uint32_t kList = 8192;
constexpr uint32_t kShort = 2048;
constexpr uint32_t kGather = 512;          // of a histogram's bin
constexpr uint32_t kSamples = 2048, kMost = 4;   // read of a row; of kMost the largest counts
constexpr uint32_t kAhead = 256 * 16 / kThreads;
// Rows up to which each workgroup of the scan finds the row's bound itself, which
// saves a launch and costs reads of 32 KB a workgroup (us, itself / a kernel, 248320:
// 1 row 16.0 / 16.9, 8 18.3 / 18.6, 16 21.9 / 21.3, 64 43 / 36).
constexpr uint32_t kOwnRows = 8;
constexpr uint32_t kOver = 0x80000000u;    // more likely tokens than kKept

struct __attribute__((packed, aligned(4))) Four {
    float v[4];
};

// What a wave of the scan says of its tokens: the largest, the sum of their
// weights relative to that, and how many are in its list.
struct Record {
    float max, sum;
    uint32_t count, pad;
};
// What the first kernel finds out of a row: the bound of its list, and the
// numbers that its weights and min_p go by.
struct __attribute__((aligned(16))) Row {
    float bound, c, c_low, floor_hi, floor_lo, pad[3];
};
struct Work {
    Record* records;       // [rows][chunks]
    float2* lists;         // [rows][chunks][kKept]: logit, index
    Row* rows;             // [rows]
    uint32_t chunks;
};

__device__ __forceinline__ bool wants_list(const Wish& w) { return w.t == 0.f || w.k != 0 || w.p < 1.f || w.m > 0.f; }
__device__ __forceinline__ bool wants_sum(const Wish& w) { return w.t > 0.f && w.k == 0 && (w.p < 1.f || !(w.m > 0.f)); }
__device__ __forceinline__ bool drawable(const Wish& w) { return w.t >= 0.f && w.t < __builtin_inff(); }

// A bound above which a row has some hundreds or thousands of its tokens, from
// 2048 of them, 512 times four beside each other: the r-th largest of the fours'
// largest (its upper 16 bits, rounded down).  Of a row of 248320, r = 6 are about 730 tokens:
// at least 40 of them but for 2 rows in a million.
// Four waves read, one finds the bound, another the row's numbers; *to holds
// them after the next barrier.
constexpr uint32_t kKeys = kSamples / kMost;
__device__ __forceinline__ void find_bound(const SampleArgs& a, uint64_t row, uint32_t* keys, Row* to) {
    constexpr int kEach = kKeys / 64;
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const int wave = this_wave();
    const float* x = a.logits + row * a.vocab;
    Four v[kKeys / 256];
#pragma unroll
    for (uint32_t i = 0; i < kKeys / 256; ++i)
        v[i] = *reinterpret_cast<const Four*>(x + (static_cast<uint64_t>(i * 256 + tid) * (a.vocab - 3)) / kKeys);
    const Wish w = wish_of(a, row);
#pragma unroll
    for (uint32_t i = 0; i < kKeys / 256; ++i) {
        uint32_t key = 0;
#pragma unroll
        for (uint32_t j = 0; j < kMost; ++j) key = max(key, key_of(v[i].v[j]) >> 16);
        keys[i * 256 + tid] = key;
    }
    __syncthreads();
    if (wave == 0) {
        uint32_t key[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) key[i] = keys[64 * i + lane];
        // (about as many tokens are listed.  Six times k, as a sample finds them, passes kList now and then from k
        // = 800 or 1000 on, us of one row and of 64: k 500 21 and 41, 800 30 and 47, 1000 33, or as 2000, and 506,
        // 2000 425 and 806)
        const uint64_t some = w.t == 0.f ? 1 : (w.k != 0 ? 6ull * w.k + 500 : 2500);
        const uint32_t least = w.t == 0.f ? 1 : 5;
        // (half of the fours at most: about 160 tokens of a wave's 1024, of which it can hand on 256)
        const uint32_t r = min(max(static_cast<uint32_t>(some * kSamples / a.vocab), least), kKeys / 2);
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
        float low = __builtin_bit_cast(float, bits & 0x80000000u ? bits & 0x7FFFFFFFu : ~bits);
        if (!(low > -3.4028235e38f)) low = -3.4028235e38f;
        if (lane == 0) to->bound = wants_list(w) && drawable(w) ? low : __builtin_inff();
    } else if (wave == 1) {
        const Weigher g = weigher_of(0.f, w.t == 0.f ? 1.f : w.t);
        const Floor f = floor_of(w.m);
        if (lane == 0) {
            to->c = g.c;
            to->c_low = g.c_low;
            to->floor_hi = f.hi;
            to->floor_lo = f.lo;
        }
    }
}
__global__ __launch_bounds__(256) void sample_bound_kernel(SampleArgs a, Work k) {
    __shared__ uint32_t keys[kKeys];
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        find_bound(a, row, keys, k.rows + row);
        __syncthreads();
    }
}

// Reads every logit once: a wave has 1024, 16 a lane.  OWN: each workgroup finds
// the row's bound for itself, while its logits are on their way.
template <bool OWN>
__global__ __launch_bounds__(256) void sample_scan_kernel(SampleArgs a, Work k) {
    __shared__ uint32_t keys[OWN ? kKeys : 1];
    __shared__ Row own;
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t chunk = blockIdx.x * 4 + static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)));
    const bool has = chunk < k.chunks;
    if (!OWN && !has) return;
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
        Row of;
        if constexpr (OWN) {
            find_bound(a, row, keys, &own);
            __syncthreads();
            of = own;
            if (blockIdx.x == 0 && threadIdx.x == 0) k.rows[row] = own;
        } else {
            of = k.rows[row];
        }
        const float bound = of.bound;
        float m = -__builtin_inff();
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bad |= !(x[i][j] < __builtin_inff());
                m = fmaxf(m, x[i][j]);
            }
        m = wave_max(m);
        if (__any(bad)) m = __builtin_inff();
        float sum = 0.f;
        if (wants_sum(w) && m > -__builtin_inff() && m < __builtin_inff()) {
            const Weigher g{m, of.c, of.c_low};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float d = x[i][j] - m;
                    // (-infinity times the low part may be no number)
                    const float t = fmaxf(fmaf(d, g.c, d * g.c_low), d * g.c - 1.f);
                    sum += d == 0.f ? 1.f : __builtin_amdgcn_exp2f(t);
                }
            sum = wave_reduce(sum);
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
        if (has && lane == 0) k.records[slot] = Record{m, sum, n <= kKept ? n : kOver, 0};
        if constexpr (OWN) __syncthreads();      // (keys and own are written again)
    }
}

// Shared memory of the kernel that picks among N tokens.
constexpr uint64_t kBelow = 1ull << 63;   // of a weight: min_p does not let the token pass
template <uint32_t N, bool DIRECT>
struct Picks {
    union {                              // (first: the functions for whole rows take it by the address of all)
        struct {
            uint64_t q[N];
            float x[N];
            uint32_t index[DIRECT ? 1 : N];
        };
        Shared row;
    };
    uint64_t weight[kThreads];
    uint32_t count[kThreads];
    uint64_t g_weight[kGather];
    uint32_t g_key[kGather], g_at[kGather];
    uint64_t sums[4][2][kWaves];     // one for each use
    float maxes[kWaves], mins[kWaves];
    uint32_t flags[kWaves];
    uint32_t bin, gathered, key, at;
    uint64_t before, inside;
};

// (The kernel that picks runs its few thousand instructions once a row, so
// their fetching is what counts: loops are not unrolled, and what is used
// twice is a function.)

// Sums of a and b over the workgroup's threads before this one, and over all.
struct Sums {
    uint64_t a_before, b_before, a_all, b_all;
};
__device__ __noinline__ Sums scan2(Lds at_sums, uint64_t a, uint64_t b) {
    uint64_t(*sums)[kWaves] = (uint64_t(*)[kWaves])at_sums;
    const int lane = threadIdx.x & 63, wave = this_wave();
    const uint64_t ua = wave_scan(a), ub = wave_scan(b);
    if (lane == 63) {
        sums[0][wave] = ua;
        sums[1][wave] = ub;
    }
    __syncthreads();
    const uint64_t sa = row_scan(sums[0][lane % kWaves]), sb = row_scan(sums[1][lane % kWaves]);
    return Sums{ua - a + (wave > 0 ? read_lane_u64(sa, wave - 1) : 0), ub - b + (wave > 0 ? read_lane_u64(sb, wave - 1) : 0),
                read_lane_u64(sa, kWaves - 1), read_lane_u64(sb, kWaves - 1)};
}

// A row's tokens in shared memory, and the bins of their histogram: bin 0 has
// the largest logits; tokens below `low` are in none.
struct Bins {
    float max, low, per;
    __device__ __forceinline__ uint32_t operator()(float x) const {
        return x >= low ? static_cast<uint32_t>(fminf((max - x) * per, kThreads - 1.f)) : 0xFFFFFFFFu;
    }
};

// Of the tokens of a bin (kGather at most, or the answer is false) the first,
// in the order of the logits, at which the running sum of what they weigh, or
// of their count, exceeds `target`: its key and place to s.key and s.at, the
// weights up to it to s.inside.
template <uint32_t N, bool DIRECT>
__device__ __noinline__ bool cut_in_bin(Lds at_s, uint32_t bin, uint32_t n, uint64_t target, bool by_count, Bins bins) {
    Picks<N, DIRECT>& s = *(Picks<N, DIRECT>*)at_s;
    const uint32_t tid = threadIdx.x;
    if (tid == 0) s.gathered = 0;
    __syncthreads();
#pragma unroll 1
    for (uint32_t i = tid; i < n; i += kThreads) {
        const float x = s.x[i];
        const uint64_t q = s.q[i];
        if (bins(x) == bin) {
            const uint32_t at = atomicAdd(&s.gathered, 1u);
            if (at < kGather) {
                s.g_key[at] = key_of(x);
                s.g_at[at] = i;
                s.g_weight[at] = q & ~kBelow;
            }
        }
    }
    __syncthreads();
    const uint32_t got = s.gathered;
    if (got > kGather) return false;
    if (tid < got) {
        const uint32_t ka = s.g_key[tid], pa = s.g_at[tid];
        const uint64_t q = s.g_weight[tid];
        uint64_t weight = 0;
        uint32_t count = 0;
#pragma unroll 4
        for (uint32_t j = 0; j < got; ++j) {
            const uint32_t kb = s.g_key[j], pb = s.g_at[j];
            const uint64_t qb = s.g_weight[j];
            const bool ahead = kb > ka || (kb == ka && pb < pa);
            weight += ahead ? qb : 0;
            count += ahead ? 1u : 0u;
        }
        const uint64_t sum = by_count ? count : weight;
        if (sum <= target && target - sum < (by_count ? 1u : q)) {
            s.key = ka;
            s.at = pa;
            s.inside = weight + q;
        }
    }
    __syncthreads();
    return true;
}

// DIRECT: rows of at most N, read here; else the row's list is.
template <uint32_t N, bool DIRECT>
__global__ __launch_bounds__(kThreads) void sample_pick_kernel(SampleArgs a, Work k) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    Picks<N, DIRECT>& s = *reinterpret_cast<Picks<N, DIRECT>*>(lds);
    const int tid = threadIdx.x, lane = tid & 63, wave = this_wave();
#pragma unroll 1
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const Wish w = wish_of(a, row);
        __syncthreads();
        s.weight[tid] = 0;
        s.count[tid] = 0;
        // the row's largest logit, its number of listed tokens, the sum of its weights
        float m = -__builtin_inff(), low = __builtin_inff();
        uint32_t n = a.vocab, flag = 0;
        Record r{-__builtin_inff(), 0.f, 0, 0};
        float2 ahead[kAhead];
        Row of_row{-__builtin_inff(), 0.f, 0.f, 0.f, 0.f, {}};
        if constexpr (!DIRECT) of_row = k.rows[row];
        const float bound = of_row.bound;
        if constexpr (DIRECT) {
            bool bad = false;
#pragma unroll 2
            for (uint32_t i = tid; i < n; i += kThreads) {
                const float x = a.logits[row * a.vocab + i];
                s.x[i] = x;
                bad |= !(x < __builtin_inff());
                m = fmaxf(m, x);
                if (x > -__builtin_inff()) low = fminf(low, x);
            }
            if (bad) m = __builtin_inff();
        } else {
            if (static_cast<uint32_t>(tid) < k.chunks) r = k.records[row * k.chunks + tid];
            // the lists' first 16 tokens, of the first 256 chunks, before their counts are known
            // (behind a list's end is memory of the workspace, read and not used)
#pragma unroll
            for (uint32_t i = 0; i < kAhead; ++i) {
                const uint32_t c = (tid >> 4) + kThreads / 16 * i;
                ahead[i] = c < k.chunks ? k.lists[(row * k.chunks + c) * kKept + (tid & 15)] : make_float2(0.f, 0.f);
            }
            m = r.max;
            flag = r.count & kOver;
        }
        m = wave_max(m);
        if constexpr (DIRECT) low = -wave_max(-low);
        flag = __any(flag != 0) ? 1u : 0u;
        if (lane == 0) {
            s.maxes[wave] = m;
            s.mins[wave] = low;
            s.flags[wave] = flag;
        }
        __syncthreads();
        m = row_max(s.maxes[lane % kWaves]);
        if constexpr (DIRECT) low = -row_max(-s.mins[lane % kWaves]);
        else flag = __any(s.flags[lane % kWaves] != 0) ? 1u : 0u;
        m = read_lane(m, 0);
        if (!(m > -__builtin_inff() && m < __builtin_inff()) || !drawable(w)) {
            if (tid == 0) no_answer(a, row);
            continue;
        }
        const bool greedy = w.t == 0.f;
        const Weigher g = DIRECT ? weigher_of(m, greedy ? 1.f : w.t) : Weigher{m, of_row.c, of_row.c_low};
        uint64_t all = 0;                        // the weights of the whole row
        if constexpr (!DIRECT) {
            // records' weights as whole numbers, and the places of their lists
            uint64_t mine = 0;
            if (wants_sum(w) && r.max > -__builtin_inff()) {
                const float2 t = g.log2_of(r.max);
                // (tokens that each weigh nothing do not together either: none of them may be drawn)
                if (g.weight_of(t) != 0) mine = static_cast<uint64_t>(static_cast<double>(r.sum * __builtin_amdgcn_exp2f(t.x) * (1.f + t.y * 0.6931471805599453f)) * 0x1p39);
            }
            const Sums of = scan2((Lds)s.sums[0], mine, r.count & ~kOver);
            all = of.a_all;
            if (!wants_list(w)) {
                // drawn from all: the record, then its tokens two a thread
                const uint64_t target = aim(w.u, max(all, uint64_t{1}));
                if (mine != 0 && of.a_before <= target && target - of.a_before < mine) {
                    s.bin = tid;
                    s.before = target - of.a_before;
                }
                __syncthreads();
                const uint32_t at = s.bin * kChunk + 2 * tid;
                const uint64_t want = s.before;
                const float u = at < a.vocab ? a.logits[row * a.vocab + at] : -__builtin_inff();
                const float v = at + 1 < a.vocab ? a.logits[row * a.vocab + at + 1] : -__builtin_inff();
                const uint64_t q = g(u), q2 = g(v);
                const Sums in = scan2((Lds)s.sums[1], q + q2, 0);
                const uint64_t place = min(want, in.a_all - 1);   // (its largest token weighs something)
                if (in.a_before <= place && place - in.a_before < q + q2) {
                    const bool second = place - in.a_before >= q;
                    answer(a, row, second ? at + 1 : at, second ? v : u, g, false, all);
                }
                continue;
            }
            n = static_cast<uint32_t>(min(of.b_all, static_cast<uint64_t>(N)));
            flag |= of.b_all > N ? 1u : 0u;
            if (flag == 0) {
                // lists into shared memory, 16 lanes a list
                s.weight[tid] = of.b_before << 32 | r.count;   // (the histogram's memory, cleared again below)
                __syncthreads();
                const uint32_t part = tid & 15;
                const auto put = [&](uint64_t of, uint32_t from, float2 v) {
                    if (from < static_cast<uint32_t>(of)) {
                        s.x[(of >> 32) + from] = v.x;
                        s.index[(of >> 32) + from] = __builtin_bit_cast(uint32_t, v.y);
                    }
                };
                uint64_t at[kAhead];
                uint32_t most = 0;
#pragma unroll
                for (uint32_t i = 0; i < kAhead; ++i) {
                    const uint32_t c = (tid >> 4) + kThreads / 16 * i;
                    at[i] = c < k.chunks ? s.weight[c] : 0;
                }
#pragma unroll
                for (uint32_t i = 0; i < kAhead; ++i) {
                    put(at[i], part, ahead[i]);
                    most = max(most, static_cast<uint32_t>(at[i]));
                }
                // what is left: longer lists, and chunks behind the first 256
                if (__any(most > 16) || k.chunks > 256) {
#pragma unroll 1
                    for (uint32_t c = tid >> 4; c < k.chunks; c += kThreads / 16) {
                        const uint64_t of_c = s.weight[c];
#pragma unroll 1
                        for (uint32_t j = c < 256 ? part + 16 : part; j < static_cast<uint32_t>(of_c); j += 16)
                            put(of_c, j, k.lists[(row * k.chunks + c) * kKept + j]);
                    }
                }
                __syncthreads();
                s.weight[tid] = 0;
            }
        }
        // tokens below `low` weigh nothing, or are in no list
        const float nothing = m - 29.2f * w.t;
        const bool complete = DIRECT || bound <= nothing;
        low = greedy ? m : fmaxf(DIRECT ? low : bound, nothing);
        const Bins bins{m, low, m > low ? (kThreads - 0.01f) / (m - low) : 0.f};
        const Floor f = DIRECT ? floor_of(greedy ? 0.f : w.m) : Floor{w.m > 0.f && !greedy, of_row.floor_hi, of_row.floor_lo};
        bool cut = false, lost = flag != 0;
        if (lost) n = 0;
        __syncthreads();
#pragma unroll 1
        for (uint32_t i = tid; i < n; i += kThreads) {
            const float x = s.x[i];
            const uint32_t bin = bins(x);
            uint64_t q = 0;
            if (bin != 0xFFFFFFFFu) {
                const float2 t = g.log2_of(x);
                q = g.weight_of(t);
                atomicAdd(&s.count[bin], 1u);
                atomicAdd(reinterpret_cast<unsigned long long*>(&s.weight[bin]), static_cast<unsigned long long>(q));
                if (x != m && !f.passes(t)) q |= kBelow;
            }
            s.q[i] = q;
        }
        __syncthreads();
        const uint32_t c_mine = s.count[tid];
        const uint64_t w_mine = s.weight[tid];
        const Sums of = scan2((Lds)s.sums[2], c_mine, w_mine);
        // (the wishes are the row's, so the workgroup goes one way)
        uint32_t key = 0, last = 0xFFFFFFFFu;
        uint64_t among = complete ? of.b_all : all;
        const uint32_t want_k = greedy ? 1u : w.k;
        if (!lost && want_k != 0) {
            if (of.a_all >= want_k) {
                if (of.a_before < want_k && of.a_before + c_mine >= want_k) {
                    s.bin = tid;
                    s.before = of.b_before;
                    s.at = want_k - static_cast<uint32_t>(of.a_before);
                }
                __syncthreads();
                const uint32_t need = s.at;
                lost = !cut_in_bin<N, DIRECT>((Lds)lds, s.bin, n, need - 1, true, bins);
                key = s.key;
                last = s.at;
                among = s.before + s.inside;
                cut = true;
            } else {
                cut = complete;                  // all that weigh anything stay
                lost = !complete;
            }
        }
        __syncthreads();
        if (!lost && !greedy && w.p < 1.f) {
            const double want = ceil(static_cast<double>(w.p) * static_cast<double>(among));
            const uint64_t target = want < 1.0 ? 0 : min(static_cast<uint64_t>(want), among) - 1;
            if (target < of.b_all) {
                if (w_mine != 0 && of.b_before <= target && target - of.b_before < w_mine) {
                    s.bin = tid;
                    s.before = target - of.b_before;
                }
                __syncthreads();
                const uint64_t in = s.before;
                lost = !cut_in_bin<N, DIRECT>((Lds)lds, s.bin, n, in, false, bins);
                key = s.key;
                last = s.at;
                cut = true;
            } else if (!cut) {
                lost = true;
            }
        }
        // (without another cut, a list that ends above what min_p lets pass is none)
        if (!cut && !complete && !(f.on && !f.passes(g.log2_of(bound)))) lost = true;
        if (lost) {
            __syncthreads();
            if (greedy) take_first(a, row, m, (Lds)lds);
            else draw_from_row(a, row, w, m, (Lds)lds);
            continue;
        }
        // the draw: a wave's tokens are consecutive, 64 a step
        const uint32_t each = ((n + kThreads - 1) / kThreads) * 64, begin = wave * each, end = min(begin + each, n);
        const auto weight = [&](uint32_t i) {
            if (i >= end) return uint64_t{0};
            const uint32_t ka = key_of(s.x[i]);
            const uint64_t q = s.q[i];
            return (ka > key || (ka == key && i <= last)) && (q & kBelow) == 0 ? q : uint64_t{0};
        };
        uint64_t sum = 0;
#pragma unroll 1
        for (uint32_t i = begin + lane; i < begin + each; i += 64) sum += weight(i);
        sum = wave_sum(sum);
        if (lane == 0) s.sums[3][0][wave] = sum;
        __syncthreads();
        const uint64_t upto_wave = row_scan(s.sums[3][0][lane % kWaves]), total = read_lane_u64(upto_wave, kWaves - 1);
        uint64_t before = read_lane_u64(upto_wave, wave) - sum;
        const uint64_t target = aim(greedy ? 0.f : w.u, total);
        if (before <= target && target - before < sum) {      // (one wave)
#pragma unroll 1
            for (uint32_t i = begin + lane; i < begin + each; i += 64) {
                const uint64_t q = weight(i);
                const uint64_t upto = wave_scan(q) + before;
                if (upto > target && upto - q <= target) answer(a, row, DIRECT ? i : s.index[i], s.x[i], g, greedy, total);
                before = read_lane_u64(upto, 63);
            }
        }
    }
}

// Rows past 2^19: a workgroup a row.
__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleArgs a) {
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 63, wave = this_wave();
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
        m = wave_max(m);
        if (__any(bad)) m = __builtin_inff();
        if (lane == 0) s.maxes[wave] = m;
        __syncthreads();
        for (int i = 0; i < kWaves; ++i) m = fmaxf(m, s.maxes[i]);
        __syncthreads();
        if (!(m > -__builtin_inff() && m < __builtin_inff()) || !drawable(w)) {
            if (tid == 0) no_answer(a, row);
        } else if (w.t == 0.f) {
            take_first(a, row, m, (Lds)&s);
        } else {
            draw_from_row(a, row, w, m, (Lds)&s);
        }
    }
}

uint32_t chunks_of(uint32_t vocab) { return (vocab + kChunk - 1) / kChunk; }
// (longer rows have more chunks than a workgroup threads: one goes over them as a whole)
bool listed(uint32_t vocab) { return vocab > kList && vocab <= kThreads * kChunk; }

template <uint32_t N, bool DIRECT>
hipError_t pick(const SampleArgs& a, const Work& k, uint32_t grid, hipStream_t s) {
    constexpr int bytes = sizeof(Picks<N, DIRECT>);
    if constexpr (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(sample_pick_kernel<N, DIRECT>), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((sample_pick_kernel<N, DIRECT>), dim3(grid), dim3(kThreads), bytes, s, a, k);
    return hipGetLastError();
}

}  // namespace

uint64_t sample_workspace_bytes(uint32_t rows, uint32_t vocab) {
    if (!listed(vocab)) return 16;
    const uint64_t slots = uint64_t{rows} * chunks_of(vocab);
    return slots * (sizeof(Record) + kKept * sizeof(float2)) + rows * sizeof(Row);
}

hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t stream) {
    const uint32_t grid = a.rows < (1u << 20) ? a.rows : (1u << 20);
    Work k{};
    if (a.vocab <= kShort) return pick<kShort, true>(a, k, grid, stream);
    if (a.vocab <= kList) return pick<kList, true>(a, k, grid, stream);
    if (!listed(a.vocab)) {
        hipLaunchKernelGGL(sample_row_kernel, dim3(grid), dim3(kThreads), 0, stream, a);
        return hipGetLastError();
    }
    k.chunks = chunks_of(a.vocab);
    const uint64_t slots = uint64_t{a.rows} * k.chunks;
    k.records = static_cast<Record*>(workspace);
    k.lists = reinterpret_cast<float2*>(k.records + slots);
    k.rows = reinterpret_cast<Row*>(k.lists + slots * kKept);
    const dim3 scan((k.chunks + 3) / 4, a.rows < 65535 ? a.rows : 65535);
    hipError_t e = hipSuccess;
    if (a.rows <= kOwnRows) {
        hipLaunchKernelGGL(sample_scan_kernel<true>, scan, dim3(256), 0, stream, a, k);
    } else {
        hipLaunchKernelGGL(sample_bound_kernel, dim3(grid), dim3(256), 0, stream, a, k);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(sample_scan_kernel<false>, scan, dim3(256), 0, stream, a, k);
    }
    e = hipGetLastError();
    return e != hipSuccess ? e : pick<kList, false>(a, k, grid, stream);
}

}  // namespace qmv
