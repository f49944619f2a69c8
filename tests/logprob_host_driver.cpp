// What qmv_logprobs' kernels list of a row, counted on the host with the
// library's own keys.  Reads lines "vocab top n_nan n_inf order seed": a row
// of n_nan NaN, n_inf -infinity and normal values else, in blocks (order 0:
// NaN first, 1: -infinity first, 2: values first) or shuffled (3).  Writes
// "E listed wrong missing" for a thread's count E of elements: keys listed for
// the row, threads whose key is not their largest, and which of the row's top
// keys are not listed.
#define __device__
#define __forceinline__ inline
#include "logprob_keys.h"

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <functional>
#include <random>
#include <vector>

template <int E>
void row(const std::vector<float>& x, uint32_t top) {
    const uint32_t vocab = static_cast<uint32_t>(x.size());
    uint64_t from = 0;
    uint32_t wrong = 0;
    std::vector<uint64_t> all;
    for (uint32_t wave = 0; wave < 4; ++wave) {
        std::vector<uint64_t> best;
        for (uint32_t tid = 64 * wave; tid < 64 * wave + 64; ++tid) {
            float v[E], m = -INFINITY;
            uint64_t largest = 0;
            for (int e = 0; e < E; ++e) {
                const uint32_t i = qmv::index_of(e, tid, 0);
                v[e] = i < vocab ? x[i] : -INFINITY;
                m = std::fmax(m, v[e]);
                if (i < vocab) {
                    all.push_back(qmv::key_of(v[e], i));
                    largest = std::max(largest, all.back());
                }
            }
            best.push_back(qmv::best_key<E>(v, m, tid, 0, vocab));
            if (best.back() != largest) ++wrong;
        }
        std::sort(best.begin(), best.end(), std::greater<uint64_t>());
        from = std::max(from, best[top - 1]);   // the wave's n-th best, 0 if it has fewer
    }
    std::sort(all.begin(), all.end(), std::greater<uint64_t>());
    uint32_t listed = 0, missing = 0;
    for (uint64_t k : all) listed += k >= std::max<uint64_t>(from, 1) ? 1 : 0;
    for (uint32_t i = 0; i < top; ++i) missing += all[i] < from ? 1 : 0;
    std::printf("%d %u %u %u\n", E, listed, wrong, missing);
}

int main() {
    uint32_t vocab, top, n_nan, n_inf, order, seed;
    while (std::scanf("%u %u %u %u %u %u", &vocab, &top, &n_nan, &n_inf, &order, &seed) == 6) {
        std::mt19937 g(seed);
        std::normal_distribution<float> normal;
        std::vector<float> x(vocab);
        for (auto& v : x) v = normal(g);
        const uint32_t rest = vocab - n_nan - n_inf;
        const uint32_t nan_at = order == 1 ? n_inf : (order == 2 ? rest : 0);
        const uint32_t inf_at = order == 1 ? 0 : (order == 2 ? rest + n_nan : n_nan);
        std::fill_n(x.begin() + nan_at, n_nan, NAN);
        std::fill_n(x.begin() + inf_at, n_inf, -INFINITY);
        if (order == 3) std::shuffle(x.begin(), x.end(), g);
        if (vocab <= 1024) row<4>(x, top);
        else if (vocab <= 2048) row<8>(x, top);
        else if (vocab <= 4096) row<16>(x, top);
        else row<32>(x, top);
    }
}
