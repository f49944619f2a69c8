// Attention over the 8-bit cache.
//
// For a query row q at position p: s_j = scale q.k_j, out = sum_j e^{s_j} v_j
// / sum_j e^{s_j} over the positions j it sees, with k_j = 2^a K_j and v_j =
// 2^b V_j (codes K, V; one scale a page and head).
//
// Few queries a key/value head (decode, and float32 prompts): exact integer
// products.  The int8 matrix cores take the codes as they lie in the cache,
// with no conversion and no shared memory; the other operand is split into
// three signed base-256 digits:
//   q = x |q|max / (127 2^16), |q|max the row's largest magnitude;
//   p = x / (127 2^16), p = e^{s - m} relative to its page's own maximum m.
// A digit's products are exact int32 sums (at most 128 * 127 * 256 < 2^23, so
// exact as float32 too), combined in float32.  Digits relative to the page's
// maximum, not to the row's, keep tokens far below the row's maximum from
// being rounded away together: a page's sums are right to 64 2^-24 of its
// own largest probability.
//
// Layout: v_mfma_i32_16x16x64_i8 gives lane l, register i the output of row
// 4 (l / 16) + i and column l % 16, and takes from lane l the 16 k-indexes
// 16 (l / 16) .. + 15.  With tokens as the rows of K q^T and row r of tile j
// read from token 16 (r / 4) + 4 j + r % 4, a lane's 16 scores (four tiles of
// 16 tokens) are those of the tokens 16 (l / 16) .. + 15 of its column: the
// very k-indexes that V^T p^T takes from it.  So probabilities go from one
// product to the next in the lane that computed them.
//
// Up to four columns (a decode step of four query heads to a key/value head,
// say) leave room for their digits beside each other: column 4 d + c is digit
// d of column c, one product takes the place of three, a score is joined by
// two rotated additions, and the output sums stay apart by digit to the end,
// one conversion and one multiply-add an output instead of five operations.
//
// Work: a workgroup of four waves has 16 columns (query row x head of one
// key/value head), or 4, and a piece of the sequence's pages; each wave takes
// every fourth page and keeps its own running maximum, sum and output, joined
// in shared memory at the end.  The pieces of a sequence are joined by a second
// kernel, in their order.  Where there are columns enough, each wave has 16 of
// its own and all of their pages, and nothing is joined.
//
// Decode is bound by memory: 32 sequences of 1000 to 4000 tokens, 32 heads on 8
// of 128, 38.2 us, 4.5 TB/s; two of up to 131072 62.0 us and 4.8 for the join,
// 5.1 TB/s (the same pages read by nothing but loads: 5.8 to 6.0); one of 100
// tokens 5.1 us, a launch and three dependent trips.  A float32 prompt of 8192
// takes 1394 us, 394 TFLOP/s, bound by the vector operations that make digits
// and join their products.  Sequences are dealt out by count, not by length: 31
// of 1000 and one of 131072 take 696 us, the long one alone 47, as eight
// workgroups, one a head, walk its pages.
#include <type_traits>

#include "kv_common.h"

namespace qmv {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPScale = 127.0f * 65536.0f;   // p = 1 as a whole number
// How the kernel for few queries deals out its work: a workgroup has 16
// columns, or 4 whose digits lie beside each other, and its waves share the
// pages; or each wave has 16 columns and all of their pages.
enum Few { kWide, kPack, kSolo };
constexpr int few_cols(Few mode) { return mode == kPack ? 4 : (mode == kWide ? 16 : 64); }   // columns of a workgroup
constexpr uint32_t kTarget = 256;              // workgroups that a launch aims at

struct AttendArgs {
    qmv_kv_cache c;
    qmv_kv_seqs s;
    const void* q;
    void* out;
    float* part;        // [pieces][rows * heads][D]: output sums
    float2* stat;       // [pieces][rows * heads]: maximum, sum
    float scale_log2;   // scale * log2(e)
    uint32_t heads, group, window, pieces;
    uint32_t per;       // pages of a piece, at least
};

// Three signed digits of each of four whole numbers |x| <= 127 * 2^16, as
// dwords of four bytes: x = d0 + 256 d1 + 65536 d2.  Given are u = x + 0x8080,
// whose lower two bytes are the digits 128 up.
__device__ __forceinline__ void digits4(const uint32_t u[4], uint32_t d[3]) {
    // bytes 0 of (u0, u1) and (u2, u3), bytes 1, bytes 2
    const uint32_t a = __builtin_amdgcn_perm(u[1], u[0], 0x05010400u);  // b0 b0' b1 b1'
    const uint32_t b = __builtin_amdgcn_perm(u[3], u[2], 0x05010400u);
    d[0] = __builtin_amdgcn_perm(b, a, 0x05040100u) ^ 0x80808080u;
    d[1] = __builtin_amdgcn_perm(b, a, 0x07060302u) ^ 0x80808080u;
    const uint32_t e = __builtin_amdgcn_perm(u[1], u[0], 0x00000602u);
    const uint32_t f = __builtin_amdgcn_perm(u[3], u[2], 0x06020000u);
    d[2] = __builtin_amdgcn_perm(f, e, 0x07060100u);
}

// The number that three digits' products stand for, times 2^-16: the lower
// two are joined as whole numbers (below 2^30 in sum).
__device__ __forceinline__ float join3(int c0, int c1, int c2) {
    return fmaf(static_cast<float>(c1 * 256 + c0), 0x1p-16f, static_cast<float>(c2));
}

__device__ __forceinline__ float xor_lane(float v, int m) { return __shfl_xor(v, m); }

// Sum of c times w of the lanes 4, 8 and 12 apart in a row of 16, the same
// bits in each: the products are rounded before they are added (fused, each
// lane would round the others' alone, and digits that are then made of a sum
// in different lanes would not be of one number).
__device__ __forceinline__ float add_slots(float c, float w) {
#pragma clang fp contract(off)
    float v = c * w;
    v += dpp_mov<0x128>(v);  // row_ror:8
    v += dpp_mov<0x124>(v);  // row_ror:4
    return v;
}

// What a workgroup's columns are.  Columns of a sequence and key/value head
// (rows * group, below 2^31) are numbered row first.
struct Columns {
    int32_t row;                 // this lane's query row, -1: none
    int32_t pos;                 // its position
    uint32_t head;
    int32_t first_pos, last_pos; // smallest and largest position of the columns
    int32_t lo, hi;              // positions that any of the columns sees: [lo, hi)
};
template <uint32_t COLS>
__device__ __forceinline__ Columns columns(const AttendArgs& a, const SeqRows& r, uint32_t kvh, uint32_t tile,
                                           uint32_t col) {
    Columns o;
    const uint32_t n = static_cast<uint32_t>(r.count) * a.group, c = tile * COLS + col;
    const uint32_t t0 = tile * COLS / a.group;
    const uint32_t t1 = min(tile * COLS + COLS - 1, n - 1) / a.group;
    const uint32_t t = c / a.group;
    o.row = c < n ? r.first + static_cast<int32_t>(t) : -1;
    o.pos = r.base + static_cast<int32_t>(t);
    o.head = kvh * a.group + (c - t * a.group);
    o.first_pos = r.base + static_cast<int32_t>(t0);
    o.last_pos = r.base + static_cast<int32_t>(t1);
    // (what a sequence claims past its table is in no page)
    const uint32_t room = min(a.s.table_stride, 0x7FFF0000u / kPage) * kPage;
    o.hi = min(max(o.last_pos + 1, 0), static_cast<int32_t>(room));
    o.lo = sees_from(a.window, max(o.first_pos, 0));
    return o;
}

template <uint32_t DT, int D, Few MODE>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void attend_few_kernel(AttendArgs a) {
    typedef typename Elem<DT>::type T;
    constexpr bool PACK = MODE == kPack, SOLO = MODE == kSolo;
    constexpr int kCols = PACK ? 4 : 16;
    constexpr int STEP = SOLO ? 1 : 4;   // waves that share the pages
    constexpr int ND = PACK ? 1 : 3;   // digits in a lane
    constexpr int KS = D / 64;     // k-steps of a score tile
    constexpr int ET = D / 16;     // tiles of output dims
    __shared__ float acc[STEP][kCols][SOLO ? 1 : D + 1];
    __shared__ float stat[STEP][kCols][2];
    __shared__ float4 part[kCols];       // what each wave's output counts for
    __shared__ uint64_t place[kCols];    // where the column goes (row * heads + head)
    const int lane = threadIdx.x & 63, quad = lane >> 4;
    const int lane16 = lane & 15, col = PACK ? lane & 3 : lane16, slot = lane16 >> 2;
    // packed: this lane's digit, its weight (slot 3: none), the bytes it takes
    // of pairs of words, and which of them are kept 128 up
    const float weight = !PACK ? 1.f : (slot == 0 ? 0x1p-16f : (slot == 1 ? 0x1p-8f : (slot == 2 ? 1.f : 0.f)));
    const uint32_t pick = slot == 3 ? 0x0C0Cu : static_cast<uint32_t>(slot * 0x101 + 0x400);
    const uint32_t pick_lo = 0x0C0C0000u | pick, pick_hi = (pick << 16) | 0x0C0Cu;
    const uint32_t lift = slot < 2 ? 0x80808080u : 0u;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t seq = blockIdx.x / a.c.kv_heads, kvh = blockIdx.x % a.c.kv_heads;
    const uint32_t piece = blockIdx.z;
    const SeqRows r = seq_rows(a.s, seq);
    const uint32_t all = static_cast<uint32_t>(r.count) * a.group;
    const uint32_t tiles = (all + kCols - 1) / kCols;
    // the last tiles see the most: they begin first
    constexpr uint32_t kOwn = SOLO ? 4 : 1;   // tiles of a workgroup
    for (uint32_t turn = kOwn * blockIdx.y + (SOLO ? wave : 0); turn < tiles; turn += kOwn * gridDim.y) {
        const uint32_t tile = tiles - 1 - turn;
        const Columns w = columns<kCols>(a, r, kvh, tile, col);
        // pages of this piece
        const int32_t p_lo = w.lo / kPage, p_hi = (w.hi + kPage - 1) / kPage;
        const int32_t per = max((p_hi - p_lo + static_cast<int32_t>(a.pieces) - 1) / static_cast<int32_t>(a.pieces),
                                static_cast<int32_t>(a.per));
        const int64_t begin = p_lo + static_cast<int64_t>(piece) * per;
        const int32_t p0 = static_cast<int32_t>(min(begin, static_cast<int64_t>(p_hi)));
        const int32_t p1 = min(p_hi - p0, per) + p0;
        const int32_t see_lo = sees_from(a.window, w.pos);
        // pages that every column sees whole: from full_lo up to full_hi
        const int32_t full_lo = (sees_from(a.window, w.last_pos) + kPage - 1) / kPage;
        const int32_t full_hi = max(w.first_pos + 1, 0) / kPage;

        // Lane i has the page ids and scales of the wave's next pages, 64 of
        // them from one trip to memory.  Keys of the next page are requested
        // as soon as this page's have been multiplied, its values while the
        // scores are formed: a wave always has keys or values on the way.
        i32x4 kf[4][KS];
        int32_t ids = -1, id = -1;
        float kss = 0.f, vss = 0.f;
        const int krow = 16 * (lane16 >> 2) + (lane16 & 3);
        // What the table says (where there is no page its first entry is read
        // and not used, so that the load waits for no branch).
        auto entry = [&](int32_t p) {
            const int32_t mine = p + STEP * lane;
            const bool there = mine < p1;        // (p1 is at most the table's length)
            const int32_t id = a.s.table[static_cast<uint64_t>(seq) * a.s.table_stride + (there ? mine : 0)];
            return there ? id : -1;
        };
        auto look = [&](int32_t id) {
            ids = id >= 0 && static_cast<uint32_t>(id) < a.c.pages ? id : -1;
            if (ids >= 0) {
                const uint64_t at = static_cast<uint64_t>(ids) * a.c.kv_heads + kvh;
                kss = a.c.k_scale[at];
                vss = a.c.v_scale[at];
            }
        };
        auto fetch = [&](int n) {
            // (where there is no page, page 0, which every cache has, is read
            // and not used: a branch here would keep two sets of registers)
            id = __builtin_amdgcn_readlane(ids, n);
            const uint64_t at = static_cast<uint64_t>(max(id, 0)) * a.c.kv_heads + kvh;
            const int8_t* kp = a.c.k + at * (kPage * D) + krow * D + 16 * quad;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    kf[j][s] = *reinterpret_cast<const i32x4*>(kp + 4 * j * D + 64 * s);
        };
        // (the query is on the way while the pages are looked up)
        const int32_t first_entry = entry(p0 + (SOLO ? 0 : wave));
        float v[KS][16];
        {
            const T* qp = static_cast<const T*>(a.q) + (static_cast<uint64_t>(w.row < 0 ? 0 : w.row) * a.heads + w.head) * D;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if (w.row >= 0) {
                    load8<DT>(qp + 64 * s + 16 * quad, v[s]);
                    load8<DT>(qp + 64 * s + 16 * quad + 8, v[s] + 8);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[s][i] = 0.f;
                }
            }
        }
        int n = 0;                               // the page's lane
        look(first_entry);
        fetch(0);

        // the query's digits
        uint32_t qd[KS][ND][4];
        float qs;
        {
            uint32_t m = 0;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 16; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[s][i]) & 0x7FFFFFFFu);
            m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
            m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
            const bool none = m >= 0x7F800000u;
            const float amax = none ? 0.f : __builtin_bit_cast(float, m);
            qs = none ? __builtin_nanf("") : amax / 127.f;        // 2^16 times the digits' unit
            // rows that hold no numbers count as 0, and small ones are moved
            // up first, where 1 / amax is finite
            const bool low = amax < 0x1p-96f;
            if (__any(none || low)) {
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[s][i] = none ? 0.f : v[s][i] * (low ? 0x1p64f : 1.f);
            }
            const float mul = amax == 0.f ? 0.f : kPScale / (low ? amax * 0x1p64f : amax);
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = static_cast<int>(rintf(v[s][4 * j + i] * mul)) + 0x8080;
                    if constexpr (PACK) {
                        qd[s][0][j] = (__builtin_amdgcn_perm(x[1], x[0], pick_lo) | __builtin_amdgcn_perm(x[3], x[2], pick_hi)) ^ lift;
                    } else {
                        uint32_t d[3];
                        digits4(x, d);
#pragma unroll
                        for (int k = 0; k < 3; ++k) qd[s][k][j] = d[k];
                    }
                }
        }

        float o[ET][4];
#pragma unroll
        for (int e = 0; e < ET; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[e][i] = 0.f;
        float m_run = -__builtin_inff(), l_run = 0.f;

        for (int32_t p = p0 + (SOLO ? 0 : wave); p < p1; p += STEP, n = (n + 1) & 63) {
            const int32_t at_id = id;
            const float kscale = read_lane(kss, n) * a.scale_log2, vscale = read_lane(vss, n);
            if (n == 63) look(entry(p + STEP));
            if (at_id < 0) {
                fetch((n + 1) & 63);
                continue;
            }
            const int8_t* vp = a.c.v + (static_cast<uint64_t>(at_id) * a.c.kv_heads + kvh) * (kPage * D);
            i32x4 vf[ET];
#pragma unroll
            for (int e = 0; e < ET; ++e)
                vf[e] = *reinterpret_cast<const i32x4*>(vp + (16 * e + lane16) * kPage + 16 * quad);
            // scores
            float sc[4][4];
            const float qk = qs * kscale * weight;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                i32x4 c[ND];
#pragma unroll
                for (int k = 0; k < ND; ++k) c[k] = i32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int k = 0; k < ND; ++k) {
                        const i32x4 b = {static_cast<int>(qd[s][k][0]), static_cast<int>(qd[s][k][1]),
                                         static_cast<int>(qd[s][k][2]), static_cast<int>(qd[s][k][3])};
                        c[k] = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[j][s], b, c[k], 0, 0, 0);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (PACK) sc[j][i] = add_slots(static_cast<float>(c[0][i]), qk);
                    else sc[j][i] = join3(c[0][i], c[1][i], c[2][i]) * qk;
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            fetch((n + 1) & 63);
            __builtin_amdgcn_sched_barrier(0);
            // what this column sees of the page: all of it in the middle of a
            // sequence, else the tokens [from, to)
            bool any = true;
            if (p < full_lo || p >= full_hi) {
                const int from = max(see_lo - p * kPage, 0);
                const int to = w.row < 0 ? 0 : min(w.pos + 1 - p * kPage, kPage);
                any = from < to;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = 16 * quad + 4 * j + i;
                        sc[j][i] = t >= from && t < to ? sc[j][i] : -__builtin_inff();
                    }
            }
            float mt = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) mt = fmaxf(mt, sc[j][i]);
            mt = max_quads(mt);
            // nothing seen, or only NaN: the maximum counts as 0 (NaN scores
            // still make the sum NaN, and so does a score of +infinity)
            const float ref = mt > -__builtin_inff() ? mt : 0.f;
            float lt[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t pd[ND][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float pr = __builtin_amdgcn_exp2f(sc[j][i] - ref);
                    lt[i] += pr;
                    // the whole number nearest to p 127 2^16 + 0x8080 < 2^23
                    // is in the low three bytes of its sum with 2^23
                    x[i] = __builtin_bit_cast(uint32_t, fmaf(pr, kPScale, 0x1p23f + 0x8080));
                }
                if constexpr (PACK) {
                    pd[0][j] = (__builtin_amdgcn_perm(x[1], x[0], pick_lo) | __builtin_amdgcn_perm(x[3], x[2], pick_hi)) ^ lift;
                } else {
                    uint32_t d[3];
                    digits4(x, d);
#pragma unroll
                    for (int k = 0; k < 3; ++k) pd[k][j] = d[k];
                }
            }
            // Sums (of this lane's tokens; the lanes' are added at the end)
            // are kept relative to the maximum of the first page seen and
            // moved to a larger one only where that is 2^40 away; a page that
            // this column does not see leaves everything as it is, whatever
            // its scales are.
            const float off = ref - m_run;
            if (__any(any && !(off <= 40.f))) {
                const float m_new = any && !(off <= 40.f) ? ref : m_run;
                const float keep = m_run == m_new ? 1.f : __builtin_amdgcn_exp2f(m_run - m_new);
                l_run *= keep;
                m_run = m_new;
#pragma unroll
                for (int e = 0; e < ET; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[e][i] *= keep;
            }
            const float add = any ? __builtin_amdgcn_exp2f(ref - m_run) : 0.f;
            const float put = any ? add * (vscale * (65536.f / kPScale)) * weight : 0.f;
            l_run += any ? add * ((lt[0] + lt[1]) + (lt[2] + lt[3])) : 0.f;
#pragma unroll
            for (int e = 0; e < ET; ++e) {
                i32x4 c[ND];
#pragma unroll
                for (int k = 0; k < ND; ++k) {
                    const i32x4 b = {static_cast<int>(pd[k][0]), static_cast<int>(pd[k][1]),
                                     static_cast<int>(pd[k][2]), static_cast<int>(pd[k][3])};
                    c[k] = __builtin_amdgcn_mfma_i32_16x16x64_i8(vf[e], b, i32x4{0, 0, 0, 0}, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (PACK) o[e][i] = fmaf(static_cast<float>(c[0][i]), put, o[e][i]);
                    else o[e][i] = fmaf(join3(c[0][i], c[1][i], c[2][i]), put, o[e][i]);
                }
                if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
        }

        l_run += xor_lane(l_run, 16);
        l_run += xor_lane(l_run, 32);
        if constexpr (SOLO) {
            if (w.row >= 0) {
                const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
                const uint64_t at = (static_cast<uint64_t>(w.row) * a.heads + w.head) * D + 4 * quad;
#pragma unroll
                for (int e = 0; e < ET; ++e) {
                    const float v[4] = {o[e][0] * inv, o[e][1] * inv, o[e][2] * inv, o[e][3] * inv};
                    if constexpr (DT == QMV_F32) {
                        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + 16 * e) = make_float4(v[0], v[1], v[2], v[3]);
                    } else {
                        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                        const bf16x4 x = {static_cast<__bf16>(v[0]), static_cast<__bf16>(v[1]), static_cast<__bf16>(v[2]), static_cast<__bf16>(v[3])};
                        *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(a.out) + at + 16 * e) = x;
                    }
                }
            }
            continue;
        }
        // the four waves' results
#pragma unroll
        for (int e = 0; e < ET; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = PACK ? add_slots(o[e][i], 1.f) : o[e][i];
                if (!PACK || slot == 0) acc[wave][col][16 * e + 4 * quad + i] = v;
            }
        if (quad == 0 && (!PACK || slot == 0)) {
            stat[wave][col][0] = m_run;
            stat[wave][col][1] = l_run;
        }
        __syncthreads();
        if (threadIdx.x < kCols) {
            const int cc = threadIdx.x;
            const uint32_t gc = tile * kCols + cc;
            float m = stat[0][cc][0], l = 0.f, f[4];
#pragma unroll
            for (int u = 1; u < 4; ++u) m = fmaxf(m, stat[u][cc][0]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                f[u] = stat[u][cc][0] == m ? 1.f : exp2f(stat[u][cc][0] - m);
                l += f[u] * stat[u][cc][1];
            }
            const uint64_t at = static_cast<uint64_t>(r.first + static_cast<int32_t>(gc / a.group)) * a.heads + kvh * a.group + gc % a.group;
            const float inv = a.pieces == 1 ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            part[cc] = make_float4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
            place[cc] = at;
            if (a.pieces != 1 && gc < all) a.stat[static_cast<uint64_t>(piece) * a.s.rows * a.heads + at] = make_float2(m, l);
        }
        __syncthreads();
        const int here = static_cast<int>(min(all - tile * kCols, static_cast<uint32_t>(kCols)));
        for (int i = threadIdx.x; i < here * D; i += 256) {
            const int cc = i / D, dim = i % D;
            const float4 f = part[cc];
            const float res = (f.x * acc[0][cc][dim] + f.y * acc[1][cc][dim]) + (f.z * acc[2][cc][dim] + f.w * acc[3][cc][dim]);
            if (a.pieces == 1) {
                if constexpr (DT == QMV_F32) static_cast<float*>(a.out)[place[cc] * D + dim] = res;
                else static_cast<__bf16*>(a.out)[place[cc] * D + dim] = static_cast<__bf16>(res);
            } else if (p0 < p1) {
                // (of a piece without pages only the statistics are read)
                a.part[(static_cast<uint64_t>(piece) * a.s.rows * a.heads + place[cc]) * D + dim] = res;
            }
        }
        __syncthreads();
    }
}

// ---- many queries a key/value head (bfloat16 prompts) -------------------------
//
// Products on v_mfma_f32_32x32x16_f16: a workgroup of eight waves has 256
// columns, each wave 32, and walks the pages that any of them sees.  A page's
// codes come from memory into registers one page ahead, are made f16 once for
// all waves on the way into shared memory (1024 + 128 + code is the f16 with
// the bits 0x6400 | (code ^ 0x80); one packed operation takes the 1152 off
// again) and lie there twice, so that one barrier a page is enough.
//
// The scores' operands are exact: a query row is scaled by a power of two to a
// largest magnitude in [2^14, 2^15) (bfloat16's 8 bits fit f16's 11; what is below
// 2^-31 of the largest is rounded to 2^-39 of it), codes are whole numbers.  The
// values' scales enter as powers of two relative to the unit of the outputs so
// far, whose exponent follows the pages' largest: code 2^(e - unit), exact in f16
// from 2^-24 to 2^5.  For a page further below, the outputs are moved to a lower
// unit and back after it, which takes nothing from them down to 2^-96 of the
// largest.  Probabilities are rounded to f16 and their sum is taken from the
// rounded ones, so that numerator and denominator agree.  They are relative to a
// running reference, times 2^3, that is moved (and the outputs scaled) where a
// page's maximum is 2^6 above it, or, where no maximum is sought, where a lane's
// sum reaches 2^15, so that they stay f16; down to 2^-17 of the reference they
// keep all of f16's bits, down to 2^-27 some.
//
// Rows and columns are arranged as above: the 32 x 32 output gives lane l,
// register 4 a + b the row 8 a + 4 (l / 32) + b and takes the k-indexes 8 (l /
// 32) + .. from it, so with row r of a tile read from token 16 (a / 2) + 8 (l
// / 32) + 4 (a % 2) + b the probabilities stay in their lanes.
//
// Shared memory: 16-byte chunks of a row are permuted by the row's number, so
// that lanes that read the same chunk of different rows do not meet in a bank
// (the stores, one to eight reads and fewer, do: 8 cycles each).
//
// Measured: a prompt of 8192 with 32 heads on 8 of 128, 592 us, 929 TFLOP/s (a
// large bfloat16 product: 1380).  By counters the matrix cores are busy in 38%
// of the SIMDs' cycles and vector instructions issue in 42%; waves wait in 32%
// of theirs (two a SIMD, a barrier a page), in 5% for shared memory, though each
// operand of a product is read from there for 32 columns alone, at 128 bytes a
// cycle as long as the product takes.  Three pieces of up to 500 rows under a
// window of 1024, 16 heads on 4 of 256, 60 us, 342 TFLOP/s: the same, and 160
// tiles for 256 compute units.

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kPBias = 3.0f;         // probabilities times 2^3
constexpr float kMoveAt = 6.0f;        // reference moved when a maximum is 2^6 above

// Columns of a workgroup of eight waves.
constexpr int many_cols(int d) { return d == 256 ? 128 : 256; }

// Row r of a score tile: its token.
__device__ __forceinline__ int token_of_row(int r) {
    const int a = r >> 3, h = (r >> 2) & 1, b = r & 3;
    return 16 * (a >> 1) + 8 * h + 4 * (a & 1) + b;
}
// Permutation of the 16-byte chunks of a row of `chunks`: 16 rows that are
// read together fall into all 16 chunks' worth of the 64 banks (two rows of 8
// chunks lie side by side in them).  Permuted by row & 7 alone, reads took
// 1.47 times as long.
template <int CHUNKS>
__device__ __forceinline__ int swizzle(int row) { return CHUNKS == 8 ? (row >> 1) & 7 : row & 15; }

// 16 codes as f16, each times mul (less = -1152 mul).
__device__ __forceinline__ void codes_to_f16(i32x4 c, f16x2 mul, f16x2 less, f16x8 out[2]) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint32_t u = static_cast<uint32_t>(c[w]) ^ 0x80808080u;
        const f16x2 lo = __builtin_elementwise_fma(
            __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)), mul, less);
        const f16x2 hi = __builtin_elementwise_fma(
            __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)), mul, less);
        out[w >> 1][4 * (w & 1)] = lo[0];
        out[w >> 1][4 * (w & 1) + 1] = lo[1];
        out[w >> 1][4 * (w & 1) + 2] = hi[0];
        out[w >> 1][4 * (w & 1) + 3] = hi[1];
    }
}
// 2^up and -1152 2^up for up from -24 to 5, as f16 twice.
__device__ __forceinline__ uint32_t f16_power(int up) {
    return (up >= -14 ? static_cast<uint32_t>(up + 15) << 10 : 1u << (up + 24)) * 0x10001u;
}
__device__ __forceinline__ uint32_t f16_less(int up) {   // 1152 = 1.125 2^10
    return (0x8080u | static_cast<uint32_t>(up + 25) << 10) * 0x10001u;
}

// Exponent of a scale, a power of two; kNone for 0, kNan for what is no number.
constexpr int kNone = -1000, kNan = 1000;
// f16 holds codes times 2^-kBelow to 2^kAbove (the packed conversion stays
// below 65504 up to there).  kFar: how far below the largest a unit goes.  A
// page's probabilities sum to less than 2^17, its outputs to 2^29, those of 2^25
// pages to 2^54: 2^72 times that is a float32.
constexpr int kAbove = 5, kBelow = 24, kFar = 72;
__device__ __forceinline__ int exponent_of(float s) {
    const uint32_t b = __builtin_bit_cast(uint32_t, s) & 0x7FFFFFFFu;
    return b < 0x00800000u ? kNone : (b >= 0x7F800000u ? kNan : static_cast<int>(b >> 23) - 127);
}

// Head dims of 256 hold too many registers for a wave of 32 columns: waves w
// and w + 4 have the same 32.  Each scores and weighs half of a page's tokens,
// they exchange the probabilities through shared memory, and each adds up half
// of the output dims.  Whether a page is masked or its maximum is sought is
// then decided for the workgroup, whose waves meet at the barriers.
template <int D>
__global__ __launch_bounds__(512, 2) void attend_many_kernel(AttendArgs a) {
    constexpr int NT = 512;
    constexpr bool PAIR = D == 256;
    constexpr int COLS = many_cols(D);
    constexpr int ST = PAIR ? 1 : 2;             // tiles of 32 tokens that a wave scores
    constexpr int KC = D / 8;                    // 16-byte chunks of a key row
    constexpr int UNITS = 2 * kPage * D / 16;    // 16-code pieces of a page: keys, then values
    constexpr int PER = UNITS / NT;
    constexpr int QS = D / 16;                   // k-steps of a score
    constexpr int ET = D / (PAIR ? 64 : 32);     // tiles of output dims that a wave adds up
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    f16x8* const kbuf = reinterpret_cast<f16x8*>(lds);                       // [2][64][KC]
    f16x8* const vbuf = kbuf + 2 * kPage * KC;                               // [2][D][8]
    // (pairs) probabilities [4 column groups][4 k-steps][64 lanes], maxima and
    // sums [4][2 halves][32], whether a page has to be done again
    f16x8* const pbuf = vbuf + 2 * D * 8;
    float* const mbuf = reinterpret_cast<float*>(pbuf + 4 * 4 * 64);
    int* const again = reinterpret_cast<int*>(mbuf + 4 * 2 * 32);            // [2]
    const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t seq = blockIdx.x / a.c.kv_heads, kvh = blockIdx.x % a.c.kv_heads;
    const uint32_t piece = blockIdx.z;
    const SeqRows r = seq_rows(a.s, seq);
    const uint32_t all = static_cast<uint32_t>(r.count) * a.group;
    const uint32_t tiles = (all + COLS - 1) / COLS;
    // the last tiles see the most: they begin first
    for (uint32_t turn = blockIdx.y; turn < tiles; turn += gridDim.y) {
        const uint32_t tile = tiles - 1 - turn;
        const int group = PAIR ? wave & 3 : wave, part = PAIR ? wave >> 2 : 0;
        const Columns w = columns<COLS>(a, r, kvh, tile, group * 32 + col);
        const int32_t p_lo = w.lo / kPage, p_hi = (w.hi + kPage - 1) / kPage;
        const int32_t per = max((p_hi - p_lo + static_cast<int32_t>(a.pieces) - 1) / static_cast<int32_t>(a.pieces),
                                static_cast<int32_t>(a.per));
        const int64_t begin = p_lo + static_cast<int64_t>(piece) * per;
        const int32_t p0 = static_cast<int32_t>(min(begin, static_cast<int64_t>(p_hi)));
        const int32_t p1 = min(p_hi - p0, per) + p0;
        const int32_t see_lo = sees_from(a.window, w.pos);
        // this wave's columns: what any sees, and the pages that all see whole
        const uint32_t c0 = tile * COLS + group * 32;
        const uint32_t n_cols = c0 < all ? min(all - c0, 32u) : 0u;
        const int32_t wf = r.base + static_cast<int32_t>(c0 / a.group);
        const int32_t wl = r.base + static_cast<int32_t>((c0 + max(n_cols, 1u) - 1) / a.group);
        const int32_t w_lo = sees_from(a.window, max(wf, 0));
        const int32_t w_hi = n_cols != 0 ? max(wl + 1, 0) : 0;
        // (as page numbers: some seen, all seen by all)
        const int32_t seen_lo = w_lo / kPage, seen_hi = (w_hi + kPage - 1) / kPage;
        // (columns without a row have zero queries and may see anything)
        const int32_t full_lo = (sees_from(a.window, PAIR ? w.last_pos : wl) + kPage - 1) / kPage;
        const int32_t full_hi = PAIR || n_cols != 0 ? max((PAIR ? w.first_pos : wf) + 1, 0) / kPage : 0;

        // the queries, f16, as the second operand of the scores
        f16x8 qf[QS];
        float qs;
        {
            const uint16_t* qp = static_cast<const uint16_t*>(a.q) +
                                 (static_cast<uint64_t>(w.row < 0 ? 0 : w.row) * a.heads + w.head) * D;
            uint4 raw[QS];
            uint32_t m = 0;
#pragma unroll
            for (int s = 0; s < QS; ++s) {
                raw[s] = make_uint4(0, 0, 0, 0);
                if (w.row >= 0) raw[s] = *reinterpret_cast<const uint4*>(qp + 16 * s + 8 * half);
            }
#pragma unroll
            for (int s = 0; s < QS; ++s) {
                const uint32_t u[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) m = max(m, max(u[i] & 0x7FFFu, (u[i] >> 16) & 0x7FFFu));
            }
            m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
            const bool zero = m == 0 || m >= 0x7F80u;
            int e = 0;
            if (!zero) (void)frexpf(__builtin_bit_cast(float, m << 16), &e);   // |q| < 2^e
            qs = m >= 0x7F80u ? __builtin_nanf("") : (zero ? 0.f : ldexpf(1.f, e - 15));
#pragma unroll
            for (int s = 0; s < QS; ++s) {
                const uint32_t u[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = __builtin_bit_cast(float, u[i] << 16), y = __builtin_bit_cast(float, u[i] & 0xFFFF0000u);
                    qf[s][2 * i] = static_cast<_Float16>(zero ? 0.f : ldexpf(a.scale_log2 < 0.f ? -x : x, 15 - e));
                    qf[s][2 * i + 1] = static_cast<_Float16>(zero ? 0.f : ldexpf(a.scale_log2 < 0.f ? -y : y, 15 - e));
                }
            }
        }
        const float q_log2 = qs * fabsf(a.scale_log2);   // (a negative scale's sign is in the queries)

        f32x16 o[ET];
#pragma unroll
        for (int e = 0; e < ET; ++e)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[e][i] = 0.f;
        float m_run = -__builtin_inff(), l_run = 0.f;   // this lane's part of the sum
        int e_ref = kNone, unit = kNone;                // largest exponent so far, that of the outputs' unit

        // Lane i has, of page at + i: its place (page id * kv_heads + head; -1:
        // none), its keys' scale and its values' scale's exponent.
        int32_t at = p0, places = -1, exps = kNone;
        float kss = 0.f;
        auto look = [&](int32_t p) {
            at = p;
            const int32_t id = p + lane < p1 ? page_id(a.c, a.s, seq, p + lane) : -1;
            places = -1;
            if (id >= 0) {
                places = id * static_cast<int32_t>(a.c.kv_heads) + static_cast<int32_t>(kvh);
                kss = a.c.k_scale[places];
                exps = exponent_of(a.c.v_scale[places]);
            }
        };
        auto place = [&](int32_t p) { return p < p1 ? __builtin_amdgcn_readlane(places, p - at) : -1; };

        // The codes of one page's keys and one's values, on the way from memory
        // while pages before are computed (where there is no page, page 0 is
        // read and not used).  A wave's pieces are all keys or all values.
        i32x4 st[PER];
        const int8_t* const k_from = a.c.k + 16 * tid;
        const int8_t* const v_from = a.c.v + 16 * tid - 8 * UNITS;
        auto fetch = [&](int32_t kp, int32_t vp) {
            const int64_t k_at = static_cast<int64_t>(max(place(kp), 0)) * (kPage * D);
            const int64_t v_at = static_cast<int64_t>(max(place(vp), 0)) * (kPage * D);
#pragma unroll
            for (int u = 0; u < PER; ++u)
                st[u] = *reinterpret_cast<const i32x4*>((wave * 64 + u * NT < UNITS / 2 ? k_from + k_at : v_from + v_at) + 16 * u * NT);
        };
        // Into shared memory; the values times 2^up (0 where that is below f16).
        auto stage = [&](int kb, int vb, int up) {
            const uint32_t v_mul = up < -kBelow ? 0u : f16_power(up), v_less = up < -kBelow ? 0u : f16_less(up);
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int i = tid + u * NT;
                // (known at compile time but for head dims of 64)
                const bool keys = UNITS / 2 % NT == 0 ? u * NT < UNITS / 2 : wave * 64 < UNITS / 2;
                f16x8 x[2];
                if (keys) {
                    codes_to_f16(st[u], __builtin_bit_cast(f16x2, f16_power(0)), __builtin_bit_cast(f16x2, f16_less(0)), x);
                    const int row = i / (D / 16), c = (2 * (i % (D / 16))) ^ swizzle<KC>(row);
                    f16x8* d = kbuf + (kb * kPage + row) * KC;
                    d[c] = x[0];
                    d[c ^ 1] = x[1];
                } else {
                    codes_to_f16(st[u], __builtin_bit_cast(f16x2, v_mul), __builtin_bit_cast(f16x2, v_less), x);
                    const int k = i - UNITS / 2, row = k >> 2, c = (2 * (k & 3)) ^ swizzle<8>(row);
                    f16x8* d = vbuf + (vb * D + row) * 8;
                    d[c] = x[0];
                    d[c ^ 1] = x[1];
                }
            }
        };
        // Settles the unit for a page's values, and what they are staged with.
        int want = kNone;                        // the unit's exponent for the page staged
        auto settle = [&](int32_t p) {
            if (place(p) < 0) return kNone;
            const int e = __builtin_amdgcn_readlane(exps, p - at);
            if (e == kNone) return kNone;
            if (e == kNan) return 0;             // (sums that see them are NaN)
            if (e - e_ref > kAbove) e_ref = e;   // (kNone: the first)
            want = e - e_ref < -kBelow ? max(e, e_ref - kFar) : e_ref;
            return e - want;
        };
        // whether this wave's columns (a pair's workgroup's) see anything of a page
        auto seen = [&](int32_t p) { return (PAIR || (p >= seen_lo && p < seen_hi)) && place(p) >= 0; };
        // Chunk 2 s + half of a row, permuted, is the row's chunk (half ^
        // permutation) with the bits of 2 s flipped.  (The addresses are hidden
        // from the compiler, which would keep one for every read in a register.)
        const uint32_t k_row = static_cast<uint32_t>((32 * part + token_of_row(col)) * KC + (half ^ swizzle<KC>(token_of_row(col))));
        const uint32_t v_row = static_cast<uint32_t>((32 * ET * part + col) * 8 + (half ^ swizzle<8>(col)));
        // N products whose operands are read from shared memory kAhead ahead.
        auto pipelined = [](auto n) {
            constexpr int kAhead = 6, N = decltype(n)::value;
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
            for (int i = 0; i < N - kAhead; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto scores = [&](int b, f32x16 (&sc)[ST]) {
            __builtin_amdgcn_sched_barrier(0);
            uint32_t from = k_row + b * kPage * KC;
            asm volatile("" : "+v"(from));
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
#pragma unroll
            for (int s = 0; s < QS; ++s)
#pragma unroll
                for (int t = 0; t < ST; ++t)
                    sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kbuf[(from ^ (2 * s)) + 32 * t * KC], qf[s], sc[t], 0, 0, 0);
            pipelined(std::integral_constant<int, ST * QS>{});
        };
        // The values' products; of pairs beside them the next page goes into
        // shared memory (three pieces of 500 under a window of 1024: 65 us with
        // one after the other, 62 so; head dims of 128 and 64, whose waves
        // drift apart by themselves, lose 2 %).
        auto values = [&](int b, const f16x8 (&pf)[4], int up) {
            __builtin_amdgcn_sched_barrier(0);
            uint32_t from = v_row + b * D * 8;
            asm volatile("" : "+v"(from));
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int e = 0; e < ET; ++e)
                    o[e] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vbuf[(from ^ (2 * s)) + 32 * e * 8], pf[s], o[e], 0, 0, 0);
            if constexpr (PAIR) {
                constexpr int kAhead = 6, N = 4 * ET, kEach = 24 * PER / N, kStore = N / (2 * PER);
                stage(b ^ 1, b ^ 1, up);
                __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    if (i < N - kAhead) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, kEach, 0);
                    if (i % kStore == kStore - 1) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            } else {
                pipelined(std::integral_constant<int, 4 * ET>{});
            }
        };
        float fm = 0.f, base = 0.f;              // p = e^(sc fm - base)
        bool begun = false;                      // every column of the wave has a reference
        // Masks the page's scores, moves the reference if it has to, settles fm and base.
        auto ready = [&](int32_t p, f32x16 (&sc)[ST]) {
            const int32_t t0 = p * kPage;
            bool any = true;
            if (p < full_lo || p >= full_hi) {
                const int from = max(see_lo - t0, 0), to = w.row < 0 ? 0 : min(w.pos + 1 - t0, kPage);
                any = from < to;
#pragma unroll
                for (int t = 0; t < ST; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int k = 32 * (t + part) + 16 * (i >> 3) + 8 * half + (i & 7);
                        sc[t][i] = k >= from && k < to ? sc[t][i] * fm : -__builtin_inff();
                    }
                fm = 1.f;
            }
            float mt = -__builtin_inff();
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) mt = fmaxf(mt, sc[t][i]);
            mt = max_halves(mt) * fm;
            if constexpr (PAIR) {
                if (half == 0) mbuf[(2 * group + part) * 32 + col] = mt;
                __syncthreads();
                mt = fmaxf(mt, mbuf[(2 * group + (part ^ 1)) * 32 + col]);
            }
            // (of a page that shows only NaN the reference is 0)
            const float ref = mt > -__builtin_inff() ? mt : (any && m_run == -__builtin_inff() ? 0.f : m_run);
            if (__any(any && !(ref - m_run <= kMoveAt))) {
                const float m_new = any && !(ref - m_run <= kMoveAt) ? ref : m_run;
                const float keep = m_run == m_new ? 1.f : __builtin_amdgcn_exp2f(m_run - m_new);
                l_run *= keep;
                m_run = m_new;
#pragma unroll
                for (int e = 0; e < ET; ++e)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[e][i] *= keep;
            }
            // (a column that has seen nothing yet: e^-inf, not inf - inf)
            base = (m_run > -__builtin_inff() ? m_run : 0.f) - kPBias;
            // (a page that all see has given every column one)
            if constexpr (PAIR) begun |= p >= full_lo && p < full_hi;
            else begun = __all(m_run > -__builtin_inff());
            if (any && __builtin_amdgcn_readlane(exps, p - at) == kNan) l_run = __builtin_nanf("");
        };
        // The probabilities, and this lane's sum of them.
        auto weights = [&](const f32x16 (&sc)[ST], f16x8 (&pf)[2 * ST]) {
            float l[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float x = __builtin_amdgcn_exp2f(fmaf(sc[t][i], fm, -base));
                    const float y = __builtin_amdgcn_exp2f(fmaf(sc[t][i + 1], fm, -base));
                    const f16x2 h = {static_cast<_Float16>(x), static_cast<_Float16>(y)};
                    const f16x2 one = {static_cast<_Float16>(1.f), static_cast<_Float16>(1.f)};
                    l[(i >> 1) & 3] = __builtin_amdgcn_fdot2(h, one, l[(i >> 1) & 3], false);
                    pf[2 * t + (i >> 3)][i & 7] = h[0];
                    pf[2 * t + (i >> 3)][(i & 7) + 1] = h[1];
                }
            return (l[0] + l[1]) + (l[2] + l[3]);
        };
        // In the middle of a sequence the maximum is not even sought: relative
        // to the reference so far the probabilities either keep their sum
        // below 2^15 (so each is at most 2^12 times that of the reference), or
        // the page is done again with its maximum.
        auto weigh = [&](int32_t p, f32x16 (&sc)[ST], f16x8 (&pf)[2 * ST]) {
            fm = q_log2 * read_lane(kss, p - at);
            const bool plain = begun && p >= full_lo && p < full_hi && __builtin_amdgcn_readlane(exps, p - at) != kNan;
            if (plain) {
                const float l = weights(sc, pf);
                if constexpr (PAIR) {
                    if (!__all(l < 32768.f) && lane == 0) again[p & 1] = 1;
#pragma unroll
                    for (int s = 0; s < 2; ++s) pbuf[(4 * group + 2 * part + s) * 64 + lane] = pf[s];
                    __syncthreads();
                    if (again[p & 1] == 0) {
                        l_run += l;
                        return;
                    }
                } else if (__all(l < 32768.f)) {
                    l_run += l;
                    return;
                }
            }
            ready(p, sc);
            l_run += weights(sc, pf);
            if constexpr (PAIR) {
#pragma unroll
                for (int s = 0; s < 2; ++s) pbuf[(4 * group + 2 * part + s) * 64 + lane] = pf[s];
                __syncthreads();
            }
        };

        auto follow = [&]() {                    // outputs so far in the unit of the page staged
            if (unit == want) return;
            const float f = ldexpf(1.f, unit - want);   // (kNone: they are 0)
            unit = want;
#pragma unroll
            for (int e = 0; e < ET; ++e)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[e][i] *= f;
        };

        if (p0 < p1) {
            look(p0);
            fetch(p0, p0);
            int up = settle(p0);
            stage(0, 0, up);
            if (PAIR && tid < 2) again[tid] = 0;
            __syncthreads();
            for (int32_t p = p0; p < p1; ++p) {
                const int b = (p - p0) & 1;
                if (p + 2 - at > 64) look(p);
                fetch(p + 1, p + 1);
                follow();
                if (seen(p)) {
                    f32x16 sc[ST];
                    scores(b, sc);
                    f16x8 pf[4];
                    if constexpr (PAIR) {
                        f16x8 mine[2];
                        weigh(p, sc, mine);
#pragma unroll
                        for (int s = 0; s < 4; ++s) pf[s] = pbuf[(4 * group + s) * 64 + lane];
                        if (tid == 0) again[(p + 1) & 1] = 0;
                        up = settle(p + 1);
                    } else {
                        weigh(p, sc, pf);
                    }
                    values(b, pf, up);
                }
                if (!PAIR || !seen(p)) {
                    up = settle(p + 1);
                    stage(b ^ 1, b ^ 1, up);
                }
                __syncthreads();
            }
        }

        // Outputs: a lane has, for its column, four dims at a time.
        float l = l_run + xor_lane(l_run, 32);
        if constexpr (PAIR) {
            __syncthreads();                     // (also: the buffers may be filled for the next tile)
            if (half == 0) mbuf[(2 * group + part) * 32 + col] = l;
            __syncthreads();
            l = mbuf[2 * group * 32 + col] + mbuf[(2 * group + 1) * 32 + col];
        }
        if (w.row >= 0) {
            const uint64_t row_at = static_cast<uint64_t>(w.row) * a.heads + w.head;
            const float v_scale = unit == kNone ? 0.f : ldexpf(1.f, unit);
            if (a.pieces == 1) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int e = 0; e < ET; ++e)
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                        bf16x4 x;
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = static_cast<__bf16>((o[e][i + k] * inv) * v_scale);
                        *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(a.out) + row_at * D + 32 * (ET * part + e) + 2 * i + 4 * half) = x;
                    }
            } else {
                const uint64_t slot = static_cast<uint64_t>(piece) * a.s.rows * a.heads + row_at;
                if (p0 < p1) {
#pragma unroll
                    for (int e = 0; e < ET; ++e)
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            *reinterpret_cast<float4*>(a.part + slot * D + 32 * (ET * part + e) + 2 * i + 4 * half) =
                                make_float4(o[e][i] * v_scale, o[e][i + 1] * v_scale, o[e][i + 2] * v_scale, o[e][i + 3] * v_scale);
                }
                if (half == 0 && part == 0) a.stat[slot] = make_float2(m_run, l);
            }
        }
    }
}

// Joins the pieces of each column: lane z has piece z's maximum and sum (at
// most 64 pieces), and the pieces' outputs are added in their order, D / 64
// values a lane, eight pieces to a trip to memory.  A wave has a column, or,
// SPLIT, a workgroup has one and its waves a quarter of the pieces each.
// Pieces from which on a workgroup has one column (one sequence of 32000
// tokens, 4 heads of 256, both kernels: 36 us with a wave a column, 25 so; 8000
// of 8 heads of 128 12.9 and 11.8; with fewer pieces no difference).
constexpr uint32_t kSplitJoin = 9;

template <uint32_t DT, int D, bool SPLIT>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
    constexpr int V = D / 64;
    __shared__ float quarter[4][D];
    const uint32_t seq = blockIdx.x / a.c.kv_heads, kvh = blockIdx.x % a.c.kv_heads;
    const int lane = threadIdx.x & 63;
    const uint32_t wave = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)));
    const SeqRows r = seq_rows(a.s, seq);
    const uint32_t n = static_cast<uint32_t>(r.count) * a.group;
    const uint64_t step = static_cast<uint64_t>(a.s.rows) * a.heads;
    const uint32_t each = SPLIT ? (a.pieces + 3) / 4 : a.pieces;
    const uint32_t from = SPLIT ? wave * each : 0, to = min(from + each, a.pieces);
    for (uint32_t gc = SPLIT ? blockIdx.y : blockIdx.y * 4 + wave; gc < n; gc += SPLIT ? gridDim.y : gridDim.y * 4) {
        const uint64_t at = static_cast<uint64_t>(r.first + static_cast<int32_t>(gc / a.group)) * a.heads + kvh * a.group + gc % a.group;
        float2 st = make_float2(-__builtin_inff(), 0.f);
        if (static_cast<uint32_t>(lane) < a.pieces) st = a.stat[lane * step + at];
        float m = st.x;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, xor_lane(m, k));
        // pieces that saw nothing have the maximum -infinity and the sum 0
        const float f = st.x == m ? 1.f : __builtin_amdgcn_exp2f(st.x - m);
        float l = f * st.y;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) l += xor_lane(l, k);
        const uint64_t used = __ballot(st.y != 0.f);
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
        const float* pp = a.part + at * D + lane * V;
        for (uint32_t z = from; z < to; z += 8) {
            float x[8][V];
            const uint64_t take = used >> z & ((1ull << min(to - z, 8u)) - 1);
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    x[u][i] = (take >> u & 1) != 0 ? pp[(z + u) * step * D + i] : 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float g = read_lane(f, (z + u) & 63);
                if ((take >> u & 1) != 0) {
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = fmaf(g, x[u][i], v[i]);
                }
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        auto store = [&](int dim, float res) {
            if constexpr (DT == QMV_F32) static_cast<float*>(a.out)[at * D + dim] = res;
            else static_cast<__bf16*>(a.out)[at * D + dim] = static_cast<__bf16>(res);
        };
        if constexpr (SPLIT) {
#pragma unroll
            for (int i = 0; i < V; ++i) quarter[wave][lane * V + i] = v[i];
            __syncthreads();
            const int dim = threadIdx.x;
            if (dim < D) store(dim, ((quarter[0][dim] + quarter[1][dim]) + (quarter[2][dim] + quarter[3][dim])) * inv);
            __syncthreads();
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) store(lane * V + i, v[i] * inv);
        }
    }
}

// Enqueues the join of up to `columns` columns a sequence and head, where there are pieces to join.
template <uint32_t DT, int D>
hipError_t join(const AttendArgs& a, uint32_t columns, hipStream_t s) {
    const uint32_t x = a.s.seqs * a.c.kv_heads;
    if (a.pieces >= kSplitJoin)
        hipLaunchKernelGGL((attend_join_kernel<DT, D, true>), dim3(x, columns < 65535 ? columns : 65535), dim3(256), 0, s, a);
    else if (a.pieces > 1)
        hipLaunchKernelGGL((attend_join_kernel<DT, D, false>), dim3(x, columns / 4 < 65535 ? (columns + 3) / 4 : 65535), dim3(256), 0, s, a);
    return hipGetLastError();
}

// The launch: tiles of 16 columns of a sequence and head, and pieces of its
// pages, so that every compute unit has a workgroup, with at least one page
// for each wave of a piece.  (One workgroup of four waves a compute unit: 2 x
// 131072 tokens 63 us, two 69, four 75; 32 x 4000 38, 40 and 43.  Two pages a
// wave at least: one sequence of 4000 tokens with 8 heads of 128 11.2 us, with 4
// of 256 17.6; one: 9.9 and 14.4.)  Short sequences stay whole, as a second
// kernel costs as much as their pages one after another, and its launch a call
// more on the host (one sequence, whole / in pieces, us in a graph: 500 tokens
// of 8 heads of 128 8.0 / 9.3, 900 10.2 / 9.5, 1000 10.5 / 9.7; of 2 heads of 64
// 1000 6.8 / 7.5, 1400 8.2 / 7.6; of 4 heads of 256 500 13.0 / 13.3, 550 14.6 /
// 13.8: the limits lie where the second launch is worth what it saves).
struct Plan {
    uint32_t tiles, pieces, per;
    Few few;
};
// Each wave has its own columns where there are waves enough that way: tiles of
// 16 columns for every SIMD (two for head dims of 64), or for few pages a tile
// fewer, kSoloPage / D a page.  A wave then makes its queries' digits once, not
// four waves the same ones, and nothing is joined.  Measured with float32 (us,
// waves share the pages / each its own), sequences x new of tokens:
//   D 128, 8 heads: 1 x 8192 of 8192 1517 / 1392, 8 x 300 of 300 72 / 29, 64 x 8
//     of 1000 38 / 35; 1 head a query head: 1 x 1000 of 1000 (504 tiles) 18 / 26
//   D 256, 4 heads: 8 x 300 of 300 148 / 42, 1 x 300 of 300 (300 tiles) 33 / 22,
//     64 x 8 of 8000 (512 tiles) 258 / 348
//   D 64, 8 heads: 8 x 300 of 300 37 / 16, 64 x 8 of 1000 (1024 tiles) 22 / 26
constexpr uint64_t kSoloPage = 8192;
Plan plan_few(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t heads, uint32_t window) {
    const uint64_t group = heads / c.kv_heads;
    const uint64_t most = s.max_new < s.rows ? (s.max_new == 0 ? 1 : s.max_new) : s.rows;
    Few mode = most * group <= 4 ? kPack : kWide;
    const uint64_t tiles16 = uint64_t{s.seqs} * c.kv_heads * ((most * group + 15) / 16);
    if (mode == kWide && (tiles16 >= (c.head_dim == 64 ? 2048u : 1024u) ||
                          tiles16 * c.head_dim >= kSoloPage * span_pages(s, window, 16)))
        mode = kSolo;
    const uint32_t kCols = few_cols(mode);
    uint64_t tiles = (most * group + kCols - 1) / kCols;
    if (tiles > 8192) tiles = 8192;
    const uint64_t pages = span_pages(s, window, kCols);
    const uint64_t wgs = uint64_t{s.seqs} * c.kv_heads * tiles;
    uint64_t pieces = (kTarget + wgs - 1) / wgs;
    if (pieces > (pages + 3) / 4) pieces = (pages + 3) / 4;
    if (pages <= (c.head_dim == 64 ? 24u : (c.head_dim == 128 ? 17u : 10u))) pieces = 1;
    if (pieces > 64) pieces = 64;
    if (pieces < 1 || mode == kSolo) pieces = 1;
    return Plan{static_cast<uint32_t>(tiles), static_cast<uint32_t>(pieces),
                static_cast<uint32_t>((pages + pieces - 1) / pieces), mode};
}

// bfloat16 queries go to the kernel for many where a sequence has columns
// enough to be worth tiles of 256 (kManyCols / D; at less the matrix cores
// multiply zeros) and the launch has work enough that its waves do not wait
// for each page by themselves: kManyWork, in products of 16 columns with a
// page, times D.  Measured (us, many / few), sequences x tokens, columns:
//   D 128, 8 heads: 1 x 2000, 256: 32 / 16; 1 x 16000, 128 and 256: 31 / 34 and
//     43 / 58; 8 x 3000, 128 and 256: 34 / 41 and 47 / 68; 64 x 1000, 128 and 256:
//     61 / 79 and 90 / 132; whole prompts 2 x 500 27 / 24, 1 x 2000 79 / 114
//   D 256, 4 heads: 1 x 16000, 64, 128 and 256: 38 / 27, 44 / 39 and 50 / 60; 8 x
//     3000, 128: 44 / 43; 64 x 1000, 64 and 128: 50 / 51 and 55 / 91
//   D 64, 8 heads: 8 x 3000, 256 and 512: 36 / 37 and 61 / 72; 64 x 1000, 256 and
//     512: 68 / 71 and 119 / 120; whole prompts 1 x 1000 36 / 24, 1 x 4000 135 / 189
// The faster one is taken at each of these but one, D 256, 1 x 16000 with 128
// columns (44 for 39), just past the limit, and one more is even (8 x 3000).
constexpr uint64_t kManyCols = 16384;
constexpr double kManyWork = 2e6;

bool is_many(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype, uint32_t heads, uint32_t window) {
    const uint64_t most = s.max_new < s.rows ? s.max_new : s.rows, cols = most * (heads / c.kv_heads);
    if (dtype != QMV_BF16 || cols * c.head_dim < kManyCols) return false;
    const double products = static_cast<double>(uint64_t{s.seqs} * c.kv_heads) * static_cast<double>((cols + 15) / 16);
    qmv_kv_seqs mean = s;   // the middle row's tokens
    mean.max_len -= static_cast<uint32_t>(most / 2 < s.max_len ? most / 2 : s.max_len);
    return products * static_cast<double>(span_pages(mean, window, 16)) * c.head_dim >= kManyWork;
}

Plan plan_many(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t heads, uint32_t window, uint32_t cols) {
    const uint64_t group = heads / c.kv_heads;
    const uint64_t most = s.max_new < s.rows ? s.max_new : s.rows;
    uint64_t tiles = (most * group + cols - 1) / cols;
    if (tiles > 65535) tiles = 65535;
    if (tiles < 1) tiles = 1;
    const uint64_t pages = span_pages(s, window, cols);
    const uint64_t wgs = uint64_t{s.seqs} * c.kv_heads * tiles;
    uint64_t pieces = 256 / wgs;
    if (pieces > pages / 8) pieces = pages / 8;
    if (pieces > 64) pieces = 64;
    if (pieces < 1) pieces = 1;
    return Plan{static_cast<uint32_t>(tiles), static_cast<uint32_t>(pieces),
                static_cast<uint32_t>((pages + pieces - 1) / pieces), kWide};
}

template <int D>
hipError_t go_many(const AttendArgs& a, const Plan& p, hipStream_t s) {
    const dim3 grid(a.s.seqs * a.c.kv_heads, p.tiles, p.pieces), block(512);
    // keys and values, f16, twice; of pairs also probabilities, maxima, flags
    constexpr uint32_t bytes = 2 * 2 * kPage * D * 2 + (D == 256 ? 4 * 4 * 64 * 16 + 4 * 2 * 32 * 4 + 16 : 0);
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(attend_many_kernel<D>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((attend_many_kernel<D>), grid, block, bytes, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : join<QMV_BF16, D>(a, p.tiles * many_cols(D), s);
}

template <uint32_t DT, int D>
hipError_t go_few(const AttendArgs& a, const Plan& p, hipStream_t s) {
    const dim3 grid(a.s.seqs * a.c.kv_heads, p.tiles, p.pieces), block(256);
    if (p.few == kPack) hipLaunchKernelGGL((attend_few_kernel<DT, D, kPack>), grid, block, 0, s, a);
    else if (p.few == kSolo) hipLaunchKernelGGL((attend_few_kernel<DT, D, kSolo>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attend_few_kernel<DT, D, kWide>), grid, block, 0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : join<DT, D>(a, p.tiles * few_cols(p.few), s);
}

Plan plan_of(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype, uint32_t heads, uint32_t window) {
    return is_many(c, s, dtype, heads, window) ? plan_many(c, s, heads, window, many_cols(static_cast<int>(c.head_dim))) : plan_few(c, s, heads, window);
}

}  // namespace

uint64_t kv_attend_workspace_bytes(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype, uint32_t heads,
                                   uint32_t window) {
    const Plan p = plan_of(c, s, dtype, heads, window);
    if (p.pieces == 1) return 0;
    return uint64_t{p.pieces} * s.rows * heads * (c.head_dim + 2) * 4;  // outputs, then statistics
}

hipError_t launch_kv_attend(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype, uint32_t heads,
                            float scale, uint32_t window, const void* q, void* out, void* workspace,
                            hipStream_t stream) {
    const Plan p = plan_of(c, s, dtype, heads, window);
    float* part = static_cast<float*>(workspace);
    const uint64_t outputs = uint64_t{p.pieces} * s.rows * heads * c.head_dim;
    const AttendArgs a{c, s, q, out, part, reinterpret_cast<float2*>(part + outputs), scale * kLog2e, heads,
                       heads / c.kv_heads, window, p.pieces, p.per};
    if (is_many(c, s, dtype, heads, window)) {
        if (c.head_dim == 64) return go_many<64>(a, p, stream);
        if (c.head_dim == 128) return go_many<128>(a, p, stream);
        return go_many<256>(a, p, stream);
    }
    if (dtype == QMV_F32) {
        if (c.head_dim == 64) return go_few<QMV_F32, 64>(a, p, stream);
        if (c.head_dim == 128) return go_few<QMV_F32, 128>(a, p, stream);
        return go_few<QMV_F32, 256>(a, p, stream);
    }
    if (c.head_dim == 64) return go_few<QMV_BF16, 64>(a, p, stream);
    if (c.head_dim == 128) return go_few<QMV_BF16, 128>(a, p, stream);
    return go_few<QMV_BF16, 256>(a, p, stream);
}

}  // namespace qmv
