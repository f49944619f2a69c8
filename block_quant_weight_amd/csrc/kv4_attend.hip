// Attention over the 4-bit cache.
//
// For a query row q at position p: s_j = scale q.k_j, out = sum_j e^{s_j} v_j
// / sum_j e^{s_j} over the positions j it sees.
//
// A stored key or value is exact in bfloat16, and one instruction makes two of
// them from their codes and their block's scale.  Both products run on the
// bfloat16 matrix cores with float32 sums; the other operand is split so that
// nothing that counts is rounded: float32 queries and probabilities into three
// bfloat16 parts (24 bits, exact), bfloat16 queries are one part, and their
// probabilities two (16 bits, where the output keeps 8; cut off, while their sum
// is of the whole ones: an output is up to 2^-16 of itself nearer to 0, 1/128 of
// its rounding).
//
// Layout: v_mfma_f32_16x16x32_bf16 takes from lane l eight k-indexes of row (or
// column) l % 16, those of group l / 16, and gives lane l, register i the
// output of row 4 (l / 16) + i and column l % 16.  The order of the k-indexes is
// free as long as both operands agree, so
//   keys: lane (t, g) has a quarter of token t's channels, from one load;
//   scores: rows are tokens, so lane (column, g) gets those of the tokens 16 T +
//     4 g + i, and these are the k-indexes that the output's product takes from
//     it: probabilities stay in the lane that computed them;
//   values: lane (c, g) has channel sixteenth c of the same tokens (the order
//     in which they lie in the cache), and row r of the m-th product is channel
//     (D / 16) r + m.
// Neither operand goes through shared memory.
//
// Work: a workgroup of four waves has 16 columns (query row x head of one
// key/value head) and a piece of the sequence's pages; each wave takes every
// fourth page and keeps its own running maximum, sum and output, joined in
// shared memory at the end.  Where columns are few (PACKED), the parts of a
// query and of a probability are columns of their own; where there are enough,
// each wave has 16 and all of their pages (SOLO).
//
// Bound by memory for long contexts: 2 x 131072 bfloat16 (32 heads on 8 of 128,
// 180 MB) 42.4 us, of which the join 5, the kernel 4.8 TB/s.  A decode step of 32
// x 1000 to 4000 in float32 (91 MB) 30.1 us: vector instructions are issued in
// half of the cycles (conversion, exponentials, parts), the rest is the first
// trips to memory, uneven ends and the join (two pages on the way instead of
// one: 35; nothing fetched behind a wave's last page: 31).
#include "kv4_common.h"

namespace qmv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// The running reference moves when a maximum is further above it: e^s stays
// below 2^8 times the reference's.
constexpr float kMoveAt = 8.f;
// How a call is dealt out: few queries to a key/value head, the waves of a
// workgroup sharing the pages (packed: a tile's columns few enough that each
// part of a probability has a column of its own, so one product takes what two
// or three took: 32 x 4000 float32 31.4 us, else 34.1) or each with its own
// columns; or many.
enum Kind { kShared, kPacked, kSolo, kMany };
template <uint32_t DT>
constexpr uint32_t kPackedCols = DT == QMV_F32 ? 4 : 8;
constexpr uint32_t kMaxPieces = 64;    // of a sequence
constexpr uint32_t kScanSeqs = 1024;   // sequences up to which pieces are made

struct Attend4Args {
    qmv_kv4_cache c;
    qmv_kv_seqs s;
    const void* q;
    void* out;
    float* part;          // [room][kv_heads * group][D]: output sums of pieces
    float2* stat;         // [room][kv_heads * group]: maximum, sum
    float scale_log2;     // |scale| * log2(e) (1 where the scale is 0)
    float move;           // what kMoveAt is of a product with a key
    uint32_t keep, flip;  // bits of a query that the scale leaves, and turns
    uint32_t heads, group, window;
    uint32_t target;      // pieces of all sequences that the launch aims at; 0: sequences stay whole
    uint32_t least;       // pages of a piece, at least
    uint32_t room;        // rows of pieces that the workspace holds
};

// Positions that a table has room for.
__device__ __forceinline__ int32_t room_of(const qmv_kv_seqs& s) {
    return static_cast<int32_t>(min(s.table_stride, 0x7FFF0000u / kPage) * kPage);
}

// Pages [lo, hi) that any row of a sequence sees.
struct Span {
    int32_t lo, hi;
};
__device__ __forceinline__ Span span_of(const Attend4Args& a, const SeqRows& r) {
    const int32_t hi = min(r.base + r.count, room_of(a.s));
    Span o;
    o.lo = sees_from(a.window, max(r.base, 0)) / kPage;
    o.hi = max((max(hi, 0) + kPage - 1) / kPage, o.lo);
    return o;
}

// How sequences are cut into pieces, the same in every wave that asks: the
// pages of all are dealt out in `target` pieces of about one size, so a long
// sequence beside short ones has more of them.  A sequence that is not whole
// keeps its pieces' sums in the workspace's rows from `first` on, piece by
// piece, its query rows one after another.
struct Piece {
    int32_t seq;                 // -1: none
    uint32_t piece, pieces;
    uint32_t first;
};
// Piece `slot` in the order of the sequences; with by_seq, piece 0 of sequence
// `slot`.  All lanes of a wave call it together.
__device__ __forceinline__ Piece find_piece(const Attend4Args& a, uint32_t slot, bool by_seq) {
    const uint32_t seqs = a.s.seqs, lane = threadIdx.x & 63;
    if (a.target == 0) return Piece{slot < seqs ? static_cast<int32_t>(slot) : -1, 0, 1, 0};
    auto look = [&](uint32_t i, uint32_t* count) {
        uint32_t pages = 0;
        *count = 0;
        if (i < seqs) {
            const SeqRows r = seq_rows(a.s, i);
            const Span sp = span_of(a, r);
            *count = static_cast<uint32_t>(r.count);
            pages = r.count > 0 ? static_cast<uint32_t>(sp.hi - sp.lo) : 0u;
        }
        return pages;
    };
    uint32_t count, mine = look(lane, &count), total = mine, most = mine;
    for (uint32_t b = 64; b < seqs; b += 64) {
        uint32_t n;
        const uint32_t p = look(b + lane, &n);
        total += p;                              // (at most 16 of 2^25 pages a lane)
        most = max(most, p);
    }
    // (2^10 sequences of 2^25 pages: their sum is held in 64 bits)
    uint64_t sum = total;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t lo = static_cast<uint32_t>(sum), hi = static_cast<uint32_t>(sum >> 32);
        sum += static_cast<uint32_t>(__shfl_xor(static_cast<int>(lo), m)) |
               static_cast<uint64_t>(static_cast<uint32_t>(__shfl_xor(static_cast<int>(hi), m))) << 32;
        most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), m)));
    }
    const uint32_t per = max(max(static_cast<uint32_t>((sum + a.target - 1) / a.target), a.least), (most + kMaxPieces - 1) / kMaxPieces);
    uint32_t before = 0, kept = 0;               // pieces, and rows of the workspace, of the sequences before
    for (uint32_t b = 0; b < seqs; b += 64) {
        if (b > 0) mine = look(b + lane, &count);
        uint32_t n = count > 0 ? max((mine + per - 1) / per, 1u) : 0u;
        // (a sequence whose sums would not fit stays whole: rows below 2^31, pieces 64 at most)
        uint64_t rows = n > 1 ? static_cast<uint64_t>(n) * count : 0u;
        uint32_t need = rows > a.room ? a.room + 1 : static_cast<uint32_t>(rows);
        uint32_t at = need, upto = n;
        // inclusive sums over the lanes before (rows held to room + 1 and at most 2^31: no overflow in 64 bits)
        uint64_t acc = need;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const uint32_t lo = static_cast<uint32_t>(__shfl_up(static_cast<int>(static_cast<uint32_t>(acc)), m));
            const uint32_t hi = static_cast<uint32_t>(__shfl_up(static_cast<int>(static_cast<uint32_t>(acc >> 32)), m));
            if (lane >= static_cast<uint32_t>(m)) acc += lo | static_cast<uint64_t>(hi) << 32;
        }
        if (kept + acc > a.room) {               // from the first that does not fit on
            if (n > 1) n = 1;
            upto = n;
        }
        at = static_cast<uint32_t>(min(kept + acc - need, static_cast<uint64_t>(a.room)));
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const uint32_t u = static_cast<uint32_t>(__shfl_up(static_cast<int>(upto), m));
            if (lane >= static_cast<uint32_t>(m)) upto += u;
        }
        const uint32_t start = before + upto - n;
        const bool hit = by_seq ? b + lane == slot : (n > 0 && slot >= start && slot - start < n);
        const uint64_t who = __ballot(hit);
        if (who != 0) {
            const int l = __builtin_ctzll(who);
            Piece o;
            o.seq = static_cast<int32_t>(b) + l;
            o.pieces = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(n), l));
            o.piece = by_seq ? 0u : slot - static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(start), l));
            o.first = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(at), l));
            return o;
        }
        before += static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(upto), 63));
        const uint64_t end = kept + (static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(acc >> 32)), 63))) << 32 |
                                     static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(acc)), 63)));
        kept = end > a.room ? a.room + 1 : static_cast<uint32_t>(end);
    }
    return Piece{-1, 0, 1, 0};
}

// What a tile of columns is.  Columns of a sequence and key/value head (rows *
// group, below 2^31) are numbered row first.
struct Columns {
    int32_t row;                 // this lane's query row in its sequence, -1: none
    int32_t pos;                 // its position
    uint32_t head;
    int32_t first_pos, last_pos; // smallest and largest position of the columns
    int32_t lo, hi;              // positions that any of the columns sees: [lo, hi)
};
template <uint32_t COLS>
__device__ __forceinline__ Columns columns(const Attend4Args& a, const SeqRows& r, uint32_t kvh, uint32_t tile, uint32_t col) {
    Columns o;
    const uint32_t n = static_cast<uint32_t>(r.count) * a.group, c = tile * COLS + col;
    const uint32_t t = c / a.group;
    o.row = c < n ? static_cast<int32_t>(t) : -1;
    o.pos = r.base + static_cast<int32_t>(t);
    o.head = kvh * a.group + (c - t * a.group);
    o.first_pos = r.base + static_cast<int32_t>(tile * COLS / a.group);
    o.last_pos = r.base + static_cast<int32_t>(min(tile * COLS + COLS - 1, n - 1) / a.group);
    o.hi = min(max(o.last_pos + 1, 0), room_of(a.s));
    o.lo = sees_from(a.window, max(o.first_pos, 0));
    return o;
}

// A float32 as N bfloat16 parts, the largest first (each cut off, so that the
// next is exact; of three the sum is the number itself).
template <int N>
__device__ __forceinline__ void split(float x, uint32_t part[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x);
        part[i] = b;                             // (the upper half is taken)
        x -= __builtin_bit_cast(float, b & 0xFFFF0000u);
    }
}
// Upper halves of two words, as a pair.
__device__ __forceinline__ uint32_t uppers(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }
__device__ __forceinline__ uint32_t lowers(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x05040100u); }

template <uint32_t DT, int D, int KIND>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void attend4_few_kernel(Attend4Args a) {
    typedef typename Elem<DT>::type T;
    constexpr bool SOLO = KIND == kSolo, PACKED = KIND == kPacked;
    constexpr int STEP = SOLO ? 1 : 4;            // waves that share the pages
    constexpr int PARTS = DT == QMV_F32 ? 3 : 2;  // of a probability
    constexpr uint32_t kCols = PACKED ? kPackedCols<DT> : 16;   // columns of a tile
    constexpr int NQ = DT == QMV_F32 && !PACKED ? 3 : 1;        // operands made of a query
    constexpr int NP = PACKED ? 1 : PARTS;                      // and of a probability
    constexpr int KS = D / 32;                    // k-steps of a score tile
    constexpr int W = D / 32;                     // words of a lane's quarter of a key, and of its four tokens' values
    constexpr int E = D / 16;                     // channels of a sixteenth, and tiles of the output
    __shared__ float acc[SOLO ? 1 : 4][SOLO ? 1 : 16][SOLO ? 1 : D + 1];
    __shared__ float stat[SOLO ? 1 : 4][16][2];
    const int lane = threadIdx.x & 63, quad = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t kvh = blockIdx.x % a.c.kv_heads;
    const Piece w0 = find_piece(a, blockIdx.x / a.c.kv_heads, false);
    if (w0.seq < 0) return;
    const uint32_t seq = static_cast<uint32_t>(w0.seq);
    const SeqRows r = seq_rows(a.s, seq);
    const uint32_t all = static_cast<uint32_t>(r.count) * a.group;
    const uint32_t tiles = (all + kCols - 1) / kCols;
    const uint32_t own = col / kCols;             // (packed: the part that the lane has)
    const Span sp = span_of(a, r);
    const int32_t per = (sp.hi - sp.lo + static_cast<int32_t>(w0.pieces) - 1) / static_cast<int32_t>(w0.pieces);
    const int32_t b0 = min(sp.lo + static_cast<int32_t>(w0.piece) * per, sp.hi), b1 = min(b0 + per, sp.hi);
    constexpr uint32_t kOwn = SOLO ? 4 : 1;       // tiles of a workgroup
    // the last tiles see the most: they begin first
    for (uint32_t turn = kOwn * blockIdx.y + (SOLO ? wave : 0); turn < tiles; turn += kOwn * gridDim.y) {
        const uint32_t tile = tiles - 1 - turn;
        const Columns w = columns<kCols>(a, r, kvh, tile, col % kCols);
        const int32_t p0 = max(b0, w.lo / kPage), p1 = min(b1, (w.hi + kPage - 1) / kPage);
        const int32_t see_lo = sees_from(a.window, w.pos);
        // pages that every column sees whole: from full_lo up to full_hi
        const int32_t full_lo = (sees_from(a.window, w.last_pos) + kPage - 1) / kPage;
        const int32_t full_hi = max(w.first_pos + 1, 0) / kPage;

        // Lane i has the id of the wave's page number i from here; keys and
        // values of the next page are on the way while one is computed.
        int32_t ids = -1;
        auto look = [&](int32_t p) {
            const int32_t mine = p + STEP * lane;
            ids = mine < p1 ? page_id(a.c, a.s, seq, mine) : -1;
        };
        uint32_t kw[4][W], vw[4][W], ks[W > 4 ? 2 : 1], vs[4];
        int32_t id = -1;
        auto fetch_k = [&](int32_t at) {
            // (where there is no page, page 0, which every cache has, is read and not used)
            const uint64_t place = static_cast<uint64_t>(max(at, 0)) * a.c.kv_heads + kvh;
            const uint8_t* kp = a.c.k + place * kCodeBytes<D> + k_at<D>(col, quad * W);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < W; ++i) kw[t][i] = reinterpret_cast<const uint32_t*>(kp + 16 * t * (D / 2))[i];
            const uint8_t* sp = a.c.k_scale + place * kScaleBytes<D> + k_scale_at<D>(col, quad * W / 4);
            ks[0] = reinterpret_cast<const uint32_t*>(sp)[0];
            if constexpr (W > 4) ks[1] = reinterpret_cast<const uint32_t*>(sp)[1];
        };
        auto fetch_v = [&](int32_t at) {
            const uint64_t place = static_cast<uint64_t>(max(at, 0)) * a.c.kv_heads + kvh;
            const uint8_t* vp = a.c.v + place * kCodeBytes<D> + v_at<D>(4 * quad, E * col);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < W; ++i) vw[t][i] = reinterpret_cast<const uint32_t*>(vp + t * 16 * (D / 2))[i];
            const uint4 s = *reinterpret_cast<const uint4*>(a.c.v_scale + place * kScaleBytes<D> + v_scale_at<D>(4 * quad, E * col / kBlock));
            vs[0] = s.x; vs[1] = s.y; vs[2] = s.z; vs[3] = s.w;
        };
        look(p0 + (SOLO ? 0 : wave));
        // the query: lane (column, g) has the channels that lane (t, g) has of a key
        bf16x8 qf[KS][NQ];
        {
            const uint64_t row = static_cast<uint64_t>(r.first + max(w.row, 0));
            const T* qp = static_cast<const T*>(a.q) + (row * a.heads + w.head) * D + quad * (D / 4);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.f;
                if (w.row >= 0) load8<DT>(qp + 8 * s, x);
                uint32_t part[8][NQ];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // (+ 0 x: an infinite query, whose products need not all be NaN, is NaN, and with a scale of 0 one that is no number too)
                    const float y = fmaf(x[i], 0.f, __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x[i]) & a.keep) ^ a.flip));
                    if constexpr (PACKED && DT == QMV_F32) {
                        uint32_t of[3];
                        split<3>(y, of);
                        part[i][0] = own == 0 ? of[0] : (own == 1 ? of[1] : (own == 2 ? of[2] : 0u));
                    } else {
                        split<NQ>(y, part[i]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                    qf[s][n] = __builtin_bit_cast(bf16x8, make_uint4(uppers(part[0][n], part[1][n]), uppers(part[2][n], part[3][n]),
                                                                     uppers(part[4][n], part[5][n]), uppers(part[6][n], part[7][n])));
            }
        }
        int n = 0;
        id = __builtin_amdgcn_readlane(ids, 0);
        fetch_k(id);
        fetch_v(id);

        const uint32_t cut1 = own >= 1 ? 0xFFFF0000u : 0u, cut2 = own >= 2 ? 0xFFFF0000u : 0u;
        f32x4 o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
        // the largest product with a key so far, as far as the reference has
        // moved; it times the scale; the sum
        float m_run = -__builtin_inff(), base = 0.f, l_run = 0.f;

        for (int32_t p = p0 + (SOLO ? 0 : wave); p < p1; p += STEP) {
            const int32_t here = id;
            if (++n == 64) {
                look(p + STEP);
                n = 0;
            }
            id = __builtin_amdgcn_readlane(ids, n);
            const bool edge = p < full_lo || p >= full_hi;
            // scores
            f32x4 sc[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                sc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const uint32_t byte = ks[s / 4] >> (8 * t) & 0xFFu;
                    const bf16x8 k = values8(kw[t][s], scale_of(byte));
#pragma unroll
                    for (int i = NQ - 1; i >= 0; --i) sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, qf[s][i], sc[t], 0, 0, 0);
                }
            }
            fetch_k(id);
            if (here >= 0) {
                if constexpr (PACKED && DT == QMV_F32) {
                    // the sum of the parts' products, the same in all of them
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float u = sc[t][i] + dpp_mov<0x128>(sc[t][i]);   // lanes 8 apart in a row of 16
                            sc[t][i] = u + dpp_mov<0x124>(u);                      // 4 apart
                        }
                }
                if (edge) {
                    // scores of what a column does not see, and values that none does: the
                    // memory behind a sequence's end may hold anything
                    const int32_t t0 = p * kPage + 4 * quad;
                    const int32_t to = w.row < 0 ? 0 : w.pos + 1;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int32_t at = t0 + 16 * t + i;
                            sc[t][i] = at >= see_lo && at < to ? sc[t][i] : -__builtin_inff();
                            if (at < w.lo || at >= w.hi) {
                                vs[t] = (vs[t] & ~(0xFFu << (8 * i))) | 127u << (8 * i);
                                if constexpr (W == 2) vw[t][i / 2] &= i % 2 == 0 ? 0xFFFF0000u : 0xFFFFu;
                                else
#pragma unroll
                                    for (int u = 0; u < W / 4; ++u) vw[t][i * (W / 4) + u] = 0u;
                            }
                        }
                    }
                }
                float mt = -__builtin_inff();
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mt = fmaxf(mt, sc[t][i]);
                mt = max_quads(mt);
                if (__any(mt > m_run + a.move || (m_run == -__builtin_inff() && mt > m_run))) {
                    const float m_new = mt > m_run + a.move || m_run == -__builtin_inff() ? fmaxf(mt, m_run) : m_run;
                    // (a column that has seen nothing yet: e^-inf, not inf - inf)
                    const float base_new = m_new > -__builtin_inff() ? m_new * a.scale_log2 : 0.f;
                    const float keep = m_run > -__builtin_inff() ? __builtin_amdgcn_exp2f(base - base_new) : 1.f;
                    m_run = m_new;
                    base = base_new;
                    l_run *= keep;
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] *= keep;
                }
                uint32_t pp[4][4][NP];
                float l = 0.f;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = __builtin_amdgcn_exp2f(fmaf(sc[t][i], a.scale_log2, -base));
                        l += x;
                        if constexpr (PACKED) {
                            // what is left of x before the lane's part: its upper half is the part
                            float y = x - __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & cut1);
                            if constexpr (DT == QMV_F32) y -= __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, y) & cut2);
                            pp[t][i][0] = __builtin_bit_cast(uint32_t, y);
                        } else {
                            split<NP>(x, pp[t][i]);
                        }
                    }
                l_run += l;
                // outputs: two steps of 32 tokens
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    bf16x8 pf[NP];
#pragma unroll
                    for (int k = 0; k < NP; ++k)
                        pf[k] = __builtin_bit_cast(bf16x8, make_uint4(uppers(pp[2 * s][0][k], pp[2 * s][1][k]), uppers(pp[2 * s][2][k], pp[2 * s][3][k]),
                                                                      uppers(pp[2 * s + 1][0][k], pp[2 * s + 1][1][k]), uppers(pp[2 * s + 1][2][k], pp[2 * s + 1][3][k])));
#pragma unroll
                    for (int b = 0; b < E / 2; ++b) {      // a byte of a sixteenth: two channels
                        uint32_t x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int t = 2 * s + j / 4, i = j % 4, at = i * (E / 2) + b;
                            const float d = scale_of(vs[t] >> (8 * i) & 0xFFu);
                            const uint32_t u = vw[t][at / 4];
                            x[j] = at % 4 == 0 ? pair_bf16<0>(u, d) : (at % 4 == 1 ? pair_bf16<1>(u, d) : (at % 4 == 2 ? pair_bf16<2>(u, d) : pair_bf16<3>(u, d)));
                        }
                        const bf16x8 even = __builtin_bit_cast(bf16x8, make_uint4(lowers(x[0], x[1]), lowers(x[2], x[3]), lowers(x[4], x[5]), lowers(x[6], x[7])));
                        const bf16x8 odd = __builtin_bit_cast(bf16x8, make_uint4(uppers(x[0], x[1]), uppers(x[2], x[3]), uppers(x[4], x[5]), uppers(x[6], x[7])));
#pragma unroll
                        for (int k = NP - 1; k >= 0; --k) {
                            o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even, pf[k], o[2 * b], 0, 0, 0);
                            o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd, pf[k], o[2 * b + 1], 0, 0, 0);
                        }
                    }
                }
            }
            fetch_v(id);
        }
        l_run += __shfl_xor(l_run, 16);
        l_run += __shfl_xor(l_run, 32);

        // where a column's output goes: into `out`, or to the piece's row
        const uint64_t piece_row = w0.first + static_cast<uint64_t>(w0.piece) * static_cast<uint32_t>(r.count);
        if constexpr (SOLO) {
            if (w.row >= 0) {
                const float inv = m_run == -__builtin_inff() && l_run == 0.f ? 0.f : 1.f / l_run;
                T* op = static_cast<T*>(a.out) + (static_cast<uint64_t>(r.first + w.row) * a.heads + w.head) * D;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        const int ch = E * (4 * quad + i) + e;
                        if constexpr (DT == QMV_F32) {
                            *reinterpret_cast<float4*>(op + ch) = make_float4(o[e][i] * inv, o[e + 1][i] * inv, o[e + 2][i] * inv, o[e + 3][i] * inv);
                        } else {
                            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                            const bf16x4 v = {static_cast<__bf16>(o[e][i] * inv), static_cast<__bf16>(o[e + 1][i] * inv),
                                              static_cast<__bf16>(o[e + 2][i] * inv), static_cast<__bf16>(o[e + 3][i] * inv)};
                            *reinterpret_cast<bf16x4*>(op + ch) = v;
                        }
                    }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[wave][col][E * (4 * quad + i) + e] = o[e][i];
            if (quad == 0) {
                stat[wave][col][0] = m_run > -__builtin_inff() ? base : -__builtin_inff();
                stat[wave][col][1] = l_run;
            }
            __syncthreads();
            // thread: a column, and a sixteenth of its channels
            const int c = threadIdx.x >> 4, part = threadIdx.x & 15;
            const uint32_t at = tile * kCols + c;
            if (static_cast<uint32_t>(c) < kCols && at < all) {
                float m = stat[0][c][0];
#pragma unroll
                for (int k = 1; k < 4; ++k) m = fmaxf(m, stat[k][c][0]);
                float f[4], l = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // (waves that saw nothing have the maximum -infinity and the sum 0)
                    f[k] = stat[k][c][0] == m ? 1.f : __builtin_amdgcn_exp2f(stat[k][c][0] - m);
                    l = fmaf(f[k], stat[k][c][1], l);
                }
                const uint32_t row = at / a.group, head = kvh * a.group + at % a.group;
                // (nothing seen: 0; a sum of 0 past float32's range: no number)
                const float inv = w0.pieces > 1 ? 1.f : (m == -__builtin_inff() && l == 0.f ? 0.f : 1.f / l);
                const uint64_t slot = (piece_row + row) * a.heads + head;
                if (w0.pieces > 1 && part == 0) a.stat[slot] = make_float2(m, l);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int ch = part + 16 * e;
                    float v = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x = acc[k][c][ch];
                        if constexpr (PACKED) {
                            x = acc[k][c + (PARTS - 1) * kCols][ch];
#pragma unroll
                            for (int b = PARTS - 2; b >= 0; --b) x += acc[k][c + b * kCols][ch];
                        }
                        v = fmaf(f[k], x, v);
                    }
                    v *= inv;
                    if (w0.pieces > 1) {
                        a.part[slot * D + ch] = v;
                    } else {
                        const uint64_t to = (static_cast<uint64_t>(r.first + static_cast<int32_t>(row)) * a.heads + head) * D + ch;
                        if constexpr (DT == QMV_F32) static_cast<float*>(a.out)[to] = v;
                        else static_cast<__bf16*>(a.out)[to] = static_cast<__bf16>(v);
                    }
                }
            }
            __syncthreads();
        }
    }
}

// ---- many queries -----------------------------------------------------------

// Many bfloat16 queries to a key/value head: a workgroup of four waves has 32
// columns a wave, and walks the pages together.  Values are made float16 once
// for all, in shared memory; keys stay codes there, which each wave turns into
// bfloat16 on the way to its products: an operand read from shared memory feeds
// one product of 32 columns, and were both of 2 bytes a value, four waves' reads
// of a page (head dims of 128: 128 KB, 128 bytes a cycle) would take as long as
// their products at the matrix cores' full rate, 1024 cycles.  With keys as codes
// they take 640; at the rate that is reached shared memory is addressed in 26% of
// the cycles, and would be in 41%.
//
// v_mfma_f32_32x32x16 takes from lane l eight k-indexes of row (or column) l %
// 32, those of half l / 32, and gives lane l, register i the output of row 8 (i
// / 4) + 4 (l / 32) + i % 4 and column l % 32.  Keys: lane (row, h) reads the 32
// codes of block 2 B + h, the operands of four k-steps.  Tokens are the rows of
// the scores, and the output's k-index 16 s + 8 h + e is token 16 s + 8 (e / 4) +
// 4 h + e % 4 of a tile of 32, register 8 s + e of the lane that scored it:
// probabilities stay in their lane.  Row r of the values in shared memory is
// channel (D / 16) (r % 16) + r / 16.
//
// Scores are bfloat16 products, exact in both operands.  The output's are
// float16: probabilities keep 11 bits there (their sum is taken of the rounded
// ones), not 8.  They are 4 at a column's reference m, e^(s - m), which moves
// once a lane's sum of a page would pass 2^15: no maximum is sought in the
// middle of a sequence.  Down to 2^-16 of the reference they keep all their
// bits, and below 2^-27 they count as 0.  A page's values are times 2^-unit,
// with a unit 4 above its largest exponent that stays while pages' largest are
// within 10 below and 13 above it, so blocks down to 2^-13 of a page's largest
// are exact whatever came before.  Blocks of zeros (all that tokens which are no
// number have, too) carry the least exponent there is: they do not lower the
// unit.  Nor does it fall further than kFar below the highest so far: outputs
// are multiplied by what it falls, and a page's are below 2^32 (probabilities
// of a column sum to less than 2^16, values are below 2^16 units), those of 2^25
// pages below 2^57: 2^64 times that is a float32.
//
// Head dims of 256 hold too many registers for a wave of 32 columns: waves w
// and w + 4 have the same 32.  Each scores half of a page's tokens, they
// exchange maxima and probabilities through shared memory, and each adds up
// half of the output channels.
//
// A page's products and exponentials are laid out so that a tile of 32 tokens'
// products are beside the other's exponentials, and the next page's values are
// staged beside the last of them: one barrier a page.  Two workgroups share a
// compute unit (216 of 256 registers), so one's barrier is the other's work.
//
// A prompt of 8192 (32 heads on 8 of 128, 550 GFLOP) takes 561 to 576 us, 970
// TFLOP/s, 70% of what a large bfloat16 product reaches.  Vector instructions (the
// exponentials, and the codes' conversion, of keys in each wave) are issued in 58%
// of the cycles and the matrix cores busy in 41%: little of one lies beside the
// other, though nothing keeps them apart.
// (Waves that read pages from memory themselves, few kernel: 874; eight waves and
// three barriers: 721.)
template <int D>
struct Many {
    static constexpr bool kPair = D == 256;
    static constexpr int kThreads = kPair ? 512 : 256, kCols = 128;
    static constexpr int kKeys = kCodeBytes<D>, kValueRow = 2 * kPage, kValues = D * kValueRow;   // bytes of a page
    // (pairs: probabilities [4 column groups][4 k-steps][64 lanes], maxima [4][2 halves][32], two flags)
    static constexpr int kExchange = kPair ? 4 * 4 * 64 * 16 + 4 * 2 * 32 * 4 + 16 : 0;
    static constexpr int kBytes = 2 * (kKeys + kValues) + kExchange + 64;   // 64: the pages' largest exponents, of each wave
};
constexpr float kSumLimit = 0x1p15f;       // of a page's probabilities in a lane
constexpr float kBias = 2.f;               // log2 of a probability at the reference
constexpr float kMoveManyAt = 4.f;
constexpr int32_t kNoUnit = -1000, kFar = 64;

template <int D>
__global__ __launch_bounds__(Many<D>::kThreads, 2) void attend4_many_kernel(Attend4Args a) {
    typedef Many<D> M;
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    constexpr bool PAIR = M::kPair;
    constexpr int QS = D / 16;                    // k-steps of a score
    constexpr int KB = D / kBlock;                // blocks of a token
    constexpr int ET = D / (PAIR ? 64 : 32);      // tiles of output channels that a wave adds up
    // pieces of 16 bytes of codes: of keys (32 channels of a token), of values (four tokens, 128 / D sixteenths)
    constexpr int PIECES = kPage * D / 32, PER = PIECES > M::kThreads / 2 ? 1 : 0;   // PER: a thread has both
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    uint8_t* const v_lds = lds + 2 * M::kKeys;
    uint8_t* const p_lds = v_lds + 2 * M::kValues;                            // (pairs)
    float* const m_lds = reinterpret_cast<float*>(p_lds + (PAIR ? 4 * 4 * 64 * 16 : 0));
    uint32_t* const again = reinterpret_cast<uint32_t*>(m_lds + (PAIR ? 4 * 2 * 32 : 0));   // (pairs) [2]: the page's probabilities once more
    uint32_t* const most = reinterpret_cast<uint32_t*>(lds + M::kBytes - 64);   // [2][8 waves]
    const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = PAIR ? wave & 3 : wave, part = PAIR ? wave >> 2 : 0;
    const uint32_t kvh = blockIdx.x % a.c.kv_heads;
    const Piece w0 = find_piece(a, blockIdx.x / a.c.kv_heads, false);
    if (w0.seq < 0) return;
    const uint32_t seq = static_cast<uint32_t>(w0.seq);
    const SeqRows r = seq_rows(a.s, seq);
    const uint32_t all = static_cast<uint32_t>(r.count) * a.group;
    const uint32_t tiles = (all + M::kCols - 1) / M::kCols;
    const Span sp = span_of(a, r);
    const int32_t per = (sp.hi - sp.lo + static_cast<int32_t>(w0.pieces) - 1) / static_cast<int32_t>(w0.pieces);
    const int32_t b0 = min(sp.lo + static_cast<int32_t>(w0.piece) * per, sp.hi), b1 = min(b0 + per, sp.hi);
    const float fm = a.scale_log2;
    // the last tiles see the most: they begin first
    for (uint32_t turn = blockIdx.y; turn < tiles; turn += gridDim.y) {
        const uint32_t tile = tiles - 1 - turn;
        const Columns w = columns<M::kCols>(a, r, kvh, tile, 32 * group + col);
        const int32_t p0 = max(b0, w.lo / kPage), p1 = min(b1, (w.hi + kPage - 1) / kPage);
        // positions that the column sees (one without a row has a zero query and sees what the last has)
        const int32_t see_hi = (w.row < 0 ? w.last_pos : w.pos) + 1, see_lo = sees_from(a.window, see_hi - 1);
        // positions that all of the wave's columns see: [full_lo, full_hi)
        const uint32_t c0 = tile * M::kCols + 32 * group;
        const int32_t full_lo = sees_from(a.window, r.base + static_cast<int32_t>(min(c0 + 31, all - 1) / a.group));
        const int32_t full_hi = r.base + static_cast<int32_t>(min(c0, all - 1) / a.group) + 1;

        // the queries, the second operand of the scores: k-step 4 B + i has channels 8 i .. 8 i + 7 of block 2 B + half
        bf16x8 qf[QS];
        {
            const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (static_cast<uint64_t>(r.first + max(w.row, 0)) * a.heads + w.head) * D + kBlock * half;
            const uint32_t flip = a.flip | a.flip >> 16;
            u16x2 high = {0, 0};                 // largest magnitudes, as bits
#pragma unroll
            for (int s = 0; s < QS; ++s) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (w.row >= 0) u = *reinterpret_cast<const uint4*>(qp + 2 * kBlock * (s / 4) + 8 * (s % 4));
                for (const uint32_t v : {u.x, u.y, u.z, u.w}) high = __builtin_elementwise_max(high, __builtin_bit_cast(u16x2, v & 0x7FFF7FFFu));
                qf[s] = __builtin_bit_cast(bf16x8, make_uint4((u.x & a.keep) ^ flip, (u.y & a.keep) ^ flip, (u.z & a.keep) ^ flip, (u.w & a.keep) ^ flip));
            }
            // (an infinite query's products need not all be NaN, nor those of a scale of 0: one NaN makes them so)
            if (max(high[0], high[1]) >= 0x7F80u) qf[0][0] = static_cast<__bf16>(__builtin_nanf(""));
        }

        // Lane i has the id of page at + i (-1: none).
        int32_t at = p0, ids = -1;
        auto look = [&](int32_t p) {
            at = p;
            ids = p + lane < p1 ? page_id(a.c, a.s, seq, p + lane) : -1;
        };
        auto place = [&](int32_t p) {
            const int32_t id = __builtin_amdgcn_readlane(ids, (p - at) & 63);
            return p < p1 ? id : -1;
        };

        // The thread's pieces of a page's keys and values, and the scales of the keys that its lane multiplies, on the
        // way from memory (where there is no page, page 0 is read and not used).
        const bool has_k = PER != 0 || tid < PIECES, has_v = PER != 0 || (tid >= PIECES && tid < 2 * PIECES);
        const int vi = PER != 0 ? tid : tid - PIECES;
        constexpr int VC = D / 8;                 // pieces (16 bytes) of a group of four tokens
        const uint32_t v_group = (vi / VC) & 15, v_piece = vi % VC;
        uint4 kc = make_uint4(0, 0, 0, 0), vc = kc;
        uint32_t vs = 0, vs_next = 0, ks[KB / 2], ks_next[KB / 2];
        auto fetch = [&](int32_t p) {
            const uint64_t pl = static_cast<uint64_t>(max(place(p), 0)) * a.c.kv_heads + kvh;
            if (has_k) kc = *reinterpret_cast<const uint4*>(a.c.k + pl * kCodeBytes<D> + 16 * tid);
            if (has_v) vc = *reinterpret_cast<const uint4*>(a.c.v + pl * kCodeBytes<D> + 16 * vi);
            // (tokens row % 16 + 16 i of block 2 B + half: byte i)
#pragma unroll
            for (int b = 0; b < KB / 2; ++b)
                ks_next[b] = *reinterpret_cast<const uint32_t*>(a.c.k_scale + pl * kScaleBytes<D> + k_scale_at<D>(col & 15, 2 * b + half));
        };
        auto fetch_next = [&](int32_t p) {
            const uint64_t pl = static_cast<uint64_t>(max(place(p), 0)) * a.c.kv_heads + kvh;
            if (has_v) vs_next = *reinterpret_cast<const uint32_t*>(a.c.v_scale + pl * kScaleBytes<D> + v_scale_at<D>(4 * v_group, v_piece * 8 / kBlock));
        };
        // (shifted so that tile t's is byte 2 t)
        auto take_scales = [&] {
#pragma unroll
            for (int b = 0; b < KB / 2; ++b) ks[b] = ks_next[b] >> (8 * (col >> 4));
        };
        // Whether a column may see token i of the thread's four, and whether one may see all of a page.
        auto seen = [&](int32_t p, int i) {
            const int32_t t = p * kPage + 4 * static_cast<int32_t>(v_group) + i;
            return (t >= w.lo) & (t < w.hi) & (place(p) >= 0);
        };
        auto whole = [&](int32_t p) { return p * kPage >= w.lo && p * kPage + kPage <= w.hi && place(p) >= 0; };
        // Exponent bytes of values that no column sees become 0.
        auto visible = [&](int32_t p, uint32_t bytes) {
            if (!whole(p)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) bytes &= seen(p, i) ? 0xFFFFFFFFu : ~(0xFFu << (8 * i));
            }
            return bytes;
        };
        // The unit's exponent (biased) of the page staged, and of the outputs.  What the waves tell each other of a page
        // ahead: 1: its largest exponent is too high for the unit so far, 2: high enough, and the largest byte above.
        int32_t want = kNoUnit, unit = kNoUnit, highest = kNoUnit;
        auto tell = [&](int32_t p) {
            if (!has_v) return;                  // (a whole wave: it says nothing)
            const uint32_t v = visible(p, vs_next), m = max(max(v & 0xFFu, v >> 8 & 0xFFu), max(v >> 16 & 0xFFu, v >> 24));
            const bool high = __any(static_cast<int32_t>(m) > want + 13), enough = __any(static_cast<int32_t>(m) >= want - 10);
            uint32_t word = 2;
            if (high || !enough) word = 1 | wave_max_u32(m) << 8;   // (also: no unit so far)
            if (lane == 0) most[8 * (p & 1) + wave] = word;
        };
        auto settle = [&](int32_t p) {
            const uint4 u = reinterpret_cast<const uint4*>(most + 8 * (p & 1))[0], v = reinterpret_cast<const uint4*>(most + 8 * (p & 1))[1];
            const uint32_t some = __builtin_amdgcn_readfirstlane(static_cast<int>((u.x | u.y | u.z | u.w) | (v.x | v.y | v.z | v.w)));
            if ((some & 1) == 0) return;
            const int32_t m = __builtin_amdgcn_readfirstlane(static_cast<int>(max(max(max(u.x, u.y), max(u.z, u.w)), max(max(v.x, v.y), max(v.z, v.w))) >> 8));
            // (0: nothing is seen; some waves may have exponents high enough where others have none)
            const bool fall = (some & 2) == 0 && m < want - 10 && m > static_cast<int32_t>(kByteMin);
            if (m != 0 && (want == kNoUnit || m > want + 13 || fall)) want = max(m + 4, highest - kFar);
            highest = max(highest, want);
        };
        // Into shared memory.  Rows of 16-byte chunks, permuted so that reads meet in no bank.
        constexpr int kKeyRow = D / 2;
        auto key_chunk = [](uint32_t row, uint32_t c) { return D == 256 ? c ^ ((row >> 1) & 7) : (D == 128 ? c ^ ((row >> 2) & 3) : c); };
        auto stage_k = [&](int32_t p) {
            const uint32_t row = tid / KB, c = tid % KB;
            if (has_k) *reinterpret_cast<uint4*>(lds + (p & 1) * M::kKeys + row * kKeyRow + 16 * key_chunk(row, c)) = kc;
        };
        // What no column sees may be anything: 0.  (Before the page goes into shared memory.)
        auto hide = [&](int32_t p) {
            if (whole(p)) return;
            vs = visible(p, vs);
            uint32_t word[4] = {vc.x, vc.y, vc.z, vc.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == 64) {                 // (token i: 16 bits of words i / 2 and 2 + i / 2)
                    const uint32_t keep = seen(p, i) ? 0xFFFFFFFFu : (i % 2 == 0 ? 0xFFFF0000u : 0xFFFFu);
                    word[i / 2] &= keep;
                    word[2 + i / 2] &= keep;
                } else if constexpr (D == 128) {
                    word[i] = seen(p, i) ? word[i] : 0u;
                } else {
                    word[i] = seen(p, 2 * (v_piece & 1) + i / 2) ? word[i] : 0u;
                }
            }
            vc = make_uint4(word[0], word[1], word[2], word[3]);
        };
        auto stage_v = [&](int32_t p) {
            if (!has_v) return;
            uint32_t word[4] = {vc.x, vc.y, vc.z, vc.w};
            if constexpr (D == 256) {
                // a piece is two tokens of a sixteenth's 16 channels, the next lane's the other two: each takes 8
                // channels of the four
                const bool odd = (v_piece & 1) != 0;
                const uint32_t a0 = dpp_u32<0xB1>(odd ? word[0] : word[1]), a1 = dpp_u32<0xB1>(odd ? word[2] : word[3]);
                const uint32_t b0 = odd ? word[1] : word[0], b1 = odd ? word[3] : word[2];
                word[0] = odd ? a0 : b0;
                word[1] = odd ? a1 : b1;
                word[2] = odd ? b0 : a0;
                word[3] = odd ? b1 : a1;
            }
            float d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t byte = static_cast<int32_t>(vs >> (8 * i) & 0xFFu);
                d[i] = scale_of(static_cast<uint32_t>(max(byte, want - 126) - want + 127));
            }
            // group 4 s + g of a page is the (0, 2, 1, 3)-th of its 16 tokens
            const uint32_t chunk = 2 * (v_group / 4) + (v_group & 1), eighth = (v_group >> 1) & 1;
            uint8_t* buf = v_lds + (p & 1) * M::kValues;
            auto row_at = [&](uint32_t row) { return buf + row * M::kValueRow + 16 * (chunk ^ ((row >> 1) & 7)) + 8 * eighth; };
            {
#pragma unroll
                for (int b = 0; b < 4; ++b) {            // a byte: two channels of four tokens
                    uint32_t x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // word i is token i, 8 channels; D 64: words 2 h and 2 h + 1 are sixteenth h's 4 channels
                        const uint32_t u = D == 64 ? word[2 * (b / 2) + i / 2] : word[i];
                        const int byte_at = D == 64 ? 2 * (i % 2) + b % 2 : b;
                        x[i] = byte_at == 0 ? pair_f16<0>(u, d[i]) : (byte_at == 1 ? pair_f16<1>(u, d[i]) : (byte_at == 2 ? pair_f16<2>(u, d[i]) : pair_f16<3>(u, d[i])));
                    }
                    // channels of the byte: sixteenth c, its channels m and m + 1: rows m * 16 + c
                    const uint32_t c = D == 64 ? 2 * v_piece + b / 2 : (D == 128 ? v_piece : v_piece / 2);
                    const uint32_t m0 = D == 64 ? 2 * (b % 2) : (D == 128 ? 0 : 8 * (v_piece & 1)) + 2 * b;
                    *reinterpret_cast<uint2*>(row_at(m0 * 16 + c)) = make_uint2(lowers(x[0], x[1]), lowers(x[2], x[3]));
                    *reinterpret_cast<uint2*>(row_at((m0 + 1) * 16 + c)) = make_uint2(uppers(x[0], x[1]), uppers(x[2], x[3]));
                }
            }
        };

        f32x16 o[ET];
        float m_run = -__builtin_inff(), l_run = 0.f;
#pragma unroll
        for (int e = 0; e < ET; ++e)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[e][i] = 0.f;
        bool begun = false;                      // every column of the wave has a reference

        // The codes of tile t of a page (32 tokens; a pair's wave has one tile, `part`), and its scores.
        auto codes = [&](int32_t p, int t, uint4 (&u)[KB / 2]) {
            const uint32_t row = 32 * t + col;
            const uint8_t* from = lds + (p & 1) * M::kKeys + row * kKeyRow;
#pragma unroll
            for (int b = 0; b < KB / 2; ++b) u[b] = *reinterpret_cast<const uint4*>(from + 16 * key_chunk(row, 2 * b + half));
        };
        auto scores = [&](const uint4 (&from)[KB / 2], int t, f32x16& sc) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = 0.f;
#pragma unroll
            for (int b = 0; b < KB / 2; ++b) {
                const uint4 u = from[b];
                const float d = scale_of(ks[b] >> (16 * t) & 0xFFu);
                const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(values8(word[i], d), qf[4 * b + i], sc, 0, 0, 0);
            }
        };
        const uint32_t v_from = static_cast<uint32_t>((32 * ET * part + col) * M::kValueRow + 16 * (half ^ ((col >> 1) & 7)));
        // The output's products of a tile's two k-steps.
        auto values = [&](int32_t p, int t, const f16x8 (&pf)[2]) {
            const uint8_t* buf = v_lds + (p & 1) * M::kValues;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int e = 0; e < ET; ++e)
                    o[e] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const f16x8*>(buf + (v_from ^ (64 * t + 32 * s)) + e * 32 * M::kValueRow), pf[s], o[e], 0, 0, 0);
        };
        // A tile's probabilities e^(sc mul - base), and their sum in the lane (of the rounded ones).
        auto weigh = [&](const f32x16& sc, float mul, float base, f16x8 (&pf)[2]) {
            const f16x2 one = {static_cast<_Float16>(1.f), static_cast<_Float16>(1.f)};
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float x = __builtin_amdgcn_exp2f(fmaf(sc[i], mul, -base));
                const float y = __builtin_amdgcn_exp2f(fmaf(sc[i + 1], mul, -base));
                const f16x2 h = {static_cast<_Float16>(x), static_cast<_Float16>(y)};
                sum[(i >> 1) & 1] = __builtin_amdgcn_fdot2(h, one, sum[(i >> 1) & 1], false);
                pf[i >> 3][i & 7] = h[0];
                pf[i >> 3][(i & 7) + 1] = h[1];
            }
            return sum[0] + sum[1];
        };
        auto scale_outputs = [&](float f) {
#pragma unroll
            for (int e = 0; e < ET; ++e)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[e][i] *= f;
        };
        // A tile's scores times fm, those that are not seen -infinity, and the largest of the column.
        auto masked = [&](int32_t t0, bool there, f32x16& sc) {
            float mt = -__builtin_inff();
            const int32_t lo = see_lo - t0 - 4 * half, hi = there ? see_hi - t0 - 4 * half : -kPage;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int32_t k = 8 * (i >> 2) + (i & 3);
                sc[i] = k >= lo && k < hi ? sc[i] * fm : -__builtin_inff();
                mt = fmaxf(mt, sc[i]);
            }
            return max_halves(mt);
        };
        // Moves the reference, where the largest score of `tokens` from t0 on is above it.
        auto refer = [&](int32_t t0, int32_t tokens, bool there, float mt) {
            // (of tokens that give only NaN the reference is 0)
            if (there && mt == -__builtin_inff() && m_run == mt && max(see_lo, t0) < min(see_hi, t0 + tokens)) mt = 0.f;
            if (__any(mt > m_run + kMoveManyAt)) {
                const float m_new = mt > m_run + kMoveManyAt ? mt : m_run;
                const float keep = m_new == m_run ? 1.f : __builtin_amdgcn_exp2f(m_run - m_new);
                m_run = m_new;
                l_run *= keep;
                scale_outputs(keep);
            }
            begun = __all(m_run > -__builtin_inff());
            return (m_run > -__builtin_inff() ? m_run : 0.f) - kBias;
        };

        if (p0 < p1) {
            look(p0);
            fetch(p0);
            fetch_next(p0);
            if (tid < 16) most[tid] = 0;
            if (PAIR && tid < 2) again[tid] = 0;
            __syncthreads();
            tell(p0);
            vs = vs_next;
            fetch_next(p0 + 1);
            stage_k(p0);
            __syncthreads();
            settle(p0);
            tell(p0 + 1);
            hide(p0);
            stage_v(p0);
            unit = want;
            __syncthreads();
            // One barrier a page: while page p is computed, p + 1 goes into the other buffers, and what p + 2 holds at
            // most is told.
#pragma unroll 1
            for (int32_t p = p0; p < p1; ++p) {
                const bool there = place(p) >= 0;
                const bool full = there && p * kPage >= full_lo && p * kPage + kPage <= full_hi;
                // (while the page's codes are on their way) the scales of its keys, and what comes after the next page
                auto ahead = [&] {
                    take_scales();
                    if (p + 3 - at > 64) look(p);
                    fetch(p + 1);
                    vs = vs_next;
                    fetch_next(p + 2);
                };
                // (no number stays none whatever the reference)
                auto fits = [&](float l) { return full && begun && !__any(l >= kSumLimit); };
                auto turn_unit = [&] {           // outputs so far in the unit of this page's values
                    if (unit == want) return;
                    scale_outputs(ldexpf(1.f, unit - want));   // (kNoUnit: they are 0)
                    unit = want;
                };
                auto stage = [&] {
                    stage_k(p + 1);
                    stage_v(p + 1);
                };
                if constexpr (PAIR) {
                    // The probabilities go through shared memory relative to the reference so far; if that does for one
                    // wave not, all take the way over the page's maximum.
                    f32x16 sc;
                    f16x8 mine[2], pf[2][2];
                    f16x8* const mail = reinterpret_cast<f16x8*>(p_lds) + 4 * group * 64 + lane;
                    auto send = [&] {
#pragma unroll
                        for (int s = 0; s < 2; ++s) mail[(2 * part + s) * 64] = mine[s];
                    };
                    {
                        uint4 u[KB / 2];
                        codes(p, part, u);
                        ahead();
                        scores(u, part, sc);
                    }
                    float l = weigh(sc, fm, m_run - kBias, mine);
                    send();
                    if (!fits(l) && lane == 0) again[p & 1] = 1;
                    __syncthreads();
                    if (again[p & 1] != 0) {
                        const float mt = masked(p * kPage + 32 * part, there, sc);
                        if (half == 0) m_lds[(2 * group + part) * 32 + col] = mt;
                        __syncthreads();
                        l = weigh(sc, 1.f, refer(p * kPage, kPage, there, fmaxf(mt, m_lds[(2 * group + (part ^ 1)) * 32 + col])), mine);
                        send();
                        __syncthreads();
                    }
                    if (tid == 0) again[(p + 1) & 1] = 0;
                    l_run += l;
                    turn_unit();
                    settle(p + 1);
                    hide(p + 1);
                    tell(p + 2);
#pragma unroll
                    for (int s = 0; s < 4; ++s) pf[s / 2][s % 2] = mail[s * 64];
                    values(p, 0, pf[0]);
                    values(p, 1, pf[1]);
                    stage();
                } else {
                    // Stretches of products of one tile beside the exponentials of the other.
                    f32x16 s0, s1;
                    f16x8 f0[2], f1[2];
                    uint4 u0[KB / 2], u1[KB / 2];
                    codes(p, 0, u0);
                    codes(p, 1, u1);
                    ahead();
                    scores(u0, 0, s0);
                    scores(u1, 1, s1);
                    float l = weigh(s0, fm, m_run - kBias, f0);
                    asm volatile("" : "+v"(l));      // (formed here, beside the products, not in the branch that takes it)
                    turn_unit();
                    if (!fits(l)) l = weigh(s0, 1.f, refer(p * kPage, 32, there, masked(p * kPage, there, s0)), f0);
                    l_run += l;
                    values(p, 0, f0);
                    l = weigh(s1, fm, m_run - kBias, f1);
                    asm volatile("" : "+v"(l));
                    if (!fits(l)) l = weigh(s1, 1.f, refer(p * kPage + 32, 32, there, masked(p * kPage + 32, there, s1)), f1);
                    l_run += l;
                    settle(p + 1);
                    hide(p + 1);
                    tell(p + 2);
                    values(p, 1, f1);
                    stage();
                }
                __syncthreads();
            }
        }
        const float v_scale = unit == kNoUnit ? 0.f : ldexpf(1.f, unit - 127);

        float l = l_run + __shfl_xor(l_run, 32);
        if constexpr (PAIR) {
            __syncthreads();
            if (half == 0) m_lds[(2 * group + part) * 32 + col] = l;
            __syncthreads();
            l = m_lds[2 * group * 32 + col] + m_lds[(2 * group + 1) * 32 + col];
            __syncthreads();
        }
        if (w.row >= 0) {
            const float inv = (w0.pieces > 1 ? 1.f : (l == 0.f ? 0.f : 1.f / l));
            const uint64_t slot = (w0.first + static_cast<uint64_t>(w0.piece) * static_cast<uint32_t>(r.count) + static_cast<uint32_t>(w.row)) * a.heads + w.head;
            const uint64_t to = (static_cast<uint64_t>(r.first + w.row) * a.heads + w.head) * D;
            if (w0.pieces > 1 && half == 0 && part == 0) a.stat[slot] = make_float2(m_run, l);
            // register 4 q + i of tile e is channel (D / 16) c + m, c = 8 (q % 2) + 4 half + i, m = 2 (e + ET part) + q / 2
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ch = D / 16 * (8 * q + 4 * half + i) + 2 * ET * part;
                    float v[2 * ET];
#pragma unroll
                    for (int e = 0; e < ET; ++e) {
                        v[2 * e] = o[e][4 * q + i] * inv * v_scale;
                        v[2 * e + 1] = o[e][8 + 4 * q + i] * inv * v_scale;
                    }
                    if (w0.pieces > 1) {
#pragma unroll
                        for (int e = 0; e < 2 * ET; e += 4) *reinterpret_cast<float4*>(a.part + slot * D + ch + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    } else {
                        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
                        for (int e = 0; e < 2 * ET; e += 4) {
                            const bf16x4 b = {static_cast<__bf16>(v[e]), static_cast<__bf16>(v[e + 1]), static_cast<__bf16>(v[e + 2]), static_cast<__bf16>(v[e + 3])};
                            *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(a.out) + to + ch + e) = b;
                        }
                    }
                }
        }
    }
}

// Joins the pieces of each column of a sequence that was cut: a wave has a
// column, lane z piece z's maximum and sum, and the pieces' outputs are added
// in their order, D / 64 values a lane.  SPREAD: the four waves of a workgroup
// have a column, each every fourth piece (columns are few and have many).
template <uint32_t DT, int D, bool SPREAD>
__global__ __launch_bounds__(256) void attend4_join_kernel(Attend4Args a) {
    constexpr int V = D / 64;
    constexpr uint32_t STEP = SPREAD ? 4 : 1, AT_ONCE = 8;
    __shared__ float acc[SPREAD ? 4 : 1][SPREAD ? D : 1];
    const int lane = threadIdx.x & 63;
    const uint32_t wave = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)));
    const Piece w = find_piece(a, blockIdx.x, true);
    if (w.seq < 0 || w.pieces <= 1) return;
    const SeqRows r = seq_rows(a.s, static_cast<uint32_t>(w.seq));
    const uint64_t n = static_cast<uint64_t>(r.count) * a.heads;
    constexpr uint32_t kOwn = SPREAD ? 1 : 4;     // columns of a workgroup
    for (uint64_t i = static_cast<uint64_t>(blockIdx.y) * kOwn + (SPREAD ? 0 : wave); i < n; i += static_cast<uint64_t>(gridDim.y) * kOwn) {
        // (a piece's rows and heads are as those of the output)
        const uint64_t from = static_cast<uint64_t>(w.first) * a.heads + i;
        float x[AT_ONCE][V];
        auto load = [&](uint32_t z) {
#pragma unroll
            for (uint32_t u = 0; u < AT_ONCE; ++u)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    x[u][k] = z + u * STEP < w.pieces ? a.part[(from + (z + u * STEP) * n) * D + lane * V + k] : 0.f;
        };
        const uint32_t z0 = SPREAD ? wave : 0;
        load(z0);
        float2 st = make_float2(-__builtin_inff(), 0.f);
        if (static_cast<uint32_t>(lane) < w.pieces) st = a.stat[from + lane * n];
        float m = st.x;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k));
        const float f = st.x == m ? 1.f : __builtin_amdgcn_exp2f(st.x - m);
        float l = f * st.y;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) l += __shfl_xor(l, k);
        float v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = 0.f;
        for (uint32_t z = z0; z < w.pieces; z += AT_ONCE * STEP) {
            if (z != z0) load(z);
#pragma unroll
            for (uint32_t u = 0; u < AT_ONCE; ++u) {
                const float g = z + u * STEP < w.pieces ? read_lane(f, static_cast<int>(z + u * STEP)) : 0.f;
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] = fmaf(g, x[u][k], v[k]);
            }
        }
        // (nothing seen: 0; a sum of 0 past float32's range: no number)
        const float inv = m == -__builtin_inff() && l == 0.f ? 0.f : 1.f / l;
        if constexpr (SPREAD) {
#pragma unroll
            for (int k = 0; k < V; ++k) acc[wave][lane * V + k] = v[k];
            __syncthreads();
            const uint64_t to = (static_cast<uint64_t>(r.first) * a.heads + i) * D + threadIdx.x;
            if (threadIdx.x < D) {
                const float y = ((acc[0][threadIdx.x] + acc[1][threadIdx.x]) + (acc[2][threadIdx.x] + acc[3][threadIdx.x])) * inv;
                if constexpr (DT == QMV_F32) static_cast<float*>(a.out)[to] = y;
                else static_cast<__bf16*>(a.out)[to] = static_cast<__bf16>(y);
            }
            __syncthreads();
        } else {
            const uint64_t to = (static_cast<uint64_t>(r.first) * a.heads + i) * D + lane * V;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if constexpr (DT == QMV_F32) static_cast<float*>(a.out)[to + k] = v[k] * inv;
                else static_cast<__bf16*>(a.out)[to + k] = static_cast<__bf16>(v[k] * inv);
            }
        }
    }
}

struct Plan {
    Kind kind;
    uint32_t tiles, target, least, slots;
    uint64_t room;
};
// Workgroups that a launch of the kernel for few aims at (us with 512, 768 and
// 1024: 32 x 4000 float32 30.1, 30.4 and 31.1; 2 x 131072 bfloat16 42.4, 44.8 and
// 44.8).
constexpr uint32_t kWorkgroups = 512;
// Columns of a call up to which a workgroup, not a wave, joins one (us, workgroup
// / wave: 64 columns of 32 pieces 38.5 / 41.1, 256 of 8 30.7 / 31.7, 1024 of 2
// 31.0 / 30.1).
constexpr uint64_t kSpreadCols = 512;
// Pages up to which a sequence is not cut: a join is a launch, of 3 to 5 us; with
// workgroups enough (kBusy) up to more (us, whole / cut, 8 heads of 128: 1 x 1000
// 10.3 / 13.8, 32 x 1000 10.4 / 16.2, 1 x 2000 12.3 / 11.8, float32 14.6 / 12.8; 16
// x 2000 12.6 / 15.5; 1 x 3000 16.0 / 11.6, 16 x 3000 17.3 / 18.6).
constexpr uint32_t kWhole = 24, kWholeBusy = 34;
constexpr uint64_t kBusy = 64;
// In the kernel for many, whose workgroups walk pages faster, and the number that
// a launch of it aims at, two a compute unit, or one in pairs of waves (us, 512 /
// 256: 1 x 16000 with 128 rows 63 / 90, 4 x 8000 with 64 53 / 66, head dims of
// 256, 2 x 16000 with 64 96 / 76); from kManyFull on a launch is not cut (16 x 4000
// with 64 rows, 256 workgroups, cut 118, else 102).
constexpr uint32_t kWholeMany = 16;
constexpr uint64_t kManyAim = 512, kManyPairs = 256, kManyFull = 192;
// Workgroups from which each wave has its own columns (us, own / shared: 64 x
// 1000 with 32 and 64 columns 30 / 33 and 35 / 53, 1024 and 2048 workgroups; at
// 512, 8 x 3000 with 128 51 / 36, 16 x 1000 with 64 22 / 26).
constexpr uint64_t kSoloFrom = 1024;
// bfloat16 queries go to the kernel for many where a sequence has columns enough
// for its tiles (kManyCols / D) and the call work enough (products of 16 columns
// with a page, times D) that its waves' waiting for each other is paid for.
// Measured (us, few / many), sequences x tokens, columns:
//   D 128, 8 heads: 1 x 16000, 64, 128 and 256: 24 / 30, 34 / 36 and 55 / 50; 8 x
//     3000, 128 and 256: 36 / 39 and 55 / 63; 64 x 1000, 128 and 256: 53 / 46 and
//     88 / 81; whole prompts 2 x 500 18 / 22, 1 x 1000 28 / 35, 1 x 2000 71 / 62
//   D 256, 4 heads: 1 x 16000, 256: 43 / 60; 8 x 3000, 128 and 256: 41 / 52 and
//     62 / 58; 64 x 1000, 128: 60 / 59; prompts 2 x 500 24 / 35, 1 x 4000 219 / 202
//   D 64, 8 heads: 8 x 3000, 256 and 512: 42 / 55 and 66 / 76; 64 x 1000, 256 and
//     512: 62 / 67 and 104 / 93; prompts 1 x 1000 21 / 33, 1 x 4000 153 / 109
constexpr uint64_t kManyCols = 16384;
constexpr double kManyWork = 7e6, kManyWork64 = 12e6;   // head dims of 64: the second

Plan plan_of(const qmv_kv4_cache& c, const qmv_kv_seqs& s, uint32_t dtype, uint32_t heads, uint32_t window) {
    const uint64_t group = heads / c.kv_heads;
    const uint64_t most = s.max_new < s.rows ? (s.max_new == 0 ? 1 : s.max_new) : s.rows;
    const uint64_t pages = span_pages(s, window, most), cols = most * group;
    Plan p{};
    // (pages of the middle row)
    qmv_kv_seqs mean = s;
    mean.max_len -= static_cast<uint32_t>(most / 2 < s.max_len ? most / 2 : s.max_len);
    const double work = static_cast<double>(uint64_t{s.seqs} * c.kv_heads) * static_cast<double>((cols + 15) / 16) *
                        static_cast<double>(span_pages(mean, window, 16)) * c.head_dim;
    if (dtype == QMV_BF16 && cols * c.head_dim >= kManyCols && work >= (c.head_dim == 64 ? kManyWork64 : kManyWork)) p.kind = kMany;
    const uint64_t wide = p.kind == kMany ? 128 : 16;
    uint64_t tiles = (cols + wide - 1) / wide;
    const uint64_t wgs = uint64_t{s.seqs} * c.kv_heads * tiles;
    if (p.kind != kMany && cols <= (dtype == QMV_F32 ? kPackedCols<QMV_F32> : kPackedCols<QMV_BF16>)) p.kind = kPacked;
    else if (p.kind != kMany && wgs >= kSoloFrom) {
        p.kind = kSolo;
        tiles = (tiles + 3) / 4;
    }
    p.tiles = static_cast<uint32_t>(tiles > 65535 ? 65535 : tiles);
    p.slots = s.seqs;
    const uint64_t whole = p.kind == kMany ? kWholeMany : (wgs >= kBusy ? kWholeBusy : kWhole);
    if (p.kind == kSolo || s.seqs > kScanSeqs || pages <= whole || (p.kind == kMany && wgs >= kManyFull)) return p;
    const uint64_t aim = p.kind == kMany ? (c.head_dim == 256 ? kManyPairs : kManyAim) : kWorkgroups;
    uint64_t target = (aim + c.kv_heads * tiles - 1) / (c.kv_heads * tiles);
    if (target < s.seqs / 2) target = s.seqs / 2;
    if (target < 1) target = 1;
    p.target = static_cast<uint32_t>(target);
    p.least = p.kind == kMany ? 8 : 4;
    p.slots = p.target + s.seqs;
    const uint64_t pieces = target < kMaxPieces ? target : kMaxPieces;
    uint64_t room = pieces * s.rows;
    if (room > p.slots * most) room = p.slots * most;
    p.room = room > 0x7FFFFFFFu ? 0x7FFFFFFFu : room;
    return p;
}

template <uint32_t DT, int D>
hipError_t go(const Attend4Args& a, const Plan& p, hipStream_t s) {
    const dim3 grid(p.slots * a.c.kv_heads, p.tiles), block(256);
    bool done = false;
    if constexpr (DT == QMV_BF16) {
        if (p.kind == kMany) {
            constexpr int bytes = Many<D>::kBytes;
            if constexpr (bytes > 65536) {
                const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(attend4_many_kernel<D>), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
                if (e != hipSuccess) return e;
            }
            hipLaunchKernelGGL((attend4_many_kernel<D>), grid, dim3(Many<D>::kThreads), bytes, s, a);
            done = true;
        }
    }
    if (done) {
    } else if (p.kind == kSolo) hipLaunchKernelGGL((attend4_few_kernel<DT, D, kSolo>), grid, block, 0, s, a);
    else if (p.kind == kPacked) hipLaunchKernelGGL((attend4_few_kernel<DT, D, kPacked>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attend4_few_kernel<DT, D, kShared>), grid, block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.target != 0) {
        const uint64_t most = a.s.max_new < a.s.rows ? a.s.max_new : a.s.rows;
        const bool spread = most * a.heads * a.s.seqs <= kSpreadCols;
        uint64_t y = spread ? most * a.heads : (most * a.heads + 3) / 4;
        if (y < 1) y = 1;
        if (y > 65535) y = 65535;
        const dim3 joins(a.s.seqs, static_cast<uint32_t>(y));
        if (spread) hipLaunchKernelGGL((attend4_join_kernel<DT, D, true>), joins, block, 0, s, a);
        else hipLaunchKernelGGL((attend4_join_kernel<DT, D, false>), joins, block, 0, s, a);
        e = hipGetLastError();
    }
    return e;
}
template <uint32_t DT>
hipError_t go(const Attend4Args& a, const Plan& p, hipStream_t s) {
    if (a.c.head_dim == 64) return go<DT, 64>(a, p, s);
    if (a.c.head_dim == 128) return go<DT, 128>(a, p, s);
    return go<DT, 256>(a, p, s);
}

}  // namespace

uint64_t kv4_attend_workspace_bytes(const qmv_kv4_cache& c, const qmv_kv_seqs& s, uint32_t dtype, uint32_t heads, uint32_t window) {
    return plan_of(c, s, dtype, heads, window).room * heads * (c.head_dim + 2) * 4;
}

hipError_t launch_kv4_attend(const qmv_kv4_cache& c, const qmv_kv_seqs& s, uint32_t dtype, uint32_t heads, float scale, uint32_t window,
                             const void* q, void* out, void* workspace, hipStream_t stream) {
    const Plan p = plan_of(c, s, dtype, heads, window);
    float* part = static_cast<float*>(workspace);
    // (a scale of 0: queries of 0)
    const float by = scale == 0.f ? 1.f : (scale < 0.f ? -scale : scale) * kLog2e;
    const Attend4Args a{c, s, q, out, part, reinterpret_cast<float2*>(part + p.room * heads * c.head_dim), by, kMoveAt / by,
                        scale == 0.f ? 0u : ~0u, scale < 0.f ? 0x80000000u : 0u, heads,
                        heads / c.kv_heads, window, p.target, p.least, static_cast<uint32_t>(p.room)};
    return dtype == QMV_F32 ? go<QMV_F32>(a, p, stream) : go<QMV_BF16>(a, p, stream);
}

}  // namespace qmv
