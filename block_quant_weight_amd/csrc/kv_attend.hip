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
//   q = x 2^(E-22), x = rint(q 2^(22-E)) with |q| < 2^E the row's largest;
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
// Work: a workgroup of four waves has 16 columns (query row x head of one
// key/value head) and a piece of the sequence's pages; each wave takes every
// fourth page and keeps its own running maximum, sum and output, joined in
// shared memory at the end.  The pieces of a sequence are joined by a second
// kernel, in their order.
#include "kv_common.h"

namespace qmv {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPScale = 127.0f * 65536.0f;   // p = 1 as a whole number
constexpr int kCols = 16;                      // columns of a workgroup

struct AttendArgs {
    qmv_kv_cache c;
    qmv_kv_seqs s;
    const void* q;
    void* out;
    float* part;        // [pieces][rows * heads][D + 2]: output sum, maximum, sum
    float scale_log2;   // scale * log2(e)
    uint32_t heads, group, window, pieces;
};

// Three signed digits of each of four whole numbers |x| <= 127 * 2^16, as
// dwords of four bytes: x = d0 + 256 d1 + 65536 d2.
__device__ __forceinline__ void digits4(const int x[4], uint32_t d[3]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = static_cast<uint32_t>(x[i] + 0x8080) ^ 0x8080u;
    // bytes 0 of (u0, u1) and (u2, u3), bytes 1, bytes 2
    const uint32_t a = __builtin_amdgcn_perm(u[1], u[0], 0x05010400u);  // b0 b0' b1 b1'
    const uint32_t b = __builtin_amdgcn_perm(u[3], u[2], 0x05010400u);
    d[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    d[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    const uint32_t e = __builtin_amdgcn_perm(u[1], u[0], 0x00000602u);
    const uint32_t f = __builtin_amdgcn_perm(u[3], u[2], 0x06020000u);
    d[2] = __builtin_amdgcn_perm(f, e, 0x07060100u);
}

__device__ __forceinline__ float xor_lane(float v, int m) { return __shfl_xor(v, m); }

// What a workgroup's columns are.
struct Columns {
    int64_t row, pos;      // this lane's query row and position (row -1: none)
    uint32_t head;
    int64_t lo, hi;        // positions that any of the 16 columns sees: [lo, hi)
};
__device__ __forceinline__ Columns columns(const AttendArgs& a, const SeqRows& r, uint32_t kvh, int64_t tile,
                                           int col) {
    Columns o;
    const int64_t n = r.count * a.group, c = tile * kCols + col;
    const int64_t t0 = tile * kCols / a.group;
    const int64_t t1 = min(tile * kCols + kCols - 1, n - 1) / a.group;
    o.row = c < n ? r.first + c / a.group : -1;
    o.pos = r.base + c / a.group;
    o.head = kvh * a.group + static_cast<uint32_t>(c % a.group);
    const int64_t first = max(r.base + t0, int64_t{0});
    o.hi = max(r.base + t1 + 1, int64_t{0});
    o.lo = a.window != 0 ? max(first - static_cast<int64_t>(a.window) + 1, int64_t{0}) : 0;
    return o;
}

template <uint32_t DT, int D>
__global__ __launch_bounds__(256) void attend_few_kernel(AttendArgs a) {
    typedef typename Elem<DT>::type T;
    constexpr int KS = D / 64;     // k-steps of a score tile
    constexpr int ET = D / 16;     // tiles of output dims
    __shared__ float acc[4][kCols][D + 1];
    __shared__ float stat[4][kCols][2];
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t seq = blockIdx.x / a.c.kv_heads, kvh = blockIdx.x % a.c.kv_heads;
    const uint32_t piece = blockIdx.z;
    const SeqRows r = seq_rows(a.s, seq);
    const int64_t tiles = (r.count * a.group + kCols - 1) / kCols;
    for (int64_t tile = blockIdx.y; tile < tiles; tile += gridDim.y) {
        const Columns w = columns(a, r, kvh, tile, col);
        // pages of this piece
        const int64_t p_lo = w.lo / kPage, p_hi = (w.hi + kPage - 1) / kPage;
        const int64_t per = (p_hi - p_lo + a.pieces - 1) / a.pieces;
        const int64_t p0 = p_lo + piece * per, p1 = min(p0 + per, p_hi);
        const int64_t see_lo = a.window != 0 ? max(w.pos - static_cast<int64_t>(a.window) + 1, int64_t{0}) : 0;

        // the query's digits
        uint32_t qd[KS][3][4];
        float qs;
        {
            float v[KS][16];
            const T* qp = static_cast<const T*>(a.q) + (static_cast<uint64_t>(w.row < 0 ? 0 : w.row) * a.heads + w.head) * D;
            uint32_t m = 0;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if (w.row >= 0) {
                    load8<DT>(qp + 64 * s + 16 * quad, v[s]);
                    load8<DT>(qp + 64 * s + 16 * quad + 8, v[s] + 8);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[s][i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[s][i]) & 0x7FFFFFFFu);
            }
            m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
            m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
            const float amax = __builtin_bit_cast(float, m);
            int e = 0;
            const bool zero = m == 0 || m >= 0x7F800000u;
            if (!zero) (void)frexpf(amax, &e);       // amax in [2^(e-1), 2^e)
            qs = m >= 0x7F800000u ? __builtin_nanf("") : (zero ? 0.f : ldexpf(1.f, e - 22));
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    int x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = zero ? 0 : static_cast<int>(rintf(ldexpf(v[s][4 * j + i], 22 - e)));
                    uint32_t d[3];
                    digits4(x, d);
#pragma unroll
                    for (int k = 0; k < 3; ++k) qd[s][k][j] = d[k];
                }
        }

        float o[ET][4];
#pragma unroll
        for (int e = 0; e < ET; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[e][i] = 0.f;
        float m_run = -__builtin_inff(), l_run = 0.f;

        for (int64_t p = p0 + wave; p < p1; p += 4) {
            const int64_t id = page_id(a.c, a.s, seq, p);
            if (id < 0) continue;
            const uint64_t at = static_cast<uint64_t>(id) * a.c.kv_heads + kvh;
            const int8_t* kp = a.c.k + at * (kPage * D);
            const int8_t* vp = a.c.v + at * (kPage * D);
            const float ks = a.c.k_scale[at], vs = a.c.v_scale[at];
            // scores
            float sc[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int8_t* kr = kp + (16 * (col >> 2) + 4 * j + (col & 3)) * D + 16 * quad;
                i32x4 c[3];
#pragma unroll
                for (int k = 0; k < 3; ++k) c[k] = i32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const i32x4 kf = *reinterpret_cast<const i32x4*>(kr + 64 * s);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const i32x4 b = {static_cast<int>(qd[s][k][0]), static_cast<int>(qd[s][k][1]),
                                         static_cast<int>(qd[s][k][2]), static_cast<int>(qd[s][k][3])};
                        c[k] = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf, b, c[k], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float t = fmaf(static_cast<float>(c[2][i]), 65536.f,
                                         fmaf(static_cast<float>(c[1][i]), 256.f, static_cast<float>(c[0][i])));
                    sc[j][i] = (t * qs) * (ks * a.scale_log2);
                }
            }
            // what this column sees of the page: tokens [from, to)
            const int from = static_cast<int>(min(max(see_lo - p * kPage, int64_t{0}), int64_t{kPage}));
            const int to = w.row < 0 ? 0 : static_cast<int>(min(max(w.pos + 1 - p * kPage, int64_t{0}), int64_t{kPage}));
            const bool any = from < to;
            float mt = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 16 * quad + 4 * j + i;
                    sc[j][i] = t >= from && t < to ? sc[j][i] : -__builtin_inff();
                    mt = fmaxf(mt, sc[j][i]);
                }
            mt = fmaxf(mt, xor_lane(mt, 16));
            mt = fmaxf(mt, xor_lane(mt, 32));
            // nothing seen, or only NaN: the maximum counts as 0 (NaN scores
            // still make the sum NaN, and so does a score of +infinity)
            const float ref = mt > -__builtin_inff() ? mt : 0.f;
            float lt = 0.f;
            uint32_t pd[3][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                int x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float pr = exp2f(sc[j][i] - ref);
                    lt += pr;
                    x[i] = static_cast<int>(rintf(fminf(pr, 1.f) * kPScale));
                }
                uint32_t d[3];
                digits4(x, d);
#pragma unroll
                for (int k = 0; k < 3; ++k) pd[k][j] = d[k];
            }
            lt += xor_lane(lt, 16);
            lt += xor_lane(lt, 32);
            // join with what came before; a page that this column does not
            // see leaves everything as it is, whatever its scales are
            const float m_new = any ? fmaxf(m_run, ref) : m_run;
            const float keep = m_run == m_new ? 1.f : exp2f(m_run - m_new);
            const float add = any ? exp2f(ref - m_new) : 0.f;
            const float put = any ? add * (vs * (1.f / kPScale)) : 0.f;
            l_run = l_run * keep + (any ? add * lt : 0.f);
            m_run = m_new;
#pragma unroll
            for (int e = 0; e < ET; ++e) {
                const i32x4 vf = *reinterpret_cast<const i32x4*>(vp + (16 * e + col) * kPage + 16 * quad);
                i32x4 c[3];
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const i32x4 b = {static_cast<int>(pd[k][0]), static_cast<int>(pd[k][1]),
                                     static_cast<int>(pd[k][2]), static_cast<int>(pd[k][3])};
                    c[k] = __builtin_amdgcn_mfma_i32_16x16x64_i8(vf, b, i32x4{0, 0, 0, 0}, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float t = fmaf(static_cast<float>(c[2][i]), 65536.f,
                                         fmaf(static_cast<float>(c[1][i]), 256.f, static_cast<float>(c[0][i])));
                    o[e][i] = fmaf(t, put, o[e][i] * keep);
                }
            }
        }

        // the four waves' results
#pragma unroll
        for (int e = 0; e < ET; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[wave][col][16 * e + 4 * quad + i] = o[e][i];
        if (quad == 0) {
            stat[wave][col][0] = m_run;
            stat[wave][col][1] = l_run;
        }
        __syncthreads();
        const int64_t n = r.count * a.group;
        for (int i = threadIdx.x; i < kCols * D; i += 256) {
            const int cc = i / D, dim = i % D;
            const int64_t gc = tile * kCols + cc;
            if (gc >= n) continue;
            float m = stat[0][cc][0], l = 0.f, v = 0.f;
#pragma unroll
            for (int u = 1; u < 4; ++u) m = fmaxf(m, stat[u][cc][0]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float f = stat[u][cc][0] == m ? 1.f : exp2f(stat[u][cc][0] - m);
                l += f * stat[u][cc][1];
                v += f * acc[u][cc][dim];
            }
            const uint64_t at = static_cast<uint64_t>(r.first + gc / a.group) * a.heads + kvh * a.group + gc % a.group;
            if (a.pieces == 1) {
                const float res = l == 0.f ? 0.f : v / l;
                if constexpr (DT == QMV_F32) static_cast<float*>(a.out)[at * D + dim] = res;
                else static_cast<__bf16*>(a.out)[at * D + dim] = static_cast<__bf16>(res);
            } else {
                float* pp = a.part + (static_cast<uint64_t>(piece) * a.s.rows * a.heads + at) * (D + 2);
                pp[dim] = v;
                if (dim == 0) {
                    pp[D] = m;
                    pp[D + 1] = l;
                }
            }
        }
        __syncthreads();
    }
}

// Joins the pieces of each column: a workgroup has the 16 columns that the
// kernel before it had.
template <uint32_t DT, int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
    const uint32_t seq = blockIdx.x / a.c.kv_heads, kvh = blockIdx.x % a.c.kv_heads;
    const SeqRows r = seq_rows(a.s, seq);
    const int64_t n = r.count * a.group;
    const int64_t tiles = (n + kCols - 1) / kCols;
    const uint64_t step = static_cast<uint64_t>(a.s.rows) * a.heads * (D + 2);
    for (int64_t tile = blockIdx.y; tile < tiles; tile += gridDim.y) {
        for (int i = threadIdx.x; i < kCols * D; i += 256) {
            const int64_t gc = tile * kCols + i / D;
            const int dim = i % D;
            if (gc >= n) continue;
            const uint64_t at = static_cast<uint64_t>(r.first + gc / a.group) * a.heads + kvh * a.group + gc % a.group;
            const float* pp = a.part + at * (D + 2);
            float m = -__builtin_inff();
            for (uint32_t z = 0; z < a.pieces; ++z) m = fmaxf(m, pp[z * step + D]);
            float l = 0.f, v = 0.f;
            for (uint32_t z = 0; z < a.pieces; ++z) {
                const float mz = pp[z * step + D];
                const float f = mz == m ? 1.f : exp2f(mz - m);
                l += f * pp[z * step + D + 1];
                v += f * pp[z * step + dim];
            }
            const float res = l == 0.f ? 0.f : v / l;
            if constexpr (DT == QMV_F32) static_cast<float*>(a.out)[at * D + dim] = res;
            else static_cast<__bf16*>(a.out)[at * D + dim] = static_cast<__bf16>(res);
        }
    }
}

// The launch: tiles of 16 columns of a sequence and head, and pieces of its
// pages so that about two workgroups a compute unit run, with at least two
// pages for each wave of a piece.
struct Plan {
    uint32_t tiles, pieces;
};
Plan plan_few(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t heads, uint32_t window) {
    const uint64_t group = heads / c.kv_heads;
    const uint64_t most = s.max_new < s.rows ? (s.max_new == 0 ? 1 : s.max_new) : s.rows;
    uint64_t tiles = (most * group + kCols - 1) / kCols;
    if (tiles > 16384) tiles = 16384;
    uint64_t span = s.max_len;
    if (window != 0 && span > uint64_t{window} + kCols) span = uint64_t{window} + kCols;
    const uint64_t pages = (span + kPage - 1) / kPage + 1;
    const uint64_t wgs = uint64_t{s.seqs} * c.kv_heads * tiles;
    uint64_t pieces = (512 + wgs - 1) / wgs;
    if (pieces > (pages + 7) / 8) pieces = (pages + 7) / 8;
    if (pieces > 256) pieces = 256;
    if (pieces < 1) pieces = 1;
    return Plan{static_cast<uint32_t>(tiles), static_cast<uint32_t>(pieces)};
}

template <uint32_t DT, int D>
hipError_t go_few(const AttendArgs& a, const Plan& p, hipStream_t s) {
    const dim3 grid(a.s.seqs * a.c.kv_heads, p.tiles, p.pieces), block(256);
    hipLaunchKernelGGL((attend_few_kernel<DT, D>), grid, block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.pieces == 1) return e;
    hipLaunchKernelGGL((attend_join_kernel<DT, D>), dim3(grid.x, p.tiles), block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

uint64_t kv_attend_workspace_bytes(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t, uint32_t heads,
                                   uint32_t window) {
    const Plan p = plan_few(c, s, heads, window);
    if (p.pieces == 1) return 0;
    return uint64_t{p.pieces} * s.rows * heads * (c.head_dim + 2) * 4;
}

hipError_t launch_kv_attend(const qmv_kv_cache& c, const qmv_kv_seqs& s, uint32_t dtype, uint32_t heads,
                            float scale, uint32_t window, const void* q, void* out, void* workspace,
                            hipStream_t stream) {
    const Plan p = plan_few(c, s, heads, window);
    const AttendArgs a{c, s, q, out, static_cast<float*>(workspace), scale * kLog2e, heads,
                       heads / c.kv_heads, window, p.pieces};
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
