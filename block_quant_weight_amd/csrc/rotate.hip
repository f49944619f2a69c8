// Norm of each query and key head with the position's rotation.
//
// For a head of n values x: r = 1 / sqrt(sum x^2 / n + eps), y = (x r) w, then
// each pair (a, b) of the first `rot` channels, of frequency f, becomes
// (a c - b s, b c + a s) with c = m cos(p f), s = m sin(p f) for position p.
//
// A head is G neighbouring lanes of 8 channels each (G the power of two that
// holds head_dim), so it is read once, its squares are summed by lane
// exchanges, the partner of a channel half a rotation away is in another lane
// of the same wave, and it is written once.  A workgroup has one row: its
// first rot / 2 threads make the row's cosines and sines, once for all heads,
// into shared memory while the first heads are on their way from memory.  The
// angle p f is taken in 64 bits and reduced to a fraction of a turn there: at
// position 10^6 float32 would be 0.03 radians off.  Squares are summed in 64
// bits too, where they cannot overflow; all else is float32.
//
// Bound by memory: 8191 rows of 32 + 8 heads of 128, float32 to bfloat16 (252 MB),
// 52 us, 4.8 TB/s, the rate of a large copy; 1500 rows of 16 + 4 heads of 256 in
// bfloat16 (31 MB) 8.0 us in a graph, 3.8 TB/s, where the launch, the first trip
// and the row's sines count; one row 3.1 us.
#include "kv_common.h"

namespace qmv {
namespace {

#pragma clang fp contract(off)

constexpr int kThreads = 256;
// Workgroups that a launch aims at, a row's heads dealt out to several where rows
// are few (us with 1024, 256 and one a row, 16 + 4 heads of 256: 1 row 3.4, 3.4
// and 4.8; 64 rows 3.6, 3.6 and 5.1; 256 rows 4.3, 5.5 and 5.5; 4096 is as 1024).
constexpr uint32_t kRotateFull = 1024;

// Sum over G neighbouring lanes, in each of them.
template <int G>
__device__ __forceinline__ double group_sum(double v) {
#pragma unroll
    for (int m = 1; m < G; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// 1 / sqrt(v): the instruction's estimate and two of Newton's steps y (3 - v
// y^2) / 2, each of which doubles its correct bits.
__device__ __forceinline__ float root(double v) {
    double y = __builtin_amdgcn_rsq(v);
    if (v > 0.0 && v < __builtin_inf()) {
#pragma unroll
        for (int i = 0; i < 2; ++i) y = fma(0.5 * y, fma(-v * y, y, 1.0), y);
    }
    return static_cast<float>(y);
}

template <uint32_t IN, uint32_t OUT, int G, bool NEIGHBOURS>
__global__ __launch_bounds__(kThreads) void rotate_kernel(RotateArgs a) {
    typedef typename Elem<IN>::type TI;
    typedef typename Elem<OUT>::type TO;
    constexpr uint32_t kHeads = kThreads / G;    // heads of a turn
    __shared__ float2 turn[kThreads];
    const uint32_t tid = threadIdx.x, lane = tid & 63, sub = tid % G;
    const uint32_t half = a.rot / 2, all = a.q.heads + a.k.heads, at = 8 * sub;
    const bool live = at < a.head_dim;
    const uint32_t first = blockIdx.y * kHeads + tid / G, step = gridDim.y * kHeads;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        auto load = [&](uint32_t head, float* x) {
            const bool key = head >= a.q.heads;
            const TI* p = static_cast<const TI*>(key ? a.k.x : a.q.x) + row * (key ? a.k.x_stride : a.q.x_stride) +
                          static_cast<uint64_t>(key ? head - a.q.heads : head) * a.head_dim + at;
            if (head < all && live) {
                load8<IN>(p, x);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.f;
            }
        };
        float x[8];
        load(first, x);
        if (tid < half) {
            // the fraction of a turn, between -1/2 and 1/2
            const double t = static_cast<double>(a.pos[row]) * static_cast<double>(a.freq[tid]) * 0.15915494309189534;
            float s, c;
            sincospif(2.f * static_cast<float>(t - rint(t)), &s, &c);
            turn[tid] = make_float2(c * a.mscale, s * a.mscale);
        }
        __syncthreads();
        // this lane's cosines and sines (a channel that stays: 1 and 0)
        float c[8], s[8];
        const bool turned = at < a.rot, upper = turned && at >= half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t j = NEIGHBOURS ? (at + i) / 2 : (upper ? at - half : at) + i;
            const float2 v = turned ? turn[j] : make_float2(1.f, 0.f);
            c[i] = v.x;
            // (the pair's first channel takes - s times the second)
            s[i] = (NEIGHBOURS ? i % 2 == 0 : !upper) ? -v.y : v.y;
        }
        // (halves: the lane of the channel half a rotation away)
        const int partner = turned ? static_cast<int>(lane) + (upper ? -1 : 1) * static_cast<int>(half / 8) : static_cast<int>(lane);
        // (the loop's bound is the workgroup's, so that all lanes of a wave exchange)
        for (uint32_t base = blockIdx.y * kHeads; base < all; base += step) {
            const uint32_t head = base + tid / G;
            const bool key = head >= a.q.heads;
            float next[8];
            load(head + step, next);
            const float* w = key ? a.k.w : a.q.w;
            if (w != nullptr) {
                double sum = 0.0;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), sum);
                const float r = root(fma(group_sum<G>(sum), a.inv_dim, static_cast<double>(a.eps)));
                if (live) {
                    const float4 lo = reinterpret_cast<const float4*>(w + at)[0], hi = reinterpret_cast<const float4*>(w + at)[1];
                    const float u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = (x[i] * r) * u[i];
                }
            }
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float other = NEIGHBOURS ? x[i ^ 1] : __shfl(x[i], partner);
                y[i] = turned ? x[i] * c[i] + other * s[i] : x[i];
            }
            if (head < all && live) {
                TO* p = static_cast<TO*>(key ? a.k.y : a.q.y) + row * (key ? a.k.y_stride : a.q.y_stride) +
                        static_cast<uint64_t>(key ? head - a.q.heads : head) * a.head_dim + at;
                store8<OUT>(p, y);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = next[i];
        }
        __syncthreads();
    }
}

template <uint32_t IN, uint32_t OUT, bool NEIGHBOURS>
hipError_t go(const RotateArgs& a, hipStream_t s) {
    const int g = a.head_dim <= 64 ? 8 : (a.head_dim <= 128 ? 16 : (a.head_dim <= 256 ? 32 : 64));
    const uint32_t per = kThreads / g, turns = (a.q.heads + a.k.heads + per - 1) / per;
    // a row's heads are dealt out to several workgroups where rows are few
    uint32_t y = a.rows >= kRotateFull ? 1 : (kRotateFull + a.rows - 1) / a.rows;
    if (y > turns) y = turns;
    if (y > 65535) y = 65535;
    const dim3 grid(a.rows < (1u << 22) ? a.rows : (1u << 22), y), block(kThreads);
    if (g == 8) hipLaunchKernelGGL((rotate_kernel<IN, OUT, 8, NEIGHBOURS>), grid, block, 0, s, a);
    else if (g == 16) hipLaunchKernelGGL((rotate_kernel<IN, OUT, 16, NEIGHBOURS>), grid, block, 0, s, a);
    else if (g == 32) hipLaunchKernelGGL((rotate_kernel<IN, OUT, 32, NEIGHBOURS>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((rotate_kernel<IN, OUT, 64, NEIGHBOURS>), grid, block, 0, s, a);
    return hipGetLastError();
}
template <uint32_t IN, uint32_t OUT>
hipError_t go(const RotateArgs& a, hipStream_t s) {
    return a.neighbours != 0 ? go<IN, OUT, true>(a, s) : go<IN, OUT, false>(a, s);
}

}  // namespace

hipError_t launch_rotate(const RotateArgs& a, uint32_t dtype, uint32_t out_dtype, hipStream_t s) {
    if (dtype == QMV_F32) return out_dtype == QMV_F32 ? go<QMV_F32, QMV_F32>(a, s) : go<QMV_F32, QMV_BF16>(a, s);
    return out_dtype == QMV_F32 ? go<QMV_BF16, QMV_F32>(a, s) : go<QMV_BF16, QMV_BF16>(a, s);
}

}  // namespace qmv
