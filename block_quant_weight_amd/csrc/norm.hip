// Root-mean-square norm with the residual's addition, in the forms that the
// products take (float32, bfloat16, Q8_0 blocks of 32).
//
// For a row of n values: h = x + res, r = 1 / sqrt(sum h^2 / n + eps),
// y = (h r) w; with Q8_0 output, per block of 32: d = amax / 127, q =
// trunc(y (127 / amax) + copysign(0.5, y)), the activation quantizer's rule.
//
// One pass over the row: a workgroup keeps it in registers (float4 i * NT +
// tid of the row in thread tid), so x and res are read once and every output
// is written from the same values.  The squares are summed in 64 bits (h^2
// is exact there), because a code lies next to a border where a last-bit
// difference of r moves it by a whole step; r and everything after it is
// float32, each operation rounded on its own, so codes do not depend on how
// a row is split over threads.  A block of 32 is eight neighbouring lanes'
// float4s: its amax is three lane exchanges.
//
// Bound by memory: 8191 x 4096 with residual and bfloat16 output 78 us, 6.0
// TB/s (a copy of a large array reaches 5.0); 512 x 4096 to Q8_0 8.6 us, 3.2
// TB/s, where the launch and one trip to memory count; one row 3.1 us, the
// same two and the sum over the workgroup.
#include "device_common.h"
#include "serve_kernels.h"

namespace qmv {
namespace {

#pragma clang fp contract(off)

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

__device__ __forceinline__ uint32_t abs_bits(float v) {
    return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}

// Loads and stores; with NT past the caches.
template <bool NT, typename V>
__device__ __forceinline__ V get(const V* p) {
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool NT, typename V>
__device__ __forceinline__ void set(V* p, V v) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// Writes float4 `i` of row `row` of every output after the sum.
template <bool NT>
__device__ __forceinline__ void put(const NormArgs& a, uint64_t row, uint32_t i, f32x4 h, float r) {
    const f32x4 w = reinterpret_cast<const f32x4*>(a.w)[i];
    const f32x4 y = (h * r) * w;
    const uint64_t at = row * a.cols + 4ull * i;
    if (a.y != nullptr) set<NT>(reinterpret_cast<f32x4*>(a.y + at), y);
    if (a.y_bf16 != nullptr) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        const bf16x4 b = {static_cast<__bf16>(y[0]), static_cast<__bf16>(y[1]),
                          static_cast<__bf16>(y[2]), static_cast<__bf16>(y[3])};
        set<NT>(reinterpret_cast<uint64_t*>(a.y_bf16 + at), __builtin_bit_cast(uint64_t, b));
    }
    if (a.q != nullptr) {
        // largest magnitude of the block, as bits: infinities and NaNs are
        // the largest of all
        const float v[4] = {y[0], y[1], y[2], y[3]};
        uint32_t m = max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3])));
        m = max(m, dpp_u32<0xB1>(m));   // lanes 1 apart
        m = max(m, dpp_u32<0x4E>(m));   // 2 apart
        m = max(m, dpp_u32<0x141>(m));  // half row mirrored: the other four
        const float amax = __builtin_bit_cast(float, m);
        float d = 0.f;
        uint32_t word = 0;
        if (m >= 0x7F800000u) {
            d = __builtin_nanf("");
        } else if (!(amax < 1e-30f)) {
            d = amax / 127.0f;
            const float id = 127.0f / amax;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float t = v[c] * id;
                const float u = truncf(t + copysignf(0.5f, v[c]));
                const int q = static_cast<int>(fminf(fmaxf(u, -127.f), 127.f));
                word |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * c);
            }
        }
        set<NT>(reinterpret_cast<uint32_t*>(a.q + at), word);
        if ((i & 7) == 0) a.d[at >> 5] = d;
    }
}

// 1 / sqrt(sum / cols + eps): the instruction's estimate and two of Newton's
// steps y (3 - v y^2) / 2, each of which doubles its correct bits (a division
// and a square root in 64 bits take several times as long, in every thread).
__device__ __forceinline__ float inv_rms(double sum, double inv_cols, float eps) {
    const double v = fma(sum, inv_cols, static_cast<double>(eps));
    double y = __builtin_amdgcn_rsq(v);
    if (v > 0.0 && v < static_cast<double>(__builtin_inff())) {
#pragma unroll
        for (int i = 0; i < 2; ++i) y = fma(0.5 * y, fma(-v * y, y, 1.0), y);
    }
    return static_cast<float>(y);
}

// NT threads a row, at most V float4s in each; LOOP: any length, the row's h
// read again for the outputs.  PAST: past the caches.
template <int NT, int V, bool LOOP, bool PAST>
__global__ __launch_bounds__(NT) void rms_norm_kernel(NormArgs a) {
    __shared__ double part[2][NT / 64];
    const uint32_t n4 = a.cols >> 2;
    const int tid = threadIdx.x;
    int flip = 0;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const f32x4* xp = reinterpret_cast<const f32x4*>(a.x + row * a.cols);
        const f32x4* rp = a.res != nullptr ? reinterpret_cast<const f32x4*>(a.res + row * a.cols) : nullptr;
        f32x4* sp = a.sum != nullptr ? reinterpret_cast<f32x4*>(a.sum + row * a.cols) : nullptr;
        f32x4 h[V];
        double s = 0.0;
        auto load = [&](uint32_t i) {
            f32x4 v = get<PAST>(xp + i);
            if (rp != nullptr) v = v + get<PAST>(rp + i);
            return v;
        };
        auto square = [&](const f32x4& v) {
            const double p = v[0], q = v[1], u = v[2], w = v[3];
            s += (p * p + q * q) + (u * u + w * w);
        };
        if constexpr (LOOP) {
            for (uint32_t i = tid; i < n4; i += NT) {
                const f32x4 v = load(i);
                square(v);
                if (sp != nullptr) sp[i] = v;
            }
        } else {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const uint32_t i = u * NT + tid;
                h[u] = i < n4 ? load(i) : f32x4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int u = 0; u < V; ++u) {
                square(h[u]);
                const uint32_t i = u * NT + tid;
                if (sp != nullptr && i < n4) set<PAST>(sp + i, h[u]);
            }
        }
        s = wave_sum(s);
        if constexpr (NT > 64) {
            if ((tid & 63) == 0) part[flip][tid >> 6] = s;
            __syncthreads();  // the other buffer is written before the next one
            s = 0.0;
#pragma unroll
            for (int w = 0; w < NT / 64; ++w) s += part[flip][w];
        }
        const float r = inv_rms(s, a.inv_cols, a.eps);
        if constexpr (LOOP) {
            // the sum may have replaced res or x: each thread reads back the
            // elements it wrote itself
            for (uint32_t i = tid; i < n4; i += NT) put<PAST>(a, row, i, sp != nullptr ? sp[i] : load(i), r);
        } else {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const uint32_t i = u * NT + tid;
                if (i < n4) put<PAST>(a, row, i, h[u], r);
            }
        }
    }
}

template <int NT, int V, bool LOOP>
hipError_t go(const NormArgs& a, hipStream_t s) {
    const uint32_t grid = a.rows < (1u << 20) ? a.rows : (1u << 20);
    // Arrays of 64 MB or more will not be found in the caches by the next
    // kernel: they go past them (8191 x 4096: 78 us, else 88).  A row too
    // long for registers is read twice, through the caches.
    if (!LOOP && uint64_t{a.rows} * a.cols * 4 >= (64u << 20))
        hipLaunchKernelGGL((rms_norm_kernel<NT, V, LOOP, !LOOP>), dim3(grid), dim3(NT), 0, s, a);
    else
        hipLaunchKernelGGL((rms_norm_kernel<NT, V, LOOP, false>), dim3(grid), dim3(NT), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
    // Two float4s a thread: 8191 x 4096 with residual and bfloat16 output 88
    // us, one 93, four 95, eight 104; one row of 4096 3.1, 3.1, 3.9 and 5.4.
    if (a.cols <= 512) return go<64, 2, false>(a, s);
    if (a.cols <= 1024) return go<128, 2, false>(a, s);
    if (a.cols <= 2048) return go<256, 2, false>(a, s);
    if (a.cols <= 4096) return go<512, 2, false>(a, s);
    if (a.cols <= 8192) return go<1024, 2, false>(a, s);
    if (a.cols <= 16384) return go<1024, 4, false>(a, s);
    return go<1024, 1, true>(a, s);
}

}  // namespace qmv
