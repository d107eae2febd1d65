// row_norm.cuh -- what the kernels over rows of bf16 values at positions share: the lanes of a row,
// its chunks of 8 values, the norm factor and the rotation in f32.
//
// A row of d values (d % 8 == 0, d <= 1024) is d / 8 chunks of 16 bytes.  L = 8, 16 or 32 lanes share a
// row; lane l of them holds chunks l, l + L, ..., so that a warp's accesses are contiguous.
#pragma once

#include "common.cuh"

namespace dsattn {
namespace rows {

constexpr int kThreads = 256;
constexpr uint32_t kAll = 0xffffffffu;

// Calls f(integral constants L, N) for a row of d values: its lanes and the chunks of a lane.
template <int V>
struct Int {
    static constexpr int value = V;
};
template <typename F>
void for_row(int d, F f) {
    if (d <= 64) f(Int<8>(), Int<1>());
    else if (d <= 128) f(Int<16>(), Int<1>());
    else if (d <= 256) f(Int<32>(), Int<1>());
    else if (d <= 512) f(Int<32>(), Int<2>());
    else f(Int<32>(), Int<4>());
}

__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// n / d and n % d for n < 2^32 with m = floor((2^32 - 1) / d) from the host: the product's high word is the
// quotient or one less.
struct Divisor {
    uint32_t d, m;
    explicit Divisor(uint32_t v = 1) : d(v), m(0xffffffffu / v) {}
    __device__ __forceinline__ uint32_t div(uint32_t n, uint32_t &rest) const {
        uint32_t q = __umulhi(n, m);
        rest = n - q * d;
        if (rest >= d) {
            rest -= d;
            ++q;
        }
        return q;
    }
};

// 1 / sqrt(ss / d + eps) from inv_d = 1 / d rounded, within 5 * 2^-24 of it: half of two roundings, and the two units
// in the last place that rsqrtf's documentation allows.
__device__ __forceinline__ float norm_factor(float ss, float inv_d, float eps) { return rsqrtf(fmaf(ss, inv_d, eps)); }

// Sum over the L lanes of a row; every lane gets it.
template <int L, typename T>
__device__ __forceinline__ T row_sum(T v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// The chunk's values times the row's factor and the weights of its columns (w: f32 [8], 16-byte aligned, or
// null).
__device__ __forceinline__ void scale8(float (&x)[8], float r, const float *__restrict__ w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], r);
    if (w) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(w)), b = __ldg(reinterpret_cast<const float4 *>(w) + 1);
        const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], f[i]);
    }
}

// Four adjacent pairs (a, b) turned by cs[j] = (cos, sin): (a c - b s, a s + b c).  Stays in f32: the
// result is rounded once, by whoever stores it.
__device__ __forceinline__ void rotate8(float (&x)[8], const float2 *__restrict__ cs) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 t = __ldg(cs + j);
        const float a = x[2 * j], b = x[2 * j + 1];
        x[2 * j] = a * t.x - b * t.y;
        x[2 * j + 1] = a * t.y + b * t.x;
    }
}

}  // namespace rows
}  // namespace dsattn
