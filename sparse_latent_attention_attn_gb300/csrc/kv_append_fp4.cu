// kv_append_fp4.cu -- the append (kv_append.cuh) in the 4-bit format: e2m1 codes, two to a byte (the even value in the low
// nibble), scale 2^k with k = ceil(log2(max(amax, 1e-4) / 6)).
//
// HBM has 2 bytes read and 17/32 written a value, 2 more with y; no pipe is full in long batches (the
// integer pipe 0.69 of its rate, issue 0.67 a cycle and scheduler, 43 % of the warps: 650 instructions a row, in chains
// of conversions, byte permutes, maxima and exponents), decode sizes are bound by latency.  Two rows of 512 in a thousand
// go through the exact path.
// Measured: 8 x 4096 rows of 512 with y, 28.7 us (650 instructions a row; its bytes alone 12.4 us; with three blocks of
// 72 registers an SM 33.3, with five of 48 30.8); 256 rows into rings 5.1 us a call in a graph.
#include "kv_append.cuh"

namespace dsattn {
namespace {

struct E2m1 {
    using Codes = uint32_t;
    static constexpr int kBorderBits = 2;

    // Exponent k of a block: the smallest with amax <= 6 * 2^k, from amax's IEEE fields (6 = 1.5 * 4).
    static __device__ __forceinline__ int block_exp(float amax) {
        const uint32_t u = __float_as_uint(amax);
        return (int)(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x400000u ? 2 : 1);
    }

    // Eight codes of z, the first in the lowest nibble; nearest, ties to even, saturating at 6.
    static __device__ __forceinline__ uint32_t codes8(const uint64_t (&zz)[4]) {
        float z[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) unpair(zz[j], z[2 * j], z[2 * j + 1]);
        uint32_t r;
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(r)
            : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
        return r;
    }

    // The values that eight codes stand for at scale sc.
    static __device__ __forceinline__ void values8(uint32_t c, float sc, float (&x)[8]) {
        uint32_t f[4];
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
            : "r"(c));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __half2float(__ushort_as_half((unsigned short)(f[j] & 0xffffu))) * sc;
            x[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(f[j] >> 16))) * sc;
        }
    }
};

}  // namespace

int launch_kv_append_fp4(const AppendCall &a, cudaStream_t stream) { return append::launch<E2m1>(append::AppendArgs(a), stream); }

}  // namespace dsattn
