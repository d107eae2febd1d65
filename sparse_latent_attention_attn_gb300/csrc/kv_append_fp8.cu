// kv_append_fp8.cu -- the append (kv_append.cuh) in the 8-bit format: e4m3 codes, scale 2^k with
// k = ceil(log2(max(amax, 1e-4) / 448)): "Module attn", act_quant_inplace and pow2_ceil.
//
// Bound by instructions, as in 4 bits (two thirds of the issue slots, no pipe full): 32 us for 8 x 4096 rows of 512, whose
// bytes alone would take 13.7; 256 rows 14.5 us a call through the binding among others, bound by the host.
#include "kv_append.cuh"

namespace dsattn {
namespace {

struct E4m3 {
    using Codes = uint64_t;
    static constexpr int kBorderBits = 4;

    // Exponent k of a block: the smallest with amax <= 448 * 2^k, from amax's IEEE fields (448 = 1.75 * 256).
    static __device__ __forceinline__ int block_exp(float amax) {
        const uint32_t u = __float_as_uint(amax);
        return (int)(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7);
    }

    // Eight codes of z, the first in the lowest byte; nearest, ties to even, saturating at 448.
    static __device__ __forceinline__ uint64_t codes8(const uint64_t (&zz)[4]) {
        float z[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) unpair(zz[j], z[2 * j], z[2 * j + 1]);
        uint64_t r;
        asm("{\n\t.reg .b16 h0, h1, h2, h3;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 h0, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 h1, %4, %3;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 h2, %6, %5;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 h3, %8, %7;\n\t"
            "mov.b64 %0, {h0, h1, h2, h3};\n\t}"
            : "=l"(r)
            : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
        return r;
    }

    // The values that eight codes stand for at scale sc.
    static __device__ __forceinline__ void values8(uint64_t c, float sc, float (&x)[8]) {
        uint32_t f[4];
        asm("{\n\t.reg .b16 h0, h1, h2, h3;\n\t"
            "mov.b64 {h0, h1, h2, h3}, %4;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, h0;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, h1;\n\t"
            "cvt.rn.f16x2.e4m3x2 %2, h2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %3, h3;\n\t}"
            : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
            : "l"(c));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __half2float(__ushort_as_half((unsigned short)(f[j] & 0xffffu))) * sc;
            x[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(f[j] >> 16))) * sc;
        }
    }
};

}  // namespace

int launch_kv_append_fp8(const AppendCall &a, cudaStream_t stream) { return append::launch<E4m3>(append::AppendArgs(a), stream); }

}  // namespace dsattn
