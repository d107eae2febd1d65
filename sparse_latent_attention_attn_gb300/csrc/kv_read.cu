// kv_read.cu -- rows of a paged cache of codes read back as bf16 rows.
//
// Value i of a row is code_i * 2^k, k the exponent of its block of 32: one f16 conversion of the code (exact), the
// power of two in f32 as two factors (exact for every k of an int8, whose extremes one factor would not hold), one
// rounding to bf16 (exact wherever bf16 holds the value: a code has at most four significant bits).
//
// Bound by HBM: 33/32 (17/32 in 4 bits) byte read and 2 written a value.  A block takes up to 64 rows: the
// first threads look up their slots, one dependent chain (list, page) for all of them, then every thread moves eight
// values a step, so that a warp stores 512 contiguous bytes, kSteps steps in flight.  Few rows are spread over more blocks.
// 16 x 4224 rows of 512 in 8 bits, whose bytes alone take 15.4 us: 18.1 us on the device (profiler, cold caches), 22.7 a call
// through the binding among others; 64 x 640 listed rows in 4 bits: 10.3 us such a call.
#include "paged_rows.cuh"
#include "row_norm.cuh"

namespace dsattn {
namespace {

using namespace rows;

constexpr int kMaxRows = 64;   // rows of a block
constexpr int kSteps = 4;

struct ReadArgs {
    const uint8_t *codes;
    const int8_t *exps;
    int64_t pages;
    Divisor page;
    const int32_t *block_table;
    int max_pages;
    const int32_t *idx, *first, *lens;
    uint16_t *y;
    uint32_t nrows;
    Divisor n;
    int per;                   // rows a block
    Divisor chunks;            // of a row
    unsigned int *status;
};

// Eight values of codes of BITS bits times 2^k, in f32.
template <int BITS>
struct Codes;
template <>
struct Codes<8> {
    using T = uint2;
    static __device__ __forceinline__ void f16(T c, uint32_t (&f)[4]) {
        const uint32_t w[2] = {c.x, c.y};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f[j]) : "h"((uint16_t)(w[j / 2] >> (16 * (j % 2)))));
    }
};
template <>
struct Codes<4> {
    using T = uint32_t;
    static __device__ __forceinline__ void f16(T c, uint32_t (&f)[4]) {
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
            : "r"(c));
    }
};

template <int BITS>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadArgs p) {
    using C = Codes<BITS>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int slot[kMaxRows];           // -1: zeros, -2: left as it is
    const uint32_t row0 = blockIdx.x * (uint32_t)p.per;
    if ((int)threadIdx.x < p.per) {
        const uint32_t row = row0 + threadIdx.x;
        int at = -2;
        if (row < p.nrows) {
            uint32_t i;
            const uint32_t bi = p.n.div(row, i);
            if (!p.lens || (int)i < __ldg(p.lens + bi)) {
                const int64_t r = p.idx ? (int64_t)__ldg(p.idx + row) : (p.first ? (int64_t)__ldg(p.first + bi) : 0) + i;
                bool bad = p.idx ? false : r < 0;
                at = -1;
                if (r >= 0) {
                    uint32_t off = 0;
                    const uint32_t pg = r <= INT32_MAX ? p.page.div((uint32_t)r, off) : UINT32_MAX;
                    const int id = pg < (uint32_t)p.max_pages ? __ldg(p.block_table + (int64_t)bi * p.max_pages + pg) : -1;
                    bad = id < 0 || id >= p.pages;
                    if (!bad) at = (int)((uint32_t)id * p.page.d + off);
                }
                if (bad) flag_status(p.status, DS_DEV_BAD_INDEX);
            }
        }
        slot[threadIdx.x] = at;
    }
    __syncthreads();
    const uint32_t units = (uint32_t)p.per * p.chunks.d, nblk = p.chunks.d / 4;
    for (uint32_t u0 = threadIdx.x; u0 < units; u0 += kThreads * kSteps) {
        typename C::T code[kSteps];
        int k[kSteps];
        int at[kSteps];
        uint32_t ch[kSteps], rw[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const uint32_t u = u0 + kThreads * i;
            rw[i] = p.chunks.div(u, ch[i]);
            at[i] = u < units ? slot[rw[i]] : -2;
            code[i] = {};
            k[i] = 0;
            if (at[i] >= 0) {
                code[i] = __ldg(reinterpret_cast<const typename C::T *>(p.codes) + (int64_t)at[i] * p.chunks.d + ch[i]);
                k[i] = __ldg(p.exps + (int64_t)at[i] * nblk + (ch[i] >> 2));
            }
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (at[i] == -2) continue;
            uint32_t f[4];
            C::f16(code[i], f);
            const int k1 = k[i] >> 1;
            const float s1 = __uint_as_float((uint32_t)(k1 + 127) << 23), s2 = __uint_as_float((uint32_t)(k[i] - k1 + 127) << 23);
            float x[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[2 * j] = __half2float(__ushort_as_half((unsigned short)(f[j] & 0xffffu))) * s1 * s2;
                x[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(f[j] >> 16))) * s1 * s2;
            }
            reinterpret_cast<uint4 *>(p.y)[(int64_t)(row0 + rw[i]) * p.chunks.d + ch[i]] = pack8(x);
        }
    }
}

template <int BITS>
int launch(const ReadCall &a, cudaStream_t stream) {
    ReadArgs p{a.codes, a.exps, a.pages, Divisor((uint32_t)a.page), a.block_table, a.max_pages, a.idx, a.first, a.lens, a.y,
               (uint32_t)((int64_t)a.b * a.n), Divisor((uint32_t)a.n), kMaxRows, Divisor((uint32_t)a.d / 8), a.status};
    // fewer rows a block until there are enough blocks for every SM (a GB300 has 152), but work for all its threads
    while (p.per > 1 && p.nrows / (uint32_t)p.per < 1024 && p.per * a.d / 8 > kThreads) p.per /= 2;
    kv_read_kernel<BITS><<<(p.nrows - 1) / (uint32_t)p.per + 1, kThreads, 0, stream>>>(p);
    return launch_status();
}

}  // namespace

int launch_kv_read_fp4(const ReadCall &a, cudaStream_t stream) { return launch<4>(a, stream); }
int launch_kv_read_fp8(const ReadCall &a, cudaStream_t stream) { return launch<8>(a, stream); }

}  // namespace dsattn
