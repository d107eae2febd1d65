// kv_append_fp4.cu -- new latent rows into a paged cache of 4-bit codes, normalised and rotated on the way.
//
// "DeepSeek V4.1", attention/query-latent: kv_norm and apply_rotary_emb on the KV row, the ring slot of a
// window row, one compressed row for each `ratio` positions (rotated to its first position).  "Module
// attn": a power-of-two scale per block of 32 with amax floored at 1e-4.  The 4-bit values (e2m1) and the
// pages are this library's: with z the row after norm and rotation, per block of 32
//     k = ceil(log2(max(amax, 1e-4) / 6)),  code_i = e2m1(z_i / 2^k), nearest, ties to the even code.
//
// A code is a decision, so it is made on the exact z: the f32 value is within 2^-21 of the magnitudes it
// was made of (each product and sum below rounds by 2^-24; the norm factor comes from a sum carried in
// two floats and one Newton step).  A value that near to a border between two codes (or a maximum that
// near to a power of two times 6) sends its warp through the same formula in 64 bits: about one row of
// 512 in a thousand.  Rows that are neither normalised nor rotated are exact in f32.
//
// Bound by HBM (2 bytes read, 17/32 written a value, 2 more with y) and at decode sizes by latency: one
// row a warp (half or a quarter for short rows), 16 bytes a lane and step; a block's maximum is two
// shuffles over its four lanes, and a warp stores 128 contiguous bytes of codes.
#include "row_norm.cuh"

namespace dsattn {
namespace {

using namespace rows;

struct AppendArgs {
    const uint16_t *x;
    int64_t x_bstride, x_tstride;
    uint16_t *y;
    uint32_t ntok;
    int s, d, rd;
    const float *weight;
    float eps;                 // 0: no norm
    const float2 *table;
    int64_t table_rows;
    const int32_t *first, *lens;
    int pos_step, base, window;
    uint8_t *codes;
    int8_t *exps;
    int64_t pages;
    int page;
    const int32_t *block_table;
    int max_pages;
    unsigned int *status;
};

// s + e == a + b exactly.
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
    s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

// 1 / sqrt(hi + lo) within 2^-24 of itself: the library's value and one Newton step whose residual is
// formed with fused products.
__device__ __forceinline__ float rsqrt_near(float hi, float lo) {
    const float r = 1.0f / sqrtf(hi);
    const float t = __fmul_rn(r, r), te = fmaf(r, r, -t);
    const float e = -fmaf(lo, t, fmaf(hi, te, fmaf(hi, t, -1.0f)));   // 1 - (hi + lo) r^2
    return fmaf(r, 0.5f * e, r);
}

// Exponent k of a block: the smallest with amax <= 6 * 2^k, from amax's IEEE fields (6 = 1.5 * 4).
__device__ __forceinline__ int block_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    return (int)(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x400000u ? 2 : 1);
}

__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// Two codes in a byte, lo in the low nibble; nearest, ties to even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
        "cvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// Whether |v| is within tol of a border between two codes.
__device__ __forceinline__ bool near_border(float v, float tol) {
    const float a = fabsf(v);
    // borders 0.25, 0.75, 1.25, 1.75 | 2.5, 3.5 | 5: the nearest border of each part
    const float b = a < 2.125f ? fminf(floorf(2.0f * a) * 0.5f + 0.25f, 1.75f) : a < 4.25f ? (a < 3.0f ? 2.5f : 3.5f) : 5.0f;
    return fabsf(a - b) <= tol;
}

// The value a code of block exponent k stands for.
__device__ __forceinline__ float code_value(uint32_t code, float sc) {
    const uint32_t m = code & 7u;
    const float a = m < 4u ? 0.5f * (float)m : m == 7u ? 6.0f : (float)(m - 2u);
    return (code & 8u ? -a : a) * sc;
}

__device__ __forceinline__ uint32_t code_of(double v) {
    const double a = fabs(v);
    const uint32_t m = (a > 0.25) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0);
    return m | (signbit(v) ? 8u : 0u);
}

// One chunk of the row in 64 bits: norm (factor r), weight, rotation.
__device__ __noinline__ void chunk64(const uint4 v, double r, const float *w, const float2 *cs, double (&z)[8]) {
    float x[8];
    unpack8(v, x);
    for (int i = 0; i < 8; ++i) z[i] = (double)x[i] * r * (w ? (double)w[i] : 1.0);
    if (cs)
        for (int j = 0; j < 4; ++j) {
            const double a = z[2 * j], b = z[2 * j + 1], c = cs[j].x, s = cs[j].y;
            z[2 * j] = a * c - b * s;
            z[2 * j + 1] = a * s + b * c;
        }
}

template <int L, int N>
__global__ void __launch_bounds__(kThreads) kv_append_fp4_kernel(const AppendArgs p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tok = blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const int lane = threadIdx.x % L;
    const uint32_t bi = tok / (uint32_t)p.s, t = tok - bi * (uint32_t)p.s;
    bool live = tok < p.ntok;
    bool stored = false;
    int64_t pos = 0, slot = 0;
    if (live) {
        const int len = p.lens ? min(__ldg(p.lens + bi), p.s) : p.s;
        const int64_t i = (int64_t)__ldg(p.first + bi) + t;
        live = (int)t < len;
        stored = live && (p.window == 0 || (int)t >= len - p.window);
        bool bad = false;
        if (live) {
            pos = i * p.pos_step;
            if (i < 0 || i > INT32_MAX || (p.rd && pos >= p.table_rows)) {
                bad = true;
                live = stored = false;
            }
        }
        if (stored) {
            const uint32_t r = (uint32_t)p.base + (p.window ? (uint32_t)i % (uint32_t)p.window : (uint32_t)i);
            const uint32_t pg = r / (uint32_t)p.page;
            const int id = pg < (uint32_t)p.max_pages ? __ldg(p.block_table + (int64_t)bi * p.max_pages + pg) : -1;
            slot = (int64_t)id * p.page + (r - pg * (uint32_t)p.page);
            if (id < 0 || id >= p.pages) {
                bad = true;
                stored = false;
            }
        }
        if (bad && lane == 0) flag_status(p.status, DS_DEV_BAD_INDEX);
    }
    live = live && (stored || p.y);
    const int nch = p.d / 8, nblk = p.d / 32;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.x + (int64_t)bi * p.x_bstride + (int64_t)t * p.x_tstride);
    uint4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = live && lane + L * i < nch ? src[lane + L * i] : make_uint4(0, 0, 0, 0);
    const bool norm = p.eps > 0.0f;
    float r = 1.0f;
    if (norm) {
        // squares of bf16 values are exact in f32; their sum is carried in two floats
        float hi = 0.0f, lo = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x[8];
            unpack8(v[i], x);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float s, e;
                two_sum(hi, __fmul_rn(x[k], x[k]), s, e);
                hi = s;
                lo = __fadd_rn(lo, e);
            }
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            const float h2 = __shfl_xor_sync(kAll, hi, o), l2 = __shfl_xor_sync(kAll, lo, o);
            float s, e;
            two_sum(hi, h2, s, e);
            hi = s;
            lo = __fadd_rn(__fadd_rn(lo, l2), e);
        }
        // (hi + lo) / d + eps: the quotient's remainder goes to the low part
        const float dd = (float)p.d;
        const float q = __fdiv_rn(hi, dd);
        const float ql = __fdiv_rn(__fadd_rn(fmaf(-q, dd, hi), lo), dd);
        float s, e;
        two_sum(q, p.eps, s, e);
        r = rsqrt_near(s, __fadd_rn(ql, e));
    }
    const int rot = (p.d - p.rd) / 8;
    const float2 *cs = p.table + pos * (p.rd / 2);
    uint32_t code[N];
    int kexp[N];
    bool near = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = lane + L * i;
        const bool in = live && c < nch;
        float x[8], mag[8];   // a value, and the magnitudes it was made of
        unpack8(v[i], x);
        if (in && norm) scale8(x, r, p.weight ? p.weight + c * 8 : nullptr);
        const bool turned = in && c >= rot;
        if (turned) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 cj = __ldg(cs + (c - rot) * 4 + j);
                const float a = x[2 * j], b = x[2 * j + 1];
                x[2 * j] = a * cj.x - b * cj.y;
                x[2 * j + 1] = a * cj.y + b * cj.x;
                mag[2 * j] = mag[2 * j + 1] = (fabsf(a) + fabsf(b)) * fmaxf(fabsf(cj.x), fabsf(cj.y));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) mag[j] = fabsf(x[j]);
        }
        float amax = 0.0f, most = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            amax = fmaxf(amax, fabsf(x[j]));
            most = fmaxf(most, mag[j]);
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
            most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
        }
        amax = fmaxf(amax, 1e-4f);
        const int k = block_exp(amax);
        const float inv = pow2(-k);
        kexp[i] = k;
        uint32_t cw = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) cw |= e2m1x2(x[2 * j] * inv, x[2 * j + 1] * inv) << (8 * j);
        code[i] = cw;
        if (in && (norm || turned)) {
            const float tol = 4.76837158e-7f * inv;   // 2^-21, in units of the block's scale
            const float top = amax * inv;             // in (3, 6]
            near |= top >= 6.0f - tol * most || top <= 3.0f + tol * most;
#pragma unroll
            for (int j = 0; j < 8; ++j) near |= near_border(x[j] * inv, tol * mag[j]);
        }
    }
    if (__any_sync(kAll, near)) {
        double r64 = 1.0;
        if (norm) {
            double ss = 0.0;
            for (int i = 0; i < N; ++i) {
                float x[8];
                unpack8(v[i], x);
                for (int k = 0; k < 8; ++k) ss += (double)x[k] * (double)x[k];
            }
            ss = row_sum<L>(ss);
            r64 = 1.0 / sqrt(ss / (double)p.d + (double)p.eps);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = lane + L * i;
            const bool in = live && c < nch;
            double z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (in)
                chunk64(v[i], r64, norm && p.weight ? p.weight + c * 8 : nullptr,
                        c >= rot ? cs + (c - rot) * 4 : nullptr, z);
            double amax = 0.0;
            for (int j = 0; j < 8; ++j) amax = fmax(amax, fabs(z[j]));
            amax = fmax(amax, __shfl_xor_sync(kAll, amax, 1));
            amax = fmax(amax, __shfl_xor_sync(kAll, amax, 2));
            amax = fmax(amax, 1e-4);
            int k = ilogb(amax) - 2;                 // amax in [4, 8) * 2^k
            if (amax > 6.0 * scalbn(1.0, k)) ++k;
            uint32_t cw = 0;
            for (int j = 0; j < 8; ++j) cw |= code_of(z[j] * scalbn(1.0, -k)) << (4 * j);
            kexp[i] = k;
            code[i] = cw;
        }
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = lane + L * i;
        if (c >= nch) continue;
        if (stored) {
            reinterpret_cast<uint32_t *>(p.codes)[slot * nch + c] = code[i];
            if ((c & 3) == 0) p.exps[slot * nblk + (c >> 2)] = (int8_t)kexp[i];
        }
        if (p.y) {
            const float sc = pow2(kexp[i]);
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = code_value((code[i] >> (4 * j)) & 15u, sc);
            reinterpret_cast<uint4 *>(p.y + (int64_t)tok * p.d)[c] = pack8(x);
        }
    }
}

}  // namespace

int launch_kv_append_fp4(const uint16_t *x, int64_t x_bstride, int64_t x_tstride, uint16_t *y, int b, int s, int d,
                         const float *weight, float eps, int rd, const float *table, int64_t table_rows,
                         const int32_t *first, const int32_t *lens, int pos_step, int base, int window, uint8_t *codes,
                         int8_t *exps, int64_t pages, int page, const int32_t *block_table, int max_pages,
                         unsigned int *status, cudaStream_t stream) {
    const AppendArgs p{x, x_bstride, x_tstride, y, (uint32_t)((int64_t)b * s), s, d, rd, weight, eps,
                       reinterpret_cast<const float2 *>(table), table_rows, first, lens, pos_step, base, window,
                       codes, exps, pages, page, block_table, max_pages, status};
    for_row(d, [&](auto l, auto n) {
        constexpr int L = decltype(l)::value;
        const uint32_t per = kThreads / L;
        kv_append_fp4_kernel<L, decltype(n)::value><<<(p.ntok + per - 1) / per, kThreads, 0, stream>>>(p);
    });
    return launch_status();
}

}  // namespace dsattn
