// kv_append_fp4.cu -- new latent rows into a paged cache of 4-bit codes, normalised and rotated on the way.
//
// "DeepSeek V4.1", attention/query-latent: kv_norm and apply_rotary_emb on the KV row, the ring slot of a
// window row, one compressed row for each `ratio` positions (rotated to its first position).  "Module
// attn": a power-of-two scale per block of 32 with amax floored at 1e-4.  The 4-bit values (e2m1) and the
// pages are this library's: with z the row after norm and rotation, per block of 32
//     k = ceil(log2(max(amax, 1e-4) / 6)),  code_i = e2m1(z_i / 2^k), nearest, ties to the even code.
//
// A code is a decision, so it is made on the exact z.  The f32 value is off by less than t of the magnitudes it was
// made of.  Its roundings, in units of 2^-24: half of those in the longest chain into the sum of squares, of N
// chunks a lane (2 N - 1 products and sums, the first square exact, 2 + 5 sums of a lane's and the lanes' parts): 5 for
// N <= 2, 7 for N = 4; 5 for the factor 1 / sqrt(ss / d + eps); two products; two for the rotation; and one for z + t
// itself: 15 for rows of up to 512, t = 16, and 17 above, t = 32.  So the codes of z + t and z - t are formed;
// where they are the same (and the block's exponent is for its maximum + t and - t) they are z's, and where a
// border lies between them the warp goes through the formula with two floats a number (to about 2^-44): two rows
// of 512 in a thousand.  Rows that are neither normalised nor rotated are exact in f32 (t = 0).
//
// HBM has 2 bytes read and 17/32 written a value, 2 more with y; no pipe is full in long batches (the
// integer pipe 0.69 of its rate, issue 0.67 a cycle and scheduler, 43 % of the warps: 650 instructions a row, in chains
// of conversions, byte permutes, maxima and exponents), decode sizes are bound by latency.  One row a warp (half
// or a quarter for short rows), 16 bytes a lane and step; a block's maximum is two shuffles over its four lanes,
// and a warp stores 128 contiguous bytes of codes.  Several rows a warp with the next one's loads ahead took as
// long or longer (four 31.5 us, two 38.2), for their registers.
// Measured: 8 x 4096 rows of 512 with y, 28.7 us (650 instructions a row; its bytes alone 12.4 us); 256 rows into
// rings 5.1 us a call in a graph.
#include "f32x2.cuh"
#include "paged_rows.cuh"
#include "row_norm.cuh"

namespace dsattn {
namespace {

using namespace rows;

struct AppendArgs {
    const uint16_t *x;
    int64_t x_bstride, x_tstride;
    uint16_t *y;
    uint32_t ntok;
    Divisor s;
    int d, rd;
    const float *weight;
    float inv_d, eps;          // eps 0: no norm
    const float2 *table;
    int64_t table_rows;
    const int32_t *first, *lens;
    int pos_step, base;
    Divisor window;            // d 0: none
    uint8_t *codes;
    int8_t *exps;
    int64_t pages;
    Divisor page;
    const int32_t *block_table;
    int max_pages;
    unsigned int *status;
};

// Exponent k of a block: the smallest with amax <= 6 * 2^k, from amax's IEEE fields (6 = 1.5 * 4).
__device__ __forceinline__ int block_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    return (int)(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x400000u ? 2 : 1);
}

__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// The eight values of a chunk in four pairs.
__device__ __forceinline__ void unpack_pairs(const uint4 v, uint64_t (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = pair(bf16_lo(w[j]), bf16_hi(w[j]));
}

// Eight codes of z, the first in the lowest nibble; nearest, ties to even, saturating at 6.
__device__ __forceinline__ uint32_t codes8(const uint64_t (&zz)[4]) {
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
__device__ __forceinline__ void values8(uint32_t c, float sc, float (&x)[8]) {
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

// ---- the same in two floats (hi + lo, good to about 2^-44), for values next to a border ----

// s + e == a + b exactly (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
    s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

struct F2 {
    float hi, lo;
};
__device__ __forceinline__ F2 times(F2 a, float b) {
    const float h = __fmul_rn(a.hi, b);
    return {h, fmaf(a.lo, b, fmaf(a.hi, b, -h))};
}
__device__ __forceinline__ F2 plus(F2 a, F2 b) {
    F2 r;
    float e;
    two_sum(a.hi, b.hi, r.hi, e);
    r.lo = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
    return r;
}

// One float that rounds like hi + lo: hi, but one unit in its last place towards lo where hi may lie on a border
// itself.  Borders (and 6 times a power of two) have at most two mantissa bits, and a unit in the last
// place moves no other such value across one.
__device__ __forceinline__ float one_float(F2 a) {
    if (a.lo == 0.0f) return a.hi;               // (a zero keeps its sign)
    float h, l;
    two_sum(a.hi, a.lo, h, l);
    const uint32_t u = __float_as_uint(h);
    if ((u & 0x1fffffu) != 0 || l == 0.0f) return h;
    return __uint_as_float((l > 0.0f) == (h > 0.0f) ? u + 1 : u - 1);
}

// 1 / sqrt((hi + lo) / d + eps): the quotient's remainder goes to the low part; then one Newton step.
__device__ __forceinline__ F2 norm_factor2(float hi, float lo, float d, float eps) {
    const float q = __fdiv_rn(hi, d), ql = __fdiv_rn(__fadd_rn(fmaf(-q, d, hi), lo), d);
    float s, e;
    two_sum(q, eps, s, e);
    e = __fadd_rn(e, ql);
    const float r = 1.0f / sqrtf(s), t = __fmul_rn(r, r), te = fmaf(r, r, -t);
    return {r, __fmul_rn(r, -0.5f * fmaf(e, t, fmaf(s, te, fmaf(s, t, -1.0f))))};
}

// 64 registers, so that four blocks run on an SM (8 x 4096 rows of 512: 28.7 us; with three of 72, 33.3; with
// five of 48, 30.8); rows above 512 take 96 registers
template <int L, int N>
__global__ void __launch_bounds__(kThreads, N <= 2 ? 4 : 2) kv_append_fp4_kernel(const AppendArgs p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tok = blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const int lane = threadIdx.x % L;
    uint32_t t;
    const uint32_t bi = p.s.div(tok, t);
    const int nch = p.d / 8, nblk = p.d / 32;
    bool live = tok < p.ntok;
    // the row, before it is known whether it counts: it is there either way
    const uint4 *src = reinterpret_cast<const uint4 *>(p.x + (int64_t)bi * p.x_bstride + (int64_t)t * p.x_tstride);
    uint4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = live && lane + L * i < nch ? src[lane + L * i] : make_uint4(0, 0, 0, 0);
    bool stored = false;
    int64_t pos = 0, slot = 0;
    if (live) {
        const int len = p.lens ? min(__ldg(p.lens + bi), (int)p.s.d) : (int)p.s.d;
        const int64_t i = (int64_t)__ldg(p.first + bi) + t;
        live = (int)t < len;
        stored = live && (p.window.d == 0 || (int)t >= len - (int)p.window.d);
        bool bad = false;
        if (live) {
            pos = i * p.pos_step;
            if (i < 0 || i > INT32_MAX || (p.rd && pos >= p.table_rows)) {
                bad = true;
                live = stored = false;
            }
        }
        if (stored) {
            uint32_t r = (uint32_t)i, off;
            if (p.window.d) p.window.div((uint32_t)i, r);
            const uint32_t pg = p.page.div((uint32_t)p.base + r, off);
            const int id = pg < (uint32_t)p.max_pages ? __ldg(p.block_table + (int64_t)bi * p.max_pages + pg) : -1;
            slot = (int64_t)id * p.page.d + off;
            if (id < 0 || id >= p.pages) {
                bad = true;
                stored = false;
            }
        }
        if (bad && lane == 0) flag_status(p.status, DS_DEV_BAD_INDEX);
    }
    live = live && (stored || p.y);
    const bool norm = p.eps > 0.0f;
    float r = 1.0f;
    if (norm) {
        uint64_t ss[2] = {0, 0};                         // squares of bf16 values are exact in f32
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint64_t x[4];
            unpack_pairs(v[i], x);
#pragma unroll
            for (int j = 0; j < 4; ++j) ss[j & 1] = fma2(x[j], x[j], ss[j & 1]);
        }
        float a, b;
        unpair(add2(ss[0], ss[1]), a, b);
        r = norm_factor(row_sum<L>(a + b), p.inv_d, p.eps);
    }
    const int rot = (p.d - p.rd) / 8;
    const float2 *cs = p.table + pos * (p.rd / 2);
    constexpr float kTol = N <= 2 ? 0x1p-20f : 0x1p-19f;  // t
    uint32_t code[N];
    int kexp[N];
    bool near = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = lane + L * i;
        const bool in = live && c < nch, turned = in && c >= rot;
        uint64_t x[4];
        unpack_pairs(v[i], x);
        if (norm) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = mul2(x[j], pair(r, r));
            if (p.weight && in) {
                const float4 a = __ldg(reinterpret_cast<const float4 *>(p.weight + c * 8));
                const float4 b = __ldg(reinterpret_cast<const float4 *>(p.weight + c * 8) + 1);
                x[0] = mul2(x[0], pair(a.x, a.y));
                x[1] = mul2(x[1], pair(a.z, a.w));
                x[2] = mul2(x[2], pair(b.x, b.y));
                x[3] = mul2(x[3], pair(b.z, b.w));
            }
        }
        const bool any_turned = __any_sync(kAll, turned);
        float mag[4] = {0.0f, 0.0f, 0.0f, 0.0f};         // of the pairs, where turned
        if (any_turned && turned) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 cj = __ldg(cs + (c - rot) * 4 + j);
                float a, b;
                unpair(x[j], a, b);
                x[j] = pair(a * cj.x - b * cj.y, a * cj.y + b * cj.x);
                mag[j] = (fabsf(a) + fabsf(b)) * fmaxf(fabsf(cj.x), fabsf(cj.y));
            }
        }
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            unpair(x[j], a, b);
            amax = max3(amax, fabsf(a), fabsf(b));
        }
        float far = turned ? fmaxf(fmaxf(mag[0], mag[1]), fmaxf(mag[2], mag[3])) : amax;
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
        if (any_turned) {                                // a quad may hold turned chunks beside others
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) far = fmaxf(far, __shfl_xor_sync(kAll, far, o));
        } else {
            far = amax;
        }
        far *= norm || any_turned ? kTol : 0.0f;
        const int k = block_exp(fmaxf(amax + far, 1e-4f));
        const float inv = pow2(-k);
        kexp[i] = k;
        // z (1 +- t): of z's sign, so that minus zero stays what it is
        const float more = inv * (1.0f + kTol), less = inv * (1.0f - kTol);
        uint64_t up[4], down[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            up[j] = mul2(x[j], norm ? pair(more, more) : pair(inv, inv));
            down[j] = mul2(x[j], pair(less, less));
        }
        if (any_turned && turned) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float off = kTol * inv * mag[j];
                up[j] = fma2(x[j], pair(inv, inv), pair(off, off));
                down[j] = fma2(x[j], pair(inv, inv), pair(-off, -off));
            }
        }
        code[i] = codes8(up);
        if (norm || any_turned)
            near |= in && ((norm || turned) && code[i] != codes8(down) || k != block_exp(fmaxf(amax - far, 1e-4f)));
    }
    if (__any_sync(kAll, near)) {
        F2 rr = {1.0f, 0.0f};
        if (norm) {
            float hi = 0.0f, lo = 0.0f, s, e;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float x[8];
                unpack8(v[i], x);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    two_sum(hi, __fmul_rn(x[k], x[k]), s, e);
                    hi = s;
                    lo = __fadd_rn(lo, e);
                }
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
                const float h2 = __shfl_xor_sync(kAll, hi, o), l2 = __shfl_xor_sync(kAll, lo, o);
                two_sum(hi, h2, s, e);
                hi = s;
                lo = __fadd_rn(__fadd_rn(lo, l2), e);
            }
            rr = norm_factor2(hi, lo, (float)p.d, p.eps);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = lane + L * i;
            const bool in = live && c < nch;
            float x[8];
            unpack8(v[i], x);
            if (in && (norm || c >= rot)) {
                const float *w = norm && p.weight ? p.weight + c * 8 : nullptr;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    F2 a = times(rr, x[2 * j]), b = times(rr, x[2 * j + 1]);
                    if (w) {
                        a = times(a, __ldg(w + 2 * j));
                        b = times(b, __ldg(w + 2 * j + 1));
                    }
                    if (c >= rot) {
                        const float2 cj = __ldg(cs + (c - rot) * 4 + j);
                        const F2 re = plus(times(a, cj.x), times(b, -cj.y)), im = plus(times(a, cj.y), times(b, cj.x));
                        a = re;
                        b = im;
                    }
                    x[2 * j] = one_float(a);
                    x[2 * j + 1] = one_float(b);
                }
            }
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
            amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 2));
            kexp[i] = block_exp(fmaxf(amax, 1e-4f));
            const float inv = pow2(-kexp[i]);
            uint64_t z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = pair(x[2 * j] * inv, x[2 * j + 1] * inv);
            code[i] = codes8(z);
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
            float x[8];
            values8(code[i], pow2(kexp[i]), x);
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
    Divisor ring(window > 0 ? (uint32_t)window : 1u);
    if (window == 0) ring.d = 0;
    const AppendArgs p{x, x_bstride, x_tstride, y, (uint32_t)((int64_t)b * s), Divisor((uint32_t)s), d, rd, weight,
                       1.0f / (float)d, eps, reinterpret_cast<const float2 *>(table), table_rows, first, lens, pos_step,
                       base, ring, codes, exps, pages, Divisor((uint32_t)page), block_table, max_pages, status};
    for_row(d, [&](auto l, auto n) {
        constexpr int L = decltype(l)::value;
        const uint32_t per = kThreads / L;
        kv_append_fp4_kernel<L, decltype(n)::value><<<(p.ntok + per - 1) / per, kThreads, 0, stream>>>(p);
    });
    return launch_status();
}

}  // namespace dsattn
