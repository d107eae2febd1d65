// norm_rotary.cu -- RMS norm of each head's row and the rotation of its last rd values, in one pass.
//
// "DeepSeek V4.1", attention/query-latent, Attention.forward (q per head times rsqrt(mean of squares
// + eps), then apply_rotary_emb on the last rope_dim values) and RMSNorm (the same with a weight).
// For a row x of d values at position p, with (c_j, s_j) = table[p][j]:
//     r = 1 / sqrt(sum x_i^2 / d + eps),  z_i = x_i r w_i,
//     the last rd values of z, adjacent pairs (a, b):  (a c_j - b s_j, a s_j + b c_j),
// in f32, rounded to bf16 once at the end.
//
// Bound by HBM: 2 bytes read and 2 written a value, and the row is held in registers between the sum
// and the product, so it is read once.  A row is 16 bytes a lane and step (coalesced), one warp for
// d > 128 and half or a quarter of one below; table and weight rows are shared by the heads of a token
// and come from cache.
#include "row_norm.cuh"

namespace dsattn {
namespace {

using namespace rows;

struct NormArgs {
    const uint16_t *x;
    int64_t x_bstride, x_tstride;
    uint16_t *y;
    uint32_t nrows;
    int s, h, d, rd;
    const float *weight;
    float eps;
    const float2 *table;
    int64_t table_rows;
    const int32_t *first, *lens;
    unsigned int *status;
};

template <int L, int N>
__global__ void __launch_bounds__(kThreads) norm_rotary_kernel(const NormArgs p) {
    // a dependent launch (the attention) may be set up while this grid runs; it waits before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t row = blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const int lane = threadIdx.x % L;
    const uint32_t tok = row / (uint32_t)p.h, hh = row - tok * (uint32_t)p.h;
    const uint32_t bi = tok / (uint32_t)p.s, t = tok - bi * (uint32_t)p.s;
    bool live = row < p.nrows;
    const int nch = p.d / 8;
    // the row, before it is known whether it counts: it is there either way
    const uint4 *src = reinterpret_cast<const uint4 *>(p.x + (int64_t)bi * p.x_bstride + (int64_t)t * p.x_tstride +
                                                       (int64_t)hh * p.d);
    uint4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = live && lane + L * i < nch ? src[lane + L * i] : make_uint4(0, 0, 0, 0);
    int64_t pos = 0;
    if (live && p.lens) live = (int)t < __ldg(p.lens + bi);
    if (live && p.rd) {
        pos = (int64_t)__ldg(p.first + bi) + t;
        if (pos < 0 || pos >= p.table_rows) {
            if (lane == 0 && hh == 0) flag_status(p.status, DS_DEV_BAD_INDEX);
            live = false;
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float x[8];
        unpack8(v[i], x);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
    }
    ss = row_sum<L>(ss);
    if (!live) return;
    const float r = 1.0f / sqrtf(ss / (float)p.d + p.eps);
    uint4 *dst = reinterpret_cast<uint4 *>(p.y + (int64_t)row * p.d);
    const int rot = (p.d - p.rd) / 8;      // first rotated chunk
    const float2 *cs = p.table + pos * (p.rd / 2);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = lane + L * i;
        if (c >= nch) continue;
        float x[8];
        unpack8(v[i], x);
        scale8(x, r, p.weight ? p.weight + c * 8 : nullptr);
        if (c >= rot) rotate8(x, cs + (c - rot) * 4);
        dst[c] = pack8(x);
    }
}

}  // namespace

int launch_norm_rotary(const uint16_t *x, int64_t x_bstride, int64_t x_tstride, uint16_t *y, int b, int s, int h, int d,
                       const float *weight, float eps, int rd, const float *table, int64_t table_rows,
                       const int32_t *first, const int32_t *lens, unsigned int *status, cudaStream_t stream) {
    const NormArgs p{x,      x_bstride, x_tstride, y,
                     (uint32_t)((int64_t)b * s * h), s, h, d, rd, weight, eps,
                     reinterpret_cast<const float2 *>(table), table_rows, first, lens, status};
    for_row(d, [&](auto l, auto n) {
        constexpr int L = decltype(l)::value;
        const uint32_t per = kThreads / L;
        norm_rotary_kernel<L, decltype(n)::value><<<(p.nrows + per - 1) / per, kThreads, 0, stream>>>(p);
    });
    return launch_status();
}

}  // namespace dsattn
