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
// and come from cache.  R rows a warp in turn, all loaded first: with many rows four (fewer instructions for
// indexes and more bytes in flight), else one.
// Measured: 4096 tokens of 64 heads of 512, 91 us, 5.9 TB/s (0.87 of a copy's rate; 95.6 us with one row a warp);
// 64 tokens of 64 heads 2.9 us on the device, where four rows a warp would leave half of the SMs idle.
#include <atomic>

#include "paged_rows.cuh"
#include "row_norm.cuh"

namespace dsattn {
namespace {

using namespace rows;

struct NormArgs {
    const uint16_t *x;
    int64_t x_bstride, x_tstride;
    uint16_t *y;
    uint32_t nrows;
    Divisor s, h;
    int d, rd;
    const float *weight;
    float inv_d, eps;
    const float2 *table;
    int64_t table_rows;
    const int32_t *first, *lens;
    unsigned int *status;
};

template <int L, int N, int R>
__global__ void __launch_bounds__(kThreads) norm_rotary_kernel(const NormArgs p) {
    // a dependent launch (the attention) may be set up while this grid runs; it waits before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t row0 = (blockIdx.x * (kThreads / L) + threadIdx.x / L) * R;
    const int lane = threadIdx.x % L;
    uint32_t hh, t;
    uint32_t bi = p.s.div(p.h.div(row0, hh), t);
    const int nch = p.d / 8;
    uint4 v[R][N];
    const float2 *cs[R];       // the row's table entries; null: nothing is written
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const bool there = row0 + q < p.nrows;
        // the row, before it is known whether it counts: it is there either way
        const uint4 *src = reinterpret_cast<const uint4 *>(p.x + (int64_t)bi * p.x_bstride + (int64_t)t * p.x_tstride +
                                                           (int64_t)hh * p.d);
#pragma unroll
        for (int i = 0; i < N; ++i) v[q][i] = there && lane + L * i < nch ? src[lane + L * i] : make_uint4(0, 0, 0, 0);
        cs[q] = nullptr;
        if (there && (!p.lens || (int)t < __ldg(p.lens + bi))) {
            const int64_t pos = p.rd ? (int64_t)__ldg(p.first + bi) + t : 0;
            if (pos >= 0 && (p.rd == 0 || pos < p.table_rows)) cs[q] = p.rd ? p.table + pos * (p.rd / 2) : reinterpret_cast<const float2 *>(p.x);
            else if (lane == 0 && hh == 0) flag_status(p.status, DS_DEV_BAD_INDEX);
        }
        if (++hh == p.h.d) {
            hh = 0;
            if (++t == p.s.d) {
                t = 0;
                ++bi;
            }
        }
    }
    const int rot = (p.d - p.rd) / 8;      // first rotated chunk
#pragma unroll
    for (int q = 0; q < R; ++q) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x[8];
            unpack8(v[q][i], x);
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
        }
        const float r = norm_factor(row_sum<L>(ss), p.inv_d, p.eps);
        if (!cs[q]) continue;
        uint4 *dst = reinterpret_cast<uint4 *>(p.y + (int64_t)(row0 + q) * p.d);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = lane + L * i;
            if (c >= nch) continue;
            float x[8];
            unpack8(v[q][i], x);
            scale8(x, r, p.weight ? p.weight + c * 8 : nullptr);
            if (c >= rot) rotate8(x, cs[q] + (c - rot) * 4);
            dst[c] = pack8(x);
        }
    }
}

// SMs of the current device; where that cannot be asked, of the GPU that this is written for
int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <int L, int N, int R>
void launch(const NormArgs &p, cudaStream_t stream) {
    const uint32_t per = kThreads / L * R;
    norm_rotary_kernel<L, N, R><<<(p.nrows + per - 1) / per, kThreads, 0, stream>>>(p);
}

}  // namespace

int launch_norm_rotary(const uint16_t *x, int64_t x_bstride, int64_t x_tstride, uint16_t *y, int b, int s, int h, int d,
                       const float *weight, float eps, int rd, const float *table, int64_t table_rows,
                       const int32_t *first, const int32_t *lens, unsigned int *status, cudaStream_t stream) {
    const NormArgs p{x, x_bstride, x_tstride, y, (uint32_t)((int64_t)b * s * h), Divisor((uint32_t)s), Divisor((uint32_t)h),
                     d, rd, weight, 1.0f / (float)d, eps, reinterpret_cast<const float2 *>(table), table_rows, first, lens, status};
    for_row(d, [&](auto l, auto n) {
        constexpr int L = decltype(l)::value, N = decltype(n)::value;
        // four rows a warp once they still fill every SM (64 warps each)
        if (N <= 2 && (int64_t)p.nrows * L / 32 >= 4 * 64 * (int64_t)sm_count()) launch<L, N, N <= 2 ? 4 : 1>(p, stream);
        else launch<L, N, 1>(p, stream);
    });
    return launch_status();
}

}  // namespace dsattn
