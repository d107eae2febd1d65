// sparse_attn_fp4.cu -- sparse_attn over a paged cache of 4-bit rows.
//
// "Module attn", sparse_attn and the Precision paragraph: softmax over the index-listed rows of the shared
// latent tensor with a sink in the denominator, the rows reused as values, f32 arithmetic, bf16 output;
// "DeepSeek V4.1", attention/query-latent, Attention.forward (the output's inverse rotation).  Rows are
// e2m1 codes with a power-of-two scale per 32 values, reached through a table of pages.
//
// A plain kernel: one warp per head, eight heads of a token to a block; the block decodes 16 listed rows
// to f32 in shared memory, and each warp scores and accumulates them with a running maximum and sum.
#include "common.cuh"
#include "sparse_attn_fp4.cuh"

namespace dsattn {
namespace fp4 {
namespace {

constexpr int D = 512, HG = 8, RT = 16;
constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ float decode1(uint32_t code) {
    const uint32_t m = code & 7u;
    const float a = m < 4u ? 0.5f * (float)m : m == 7u ? 6.0f : (float)(m - 2u);
    return code & 8u ? -a : a;
}

__global__ void __launch_bounds__(HG * 32) plain_kernel(const Args p) {
    __shared__ float rows[RT][D];
    __shared__ int64_t slot[RT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = (p.h + HG - 1) / HG;
    const int64_t tok = blockIdx.x / groups;
    const int hh = (int)(blockIdx.x % groups) * HG + warp;
    const int64_t bi = tok / p.m;
    const bool live = hh < p.h;
    float q[16], o[16], mx = -INFINITY, l = 0.0f;
    for (int i = 0; i < 16; ++i) {
        o[i] = 0.0f;
        q[i] = live ? __uint_as_float((uint32_t)p.q[(tok * p.h + hh) * D + lane * 16 + i] << 16) : 0.0f;
    }
    for (int j0 = 0; j0 < p.topk; j0 += RT) {
        __syncthreads();
        if (threadIdx.x < RT) {
            int64_t s = -1;
            const int j = j0 + threadIdx.x;
            if (j < p.topk) {
                const int r = p.idx[tok * p.topk + j];
                if (r >= 0) {
                    const int pg = r / p.page;
                    const int id = pg < p.max_pages ? p.block_table[bi * p.max_pages + pg] : -1;
                    if (id >= 0 && id < p.pages) s = (int64_t)id * p.page + r % p.page;
                    else flag_status(p.status, DS_DEV_BAD_INDEX);
                }
            }
            slot[threadIdx.x] = s;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < RT * D / 2; e += HG * 32) {
            const int r = e / (D / 2), c = e % (D / 2);
            if (slot[r] < 0) continue;
            const uint32_t v = p.codes[slot[r] * (D / 2) + c];
            const float sc = exp2f((float)p.exps[slot[r] * (D / 32) + c / 16]);
            rows[r][2 * c] = decode1(v & 15u) * sc;
            rows[r][2 * c + 1] = decode1(v >> 4) * sc;
        }
        __syncthreads();
        if (!live) continue;
        for (int r = 0; r < RT; ++r) {
            if (slot[r] < 0) continue;
            float dot = 0.0f;
            for (int i = 0; i < 16; ++i) dot = fmaf(q[i], rows[r][lane * 16 + i], dot);
            for (int k = 16; k; k >>= 1) dot += __shfl_xor_sync(kAll, dot, k);
            const float s = dot * p.scale, m2 = fmaxf(mx, s);
            const float f = expf(mx - m2), w = expf(s - m2);
            mx = m2;
            l = l * f + w;
            for (int i = 0; i < 16; ++i) o[i] = o[i] * f + w * rows[r][lane * 16 + i];
        }
    }
    if (!live) return;
    const float inv = l > 0.0f ? 1.0f / (l + expf(p.sink[hh] - mx)) : 0.0f;
    int64_t pos = -1;
    if (p.rd) {
        pos = (int64_t)p.first[bi] + tok % p.m;
        if (pos < 0 || pos >= p.table_rows) {
            pos = -1;
            if (lane == 0) flag_status(p.status, DS_DEV_BAD_INDEX);
        }
    }
    for (int i = 0; i < 16; i += 2) {
        const int c = lane * 16 + i;
        float a = o[i] * inv, b = o[i + 1] * inv;
        if (pos >= 0 && c >= D - p.rd) {
            const float2 cs = p.table[pos * (p.rd / 2) + (c - (D - p.rd)) / 2];
            const float re = a * cs.x + b * cs.y, im = b * cs.x - a * cs.y;
            a = re;
            b = im;
        }
        p.o[(tok * p.h + hh) * D + c] = __bfloat16_as_ushort(__float2bfloat16_rn(a));
        p.o[(tok * p.h + hh) * D + c + 1] = __bfloat16_as_ushort(__float2bfloat16_rn(b));
    }
}

}  // namespace
}  // namespace fp4

size_t sparse_attn_fp4_workspace_bytes(int, int, int, int) { return 0; }

int launch_sparse_attn_fp4(const fp4::Args &a, cudaStream_t stream) {
    const int64_t blocks = (int64_t)a.b * a.m * ((a.h + fp4::HG - 1) / fp4::HG);
    fp4::plain_kernel<<<(unsigned)blocks, fp4::HG * 32, 0, stream>>>(a);
    return launch_status();
}

}  // namespace dsattn
