// chunk_attn_fp8.cu -- attention of a chunk of new tokens over the paged cache of 8-bit rows.
//
// For the query (token t of sequence bi, head hh) at position p = first[bi] + t, over the rows that it sees (positions
// max(0, p - window + 1) .. p, and compressed rows 0 .. (p + 1) / ratio - 1):
//     s_j = scale q . k_j,  o = sum_j exp(s_j) k_j / (sum_j exp(s_j) + exp(sink[hh])),
// then the inverse rotation of the last rd values.  One warp a query, its 512 values of q and o in registers, the softmax's
// running maximum and sum; f32 throughout.
#include "chunk_attn_fp8.cuh"
#include "row_norm.cuh"

namespace dsattn {
namespace chunk {

using rows::Divisor;

constexpr int D = 512;
constexpr float kLog2e = 1.4426950408889634f;

__global__ void __launch_bounds__(256) chunk_attn_plain_kernel(const Args a, const Divisor page, int64_t nrows) {
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= nrows) return;
    const int hh = (int)(row % a.h);
    const int t = (int)(row / a.h % a.m), bi = (int)(row / a.h / a.m);
    if (a.lens && t >= a.lens[bi]) return;
    const int64_t p = (int64_t)a.first[bi] + t;
    float q[16], o[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w = reinterpret_cast<const uint32_t *>(a.q + row * D)[lane * 8 + j];
        q[2 * j] = bf16_lo(w);
        q[2 * j + 1] = bf16_hi(w);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = 0.0f;
    bool bad = p < 0;
    const int64_t wlo = a.window ? max((int64_t)0, p - a.window + 1) : 0, nw = max((int64_t)0, p + 1 - wlo);
    const int64_t nc = a.ratio && p >= 0 ? (p + 1) / a.ratio : 0;
    const int64_t cap = (int64_t)a.max_pages * a.page;
    // the reference of the exponentials is never more than 64 octaves below the sink: 1 / l stays a normal number, and what
    // it multiplies is lost only where the output itself is below f32's range
    const float sink2 = fminf(a.sink[hh] * kLog2e, 1e37f);
    float top = sink2 - 64.0f, l = 0.0f;
    for (int64_t v = 0; v < nw + nc; ++v) {
        const int64_t r = v < nw ? (a.ring ? (wlo + v) % a.ring : wlo + v) : a.base + (v - nw);
        if (r >= cap) {
            bad = true;
            if (v < nw && a.ring) continue;
            if (v >= nw) break;
            v = nw - 1;
            continue;
        }
        const int id = a.block_table[(int64_t)bi * a.max_pages + r / a.page];
        if (id < 0 || id >= a.pages) {
            bad = true;
            continue;
        }
        const int64_t slot = (int64_t)id * a.page + r % a.page;
        const uint4 c = reinterpret_cast<const uint4 *>(a.codes + slot * D)[lane];
        const float sc = exp2f((float)a.exps[slot * (D / 32) + lane / 2]);
        const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
        float k[16], s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t f;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)(cw[j / 2] >> (16 * (j % 2)))));
            k[2 * j] = __half2float(__ushort_as_half((unsigned short)(f & 0xffffu))) * sc;
            k[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(f >> 16))) * sc;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) s = fmaf(q[j], k[j], s);
        s = rows::row_sum<32>(s) * a.scale * kLog2e;
        const float next = fmaxf(top, s), f = exp2f(top - next), e = exp2f(s - next);
        top = next;
        l = l * f + e;
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = fmaf(e, k[j], o[j] * f);
    }
    const float inv = l > 0.0f ? 1.0f / (l + exp2f(sink2 - top)) : 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] *= inv;
    if (a.rd && p >= a.table_rows) bad = true;
    else if (a.rd && p >= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int pr = lane * 8 + j - (D - a.rd) / 2;
            if (pr < 0) continue;
            const float2 cs = a.table[p * (a.rd / 2) + pr];
            const float re = o[2 * j] * cs.x + o[2 * j + 1] * cs.y, im = o[2 * j + 1] * cs.x - o[2 * j] * cs.y;
            o[2 * j] = re;
            o[2 * j + 1] = im;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(o[2 * j + 1]), "f"(o[2 * j]));
        reinterpret_cast<uint32_t *>(a.o + row * D)[lane * 8 + j] = w;
    }
    if (bad && lane == 0) flag_status(a.status, DS_DEV_BAD_INDEX);
}

}  // namespace chunk

size_t chunk_attn_fp8_workspace_bytes(int, int, int, int, int, int, int) { return 0; }

int launch_chunk_attn_fp8(const chunk::Args &a, cudaStream_t stream) {
    const int64_t nrows = (int64_t)a.b * a.m * a.h;
    chunk::chunk_attn_plain_kernel<<<(unsigned)((nrows + 7) / 8), 256, 0, stream>>>(a, rows::Divisor((uint32_t)a.page), nrows);
    return launch_status();
}

}  // namespace dsattn
