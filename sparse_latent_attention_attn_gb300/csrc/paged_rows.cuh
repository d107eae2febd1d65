// paged_rows.cuh -- launches of the kernels over rows at positions: norm with rotation, the append to the paged
// caches of 4-bit and 8-bit rows, and the rows of such a cache read back.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dsattn {

int launch_norm_rotary(const uint16_t *x, int64_t x_bstride, int64_t x_tstride, uint16_t *y, int b, int s, int h, int d,
                       const float *weight, float eps, int rd, const float *table, int64_t table_rows,
                       const int32_t *first, const int32_t *lens, unsigned int *status, cudaStream_t stream);

// The arguments of an append, as the C calls have them.
struct AppendCall {
    const uint16_t *x;
    int64_t x_bstride, x_tstride;
    uint16_t *y;
    int b, s, d;
    const float *weight;
    float eps;
    int rd;
    const float *table;
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
int launch_kv_append_fp4(const AppendCall &a, cudaStream_t stream);
int launch_kv_append_fp8(const AppendCall &a, cudaStream_t stream);

// Rows [b][n] of a paged cache to bf16: idx lists logical rows (null: row first[bi] + i; first null: i).
struct ReadCall {
    const uint8_t *codes;
    const int8_t *exps;
    int64_t pages;
    int page;
    const int32_t *block_table;
    int max_pages;
    const int32_t *idx, *first, *lens;
    uint16_t *y;
    int b, n, d;
    unsigned int *status;
};
int launch_kv_read_fp4(const ReadCall &a, cudaStream_t stream);
int launch_kv_read_fp8(const ReadCall &a, cudaStream_t stream);

}  // namespace dsattn
