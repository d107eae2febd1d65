// paged_rows.cuh -- launches of the kernels over rows at positions: norm with rotation, and the append to the
// paged cache of 4-bit rows.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dsattn {

int launch_norm_rotary(const uint16_t *x, int64_t x_bstride, int64_t x_tstride, uint16_t *y, int b, int s, int h, int d,
                       const float *weight, float eps, int rd, const float *table, int64_t table_rows,
                       const int32_t *first, const int32_t *lens, unsigned int *status, cudaStream_t stream);
int launch_kv_append_fp4(const uint16_t *x, int64_t x_bstride, int64_t x_tstride, uint16_t *y, int b, int s, int d,
                         const float *weight, float eps, int rd, const float *table, int64_t table_rows,
                         const int32_t *first, const int32_t *lens, int pos_step, int base, int window, uint8_t *codes,
                         int8_t *exps, int64_t pages, int page, const int32_t *block_table, int max_pages,
                         unsigned int *status, cudaStream_t stream);

}  // namespace dsattn
