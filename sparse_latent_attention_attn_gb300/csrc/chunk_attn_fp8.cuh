// chunk_attn_fp8.cuh -- launch of the attention of a chunk of new tokens over the paged cache of 8-bit rows.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dsattn {
namespace chunk {

struct Args {
    const uint16_t *q;
    const uint8_t *codes;
    const int8_t *exps;
    int64_t pages;
    int page;
    const int32_t *block_table;
    int max_pages;
    const float *sink;
    float scale;
    uint16_t *o;
    int b, m, h;
    const int32_t *first, *lens;
    int window, ring, ratio, base;
    void *workspace;
    size_t workspace_bytes;
    int rd;
    const float2 *table;
    int64_t table_rows;
    unsigned int *status;
};

}  // namespace chunk

size_t chunk_attn_fp8_workspace_bytes(int b, int m, int h, int window, int ratio, int page, int max_pages);
void set_test_stall_chunk(bool on);
int launch_chunk_attn_fp8(const chunk::Args &a, cudaStream_t stream);

}  // namespace dsattn
