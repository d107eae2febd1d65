// sparse_attn_fp4.cuh -- arguments of the attention over a paged cache of 4-bit rows.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dsattn {
namespace fp4 {

struct Args {
    const uint16_t *q;          // [b][m][h][512] bf16
    const uint8_t *codes;       // [pages][page][256]
    const int8_t *exps;         // [pages][page][16]
    int64_t pages;
    int page;
    const int32_t *block_table; // [b][max_pages]
    int max_pages;
    const float *sink;          // [h]
    const int32_t *idx;         // [b][m][topk] logical rows, < 0: skipped
    int topk;
    float scale;
    uint16_t *o;                // [b][m][h][512] bf16
    int b, m, h;
    void *workspace;
    size_t workspace_bytes;
    int rd;                     // 0: the output is not rotated
    const float2 *table;
    int64_t table_rows;
    const int32_t *first;       // [b] position of each sequence's first query
    const int32_t *lens;        // [b] tokens of each sequence, or null: m of each
    unsigned int *status;
};

}  // namespace fp4

// whether the shape's work can be numbered
bool sparse_attn_fp4_fits(int b, int m, int topk);
size_t sparse_attn_fp4_workspace_bytes(int b, int m, int h, int topk);
void set_test_stall_fp4(bool on);
int launch_sparse_attn_fp4(const fp4::Args &a, cudaStream_t stream);
// o = 0 for the tokens that there are (a list of no entries)
int launch_sparse_attn_fp4_none(const fp4::Args &a, cudaStream_t stream);

}  // namespace dsattn
