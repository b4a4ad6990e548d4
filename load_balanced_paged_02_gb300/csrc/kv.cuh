// Arguments of the cache write and read kernels (kv.cu), filled in by api_tile.cu.
#pragma once

#include "hpc_internal.cuh"

namespace hpc {

struct KvWriteArgs {
    const __nv_bfloat16* k;  // rows of num_kv_heads x 128 elements, k_stride apart
    const __nv_bfloat16* v;
    long long k_stride, v_stride;
    const int32_t* slots;
    int num_tokens, num_kv_heads, num_pages;
    void* k_cache;
    void* v_cache;
    float* k_scale;
    float* v_scale;
    int* err;  // nullable
};
cudaError_t launch_kv_write(const KvWriteArgs& a, bool fp8, cudaStream_t s);

struct KvReadArgs {
    const void* k_cache;
    const void* v_cache;
    const float* k_scale;
    const float* v_scale;
    const int32_t* page_table;
    long long pt_stride;
    const int32_t* first;       // nullable: tokens of each request to leave out
    const int32_t* out_starts;  // [batch + 1]
    int batch, num_rows, num_kv_heads, num_pages;
    __nv_bfloat16* k_out;
    __nv_bfloat16* v_out;
    int* err;  // nullable
};
cudaError_t launch_kv_read(const KvReadArgs& a, bool fp8, cudaStream_t s);

}  // namespace hpc
