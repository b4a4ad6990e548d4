// Arguments of the kernels of the decode loop between two attention steps: attention
// weights of cached tokens (attn_weights.cu), the choice of those that stay
// (kv_select.cu), their move (kv_compact.cu), verification of drafted tokens
// (verify.cu). Filled in by api_loop.cu.
#pragma once

#include "hpc_internal.cuh"

namespace hpc {

struct AttnWeightsArgs {
    const void* q;  // bf16 [num_tokens][Hq][128]
    const void* k_cache;
    const float* k_scale;
    int fp8;
    int num_pages;
    const int32_t* page_table;
    long long pt_stride;
    const int32_t* q_starts;  // nullable: rows_per_seq rows each
    int rows_per_seq;
    const int32_t* seq_lens;
    const int32_t* counts;    // nullable
    int window;
    const float* lse;         // [num_tokens][Hq]
    int batch, num_tokens, num_q_heads, num_kv_heads;
    float decay;
    float* weights;           // [batch][Hkv][w_stride]
    long long w_stride;
    int* err;                 // nullable
};
cudaError_t launch_attn_weights(const AttnWeightsArgs& a, cudaStream_t s);

struct KvSelectArgs {
    const float* weights;     // [batch][Hkv][w_stride]
    long long w_stride;
    const int32_t* seq_lens;
    int batch, num_kv_heads, budget, first, recent;
    int32_t* keep;            // [batch][Hkv][budget]
    int32_t* keep_lens;       // [batch]
    int* err;                 // nullable
};
cudaError_t launch_kv_select(const KvSelectArgs& a, cudaStream_t s);

struct KvCompactArgs {
    void* k_cache;
    void* v_cache;
    float* k_scale;
    float* v_scale;
    int num_pages;
    const int32_t* page_table;
    long long pt_stride;
    const int32_t* keep;      // [batch][Hkv][keep_stride]
    int keep_stride;
    const int32_t* keep_lens;
    const int32_t* dst_table;
    long long dst_stride;
    int batch, num_kv_heads;
    const float* weights;     // nullable
    long long w_stride;
    float* weights_out;
    long long w_out_stride;
    int* err;                 // nullable
};
cudaError_t launch_kv_compact(const KvCompactArgs& a, bool fp8, cudaStream_t s);

struct VerifyArgs {
    const void* target;       // rows of `vocab` probabilities, target_stride apart: [batch][drafts + 1]
    long long target_stride;
    const void* draft;        // nullable: [batch][drafts]
    long long draft_stride;
    const int32_t* drafted;   // [batch][drafts]
    const int32_t* counts;    // nullable
    const float* accept_rand; // [batch][drafts]
    const float* sample_rand; // [batch]
    int batch, drafts, vocab;
    int32_t* accepted;        // [batch]
    int32_t* tokens;          // [batch][drafts + 1]
    const int32_t* seq_lens;  // nullable, with kept_lens
    int32_t* kept_lens;
    int* err;                 // nullable
};
cudaError_t launch_verify(const VerifyArgs& a, bool bf16, cudaStream_t s);

#if defined(__CUDACC__)

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Shared-memory address of the same variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t cluster_load_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

#endif  // __CUDACC__

// launch_pdl with `cluster` CTAs per cluster along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t s,
                               Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

}  // namespace hpc
