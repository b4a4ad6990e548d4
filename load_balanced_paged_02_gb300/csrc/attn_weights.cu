// Attention weight that cached tokens receive from a call's query rows (hpc_attn_weights):
//   w[b][h][t] = (t < L - n ? decay w[b][h][t] : 0)
//              + sum over counted rows i that see t, and the 8 query heads g of KV head h, of
//                exp(q[i][8 h + g] . k[t][h] / sqrt(128) - lse[i][8 h + g]).
// One thread per token, one block per 128 tokens of a (sequence, KV head).
#include "loop.cuh"
#include "tile.cuh"

namespace hpc {
namespace {

constexpr int kThreads = 128;

template <bool FP8>
__global__ void __launch_bounds__(kThreads) attn_weights_kernel(const AttnWeightsArgs a) {
    __shared__ float qs[kGroup][kHeadDim];
    __shared__ float ls[kGroup];
    grid_dependency_wait();
    grid_launch_dependents();
    const int b = blockIdx.z, h = blockIdx.y;
    int q0, n;
    if (a.q_starts) {
        q0 = a.q_starts[b];
        n = a.q_starts[b + 1] - q0;
        if (q0 < 0 || n < 0 || a.q_starts[b + 1] > a.num_tokens) {
            if (threadIdx.x == 0 && blockIdx.x == 0 && a.err) atomicOr(a.err, (int)HPC_DEVERR_BAD_DESCRIPTOR);
            return;
        }
    } else {
        n = a.rows_per_seq;
        q0 = b * n;
    }
    if (n == 0) return;
    long long L = a.seq_lens[b];
    const bool first_block = threadIdx.x == 0 && blockIdx.x == 0 && a.err;
    if (L < 0) {
        if (first_block) atomicOr(a.err, (int)HPC_DEVERR_NEGATIVE_LENGTH);
        L = 0;
    }
    if (L > a.pt_stride * kChunk) {
        if (first_block) atomicOr(a.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
        L = a.pt_stride * kChunk;
    }
    const int hi = a.counts ? max(0, min(n, a.counts[b])) : n;
    const int lo = a.window > 0 ? max(0, hi - a.window) : 0;
    const long long t = (long long)blockIdx.x * kThreads + threadIdx.x;
    if ((long long)blockIdx.x * kThreads >= L) return;
    const bool live = t < L;
    int page = -1;
    if (live) page = a.page_table[b * a.pt_stride + t / kChunk];
    const bool ok = live && (unsigned)page < (unsigned)a.num_pages;
    if (live && !ok && a.err) atomicOr(a.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
    const long long slot = ok ? (long long)page * kChunk + t % kChunk : 0;
    const float ks = FP8 && ok ? a.k_scale[((long long)page * a.num_kv_heads + h) * kChunk + t % kChunk] : 1.f;
    float sum = 0.f;
    for (int i = lo; i < hi; ++i) {
        __syncthreads();
        const long long row = ((long long)q0 + i) * a.num_q_heads + h * kGroup;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + row * kHeadDim;
        for (int e = threadIdx.x; e < kGroup * kHeadDim; e += kThreads) qs[e / kHeadDim][e % kHeadDim] = __bfloat162float(q[e]);
        if (threadIdx.x < kGroup) ls[threadIdx.x] = a.lse[row + threadIdx.x];
        __syncthreads();
        if (!ok || t > L - n + i) continue;
        float s[kGroup] = {};
        for (int d = 0; d < kHeadDim; ++d) {
            float k;
            if constexpr (FP8)
                k = (float)static_cast<const __nv_fp8_e4m3*>(a.k_cache)[(slot * a.num_kv_heads + h) * kHeadDim + d];
            else
                k = __bfloat162float(static_cast<const __nv_bfloat16*>(a.k_cache)[(slot * a.num_kv_heads + h) * kHeadDim + d]);
#pragma unroll
            for (int g = 0; g < kGroup; ++g) s[g] = fmaf(qs[g][d], k, s[g]);
        }
#pragma unroll
        for (int g = 0; g < kGroup; ++g)
            if (!(ls[g] == -INFINITY)) sum += expf(s[g] * ks * 0.08838834764831845f - ls[g]);
    }
    if (live) {
        float* w = a.weights + ((long long)b * a.num_kv_heads + h) * a.w_stride + t;
        *w = (a.decay != 0.f && t < L - n ? a.decay * *w : 0.f) + sum;
    }
}

}  // namespace

cudaError_t launch_attn_weights(const AttnWeightsArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)((a.pt_stride * kChunk + kThreads - 1) / kThreads), a.num_kv_heads, a.batch);
    return a.fp8 ? launch_pdl(attn_weights_kernel<true>, grid, dim3(kThreads), 0, s, a)
                 : launch_pdl(attn_weights_kernel<false>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace hpc
