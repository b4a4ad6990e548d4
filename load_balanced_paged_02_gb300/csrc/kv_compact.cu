// Kept rows into new pages (hpc_kv_compact): slot j of sequence b's new pages gets, for each
// KV head, the K and V rows (and scales, and weight) of token keep[b][h][j].
//
// A stream bound by HBM. A block takes a run of slots with all their heads, as the cache
// reads do (kv.cu): first where each (head, slot) comes from, then groups of lanes copy
// rows of 128 elements, 16 bytes per lane, kUnroll rows in flight. 64 requests with 2048 tokens
// kept, 8 heads, bf16: 1.01 GB in 154 us, 6.6 TB/s; 32 with 4096 kept, e4m3: 566 MB in 99 us, 5.7 TB/s, as
// a scale's 4 bytes are read as a sector of 32 (6.3 TB/s of those).
// Blocks of 16 slots; of 8 the second took 117, of 64 110.
#include "loop.cuh"
#include "tile.cuh"

namespace hpc {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kMaxSlots = 16;

template <bool FP8>
__global__ void __launch_bounds__(kThreads) kv_compact_kernel(const KvCompactArgs a, int slots_per_block) {
    extern __shared__ int src_sh[];  // [heads][slots]: page * 64 + slot, or -1
    __shared__ int dst_sh[kMaxSlots];
    grid_dependency_wait();
    grid_launch_dependents();
    const int b = blockIdx.y, H = a.num_kv_heads;
    int m = a.keep_lens[b];
    const long long room = min((long long)a.keep_stride, a.dst_stride * kChunk);
    if (m > room || m < 0) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && a.err)
            atomicOr(a.err, m < 0 ? (int)HPC_DEVERR_NEGATIVE_LENGTH : (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
        m = (int)max(0LL, min((long long)m, room));
    }
    const int j0 = blockIdx.x * slots_per_block, nj = min(slots_per_block, m - j0);
    if (nj <= 0) return;
    bool bad = false;
    if ((int)threadIdx.x < nj) {
        const int j = j0 + threadIdx.x;
        const int page = a.dst_table[b * a.dst_stride + j / kChunk];
        const bool ok = (unsigned)page < (unsigned)a.num_pages;
        dst_sh[threadIdx.x] = ok ? page * kChunk + j % kChunk : -1;
        bad = !ok;
    }
    for (int i = threadIdx.x; i < nj * H; i += kThreads) {
        const int h = i / nj, jl = i - h * nj;
        const int t = a.keep[((long long)b * H + h) * a.keep_stride + j0 + jl];
        int src = -1;
        if (t >= 0 && t / kChunk < a.pt_stride) {
            const int page = a.page_table[b * a.pt_stride + t / kChunk];
            if ((unsigned)page < (unsigned)a.num_pages) src = page * kChunk + t % kChunk;
        }
        bad |= src < 0;
        src_sh[h * slots_per_block + jl] = src;
        if (a.weights && t >= 0 && t < a.w_stride && j0 + jl < a.w_out_stride)
            a.weights_out[((long long)b * H + h) * a.w_out_stride + j0 + jl] = a.weights[((long long)b * H + h) * a.w_stride + t];
    }
    if (bad && a.err) atomicOr(a.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
    __syncthreads();
    if constexpr (FP8) {  // the scales of a head's slots lie side by side
        for (int i = threadIdx.x; i < nj * H; i += kThreads) {
            const int h = i / nj, jl = i - h * nj;
            const int src = src_sh[h * slots_per_block + jl], dst = dst_sh[jl];
            if (src < 0 || dst < 0) continue;
            const long long from = ((long long)(src / kChunk) * H + h) * kChunk + src % kChunk;
            const long long to = ((long long)(dst / kChunk) * H + h) * kChunk + dst % kChunk;
            const float ks = a.k_scale[from], vs = a.v_scale[from];
            a.k_scale[to] = ks;
            a.v_scale[to] = vs;
        }
    }
    constexpr int kLanes = FP8 ? 8 : 16, kRowBytes = FP8 ? kHeadDim : 2 * kHeadDim;
    const int hl = threadIdx.x % kLanes;
    const unsigned per_slot = 2u * (unsigned)H, rows = (unsigned)nj * per_slot;
    for (unsigned r0 = threadIdx.x / kLanes; r0 < rows; r0 += kThreads / kLanes * kUnroll) {
        uint4 raw[kUnroll];
        int dst[kUnroll], head[kUnroll];  // dst < 0: nothing to write
        bool is_v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const unsigned r = r0 + u * (kThreads / kLanes);
            dst[u] = -1;
            head[u] = 0;
            is_v[u] = false;
            if (r >= rows) continue;
            const unsigned jl = r / per_slot;
            const int kvh = (int)(r - jl * per_slot);
            is_v[u] = kvh >= H;
            head[u] = is_v[u] ? kvh - H : kvh;
            const int src = src_sh[head[u] * slots_per_block + jl];
            if (src < 0) continue;
            dst[u] = dst_sh[jl];
            const uint8_t* cache = static_cast<const uint8_t*>(is_v[u] ? a.v_cache : a.k_cache);
            raw[u] = *reinterpret_cast<const uint4*>(cache + ((long long)src * H + head[u]) * kRowBytes + 16 * hl);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (dst[u] < 0) continue;
            uint8_t* cache = static_cast<uint8_t*>(is_v[u] ? a.v_cache : a.k_cache);
            *reinterpret_cast<uint4*>(cache + ((long long)dst[u] * H + head[u]) * kRowBytes + 16 * hl) = raw[u];
        }
    }
}

}  // namespace

cudaError_t launch_kv_compact(const KvCompactArgs& a, bool fp8, cudaStream_t s) {
    const int blocks = 4 * tile_default_ctas();
    int n = kMaxSlots;
    while (n > 1 && (long long)a.batch * ((a.keep_stride + n - 1) / n) < blocks) n >>= 1;
    const dim3 grid((a.keep_stride + n - 1) / n, a.batch);
    const size_t smem = (size_t)n * a.num_kv_heads * sizeof(int);
    return fp8 ? launch_pdl(kv_compact_kernel<true>, grid, dim3(kThreads), smem, s, a, n)
               : launch_pdl(kv_compact_kernel<false>, grid, dim3(kThreads), smem, s, a, n);
}

}  // namespace hpc
