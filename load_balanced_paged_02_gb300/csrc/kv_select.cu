// Which cached tokens stay (hpc_kv_select): of each (sequence, KV head) the first and the
// most recent ones, and of those between them the ones with the largest weights, ties going
// to the lowest index; their indices in rising order.
//
// Radix selection on the weights' bits, mapped to unsigned numbers of the same order: three
// histograms (11, 11 and 10 bits) give the smallest weight that stays and how many of its
// equals do; then one ordered pass writes the indices. A cluster of CTAs takes a row, each
// CTA a contiguous part of its tokens, kept in shared memory as far as it has room; the
// histograms are summed over the cluster through distributed shared memory.
#include "loop.cuh"
#include "tile.cuh"

#include <atomic>

namespace hpc {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kPasses = 3;
constexpr int kMaxCluster = 8;
// Keys that a CTA keeps in shared memory: with the histograms 96 KB, so that two CTAs fit an SM.
constexpr int kCached = 16384;

struct Smem {
    uint32_t hist[kPasses][kBins];
    uint32_t scan[kWarps];
    uint32_t found[4];          // bin, count above it, count in it
    uint32_t above, equal;      // of this CTA's part
    uint32_t warp_above[kWarps], warp_equal[kWarps];
    uint32_t keys[kCached];
};

// Unsigned numbers in the order of the floats; -0 counts as 0, and NaN as less than all.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 is 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads) kv_select_kernel(const KvSelectArgs a, int cluster) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int rank = (int)(blockIdx.x % (unsigned)cluster);
    const long long row = blockIdx.x / (unsigned)cluster;  // b * Hkv + h
    const int b = (int)(row / a.num_kv_heads);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kPasses * kBins; i += kThreads) (&sm.hist[0][0])[i] = 0u;
    grid_dependency_wait();
    grid_launch_dependents();
    long long L64 = a.seq_lens[b];
    if (tid == 0 && a.err) {
        if (L64 < 0) atomicOr(a.err, (int)HPC_DEVERR_NEGATIVE_LENGTH);
        if (L64 > a.w_stride) atomicOr(a.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
    }
    const int L = (int)max(0LL, min(L64, a.w_stride));
    const int kept = min(L, a.budget);
    if (rank == 0 && tid == 0 && row % a.num_kv_heads == 0) a.keep_lens[b] = kept;
    int32_t* keep = a.keep + row * a.budget;
    const int step = cluster * kThreads, at = rank * kThreads + tid;
    if (L <= a.budget) {
        for (int i = at; i < a.budget; i += step) keep[i] = i < L ? i : -1;
        return;
    }
    for (int i = at; i < a.first; i += step) keep[i] = i;
    for (int i = at; i < a.recent; i += step) keep[a.budget - a.recent + i] = L - a.recent + i;
    uint32_t need = (uint32_t)(a.budget - a.first - a.recent);
    if (need == 0) return;
    const float* w = a.weights + row * a.w_stride + a.first;
    const int M = L - a.recent - a.first;
    const int part = (M + cluster - 1) / cluster;
    const int lo = min(M, rank * part), n = min(M, lo + part) - lo;
    w += lo;
    uint32_t prefix = 0, mask = 0;
    for (int pass = 0; pass < kPasses; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit = pass == 2 ? 1023u : 2047u;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            uint32_t key;
            if (pass == 0) {
                key = order_key(w[i]);
                if (i < kCached) sm.keys[i] = key;
            } else {
                key = i < kCached ? sm.keys[i] : order_key(w[i]);
            }
            if ((key & mask) == prefix) atomicAdd(&sm.hist[pass][(key >> shift) & digit], 1u);
        }
        if (cluster > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        // two bins per thread, the largest first
        uint32_t c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int bin = kBins - 1 - (2 * tid + k);
            c[k] = 0;
            for (int r = 0; r < cluster; ++r) c[k] += cluster > 1 ? cluster_load_u32(cluster_addr(&sm.hist[pass][bin], r)) : sm.hist[pass][bin];
        }
        uint32_t sum = c[0] + c[1], incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sm.scan[warp] = incl;
        __syncthreads();
        uint32_t before = 0;
        for (int k = 0; k < warp; ++k) before += sm.scan[k];
        const uint32_t e0 = before + incl - sum, e1 = e0 + c[0];
        if (e0 < need && need <= e0 + c[0]) {
            sm.found[0] = kBins - 1 - 2 * tid;
            sm.found[1] = e0;
        }
        if (e1 < need && need <= e1 + c[1]) {
            sm.found[0] = kBins - 2 - 2 * tid;
            sm.found[1] = e1;
        }
        __syncthreads();
        prefix |= sm.found[0] << shift;
        mask |= digit << shift;
        need -= sm.found[1];
    }
    // `prefix` is the smallest key that stays, `need` of its equals do. Each warp takes a
    // contiguous part: counts first, then places.
    const int wpart = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int w0 = min(n, warp * wpart), w1 = min(n, w0 + wpart);
    uint32_t above = 0, equal = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t key = i < kCached ? sm.keys[i] : order_key(w[i]);
        above += key > prefix;
        equal += key == prefix;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        sm.warp_above[warp] = above;
        sm.warp_equal[warp] = equal;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t x = 0, y = 0;
        for (int k = 0; k < kWarps; ++k) {
            x += sm.warp_above[k];
            y += sm.warp_equal[k];
        }
        sm.above = x;
        sm.equal = y;
    }
    if (cluster > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    uint32_t na = 0, ne = 0;  // of the tokens before this warp's
    for (int r = 0; r < rank; ++r) {
        na += cluster_load_u32(cluster_addr(&sm.above, r));
        ne += cluster_load_u32(cluster_addr(&sm.equal, r));
    }
    for (int k = 0; k < warp; ++k) {
        na += sm.warp_above[k];
        ne += sm.warp_equal[k];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < w1 ? (i < kCached ? sm.keys[i] : order_key(w[i])) : 0u;
        const uint32_t ma = __ballot_sync(0xffffffffu, i < w1 && key > prefix);
        const uint32_t me = __ballot_sync(0xffffffffu, i < w1 && key == prefix);
        const uint32_t ea = na + __popc(ma & below), ee = ne + __popc(me & below);
        const bool stays = (ma >> lane & 1u) || ((me >> lane & 1u) && ee < need);
        if (stays) keep[a.first + ea + min(ee, need)] = a.first + lo + i;
        na += __popc(ma);
        ne += __popc(me);
    }
    if (cluster > 1) {  // the counts are read by the other CTAs
        cluster_arrive();
        cluster_wait();
    }
}

}  // namespace

cudaError_t launch_kv_select(const KvSelectArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&kv_select_kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sizeof(Smem));
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e;
        }
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    const long long rows = (long long)a.batch * a.num_kv_heads;
    int cluster = 1;
    while (cluster < kMaxCluster && rows * cluster < 2LL * tile_default_ctas() && a.w_stride > 2048LL * cluster) cluster *= 2;
    return launch_pdl_cluster(kv_select_kernel, dim3((unsigned)(rows * cluster)), dim3(kThreads), sizeof(Smem), cluster, s, a, cluster);
}

}  // namespace hpc
