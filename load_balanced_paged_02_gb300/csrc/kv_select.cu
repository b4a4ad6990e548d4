// Which cached tokens stay (hpc_kv_select): of each (sequence, KV head) the first and the
// most recent ones, and of those between them the ones with the largest weights, ties going
// to the lowest index; their indices in rising order.
//
// Radix selection on the weights' bits, mapped to unsigned numbers of the same order: three
// histograms (11, 11 and 10 bits) give the smallest weight that stays and how many of its
// equals do. The keys stay in shared memory, and all of them are gone through three times:
// loaded and put into the first histogram; looked through for the ones in the bin found,
// which go to a list that gives the other two histograms (a bin of too many is gone through
// again instead); and written, each thread a run of its own at the place that the counts
// give. Nothing in these loops branches on a key.
//
// A CTA takes a row. Rows differ in length, and the time is that of the longest, so where
// the array has room for more than 8192 tokens CTAs have 1024 threads and take the rows in
// order of falling length (512 rows of lengths log-uniform in [128, 65536]: 41 us, in the
// batch's order 52; 512 rows of 4096 tokens with 512 threads 21 us, with 1024 and in order 35).
// Where rows are fewer than SMs, clusters of up to 8 CTAs share each, a contiguous part of its
// tokens for each CTA, and sum the histograms through distributed shared memory (8 rows of
// 262144: 28 us, 317 by single CTAs of 512 threads). Clusters for every row, whose CTAs leave
// where it is short, are placed as one and took 64 us for the first batch. What bounds a row
// is the instructions of the three passes, about 30 for 32 keys each, and five barriers.
#include "loop.cuh"
#include "tile.cuh"

#include <atomic>

namespace hpc {
namespace {

constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kLeastPart = 4096;                 // tokens of a CTA at least, before another takes part
constexpr int kChunkKeys = 32768;                // keys that a CTA keeps in shared memory
constexpr int kList = 4096;                      // keys of one bin that the list has room for
constexpr int kLoads = 8;                        // keys that a thread has on their way at once
constexpr int kOrdered = 1024;                   // batches up to this are taken in order of length

struct Smem {
    uint32_t hist[2][kBins + 32];  // a lane that has nothing to count adds behind the bins: no branch
    uint2 list[kList + 32];        // key and place (likewise)
    uint32_t scan[32], scan2[32];
    uint32_t owned[1024];          // per thread: its tokens of the list, as counted by `count`
    uint32_t found[2];             // bin, tokens in higher bins
    uint32_t above, equal;         // tokens of this CTA's part
    uint32_t listed;
    int32_t request;
    uint32_t keys[1];              // [the longest part, at most kChunkKeys, and 1024 kLoads more]
};

// Unsigned numbers in the order of the floats; -0 counts as 0, and NaN as less than all.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 is 0
    const uint32_t k = u ^ (uint32_t)((int32_t)u >> 31 | (int32_t)0x80000000);
    return x != x ? 0u : k;
}

__device__ __forceinline__ void store_if(uint32_t yes, int32_t* p, int32_t v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p st.global.b32 [%1], %2;\n\t}" ::"r"(yes), "l"(p), "r"(v) : "memory");
}

// The sum of x over the threads before this one.
template <int kThreads>
__device__ __forceinline__ uint32_t block_before(uint32_t* scan, uint32_t x, int lane, int warp) {
    uint32_t incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < warp ? scan[lane] : 0u) + incl - x;
}

// Bins [first, first + N) summed over the cluster's `active` CTAs.
template <int N>
__device__ __forceinline__ void cluster_bins(const uint32_t* hist, int first, int active, uint32_t (&sum)[N]) {
    if (active == 1) {
#pragma unroll
        for (int k = 0; k < N; ++k) sum[k] = hist[first + k];
        return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] = 0;
    uint32_t x[kMaxCluster][N];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
        if (r >= active) break;
        const uint32_t at = cluster_addr(hist + first, r);
#pragma unroll
        for (int k = 0; k < N; k += 2)
            asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(x[r][k]), "=r"(x[r][k + 1]) : "r"(at + 4 * k));
    }
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
        if (r >= active) break;
#pragma unroll
        for (int k = 0; k < N; ++k) sum[k] += x[r][k];
    }
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1536 / kThreads) kv_select_kernel(const KvSelectArgs a, int cluster) {
    constexpr int kWarps = kThreads / 32, kOwnBins = kBins / kThreads;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int rank = (int)(blockIdx.x % (unsigned)cluster);
    const long long turn = blockIdx.x / (unsigned)cluster;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < 2 * (kBins + 32); i += kThreads) (&sm.hist[0][0])[i] = 0u;
    sm.owned[tid] = 0u;
    if (tid == 0) sm.listed = 0u;
    grid_dependency_wait();
    grid_launch_dependents();
    int b = (int)(turn / a.num_kv_heads);
    if (kThreads == 1024 && a.batch > 1 && a.batch <= kOrdered) {
        // the request that has b longer ones (of equals, the ones before it)
        int32_t* lens = reinterpret_cast<int32_t*>(sm.keys);
        for (int i = tid; i < a.batch; i += kThreads) lens[i] = a.seq_lens[i];
        __syncthreads();
        for (int i = tid; i < a.batch; i += kThreads) {
            const int mine = lens[i];
            int longer = 0;
#pragma unroll 4
            for (int k = 0; k < a.batch; ++k) longer += lens[k] > mine || (lens[k] == mine && k < i);
            if (longer == b) sm.request = i;
        }
        __syncthreads();
        b = sm.request;
        __syncthreads();  // (the keys take the place of the lengths)
    }
    const long long row = (long long)b * a.num_kv_heads + turn % a.num_kv_heads;
    const long long L64 = a.seq_lens[b];
    const int L = (int)max(0LL, min(L64, a.w_stride));
    // the middle, from which tokens are chosen, and the CTAs that share it
    const int M = L <= a.budget ? 0 : L - a.recent - a.first;
    const int part = max((M + cluster - 1) / cluster, kLeastPart);
    const int active = max(1, (M + part - 1) / part);
    if (rank >= active) return;  // a cluster's barrier waits for the CTAs that are there
    if (rank == 0 && tid == 0) {
        if (row % a.num_kv_heads == 0) a.keep_lens[b] = min(L, a.budget);
        if (a.err && L64 < 0) atomicOr(a.err, (int)HPC_DEVERR_NEGATIVE_LENGTH);
        if (a.err && L64 > a.w_stride) atomicOr(a.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
    }
    int32_t* keep = a.keep + row * a.budget;
    const int step = active * kThreads, at = rank * kThreads + tid;
    if (L <= a.budget) {
        for (int i = at; i < a.budget; i += step) keep[i] = i < L ? i : -1;
        return;
    }
    for (int i = at; i < a.first; i += step) keep[i] = i;
    for (int i = at; i < a.recent; i += step) keep[a.budget - a.recent + i] = L - a.recent + i;
    uint32_t need = (uint32_t)(a.budget - a.first - a.recent);
    if (need == 0) return;
    const int lo = rank * part, n = min(M, lo + part) - lo;
    const float* w = a.weights + row * a.w_stride + a.first + lo;

    // A chunk of up to kChunkKeys tokens in shared memory; each thread has a run of them, of odd
    // length, so that the lanes' reads fall into different banks.
    const int chunks = (n + kChunkKeys - 1) / kChunkKeys;
    int c0 = 0, m = 0, run = 0;  // the chunk's first token, its tokens, and a thread's
    auto load = [&](int c, uint32_t* hist) {  // hist: the first histogram, or null
        if (chunks > 1) __syncthreads();
        c0 = c * kChunkKeys;
        m = min(kChunkKeys, n - c0);
        run = ((m + kThreads - 1) / kThreads) | 1;
#pragma unroll 1
        for (int i = tid; i < m; i += kThreads * kLoads) {
            float x[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
                if (i + kThreads * k < m) x[k] = __ldg(w + c0 + i + kThreads * k);
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const uint32_t key = order_key(x[k]);
                const bool in = i + kThreads * k < m;
                sm.keys[i + kThreads * k] = key;
                if (hist) atomicAdd(&hist[in ? key >> 21 : kBins + lane], 1u);
            }
        }
    };
    // Of the bins of a histogram, the one with the token number `need` from the largest down.
    auto find = [&](const uint32_t* hist) {
        if (active > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        uint32_t v[kOwnBins], sum = 0;
        const int first_bin = kBins - kOwnBins * (tid + 1);
        cluster_bins<kOwnBins>(hist, first_bin, active, v);
#pragma unroll
        for (int k = 0; k < kOwnBins; ++k) sum += v[k];
        uint32_t higher = block_before<kThreads>(sm.scan, sum, lane, warp);
#pragma unroll
        for (int k = kOwnBins - 1; k >= 0; --k) {
            if (higher < need && need <= higher + v[k]) {
                sm.found[0] = first_bin + k;
                sm.found[1] = higher;
            }
            higher += v[k];
        }
        __syncthreads();
        need -= sm.found[1];
        return sm.found[0];
    };
    for (int c = 0; c < chunks; ++c) load(c, sm.hist[0]);
    const uint32_t top = find(sm.hist[0]);
    // the keys of that bin; and how many of this thread's run are above it (one chunk only)
    uint32_t mine = 0;  // above in the upper, equals in the lower half word
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) {
            load(c, nullptr);
            __syncthreads();
        }
        const int i0 = min(m, tid * run), i1 = min(m, i0 + run);
#pragma unroll 1
        for (int i = i0; i < i1; i += kLoads) {
            uint32_t key[kLoads], in_bin = 0;
#pragma unroll
            for (int k = 0; k < kLoads; ++k) key[k] = sm.keys[i + k];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const uint32_t in = i + k < i1, d = key[k] >> 21;
                mine += (in & (d > top)) << 16;
                in_bin |= (in & (d == top)) << k;
            }
            if (in_bin) {
                uint32_t place = atomicAdd(&sm.listed, (uint32_t)__popc(in_bin));
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    sm.list[(in_bin >> k & 1u) && place < kList ? place : kList + lane] = make_uint2(key[k], (uint32_t)tid);
                    place += in_bin >> k & 1u;
                }
            }
        }
    }
    __syncthreads();
    const int listed = (int)sm.listed;
    const bool all = listed > kList;  // too many: gone through again
    // histogram of (key >> shift) & digit of the keys with key & mask == prefix
    auto refine = [&](uint32_t* hist, uint32_t prefix, uint32_t mask, int shift, uint32_t digit) {
        if (!all) {
            for (int i = tid; i < listed; i += kThreads) {
                const uint32_t key = sm.list[i].x;
                atomicAdd(&hist[(key & mask) == prefix ? (key >> shift) & digit : kBins + lane], 1u);
            }
            return;
        }
        for (int c = 0; c < chunks; ++c) {
            if (chunks > 1) {
                load(c, nullptr);
                __syncthreads();
            }
#pragma unroll 1
            for (int i = tid; i < m; i += kThreads * kLoads) {
                uint32_t key[kLoads];
#pragma unroll
                for (int k = 0; k < kLoads; ++k) key[k] = sm.keys[i + kThreads * k];
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const bool one = i + kThreads * k < m && (key[k] & mask) == prefix;
                    atomicAdd(&hist[one ? (key[k] >> shift) & digit : kBins + lane], 1u);
                }
            }
        }
    };
    uint32_t prefix = top << 21;
    refine(sm.hist[1], prefix, 0xffe00000u, 10, 2047u);
    prefix |= find(sm.hist[1]) << 10;
    // (the third histogram takes the first one's place, which every CTA read before the second's barrier)
    for (int i = tid; i < kBins; i += kThreads) sm.hist[0][i] = 0u;
    __syncthreads();
    refine(sm.hist[0], prefix, 0xfffffc00u, 0, 1023u);
    prefix |= find(sm.hist[0]);

    // `prefix` is the smallest key that stays, and `need` of its equals do. Counts first, above
    // in the upper and equals in the lower half of a word (a chunk has fewer than 2^16), then places.
    auto weigh = [&](uint32_t key) { return ((uint32_t)(key > prefix) << 16) + (uint32_t)(key == prefix); };
    static_assert(kChunkKeys < 65536, "counts of a chunk in half words");
    auto count = [&]() {  // of the run in the chunk that is there
        uint32_t x = 0;
        const int i1 = min(m, (tid + 1) * run);
#pragma unroll 8
        for (int i = min(m, tid * run); i < i1; ++i) x += weigh(sm.keys[i]);
        return x;
    };
    const bool again = all || chunks > 1;  // the counts are taken from all the keys, or from the list's
    if (!again) {
        for (int i = tid; i < listed; i += kThreads) {
            const uint2 x = sm.list[i];
            atomicAdd(&sm.owned[x.y], weigh(x.x));
        }
        __syncthreads();
        mine += sm.owned[tid];
    }
    uint32_t na = 0, ne = 0;  // kept for certain, and equals, among the tokens before this chunk
    if (active > 1) {
        uint32_t above = again ? 0 : mine >> 16, equal = again ? 0 : mine & 0xffffu;
        for (int c = 0; again && c < chunks; ++c) {
            if (chunks > 1) {
                load(c, nullptr);
                __syncthreads();
            }
            const uint32_t x = count();
            above += x >> 16;
            equal += x & 0xffffu;
        }
        above = __reduce_add_sync(0xffffffffu, above);
        equal = __reduce_add_sync(0xffffffffu, equal);
        if (lane == 0) {
            sm.scan[warp] = above;
            sm.scan2[warp] = equal;
        }
        __syncthreads();
        if (warp == 0) {
            above = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm.scan[lane] : 0u);
            equal = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm.scan2[lane] : 0u);
            if (lane == 0) {
                sm.above = above;
                sm.equal = equal;
            }
        }
        cluster_arrive();
        cluster_wait();
        uint32_t x = 0, y = 0;
        if (lane < rank) {
            x = cluster_load_u32(cluster_addr(&sm.above, lane));
            y = cluster_load_u32(cluster_addr(&sm.equal, lane));
        }
        na = __reduce_add_sync(0xffffffffu, x);
        ne = __reduce_add_sync(0xffffffffu, y);
        cluster_arrive();  // (waited for at the end: the others read this CTA's counts)
    }
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) load(c, nullptr);
        __syncthreads();
        if (again) mine = count();
        const uint32_t before = block_before<kThreads>(sm.scan, mine, lane, warp);
        uint32_t above = na + (before >> 16), equal = ne + (before & 0xffffu);
        const int i0 = min(m, tid * run), i1 = min(m, i0 + run);
        const int32_t first_token = a.first + lo + c0;
#pragma unroll 1
        for (int i = i0; i < i1; i += kLoads) {
            uint32_t key[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) key[k] = sm.keys[i + k];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const uint32_t in = i + k < i1, more = in & (key[k] > prefix), same = in & (key[k] == prefix);
                store_if(more | (same & (equal < need)), keep + a.first + above + min(equal, need), first_token + i + k);
                above += more;
                equal += same;
            }
        }
        if (chunks > 1) {
            if (tid == kThreads - 1) {
                sm.scan2[0] = above;
                sm.scan2[1] = equal;
            }
            __syncthreads();
            na = sm.scan2[0];
            ne = sm.scan2[1];
        }
    }
    if (active > 1) cluster_wait();
}

template <int kThreads>
cudaError_t launch(const KvSelectArgs& a, int cluster, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    constexpr size_t kMost = sizeof(Smem) + (kChunkKeys + kThreads * kLoads) * sizeof(uint32_t);
    static_assert(kMost <= 232448, "over the 227 KB shared-memory limit of a CTA");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&kv_select_kernel<kThreads>), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e;
        }
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    long long part = (a.w_stride + cluster - 1) / cluster;
    if (part < kLeastPart) part = kLeastPart;
    if (part > kChunkKeys) part = kChunkKeys;
    part += kThreads * kLoads;  // written or read past the last key, and not used
    return launch_pdl_cluster(kv_select_kernel<kThreads>, dim3((unsigned)((long long)a.batch * a.num_kv_heads * cluster)), dim3(kThreads),
                              sizeof(Smem) + (size_t)part * sizeof(uint32_t), cluster, s, a, cluster);
}

}  // namespace

cudaError_t launch_kv_select(const KvSelectArgs& a, cudaStream_t s) {
    // several CTAs per row only while every one of them has an SM of its own
    const long long rows = (long long)a.batch * a.num_kv_heads, sms = tile_default_ctas();
    int cluster = 1;
    while (cluster < kMaxCluster && rows * cluster * 2 <= sms && a.w_stride > (long long)kLeastPart * cluster) cluster *= 2;
    return a.w_stride > 8192 ? launch<1024>(a, cluster, s) : launch<512>(a, cluster, s);
}

}  // namespace hpc
