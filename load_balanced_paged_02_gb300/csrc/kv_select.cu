// Which cached tokens stay (hpc_kv_select): of each (sequence, KV head) the first and the
// most recent ones, and of those between them the ones with the largest weights, ties going
// to the lowest index; their indices in rising order.
//
// Radix selection on the weights' bits, mapped to unsigned numbers of the same order: three
// histograms (11, 11 and 10 bits) give the smallest weight that stays and how many of its
// equals do. All weights are gone through twice: for the first histogram, by their own upper bits
// (its bins are brought in order when it is summed), and for the list of those that reach the bin
// found, which each warp keeps in shared memory for its part of the row, in order. Whatever
// follows, the other two histograms, the counts and the indices, needs the lists alone. A warp
// that has more of them than its list has room for goes through its part again each time (24 x 8
// rows of 65536, half of them kept: 70 us; through the rows in shared memory, as before the lists, 99).
//
// A CTA of 512 threads takes a row, two of them an SM: a row's fixed costs, five barriers and
// the round trips between them, about 5 us, are covered by the other's (512 rows of lengths
// log-uniform in [128, 65536]: 23 us; one CTA of 1024 threads per SM 29, four of 256 25). Where the
// array has room for more than 8192 tokens they take the rows in order of falling length
// (in the batch's order 27; finding the order costs rows of 4096 tokens 2 us of 19). Where rows are
// fewer than SMs, clusters of up to 8 CTAs share each, a contiguous part of its tokens for
// each CTA, and sum the histograms through distributed shared memory: 64 groups of bins, then
// the one group's (8 rows of 262144: 19 us, 137 by single CTAs; whole histograms, read by
// every CTA, 23). Clusters for every row, whose CTAs leave where it is short, are
// placed as one and took 64 us for the first batch. What bounds a row of 65536 is its two
// passes, 5 us each for one CTA, at about 15 instructions for 32 weights.
#include "loop.cuh"
#include "tile.cuh"

#include <atomic>
#include <climits>

namespace hpc {
namespace {

constexpr int kBins = 2048;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kLeastPart = 4096;                 // tokens of a CTA at least, before another takes part
constexpr int kMostListed = 640;                 // tokens that a warp's list has room for at most
constexpr int kLoads = 8;                        // weights that a thread has on their way at once
constexpr long long kShort = 8192;               // rows up to this are taken as they come
constexpr int kOrdered = 1024;                   // batches up to this are taken in order of length

struct Smem {
    uint32_t hist[3][kBins];
    uint32_t group[3][kBins / 32];
    uint32_t scan[32], scan2[32];
    uint32_t found[2];             // bin, and how many of its tokens stay
    uint32_t above, equal;         // tokens of this CTA's part
    int32_t request;
    uint2 list[1];                 // [warps][room]: weight and place
};

// Unsigned numbers in the order of the floats x + 0 (-0 counts as 0), NaN as less than all.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x);
    const uint32_t k = u ^ (uint32_t)((int32_t)u >> 31 | (int32_t)0x80000000);
    return x != x ? 0u : k;
}

// The first histogram is of the weights' own upper 11 bits (an addition's NaN is 0x7fffffff): where
// bin number `o` of order_key's is in it.
__device__ __forceinline__ int bin_of(int o) {
    if (o == 0) return 1023;     // NaN
    if (o == 2047) return 2047;  // (what would be NaN of the other sign: none)
    return o >= 1024 ? o - 1024 : 2047 - o;
}

__global__ void __launch_bounds__(kThreads, 2) kv_select_kernel(const KvSelectArgs a, int cluster, int room, bool ordered) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int rank = (int)(blockIdx.x % (unsigned)cluster);
    const long long turn = blockIdx.x / (unsigned)cluster;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < 3 * kBins; i += kThreads) (&sm.hist[0][0])[i] = 0u;
    grid_dependency_wait();
    grid_launch_dependents();
    int b = (int)(turn / a.num_kv_heads);
    if (ordered && a.batch > 1 && a.batch <= kOrdered) {
        // the request that has b longer ones (of equals, the ones before it)
        int32_t* lens = reinterpret_cast<int32_t*>(sm.list);
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
        __syncthreads();  // (the list takes the place of the lengths)
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

    // This warp's tokens: [s0, s1) of the middle.
    const int lo = rank * part, n = min(M, lo + part) - lo;
    const int seg = ((n + kWarps - 1) / kWarps + 31) & ~31;
    const int s0 = lo + min(n, warp * seg), s1 = lo + min(n, (warp + 1) * seg);
    const float* w = a.weights + row * a.w_stride + a.first;
    const uint32_t before_me = (1u << lane) - 1u;
    // f(weight + 0, place, whether there is one) for all of them in order, 32 at a time.
    auto sweep = [&](auto&& f) {
        const float* at = w + lane;
        int i = s0;
        float x[kLoads];
        if (i + 32 * kLoads <= s1) {
#pragma unroll
            for (int k = 0; k < kLoads; ++k) x[k] = at[i + 32 * k];
            bool next;
#pragma unroll 1
            do {
                next = i + 2 * 32 * kLoads <= s1;
                float y[kLoads];
                if (next) {
#pragma unroll
                    for (int k = 0; k < kLoads; ++k) y[k] = at[i + 32 * (kLoads + k)];
                }
#pragma unroll
                for (int k = 0; k < kLoads; ++k) f(x[k] + 0.f, i + 32 * k + lane, true);
                i += 32 * kLoads;
#pragma unroll
                for (int k = 0; k < kLoads; ++k) x[k] = y[k];
            } while (next);
        }
        if (i >= s1) return;
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            if (i + 32 * k + lane < s1) x[k] = at[i + 32 * k];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            if (i + 32 * k >= s1) break;
            f(x[k] + 0.f, i + 32 * k + lane, i + 32 * k + lane < s1);
        }
    };
    // Of the bins of a histogram, the one with the token number `need` from the largest down. In
    // a cluster first among groups of 32 bins, then in the group, both summed over its CTAs.
    auto find = [&](int turn) {
        const uint32_t* hist = sm.hist[turn];
        auto at = [&](int bin) { return hist + (turn == 0 ? bin_of(bin) : bin); };
        __syncthreads();
        if (active == 1) {  // each thread a few bins
            constexpr int kOwn = kBins / kThreads;
            uint32_t v[kOwn], sum = 0;
            const int first_bin = kBins - kOwn * (tid + 1);
#pragma unroll
            for (int k = 0; k < kOwn; ++k) sum += v[k] = *at(first_bin + k);
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (lane == 31) sm.scan[warp] = incl;
            __syncthreads();
            uint32_t higher = __reduce_add_sync(0xffffffffu, lane < warp ? sm.scan[lane] : 0u) + incl - sum;
#pragma unroll
            for (int k = kOwn - 1; k >= 0; --k) {
                if (higher < need && need <= higher + v[k]) {
                    sm.found[0] = first_bin + k;
                    sm.found[1] = need - higher;
                }
                higher += v[k];
            }
            __syncthreads();
            need = sm.found[1];
            return sm.found[0];
        }
        for (int g = warp; g < kBins / 32; g += kWarps) {
            const uint32_t x = __reduce_add_sync(0xffffffffu, *at(32 * g + lane));
            if (lane == 0) sm.group[turn][g] = x;
        }
        cluster_arrive();
        cluster_wait();
        if (warp == 0) {
            auto total = [&](const uint32_t* p) {
                uint32_t x[kMaxCluster], sum = 0;
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) x[r] = r < active ? cluster_load_u32(cluster_addr(p, r)) : 0u;
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) sum += x[r];
                return sum;
            };
            // lane 0 has the highest; the lane that reaches `need`, which becomes what is left of it there
            auto lane_of = [&](uint32_t x) {
                uint32_t incl = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                const int l = __ffs(__ballot_sync(0xffffffffu, incl >= need)) - 1;
                need -= __shfl_sync(0xffffffffu, incl - x, l);
                return l;
            };
            const uint32_t x = total(&sm.group[turn][63 - 2 * lane]), y = total(&sm.group[turn][62 - 2 * lane]);
            const int l = lane_of(x + y);
            const uint32_t higher = __shfl_sync(0xffffffffu, x, l);
            const bool second = need > higher;
            if (second) need -= higher;
            const int g = 63 - 2 * l - (second ? 1 : 0), bin = 32 * g + 31 - lane_of(total(at(32 * g + 31 - lane)));
            if (lane == 0) {
                sm.found[0] = (uint32_t)bin;
                sm.found[1] = need;
            }
        }
        __syncthreads();
        need = sm.found[1];
        return sm.found[0];
    };
    sweep([&](float x, int, bool in) {
        if (in) atomicAdd(&sm.hist[0][__float_as_uint(x) >> 21], 1u);
    });
    uint32_t prefix = find(0) << 21;

    // Only keys from here on can stay: the warp's list of them, in order
    uint2* list = sm.list + warp * room;
    int listed = 0;
    const float least = __uint_as_float(prefix ^ (prefix & 0x80000000u ? 0x80000000u : 0xffffffffu));
    if (prefix < 0x00800000u) {
        listed = INT_MAX;  // down to -infinity or NaN: no number is the least
    } else {
        sweep([&](float x, int i, bool in) {
            const bool stays = in && x >= least;
            const uint32_t those = __ballot_sync(0xffffffffu, stays);
            const int place = listed + __popc(those & before_me);
            if (stays && place < room) list[place] = make_uint2(__float_as_uint(x), (uint32_t)i);
            listed += __popc(those);
        });
    }
    __syncwarp();
    // f(key, place, whether there is one) for the list's, or, where it had no room for them, for all again.
    auto candidates = [&](auto&& f) {
        if (listed > room) {
            sweep([&](float x, int i, bool in) { f(order_key(x), i, in); });
            return;
        }
#pragma unroll 2
        for (int i = 0; i < listed; i += 32) {
            const uint2 x = i + lane < listed ? list[i + lane] : make_uint2(0u, 0u);
            f(order_key(__uint_as_float(x.x)), (int)x.y, i + lane < listed);
        }
    };
    candidates([&](uint32_t key, int, bool in) {
        if (in && key >> 21 == prefix >> 21) atomicAdd(&sm.hist[1][key >> 10 & 2047u], 1u);
    });
    prefix |= find(1) << 10;
    candidates([&](uint32_t key, int, bool in) {
        if (in && key >> 10 == prefix >> 10) atomicAdd(&sm.hist[2][key & 1023u], 1u);
    });
    prefix |= find(2);

    // `prefix` is the smallest key that stays, and `need` of its equals do. First how many are before this warp's.
    uint32_t above = 0, equal = 0;
    candidates([&](uint32_t key, int, bool in) {
        above += in && key > prefix;
        equal += in && key == prefix;
    });
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        sm.scan[warp] = above;
        sm.scan2[warp] = equal;
    }
    __syncthreads();
    const uint32_t above_of = lane < kWarps ? sm.scan[lane] : 0u, equal_of = lane < kWarps ? sm.scan2[lane] : 0u;
    above = __reduce_add_sync(0xffffffffu, lane < warp ? above_of : 0u);
    equal = __reduce_add_sync(0xffffffffu, lane < warp ? equal_of : 0u);
    if (active > 1) {
        if (warp == 0) {
            const uint32_t x = __reduce_add_sync(0xffffffffu, above_of), y = __reduce_add_sync(0xffffffffu, equal_of);
            if (lane == 0) {
                sm.above = x;
                sm.equal = y;
            }
        }
        cluster_arrive();
        cluster_wait();
        uint32_t x = 0, y = 0;
        if (lane < rank) {
            x = cluster_load_u32(cluster_addr(&sm.above, lane));
            y = cluster_load_u32(cluster_addr(&sm.equal, lane));
        }
        above += __reduce_add_sync(0xffffffffu, x);
        equal += __reduce_add_sync(0xffffffffu, y);
        cluster_arrive();  // (waited for at the end: the others read this CTA's counts)
    }
    keep += a.first;
    candidates([&](uint32_t key, int i, bool in) {
        const bool more = in && key > prefix, same = in && key == prefix;
        const uint32_t mores = __ballot_sync(0xffffffffu, more), sames = __ballot_sync(0xffffffffu, same);
        const uint32_t equals = equal + __popc(sames & before_me);
        if (more || (same && equals < need)) keep[above + __popc(mores & before_me) + min(equals, need)] = a.first + i;
        above += __popc(mores);
        equal += __popc(sames);
    });
    if (active > 1) cluster_wait();
}

cudaError_t launch(const KvSelectArgs& a, int cluster, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    constexpr size_t kMost = sizeof(Smem) + kWarps * kMostListed * sizeof(uint2);
    static_assert(kMost <= 115712, "two CTAs per SM");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&kv_select_kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e;
        }
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    long long room = (a.w_stride + cluster - 1) / cluster;  // a warp's tokens of the longest part
    if (room < kLeastPart) room = kLeastPart;
    room = ((room + kWarps - 1) / kWarps + 31) / 32 * 32;
    if (room > kMostListed) room = kMostListed;
    const size_t smem = sizeof(Smem) + kWarps * (size_t)room * sizeof(uint2);
    return launch_pdl_cluster(kv_select_kernel, dim3((unsigned)((long long)a.batch * a.num_kv_heads * cluster)), dim3(kThreads), smem,
                              cluster, s, a, cluster, (int)room, a.w_stride > kShort);
}

}  // namespace

cudaError_t launch_kv_select(const KvSelectArgs& a, cudaStream_t s) {
    // several CTAs per row only while every one of them has an SM of its own
    const long long rows = (long long)a.batch * a.num_kv_heads, sms = tile_default_ctas();
    int cluster = 1;
    while (cluster < kMaxCluster && rows * cluster * 2 <= sms && a.w_stride > (long long)kLeastPart * cluster) cluster *= 2;
    return launch(a, cluster, s);
}

}  // namespace hpc
