// Verification of drafted tokens (hpc_verify_drafts). Draft i of a request is accepted while
//   u_i q_i(d_i) < p_i(d_i)
// (p_i the target's, q_i the draft's probabilities, u_i a given random number); at the first
// refusal r the next token is drawn from max(p_r - q_r, 0), after the last draft from p_r, as
// the least v whose running sum exceeds u times the whole sum.
//
// A token is a whole number, so a sum that is off by a rounding in 32 bits would now and then
// answer with a neighbour. Differences and sums are therefore kept as unevaluated pairs of
// floats (Knuth's two-sum and its difference form: exact errors, The Art of Computer
// Programming, vol. 2, 4.2.2), which holds 48 bits at the rate of 32-bit additions; 64-bit
// ones would bound the kernel. Per-thread sums are joined in 64 bits.
//
// Only row r of p and q is read whole. A cluster of CTAs takes a request, each warp a
// contiguous part of the vocabulary; the parts' sums say which warp holds the token, and
// that warp alone goes through its part again.
#include "loop.cuh"
#include "tile.cuh"

namespace hpc {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kRun = 8;  // consecutive entries of a lane in the second pass
constexpr float kMost = 18446744073709551616.f;  // entries from 2^64 on count as 0

struct Pair {
    float s, e;
};

// The weight of an entry, exact as s + e: p, or p - q where that is above 0.
__device__ __forceinline__ Pair entry(float p, float q, bool both) {
    if (!both) q = 0.f;
    const float s = p - q;
    const float bb = s - p;
    const float e = (p - (s - bb)) - (q + bb);
    const bool ok = s > 0.f && s < kMost;
    return Pair{ok ? s : 0.f, ok ? e : 0.f};
}

__device__ __forceinline__ void add(Pair& a, const Pair& x) {
    const float t = a.s + x.s;
    const float bb = t - a.s;
    a.e += ((a.s - (t - bb)) + (x.s - bb)) + x.e;
    a.s = t;
}

template <bool BF16>
__device__ __forceinline__ float load(const void* p, long long i) {
    if constexpr (BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    else
        return static_cast<const float*>(p)[i];
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a, int cluster) {
    __shared__ int accepted_sh;
    __shared__ double warp_sum[kWarps];
    __shared__ double cta_sum[2];  // of the residual, and of p alone
    const int rank = (int)(blockIdx.x % (unsigned)cluster);
    const long long b = blockIdx.x / (unsigned)cluster;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int count = a.counts ? max(0, min(a.drafts, a.counts[b])) : a.drafts;
    if (warp == 0) {
        bool yes = false;
        if (lane < count) {
            const int d = a.drafted[b * a.drafts + lane];
            if ((unsigned)d < (unsigned)a.vocab) {
                const float p = load<BF16>(a.target, (b * (a.drafts + 1) + lane) * a.target_stride + d);
                const float q = a.draft ? load<BF16>(a.draft, (b * a.drafts + lane) * a.draft_stride + d) : 1.f;
                yes = (double)a.accept_rand[b * a.drafts + lane] * (double)q < (double)p;
            } else if (rank == 0 && a.err) {
                atomicOr(a.err, (int)HPC_DEVERR_BAD_TOKEN);
            }
        }
        const uint32_t no = ~__ballot_sync(0xffffffffu, yes);
        const int r = min(count, no ? __ffs(no) - 1 : 32);
        if (lane == 0) accepted_sh = r;
        if (rank == 0) {
            if (lane < r) a.tokens[b * (a.drafts + 1) + lane] = a.drafted[b * a.drafts + lane];
            if (lane > r && lane <= a.drafts) a.tokens[b * (a.drafts + 1) + lane] = -1;
            if (lane == 0) {
                a.accepted[b] = r;
                if (a.kept_lens) a.kept_lens[b] = max(0, a.seq_lens[b] - (a.drafts - r));
            }
        }
    }
    __syncthreads();
    const int r = accepted_sh;
    const bool refused = r < count;
    constexpr int kSize = BF16 ? 2 : 4;
    const void* p = static_cast<const uint8_t*>(a.target) + (b * (a.drafts + 1) + r) * a.target_stride * kSize;
    const void* q = refused && a.draft ? static_cast<const uint8_t*>(a.draft) + (b * a.drafts + r) * a.draft_stride * kSize : nullptr;
    // without the draft's probabilities a refused token alone is out
    int out = refused && !a.draft ? a.drafted[b * a.drafts + r] : -1;
    const long long parts = (long long)cluster * kWarps;
    const long long part = ((a.vocab + parts - 1) / parts + 31) / 32 * 32;
    const long long v0 = min((long long)a.vocab, (rank * kWarps + warp) * part), v1 = min((long long)a.vocab, v0 + part);
    double pre = 0., border = 0.;  // the sum before this CTA's part, and u times the whole sum
    int owner = -1;  // the CTA of the cluster that holds the token
    for (int mode = 0; mode < 2; ++mode) {
        if (mode == 1) {  // nothing is left of the row: the target's probabilities alone
            q = nullptr;
            out = -1;
        }
        Pair acc{0.f, 0.f};
        for (long long v = v0 + lane; v < v1; v += 32) {
            Pair x = entry(load<BF16>(p, v), q ? load<BF16>(q, v) : 0.f, q != nullptr);
            if (v == out) x = Pair{0.f, 0.f};
            add(acc, x);
        }
        double s = (double)acc.s + (double)acc.e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) warp_sum[warp] = s;
        __syncthreads();
        if (tid == 0) {
            double c = 0.;
            for (int k = 0; k < kWarps; ++k) c += warp_sum[k];
            cta_sum[mode] = c;
        }
        if (cluster > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        double sums[kMaxCluster];
        double total = 0.;
        for (int k = 0; k < cluster; ++k) {
            sums[k] = cluster > 1 ? cluster_load_f64(cluster_addr(&cta_sum[mode], k)) : cta_sum[mode];
            total += sums[k];
        }
        if (total > 0.) {
            border = (double)a.sample_rand[b] * total;
            double c = 0.;
            for (int k = 0; k < cluster; ++k) {
                if (sums[k] > 0.) {
                    owner = k;
                    pre = c;
                    if (c + sums[k] > border) break;
                }
                c += sums[k];
            }
            break;
        }
    }
    if (cluster > 1) cluster_arrive();
    if (owner < 0) {
        if (rank == 0 && tid == 0) a.tokens[b * (a.drafts + 1) + r] = -1;
    } else if (owner == rank) {
        int mine = -1;
        double c = pre;
        for (int k = 0; k < kWarps; ++k) {
            if (warp_sum[k] > 0.) {
                mine = k;
                pre = c;
                if (c + warp_sum[k] > border) break;
            }
            c += warp_sum[k];
        }
        if (warp == mine) {
            long long token = -1, last = -1;
            for (long long i = v0; i < v1; i += 32 * kRun) {
                double x[kRun], s = 0.;
                int top = -1;
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    const long long v = i + lane * kRun + k;
                    Pair y{0.f, 0.f};
                    if (v < v1 && v != out) y = entry(load<BF16>(p, v), q ? load<BF16>(q, v) : 0.f, q != nullptr);
                    x[k] = (double)y.s + (double)y.e;
                    if (y.s > 0.f) top = k;
                    s += x[k];
                }
                double incl = s;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                const uint32_t over = __ballot_sync(0xffffffffu, s > 0. && pre + incl > border);
                const uint32_t some = __ballot_sync(0xffffffffu, top >= 0);
                if (some) {
                    const int l = 31 - __clz(some);
                    last = i + l * kRun + __shfl_sync(0xffffffffu, top, l);
                }
                if (over) {
                    const int l = __ffs(over) - 1;
                    double upto = pre + (incl - s);
                    int at = -1;
#pragma unroll
                    for (int k = 0; k < kRun; ++k) {
                        upto += x[k];
                        if (at < 0 && x[k] > 0. && upto > border) at = k;
                    }
                    if (at < 0) at = top;  // the lane's sum was rounded up past the border
                    token = i + l * kRun + __shfl_sync(0xffffffffu, at, l);
                    break;
                }
                pre += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) a.tokens[b * (a.drafts + 1) + r] = (int32_t)(token >= 0 ? token : last);
        }
    }
    if (cluster > 1) cluster_wait();  // the others read this CTA's sums
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, bool bf16, cudaStream_t s) {
    int cluster = 1;
    while (cluster < kMaxCluster && (long long)a.batch * cluster < tile_default_ctas() && a.vocab > 4096LL * cluster) cluster *= 2;
    const dim3 grid((unsigned)((long long)a.batch * cluster));
    return bf16 ? launch_pdl_cluster(verify_kernel<true>, grid, dim3(kThreads), 0, cluster, s, a, cluster)
                : launch_pdl_cluster(verify_kernel<false>, grid, dim3(kThreads), 0, cluster, s, a, cluster);
}

}  // namespace hpc
