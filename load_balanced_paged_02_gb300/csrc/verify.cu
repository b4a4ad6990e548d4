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
// ones are so slow here (a warp's addition takes 16 cycles of its SM and more) that joining
// the threads' sums with them alone took 10 us; only the comparisons with the border are in
// 64 bits, in one warp.
//
// Only row r of p and q is read whole. A cluster of CTAs takes a request, each warp a
// contiguous part of the vocabulary; the parts' sums say which warp holds the token, and
// that warp alone goes through its part again, 2048 entries at a time in shared memory.
//
// The rows' bytes are the floor (256 requests of 131072 entries in 32 bits, target and draft:
// 268 MB, 40 us at the rate of a copy); 50-52 us is what it takes, 5.3 TB/s. Without the
// search it takes 47: a request begins with three round trips in a row (count, drafted token,
// its probabilities) and ends with two more, which the SM's other CTAs cover in part. In bf16 (512
// requests, 49 us) the issue slots are 55 % busy; rows off 16 bytes have fewer loads on their way (128
// requests of 100003 entries 27 us for 15 us of bytes), and so has the part that holds a certain
// draft that was refused (256 requests 49 us for 20).
#include "loop.cuh"
#include "tile.cuh"

#include <atomic>

namespace hpc {
namespace {

constexpr int kAhead = 4;
constexpr int kMaxCluster = 8;
constexpr int kPart = 256;  // a warp's part is a multiple of this many entries
constexpr float kMost = 18446744073709551616.f;  // entries from 2^64 on count as 0

struct Pair {
    float s, e;
};

// What of the draft's probability counts beside p >= 0: at most p, so that the difference is not
// below 0; 0 where q's sign is set; p, which leaves nothing, where q is NaN or infinite. Floats
// that are not negative have the order of their bits, so that this is one instruction.
__device__ __forceinline__ float within(float q, float p) {
    int32_t d;
    asm("min.relu.s32 %0, %1, %2;" : "=r"(d) : "r"(__float_as_int(q)), "r"(__float_as_int(p)));
    return __int_as_float(d);
}

// The weight of an entry, exact as s + e: p, or p - q, where that is below 2^64. As p' >= q' >= 0
// the difference's error is (p' - s) - q'.
__device__ __forceinline__ Pair entry(float p, float q, bool both) {
    p = fmaxf(p, 0.f);  // (the number where p is NaN)
    q = both ? within(q, p) : 0.f;
    const float s = p - q;
    const float e = (p - s) - q;
    const bool ok = s < kMost;
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

// Value k of 16 bytes of a row.
template <bool BF16>
__device__ __forceinline__ float at_k(const uint4& r, int k) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (BF16) return __uint_as_float(k & 1 ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
    return __uint_as_float(w[k]);
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two pairs side by side, in 64-bit registers: two additions for one issue slot.
struct Pair2 {
    uint64_t s, e;
};
__device__ __forceinline__ uint64_t pack(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 unpack(uint64_t v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ void add(Pair2& a, uint64_t s) {  // e is left alone where it is 0
    const uint64_t t = add2(a.s, s), bb = sub2(t, a.s);
    a.e = add2(a.e, add2(sub2(a.s, sub2(t, bb)), sub2(s, bb)));
    a.s = t;
}

// Two entries; a weight from 2^64 on makes the sum too large, which the caller sees.
template <bool BOTH>
__device__ __forceinline__ void add_entries(Pair2& acc, float p0, float p1, float q0, float q1) {
    p0 = fmaxf(p0, 0.f);
    p1 = fmaxf(p1, 0.f);
    if constexpr (BOTH) {
        const uint64_t p = pack(p0, p1), q = pack(within(q0, p0), within(q1, p1));
        const uint64_t s = sub2(p, q);
        acc.e = add2(acc.e, sub2(sub2(p, s), q));
        add(acc, s);
    } else {
        add(acc, pack(p0, p1));
    }
}

// A lane's part of the sum over entries [v0, v1) of a row. EACH looks at every entry on its
// own, for parts with an entry that is left out (`out`) or too large to be a probability.
// Rows on 16-byte boundaries come through shared memory, kAhead pieces of 16 bytes per lane
// and row on their way without a register: `ring` is this thread's [kAhead][2], kThreads apart.
template <int kThreads, bool BF16, bool BOTH, bool EACH>
__device__ __forceinline__ Pair lane_sum(const void* p, const void* q, long long v0, long long v1, int out, int lane, uint4* ring) {
    constexpr int kVec = BF16 ? 8 : 4, kSize = BF16 ? 2 : 4;
    Pair one{0.f, 0.f};
    Pair2 two{0, 0};
    long long v = v0;
    const bool wide = ((reinterpret_cast<uintptr_t>(p) | (BOTH ? reinterpret_cast<uintptr_t>(q) : 0)) & 15) == 0;
    if (!EACH && wide) {
        const int n = (int)((v1 - v0) / (32 * kVec));  // pieces of a lane
        const uint8_t* ps = static_cast<const uint8_t*>(p) + v0 * kSize + lane * 16;
        const uint8_t* qs = BOTH ? static_cast<const uint8_t*>(q) + v0 * kSize + lane * 16 : nullptr;
        auto fetch = [&](int i) {
            if (i < n) {
                copy16(ring + (i % kAhead) * 2 * kThreads, ps + i * 512);
                if (BOTH) copy16(ring + ((i % kAhead) * 2 + 1) * kThreads, qs + i * 512);
            }
            copy_commit();
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            copy_wait<kAhead - 1>();
            const uint4 x = ring[(i % kAhead) * 2 * kThreads];
            const uint4 y = BOTH ? ring[((i % kAhead) * 2 + 1) * kThreads] : make_uint4(0u, 0u, 0u, 0u);
            fetch(i + kAhead);
#pragma unroll
            for (int k = 0; k < kVec; k += 2)
                add_entries<BOTH>(two, at_k<BF16>(x, k), at_k<BF16>(x, k + 1), at_k<BF16>(y, k), at_k<BF16>(y, k + 1));
        }
        copy_wait<0>();
        v += (long long)n * 32 * kVec;
    }
    for (; v < v1; v += 32 * 8) {
        float x[8], y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const long long i = v + 32 * u + lane;
            x[u] = i < v1 ? load<BF16>(p, i) : 0.f;
            y[u] = BOTH && i < v1 ? load<BF16>(q, i) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
            if constexpr (EACH) {
#pragma unroll
                for (int k = u; k < u + 2; ++k)
                    if (v + 32 * k + lane != out) add(one, entry(x[k], y[k], BOTH));
            } else {
                add_entries<BOTH>(two, x[u], x[u + 1], y[u], y[u + 1]);
            }
        }
    }
    if (!EACH) {
        const float2 s = unpack(two.s), e = unpack(two.e);
        one = Pair{s.x, e.x};
        add(one, Pair{s.y, e.y});
    }
    return one;
}

// (out of line: it is rare, and would take registers from the usual path)
template <int kThreads, bool BF16>
__device__ __noinline__ Pair lane_sum_each(const void* p, const void* q, long long v0, long long v1, int out, int lane) {
    return q ? lane_sum<kThreads, BF16, true, true>(p, q, v0, v1, out, lane, nullptr)
             : lane_sum<kThreads, BF16, false, true>(p, q, v0, v1, out, lane, nullptr);
}

template <int kThreads, bool BF16>
__device__ __forceinline__ Pair lane_sum(const void* p, const void* q, long long v0, long long v1, int out, int lane, uint4* ring) {
    if (out < v0 || out >= v1) {
        const Pair x = q ? lane_sum<kThreads, BF16, true, false>(p, q, v0, v1, -1, lane, ring) : lane_sum<kThreads, BF16, false, false>(p, q, v0, v1, -1, lane, ring);
        if (__all_sync(0xffffffffu, x.s < kMost)) return x;
    }
    return lane_sum_each<kThreads, BF16>(p, q, v0, v1, out, lane);
}

__device__ __forceinline__ Pair shfl_up(const Pair& x, int o) {
    return Pair{__shfl_up_sync(0xffffffffu, x.s, o), __shfl_up_sync(0xffffffffu, x.e, o)};
}

// Sum of the lanes up to this one.
__device__ __forceinline__ Pair scan(Pair x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair y = shfl_up(x, o);
        if (lane >= o) add(x, y);
    }
    return x;
}

__device__ __forceinline__ double value(const Pair& x) { return (double)x.s + (double)x.e; }

// The first lane whose sum, after `before`, exceeds the border, or else the last with a weight at
// all (32 if `more` are to come); -1 if there is none. `before` becomes the sum before that lane.
__device__ __forceinline__ int find(const Pair& x, Pair& before, double& border, int lane, bool more = false) {
    const Pair incl = scan(x, lane);
    Pair upto = before;
    add(upto, incl);
    const bool some = x.s > 0.f;
    const uint32_t over = __ballot_sync(0xffffffffu, some && value(upto) > border), any = __ballot_sync(0xffffffffu, some);
    if (!any) return -1;
    const int l = over ? __ffs(over) - 1 : more ? 32 : 31 - __clz(any);
    if (!over && !more) border = INFINITY;  // the last one it stays
    if (l > 0) add(before, Pair{__shfl_sync(0xffffffffu, incl.s, l - 1), __shfl_sync(0xffffffffu, incl.e, l - 1)});
    return l;
}

// What the warp that looks for the token has a piece of the rows copied into: 32 lines, one for
// a lane, of 1 << log entries each (up to kLine), with room for 16 bytes more, so that the lanes'
// reads of 16 bytes fall into different banks.
constexpr int kLine = 64;
constexpr int kLeastLog = 3;  // 16 bytes of the shorter type
template <bool BF16>
struct Desk {
    static constexpr int kSize = BF16 ? 2 : 4, kPer16 = 16 / kSize;
    static constexpr int kStride = kLine * kSize + 16;
    static constexpr int kBytes = 32 * kStride;
};

// Entries [v0, v1) of a row, at most 32 << log, to the desk, zeros behind them: all of them on their
// way at once, as a round trip takes microseconds while others stream.
template <bool BF16>
__device__ __forceinline__ void to_desk(uint8_t* desk, const void* row, long long v0, long long v1, int log, int lane) {
    using D = Desk<BF16>;
    const int n = (int)(v1 - v0);
    const uint8_t* src = static_cast<const uint8_t*>(row) + v0 * D::kSize;
    if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
        const int per = log - (BF16 ? 3 : 2);  // of them in a line, as a power of two
#pragma unroll 4
        for (int i = lane; i < 32 << per; i += 32) {
            uint8_t* to = desk + (i >> per) * D::kStride + (i & (1 << per) - 1) * 16;
            const int bytes = max(0, min(16, (n - i * D::kPer16) * D::kSize));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(src + (bytes ? i * 16 : 0)), "r"(bytes) : "memory");
        }
    } else {
#pragma unroll 8
        for (int i = lane; i < 32 << log; i += 32) {
            uint8_t* to = desk + (i >> log) * D::kStride + (i & (1 << log) - 1) * D::kSize;
            if constexpr (BF16)
                *reinterpret_cast<uint16_t*>(to) = i < n ? reinterpret_cast<const uint16_t*>(src)[i] : (uint16_t)0;
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to)), "l"(src + (i < n ? i * 4 : 0)), "r"(i < n ? 4 : 0)
                             : "memory");
        }
    }
}

// The least entry of [w0, w1) whose running sum, from `before` on, exceeds the border, by a warp;
// should rounding leave none over it, the last entry with a weight. First the line, then the pair
// of entries, then the entry.
template <bool BF16>
__device__ __forceinline__ int search(uint8_t* desk, const void* p, const void* q, long long w0, long long w1, int out, Pair before, double border,
                                   int lane) {
    using D = Desk<BF16>;
    const uint8_t* pl = desk + lane * D::kStride;
    long long found = -1;
    for (long long v0 = w0;; v0 += 32 * kLine) {
        if (v0 >= w1) {  // no later part had a weight after all: the last entry with one is in an earlier part
            if (found < 0) return (int)w0;
            v0 = found;
            w1 = min(w1, v0 + 32 * kLine);
            border = INFINITY;
        }
        const long long v1 = min(w1, v0 + 32 * kLine);
        int log = kLeastLog;
        while (32 << log < v1 - v0) ++log;
        __syncwarp();
        to_desk<BF16>(desk, p, v0, v1, log, lane);
        if (q) to_desk<BF16>(desk + D::kBytes, q, v0, v1, log, lane);
        copy_commit();
        copy_wait<0>();
        __syncwarp();
        if (out >= v0 && out < v1 && lane == 0) {  // an entry that is left out
            const int i = (int)(out - v0);
            uint8_t* at = desk + (i >> log) * D::kStride + (i & (1 << log) - 1) * D::kSize;
            if constexpr (BF16)
                *reinterpret_cast<uint16_t*>(at) = 0;
            else
                *reinterpret_cast<float*>(at) = 0.f;
        }
        __syncwarp();
        Pair s[4] = {};
#pragma unroll 2
        for (int i = 0; i < 1 << log; i += D::kPer16) {
            const uint4 x = *reinterpret_cast<const uint4*>(pl + i * D::kSize);
            const uint4 y = q ? *reinterpret_cast<const uint4*>(pl + D::kBytes + i * D::kSize) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < D::kPer16; ++k) add(s[k & 3], entry(at_k<BF16>(x, k), at_k<BF16>(y, k), q != nullptr));
        }
        add(s[0], s[1]);
        add(s[2], s[3]);
        add(s[0], s[2]);
        const int line = find(s[0], before, border, lane, v1 < w1);
        if (line < 0) continue;
        found = v0;
        if (line == 32) continue;
        Pair e[2], two{0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint8_t* at = desk + line * D::kStride + (2 * lane + k) * D::kSize;
            e[k] = Pair{0.f, 0.f};
            if (2 * lane + k < 1 << log) e[k] = entry(load<BF16>(at, 0), q ? load<BF16>(at + D::kBytes, 0) : 0.f, q != nullptr);
            add(two, e[k]);
        }
        const int l = find(two, before, border, lane);
        Pair first = before;
        add(first, e[0]);
        const bool second = !(e[0].s > 0.f) || (e[1].s > 0.f && !(value(first) > border));
        return (int)(v0 + (line << log) + 2 * l + __shfl_sync(0xffffffffu, (int)second, l));
    }
}

template <int kThreads, bool BF16>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) verify_kernel(const VerifyArgs a, int cluster) {
    constexpr int kWarps = kThreads / 32;
    extern __shared__ uint4 ring[];  // [kAhead][2][kThreads]
    __shared__ int accepted_sh, again_sh;
    __shared__ Pair warp_sum[kWarps];
    __shared__ Pair cta_sum[2];  // of the row's weights, and of p alone
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
                yes = (double)a.accept_rand[b * a.drafts + lane] * (double)(signbit(q) ? 0.f : q) < (double)p && p < kMost;
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
                if (a.kept_lens) a.kept_lens[b] = max(0, max(0, a.seq_lens[b]) - (a.drafts - r));
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
    const long long part = ((a.vocab + parts - 1) / parts + kPart - 1) / kPart * kPart;
    const long long v0 = min((long long)a.vocab, (rank * kWarps + warp) * part), v1 = min((long long)a.vocab, v0 + part);
    int owner = -1;      // warp 0: the CTA of the cluster that holds the token
    Pair before{0.f, 0.f};  // the sum before its part
    double border = 0.;  // u times the whole sum
    for (int mode = 0; mode < 2; ++mode) {
        if (mode == 1) {  // nothing is left of the row: the target's probabilities alone
            q = nullptr;
            out = -1;
        }
        Pair s = lane_sum<kThreads, BF16>(p, q, v0, v1, out, lane, ring + tid);
        s = scan(s, lane);
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        if (warp == 0) {
            s = scan(lane < kWarps ? warp_sum[lane] : Pair{0.f, 0.f}, lane);
            if (lane == 31) cta_sum[mode] = s;
        }
        if (cluster > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        if (warp == 0) {
            Pair c{0.f, 0.f};
            if (lane < cluster) {
                const uint32_t at = cluster_addr(&cta_sum[mode], lane);
                c = Pair{__uint_as_float(cluster_load_u32(at)), __uint_as_float(cluster_load_u32(at + 4))};
            }
            const Pair all = scan(c, lane);
            const double total = (double)__shfl_sync(0xffffffffu, all.s, 31) + (double)__shfl_sync(0xffffffffu, all.e, 31);
            border = (double)a.sample_rand[b] * total;
            owner = find(c, before, border, lane);
            if (lane == 0) again_sh = owner < 0;
        }
        __syncthreads();
        if (!again_sh) break;
    }
    if (cluster > 1) cluster_arrive();
    if (warp == 0) {
        int32_t* token = a.tokens + b * (a.drafts + 1) + r;
        if (owner < 0) {
            if (rank == 0 && lane == 0) *token = -1;
        } else if (owner == rank) {
            const int w = find(lane < kWarps ? warp_sum[lane] : Pair{0.f, 0.f}, before, border, lane);
            const long long w0 = min((long long)a.vocab, (rank * kWarps + w) * part), w1 = min((long long)a.vocab, w0 + part);
            // (the CTA is done with the ring)
            const int v = search<BF16>(reinterpret_cast<uint8_t*>(ring), p, q, w0, w1, out, before, border, lane);
            if (lane == 0) *token = v;
        }
    }
    if (cluster > 1) cluster_wait();  // the others read this CTA's sums
}

template <int kThreads, bool BF16>
cudaError_t launch(const VerifyArgs& a, int cluster, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    constexpr size_t kRing = sizeof(uint4) * kAhead * 2 * kThreads, kDesk = 2 * Desk<BF16>::kBytes;  // one in the other's place
    constexpr size_t kSmem = kRing > kDesk ? kRing : kDesk;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&verify_kernel<kThreads, BF16>), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e;
        }
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_pdl_cluster(verify_kernel<kThreads, BF16>, dim3((unsigned)((long long)a.batch * cluster)), dim3(kThreads), kSmem, cluster, s, a, cluster);
}

}  // namespace

template <int kThreads>
cudaError_t launch_of(const VerifyArgs& a, bool bf16, long long sms, cudaStream_t s) {
    int cluster = 1;
    while (cluster < kMaxCluster && a.batch * cluster < 1024 / kThreads * sms && a.vocab > 4096LL * cluster) cluster *= 2;
    return bf16 ? launch<kThreads, true>(a, cluster, s) : launch<kThreads, false>(a, cluster, s);
}

// CTAs per request: more of them until the SMs have as many as they take, 1024 threads each. Of
// 512 threads while a request's eight leave an SM two or fewer, of 256 up to four, of 128 from there on.
// us for 131072 entries with the draft's, 512 / 256 / 128 threads: 1 request 11.1 / 12.6 / 12.1, 40
// in float32 - / 14.9 / 16.9, 100 in bf16 - / 21.8 / 19.5, 256 72.7 / 53.7 / 53.4, 512 in bf16 - / 62.1 / 59.1;
// 128 requests of 100003 entries 39.8 / 28.8 / 26.6. Half as many CTAs of 128 threads: 256 requests 57.
cudaError_t launch_verify(const VerifyArgs& a, bool bf16, cudaStream_t s) {
    const long long sms = tile_default_ctas(), most = (long long)a.batch * kMaxCluster;
    if (most <= 2 * sms) return launch_of<512>(a, bf16, sms, s);
    if (most <= 4 * sms) return launch_of<256>(a, bf16, sms, s);
    return launch_of<128>(a, bf16, sms, s);
}

}  // namespace hpc
