// Attention weight that cached tokens receive from a call's query rows (hpc_attn_weights):
//   w[b][h][t] = (t < L - n ? decay w[b][h][t] : 0)
//              + sum over counted rows i that see t, and the 8 query heads g of KV head h, of
//                exp(q[i][8 h + g] . k[t][h] / sqrt(128) - lse[i][8 h + g]).
//
// The scores are S = K . Q^T on tcgen05 tensor cores with the cache's tokens as the 128 rows
// (M) of the accumulator and the query rows of a KV head, 8 heads each, as its columns (N):
// a token is then a TMEM lane, one thread holds all its scores, and the sum over rows and
// heads is a chain of additions in that thread, without a shuffle or an atomic. K goes from
// the page into shared memory by TMA and into the product as it is, e4m3 codes too (the
// query is split into two e4m3 numbers, whose products add up in the accumulator; the key's
// scale multiplies the score). One CTA per SM, 12 warps
// (three per sub-partition, so that a thread can have 168 registers):
//   * warp 0, producer: tiles of 128 tokens (two pages) into a ring of stages;
//   * warp 1, issuer: the MMAs of each tile with every query slot, 16 rows (128 columns) a slot;
//   * warps 2 and 3, stagers: query rows into the slots (4, so that a pass takes up to
//     64 rows), bf16 as they are or split, with each row's constants;
//   * warps 4-7 and 8-11, two groups that take the even and the odd tiles: exp2 and sums.
// More than 64 rows are several passes over the CTA's tiles, the last rows (which see most)
// first; a token's thread is the same in each, so it adds to what it wrote itself.
//
// All tiles, walked KV head by KV head and sequence by sequence, are cut into runs of equal
// cost, one per CTA; each CTA finds its run from the lengths (there is no map and no
// workspace). A tile costs the rows that see it, at least kTileCost: below that many rows the
// key's bytes bound it, above the exponentials.
// Every wait is bounded (2 s); on expiry the CTA reports HPC_DEVERR_WAIT_TIMEOUT, gives
// copies and MMAs in flight time to end, frees its TMEM and returns.
#include <atomic>
#include <cstring>

#include "attn_common.cuh"
#include "loop.cuh"
#include "tcgen05.cuh"
#include "tile.cuh"

namespace hpc {
namespace {

using namespace attn;

constexpr int kTile = 128;                    // tokens of a tile: two pages
constexpr int kSlotRows = 16;                 // query rows of a slot
constexpr int kCols = kSlotRows * kGroup;     // accumulator columns of a slot
constexpr int kSlots = 4;
constexpr int kPassRows = kSlots * kSlotRows;
constexpr int kSlotBytes = 32768;             // bf16 [2 dim halves][128][128 B], or e4m3 [hi, lo][128][128 B]
constexpr int kThreads = 384;
constexpr int kStagers = 64;
constexpr uint32_t kTmemCols = 512;           // two accumulators of 128 columns per group
constexpr int kTileCost = 24;                 // query rows
constexpr int kSeqCost = 8;                   // a sequence's start in a CTA, in rows
constexpr int kMostRows = 65536;              // rows counted in a tile's cost at most (sums stay in 64 bits)
constexpr float kLog2e = 1.4426950408889634f;

template <bool FP8>
struct Layout {
    static constexpr int kStages = FP8 ? 5 : 3;
    static constexpr int kStageBytes = FP8 ? 16384 : 32768;
    static constexpr size_t kQ = (size_t)kStages * kStageBytes;
    static constexpr size_t kNl = kQ + kSlots * kSlotBytes;                   // float [slot][128]: -lse log2(e)
    static constexpr size_t kQc = kNl + kSlots * kCols * 4;                   // e4m3: float [slot][128]: score factors
    static constexpr size_t kScan = kQc + (FP8 ? kSlots * kCols * 4 : 0);     // int64 [warps]
    static constexpr size_t kRun = kScan + kThreads / 32 * 8;                 // int [8]
    static constexpr size_t kBars = kRun + 32;
    static constexpr int kNumBars = 2 * kStages + 2 * kSlots + 8;
    static constexpr size_t kTmemSlot = kBars + kNumBars * 8;
    static constexpr size_t kFlag = kTmemSlot + 4;
    static constexpr size_t kTotal = kFlag + 4;
    static_assert(kTotal <= 232448, "over the 227 KB shared-memory limit of a CTA");
};

struct WeightParams {
    const __nv_bfloat16* q;
    const int32_t* page_table;
    long long pt_stride;
    const int32_t* q_starts;
    const int32_t* seq_lens;
    const int32_t* counts;
    const float* k_scale;
    const float* lse;
    float* weights;
    long long w_stride;
    int* err;
    int rows_per_seq, window, batch, num_tokens, num_q_heads, num_kv_heads, num_pages;
    int max_len;
    float decay;
};

// A sequence: rows [lo, hi) of its n count, of which row i sees the tokens up to p0 + i.
struct Seq {
    int q0, lo, hi, L, p0, tiles;
};

template <bool REPORT>
__device__ __forceinline__ Seq seq_of(const WeightParams& p, int b) {
    Seq s{0, 0, 0, 0, 0, 0};
    int n = p.rows_per_seq;
    if (p.q_starts) {
        s.q0 = p.q_starts[b];
        const int end = p.q_starts[b + 1];
        if (s.q0 < 0 || end < s.q0 || end > p.num_tokens) {
            if (REPORT && p.err) atomicOr(p.err, (int)HPC_DEVERR_BAD_DESCRIPTOR);
            return s;
        }
        n = end - s.q0;
    } else {
        s.q0 = b * n;
    }
    const int len = p.seq_lens[b];
    if (REPORT && p.err && n > 0) {
        if (len < 0) atomicOr(p.err, (int)HPC_DEVERR_NEGATIVE_LENGTH);
        if (len > p.max_len) atomicOr(p.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
    }
    s.L = max(0, min(len, p.max_len));
    if (n == 0) s.L = 0;
    s.hi = p.counts ? max(0, min(n, p.counts[b])) : n;
    s.lo = p.window > 0 ? max(0, s.hi - p.window) : 0;
    s.p0 = s.L - n;
    s.tiles = (int)(((long long)s.L + kTile - 1) / kTile);
    return s;
}

// Cost of a sequence's tiles [0, j): tile i costs min(rows, a - 128 i), a the tokens that the
// last counted row sees, and kTileCost at least.
__device__ __forceinline__ long long units_before(const Seq& s, int j) {
    if (j == 0) return 0;
    const long long rows = min(s.hi - s.lo, kMostRows), a = (long long)s.hi + s.p0;
    long long u = kSeqCost;
    if (rows <= kTileCost) return u + (long long)kTileCost * j;
    const long long j1 = a >= rows ? (a - rows) / kTile + 1 : 0, j2 = a >= kTileCost ? (a - kTileCost) / kTile + 1 : 0;
    const long long m1 = min((long long)j, j1), m2 = min((long long)j, j2);
    return u + rows * m1 + (m2 - m1) * a - 64 * (m1 + m2 - 1) * (m2 - m1) + kTileCost * (j - m2);
}

// The first tile with at least u units before it.
__device__ __forceinline__ int tile_at(const Seq& s, long long u) {
    int lo = 0, hi = s.tiles;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (units_before(s, mid) >= u)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// One pass of a CTA over its tiles of a sequence and KV head: rows [lo, hi) of it, tiles
// [j0, j1), of which the rows see those before jl.
struct Pass {
    int h, b, q0, lo, hi, p0, L;
    int j0, jl, j1;
    int first;  // the pass that takes over or clears what was there
    __device__ __forceinline__ int slots() const { return (hi - lo + kSlotRows - 1) / kSlotRows; }
};

struct PassWalk {
    int h, b, j;      // next sequence and its first tile
    int h1, b1, j1;   // the run's end
    Seq s;            // current sequence, its place and its tiles [ja, jb)
    int hs, bs, ja, jb;
    int top;          // its rows [lo, top) are still to be passed over

    __device__ __forceinline__ void start(const int* run) {
        h = run[0];
        b = run[1];
        j = run[2];
        h1 = run[3];
        b1 = run[4];
        j1 = run[5];
        s = Seq{0, 0, 0, 0, 0, 0};
        hs = bs = ja = jb = top = 0;
    }

    // Tiles before the limit of what row top - 1 sees, within [ja, jb].
    __device__ __forceinline__ int seen() const {
        const long long a = (long long)top + s.p0;
        return top <= s.lo || a <= 0 ? ja : (int)max((long long)ja, min((long long)jb, (a + kTile - 1) / kTile));
    }

    __device__ __forceinline__ bool next(const WeightParams& p, Pass& x) {
        int jl = seen();
        x.first = jl == ja;  // nothing is left of the current sequence
        if (x.first) {
            do {
                if (h > h1 || (h == h1 && (b > b1 || (b == b1 && j >= j1)))) return false;
                s = seq_of<false>(p, b);
                hs = h;
                bs = b;
                ja = j;
                jb = h == h1 && b == b1 ? j1 : s.tiles;
                j = 0;
                if (++b >= p.batch) {
                    b = 0;
                    ++h;
                }
            } while (jb <= ja);
            top = s.hi;
            jl = seen();
        }
        x.h = hs;
        x.b = bs;
        x.q0 = s.q0;
        x.p0 = s.p0;
        x.L = s.L;
        x.hi = top;
        top = x.lo = max(s.lo, top - kPassRows);
        x.j0 = ja;
        x.jl = jl;
        x.j1 = x.first ? jb : jl;
        return true;
    }
};

// Every lane's wait has to succeed: a warp goes on, or gives up, as one.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    const bool ok = wait_bounded(bar, parity, abort_flag, kWaitLimitNs);
    return __all_sync(0xffffffffu, ok);
}

// 32 lanes from the warp's base lane x N consecutive columns: register k of thread t is
// lane t, column k.
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// Pairs of floats in one 64-bit register: two additions or products for one issue slot.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t exp2_2(uint64_t x) {
    const float2 v = unpair(x);
    return pair(fast_exp2(v.x), fast_exp2(v.y));
}

// The weights of one query row's 8 heads for the thread's token, as two sums of four. s: the
// scores; nl, qc: the row's constants in shared memory; factor: twice the token's.
template <bool FP8>
__device__ __forceinline__ uint64_t row_weight(const uint32_t* s, const float* nl, const float* qc, uint64_t factor) {
    uint64_t e[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(nl + 4 * k);
        const uint64_t x = pair(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1]));
        const uint64_t y = pair(__uint_as_float(s[4 * k + 2]), __uint_as_float(s[4 * k + 3]));
        if constexpr (FP8) {
            const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(qc + 4 * k);
            e[2 * k] = exp2_2(fma2(mul2(x, factor), c.x, l.x));
            e[2 * k + 1] = exp2_2(fma2(mul2(y, factor), c.y, l.y));
        } else {
            e[2 * k] = exp2_2(fma2(x, factor, l.x));
            e[2 * k + 1] = exp2_2(fma2(y, factor, l.y));
        }
    }
    return add2(add2(e[0], e[1]), add2(e[2], e[3]));
}

// Rows [r, r + 4) of a slot, those there are: added where they see the token (MASK; else
// all of them do).
template <bool FP8, bool MASK>
__device__ __forceinline__ void four_rows(const uint32_t (&s)[32], int r, int rows, int sees, const float* nl, const float* qc,
                                          uint64_t factor, uint64_t& sum) {
    nl += r * kGroup;
    qc += r * kGroup;
    if (r + 4 <= rows) {
        uint64_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = row_weight<FP8>(s + 8 * k, nl + k * kGroup, qc + k * kGroup, factor);
            if (MASK && r + k < sees) w[k] = 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) sum = add2(sum, w[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (r + k < rows) {
                const uint64_t w = row_weight<FP8>(s + 8 * k, nl + k * kGroup, qc + k * kGroup, factor);
                if (!MASK || r + k >= sees) sum = add2(sum, w);
            }
        }
    }
}

// All rows of a slot.
template <bool FP8, bool MASK>
__device__ __forceinline__ void slot_rows(uint32_t ta, int rows, int sees, const float* nl, const float* qc, uint64_t factor,
                                          uint64_t& sum) {
#pragma unroll 1
    for (int r = 0; r < rows; r += 4) {
        uint32_t v[32];
        tmem_ld_x32(ta + r * kGroup, v);
        tmem_ld_wait();
        four_rows<FP8, MASK>(v, r, rows, sees, nl, qc, factor, sum);
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    attn_weights_kernel(const __grid_constant__ CUtensorMap tm_k, const WeightParams p) {
    using LY = Layout<FP8>;
    constexpr int NS = LY::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + LY::kBars);
    uint64_t* empty = full + NS;
    uint64_t* qfull = empty + NS;
    uint64_t* qfree = qfull + kSlots;
    uint64_t* accfull = qfree + kSlots;  // accumulator 2 g + (turn of group g) % 2
    uint64_t* accfree = accfull + 4;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + LY::kTmemSlot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + LY::kFlag);
    int* run = reinterpret_cast<int*>(smem + LY::kRun);
    float* nl = reinterpret_cast<float*>(smem + LY::kNl);
    float* qc = reinterpret_cast<float*>(smem + LY::kQc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&qfull[i], kStagers);
            mbar_init(&qfree[i], 1 + 8);  // the MMAs; both groups' warps
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accfree[i], 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(const_cast<uint32_t*>(tmem_slot))),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- this CTA's run: each thread sums a range of sequences, then the two borders are
    // looked up by the threads whose ranges hold them
    {
        long long* scan = reinterpret_cast<long long*>(smem + LY::kScan);
        const int per = (p.batch + kThreads - 1) / kThreads;
        const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
        long long sum = 0;
        for (int b = b0; b < b1; ++b) {
            const Seq s = blockIdx.x == 0 ? seq_of<true>(p, b) : seq_of<false>(p, b);
            sum += units_before(s, s.tiles);
        }
        long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        long long before = incl - sum, per_head = 0;
        for (int k = 0; k < kThreads / 32; ++k) {
            if (k < warp) before += scan[k];
            per_head += scan[k];
        }
        const long long total = per_head * p.num_kv_heads;
        const long long bucket = max((total + gridDim.x - 1) / gridDim.x, (long long)kTileCost);
#pragma unroll 1
        for (int end = 0; end < 2; ++end) {
            const long long u = min(total, (long long)(blockIdx.x + end) * bucket);
            int* at = run + 3 * end;
            if (u >= total) {
                if (tid == 0) {
                    at[0] = p.num_kv_heads;
                    at[1] = 0;
                    at[2] = 0;
                }
                continue;
            }
            const int h = (int)(u / per_head);
            const long long rem = u - h * per_head;
            if (rem >= before && rem < before + sum) {
                long long c = before;
                for (int b = b0; b < b1; ++b) {
                    const Seq s = seq_of<false>(p, b);
                    const long long all = units_before(s, s.tiles);
                    if (rem < c + all) {
                        at[0] = h;
                        at[1] = b;
                        at[2] = tile_at(s, rem - c);
                        break;
                    }
                    c += all;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    PassWalk walk;
    walk.start(run);
    Pass x;
    bool ok = true;

    if (warp == 0) {
        // ============================ producer: the tiles that counted rows see
        const uint64_t pol = l2_evict_first_policy();
        uint32_t seq = 0;
        auto pages = [&](const Pass& y, int j) {  // the lanes' page ids of tiles j, j + 1, ...
            const int c = 2 * j + lane;
            return c < 2 * y.jl && (long long)c * kChunk < y.L ? p.page_table[y.b * p.pt_stride + c] : -1;
        };
        bool have = walk.next(p, x);
        int pg = have ? pages(x, x.j0) : -1;
        while (have && ok) {
            Pass y;  // the pass after, whose first pages are on their way meanwhile
            const bool have2 = walk.next(p, y);
            const int pg2 = have2 ? pages(y, y.j0) : -1;
            for (int j = x.j0; j < x.jl && ok; j += 16) {
                if (j != x.j0) pg = pages(x, j);
                const int nt = min(16, x.jl - j);
                for (int k = 0; k < nt; ++k, ++seq) {
                    int page[2], there = 0;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        page[u] = __shfl_sync(0xffffffffu, pg, 2 * k + u);
                        if ((unsigned)page[u] < (unsigned)p.num_pages)
                            there |= 1 << u;
                        else if (lane == 0 && p.err && (long long)(2 * (j + k) + u) * kChunk < x.L)
                            atomicOr(p.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
                    }
                    const uint32_t st = seq % NS;
                    if (lane == 0) {
                        ok = wait_bounded(&empty[st], ((seq / NS) & 1) ^ 1, abort_flag, kWaitLimitNs);
                        if (ok) {
                            if (there == 0) {
                                mbar_arrive(&full[st]);
                            } else {
                                constexpr uint32_t kPageBytes = FP8 ? 8192 : 16384;
                                mbar_arrive_expect_tx(&full[st], (there == 3 ? 2 : 1) * kPageBytes);
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    if (!(there >> u & 1)) continue;
                                    uint8_t* dst = smem + st * LY::kStageBytes + u * 8192;
                                    tma_load_3d(dst, &tm_k, &full[st], 0, x.h, page[u] * kChunk, pol);
                                    if constexpr (!FP8)
                                        tma_load_3d(dst + 16384, &tm_k, &full[st], 64, x.h, page[u] * kChunk, pol);
                                }
                            }
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                }
            }
            x = y;
            pg = pg2;
            have = have2;
        }
        // copies in flight land before the CTA can end
        if (lane == 0)
            for (uint32_t k = seq > (uint32_t)NS ? seq - NS : 0u; k < seq; ++k)
                wait_bounded(&full[k % NS], (k / NS) & 1, nullptr, kDrainLimitNs);
    } else if (warp == 1) {
        // ============================ MMA issuer (one lane; the warp goes along)
        const uint32_t el = elect_lane();
        constexpr uint32_t kId = FP8 ? idesc_e4m3(kTile, 0) : idesc_16bit(false, kTile, 0, 0);
        // descriptors of the first stage and slot; the others lie at fixed distances (in
        // 16-byte units, the low bits of a descriptor)
        const uint64_t dk = sdesc_sw128(smem_u32(smem), 16, 1024), dq = sdesc_sw128(smem_u32(smem + LY::kQ), 16, 1024);
        uint32_t seq = 0, qseq = 0, turn0 = 0, turn1 = 0;
        while (ok && walk.next(p, x)) {
            const int ns = x.slots();
            for (int j = x.j0; j < x.jl && ok; ++j, ++seq) {
                const uint32_t st = seq % NS, g = j & 1;
                ok = warp_wait(&full[st], (seq / NS) & 1, abort_flag);
                const uint64_t k = dk + st * (LY::kStageBytes >> 4);
                for (int s = 0; s < ns && ok; ++s) {
                    const uint32_t sl = (qseq + s) % kSlots;
                    if (j == x.j0) ok = warp_wait(&qfull[sl], ((qseq + s) / kSlots) & 1, abort_flag);
                    const uint32_t c = g ? turn1++ : turn0++;
                    const uint32_t acc = 2 * g + (c & 1);
                    if (ok) ok = warp_wait(&accfree[acc], ((c >> 1) & 1) ^ 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const int rows = min(kSlotRows, x.hi - x.lo - s * kSlotRows);
                    const uint32_t id = kId | (uint32_t)((rows + 1) / 2) << 18;  // columns: a multiple of 16
                    const uint64_t q = dq + sl * (kSlotBytes >> 4);
                    const uint32_t d = tmem + acc * kCols;
                    if constexpr (FP8) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            umma_e4m3_el(el, d, k + kk * 2, q + kk * 2, id, kk > 0);
                            umma_e4m3_el(el, d, k + kk * 2, q + 1024 + kk * 2, id, 1);
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint32_t off = (kk >> 2) * 1024 + (kk & 3) * 2;
                            umma_f16_el(el, d, k + off, q + off, id, kk > 0);
                        }
                    }
                    umma_commit_el(el, &accfull[acc]);
                    if (j + 1 == x.jl) umma_commit_el(el, &qfree[sl]);
                }
                if (ok) umma_commit_el(el, &empty[st]);
            }
            if (x.jl > x.j0) qseq += ns;
        }
    } else if (warp >= 4) {
        // ============================ groups g = 0, 1: tiles j with j % 2 == g; thread = token
        const int g = (warp >> 2) - 1, wq = warp & 3;
        constexpr float kScale = kLog2e * 0.08838834764831845f;  // log2(e) / sqrt(128)
        // What a tile needs from memory comes a tile ahead, its page id two tiles: across
        // passes too, unless a pass goes on from the sums of the one before.
        struct Token {
            float old, factor;
            bool there;
        };
        auto first_tile = [&](const Pass& y) { return y.j0 + ((y.j0 & 1) ^ g); };
        auto page_of = [&](const Pass& y, int j) {
            const int c = 2 * j + (wq >> 1);
            return j < y.j1 && (long long)c * kChunk < y.L ? p.page_table[y.b * p.pt_stride + c] : -1;
        };
        auto fetch = [&](const Pass& y, int j, int page) {
            Token k{0.f, kScale, (unsigned)page < (unsigned)p.num_pages};
            const int t = j * kTile + 32 * wq + lane;
            if (j < y.j1 && t < (y.first ? y.p0 : y.L) && !(y.first && p.decay == 0.f))
                k.old = p.weights[((long long)y.b * p.num_kv_heads + y.h) * p.w_stride + t];
            if (FP8 && k.there) k.factor = p.k_scale[((long long)page * p.num_kv_heads + y.h) * kChunk + (t & (kChunk - 1))];
            return k;
        };
        uint32_t qseq = 0, turn = 0;
        bool have = walk.next(p, x);
        Token ahead{0.f, 0.f, false};
        int page = -1;  // of the tile after the one ahead
        if (have) {
            ahead = fetch(x, first_tile(x), page_of(x, first_tile(x)));
            page = page_of(x, first_tile(x) + 2);
        }
        while (have && ok) {
            Pass y;
            have = walk.next(p, y);
            const int jy = have ? first_tile(y) : 0;
            const int page_y = have ? page_of(y, jy) : -1;
            const int ns = x.slots();
            float* wrow = p.weights + ((long long)x.b * p.num_kv_heads + x.h) * p.w_stride;
            bool any = false;      // this group has seen the pass's slots
            bool fetched = false;  // ahead is of the next pass
            for (int j = first_tile(x); j < x.j1; j += 2) {
                const int t = j * kTile + 32 * wq + lane;
                const Token now = ahead;
                if (j + 2 < x.j1) {
                    ahead = fetch(x, j + 2, page);
                    page = page_of(x, j + 4);
                } else if (have && y.first) {
                    ahead = fetch(y, jy, page_y);
                    page = page_of(y, jy + 2);
                    fetched = true;
                }
                float sum = 0.f;
                if (j < x.jl) {
                    uint64_t sum2 = 0;
                    const uint64_t factor = pair(now.factor, now.factor);
                    for (int s = 0; s < ns; ++s) {
                        const uint32_t sl = (qseq + s) % kSlots;
                        if (!any) ok = warp_wait(&qfull[sl], ((qseq + s) / kSlots) & 1, abort_flag);
                        const uint32_t acc = 2 * g + (turn & 1);
                        if (ok) ok = warp_wait(&accfull[acc], (turn >> 1) & 1, abort_flag);
                        if (!ok) break;
                        ++turn;
                        tc_fence_after();
                        const int r0 = x.lo + s * kSlotRows, rows = min(kSlotRows, x.hi - r0);
                        const uint32_t ta = tmem + ((uint32_t)(32 * wq) << 16) + acc * kCols;
                        const float* nls = nl + sl * kCols;
                        const float* qcs = qc + sl * kCols;
                        // rows of the slot from t - p0 - r0 on see token t: all of them before the last tiles
                        if (j * kTile + kTile - 1 <= (long long)x.p0 + r0)
                            slot_rows<FP8, false>(ta, rows, 0, nls, qcs, factor, sum2);
                        else
                            slot_rows<FP8, true>(ta, rows, t - x.p0 - r0, nls, qcs, factor, sum2);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&accfree[acc]);
                    }
                    if (!ok) break;
                    any = true;
                    const float2 v = unpair(sum2);
                    if (now.there) sum = v.x + v.y;
                }
                if (t < x.L) wrow[t] = (x.first ? p.decay * now.old : now.old) + sum;
            }
            if (x.jl > x.j0) {
                // the slots are this pass's until both groups have seen them
                for (int s = 0; s < ns && ok; ++s) {
                    const uint32_t sl = (qseq + s) % kSlots;
                    if (!any) ok = warp_wait(&qfull[sl], ((qseq + s) / kSlots) & 1, abort_flag);
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(&qfree[sl]);
                }
                qseq += ns;
            }
            if (have && !fetched) {
                ahead = fetch(y, jy, page_y);
                page = page_of(y, jy + 2);
            }
            x = y;
        }
    } else {
        // ============================ stagers: query rows into slots
        const int sid = (warp - 2) * 32 + lane;
        uint32_t qseq = 0;
        while (ok && walk.next(p, x)) {
            if (x.jl <= x.j0) continue;
            const int ns = x.slots();
            for (int s = 0; s < ns && ok; ++s, ++qseq) {
                const uint32_t sl = qseq % kSlots;
                ok = warp_wait(&qfree[sl], ((qseq / kSlots) & 1) ^ 1, abort_flag);
                if (!ok) break;
                const int r0 = x.lo + s * kSlotRows, rows = min(kSlotRows, x.hi - r0);
                uint8_t* slot = smem + LY::kQ + sl * kSlotBytes;
                const long long row0 = ((long long)x.q0 + r0) * p.num_q_heads + x.h * kGroup;
                for (int c = sid; c < rows * kGroup; c += kStagers) {
                    const float l = p.lse[row0 + (long long)(c / kGroup) * p.num_q_heads + c % kGroup];
                    nl[sl * kCols + c] = l == -INFINITY ? -INFINITY : -l * kLog2e;  // a row of -inf: no weight
                }
                if constexpr (!FP8) {
                    // a head's 16 pieces of 16 bytes by 16 threads, eight rows at once
                    const int c = sid & 15;
                    const long long step = (long long)p.num_q_heads * kHeadDim;
                    for (int i = 0; i < 2 * rows; i += 8) {  // i: 2 row + half of the heads
                        uint4 v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int head = (sid >> 4) + 4 * (k & 1), r = (i + k) >> 1;
                            if (i + k < 2 * rows) v[k] = *reinterpret_cast<const uint4*>(p.q + row0 * kHeadDim + r * step + head * kHeadDim + c * 8);
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int head = (sid >> 4) + 4 * (k & 1), r = (i + k) >> 1;
                            if (i + k < 2 * rows)
                                *reinterpret_cast<uint4*>(slot + (c >> 3) * 16384 + (r * kGroup + head) * 128 + (((c & 7) ^ head) << 4)) = v[k];
                        }
                    }
                } else {
                    // two threads per row of 128: half hh of its dims each, split into hi and lo codes
                    for (int c0 = 0; c0 < rows * kGroup; c0 += kStagers / 2) {
                        const int c = c0 + (sid >> 1), hh = sid & 1;
                        const bool in = c < rows * kGroup;
                        const __nv_bfloat16* src =
                            p.q + (row0 + (long long)(c / kGroup) * p.num_q_heads + c % kGroup) * kHeadDim + hh * 64;
                        uint4 raw[8];
                        float amax = 0.f;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            raw[k] = in ? reinterpret_cast<const uint4*>(src)[k] : make_uint4(0, 0, 0, 0);
                            const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[m] << 16)), fabsf(__uint_as_float(w[m] & 0xffff0000u))));
                        }
                        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                        // the smallest power of two 2^ex with amax / 2^ex <= 448: q / 2^ex is exact
                        float up = 1.f, down = 1.f;
                        if (amax > 0.f && amax <= 3.0e38f) {
                            int e;
                            const float m = frexpf(amax * (1.f / 448.f), &e);
                            const int ex = m == 0.5f ? e - 1 : e;
                            up = ldexpf(1.f, ex);
                            down = ldexpf(1.f, -ex);
                        }
                        if (in && hh == 0) qc[sl * kCols + c] = up * (kLog2e * 0.08838834764831845f);
#pragma unroll
                        for (int c2 = 0; c2 < 4; ++c2) {
                            uint2 hp[2], lp[2];
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const uint4 x4 = raw[2 * c2 + u];
                                const uint32_t w[4] = {x4.x, x4.y, x4.z, x4.w};
                                float y[8];
#pragma unroll
                                for (int m = 0; m < 4; ++m) {
                                    y[2 * m] = __uint_as_float(w[m] << 16) * down;
                                    y[2 * m + 1] = __uint_as_float(w[m] & 0xffff0000u) * down;
                                }
                                split_e4m3x8(y, hp[u], lp[u]);
                            }
                            if (in) {
                                const int off = c * 128 + (((4 * hh + c2) ^ (c & 7)) << 4);
                                *reinterpret_cast<uint4*>(slot + off) = make_uint4(hp[0].x, hp[0].y, hp[1].x, hp[1].y);
                                *reinterpret_cast<uint4*>(slot + 16384 + off) = make_uint4(lp[0].x, lp[0].y, lp[1].x, lp[1].y);
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&qfull[sl]);
            }
        }
    }
    if (!ok && lane == 0) {
        *abort_flag = 1;
        if (p.err) atomicOr(p.err, (int)HPC_DEVERR_WAIT_TIMEOUT);
    }
    // all roles done: in the normal path every MMA has completed before the groups' last
    // waits; after a timeout work in flight gets a bounded drain
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        if (*abort_flag) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < kDrainLimitNs) {
            }
        }
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <bool FP8>
cudaError_t launch(const CUtensorMap& tm_k, const WeightParams& p, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&attn_weights_kernel<FP8>),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<FP8>::kTotal);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e;
        }
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    const int ctas = tile_default_ctas();
    if (ctas < 1) return cudaErrorUnknown;
    return launch_pdl(attn_weights_kernel<FP8>, dim3(ctas), dim3(kThreads), Layout<FP8>::kTotal, s, tm_k, p);
}

}  // namespace

cudaError_t launch_attn_weights(const AttnWeightsArgs& a, cudaStream_t s) {
    CUtensorMap tm_k;
    memset(&tm_k, 0, sizeof tm_k);
    if (!make_kv_map(&tm_k, a.k_cache, a.fp8, a.num_pages, a.num_kv_heads)) return cudaErrorInvalidValue;
    WeightParams p;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.page_table = a.page_table;
    p.pt_stride = a.pt_stride;
    p.q_starts = a.q_starts;
    p.seq_lens = a.seq_lens;
    p.counts = a.counts;
    p.k_scale = a.k_scale;
    p.lse = a.lse;
    p.weights = a.weights;
    p.w_stride = a.w_stride;
    p.err = a.err;
    p.rows_per_seq = a.rows_per_seq;
    p.window = a.window;
    p.batch = a.batch;
    p.num_tokens = a.num_tokens;
    p.num_q_heads = a.num_q_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.num_pages = a.num_pages;
    const long long most = a.pt_stride * kChunk;
    p.max_len = most > kMaxKeys ? kMaxKeys : (int)most;
    p.decay = a.decay;
    return a.fp8 ? launch<true>(tm_k, p, s) : launch<false>(tm_k, p, s);
}

}  // namespace hpc
