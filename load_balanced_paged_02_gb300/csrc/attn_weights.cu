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
// scale multiplies the score). One CTA per SM, 20 warps (five per sub-partition, so that a
// thread can have 96 registers):
//   * warp 0, producer: the passes (below) to the other warps, and tiles of 128 tokens (two
//     pages) into a ring of stages;
//   * warps 1 and 2, issuers that take turns by tiles: MMAs with every query slot, 8
//     rows (64 columns) a slot. One issuer's waits and commits took 0.39 us a tile, more than
//     an e4m3 tile's bytes;
//   * warp 3, stager: query rows into the slots (a pass takes up to 32 rows, four of five
//     slots) by TMA, e4m3 splits, each row's constants;
//   * warps 4-19, four groups: exp2 and sums, a tile by one of them, or, where a sequence has
//     more than 8 rows, by two that share its slots. A group has two
//     accumulators, one filled while the other is read.
// More than 32 rows are several passes over the CTA's tiles, the last rows (which see most)
// first; a token's thread is the same in each, so it adds to what it wrote itself.
//
// All tiles, walked KV head by KV head and sequence by sequence, are cut into runs of equal
// cost, one per CTA; each CTA finds its run from the lengths (there is no map and no
// workspace). A tile costs the rows that see it, at least kTileCost: below that many rows the
// key's bytes bound it, above the exponentials (30 sequences of one row among 6 of 64: 168 us with
// 16, 212 with 8, 166 with 12, 197 with 24). A sequence's start costs kSeqCost (512 of up to 512
// tokens: 86 us with 4, 88 with none).
//
// What it measured, bf16 unless said, 8 KV heads, lengths log-uniform: 64 sequences of one row,
// up to 65536 tokens, 277 us, 6.6 TB/s: HBM. 48 of four rows over e4m3, 121 us, 6.0 TB/s:
// an issuer takes 880 clocks for a tile's waits, products and commits beside the summing warps, and the
// keys come once in 800 (as fast with 6 stages as with 11). 10 of 32 rows, up to 32768 tokens,
// 93 us, 3.8 TB/s and 940 TFLOP/s: issue slots 55 % busy, exp2 42 %, the tensor core 42 % (a product of 64
// columns takes 48 clocks for its operands' bytes, where its arithmetic takes 34). The products alone would
// take 85, the sums alone 87, neither 64. Two slots in one product of 128 columns: 91 us, but rows of 4
// or 16 then take 3 to 5 % more; an issuer per group: registers for 22 warps are too few; half a slot's scores on
// their way while the other half is summed: as before. The same windows over e4m3: 128 us. All 8192 rows of a
// prompt: 1.62 ms, over e4m3 4.76 ms, where a pass's slots are for 3 to 4 tiles of a CTA.
// Every wait is bounded (2 s); on expiry the CTA reports HPC_DEVERR_WAIT_TIMEOUT, gives
// copies and MMAs in flight time to end, frees its TMEM and returns.
#include <atomic>
#include <climits>
#include <cstring>

#include "attn_common.cuh"
#include "loop.cuh"
#include "tcgen05.cuh"
#include "tile.cuh"

namespace hpc {
namespace {

using namespace attn;

constexpr int kTile = 128;                    // tokens of a tile: two pages
constexpr int kSlotRows = 8;                  // query rows of a slot
constexpr int kCols = kSlotRows * kGroup;     // accumulator columns of a slot
constexpr int kSlots = 5;
constexpr int kPassRows = 32;                 // the fifth slot is filled for the pass after
constexpr int kSlotBytes = 16384;             // bf16 [2 dim halves][64][128 B], or e4m3 [hi, lo][64][128 B]
constexpr int kSlotHalf = kSlotBytes / 2;
constexpr int kThreads = 640;
constexpr int kGroups = 4;
constexpr uint32_t kTmemCols = 512;           // two accumulators of 64 columns per group
constexpr int kPasses = 4;                    // passes that the other warps may be behind the producer
constexpr int kPassInts = 12;
constexpr int kTileCost = 16;                 // query rows
constexpr int kSeqCost = 4;                   // a sequence's start in a CTA, in rows
constexpr int kMostRows = 65536;              // rows counted in a tile's cost at most (sums stay in 64 bits)
constexpr float kLog2e = 1.4426950408889634f;

template <bool FP8>
struct Layout {
    static constexpr int kStages = FP8 ? 8 : 4;
    static constexpr int kStageBytes = FP8 ? 16384 : 32768;
    static constexpr size_t kQ = (size_t)kStages * kStageBytes;
    static constexpr size_t kNl = kQ + kSlots * kSlotBytes;                   // float [slot][64]: -lse log2(e)
    static constexpr size_t kQc = kNl + kSlots * kCols * 4;                   // e4m3: float [2][slot][64]: score factors
    static constexpr size_t kScan = kQc + (FP8 ? 2 * kSlots * kCols * 4 : 0); // int64 [warps]
    static constexpr size_t kBorder = kScan + kThreads / 32 * 8;              // Border [4]
    static constexpr size_t kRun = kBorder + 64;                              // int [8]
    static constexpr size_t kPass = kRun + 32;                                // Pass [kPasses]
    static constexpr size_t kPart = kPass + kPasses * kPassInts * 4;          // float [2][2][128]: sums of upper groups
    static constexpr size_t kBars = kPart + 4 * kTile * 4;
    static constexpr int kNumBars = 3 * kStages + 3 * kSlots + 4 * kGroups + 2 * kPasses + 8;
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
    // (every load before the first is used)
    const int len = p.seq_lens[b], count = p.counts ? p.counts[b] : INT_MAX;
    const int begin = p.q_starts ? p.q_starts[b] : b * p.rows_per_seq, end = p.q_starts ? p.q_starts[b + 1] : begin + p.rows_per_seq;
    Seq s{0, 0, 0, 0, 0, 0};
    if (begin < 0 || end < begin || end > p.num_tokens) {
        if (REPORT && p.err) atomicOr(p.err, (int)HPC_DEVERR_BAD_DESCRIPTOR);
        return s;
    }
    const int n = end - begin;
    if (REPORT && p.err && n > 0) {
        if (len < 0) atomicOr(p.err, (int)HPC_DEVERR_NEGATIVE_LENGTH);
        if (len > p.max_len) atomicOr(p.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
    }
    s.q0 = begin;
    s.L = n > 0 ? max(0, min(len, p.max_len)) : 0;
    s.hi = max(0, min(n, count));
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

// The first tile with at least u units before it, by a warp: 32 places at a time.
__device__ __forceinline__ int tile_at(const Seq& s, long long u, int lane) {
    int lo = 0, hi = s.tiles;  // the answer is in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = min(hi, lo + lane * step);
        const uint32_t enough = __ballot_sync(0xffffffffu, units_before(s, at) >= u);
        if (enough == 0) {
            lo = min(hi, lo + 31 * step) + 1;  // behind the last place
            if (lo > hi) lo = hi;
        } else {
            const int k = __ffs(enough) - 1;
            hi = min(hi, lo + k * step);
            if (k > 0) lo = min(hi, lo + (k - 1) * step + 1);
            else lo = hi;
        }
    }
    return lo;
}

// Where a CTA's run begins or ends: rem units into the tiles of a KV head and sequence.
struct Border {
    long long rem;
    int h, b;
};

// One pass of a CTA over its tiles of a sequence and KV head: rows [lo, hi) of it, tiles
// [j0, j1), of which the rows see those before jl.
struct alignas(16) Pass {
    int h, b, q0, lo, hi, p0, L;  // h < 0: the run is over
    int j0, jl, j1;
    int first;  // the pass that takes over or clears what was there
    // Tile j is number n = j + shift: issuer n % 2 has it. Of a sequence of up to 8 rows group n %
    // 4 sums it (shift below 4); of one of more rows groups n % 2 and n % 2 + 2 do, the even
    // and the odd slots.
    int shift;
    __device__ __forceinline__ bool split() const { return shift >= kGroups; }
    __device__ __forceinline__ int slots() const { return (hi - lo + kSlotRows - 1) / kSlotRows; }
};

static_assert(sizeof(Pass) == kPassInts * 4, "pass ring");

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
        x.shift = ((hs + bs) & (kGroups - 1)) + (s.hi - s.lo > kSlotRows ? kGroups : 0);  // short sequences fall to all groups
        return true;
    }
};

__device__ __forceinline__ void tma_load_3d_nohint(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

// A warp goes on, or gives up, as one: its lanes test the barrier together, without a branch of their own.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((it & 15) == 0 && __any_sync(0xffffffffu, *abort_flag != 0 || global_timer_ns() - t0 > kWaitLimitNs)) return false;
    }
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
            e[2 * k] = fma2(mul2(x, factor), c.x, l.x);
            e[2 * k + 1] = fma2(mul2(y, factor), c.y, l.y);
        } else {
            e[2 * k] = fma2(x, factor, l.x);
            e[2 * k + 1] = fma2(y, factor, l.y);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = exp2_2(e[k]);
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
#pragma unroll
    for (int r = 0; r < kSlotRows; r += 4) {
        if (r >= rows) break;
        uint32_t v[32];
        tmem_ld_x32(ta + r * kGroup, v);
        tmem_ld_wait();
        four_rows<FP8, MASK>(v, r, rows, sees, nl, qc, factor, sum);
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    attn_weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q1,
                        const __grid_constant__ CUtensorMap tm_q4, const WeightParams p) {
    using LY = Layout<FP8>;
    constexpr int NS = LY::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    // one per issuer and stage, as an issuer sees the stages that its tiles are in alone
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + LY::kBars);
    uint64_t* empty = full + 2 * NS;
    uint64_t* qfull = empty + NS;
    uint64_t* qfree = qfull + kSlots;
    uint64_t* qraw = qfree + kSlots;          // e4m3: the copies of a slot's rows
    uint64_t* accfull = qraw + kSlots;        // accumulator 2 g + (turn of group g) % 2
    uint64_t* accfree = accfull + 2 * kGroups;
    uint64_t* passfull = accfree + 2 * kGroups;
    uint64_t* passfree = passfull + kPasses;
    uint64_t* partfull = passfree + kPasses;  // buffer 2 (issuer) + (meeting) % 2
    uint64_t* partfree = partfull + 4;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + LY::kTmemSlot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + LY::kFlag);
    Pass* passes = reinterpret_cast<Pass*>(smem + LY::kPass);
    int* run = reinterpret_cast<int*>(smem + LY::kRun);
    float* part = reinterpret_cast<float*>(smem + LY::kPart);
    float* nl = reinterpret_cast<float*>(smem + LY::kNl);
    float* qc = reinterpret_cast<float*>(smem + LY::kQc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid < LY::kNumBars) {  // arrivals that each barrier waits for, in the order above
        int i = tid;
        uint32_t n = 1;  // full, empty, qraw, accfull and passfull
        if ((i -= 3 * NS) >= 0 && i < kSlots) n = FP8 ? 1 : 2;                     // qfull: the split; or copies and constants
        if ((i -= kSlots) >= 0 && i < kSlots) n = 2 + 4 * kGroups;                 // qfree: both issuers' MMAs; the groups' warps
        if ((i -= 2 * kSlots + 2 * kGroups) >= 0 && i < 2 * kGroups) n = 4;        // accfree: a group's warps
        if ((i -= 2 * kGroups + kPasses) >= 0 && i < kPasses) n = 3 + 4 * kGroups; // passfree: issuers, stager, the groups' warps
        if ((i -= kPasses) >= 0) n = 4;                                            // partfull and partfree: a group's warps
        mbar_init(&full[tid], n);
        fence_mbar_init();
    }
    if (tid == 0) *abort_flag = 0;
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
        // which sequence each border falls into, by the thread that has summed it
        Border* border = reinterpret_cast<Border*>(smem + LY::kBorder);
        if (warp < 2) {  // the head of each border: how many end before it
            const long long u = (long long)(blockIdx.x + warp) * bucket;
            int h = 0;
            for (int i = lane; i < p.num_kv_heads; i += 32) h += (i + 1) * per_head <= u;
            h = u < total ? __reduce_add_sync(0xffffffffu, h) : p.num_kv_heads;
            if (lane == 0) border[warp] = Border{u < total ? u - h * per_head : 0, h, 0};
        }
        __syncthreads();
#pragma unroll
        for (int end = 0; end < 2; ++end) {
            const int h = border[end].h;
            long long rem = border[end].rem - before;
            if (h < p.num_kv_heads && rem >= 0 && rem < sum) {
                for (int b = b0; b < b1; ++b) {
                    const Seq s = seq_of<false>(p, b);
                    const long long all = units_before(s, s.tiles);
                    if (rem < all) {
                        border[2 + end] = Border{rem, h, b};
                        break;
                    }
                    rem -= all;
                }
            }
        }
        __syncthreads();
        // and which tile, by a warp for each
        if (warp < 2) {
            const Border x = border[warp].h < p.num_kv_heads ? border[2 + warp] : border[warp];
            int j = 0;
            if (x.rem > 0) j = tile_at(seq_of<false>(p, x.b), x.rem, lane);
            if (lane == 0) {
                run[3 * warp] = x.h;
                run[3 * warp + 1] = x.b;
                run[3 * warp + 2] = j;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;
    // Pass number k as the producer told it.
    auto pass_ready = [&](uint32_t k) { return warp_wait(&passfull[k % kPasses], (k / kPasses) & 1, abort_flag); };
    auto pass_done = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&passfree[k % kPasses]);
    };

    if (warp == 0) {
        // ============================ producer: passes, and the tiles that counted rows see
        const uint64_t pol = l2_evict_first_policy();
        PassWalk walk;
        walk.start(run);
        Pass x, y;
        uint32_t seq = 0, k = 0;
        uint32_t uses[2] = {0, 0};  // bit st: of barrier st of an issuer, odd or even
        auto publish = [&](uint32_t n, bool have, Pass& z) {
            if (!have) z.h = -1;
            if (n >= (uint32_t)kPasses && !warp_wait(&passfree[n % kPasses], ((n / kPasses) - 1) & 1, abort_flag)) return false;
            if (lane == 0) {
                passes[n % kPasses] = z;
                mbar_arrive(&passfull[n % kPasses]);
            }
            return true;
        };
        auto pages = [&](const Pass& z, int j) {  // the lanes' page ids of tiles j, j + 1, ...
            const int c = 2 * j + lane;
            return c < 2 * z.jl && (long long)c * kChunk < z.L ? p.page_table[z.b * p.pt_stride + c] : -1;
        };
        bool have = walk.next(p, x);
        ok = publish(0, have, x);
        int pg = have ? pages(x, x.j0) : -1;
        while (have && ok) {
            // the pass after, whose first pages are on their way meanwhile
            have = walk.next(p, y);
            ok = publish(++k, have, y);
            const int pg2 = have ? pages(y, y.j0) : -1;
            for (int j = x.j0; j < x.jl && ok; j += 16) {
                // (16 tiles' page ids are on their way while the 16 before are copied)
                const int pg3 = pages(x, j + 16);
                const int nt = min(16, x.jl - j);
                for (int i = 0; i < nt; ++i, ++seq) {
                    int page[2], there = 0;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        page[u] = __shfl_sync(0xffffffffu, pg, 2 * i + u);
                        if ((unsigned)page[u] < (unsigned)p.num_pages)
                            there |= 1 << u;
                        else if (lane == 0 && p.err && (long long)(2 * (j + i) + u) * kChunk < x.L)
                            atomicOr(p.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
                    }
                    const uint32_t st = seq % NS;
                    ok = warp_wait(&empty[st], ((seq / NS) & 1) ^ 1, abort_flag);
                    if (!ok) break;
                    uint64_t* bar = full + ((j + i + x.shift) & 1) * NS + st;
                    if (lane == 0) {
                        if (there == 0) {
                            mbar_arrive(bar);
                        } else {
                            constexpr uint32_t kPageBytes = FP8 ? 8192 : 16384;
                            mbar_arrive_expect_tx(bar, (there == 3 ? 2 : 1) * kPageBytes);
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                if (!(there >> u & 1)) continue;
                                uint8_t* dst = smem + st * LY::kStageBytes + u * 8192;
                                tma_load_3d(dst, &tm_k, bar, 0, x.h, page[u] * kChunk, pol);
                                if constexpr (!FP8) tma_load_3d(dst + 16384, &tm_k, bar, 64, x.h, page[u] * kChunk, pol);
                            }
                        }
                    }
                    uses[0] ^= ((j + i + x.shift) & 1) == 0 ? 1u << st : 0u;
                    uses[1] ^= ((j + i + x.shift) & 1) == 1 ? 1u << st : 0u;
                    __syncwarp();
                }
                pg = pg3;
            }
            x = y;
            pg = pg2;
        }
        // copies in flight land before the CTA can end: each barrier's last use
        if (lane == 0)
            for (int i = 0; i < 2 * NS; ++i)
                wait_bounded(&full[i], (uses[i / NS] >> (i % NS) & 1) ^ 1, nullptr, kDrainLimitNs);
    } else if (warp <= 2) {
        // ============================ issuers: warp 1 the even, warp 2 the odd turns (one lane issues;
        // the warp goes along)
        const uint32_t el = elect_lane();
        const int odd = warp - 1;
        constexpr uint32_t kId = FP8 ? idesc_e4m3(kTile, 0) : idesc_16bit(false, kTile, 0, 0);
        // descriptors of the first stage and slot; the others lie at fixed distances (in
        // 16-byte units, the low bits of a descriptor)
        const uint64_t dk = sdesc_sw128(smem_u32(smem), 16, 1024), dq = sdesc_sw128(smem_u32(smem + LY::kQ), 16, 1024);
        // accumulators of this issuer's two groups so far; bit st of uses: its uses of stage st, odd or even
        uint32_t seq = 0, qseq = 0, uses = 0, turn0 = 0, turn1 = 0;
        for (uint32_t k = 0; ok; ++k) {
            ok = pass_ready(k);
            if (!ok) break;
            const Pass& z = passes[k % kPasses];
            const int j0 = z.j0, jl = z.jl, rows_all = z.hi - z.lo, shift = z.shift;
            if (z.h < 0) break;
            pass_done(k);
            if (jl <= j0) continue;
            const int ns = (rows_all + kSlotRows - 1) / kSlotRows;
            int j = j0 + ((j0 + shift + odd) & 1);
            seq += j - j0;
            if (j >= jl) {  // none of the tiles is this issuer's
                for (int s = 0; s < ns && ok; ++s) {
                    ok = warp_wait(&qfull[(qseq + s) % kSlots], ((qseq + s) / kSlots) & 1, abort_flag);
                    if (ok && lane == 0) mbar_arrive(&qfree[(qseq + s) % kSlots]);
                }
                seq -= j - jl;
                qseq += ns;
                continue;
            }
            bool fresh = true;
            for (; j < jl && ok; j += 2, seq += 2) {
                const uint32_t st = seq % NS;
                ok = warp_wait(&full[odd * NS + st], uses >> st & 1, abort_flag);
                uses ^= 1u << st;
                const uint64_t dks = dk + st * (LY::kStageBytes >> 4);
                for (int s = 0; s < ns && ok; ++s) {
                    const uint32_t sl = (qseq + s) % kSlots;
                    if (fresh) ok = warp_wait(&qfull[sl], ((qseq + s) / kSlots) & 1, abort_flag);
                    const bool upper = shift >= kGroups ? s & 1 : (j + shift) >> 1 & 1;  // group odd + 2, or odd
                    const uint32_t c = upper ? turn1++ : turn0++;
                    const uint32_t acc = 2 * (odd + 2 * upper) + (c & 1);
                    if (ok) ok = warp_wait(&accfree[acc], ((c >> 1) & 1) ^ 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const int rows = min(kSlotRows, rows_all - s * kSlotRows);
                    const uint32_t id = kId | (uint32_t)((rows + 1) / 2) << 18;  // columns: a multiple of 16
                    const uint64_t q = dq + sl * (kSlotBytes >> 4);
                    const uint32_t d = tmem + acc * kCols;
                    if constexpr (FP8) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            umma_e4m3_el(el, d, dks + kk * 2, q + kk * 2, id, kk > 0);
                            umma_e4m3_el(el, d, dks + kk * 2, q + (kSlotHalf >> 4) + kk * 2, id, 1);
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_f16_el(el, d, dks + (kk >> 2) * 1024 + (kk & 3) * 2, q + (kk >> 2) * (kSlotHalf >> 4) + (kk & 3) * 2, id,
                                        kk > 0);
                    }
                    umma_commit_el(el, &accfull[acc]);
                    if (j + 2 >= jl) umma_commit_el(el, &qfree[sl]);
                }
                if (ok) umma_commit_el(el, &empty[st]);
                fresh = false;
            }
            seq -= j - jl;
            qseq += ns;
        }
    } else if (warp == 3) {
        // ============================ stager: query rows into slots
        uint32_t qseq = 0;
        for (uint32_t k = 0; ok; ++k) {
            ok = pass_ready(k);
            if (!ok) break;
            const Pass x = passes[k % kPasses];
            if (x.h < 0) break;
            pass_done(k);
            if (x.jl <= x.j0) continue;
            const int ns = x.slots();
            for (int s = 0; s < ns && ok; ++s, ++qseq) {
                const uint32_t sl = qseq % kSlots;
                ok = warp_wait(&qfree[sl], ((qseq / kSlots) & 1) ^ 1, abort_flag);
                if (!ok) break;
                const int r0 = x.lo + s * kSlotRows, rows = min(kSlotRows, x.hi - r0);
                uint8_t* slot = smem + LY::kQ + sl * kSlotBytes;
                uint64_t* bar = FP8 ? &qraw[sl] : &qfull[sl];
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, (uint32_t)rows * (2 * kGroup * 128));
                    for (int r = 0; r < rows;) {  // four rows a copy, then one
                        const int n = rows - r >= 4 ? 4 : 1;
                        const CUtensorMap* tm = n == 4 ? &tm_q4 : &tm_q1;
                        uint8_t* dst = slot + r * (kGroup * 128);
                        tma_load_3d_nohint(dst, tm, bar, 0, x.h * kGroup, x.q0 + r0 + r);
                        tma_load_3d_nohint(dst + kSlotHalf, tm, bar, 64, x.h * kGroup, x.q0 + r0 + r);
                        r += n;
                    }
                }
                const long long row0 = ((long long)x.q0 + r0) * p.num_q_heads + x.h * kGroup;
                for (int c = lane; c < rows * kGroup; c += 32) {
                    const float l = p.lse[row0 + (long long)(c / kGroup) * p.num_q_heads + c % kGroup];
                    nl[sl * kCols + c] = l == -INFINITY ? -INFINITY : -l * kLog2e;  // a row of -inf: no weight
                }
                if constexpr (FP8) {
                    ok = warp_wait(bar, (qseq / kSlots) & 1, abort_flag);
                    if (!ok) break;
                    for (int c0 = 0; c0 < rows * kGroup; c0 += 16) {
                        const int c = c0 + (lane >> 1);
                        const bool in = c < rows * kGroup;
                        const float up = split_query_row(slot, c, lane & 1, in, in);
                        if (in && (lane & 1) == 0) {
                            const float f = up * (kLog2e * 0.08838834764831845f);
                            qc[sl * kCols + c] = f;
                            qc[(kSlots + sl) * kCols + c] = up > 3.4e38f ? f : fminf(f * 0x1p64f, 3.4e38f);
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&qfull[sl]);
            }
        }
        // copies in flight land before the CTA can end
        if (lane == 0)
            for (uint32_t i = qseq > (uint32_t)kSlots ? qseq - kSlots : 0u; i < qseq; ++i)
                wait_bounded(FP8 ? &qraw[i % kSlots] : &qfull[i % kSlots], (i / kSlots) & 1, nullptr, kDrainLimitNs);
    } else {
        // ============================ groups g = 0 .. 3: thread = token of every fourth tile
        const int g = (warp >> 2) - 1, wq = warp & 3;
        constexpr float kScale = kLog2e * 0.08838834764831845f;  // log2(e) / sqrt(128)
        const bool upper = g >= 2;
        // This warp's part of a pass: tiles j, j + step, ... below j1, of which those below jl have
        // accumulators. A tile's half of 64 tokens is page pages[2 j] while 2 j < num_pages; the
        // thread's token is number 128 j + mine, its weight weights[128 j], read below `read` and
        // written below `write`.
        const int mine = 32 * wq + lane;
        struct View {
            const int32_t* pages;
            float* weights;
            const float* scales;
            int j, step, num_pages, read, write;
        };
        auto view = [&](const Pass& y) {
            View v;
            v.step = y.split() ? 2 : kGroups;
            v.j = y.j0 + ((g - y.shift - y.j0) & (v.step - 1));
            v.pages = p.page_table + y.b * p.pt_stride + (wq >> 1);
            v.num_pages = min(2 * y.j1, (y.L + kChunk - 1) / kChunk) - (wq >> 1);
            v.weights = p.weights + ((long long)y.b * p.num_kv_heads + y.h) * p.w_stride + mine;
            v.scales = FP8 ? p.k_scale + y.h * kChunk + (mine & (kChunk - 1)) : nullptr;
            const bool quiet = y.split() && upper;  // the other group of the tile has the sums
            v.read = quiet ? 0 : !y.first ? y.L : p.decay != 0.f ? y.p0 : 0;
            v.write = quiet ? 0 : y.L;
            return v;
        };
        // What a tile needs from memory comes a tile of the group ahead, its page id two: across
        // passes too, unless a pass goes on from the sums of the one before.
        float old = 0.f, factor = kScale;
        bool there = false;
        int page = -1;  // of the tile after the one ahead
        auto page_of = [&](const View& v, int j) { return 2 * j < v.num_pages ? v.pages[2 * j] : -1; };
        auto fetch = [&](const View& v, int j, int pg) {
            there = (unsigned)pg < (unsigned)p.num_pages;
            old = 0.f;
            if (j * kTile + mine < v.read) old = v.weights[(long long)j * kTile];
            if (FP8 && there) factor = v.scales[(long long)pg * p.num_kv_heads * kChunk];
        };
        uint32_t sl0 = 0, sl_lap = 0;  // the pass's first slot, and its lap's parity
        uint32_t turn = 0, met = 0;    // accumulators; meetings with the other group of the tile
        View v{};
        ok = pass_ready(0);
        if (ok && passes[0].h >= 0) {
            v = view(passes[0]);
            fetch(v, v.j, page_of(v, v.j));
            page = page_of(v, v.j + v.step);
        }
        for (uint32_t k = 0; ok; ++k) {
            const Pass& x = passes[k % kPasses];  // stays until this warp is done with it
            if (x.h < 0) break;
            ok = pass_ready(k + 1);
            if (!ok) break;
            const Pass& y = passes[(k + 1) % kPasses];
            int page_y = -1;
            if (y.h >= 0) {
                const View w = view(y);
                page_y = page_of(w, w.j);
            }
            const int rows_all = x.hi - x.lo, ns = x.slots(), j1 = x.j1, jl = x.jl;
            const int p0 = x.p0 + x.lo;  // the last token that the pass's first row sees
            const int first_slot = x.split() && upper ? 1 : 0, slot_step = x.split() ? 2 : 1;
            const bool meet = x.split() && ns > 1, first = x.first;
            bool any = false;      // this warp has seen the pass's slots
            bool fetched = false;  // what is ahead is of the next pass
            int j = v.j;
            for (; j < j1; j += v.step) {
                const float now_old = first ? p.decay * old : old;
                const bool now_there = there;
                const int t = j * kTile + mine;
                // Sums of products, up to 2^25, times a scale from 2^103 on are beyond float32 even where a tiny query's
                // score is not: such warps take 2^64 from the scales and give it to the rows' factors.
                const bool large = FP8 && __any_sync(0xffffffffu, t < x.L && fabsf(factor) >= 0x1p100f);
                const float now_scale = large ? factor * 0x1p-64f : factor;
                const uint64_t now_factor = pair(now_scale, now_scale);
                const float* qct = large ? qc + kSlots * kCols : qc;
                float* to = v.weights + (long long)j * kTile;
                const bool writes = t < v.write;
                const int next = j + v.step;
                if (next < j1) {
                    fetch(v, next, page);
                    page = page_of(v, next + v.step);
                } else if (y.h >= 0 && y.first) {
                    v = view(y);
                    fetch(v, v.j, page_y);
                    page = page_of(v, v.j + v.step);
                    fetched = true;
                }
                float sum = 0.f;
                if (j < jl) {
                    uint64_t sum2 = 0;
                    const bool clear = (j + 1) * kTile - 1 <= p0;  // every row sees every token
                    for (int s = first_slot; s < ns; s += slot_step) {
                        const uint32_t over = sl0 + s >= kSlots, sl = sl0 + s - (over ? kSlots : 0);
                        if (!any) ok = warp_wait(&qfull[sl], (sl_lap ^ over) & 1, abort_flag);
                        const uint32_t acc = 2 * g + (turn & 1);
                        if (ok) ok = warp_wait(&accfull[acc], (turn >> 1) & 1, abort_flag);
                        if (!ok) break;
                        ++turn;
                        tc_fence_after();
                        const int rows = min(kSlotRows, rows_all - s * kSlotRows);
                        const uint32_t ta = tmem + ((uint32_t)(32 * wq) << 16) + acc * kCols;
                        if (clear && rows == kSlotRows)
                            slot_rows<FP8, false>(ta, kSlotRows, 0, nl + sl * kCols, qct + sl * kCols, now_factor, sum2);
                        else  // row r of the slot sees the token from t - p0 - 8 s on
                            slot_rows<FP8, true>(ta, rows, t - p0 - s * kSlotRows, nl + sl * kCols, qct + sl * kCols, now_factor, sum2);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&accfree[acc]);
                    }
                    if (!ok) break;
                    any = true;
                    const float2 both = unpair(sum2);
                    sum = both.x + both.y;
                    if (meet) {
                        // the upper group's sum to the lower one's thread of the token, through one of two buffers
                        const uint32_t at = 2 * (g & 1) + (met & 1), turns = met >> 1;
                        float* half = part + at * kTile + mine;
                        ++met;
                        if (upper) {
                            ok = warp_wait(&partfree[at], (turns & 1) ^ 1, abort_flag);
                            if (!ok) break;
                            *half = sum;
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&partfull[at]);
                        } else {
                            ok = warp_wait(&partfull[at], turns & 1, abort_flag);
                            if (!ok) break;
                            sum += *half;
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&partfree[at]);
                        }
                    }
                    if (!now_there) sum = 0.f;
                }
                if (writes) *to = now_old + sum;
                if (fetched) break;
            }
            if (!ok) break;
            if (jl > x.j0) {
                // the slots are this pass's until every warp has seen them
                for (int s = 0; s < ns && ok; ++s) {
                    const uint32_t over = sl0 + s >= kSlots, sl = sl0 + s - (over ? kSlots : 0);
                    ok = warp_wait(&qfull[sl], (sl_lap ^ over) & 1, abort_flag);
                    if (ok && lane == 0) mbar_arrive(&qfree[sl]);
                }
                sl0 += ns;
                if (sl0 >= (uint32_t)kSlots) {
                    sl0 -= kSlots;
                    sl_lap ^= 1;
                }
            }
            if (y.h >= 0 && !fetched) {
                v = view(y);
                fetch(v, v.j, page_y);
                page = page_of(v, v.j + v.step);
            }
            pass_done(k);
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

// 3-D map over the query rows [num_tokens][Hq][128] bf16: box = 64 dims x 8 heads x `rows`,
// 128-byte swizzle (rows of an MMA operand tile).
bool make_q_rows_map(CUtensorMap* map, const void* q, int num_tokens, int Hq, int rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)Hq, (cuuint64_t)num_tokens};
    cuuint64_t strides[2] = {kHeadDim * 2, (cuuint64_t)Hq * kHeadDim * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)kGroup, (cuuint32_t)rows};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

template <bool FP8>
cudaError_t launch(const CUtensorMap (&maps)[3], const WeightParams& p, cudaStream_t s) {
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
    return launch_pdl(attn_weights_kernel<FP8>, dim3(ctas), dim3(kThreads), Layout<FP8>::kTotal, s, maps[0], maps[1], maps[2], p);
}

}  // namespace

cudaError_t launch_attn_weights(const AttnWeightsArgs& a, cudaStream_t s) {
    CUtensorMap maps[3];  // K; one and four rows of Q
    memset(maps, 0, sizeof maps);
    if (!make_kv_map(&maps[0], a.k_cache, a.fp8, a.num_pages, a.num_kv_heads) ||
        !make_q_rows_map(&maps[1], a.q, a.num_tokens, a.num_q_heads, 1) ||
        !make_q_rows_map(&maps[2], a.q, a.num_tokens, a.num_q_heads, 4))
        return cudaErrorInvalidValue;
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
    return a.fp8 ? launch<true>(maps, p, s) : launch<false>(maps, p, s);
}

}  // namespace hpc
