// Prompt attention and shared-prefix attention on the fifth-generation tensor
// cores, over the paged cache. Both are the same product: a tile of query tokens
// x 8 query heads against a run of 128-token KV blocks, with the running maximum
// and sum of a softmax:
//   S_j = Q K_j^T,  m = max(m, rowmax S_j),  P_j = exp(S_j - m),
//   l += rowsum P_j,  O += P_j V_j   (O and l scaled when m moves),
// then O / l and m + ln l. Prompts add the causal limit (query token t of a
// sequence of n tokens and L keys sees keys [0, L - n + t]); a prefix is seen
// whole by every row of its group. A tile map (tile.cuh) gives every worker an
// equal run of blocks; a tile that falls to one worker is written to the output,
// a cut one (and every prefix piece) as normalised float32 rows with their LSE,
// which the kernels in tile_combine.cu merge.
//
// One CTA per SM, 12 warps (e4m3: 16). A tile of 32 query tokens (two halves of
// 128 rows) belongs to one CTA (CG = 1), one of 64 to a pair of CTAs (CG = 2)
// whose products run on both SMs' tensor cores at once (cta_group::2, M = 256):
// each CTA keeps its own query rows, scores and sums, and loads only half of every
// K and V block (one page of K, one dim half of V), which halves the copies and the
// shared memory that the products read. The leader (rank 0) issues for both.
//  * warps 0-3 and 4-7, the softmax warpgroups of the two halves, a page of 64 keys
//    at a time: one thread per query row (e4m3: four threads per four rows). Scores
//    come from TMEM, P goes back over them as 16-bit pairs (the A operand of the
//    second product). The reference m is not the running maximum itself: P is made
//    against m as it stands, and its sum, which is needed anyway, tells whether the
//    maximum has to be looked at (kSumLimit). O is scaled in TMEM only then. P is
//    relative to m, so bf16 loses nothing by a P above 1, and f16 holds up to 65504.
//  * warp 8, producer: one thread issues TMA copies of the tile's query rows
//    and of K_0 V_0 K_1 V_1 ... into a ring of stages, pages through the table.
//  * warp 9, issuer: the MMAs in the order
//      S0(0) S1(0) | PV0(0) S0(1) PV1(0) S1(1) | PV0(1) ...
//    so that one half's products run while the other half's softmax does. MMAs
//    run in the order of their issue, so S(j+1) may overwrite P(j) once PV(j) has
//    been issued. In the other CTA of a pair this warp tells the leader which of
//    its blocks have landed.
//  * e4m3, warps 12-15: the query rows split into two e4m3 tiles of codes
//    (Q = (Q_hi + Q_lo) 2^e, as in attn_tc.cu), so that Q K^T runs on the K
//    codes as they are; V widened to f16 (code x scale) into a ring of its own.
// Every wait is bounded; on expiry the CTA records HPC_DEVERR_WAIT_TIMEOUT.
//
// Bound by: the tensor core and its power, over bf16 caches. Prompt of 8192 tokens,
// 64 / 8 heads: 670 to 682 us called back to back, 1610 to 1640 TFLOP/s (0.93 to 0.95 of
// the library's 8192^3 product over seconds), 648 to 662 us in short replays (0.87 to
// 0.89 of it in bursts); the tensor pipe is active for 75 % of the
// cycles and the clock falls from 2070 to 1750-1790 MHz at the board's power limit. A
// half's chain (its scores, 750 clocks of softmax per page, its product) leaves the
// rest: measured per block of two halves 2900 clocks of which 2048 are MMAs. Over
// e4m3 caches the softmax threads set the pace (the key scales' products and the
// other layout cost half as much again, the widening of V takes turns from them):
// 128 requests over a 65536-token prefix 210 us, 158 us over a bf16 cache.
// Few blocks (8192-token prefix, 64 requests: 22 us for seven blocks per CTA) are
// bound by latency: 1.4 us a block, 2.5 us to the first one, 3.2 us for a tile's
// float32 rows.
//
// What else was measured (8192-token prompt unless said otherwise):
//  * the maximum of each block taken before its P goes out: 749 us; page by page:
//    734 us; the sum as the test, and one barrier per block for K and V in place of
//    two (four in a pair: each test costs the issuer 150 to 200 clocks): 680 us.
//  * two threads per row (16 softmax warps of 96 registers): 775 against 735 us.
//  * scores double-buffered as two products of 64 keys: 811 us (an MMA of N = 64
//    takes 48 clocks, not 32). An issuer that polls for whichever half is ready:
//    1184 us; an issuer warp per half: 892 us (their tests take issue slots from the
//    softmax warps of the same scheduler).
//  * e4m3 with a thread per row, each reading all of a page's key scales from shared
//    memory: 512-token pieces of four prompts beside 28 single tokens 615 us, not 588.
//    V widened by rows of a thread, one 16-byte piece after the other: 548 us.
//  * output rows with the next columns' load under way: 668 against 660 us.
#include <atomic>
#include <cstring>

#include "attn_common.cuh"
#include "tcgen05.cuh"
#include "tile.cuh"

namespace hpc {
namespace {

using attn::kDrainLimitNs;
using attn::kLn2;
using attn::kNegInf;
using attn::kWaitLimitNs;
using attn::wait_bounded;

constexpr int kHalfRows = 128;
constexpr int kQBytes = 32768;           // a half's query rows: [2 dim halves][128 rows][128 B]
// 64 keys' P that add up to more than 2^10 hold one above 2^4: then the row's reference
// moves to their maximum. Up to there every P is at most 2^10.
constexpr float kSumLimit = 1024.f;
// Over e4m3 caches P is f16, whose normal numbers end at 2^-14 and whose last one is 2^-24:
// its reference is 2^5 below the maximum, so that weights down to 2^-30 of the largest have
// a part in O as they have in the sum, and P is at most 2^15.
constexpr float kHeadroom = 5.f, kSumLimitF16 = 32.f * kSumLimit;
static_assert(kSumLimitF16 <= 65504.f, "a P may be as large as its row's sum");
constexpr int kMetaRing = 8;             // blocks whose page checks (and, e4m3, scales) are kept
constexpr int kWide = 2;                 // e4m3: f16 V tiles
constexpr int kOutBytes = 2048;          // a softmax warp's staging of 32 output rows x 64 B
constexpr uint32_t kTmemCols = 512;      // S of half t at column 128 t (P over its first 64), O at 256 + 128 t

template <bool FP8, int CG>
struct Cfg {
    static constexpr int kStageBytes = (FP8 ? 16384 : 32768) / CG;  // 128 tokens of K or of V, or this CTA's half
    static constexpr int kWideBytes = 32768 / CG;
    static constexpr int kSlots = 2 * CG;  // blocks in the ring: a K stage and a V stage each
    static constexpr int kStages = 2 * kSlots;
    static_assert(kSlots <= kMetaRing, "slots");
    static constexpr int kWarps = FP8 ? 16 : 12;
    static constexpr int kThreads = kWarps * 32;
    // registers per thread after the split (setmaxnreg): the launch's total, 384 x
    // 168 or 512 x 128, is what the two softmax warpgroups and the others share
    static constexpr int kRegsSoftmax = FP8 ? 168 : 208;
    static constexpr int kRegsOther = 88;
    static_assert(256 * kRegsSoftmax + (kThreads - 256) * kRegsOther <= kThreads * (FP8 ? 128 : 168), "register split");
};

template <bool FP8, int CG>
struct Smem {
    using C = Cfg<FP8, CG>;
    static constexpr size_t kQ = 0;
    static constexpr size_t kRing = kQ + 2 * kQBytes;
    static constexpr size_t kWideV = kRing + (size_t)C::kStages * C::kStageBytes;
    static constexpr size_t kOut = kWideV + (FP8 ? (size_t)kWide * C::kWideBytes : 0);
    static constexpr size_t kKs = kOut + 8 * kOutBytes;                        // float [ring][128] K scales
    static constexpr size_t kVs = kKs + (FP8 ? kMetaRing * 512 : 0);           // float [ring][128] V scales
    static constexpr size_t kQs = kVs + (FP8 ? kMetaRing * 512 : 0);           // float [2 parities][2 halves][128]
    static constexpr size_t kMeta = kQs + (FP8 ? 2048 : 0);
    static constexpr size_t kBars = kMeta + kMetaRing * 4;
    // full (slots), empty (stages); qfull, qempty, sfull, pfull (2), pvdone, ofull,
    // ofree (halves); e4m3: q8full (halves), wfull, wempty (wide tiles)
    static constexpr int kNumBars = 3 * C::kSlots + 16 + (FP8 ? 2 + 2 * kWide : 0);
    static constexpr size_t kTmemSlot = kBars + kNumBars * 8;
    static constexpr size_t kFlag = kTmemSlot + 8;
    static constexpr size_t kAlloc = kFlag + 8 + 1024;
    static_assert(kAlloc <= 232448, "over the 227 KB shared-memory limit of a CTA");
    static_assert(kWideV % 1024 == 0 && kOut % 1024 == 0, "swizzled tiles need 1 KB alignment");
};

// ------------------------------------------------------------------ waits and arrivals

// A whole warp waits; one answer for all its lanes. (The issuer meets most of its
// barriers ready: a test and a vote are all that it then pays.)
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, kWaitLimitNs));
}

// Arrives on the leader's barrier at this address (this CTA's own for CG 1).
template <int CG>
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    if constexpr (CG == 1) {
        mbar_arrive(bar);
    } else {
        asm volatile(
            "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
            "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
            : "memory");
    }
}

template <int CG>
__device__ __forceinline__ void cluster_sync_all() {
    if constexpr (CG == 2) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
}

struct TileParams {
    const int32_t* plan;
    long long seqs_off;
    const int32_t* page_table;
    long long pt_stride;
    int* err;
    int S, mode, q_len, num_tokens, num_q_heads, num_pages, num_kv_heads;
    float* split_o;
    float* split_lse;
    __nv_bfloat16* out;
    float* out_lse;
    float scale_log2;
};

// The operands as they are in memory, for redo_rows. (A parameter of its own: within
// TileParams they make the bf16 instances spill.)
struct TileSources {
    const __nv_bfloat16* q;
    const void* k_cache;
    const void* v_cache;
    const float* k_scale;
    const float* v_scale;
};

__device__ __forceinline__ void tma_load_3d_plain(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                                  int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_2d_plain(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}

// D (TMEM) (+)= A . B^T for one CTA, or for a pair at once (each CTA's rows of A
// and D, half of B from each). ss: A and B in shared memory; ts: A (16-bit,
// K-major) in TMEM, lane = row, two elements of K per column.
// The whole warp runs these with the same operands and only its elected lane (el)
// issues: the operands then stay in uniform registers. Inside an `if (lane == 0)`
// they were moved there for every instruction, and with two busy softmax warps on
// the same scheduler the issue, not the tensor core, set the pace (a product pair
// of 16 MMAs took 1670 clocks in place of 1024).
template <int CG>
__device__ __forceinline__ void mma_ss_16(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void mma_ss_e4m3(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void mma_ts_16(uint32_t el, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
            : "memory");
}

// Arrives on bar (in both CTAs of a pair) once the MMAs issued before are done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t el, uint64_t* bar) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
            "r"(el)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3), "r"(el)
            : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e;
}

// 32 columns of this thread's lane (32x32b shape: thread t of a warp holds lane t
// of the warp's quarter).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]),
        "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]),
        "f"(r[18]), "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]),
        "f"(r[27]), "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// 64 columns of 16 lanes (16x256b shape): register 4 j + 2 k + e of thread t holds
// lane t / 4 + 8 k, column 8 j + 2 (t % 4) + e.
__device__ __forceinline__ void tmem_ld16x(uint32_t taddr, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr)
        : "memory");
}

// 32 columns of 16 lanes (16x128b shape): register 2 j + k of thread t goes to lane
// t / 4 + 8 k, column 4 j + t % 4.
__device__ __forceinline__ void tmem_st16x(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Values of four rows per thread (row t / 4 + 8 i of the warp's 32, the same in the
// row's four threads) -> the value of row `lane`.
__device__ __forceinline__ float row_value(const float (&x)[4], int lane) {
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float z = __shfl_sync(0xffffffffu, x[i], 4 * (lane & 7));
        if ((lane >> 3) == i) y = z;
    }
    return y;
}

// (a.x b.x + c.x, a.y b.y + c.y) and (a.x + b.x, a.y + b.y) in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Barrier 1 over the 128 threads of warps 12-15.
__device__ __forceinline__ void named_sync_128() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool named_any_128(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.red.or.pred.aligned q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// Two e4m3 codes of two f16 numbers (round to nearest even, saturated), and back.
__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(uint32_t x) {
    uint16_t y;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
    return y;
}

// This thread's row of O times al.
__device__ __forceinline__ void scale_o(uint32_t ocol, float al) {
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        float o[32];
        tmem_ld32(ocol + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= al;
        tmem_st32(ocol + c, o);
    }
}

// One half's bf16 query rows -> e4m3 hi / lo tiles in place ([128 rows][128 B]
// each) and their power-of-two row scales. Lanes 4 j .. 4 j + 3 of warp wq take row
// 32 wq + j + 8 u, u < 4; lane quarter qq reads bf16 dims [32 qq, 32 qq + 32), which
// sit where row r of the hi tile (qq < 2) or of the lo tile goes, and writes the hi
// and lo codes of its dims once all four have read.
// An element x / scale, at most 448, has eight significant bits: an f16 number without
// loss from 2^-17 on (below, both codes are zero). hi is its rounding to e4m3's four
// bits, lo the exact remainder's (its loss: split_e4m3x8). In f16 pairs a row takes a
// third fewer instructions than in float32, and a tile of few blocks waits for its rows.
__device__ __forceinline__ void split_query_rows(uint8_t* qt, float* qs, int wq, int lane) {
#pragma unroll 1
    for (int u0 = 0; u0 < 4; ++u0) {
        const int qq = lane & 3;
        uint4 raw[1][4];
        float amax[1], qinv[1];
#pragma unroll
        for (int u = 0; u < 1; ++u) {
            const int r = 32 * wq + 8 * (u0 + u) + (lane >> 2);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                raw[u][c] = *reinterpret_cast<const uint4*>(qt + (qq >> 1) * 16384 + r * 128 + (((4 * (qq & 1) + c) ^ (r & 7)) << 4));
        }
#pragma unroll
        for (int u = 0; u < 1; ++u) {
            __nv_bfloat162 am2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t w[4] = {raw[u][c].x, raw[u][c].y, raw[u][c].z, raw[u][c].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t x = w[j] & 0x7fff7fffu;
                    am2 = __hmax2(am2, *reinterpret_cast<const __nv_bfloat162*>(&x));
                }
            }
            amax[u] = fmaxf(__low2float(am2), __high2float(am2));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1)
#pragma unroll
            for (int u = 0; u < 1; ++u) amax[u] = fmaxf(amax[u], __shfl_xor_sync(0xffffffffu, amax[u], o));
        __syncwarp();  // the rows' other lanes have read them
#pragma unroll
        for (int u = 0; u < 1; ++u) {
            // the smallest power of two 2^ex with amax / 2^ex <= 448 = 1.75 2^8: q / 2^ex is exact
            // (rows under 2^-90 keep fewer bits: their scores are 0 to float32 anyway; an
            // infinite element makes the row's scores infinite or NaN)
            const uint32_t ab = __float_as_uint(amax[u]);
            const int ex = max((int)(ab >> 23) - 127 - 8 + ((ab & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
            float qscale = 1.f;
            qinv[u] = 1.f;
            if (amax[u] > 3.4e38f) {
                qscale = amax[u];
            } else if (amax[u] > 0.f) {
                qscale = __uint_as_float((uint32_t)(127 + ex) << 23);
                qinv[u] = __uint_as_float((uint32_t)(127 - ex) << 23);
            }
            if (qq == 0) qs[32 * wq + 8 * (u0 + u) + (lane >> 2)] = qscale;
        }
#pragma unroll
        for (int u = 0; u < 1; ++u) {
            const int r = 32 * wq + 8 * (u0 + u) + (lane >> 2);
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2) {
                uint32_t hp[4], lp[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint4 x4 = raw[u][2 * c2 + (v >> 1)];
                    const uint32_t w[2] = {v & 1 ? x4.z : x4.x, v & 1 ? x4.w : x4.y};
                    uint16_t h[2], l[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 y = mul2(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)),
                                              make_float2(qinv[u], qinv[u]));
                        const uint32_t x = pack_f16x2(y.x, y.y);
                        h[j] = f16x2_to_e4m3x2(x);
                        const uint32_t hb = e4m3x2_to_f16x2(h[j]);
                        const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&hb));
                        l[j] = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&rest));
                    }
                    hp[v] = h[0] | (uint32_t)h[1] << 16;
                    lp[v] = l[0] | (uint32_t)l[1] << 16;
                }
                const int off = r * 128 + (((2 * qq + c2) ^ (r & 7)) << 4);
                *reinterpret_cast<uint4*>(qt + off) = make_uint4(hp[0], hp[1], hp[2], hp[3]);
                *reinterpret_cast<uint4*>(qt + 16384 + off) = make_uint4(lp[0], lp[1], lp[2], lp[3]);
            }
        }
    }
}

// 128 tokens of V codes -> an f16 tile (code x scale, rounded to f16; rows from
// nv on zero), [dim halves][128 rows][128 B] swizzled: both dim halves from rows of
// 128 swizzled bytes (CG 1), or this CTA's half from plain rows of 64 bytes (CG 2).
// The scale is taken as (f 2^a) (2^b) with 1 <= |f| < 2, so that a scale far below
// f16's smallest normal number keeps its bits until the last product. Thread tg takes
// row tg: one scale and one look at it per block, and stores that spread over all
// banks (so do the loads of swizzled rows; plain rows of 64 bytes take four turns, an
// eighth of what the stores of the block take).
template <int CG>
__device__ __forceinline__ void widen_v(const uint8_t* codes, const float* vs, uint8_t* wide, int nv, int tg) {
    const bool in = tg < nv;
    const float sv = in ? vs[tg] : 0.f;
    const uint32_t sb = __float_as_uint(sv);
    const int e = (int)((sb >> 23) & 255u) - 127;
    // one product where the scale is a normal f16 number (or zero) in all the warp's rows
    const bool small = __any_sync(0xffffffffu, sv != 0.f && e < -14);
    uint32_t s2 = pack_f16x2(sv, sv), p2 = 0;
    if (small) {
        // f 2^a (NaN or infinity stay what they are) and 2^b, b = e - a (0 where it underflows)
        const int a = e < -14 ? -10 : 0;
        const float fa = e == 128 ? sv : __uint_as_float((sb & 0x807fffffu) | (uint32_t)(127 + a) << 23);
        const float fb = e == 128 ? 1.f : __uint_as_float((uint32_t)max(e - a + 127, 0) << 23);
        s2 = pack_f16x2(fa, fa), p2 = pack_f16x2(fb, fb);
    }
    // One piece after the other: batches of loads and stores, which end sooner, hold up the
    // softmax warps (pieces and decode, tile 32: four at once 619 us, two 584, one 546).
#pragma unroll 1
    for (int c16 = 0; c16 < 8 / CG; ++c16) {
        uint4 w = *reinterpret_cast<const uint4*>(CG == 1 ? codes + tg * 128 + ((c16 ^ (tg & 7)) << 4) : codes + tg * 64 + c16 * 16);
        if (!in) w = make_uint4(0, 0, 0, 0);
        uint4 vl, vh;
        e4m3x4_to_f16x2x2(w.x, vl.x, vl.y);
        e4m3x4_to_f16x2x2(w.y, vl.z, vl.w);
        e4m3x4_to_f16x2x2(w.z, vh.x, vh.y);
        e4m3x4_to_f16x2x2(w.w, vh.z, vh.w);
        vl.x = hmul2_u32(vl.x, s2), vl.y = hmul2_u32(vl.y, s2), vl.z = hmul2_u32(vl.z, s2), vl.w = hmul2_u32(vl.w, s2);
        vh.x = hmul2_u32(vh.x, s2), vh.y = hmul2_u32(vh.y, s2), vh.z = hmul2_u32(vh.z, s2), vh.w = hmul2_u32(vh.w, s2);
        if (small) {
            vl.x = hmul2_u32(vl.x, p2), vl.y = hmul2_u32(vl.y, p2), vl.z = hmul2_u32(vl.z, p2), vl.w = hmul2_u32(vl.w, p2);
            vh.x = hmul2_u32(vh.x, p2), vh.y = hmul2_u32(vh.y, p2), vh.z = hmul2_u32(vh.z, p2), vh.w = hmul2_u32(vh.w, p2);
        }
        uint8_t* dst = wide + (c16 >> 2) * 16384 + tg * 128;
        const int f0 = 2 * (c16 & 3);
        *reinterpret_cast<uint4*>(dst + ((f0 ^ (tg & 7)) << 4)) = vl;
        *reinterpret_cast<uint4*>(dst + (((f0 + 1) ^ (tg & 7)) << 4)) = vh;
    }
}

// Rows [nv, end of their page) of a bf16 V tile to zero: slots behind the
// sequence's last token may hold any bits, and 0 x NaN would reach the sums. Done by
// one warp. (Rows of pages that were not loaded came as zeros.)
template <int CG>
__device__ __forceinline__ void zero_tail(uint8_t* vt, int nv, int lane) {
    const int lo = max(nv, 0), hi = (lo + kChunk - 1) / kChunk * kChunk;
    constexpr int kPieces = 16 / CG;  // 16-byte pieces of a row
    for (int i = lane; i < (hi - lo) * kPieces; i += 32) {
        const int row = lo + i / kPieces, part = i % kPieces;
        *reinterpret_cast<uint4*>(vt + (part >> 3) * 16384 + row * 128 + (part & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// acc + 0 x for two bf16 numbers, or for one float: stays zero unless one is infinite or NaN
__device__ __forceinline__ uint32_t wild2(uint32_t x, uint32_t acc) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(acc));
    return d;
}
__device__ __forceinline__ float wild1(float x, float acc) {
    float d;
    asm("fma.rn.f32 %0, %1, 0f00000000, %2;" : "=f"(d) : "f"(x), "f"(acc));
    return d;
}

// Eight elements of a cache row, from element `at` on (e4m3: without their scale).
template <bool FP8>
__device__ __forceinline__ void cache8(const void* cache, long long at, float (&x)[8]) {
    if constexpr (FP8) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + at);
        uint32_t h[4];
        e4m3x4_to_f16x2x2(w.x, h[0], h[1]);
        e4m3x4_to_f16x2x2(w.y, h[2], h[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(cache) + at);
        const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(h[i] << 16), x[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
    }
}

// Rows of an item of a prompt whose sums came out infinite or NaN. In blocks of which a row
// does not see every key, the products multiply values that it must not see by zero, and 0
// x inf is NaN. So where such keys of the item hold a value that is not finite, the warp
// computes its rows again, key by key over those that the row sees, in float32 (m and inv
// are right: values have no part in them). `rows`: the warp's rows to look at; lim0: the
// keys that its first token sees. Not entered while all values are finite; a tile over 8192
// keys then takes 18 ms. (Looking at V before the products instead, in the issuer, in a
// warp of its own or while it is widened, cost every prompt 2 to 5 %, e4m3 9 %. With the look
// at the rows on their way out an 8192-token prompt takes 647 us, 648 before; e4m3 pieces and
// decode 554, 544 before, a 65536-token prefix 260, 265 before.)
template <bool FP8>
__device__ __forceinline__ void redo_rows(const TileParams& p, const TileSources& src, const TileItem& it, uint32_t rows, int lim0, int tok0, float m,
                                          float inv, bool direct, long long split_row0, int lane) {
    // the sequence, found again by its first query token
    const int4* seqs = reinterpret_cast<const int4*>(p.plan + p.seqs_off);
    int s0 = 0, s1 = p.S;
    while (s1 - s0 > 1) {
        const int mid = (s0 + s1) >> 1;
        if (seqs[mid].x <= it.q0)
            s0 = mid;
        else
            s1 = mid;
    }
    const int32_t* const table = p.page_table + (long long)s0 * p.pt_stride;
    // element and scale of key k's row; false: no valid page
    auto locate = [&](int k, long long& at, long long& sc) {
        const int c = k / kChunk, off = k % kChunk;
        const int page = c < p.pt_stride ? table[c] : -1;
        at = (((long long)page * kChunk + off) * p.num_kv_heads + it.h) * kHeadDim;
        sc = ((long long)page * p.num_kv_heads + it.h) * kChunk + off;
        return (unsigned)page < (unsigned)p.num_pages;
    };
    const int k_end = min(it.L, it.b1 * kBlock);
    float wild = 0.f;
#pragma unroll 1
    for (int k = max(max(lim0, 0), it.b0 * kBlock) + (lane >> 4); k < k_end; k += 2) {  // 16 lanes a row of V
        long long at, sc;
        float x[8];
        if (!locate(k, at, sc)) continue;
        cache8<FP8>(src.v_cache, at + 8 * (lane & 15), x);
        // (past f16's range counts as infinite: widen_v makes it so)
        if constexpr (FP8) wild = fabsf(src.v_scale[sc]) * 448.f <= 65504.f ? wild : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) wild = wild1(x[i], wild);
    }
    if (!__any_sync(0xffffffffu, wild != 0.f)) return;  // infinite or NaN for other reasons
    const long long step = (long long)p.num_kv_heads * kHeadDim;  // from key to key of a page
    // a token's eight rows at once: they see the same keys
#pragma unroll 1
    for (int u = 0; u < 4; ++u) {
        if (((rows >> (8 * u)) & 0xffu) == 0) continue;
        const int lim = min(k_end, lim0 + u);
        const long long qrow = (long long)(it.q0 + tok0 + u) * p.num_q_heads + it.h * kGroup;
        float o[kGroup][4];  // dims 4 lane ..
#pragma unroll
        for (int g = 0; g < kGroup; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[g][i] = 0.f;
#pragma unroll 1
        for (int k0 = it.b0 * kBlock; k0 < lim; k0 += 32) {  // 32 keys lie in one page
            long long at, sc;
            if (!locate(k0, at, sc)) continue;
            const int n = min(32, lim - k0);
            float w[kGroup];  // of key k0 + lane
#pragma unroll
            for (int g = 0; g < kGroup; ++g) w[g] = 0.f;
            if (lane < n) {
#pragma unroll 2
                for (int c = 0; c < kHeadDim; c += 8) {
                    float x[8];
                    cache8<FP8>(src.k_cache, at + lane * step + c, x);
#pragma unroll
                    for (int g = 0; g < kGroup; ++g) {
                        float y[8];
                        cache8<false>(src.q, (qrow + g) * kHeadDim + c, y);
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[g] = fmaf(x[i], y[i], w[g]);
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < kGroup; ++g) {
                if constexpr (FP8) w[g] *= src.k_scale[sc + lane];
                w[g] = fast_exp2(fmaf(w[g], p.scale_log2, -__shfl_sync(0xffffffffu, m, 8 * u + g)));
                if constexpr (FP8) w[g] *= src.v_scale[sc + lane];
            }
#pragma unroll 4
            for (int j = 0; j < n; ++j) {
                float x[4];
                if constexpr (FP8) {
                    uint32_t h[2];
                    e4m3x4_to_f16x2x2(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(src.v_cache) + at + j * step + 4 * lane),
                                      h[0], h[1]);
                    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h[0])),
                                 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h[1]));
                    x[0] = f0.x, x[1] = f0.y, x[2] = f1.x, x[3] = f1.y;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(src.v_cache) + at + j * step + 4 * lane);
                    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
                    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
                }
#pragma unroll
                for (int g = 0; g < kGroup; ++g) {
                    const float f = __shfl_sync(0xffffffffu, w[g], j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[g][i] = fmaf(f, x[i], o[g][i]);
                }
            }
        }
#pragma unroll
        for (int g = 0; g < kGroup; ++g) {
            const float f = __shfl_sync(0xffffffffu, inv, 8 * u + g);
            if (((rows >> (8 * u + g)) & 1u) == 0) continue;
            if (direct)
                *reinterpret_cast<uint2*>(p.out + (qrow + g) * kHeadDim + 4 * lane) =
                    make_uint2(pack_bf16x2(o[g][0] * f, o[g][1] * f), pack_bf16x2(o[g][2] * f, o[g][3] * f));
            else
                *reinterpret_cast<float4*>(p.split_o + (split_row0 + 8 * u + g) * kHeadDim + 4 * lane) =
                    make_float4(o[g][0] * f, o[g][1] * f, o[g][2] * f, o[g][3] * f);
        }
    }
}

template <bool FP8, int CG>
__global__ void __launch_bounds__(Cfg<FP8, CG>::kThreads, 1)
    tile_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_ks,
                     const __grid_constant__ CUtensorMap tm_vs, const TileParams p,
                     const __grid_constant__ TileSources src) {
    using C = Cfg<FP8, CG>;
    using LY = Smem<FP8, CG>;
    constexpr int NB = C::kSlots;
    constexpr int T = kTileCta * CG;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + LY::kBars);
    uint64_t* empty = full + NB;   // K and V stage of slot i at 2 i and 2 i + 1
    uint64_t* qfull = empty + 2 * NB;
    uint64_t* qempty = qfull + 2;
    uint64_t* sfull = qempty + 2;
    uint64_t* pfull = sfull + 2;
    uint64_t* pvdone = pfull + 4;  // (two P barriers per half: its first 64 keys, its last)
    uint64_t* ofull = pvdone + 2;  // pvdone: the product with the first 64 is done
    uint64_t* ofree = ofull + 2;
    uint64_t* q8full = ofree + 2;  // e4m3 from here on
    uint64_t* wfull = q8full + 2;
    uint64_t* wempty = wfull + kWide;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + LY::kTmemSlot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + LY::kFlag);
    volatile int* meta = reinterpret_cast<volatile int*>(smem + LY::kMeta);
    uint8_t* qbuf = smem + LY::kQ;
    uint8_t* ring = smem + LY::kRing;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0, worker = (int)blockIdx.x / CG;
    if (threadIdx.x == 0) {
        // the leader of a pair is also told when the other CTA's copies have landed
        const int told = CG == 2 && rank == 0 ? 2 : 1;
        for (int i = 0; i < NB; ++i) {
            mbar_init(&full[i], told);
            mbar_init(&empty[2 * i], 1);
            mbar_init(&empty[2 * i + 1], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&qfull[t], FP8 ? 1 : told);
            mbar_init(&qempty[t], 1);
            mbar_init(&sfull[t], 1);
            mbar_init(&pfull[2 * t], 4 * CG);  // one arrival per softmax warp
            mbar_init(&pfull[2 * t + 1], 4 * CG);
            mbar_init(&pvdone[t], 1);
            mbar_init(&ofull[t], 1);
            mbar_init(&ofree[t], 4 * CG);
        }
        if constexpr (FP8) {
            for (int t = 0; t < 2; ++t) mbar_init(&q8full[t], 4 * CG);
            for (int i = 0; i < kWide; ++i) {
                mbar_init(&wfull[i], CG);
                mbar_init(&wempty[i], 1);
            }
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(const_cast<uint32_t*>(tmem_slot))),
                         "r"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(const_cast<uint32_t*>(tmem_slot))),
                         "r"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all<CG>();  // the other CTA's barriers are set up too
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();  // the map, the query and the new tokens' keys come from the kernels before
    grid_launch_dependents();

    TileWalk<T> walk;
    walk.start(p.plan, worker);
    auto next = [&](TileItem& x) { return walk.next(x, p.S, p.mode, reinterpret_cast<const int4*>(p.plan + p.seqs_off)); };
    TileItem it;
    bool ok = true;

    if (!tile_map_is(p.plan, p.S, p.num_kv_heads, (int)gridDim.x / CG, p.num_tokens, p.mode, p.q_len, T)) {
        if (threadIdx.x == 0) atomicOr(p.err, (int)HPC_DEVERR_BAD_DESCRIPTOR);
    } else if (warp >= 8 && warp < 12) {
        reg_dec<C::kRegsOther>();
        if (warp == 8) {
            // ============================ producer
            uint32_t blks = 0, started = 0;  // blocks filled, and begun
            int nd[2] = {0, 0};
            while (ok && next(it)) {
                if (lane == 0) {
                    for (int t = 0; t < 2 && ok; ++t) {
                        if (it.i * T + t * kHalfTokens * CG >= it.n) break;
                        // rows past the sequence's last token load whatever follows (zeros
                        // past the last query row); they are computed and not written
                        const int tok = it.q0 + it.i * T + (t * CG + rank) * kHalfTokens;
                        ok = wait_bounded(&qempty[t], (nd[t] & 1) ^ 1, abort_flag, kWaitLimitNs);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&qfull[t], kQBytes);
                        tma_load_3d_plain(qbuf + t * kQBytes, &tm_q, &qfull[t], 0, it.h * kGroup, tok);
                        tma_load_3d_plain(qbuf + t * kQBytes + kQBytes / 2, &tm_q, &qfull[t], 64, it.h * kGroup, tok);
                        ++nd[t];
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                const int32_t* prow = p.page_table + (long long)it.s * p.pt_stride;
                const int pages = (int)(((long long)it.L + kChunk - 1) / kChunk);
                for (int c0 = 2 * it.b0; c0 < 2 * it.b1 && ok; c0 += 32) {
                    const int c = c0 + lane;
                    // a page past the last or with an id out of range becomes the page after
                    // the pool's last one: the copy fills its rows with zeros. (Pages past the
                    // table's row: only a map planned since for a wider table has such.)
                    int page = p.num_pages;
                    if (c < 2 * it.b1 && c < pages) {
                        page = c < p.pt_stride ? prow[c] : -1;
                        if ((unsigned)page >= (unsigned)p.num_pages) {
                            atomicOr(p.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
                            page = p.num_pages;
                        }
                    }
                    const int nb = min(16, it.b1 - (c0 >> 1));
                    for (int b = 0; b < nb && ok; ++b, ++blks) {
                        const int pg0 = __shfl_sync(0xffffffffu, page, 2 * b);
                        const int pg1 = __shfl_sync(0xffffffffu, page, 2 * b + 1);
                        if (lane == 0) {
                            const uint32_t slot = blks % NB;
                            for (int kvi = 0; kvi < 2 && ok; ++kvi) {
                                ok = wait_bounded(&empty[2 * slot + kvi], ((blks / NB) & 1) ^ 1, abort_flag, kWaitLimitNs);
                                if (!ok) break;
                                if (kvi == 0) {
                                    meta[blks % kMetaRing] = (pg0 < p.num_pages ? 1 : 0) | (pg1 < p.num_pages ? 2 : 0);
                                    mbar_arrive_expect_tx(&full[slot], 2 * (C::kStageBytes + (FP8 ? kBlock * 4 : 0)));
                                    started = blks + 1;
                                }
                                const CUtensorMap* tm = kvi == 0 ? &tm_k : &tm_v;
                                uint8_t* dst = ring + (size_t)(2 * slot + kvi) * C::kStageBytes;
                                if constexpr (FP8) {
                                    float* sc = reinterpret_cast<float*>(smem + (kvi == 0 ? LY::kKs : LY::kVs)) +
                                                (blks % kMetaRing) * kBlock;
                                    const CUtensorMap* ts = kvi == 0 ? &tm_ks : &tm_vs;
                                    tma_load_2d_plain(sc, ts, &full[slot], 0, pg0 * p.num_kv_heads + it.h);
                                    tma_load_2d_plain(sc + kChunk, ts, &full[slot], 0, pg1 * p.num_kv_heads + it.h);
                                }
                                if constexpr (CG == 2) {
                                    // K: this CTA's page, both dim halves; V: both pages, this CTA's dim half
                                    if (kvi == 0) {
                                        const int tok = (rank ? pg1 : pg0) * kChunk;
                                        tma_load_3d_plain(dst, tm, &full[slot], 0, it.h, tok);
                                        if constexpr (!FP8) tma_load_3d_plain(dst + 8192, tm, &full[slot], 64, it.h, tok);
                                    } else {
                                        tma_load_3d_plain(dst, tm, &full[slot], 64 * rank, it.h, pg0 * kChunk);
                                        tma_load_3d_plain(dst + (FP8 ? 4096 : 8192), tm, &full[slot], 64 * rank, it.h, pg1 * kChunk);
                                    }
                                } else {
                                    tma_load_3d_plain(dst, tm, &full[slot], 0, it.h, pg0 * kChunk);
                                    tma_load_3d_plain(dst + 8192, tm, &full[slot], 0, it.h, pg1 * kChunk);
                                    if constexpr (!FP8) {
                                        tma_load_3d_plain(dst + 16384, tm, &full[slot], 64, it.h, pg0 * kChunk);
                                        tma_load_3d_plain(dst + 24576, tm, &full[slot], 64, it.h, pg1 * kChunk);
                                    }
                                }
                            }
                        }
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                    }
                }
            }
            // no copy is in flight when the CTA ends, whichever way the walk ended
            if (lane == 0) {
                for (uint32_t k = started > (uint32_t)NB ? started - NB : 0u; k < started; ++k)
                    wait_bounded(&full[k % NB], (k / NB) & 1, nullptr, kDrainLimitNs);
                for (int t = 0; t < 2; ++t)
                    if (nd[t] > 0) wait_bounded(&qfull[t], (nd[t] - 1) & 1, nullptr, kDrainLimitNs);
            }
        } else if (warp == 9 && rank == 0) {
            // ============================ issuer
            constexpr uint32_t kIdS = FP8 ? idesc_e4m3(CG * kHalfRows, kBlock) : idesc_16bit(false, CG * kHalfRows, kBlock, 0);
            constexpr uint32_t kIdO = idesc_16bit(FP8, CG * kHalfRows, kHeadDim, 1);
            constexpr uint32_t kKHalf = 16384 / CG;  // bytes of a K tile's dim half
            uint32_t blks = 0;          // blocks
            uint32_t np[2] = {0, 0};    // P tiles taken
            int nd[2] = {0, 0};         // items
            // block number k is filled (in both CTAs)
            auto wait_block = [&](uint32_t k) { return wait_warp(&full[k % NB], (k / NB) & 1, abort_flag); };
            const uint32_t el = elect_one();
            // descriptors of the first query tile, stage and V tile; the others lie at
            // fixed distances (in 16-byte units, the low bits of a descriptor)
            const uint64_t dq = sdesc_sw128(smem_u32(qbuf), 16, 1024), dk = sdesc_sw128(smem_u32(ring), 16, 1024);
            const uint64_t dv = sdesc_sw128(smem_u32(FP8 ? smem + LY::kWideV : ring), 16384, 1024);
            // S of half t from the K tile in slot sl
            auto issue_s = [&](int t, uint32_t sl) {
                const uint64_t q = dq + (uint32_t)t * (kQBytes >> 4), k = dk + sl * (2 * C::kStageBytes >> 4);
                if constexpr (FP8) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        mma_ss_e4m3<CG>(el, tmem + 128 * t, q + kk * 2, k + kk * 2, kIdS, kk > 0);
                        mma_ss_e4m3<CG>(el, tmem + 128 * t, q + 1024 + kk * 2, k + kk * 2, kIdS, 1);
                    }
                } else {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ss_16<CG>(el, tmem + 128 * t, q + (kk >> 2) * 1024 + (kk & 3) * 2,
                                      k + (kk >> 2) * (kKHalf >> 4) + (kk & 3) * 2, kIdS, kk > 0);
                }
                mma_commit<CG>(el, &sfull[t]);
            };
            while (ok && next(it)) {
                const int halves = it.n - it.i * T > kHalfTokens * CG ? 2 : 1;
                // first S of both halves
                ok = wait_block(blks);
                for (int t = 0; t < halves && ok; ++t) {
                    ok = wait_warp(FP8 ? &q8full[t] : &qfull[t], nd[t] & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    issue_s(t, blks % NB);
                    if (it.b1 - it.b0 == 1) mma_commit<CG>(el, &qempty[t]);
                    if (t == halves - 1) mma_commit<CG>(el, &empty[2 * (blks % NB)]);
                }
                for (int b = it.b0; b < it.b1 && ok; ++b, ++blks) {
                    const uint32_t vst = 2 * (blks % NB) + 1, after = (blks + 1) % NB;
                    const bool more = b + 1 < it.b1;
                    uint8_t* vt = FP8 ? smem + LY::kWideV + (blks % kWide) * C::kWideBytes : ring + (size_t)vst * C::kStageBytes;
                    const uint64_t v = dv + (FP8 ? (blks % kWide) * (C::kWideBytes >> 4) : vst * (C::kStageBytes >> 4));
                    if constexpr (FP8) {
                        ok = wait_warp(&wfull[blks % kWide], (blks / kWide) & 1, abort_flag);
                        if (!ok) break;
                    } else {
                        const int nv = it.L - b * kBlock;
                        if (nv < kBlock && (nv & (kChunk - 1)) != 0) zero_tail<CG>(vt, nv, lane);
                    }
                    for (int t = 0; t < halves && ok; ++t) {
                        // the first product of an item overwrites O: the item before must have left it
                        if (b == it.b0 && nd[t] > 0) ok = wait_warp(&ofree[t], (nd[t] - 1) & 1, abort_flag);
                        // P comes in two parts, so that its first product runs while the softmax
                        // still works on the second
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            ok = ok && wait_warp(&pfull[2 * t + u], np[t] & 1, abort_flag);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int kk = 4 * u; kk < 4 * u + 4; ++kk)
                                mma_ts_16<CG>(el, tmem + 256 + 128 * t, tmem + 128 * t + kk * 8, v + kk * 128, kIdO,
                                              b > it.b0 || kk > 0);
                            if (u == 0) mma_commit<CG>(el, &pvdone[t]);
                        }
                        if (!ok) break;
                        ++np[t];
                        if (t == halves - 1) mma_commit<CG>(el, FP8 ? &wempty[blks % kWide] : &empty[vst]);
                        if (more) {
                            if (t == 0) {
                                ok = wait_block(blks + 1);
                                if (!ok) break;
                                tc_fence_after();
                            }
                            issue_s(t, after);
                            if (b + 2 == it.b1) mma_commit<CG>(el, &qempty[t]);
                            if (t == halves - 1) mma_commit<CG>(el, &empty[2 * after]);
                        } else {
                            mma_commit<CG>(el, &ofull[t]);
                        }
                    }
                }
                for (int t = 0; t < halves; ++t) ++nd[t];
            }
        } else if (warp == 9) {
            // ============================ the other CTA of a pair: its filled query rows and
            // slots, told to the leader in order
            uint32_t blks = 0;
            int nd[2] = {0, 0};
            while (ok && next(it)) {
                const int halves = it.n - it.i * T > kHalfTokens * CG ? 2 : 1;
                if constexpr (!FP8)
                    for (int t = 0; t < halves && ok; ++t, ++nd[t - 1]) {
                        ok = wait_warp(&qfull[t], nd[t] & 1, abort_flag);
                        if (ok && lane == 0) arrive_leader<CG>(&qfull[t]);
                    }
                for (int b = it.b0; b < it.b1 && ok; ++b, ++blks) {
                    ok = wait_warp(&full[blks % NB], (blks / NB) & 1, abort_flag);
                    if (!ok) break;
                    if constexpr (!FP8) {
                        const int nv = it.L - b * kBlock;
                        if (nv < kBlock && (nv & (kChunk - 1)) != 0)
                            zero_tail<CG>(ring + (size_t)(2 * (blks % NB) + 1) * C::kStageBytes, nv, lane);
                    }
                    if (lane == 0) arrive_leader<CG>(&full[blks % NB]);
                }
            }
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            atomicOr(p.err, (int)HPC_DEVERR_WAIT_TIMEOUT);
        }
    } else if (warp >= 12) {
        // ============================ e4m3: query rows split, V widened
        if constexpr (FP8) {
            reg_dec<C::kRegsOther>();
            const int tg = threadIdx.x & 127, wq = warp & 3;
            uint32_t blks = 0;
            int nd[2] = {0, 0};
            while (ok && next(it)) {
                const int halves = it.n - it.i * T > kHalfTokens * CG ? 2 : 1;
                for (int t = 0; t < halves && ok; ++t) {
                    ok = wait_warp(&qfull[t], nd[t] & 1, abort_flag);
                    if (!ok) break;
                    split_query_rows(qbuf + t * kQBytes, reinterpret_cast<float*>(smem + LY::kQs) + (nd[t] & 1) * 256 + t * 128,
                                     wq, lane);
                    ++nd[t];
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_leader<CG>(&q8full[t]);
                }
                // (a warp that gave up must not leave the others at a barrier)
                ok = !named_any_128(!ok);
                for (int b = it.b0; b < it.b1 && ok; ++b, ++blks) {
                    const uint32_t st = 2 * (blks % NB) + 1;  // V of the CTA's block number blks
                    ok = wait_warp(&wempty[blks % kWide], ((blks / kWide) & 1) ^ 1, abort_flag) &&
                         wait_warp(&full[blks % NB], (blks / NB) & 1, abort_flag);
                    ok = !named_any_128(!ok);
                    if (!ok) break;
                    widen_v<CG>(ring + (size_t)st * C::kStageBytes,
                                reinterpret_cast<const float*>(smem + LY::kVs) + (blks % kMetaRing) * kBlock,
                                smem + LY::kWideV + (blks % kWide) * C::kWideBytes, it.L - b * kBlock, tg);
                    fence_proxy_async_smem();
                    named_sync_128();
                    if (tg == 0) {
                        arrive_leader<CG>(&wfull[blks % kWide]);
                        mbar_arrive(&empty[st]);
                    }
                }
            }
            if (!ok && lane == 0) {
                *abort_flag = 1;
                atomicOr(p.err, (int)HPC_DEVERR_WAIT_TIMEOUT);
            }
        }
    } else {
        reg_inc<C::kRegsSoftmax>();
        // ============================ softmax warpgroup of half t, one thread per row
        const int t = warp >> 2;
        const uint32_t lane_addr = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t scol = tmem + lane_addr + 128 * t, ocol = tmem + lane_addr + 256 + 128 * t;
        const int half_tok = (t * CG + rank) * kHalfTokens;  // the half's first token in the tile
        uint8_t* stage = smem + LY::kOut + warp * kOutBytes;
        uint32_t blks = 0;  // blocks of this CTA
        uint32_t ns = 0;    // score tiles of this half
        int nd = 0;
        while (ok && next(it)) {
            if (it.n - it.i * T <= t * kHalfTokens * CG) {  // an empty half
                blks += it.b1 - it.b0;
                continue;
            }
            // keys that this row sees, and those that the warp's first row does; rows past the
            // sequence's last token (computed, not written) see no more than the sequence has
            const int lim0 = it.L - it.n + it.i * T + half_tok + 4 * (warp & 3) + 1;
            const int lim_w = p.mode == kModePrefix ? it.L : min(it.L, lim0);
            const int lim = p.mode == kModePrefix ? it.L : min(it.L, lim0 + lane / kGroup);
            float m = kNegInf, l = 0.f;  // reference maximum (log2 domain) and sum
            const float sc = p.scale_log2;
            // e4m3: the same of the four rows that the thread has parts of
            float mq[4], lq[4], scq[4];
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) mq[i] = kNegInf, lq[i] = 0.f;
            }
            for (int b = it.b0; b < it.b1; ++b, ++blks, ++ns) {
                if (!wait_warp(&sfull[t], ns & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // which of the block's keys this row sees
                const int nv_w = lim_w - b * kBlock, pages_ok = meta[blks % kMetaRing];
                if constexpr (FP8) {
                    // The key scales come from shared memory, and with a row per thread every
                    // thread would read them all. Here a thread has parts of four rows: query
                    // head hq of the warp's tokens i = 2 gi + k, columns 8 j + 2 cq and the next
                    // (the 16x256b shape's layout, for TMEM lanes 16 gi ..): a quarter of them.
                    const int hq = lane >> 2, cq = lane & 3;
                    const int left = it.L - b * kBlock - 2 * cq;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float s[2][32];  // [gi][4 j + 2 k + column parity]
                        tmem_ld16x(scol + kChunk * u, s[0]);
                        tmem_ld16x(scol + kChunk * u + (16u << 16), s[1]);
                        const bool page_ok = (pages_ok >> u) & 1;
                        tmem_ld_wait();
                        if (u == 0 && b == it.b0) {
                            // (the scores exist, so the splitter's row scales do too)
                            const float* qs = reinterpret_cast<const float*>(smem + LY::kQs) + (nd & 1) * 256 + t * 128 + 32 * (warp & 3) + hq;
#pragma unroll
                            for (int i = 0; i < 4; ++i) scq[i] = sc * qs[8 * i];
                        }
                        const float2* ks = reinterpret_cast<const float2*>(smem + LY::kKs + (blks % kMetaRing) * 512) + 32 * u + cq;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 f = ks[4 * j];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float* x = s[i >> 1] + 4 * j + 2 * (i & 1);
                                const float2 y = mul2(make_float2(x[0], x[1]), f);
                                x[0] = y.x, x[1] = y.y;
                            }
                        }
                        if (nv_w < kChunk * (u + 1) || !page_ok) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int see = p.mode == kModePrefix ? left : min(left, lim0 + i - b * kBlock - 2 * cq);
                                const int n = page_ok ? see - kChunk * u : 0;
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    float* x = s[i >> 1] + 4 * j + 2 * (i & 1);
                                    if (8 * j >= n) x[0] = kNegInf;
                                    if (8 * j + 1 >= n) x[1] = kNegInf;
                                }
                            }
                        }
                        // P of the page, to TMEM as f16 pairs; the thread's parts of the rows' sums
                        float sum[4] = {0.f, 0.f, 0.f, 0.f}, neg[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) neg[i] = -mq[i];  // (no finite sum where mq is not)
                        auto exps = [&]() {
#pragma unroll
                            for (int gi = 0; gi < 2; ++gi) {
                                uint32_t pk[16];
                                float2 a[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                                for (int j = 0; j < 8; ++j)
#pragma unroll
                                    for (int k = 0; k < 2; ++k) {
                                        const int i = 2 * gi + k;
                                        const float* y = s[gi] + 4 * j + 2 * k;
                                        float2 x = fma2(make_float2(y[0], y[1]), make_float2(scq[i], scq[i]), make_float2(neg[i], neg[i]));
                                        x.x = fast_exp2(x.x);
                                        x.y = fast_exp2(x.y);
                                        a[k] = add2(a[k], x);
                                        pk[2 * j + k] = pack_f16x2(x.x, x.y);
                                    }
                                tmem_st16x(scol + ((uint32_t)(16 * gi) << 16) + 32 * u, pk);
                                sum[2 * gi] = a[0].x + a[0].y;
                                sum[2 * gi + 1] = a[1].x + a[1].y;
                            }
                        };
                        // As below, the sum being of 16 keys, and the second pass by the same
                        // instructions: a tile of few blocks waits for the instruction cache (32
                        // prompts of 512 tokens behind 88: 324 us with a copy of its own, 306 so;
                        // over bf16 caches the copy is the faster form, 650 against 690 us for an
                        // 8192-token prompt).
                        bool take = __all_sync(0xffffffffu, mq[0] == kNegInf && mq[1] == kNegInf && mq[2] == kNegInf && mq[3] == kNegInf);
                        bool taken = false;
#pragma unroll 1
                        for (;;) {
                            if (!take) {
                                exps();
                                bool high = false;
#pragma unroll
                                for (int i = 0; i < 4; ++i) high |= !(sum[i] <= kSumLimitF16 / 4);
                                if (taken || !__any_sync(0xffffffffu, high)) break;
                            }
                            take = false;
                            taken = true;
                            float al[4];
                            bool resc = false;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float* x = s[i >> 1] + 2 * (i & 1);
                                float mx = fmaxf(x[0], x[1]);
#pragma unroll
                                for (int j = 1; j < 8; ++j) mx = max3(mx, x[4 * j], x[4 * j + 1]);
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                                mx = fmaf(fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)), scq[i], -kHeadroom);
                                float all = sum[i];  // the row's
                                all += __shfl_xor_sync(0xffffffffu, all, 1);
                                all += __shfl_xor_sync(0xffffffffu, all, 2);
                                const bool move = mq[i] == kNegInf ? mx != kNegInf : mx > mq[i] && !(all <= kSumLimitF16);
                                al[i] = move && mq[i] != kNegInf ? fast_exp2(mq[i] - mx) : 1.f;
                                resc |= move && mq[i] != kNegInf;
                                if (move) mq[i] = mx;
                                neg[i] = mq[i] == kNegInf ? 0.f : -mq[i];
                                lq[i] *= al[i];
                            }
                            if (__any_sync(0xffffffffu, resc)) {
                                if (u == 1 && !wait_warp(&pvdone[t], ns & 1, abort_flag)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                scale_o(ocol, row_value(al, lane));
                            }
                        }
                        if (!ok) break;
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_leader<CG>(&pfull[2 * t + u]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) lq[i] += sum[i];
                    }
                } else {
                    const int nv = lim - b * kBlock;
                    // A page's 64 keys at a time: their product with V runs while the softmax works
                    // on the next ones.
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float s[kChunk];
                        tmem_ld32(scol + kChunk * u, s);
                        tmem_ld32(scol + kChunk * u + 32, s + 32);
                        const bool page_ok = (pages_ok >> u) & 1;
                        tmem_ld_wait();
                        if (nv_w < kChunk * (u + 1) || !page_ok) {
                            const int n = page_ok ? nv - kChunk * u : 0;
#pragma unroll
                            for (int c = 0; c < kChunk; ++c)
                                if (c >= n) s[c] = kNegInf;
                        }
                        // P = exp2(s sc - m), to TMEM as 16-bit pairs; returns the sum
                        auto exps = [&](float neg) {
                            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                            for (int c = 0; c < kChunk; c += 32) {
                                uint32_t pk[16];
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    float2 x = fma2(make_float2(s[c + 2 * i], s[c + 2 * i + 1]), make_float2(sc, sc), make_float2(neg, neg));
                                    x.x = fast_exp2(x.x);
                                    x.y = fast_exp2(x.y);
                                    sum[i & 1] = add2(sum[i & 1], x);
                                    pk[i] = pack_bf16x2(x.x, x.y);
                                }
                                tmem_st16(scol + (kChunk * u + c) / 2, pk);
                            }
                            return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                        };
                        // Against the reference as it stands. The sum tells whether that still serves:
                        // one up to kSumLimit bounds every P. Only where it is above, or where a row has
                        // no reference yet, the keys' maximum is taken and they are done again.
                        // (A row's own sum decides, so that its result does not depend on the warp's
                        // other rows.)
                        const bool fresh = m == kNegInf, all_fresh = __all_sync(0xffffffffu, fresh);
                        float sum = 0.f;
                        if (!all_fresh) sum = exps(-m);  // (not finite where m is not)
                        if (all_fresh || __any_sync(0xffffffffu, !(sum <= kSumLimit))) {
                            float mx[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) mx[i] = fmaxf(s[i], s[60 + i]);
#pragma unroll
                            for (int c = 4; c < 60; c += 8)
#pragma unroll
                                for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], s[c + i], s[c + 4 + i]);
                            const float mraw = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * sc;
                            const bool move = fresh ? mraw != kNegInf : mraw > m && !(sum <= kSumLimit);
                            const bool resc = move && m != kNegInf;
                            if (__any_sync(0xffffffffu, resc)) {
                                // O holds everything before these keys once their predecessors' product
                                // is done: the last block's is (it was issued before this block's
                                // scores), the first page's of this block says so
                                if (u == 1 && !wait_warp(&pvdone[t], ns & 1, abort_flag)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                const float al = resc ? fast_exp2(m - mraw) : 1.f;
                                scale_o(ocol, al);
                                l *= al;
                            }
                            if (move) m = mraw;
                            sum = exps(m == kNegInf ? 0.f : -m);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_leader<CG>(&pfull[2 * t + u]);
                        l += sum;
                    }
                }
                if (!ok) break;
            }
            if (!ok) break;
            // ---- the tile's rows
            if (!wait_warp(&ofull[t], nd & 1, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lq[i] += __shfl_xor_sync(0xffffffffu, lq[i], 1);
                    lq[i] += __shfl_xor_sync(0xffffffffu, lq[i], 2);
                }
                m = row_value(mq, lane);
                l = row_value(lq, lane);
            }
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            const float lse = l > 0.f || l != l ? (m == kNegInf ? 0.f : m) * kLn2 + logf(l) : kNegInf;
            const bool direct = p.mode == kModePrefill && it.whole;
            const int tok0 = it.i * T + half_tok;        // the half's first token in the sequence
            const int wtok = 4 * (warp & 3);             // the warp's first token in the half
            const int live = it.n - tok0 - wtok;         // the warp's tokens that exist
            // Rows go out 64 bytes at a time, through shared memory: the warp then writes 64
            // bytes of one token's eight rows at once (lane / 4: query head, lane % 4: 16-byte
            // piece), its four tokens one after the other.
            const int sw = (lane >> 1) & 3, hd = lane >> 2;
            uint4* const put = reinterpret_cast<uint4*>(stage + lane * 64);
            const uint8_t* const get = stage + hd * 64 + (((lane & 3) ^ ((hd >> 1) & 3)) << 4);
            uint32_t wild = 0;  // not zero: this thread's row has an infinity or NaN
            if (direct) {
                const long long row0 = (long long)(it.q0 + tok0 + wtok) * p.num_q_heads + it.h * kGroup;
                const long long step = (long long)p.num_q_heads * kHeadDim;
                __nv_bfloat16* dst = p.out + (row0 + hd) * kHeadDim + 8 * (lane & 3);
#pragma unroll 1
                for (int c = 0; c < 128; c += 32, dst += 32) {
                    float o[32];
                    tmem_ld32(ocol + c, o);
                    tmem_ld_wait();
                    // rows that saw nothing are zero, whatever O holds
                    if (inv == 0.f) {
#pragma unroll
                        for (int u = 0; u < 32; ++u) o[u] = 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint4 x = make_uint4(pack_bf16x2(o[8 * u] * inv, o[8 * u + 1] * inv),
                                                   pack_bf16x2(o[8 * u + 2] * inv, o[8 * u + 3] * inv),
                                                   pack_bf16x2(o[8 * u + 4] * inv, o[8 * u + 5] * inv),
                                                   pack_bf16x2(o[8 * u + 6] * inv, o[8 * u + 7] * inv));
                        put[u ^ sw] = x;
                        wild = wild2(x.x, wild2(x.y, wild2(x.z, wild2(x.w, wild))));
                    }
                    __syncwarp();
                    uint4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(get + 512 * i);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < live) *reinterpret_cast<uint4*>(dst + i * step) = v[i];
                    __syncwarp();
                }
                // this thread's own row: token lane / 8 of the warp, query head lane % 8
                if (p.out_lse && (lane >> 3) < live) p.out_lse[row0 + (long long)(lane >> 3) * p.num_q_heads + (lane & 7)] = lse;
            } else {
                const long long row0 = tile_slot(p.mode, worker, it) * (T * kGroup) + (half_tok + wtok) * kGroup;
                float* dst = p.split_o + (row0 + hd) * kHeadDim + 4 * (lane & 3);
#pragma unroll 1
                for (int c = 0; c < 128; c += 16, dst += 16) {
                    float o[16];
                    tmem_ld16(ocol + c, o);
                    tmem_ld_wait();
                    if (inv == 0.f) {
#pragma unroll
                        for (int u = 0; u < 16; ++u) o[u] = 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float4 x = make_float4(o[4 * u] * inv, o[4 * u + 1] * inv, o[4 * u + 2] * inv, o[4 * u + 3] * inv);
                        reinterpret_cast<float4*>(put)[u ^ sw] = x;
                        wild |= __float_as_uint(wild1(x.x, wild1(x.y, wild1(x.z, wild1(x.w, 0.f)))));
                    }
                    __syncwarp();
                    float4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float4*>(get + 512 * i);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < live) *reinterpret_cast<float4*>(dst + i * kGroup * kHeadDim) = v[i];
                    __syncwarp();
                }
                if ((lane >> 3) < live) p.split_lse[row0 + lane] = lse;
            }
            const uint32_t again = __ballot_sync(0xffffffffu, wild != 0 && (lane >> 3) < live);
            if (again != 0 && p.mode == kModePrefill)
                redo_rows<FP8>(p, src, it, again, it.L - it.n + tok0 + wtok + 1, tok0 + wtok, m, inv, direct,
                               tile_slot(p.mode, worker, it) * (T * kGroup) + (half_tok + wtok) * kGroup, lane);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader<CG>(&ofree[t]);
            ++nd;
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            atomicOr(p.err, (int)HPC_DEVERR_WAIT_TIMEOUT);
        }
    }
    // normal end: every MMA was waited for by an epilogue; after a timeout give
    // what is in flight a bounded time
    __syncwarp();
    if (*abort_flag && warp == 0) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < kDrainLimitNs) {
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all<CG>();  // no CTA of a pair ends while the other still works with it
    tc_fence_after();
    if (warp == 0) {
        if constexpr (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// 3-D map over the query [tokens][Hq][128] bf16: box = 64 dims x 8 heads x 16
// tokens, 128-byte swizzle (half of an MMA operand tile).
bool make_tile_q_map(CUtensorMap* map, const void* q, int tokens, int Hq) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)Hq, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {kHeadDim * 2, (cuuint64_t)Hq * kHeadDim * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)kGroup, (cuuint32_t)kHalfTokens};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map over an e4m3 cache's V codes with boxes of 64 dims x 64 tokens, rows
// as they are: one CTA's half of a page.
bool make_v_half_map(CUtensorMap* map, const void* base, int num_pages, int Hkv) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)Hkv, (cuuint64_t)num_pages * kChunk};
    cuuint64_t strides[2] = {kHeadDim, (cuuint64_t)Hkv * kHeadDim};
    cuuint32_t box[3] = {64u, 1u, (cuuint32_t)kChunk};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP8, int CG>
cudaError_t launch(const CUtensorMap (&maps)[5], const TileParams& p, const TileSources& src, int workers, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&tile_attn_kernel<FP8, CG>),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<FP8, CG>::kAlloc);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(workers * CG);
    cfg.blockDim = dim3(Cfg<FP8, CG>::kThreads);
    cfg.dynamicSmemBytes = Smem<FP8, CG>::kAlloc;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, tile_attn_kernel<FP8, CG>, maps[0], maps[1], maps[2], maps[3], maps[4], p, src);
    // a refused launch is reported through the return value, not left pending
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

}  // namespace

int tile_default_ctas() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return sms;
}

cudaError_t launch_tile_attn(const TileAttnArgs& a, cudaStream_t s) {
    CUtensorMap maps[5];  // K, V, Q, K scales, V scales (the last two e4m3 only)
    memset(maps, 0, sizeof maps);
    const bool pair = a.tile_tokens == kTilePair;
    if (!make_kv_map(&maps[0], a.k_cache, a.fp8, a.num_pages, a.num_kv_heads) ||
        !(a.fp8 && pair ? make_v_half_map(&maps[1], a.v_cache, a.num_pages, a.num_kv_heads)
                        : make_kv_map(&maps[1], a.v_cache, a.fp8, a.num_pages, a.num_kv_heads)) ||
        !make_tile_q_map(&maps[2], a.q, a.num_tokens, a.num_q_heads))
        return cudaErrorInvalidValue;
    if (a.fp8 && (!make_scale_map(&maps[3], a.k_scale, a.num_pages, a.num_kv_heads) ||
                  !make_scale_map(&maps[4], a.v_scale, a.num_pages, a.num_kv_heads)))
        return cudaErrorInvalidValue;
    TileParams p;
    memset(&p, 0, sizeof p);
    p.plan = a.plan;
    p.seqs_off = tile_layout(a.S, a.num_workers).seqs;
    p.page_table = a.page_table;
    p.pt_stride = a.pt_stride;
    p.err = a.plan + kTError;
    p.S = a.S;
    p.mode = a.mode;
    p.q_len = a.q_len;
    p.num_tokens = a.num_tokens;
    p.num_q_heads = a.num_q_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.num_pages = a.num_pages;
    p.split_o = a.split_o;
    p.split_lse = a.split_lse;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.out_lse = a.out_lse;
    const TileSources src{static_cast<const __nv_bfloat16*>(a.q), a.k_cache, a.v_cache, a.k_scale, a.v_scale};
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)kHeadDim);
    if (pair)
        return a.fp8 ? launch<true, 2>(maps, p, src, a.num_workers, s) : launch<false, 2>(maps, p, src, a.num_workers, s);
    return a.fp8 ? launch<true, 1>(maps, p, src, a.num_workers, s) : launch<false, 1>(maps, p, src, a.num_workers, s);
}

}  // namespace hpc
