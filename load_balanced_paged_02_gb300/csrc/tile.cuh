// Tile maps: the work of prompt attention (hpc_prefill_*) and of shared-prefix
// attention (hpc_prefix_*) as tiles of 32 or 64 query tokens x the 8 query heads
// of one KV head, each over a run of 128-token KV blocks. Layout of the map and
// the walk over it, shared by the planner, the attention kernel and the
// kernels that merge split tiles.
//
// Sequence s (a prompt, or a group of requests behind one prefix) has n query
// tokens and L keys. With T tokens per tile (32: a CTA takes a tile; 64: a pair of
// CTAs does), tile i holds query tokens [T i, min(n, T i + T)) and
//   prompts:  the keys before L - n + min(n, T i + T) (causal: query token t
//             sits at position L - n + t), at least one block, so that rows
//             without a visible key are written too;
//   prefixes: all L keys (no tile where L is 0).
// The walk is KV head by KV head, sequence by sequence, tile by tile, block by
// block; worker j (a CTA or a pair) gets units [j * bucket, (j + 1) * bucket) of
// it, where a tile is
// kTileCost units of fixed cost followed by one unit per block. A
// boundary inside the fixed cost is a boundary before block 0.
#pragma once

#include "hpc_internal.cuh"

namespace hpc {

constexpr int kHalfTokens = 16;                   // query tokens of an MMA's 128 rows
constexpr int kTileCta = 2 * kHalfTokens, kTilePair = 4 * kHalfTokens;
constexpr int kBlock = 128;                       // keys of a block: two pages
// Most keys of a sequence: a tile's limits, up to T past the last key, stay in int32.
constexpr int kMaxKeys = 2147483647 - 255;
constexpr int kModePrefill = 0, kModePrefix = 1;

enum TileHdrSlot {
    kTUnitsPerHead = 0,   // int64
    kTBucket = 2,         // int64
    kTUsedWorkers = 4,
    kTBatch = 5,
    kTNumKvHeads = 6,
    kTNumWorkers = 7,
    kTNumTokens = 8,
    kTMode = 9,
    kTTilesPerHead = 10,
    kTQLen = 11,
    kTError = 12,
    kTTileTokens = 13,
};

// Offsets (int32 units) of the sections of a tile map.
struct TileLayout {
    long long starts, seqs, units, total_ints;
};

__host__ __device__ inline TileLayout tile_layout(long long S, long long C) {
    TileLayout L;
    L.starts = kHdrInts;                      // [C + 1] rows of 8: {kv head, sequence, tile, block} and the sequence's row of seqs
    L.seqs = L.starts + (C + 1) * 8;          // [S] rows of 4: {first query token, n, L, tiles of the sequences before}
    L.units = L.seqs + S * 4;                 // int64 [S + 1]: units of the sequences before
    L.total_ints = L.units + (S + 1) * 2;
    return L;
}

// A tile's start and end in blocks: its query rows, the pipeline's first turn, its output
// rows. Packed prompts of 100 to 6000 tokens: cost 1 1123 us, 2 1100, 3 1109, 4 1121;
// one of 8192 tokens 677, 665, 657, 662; groups of 16, 5, 1 and 42 requests without it
// 121 us, 2 115, 4 116.
constexpr int kTileCost = 2;

__host__ __device__ inline int tile_count(int n, int T) { return (n + T - 1) / T; }

// Blocks of tile i.
__host__ __device__ inline int tile_blocks(int mode, int n, int L, int i, int T) {
    if (mode == kModePrefix) return (int)(((long long)L + kBlock - 1) / kBlock);
    const long long t1 = (long long)T * (i + 1) < n ? (long long)T * (i + 1) : n;
    const long long e = (long long)L - n + t1;  // keys the tile's last query token sees
    return e <= kBlock ? 1 : (int)((e + kBlock - 1) / kBlock);
}

// sum of max(1, floor(m / R)) over m < x, up to a constant
__host__ __device__ inline long long step_sum(long long x, int R) {
    if (x <= 2 * R) return x;
    const long long q = x / R, s = x % R;
    return 2 * R + (R * (q * (q - 1) / 2) + s * q) - R;  // sum of floor(m / R) over 2 R <= m < x, plus 2 R
}

// Units of tiles [0, i) of a sequence, i <= tile_count. Every tile but the last
// has T query tokens, so tile j's last key is at L - n + T (j + 1) and, with R = 128
// / T, it has max(1, floor((a + j) / R)) blocks, a = floor((L - n + T + 127) / T).
__host__ __device__ inline long long tile_units(int mode, int n, int L, int i, int T) {
    if (i <= 0) return 0;
    if (mode == kModePrefix) return (long long)i * (tile_blocks(mode, n, L, 0, T) + kTileCost);
    const int nt = tile_count(n, T);
    const int full = i < nt ? i : nt - 1;
    const long long x = (long long)L - n + T + kBlock - 1;
    const long long a = x >= 0 ? x / T : -((-x + T - 1) / T);
    long long u = step_sum(a + full, kBlock / T) - step_sum(a, kBlock / T) + (long long)i * kTileCost;
    if (i == nt) u += tile_blocks(mode, n, L, nt - 1, T);
    return u;
}

// ----------------------------------------------------------------- launchers

struct TilePlanArgs {
    const int32_t* q_starts;
    const int32_t* lens;
    int S, num_tokens, Hkv, C, min_blocks, max_len, mode, q_len, T;
    int32_t* buf;
};
cudaError_t launch_tile_plan(const TilePlanArgs& a, cudaStream_t s);
// The same and the decode planner's map (launch_plan), in one launch.
cudaError_t launch_both_plans(const TilePlanArgs& a, const int32_t* seq_lens, int B, int Hkv, int C, int m, int32_t* buf,
                              cudaStream_t s);

struct TileAttnArgs {
    const void* q;  // bf16 [num_tokens][Hq][128]
    const void* k_cache;
    const void* v_cache;
    const float* k_scale;
    const float* v_scale;
    int fp8;
    int num_pages;
    const int32_t* page_table;
    int pt_stride;
    int S, num_tokens, num_q_heads, num_kv_heads;
    int32_t* plan;
    int num_workers, mode, tile_tokens, q_len;
    float* split_o;
    float* split_lse;
    void* out;       // prompts only
    float* out_lse;  // prompts only, nullable
};
cudaError_t launch_tile_attn(const TileAttnArgs& a, cudaStream_t s);
int tile_default_ctas();  // SMs of the current device (0: it cannot be asked)

cudaError_t launch_prefill_combine(const int32_t* plan, int S, int num_tokens, int Hq, int C, int T, const float* split_o,
                                   const float* split_lse, void* out, float* out_lse, cudaStream_t s);

cudaError_t launch_prefix_combine(const int32_t* prefix_plan, int S, int prefix_workers, int T, const float* prefix_o,
                                  const float* prefix_lse, const int32_t* plan, int ctas, const float* split_o,
                                  const float* split_lse, __nv_bfloat16* out, float* out_lse, int B, int Hq, int Hkv,
                                  int q_len, cudaStream_t s);

#if defined(__CUDACC__)

// Whether a map in device memory has the sizes that the call describes (another may have
// been planned into its buffer since).
__device__ __forceinline__ bool tile_map_is(const int32_t* plan, int S, int Hkv, int C, int num_tokens, int mode, int q_len,
                                            int T) {
    const int4 a = *reinterpret_cast<const int4*>(plan + 4), b = *reinterpret_cast<const int4*>(plan + 8);
    return a.y == S && a.z == Hkv && a.w == C && b.x == num_tokens && b.y == mode && b.w == q_len &&
           plan[kTTileTokens] == T;
}
static_assert(kTBatch == 5 && kTNumKvHeads == 6 && kTNumWorkers == 7 && kTNumTokens == 8 && kTMode == 9 && kTQLen == 11,
              "header words");

struct TilePos {
    int h, s, i, blk;
};

// One piece of work: blocks [b0, b1) of tile i of sequence s for KV head h.
struct TileItem {
    int h, i, s;
    int q0, n, L;    // the sequence's first query token, its query tokens and keys
    int b0, b1;
    int whole;       // all of the tile's blocks
    int tile;        // number of the tile in the walk
};

// Walks the items of one worker's part of the map.
template <int T>
struct TileWalk {
    int tiles_per_head;
    TilePos at, end;
    int4 q;  // at.s's row of seqs

    __device__ __forceinline__ void start(const int32_t* plan, int worker) {
        const int4* st = reinterpret_cast<const int4*>(plan + kHdrInts + (long long)worker * 8);
        const int4 a = st[0], e = st[2];
        q = st[1];
        at = TilePos{a.x, a.y, a.z, a.w};
        end = TilePos{e.x, e.y, e.z, e.w};
        tiles_per_head = plan[kTTilesPerHead];
    }

    // The next item; false at the end of the worker's part. (What the call knows is given
    // each time, from its parameters, and takes no registers in between.)
    __device__ __forceinline__ bool next(TileItem& it, int S, int mode, const int4* seqs) {
        for (;;) {
            const bool last = at.h == end.h && at.s == end.s && at.i == end.i;
            if (last && at.blk >= end.blk) return false;
            const int blocks = tile_blocks(mode, q.y, q.z, at.i, T);
            it.h = at.h;
            it.s = at.s;
            it.i = at.i;
            it.q0 = q.x;
            it.n = q.y;
            it.L = q.z;
            it.b0 = at.blk;
            it.b1 = last ? end.blk : blocks;
            it.whole = it.b0 == 0 && it.b1 == blocks;
            it.tile = at.h * tiles_per_head + q.w + at.i;
            if (last) {
                at.blk = end.blk;
            } else {
                at.blk = 0;
                if (++at.i >= tile_count(q.y, T)) {
                    at.i = 0;
                    // the next sequence that has tiles (the walk ends at `end`, which
                    // has, or at the head after the last)
                    do {
                        if (++at.s >= S) {
                            at.s = 0;
                            ++at.h;
                        }
                        if (at.h > end.h || (at.h == end.h && at.s > end.s)) {
                            at = end;
                            break;
                        }
                        q = seqs[at.s];
                        if (at.h == end.h && at.s == end.s) break;
                        if (q.y > 0 && (mode == kModePrefill || q.z > 0)) break;
                    } while (true);
                }
            }
            if (it.b1 > it.b0) return true;
        }
    }
};

// Row of the split buffers where a piece of a tile goes, in units of a tile's
// rows. Prompts: only cut tiles have pieces; a worker has at most one that goes on
// from the worker before and one that starts there. Prefixes: every piece; from one
// piece to the next the tile number, the worker number or both grow.
__device__ __forceinline__ long long tile_slot(int mode, int worker, const TileItem& it) {
    return mode == kModePrefill ? 2LL * worker + (it.b0 == 0 ? 1 : 0) : (long long)it.tile + worker;
}

#endif  // __CUDACC__

}  // namespace hpc
