// Planner of tile maps (integer only, one block): sequence table and unit
// prefix sums by block scans, then every worker's start by a binary search over
// the sequences and one over the tiles of the sequence found, whose unit sums
// have a closed form (tile_units). The same load balancing as the decode
// planner's (equal runs of one walk over all KV heads), with tiles of a prompt
// in place of requests.
//
// A block of 1024 threads runs tile_plan_block: alone (tile_plan.cu), or beside the
// decode planner's blocks (plan.cu). Bound by latency: 3.5 us for a prefix, 4.5 us for
// 4 to 60 prompts, launch included (7 us with the tile size as a variable, whose closed
// forms then divide in 64 bits, and a scan for each of the two sums).
#pragma once

#include "tile.cuh"

namespace hpc {
namespace tileplan {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Exclusive scans of two values over the block; the totals receive the sums. All
// threads call it.
__device__ __forceinline__ void scan_exclusive(long long& v, int& w, long long& v_total, int& w_total, long long* v_sums,
                                               int* w_sums) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    long long x = v;
    int y = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, x, o);
        const int b = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) x += a, y += b;
    }
    if (lane == 31) v_sums[wp] = x, w_sums[wp] = y;
    __syncthreads();
    if (wp == 0) {
        long long c = v_sums[lane];
        int d = w_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long a = __shfl_up_sync(0xffffffffu, c, o);
            const int b = __shfl_up_sync(0xffffffffu, d, o);
            if (lane >= o) c += a, d += b;
        }
        v_sums[lane] = c, w_sums[lane] = d;
    }
    __syncthreads();
    v = x - v + (wp > 0 ? v_sums[wp - 1] : 0);
    w = y - w + (wp > 0 ? w_sums[wp - 1] : 0);
    v_total = v_sums[kWarps - 1];
    w_total = w_sums[kWarps - 1];
    __syncthreads();
}

// Exclusive running maximum of values >= 0 over the block; the total receives the maximum.
// All threads call it.
__device__ __forceinline__ int max_exclusive(int v, int& total, int* sums) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = max(x, a);
    }
    if (lane == 31) sums[wp] = x;
    __syncthreads();
    int before = 0;  // of the warps before, and of the lanes before
    total = 0;
    for (int k = 0; k < kWarps; ++k) {
        total = max(total, sums[k]);
        if (k == wp - 1) before = total;
    }
    const int left = __shfl_up_sync(0xffffffffu, x, 1);
    __syncthreads();
    return lane > 0 ? max(before, left) : before;
}

// T is a constant here, so that the closed forms of tile_units divide by shifts.
template <int T>
__device__ __forceinline__ void tile_plan_block(const TilePlanArgs& a) {
    __shared__ long long unit_sums[kWarps];
    __shared__ int tile_sums[kWarps];
    __shared__ int err_sh;
    const int32_t* const q_starts = a.q_starts;
    const int32_t* const lens = a.lens;
    const int S = a.S, num_tokens = a.num_tokens, Hkv = a.Hkv, C = a.C, min_blocks = a.min_blocks, max_len = a.max_len,
              mode = a.mode, q_len = a.q_len;
    int32_t* const buf = a.buf;
    const TileLayout lay = tile_layout(S, C);
    int4* seqs = reinterpret_cast<int4*>(buf + lay.seqs);
    long long* units = reinterpret_cast<long long*>(buf + lay.units);
    if (threadIdx.x == 0) err_sh = 0;  // (the loop's first barrier comes before any use)
    long long unit_base = 0;
    int tile_base = 0;
    int err = 0;
    // A query row belongs to one sequence: split rows are counted on that. While no sequence's
    // starts decrease or leave the range, every sequence begins where the one before ends; from
    // the first one that does, each has to begin at or past the ends of all before it.
    bool apart = true;
    int ends = 0;  // the largest end so far of a sequence whose starts are in order (kept once !apart)
    for (int s0 = 0; s0 < S; s0 += kThreads) {
        const int s = s0 + threadIdx.x;
        int q0 = 0, n = 0, L = 0;
        bool fits = true;
        if (s < S) {
            const long long a = (long long)q_starts[s] * q_len, b = (long long)q_starts[s + 1] * q_len;
            L = lens[s];
            if (L < 0) {
                err |= (int)HPC_DEVERR_NEGATIVE_LENGTH;
                L = 0;
            }
            if (L > max_len) {  // no page ids beyond the table's row
                err |= (int)HPC_DEVERR_PAGE_OUT_OF_RANGE;
                L = max_len;
            }
            fits = a >= 0 && b >= a && b <= num_tokens;
            if (fits) {
                q0 = (int)a;
                n = (int)(b - a);
            }
        }
        if (__syncthreads_or(!fits) && apart) {
            apart = false;
            ends = s0 > 0 ? q_starts[s0] * q_len : 0;  // (in range: all before were in order)
        }
        if (!apart) {
            int most;
            const int before = max(ends, max_exclusive(fits ? q0 + n : 0, most, tile_sums));
            ends = max(ends, most);
            if (s < S && (!fits || q0 < before)) {
                err |= (int)HPC_DEVERR_BAD_DESCRIPTOR;
                q0 = before;  // first rows never fall: prefix_combine_kernel searches them
                n = 0;
            }
        }
        const bool any = n > 0 && (mode == kModePrefill || L > 0);
        const int tiles = any ? tile_count(n, T) : 0;
        long long u = any ? tile_units(mode, n, L, tiles, T) : 0, u_total;
        int t = tiles, t_total;
        scan_exclusive(u, t, u_total, t_total, unit_sums, tile_sums);
        if (s < S) {
            seqs[s] = make_int4(q0, n, L, tile_base + t);
            units[s] = unit_base + u;
        }
        unit_base += u_total;
        tile_base += t_total;
    }
    if (err) atomicOr(&err_sh, err);
    if (threadIdx.x == 0) units[S] = unit_base;
    __syncthreads();
    const long long per_head = unit_base, total = per_head * Hkv;
    const long long floor_units = min_blocks > 0 ? min_blocks : 1;
    long long bucket = (total + C - 1) / C;
    if (bucket < floor_units) bucket = floor_units;
    if (threadIdx.x < kHdrInts) {
        const int used = (int)((total + bucket - 1) / bucket);
        int v = 0;
        switch (threadIdx.x) {
            case kTUnitsPerHead: v = (int)(per_head & 0xffffffffLL); break;
            case kTUnitsPerHead + 1: v = (int)(per_head >> 32); break;
            case kTBucket: v = (int)(bucket & 0xffffffffLL); break;
            case kTBucket + 1: v = (int)(bucket >> 32); break;
            case kTUsedWorkers: v = used; break;
            case kTBatch: v = S; break;
            case kTNumKvHeads: v = Hkv; break;
            case kTNumWorkers: v = C; break;
            case kTNumTokens: v = num_tokens; break;
            case kTMode: v = mode; break;
            case kTTilesPerHead: v = tile_base; break;
            case kTQLen: v = q_len; break;
            case kTError: v = err_sh; break;
            case kTTileTokens: v = T; break;
        }
        buf[threadIdx.x] = v;
    }
    for (int j = threadIdx.x; j <= C; j += kThreads) {
        const long long g = (long long)j * bucket;
        int4 a = make_int4(Hkv, 0, 0, 0), b = make_int4(0, 0, 0, 0);
        if (g < total) {
            const int h = (int)(g / per_head);
            const long long r = g - h * per_head;
            int lo = 0, hi = S;  // the last sequence with units[s] <= r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (units[mid] <= r)
                    lo = mid;
                else
                    hi = mid;
            }
            const int4 q = seqs[lo];
            const long long u = r - units[lo];
            int i0 = 0, i1 = tile_count(q.y, T);  // the last tile with tile_units <= u
            while (i1 - i0 > 1) {
                const int mid = (i0 + i1) >> 1;
                if (tile_units(mode, q.y, q.z, mid, T) <= u)
                    i0 = mid;
                else
                    i1 = mid;
            }
            const long long blk = u - tile_units(mode, q.y, q.z, i0, T) - kTileCost;
            a = make_int4(h, lo, i0, blk > 0 ? (int)blk : 0);
            b = q;
        }
        int4* st = reinterpret_cast<int4*>(buf + lay.starts) + 2 * j;
        st[0] = a;
        st[1] = b;
    }
}

}  // namespace tileplan
}  // namespace hpc
