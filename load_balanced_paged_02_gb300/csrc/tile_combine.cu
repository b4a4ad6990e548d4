// Merging the pieces of cut tiles (tile.cuh): partial rows o_i (normalised) with
// natural-log LSEs lse_i give out = sum w_i o_i / sum w_i with
// w_i = exp(lse_i - max), and lse = max + ln sum w_i, as in combine.cu.
//
// prefill_combine_kernel: for every worker whose part of the walk ends inside a
// tile that began there, the tile's pieces from that worker on (at most one per
// worker) into the output rows; whole tiles were written by the attention kernel.
// prefix_combine_kernel: for every (request, new token, query head) the pieces
// of its group's prefix tile and the splits of its own suffix.
// Both: a warp per few rows, lane k owning dims [4 k, 4 k + 4). Bound by the reads
// of the partial rows, mostly from L2 (20 MB of an 8192-token prefix and 64 requests
// in 5.6 us, 3.6 TB/s), and by launch latency and a chain of dependent loads for small
// batches (4.7 us).
#include "tile.cuh"

namespace hpc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 8;
// Rows that a warp merges at once. Prefixes: two (64 requests over an 8192-token prefix
// 5.6 us; four 6.8 us, one 8.3 us: more warps against more loads of the same map). Prompts:
// four, with as many blocks per tile as it has rows for (four short prompts 4.9 us, 6.4 us
// in two turns of half as many; two rows 5.8 us and more).
constexpr int kPromptRows = 4, kPrefixRows = 2;
constexpr int prompt_parts(int T) { return T * kGroup / (kWarps * kPromptRows); }  // blocks per tile

__device__ __forceinline__ void store_row(__nv_bfloat16* out, long long row, int lane, const float4& v) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    uint2 w;
    w.x = *reinterpret_cast<uint32_t*>(&lo);
    w.y = *reinterpret_cast<uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(out + row * kHeadDim + 4 * lane) = w;
}

// Partial rows at equal distances: run.n of them, the first at row run.row of (o,
// lse), run.step rows apart.
struct Run {
    const float* o;
    const float* lse;
    long long row, step;
    int n;
};

// A warp merges two runs into kRows neighbouring rows (query heads of one token): v[r]
// gets dims [4 k, 4 k + 4) of row r (k the lane), lse the LSE of row lane / kBatch. A
// piece without a visible key (LSE -inf) has weight 0 and is not added. The warp holds
// the LSEs of kBatch pieces at once: lane kBatch r + i has piece i of row r.
template <int kRows>
__device__ __forceinline__ void merge_runs(const Run& a, const Run& b, int lane, float4 (&v)[kRows], float& lse) {
    constexpr int kBatch = 32 / kRows;
    static_assert(kGroup % kRows == 0, "rows of one token");
    const int n = a.n + b.n, lr = lane / kBatch, li = lane % kBatch;
    float m = -INFINITY, sum = 0.f;  // of row lr
#pragma unroll
    for (int r = 0; r < kRows; ++r) v[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += kBatch) {
        const int i = i0 + li;
        float l = -INFINITY;
        if (i < a.n)
            l = a.lse[a.row + i * a.step + lr];
        else if (i < n)
            l = b.lse[b.row + (i - a.n) * b.step + lr];
        // the first pieces' rows are on their way while the weights are made
        const int cnt = min(kBatch, n - i0);
        float4 x[2][kRows];
        auto load = [&](int k, float4 (&y)[kRows]) {
            const int j = i0 + k;
            const float* src = j < a.n ? a.o + (a.row + j * a.step) * kHeadDim : b.o + (b.row + (j - a.n) * b.step) * kHeadDim;
#pragma unroll
            for (int r = 0; r < kRows; ++r) y[r] = *reinterpret_cast<const float4*>(src + r * kHeadDim + 4 * lane);
        };
        load(0, x[0]);
        if (cnt > 1) load(1, x[1]);
        // (fmaxf passes a NaN over; its weight stays NaN)
        float M = l;
#pragma unroll
        for (int o = kBatch / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        M = fmaxf(M, m);
        const float old = m == -INFINITY ? 0.f : exp2f((m - M) * kLog2e);  // what the sums so far still weigh
        m = M;
        const float w = l == -INFINITY ? 0.f : exp2f((l - (M == -INFINITY ? 0.f : M)) * kLog2e);
        float ws = w;
#pragma unroll
        for (int o = kBatch / 2; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
        sum = sum * old + ws;
        if (i0 > 0) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float f = __shfl_sync(0xffffffffu, old, r * kBatch);
                v[r].x *= f, v[r].y *= f, v[r].z *= f, v[r].w *= f;
            }
        }
        for (int k = 0; k < cnt; k += 2) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (k + u >= cnt) break;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float f = __shfl_sync(0xffffffffu, w, r * kBatch + k + u);
                    if (f != 0.f) {
                        v[r].x += f * x[u][r].x;
                        v[r].y += f * x[u][r].y;
                        v[r].z += f * x[u][r].z;
                        v[r].w += f * x[u][r].w;
                    }
                }
                if (k + u + 2 < cnt) load(k + u + 2, x[u]);
            }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    lse = sum == 0.f ? -INFINITY : m + logf(sum);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const float f = __shfl_sync(0xffffffffu, inv, r * kBatch);
        v[r] = make_float4(v[r].x * f, v[r].y * f, v[r].z * f, v[r].w * f);
    }
}

// Writes merged rows to output rows orow, orow + 1, ...
template <int kRows>
__device__ __forceinline__ void store_rows(__nv_bfloat16* out, float* out_lse, long long orow, int lane,
                                           const float4 (&v)[kRows], float lse) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) store_row(out, orow + r, lane, v[r]);
    constexpr int kBatch = 32 / kRows;
    if (out_lse && lane % kBatch == 0) out_lse[orow + lane / kBatch] = lse;
}

template <int T>
__global__ void __launch_bounds__(kWarps * 32)
    prefill_combine_kernel(const int32_t* plan, long long seqs_off, long long units_off, int S, int num_tokens, int Hq,
                           const float* split_o, const float* split_lse, __nv_bfloat16* out, float* out_lse) {
    grid_dependency_wait();  // the pieces come from the attention kernel
    grid_launch_dependents();
    const int4* starts = reinterpret_cast<const int4*>(plan + kHdrInts);
    const int j = blockIdx.x;
    if (!tile_map_is(plan, S, Hq / kGroup, gridDim.x, num_tokens, kModePrefill, 1, T)) return;
    const int4 a = starts[2 * j], e = starts[2 * (j + 1)];
    // the tile at the end of worker j's part is cut there, and began in it
    if (e.w == 0) return;
    const bool same = a.x == e.x && a.y == e.y && a.z == e.z;
    if (same && a.w > 0) return;
    const int4 q = reinterpret_cast<const int4*>(plan + seqs_off)[e.y];
    const long long per_head = *reinterpret_cast<const long long*>(plan + kTUnitsPerHead);
    const long long bucket = *reinterpret_cast<const long long*>(plan + kTBucket);
    const long long end = e.x * per_head + reinterpret_cast<const long long*>(plan + units_off)[e.y] +
                          tile_units(kModePrefill, q.y, q.z, e.z + 1, T);
    const int last = (int)((end - 1) / bucket);  // the worker with the tile's last block
    constexpr int kRows = kPromptRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = (blockIdx.y * kWarps + warp) * kRows;
    const int tok = e.z * T + r / kGroup;
    if (tok >= q.y) return;
    // worker j's piece, and one of every worker after it up to the last
    const Run head{split_o, split_lse, (2LL * j + 1) * (T * kGroup) + r, 0, 1};
    const Run rest{split_o, split_lse, (2LL * j + 2) * (T * kGroup) + r, 2LL * T * kGroup, last - j};
    float4 v[kRows];
    float lse;
    merge_runs(head, rest, lane, v, lse);
    store_rows(out, out_lse, (long long)(q.x + tok) * Hq + e.x * kGroup + r % kGroup, lane, v, lse);
}

template <int T>
__global__ void __launch_bounds__(kWarps * 32)
    prefix_combine_kernel(const int32_t* prefix_plan, long long seqs_off, long long units_off, int S, int workers,
                          const float* prefix_o, const float* prefix_lse, const int32_t* pair_nsplit,
                          const int32_t* pair_split0, const float* split_o, const float* split_lse, __nv_bfloat16* out,
                          float* out_lse, int B, int Hq, int Q) {
    grid_dependency_wait();  // the pieces come from the attention kernels
    grid_launch_dependents();
    constexpr int kRows = kPrefixRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long orow = ((long long)blockIdx.x * kWarps + warp) * kRows;  // (request, new token, query head)
    if (orow >= (long long)B * Q * Hq) return;
    const int tok = (int)(orow / Hq), qh = (int)(orow % Hq);
    const int h = qh / kGroup, j = qh % kGroup, b = tok / Q, qi = tok % Q;
    const long long pair = (long long)h * B + b;
    const long long rs = (long long)Q * kGroup;
    const Run own{split_o, split_lse, pair_split0[pair] * rs + qi * kGroup + j, rs, pair_nsplit[pair]};
    Run prefix{prefix_o, prefix_lse, 0, (long long)T * kGroup, 0};
    // the group whose query tokens hold this one: the last that starts at or before it
    const int4* seqs = reinterpret_cast<const int4*>(prefix_plan + seqs_off);
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seqs[mid].x <= tok)
            lo = mid;
        else
            hi = mid;
    }
    const int4 q = seqs[lo];
    if (tok >= q.x && tok < q.x + q.y && q.z > 0 &&
        tile_map_is(prefix_plan, S, Hq / kGroup, workers, B * Q, kModePrefix, Q, T)) {
        const long long per_head = *reinterpret_cast<const long long*>(prefix_plan + kTUnitsPerHead);
        const long long bucket = *reinterpret_cast<const long long*>(prefix_plan + kTBucket);
        const int i = (tok - q.x) / T, r = (tok - q.x) % T * kGroup + j;
        const int blocks = tile_blocks(kModePrefix, q.y, q.z, i, T);
        const long long g0 = h * per_head + reinterpret_cast<const long long*>(prefix_plan + units_off)[lo] +
                             (long long)i * (blocks + kTileCost) + kTileCost;
        const long long tile = (long long)h * prefix_plan[kTTilesPerHead] + q.w + i;
        const long long c0 = g0 / bucket;  // one piece per worker that the tile's blocks touch
        prefix.row = (tile + c0) * (T * kGroup) + r;
        prefix.n = (int)((g0 + blocks - 1) / bucket - c0) + 1;
    }
    float4 v[kRows];
    float lse;
    merge_runs(prefix, own, lane, v, lse);
    store_rows(out, out_lse, orow, lane, v, lse);
}

}  // namespace

cudaError_t launch_prefill_combine(const int32_t* plan, int S, int num_tokens, int Hq, int C, int T, const float* split_o,
                                   const float* split_lse, void* out, float* out_lse, cudaStream_t s) {
    const TileLayout t = tile_layout(S, C);
    return launch_pdl(T == kTilePair ? prefill_combine_kernel<kTilePair> : prefill_combine_kernel<kTileCta>,
                      dim3(C, prompt_parts(T)), dim3(kWarps * 32), 0, s, plan, t.seqs, t.units, S, num_tokens, Hq, split_o,
                      split_lse, static_cast<__nv_bfloat16*>(out), out_lse);
}

cudaError_t launch_prefix_combine(const int32_t* prefix_plan, int S, int prefix_workers, int T, const float* prefix_o,
                                  const float* prefix_lse, const int32_t* plan, int ctas, const float* split_o,
                                  const float* split_lse, __nv_bfloat16* out, float* out_lse, int B, int Hq, int Hkv,
                                  int q_len, cudaStream_t s) {
    const TileLayout t = tile_layout(S, prefix_workers);
    const PlanLayout L = plan_layout(B, Hkv, ctas);
    const long long rows = (long long)B * q_len * Hq;
    const long long blocks = (rows / kPrefixRows + kWarps - 1) / kWarps;
    return launch_pdl(T == kTilePair ? prefix_combine_kernel<kTilePair> : prefix_combine_kernel<kTileCta>,
                      dim3((unsigned)blocks), dim3(kWarps * 32), 0, s, prefix_plan, t.seqs, t.units, S, prefix_workers, prefix_o,
                      prefix_lse, plan + L.pair_nsplit, plan + L.pair_split0, split_o, split_lse, out, out_lse, B, Hq, q_len);
}

}  // namespace hpc
