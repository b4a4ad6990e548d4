// Merging the pieces of cut tiles (tile.cuh): partial rows o_i (normalised) with
// natural-log LSEs lse_i give out = sum w_i o_i / sum w_i with
// w_i = exp(lse_i - max), and lse = max + ln sum w_i, as in combine.cu.
//
// prefill_combine_kernel: for every worker whose part of the walk ends inside a
// tile that began there, the tile's pieces from that worker on (at most one per
// worker) into the output rows; whole tiles were written by the attention kernel.
// prefix_combine_kernel: for every (request, new token, query head) the pieces
// of its group's prefix tile and the splits of its own suffix.
// Both: a warp per row, lane k owning dims [4 k, 4 k + 4). Bound by the reads of
// the partial rows, mostly from L2, and by launch latency for small batches.
#include "tile.cuh"

namespace hpc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 8;
constexpr int kParts = 8;  // blocks per tile

__device__ __forceinline__ void store_row(__nv_bfloat16* out, long long row, int lane, const float4& v) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    uint2 w;
    w.x = *reinterpret_cast<uint32_t*>(&lo);
    w.y = *reinterpret_cast<uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(out + row * kHeadDim + 4 * lane) = w;
}

// Running merge of partial rows.
struct Merge {
    float m = -INFINITY, w = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);

    __device__ __forceinline__ void add(float lse, const float4& o) {
        if (lse == -INFINITY) return;  // a piece without a visible key
        const float M = fmaxf(m, lse);
        const float a = m == -INFINITY ? 0.f : exp2f((m - M) * kLog2e), b = exp2f((lse - M) * kLog2e);
        m = M;
        w = w * a + b;
        acc.x = acc.x * a + o.x * b;
        acc.y = acc.y * a + o.y * b;
        acc.z = acc.z * a + o.z * b;
        acc.w = acc.w * a + o.w * b;
    }
    __device__ __forceinline__ float lse() const { return w == 0.f ? -INFINITY : m + logf(w); }
    __device__ __forceinline__ float4 row() const {
        const float inv = w == 0.f ? 0.f : 1.f / w;
        return make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
};

__global__ void __launch_bounds__(kWarps * 32)
    prefill_combine_kernel(const int32_t* plan, long long seqs_off, int Hq, int C, int T,
                           const float* split_o, const float* split_lse,
                           __nv_bfloat16* out, float* out_lse) {
    grid_dependency_wait();  // the pieces come from the attention kernel
    grid_launch_dependents();
    const int4* starts = reinterpret_cast<const int4*>(plan + kHdrInts);
    const int j = blockIdx.x;
    const int4 a = starts[2 * j], e = starts[2 * (j + 1)];
    // the tile at the end of worker j's part is cut there, and began in it
    if (e.w == 0) return;
    const bool same = a.x == e.x && a.y == e.y && a.z == e.z;
    if (same && a.w > 0) return;
    int pieces = 2;  // worker j's and the next ones', until one reaches the tile's end
    for (int k = j + 1; k < C; ++k) {
        const int4 f = starts[2 * (k + 1)];
        if (!(f.x == e.x && f.y == e.y && f.z == e.z && f.w > 0)) break;
        ++pieces;
    }
    const int4 q = reinterpret_cast<const int4*>(plan + seqs_off)[e.y];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = blockIdx.y * kWarps + warp; r < T * kGroup; r += kParts * kWarps) {
        const int tok = e.z * T + r / kGroup;
        if (tok >= q.y) break;
        Merge mg;
        for (int u = 0; u < pieces; ++u) {
            const long long row = (u == 0 ? 2LL * j + 1 : 2LL * (j + u)) * (T * kGroup) + r;
            mg.add(split_lse[row], *reinterpret_cast<const float4*>(split_o + row * kHeadDim + 4 * lane));
        }
        const long long orow = (long long)(q.x + tok) * Hq + e.x * kGroup + r % kGroup;
        store_row(out, orow, lane, mg.row());
        if (out_lse && lane == 0) out_lse[orow] = mg.lse();
    }
}

__global__ void __launch_bounds__(kWarps * 32)
    prefix_combine_kernel(const int32_t* prefix_plan, long long seqs_off, long long units_off, int S, int T,
                          const float* prefix_o, const float* prefix_lse,
                          const int32_t* pair_nsplit, const int32_t* pair_split0,
                          const float* split_o, const float* split_lse,
                          __nv_bfloat16* out, float* out_lse, int B, int Hq, int Q) {
    grid_dependency_wait();  // the pieces come from the attention kernels
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long orow = (long long)blockIdx.x * kWarps + warp;  // (request, new token, query head)
    if (orow >= (long long)B * Q * Hq) return;
    const int tok = (int)(orow / Hq), qh = (int)(orow % Hq);
    const int h = qh / kGroup, j = qh % kGroup, b = tok / Q, qi = tok % Q;
    Merge mg;
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
    if (tok >= q.x && tok < q.x + q.y && q.z > 0) {
        const long long* units = reinterpret_cast<const long long*>(prefix_plan + units_off);
        const long long per_head = *reinterpret_cast<const long long*>(prefix_plan + kTUnitsPerHead);
        const long long bucket = *reinterpret_cast<const long long*>(prefix_plan + kTBucket);
        const int i = (tok - q.x) / T, r = (tok - q.x) % T * kGroup + j;
        const int blocks = tile_blocks(kModePrefix, q.y, q.z, i, T);
        const long long g0 = h * per_head + units[lo] + (long long)i * blocks;
        const long long tile = (long long)h * prefix_plan[kTTilesPerHead] + q.w + i;
        for (long long c = g0 / bucket; c <= (g0 + blocks - 1) / bucket; ++c) {
            const long long row = (tile + c) * (T * kGroup) + r;
            mg.add(prefix_lse[row], *reinterpret_cast<const float4*>(prefix_o + row * kHeadDim + 4 * lane));
        }
    }
    const long long pair = (long long)h * B + b;
    const int n = pair_nsplit[pair];
    const long long s0 = pair_split0[pair];
    for (int u = 0; u < n; ++u) {
        const long long row = ((s0 + u) * Q + qi) * kGroup + j;
        mg.add(split_lse[row], *reinterpret_cast<const float4*>(split_o + row * kHeadDim + 4 * lane));
    }
    store_row(out, orow, lane, mg.row());
    if (out_lse && lane == 0) out_lse[orow] = mg.lse();
}

}  // namespace

cudaError_t launch_prefill_combine(const int32_t* plan, int S, int Hq, int C, int T, const float* split_o,
                                   const float* split_lse, void* out, float* out_lse, cudaStream_t s) {
    return launch_pdl(prefill_combine_kernel, dim3(C, kParts), dim3(kWarps * 32), 0, s, plan, tile_layout(S, C).seqs, Hq, C, T,
                      split_o, split_lse, static_cast<__nv_bfloat16*>(out), out_lse);
}

cudaError_t launch_prefix_combine(const int32_t* prefix_plan, int S, int prefix_workers, int T, const float* prefix_o,
                                  const float* prefix_lse, const int32_t* plan, int ctas, const float* split_o,
                                  const float* split_lse, __nv_bfloat16* out, float* out_lse, int B, int Hq, int Hkv,
                                  int q_len, cudaStream_t s) {
    const TileLayout t = tile_layout(S, prefix_workers);
    const PlanLayout L = plan_layout(B, Hkv, ctas);
    const long long blocks = ((long long)B * q_len * Hq + kWarps - 1) / kWarps;
    return launch_pdl(prefix_combine_kernel, dim3((unsigned)blocks), dim3(kWarps * 32), 0, s, prefix_plan, t.seqs, t.units,
                      S, T, prefix_o, prefix_lse, plan + L.pair_nsplit, plan + L.pair_split0, split_o, split_lse, out, out_lse,
                      B, Hq, q_len);
}

}  // namespace hpc
