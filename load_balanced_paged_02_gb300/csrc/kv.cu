// The paged cache written and read back outside the fused prologue.
//
// hpc_kv_write: K and V rows (bf16, any token stride) into the slots the mapping
// names, as bf16 or as e4m3 codes with one float32 scale per (token, KV head):
// scale = amax / 448 (1 if all are 0), code = rne(x / scale), the rule of the
// prologue. hpc_kv_read: tokens of each request, packed, as bf16; e4m3 values
// are code x scale in float32, rounded once.
//
// Both are streams, bound by HBM for long calls and by launch latency for a decode
// step's. A block takes a run of tokens (16 at most, fewer while that leaves SMs
// without blocks) with all their heads of K and V; groups of lanes take one row of
// 128 elements each, 16 bytes per lane and load, and kUnroll rows are loaded before
// the first is used. Blocks of 16 tokens measured best (155k tokens at 8 heads, e4m3
// read: 64 tokens 170 us, 32 161 us, 16 156 us).
#include "kv.cuh"
#include "tile.cuh"

namespace hpc {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;         // rows that a reading group of lanes loads at once
constexpr int kWriteRows = 2;      // and a writing one
constexpr int kMaxTokens = 16;     // tokens of a block at most
constexpr int kSmemStarts = 1025;  // out_starts kept in shared memory up to this many
constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ void unpack8(const uint4& r, float (&y)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        y[2 * k] = __uint_as_float(w[k] << 16);
        y[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint2 pack_e4m3x8(const float (&y)[8]) {
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        c[k] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * k], y[2 * k + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Eight lanes per row (lane k: elements [16 k, 16 k + 16)); row r of the block is
// token r / (2 Hkv), K heads before V heads. Fewer lanes per row share its index
// arithmetic, scale and maximum: sixteen took 15.9 us for 8192 tokens at 8 heads.
template <bool FP8>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteArgs a, int tokens_per_block) {
    constexpr int kLanes = 8, kGroups = kThreads / kLanes;
    grid_dependency_wait();  // the projection may still be finishing
    grid_launch_dependents();
    const int hl = threadIdx.x % kLanes;
    const unsigned mask = 0xffu << (threadIdx.x & 24);
    const int t0 = blockIdx.x * tokens_per_block, nt = min(tokens_per_block, a.num_tokens - t0);
    const unsigned per_token = 2u * (unsigned)a.num_kv_heads, rows = (unsigned)nt * per_token;
    for (unsigned r0 = threadIdx.x / kLanes; r0 < rows; r0 += kGroups * kWriteRows) {
        uint4 raw[kWriteRows][2];
        int slot[kWriteRows], kvh[kWriteRows];
#pragma unroll
        for (int u = 0; u < kWriteRows; ++u) {
            const unsigned r = r0 + u * kGroups;
            slot[u] = -1;
            kvh[u] = 0;
            if (r < rows) {
                const unsigned tl = r / per_token;
                const int t = t0 + (int)tl;
                kvh[u] = (int)(r - tl * per_token);
                slot[u] = a.slots[t];
                const bool is_v = kvh[u] >= a.num_kv_heads;
                const __nv_bfloat16* src = is_v ? a.v + t * a.v_stride + (kvh[u] - a.num_kv_heads) * kHeadDim
                                                : a.k + t * a.k_stride + kvh[u] * kHeadDim;
                raw[u][0] = reinterpret_cast<const uint4*>(src)[2 * hl];
                raw[u][1] = reinterpret_cast<const uint4*>(src)[2 * hl + 1];
            }
        }
#pragma unroll
        for (int u = 0; u < kWriteRows; ++u) {
            if (slot[u] < 0) continue;  // padding (or no row): uniform over the row's lanes
            const int page = slot[u] / kChunk, off = slot[u] % kChunk;
            if (page >= a.num_pages) {
                if (hl == 0 && a.err) atomicOr(a.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
                continue;
            }
            const bool is_v = kvh[u] >= a.num_kv_heads;
            const int h = is_v ? kvh[u] - a.num_kv_heads : kvh[u];
            void* cache = is_v ? a.v_cache : a.k_cache;
            const long long dst = ((long long)slot[u] * a.num_kv_heads + h) * kHeadDim + 16 * hl;
            if constexpr (!FP8) {
                uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + dst);
                out[0] = raw[u][0];
                out[1] = raw[u][1];
            } else {
                float y[2][8];
                unpack8(raw[u][0], y[0]);
                unpack8(raw[u][1], y[1]);
                float am = fmaxf(fabsf(y[0][0]), fabsf(y[1][0]));
#pragma unroll
                for (int k = 1; k < 8; ++k) am = max3(am, fabsf(y[0][k]), fabsf(y[1][k]));
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(mask, am, o));
                float scale = __fdiv_rn(am, kE4m3Max);
                if (!(scale > 0.f)) scale = 1.f;
                // x / scale, correctly rounded, by Markstein's correction step (IBM J. Res. Dev.
                // 34(1), 1990): y = RN(1 / scale), q = RN(x y), r = RN(x - q scale), RN(q + r y).
                // His theorem asks for a q within one ulp. That may be missed here (1.4 ulp), but
                // while nothing leaves the normal range the answer is one of 128 x 128, for the
                // significands of the row's largest element and of x, and all of them are the
                // rounded quotients (checked one by one in the tests). From 1e-24 on the residual of
                // a quotient that has a code above zero (2^-11 and more) is no subnormal number.
                if (scale >= 1e-24f && scale <= 1e30f) {
                    const float inv = __frcp_rn(scale);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float x = y[k >> 3][k & 7], q = x * inv;
                        y[k >> 3][k & 7] = fmaf(fmaf(-q, scale, x), inv, q);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) y[k >> 3][k & 7] = __fdiv_rn(y[k >> 3][k & 7], scale);
                }
                const uint2 lo = pack_e4m3x8(y[0]), hi = pack_e4m3x8(y[1]);
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(cache) + dst) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                if (hl == 0)
                    (is_v ? a.v_scale : a.k_scale)[((long long)page * a.num_kv_heads + h) * kChunk + off] = scale;
            }
        }
    }
}

// First the block's tokens, one per thread: the request by a search in out_starts,
// then the page. Then 16 lanes (bf16) or 8 (e4m3, 16 codes each) per row.
template <bool FP8>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadArgs a, int tokens_per_block) {
    __shared__ int starts[kSmemStarts];
    __shared__ int src_sh[kMaxTokens];  // page * 64 + slot; -1: no valid page (zeros); -2: no request's row
    grid_dependency_wait();             // the cache may still be being written
    grid_launch_dependents();
    const bool in_smem = a.batch + 1 <= kSmemStarts;
    if (in_smem) {
        for (int i = threadIdx.x; i <= a.batch; i += kThreads) starts[i] = a.out_starts[i];
        __syncthreads();
    }
    const int* st = in_smem ? starts : a.out_starts;
    const int t0 = blockIdx.x * tokens_per_block, nt = min(tokens_per_block, a.num_rows - t0);
    if ((int)threadIdx.x < nt) {
        const int tok = t0 + threadIdx.x;
        int lo = 0, hi = a.batch;  // the last request that starts at or before the row
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (st[mid] <= tok)
                lo = mid;
            else
                hi = mid;
        }
        int src = -2;
        if (tok >= st[lo] && tok < st[lo + 1]) {
            src = -1;
            const long long pos = (long long)tok - st[lo] + (a.first ? a.first[lo] : 0);
            int page = -1;
            if (pos >= 0 && pos / kChunk < a.pt_stride) page = a.page_table[(long long)lo * a.pt_stride + pos / kChunk];
            if ((unsigned)page < (unsigned)a.num_pages)
                src = page * kChunk + (int)(pos % kChunk);
            else if (a.err)
                atomicOr(a.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
        }
        src_sh[threadIdx.x] = src;
    }
    __syncthreads();
    constexpr int kLanes = FP8 ? 8 : 16;
    const int hl = threadIdx.x % kLanes;
    const unsigned per_token = 2u * (unsigned)a.num_kv_heads, rows = (unsigned)nt * per_token;
    for (unsigned r0 = threadIdx.x / kLanes; r0 < rows; r0 += kThreads / kLanes * kUnroll) {
        uint4 raw[kUnroll];
        float scale[kUnroll];
        long long dst[kUnroll];  // element of k_out or v_out; -1: nothing to write
        bool is_v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const unsigned r = r0 + u * (kThreads / kLanes);
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            scale[u] = 0.f;
            dst[u] = -1;
            is_v[u] = false;
            if (r >= rows) continue;
            const unsigned tl = r / per_token;
            const int kvh = (int)(r - tl * per_token);
            const int src = src_sh[tl];
            is_v[u] = kvh >= a.num_kv_heads;
            const int h = is_v[u] ? kvh - a.num_kv_heads : kvh;
            if (src == -2) continue;
            dst[u] = ((long long)(t0 + (int)tl) * a.num_kv_heads + h) * kHeadDim + hl * (kHeadDim / kLanes);
            if (src < 0) continue;
            const long long at = ((long long)src * a.num_kv_heads + h) * kHeadDim + hl * (kHeadDim / kLanes);
            const void* cache = is_v[u] ? a.v_cache : a.k_cache;
            if constexpr (FP8) {
                raw[u] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(cache) + at);
                scale[u] = (is_v[u] ? a.v_scale : a.k_scale)[((long long)(src / kChunk) * a.num_kv_heads + h) * kChunk + src % kChunk];
            } else {
                raw[u] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(cache) + at);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (dst[u] < 0) continue;
            uint4* out = reinterpret_cast<uint4*>((is_v[u] ? a.v_out : a.k_out) + dst[u]);
            if constexpr (FP8) {
                const uint32_t c[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t f[2];
                    e4m3x4_to_f16x2x2(c[k], f[0], f[1]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f[j]));
                        w[2 * k + j] = pack_bf16x2(x.x * scale[u], x.y * scale[u]);
                    }
                }
                out[0] = make_uint4(w[0], w[1], w[2], w[3]);
                out[1] = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
                out[0] = raw[u];
            }
        }
    }
}

// Tokens of a block: as many as leave four blocks per SM, at most kMaxTokens.
int tokens_per_block(int tokens) {
    const int blocks = 4 * tile_default_ctas();
    int n = kMaxTokens;
    while (n > 1 && (tokens + n - 1) / n < blocks) n >>= 1;
    return n;
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, bool fp8, cudaStream_t s) {
    const int n = tokens_per_block(a.num_tokens);
    const dim3 grid((a.num_tokens + n - 1) / n);
    return fp8 ? launch_pdl(kv_write_kernel<true>, grid, dim3(kThreads), 0, s, a, n)
               : launch_pdl(kv_write_kernel<false>, grid, dim3(kThreads), 0, s, a, n);
}

cudaError_t launch_kv_read(const KvReadArgs& a, bool fp8, cudaStream_t s) {
    const int n = tokens_per_block(a.num_rows);
    const dim3 grid((a.num_rows + n - 1) / n);
    return fp8 ? launch_pdl(kv_read_kernel<true>, grid, dim3(kThreads), 0, s, a, n)
               : launch_pdl(kv_read_kernel<false>, grid, dim3(kThreads), 0, s, a, n);
}

}  // namespace hpc
