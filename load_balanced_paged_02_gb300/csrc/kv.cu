// The paged cache written and read back outside the fused prologue.
//
// hpc_kv_write: K and V rows (bf16, any token stride) into the slots the mapping
// names, as bf16 or as e4m3 codes with one float32 scale per (token, KV head):
// scale = amax / 448 (1 if all are 0), code = rne(x / scale), the rule of the
// prologue. hpc_kv_read: tokens of each request, packed, as bf16; e4m3 values
// are code x scale in float32, rounded once.
//
// Both are streams: a half-warp per (token, head) row, K or V, 16 bytes of bf16
// per lane (a 256-byte row in one access of the half-warp), kRows rows per
// half-warp loaded before any is used. Bound by HBM for long calls, by launch
// latency for a decode step's.
#include "kv.cuh"

namespace hpc {
namespace {

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;
constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ void unpack8(const uint4& r, float (&y)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        y[2 * k] = __uint_as_float(w[k] << 16);
        y[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint2 pack_e4m3x8(const float (&y)[8]) {
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        c[k] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * k], y[2 * k + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Row index -> (token, K or V, head): heads fastest, so that a token's slot is
// read by neighbouring half-warps and its K rows are contiguous.
template <bool FP8, int ROWS>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteArgs a) {
    grid_dependency_wait();  // the projection may still be finishing
    grid_launch_dependents();
    const int hl = threadIdx.x & 15;
    const unsigned mask = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
    const long long rows = (long long)a.num_tokens * 2 * a.num_kv_heads;
    const long long first = ((long long)blockIdx.x * kHalfWarps + (threadIdx.x >> 4)) * ROWS;
    uint4 raw[ROWS];
    int slot[ROWS], kvh[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const long long r = first + u;
        slot[u] = -1;
        kvh[u] = 0;
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
            const int t = (int)(r / (2 * a.num_kv_heads));
            kvh[u] = (int)(r % (2 * a.num_kv_heads));
            slot[u] = a.slots[t];
            const bool is_v = kvh[u] >= a.num_kv_heads;
            const __nv_bfloat16* src = is_v ? a.v + (long long)t * a.v_stride + (long long)(kvh[u] - a.num_kv_heads) * kHeadDim
                                            : a.k + (long long)t * a.k_stride + (long long)kvh[u] * kHeadDim;
            raw[u] = reinterpret_cast<const uint4*>(src)[hl];
        }
    }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        if (slot[u] < 0) continue;  // padding (or no row): uniform over the half-warp
        if (slot[u] / kChunk >= a.num_pages) {
            if (hl == 0 && a.err) atomicOr(a.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
            continue;
        }
        const bool is_v = kvh[u] >= a.num_kv_heads;
        const int h = is_v ? kvh[u] - a.num_kv_heads : kvh[u];
        void* cache = is_v ? a.v_cache : a.k_cache;
        const long long dst = ((long long)slot[u] * a.num_kv_heads + h) * kHeadDim + 8 * hl;
        if constexpr (!FP8) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + dst) = raw[u];
        } else {
            float y[8];
            unpack8(raw[u], y);
            float am = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) am = fmaxf(am, fabsf(y[k]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(mask, am, o));
            float scale = __fdiv_rn(am, kE4m3Max);
            if (!(scale > 0.f)) scale = 1.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __fdiv_rn(y[k], scale);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + dst) = pack_e4m3x8(y);
            if (hl == 0)
                (is_v ? a.v_scale : a.k_scale)[((long long)(slot[u] / kChunk) * a.num_kv_heads + h) * kChunk + slot[u] % kChunk] =
                    scale;
        }
    }
}

// One block per (64-row piece of a request's output, ...): see launch_kv_read.
template <bool FP8, int ROWS>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadArgs a) {
    grid_dependency_wait();  // the cache may still be being written
    grid_launch_dependents();
    const int hl = threadIdx.x & 15;
    const long long rows = (long long)a.num_rows * 2 * a.num_kv_heads;
    const long long first = ((long long)blockIdx.x * kHalfWarps + (threadIdx.x >> 4)) * ROWS;
    if (first >= rows) return;
    // request of the first row's token: the last one that starts at or before it
    int tok = (int)(first / (2 * a.num_kv_heads)), b = 0;
    {
        int lo = 0, hi = a.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.out_starts[mid] <= tok)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
    }
    int bs = a.out_starts[b], be = a.out_starts[b + 1];
    long long src[ROWS];
    int kvh[ROWS], trow[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const long long r = first + u;
        trow[u] = -1;
        src[u] = -1;
        kvh[u] = 0;
        if (r >= rows) continue;
        tok = (int)(r / (2 * a.num_kv_heads));
        kvh[u] = (int)(r % (2 * a.num_kv_heads));
        while (tok >= be && b + 1 < a.batch) {
            ++b;
            bs = be;
            be = a.out_starts[b + 1];
        }
        if (tok < bs || tok >= be) continue;  // a row of no request: left as it is
        trow[u] = tok;
        const long long pos = (long long)tok - bs + (a.first ? a.first[b] : 0);
        int page = -1;
        if (pos >= 0 && pos / kChunk < a.pt_stride) page = a.page_table[(long long)b * a.pt_stride + pos / kChunk];
        if ((unsigned)page < (unsigned)a.num_pages)
            src[u] = (long long)page * kChunk + pos % kChunk;
        else if (hl == 0 && a.err)
            atomicOr(a.err, (int)HPC_DEVERR_PAGE_OUT_OF_RANGE);
    }
    uint4 raw[ROWS];
    float scale[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        raw[u] = make_uint4(0u, 0u, 0u, 0u);  // tokens without a valid page read as zeros
        scale[u] = 0.f;
        if (src[u] < 0) continue;
        const bool is_v = kvh[u] >= a.num_kv_heads;
        const int h = is_v ? kvh[u] - a.num_kv_heads : kvh[u];
        const long long at = (src[u] * a.num_kv_heads + h) * kHeadDim + 8 * hl;
        if constexpr (FP8) {
            const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(is_v ? a.v_cache : a.k_cache) + at);
            raw[u].x = c.x;
            raw[u].y = c.y;
            scale[u] = (is_v ? a.v_scale : a.k_scale)[(src[u] / kChunk * a.num_kv_heads + h) * kChunk + src[u] % kChunk];
        } else {
            raw[u] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(is_v ? a.v_cache : a.k_cache) + at);
        }
    }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        if (trow[u] < 0) continue;
        const bool is_v = kvh[u] >= a.num_kv_heads;
        const int h = is_v ? kvh[u] - a.num_kv_heads : kvh[u];
        uint4 o = raw[u];
        if constexpr (FP8) {
            uint32_t f[4];
            e4m3x4_to_f16x2x2(raw[u].x, f[0], f[1]);
            e4m3x4_to_f16x2x2(raw[u].y, f[2], f[3]);
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f[k]));
                w[k] = pack_bf16x2(x.x * scale[u], x.y * scale[u]);
            }
            o = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __nv_bfloat16* dst = (is_v ? a.v_out : a.k_out) + ((long long)trow[u] * a.num_kv_heads + h) * kHeadDim + 8 * hl;
        *reinterpret_cast<uint4*>(dst) = o;
    }
}

constexpr int kRowsMany = 4;

template <typename K1, typename K4, typename A>
cudaError_t launch_rows(K1 one, K4 many, long long rows, const A& a, cudaStream_t s) {
    // a row per half-warp while that leaves the GPU's blocks unfilled, else several
    const bool few = rows <= 152LL * 8 * kHalfWarps;
    const int per = few ? 1 : kRowsMany;
    const long long blocks = (rows + (long long)kHalfWarps * per - 1) / ((long long)kHalfWarps * per);
    return few ? launch_pdl(one, dim3((unsigned)blocks), dim3(kThreads), 0, s, a)
               : launch_pdl(many, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, bool fp8, cudaStream_t s) {
    const long long rows = (long long)a.num_tokens * 2 * a.num_kv_heads;
    return fp8 ? launch_rows(kv_write_kernel<true, 1>, kv_write_kernel<true, kRowsMany>, rows, a, s)
               : launch_rows(kv_write_kernel<false, 1>, kv_write_kernel<false, kRowsMany>, rows, a, s);
}

cudaError_t launch_kv_read(const KvReadArgs& a, bool fp8, cudaStream_t s) {
    const long long rows = (long long)a.num_rows * 2 * a.num_kv_heads;
    return fp8 ? launch_rows(kv_read_kernel<true, 1>, kv_read_kernel<true, kRowsMany>, rows, a, s)
               : launch_rows(kv_read_kernel<false, 1>, kv_read_kernel<false, kRowsMany>, rows, a, s);
}

}  // namespace hpc
