// tcgen05 wrappers shared by the kernels on the fifth-generation tensor cores
// (attn_tc.cu, tile_attn.cu): descriptors, MMAs into TMEM accumulators, commits
// and fences.
#pragma once

#include "hpc_internal.cuh"

namespace hpc {

// Shared-memory matrix descriptor, 128-byte swizzle (rows of 128 B, 8-row
// atoms of 1024 B): start address, leading / stride byte offsets, the sm_100
// descriptor version (bit 46) and the swizzle mode (2 = 128B, bits 61-63).
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor of kind::f16: f32 accumulator, A and B both f16
// (f16 = true) or both bf16, M x N, A K-major, B K-major (b_mn = 0) or
// MN-major (b_mn = 1).
__host__ __device__ constexpr uint32_t idesc_16bit(bool f16, int M, int N, int b_mn) {
    return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
static_assert(idesc_16bit(false, 64, 64, 0) == ((1u << 4) | (1u << 7) | (1u << 10) | (8u << 17) | (4u << 24)),
              "bf16 descriptor");
static_assert(idesc_16bit(true, 64, 128, 1) == ((1u << 4) | (1u << 16) | (16u << 17) | (4u << 24)),
              "f16 descriptor");

// D (TMEM) (+)= A . B^T from shared-memory descriptors; the operand type
// comes from the instruction descriptor.
__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Instruction descriptor of kind::f8f6f4 with e4m3 A and B (format 0), f32
// accumulator, M x N, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D (TMEM) (+)= A . B^T, e4m3 operands from shared-memory descriptors (32
// elements of K per instruction).
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Arrives on bar once every MMA this thread issued before it has completed.
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// The same three for a whole warp with equal operands, of which the elected lane (el)
// issues: the operands stay in uniform registers (an `if (lane == 0)` around the forms
// above moves them there for every instruction).
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e;
}
__device__ __forceinline__ void umma_f16_el(uint32_t el, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
        : "memory");
}
__device__ __forceinline__ void umma_e4m3_el(uint32_t el, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
        : "memory");
}
__device__ __forceinline__ void umma_commit_el(uint32_t el, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(el)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Eight floats (exact multiples of the row scale's inverse, |x| <= 448) ->
// eight e4m3 "hi" codes (round to nearest even) and eight "lo" codes of the
// remainders x - hi. A bf16 value has eight significant bits; rounding it to
// e4m3's four leaves a remainder of at most four, so hi + lo is x exactly
// unless the remainder falls below e4m3's smallest subnormal (2^-9), i.e. for
// |x| < 2^-2 (elements under 2^-11 of the row maximum). Byte i of the
// outputs holds element i.
__device__ __forceinline__ void split_e4m3x8(const float (&x)[8], uint2& hi, uint2& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_fp8x2_storage_t hc =
            __nv_cvt_float2_to_fp8x2(make_float2(x[2 * j], x[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(hc, __NV_E4M3);
        const float2 hv = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        const __nv_fp8x2_storage_t lc = __nv_cvt_float2_to_fp8x2(
            make_float2(x[2 * j] - hv.x, x[2 * j + 1] - hv.y), __NV_SATFINITE, __NV_E4M3);
        h[j] = hc;
        l[j] = lc;
    }
    hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}

// The power of two 2^ex that a query row of largest magnitude amax is divided by before it is
// split, the smallest with amax / 2^ex <= 448 = 1.75 2^8 (q / 2^ex is exact then), and its
// inverse. Both stay finite: ex is -126 at least, where rows under 2^-117 begin to lose bits
// (half a code's step of 2^-9, 2^-136 an element). An infinite element makes the row's scores
// infinite or NaN.
__device__ __forceinline__ void query_row_scale(float amax, float& scale, float& inverse) {
    const uint32_t ab = __float_as_uint(amax);
    const int ex = max((int)(ab >> 23) - 127 - 8 + ((ab & 0x7fffffu) > 0x600000u ? 1 : 0), -126);
    scale = inverse = 1.f;
    if (amax > 3.4e38f) {
        scale = amax;
    } else if (amax > 0.f) {
        scale = __uint_as_float((uint32_t)(127 + ex) << 23);
        inverse = __uint_as_float((uint32_t)(127 - ex) << 23);
    }
}

// Row r of a tile of bf16 queries in shared memory ([2 dim halves][64 rows][128 B], swizzled)
// into hi and lo e4m3 tiles ([64 rows][128 B] each) in its place, by two lanes: half hh reads
// dims [64 hh, 64 hh + 64), which sit where row r of the hi tile (hh = 0) or of the lo tile
// goes, and writes the hi and lo codes of its dims once both have read. A row that is not `in`
// is zeros; `write` says whether codes are stored. Returns the row's scale.
__device__ __forceinline__ float split_query_row(uint8_t* tile, int r, int hh, bool in, bool write) {
    constexpr int kHalf = 64 * 128;
    uint4 raw[8];
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        raw[c] = in ? *reinterpret_cast<const uint4*>(tile + hh * kHalf + r * 128 + ((c ^ (r & 7)) << 4)) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    __syncwarp();  // the partner lane has read its half row
    float scale, inverse;
    query_row_scale(amax, scale, inverse);
#pragma unroll
    for (int c2 = 0; c2 < 4; ++c2) {
        // bf16 pieces c = 2 c2 + u (dims 64 hh + 8 c ...) -> bytes 8 u of the e4m3 row's
        // 16-byte piece 4 hh + c2
        uint2 hp[2], lp[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint4 x4 = raw[2 * c2 + u];
            const uint32_t w[4] = {x4.x, x4.y, x4.z, x4.w};
            float y[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[2 * j] = __uint_as_float(w[j] << 16) * inverse;
                y[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * inverse;
            }
            split_e4m3x8(y, hp[u], lp[u]);
        }
        if (write) {
            const int off = r * 128 + (((4 * hh + c2) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(tile + off) = make_uint4(hp[0].x, hp[0].y, hp[1].x, hp[1].y);
            *reinterpret_cast<uint4*>(tile + kHalf + off) = make_uint4(lp[0].x, lp[0].y, lp[1].x, lp[1].y);
        }
    }
    __syncwarp();
    return scale;
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

}  // namespace hpc
