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

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

}  // namespace hpc
