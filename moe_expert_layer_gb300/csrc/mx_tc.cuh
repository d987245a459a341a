// The block-scaled tcgen05 product of MXFP4 operands: instruction wrappers and the scale
// layout in tensor memory, shared by the grouped product and the few-token layer.
//
//   D[128 x N] (+)= A[128 x 64] * B[N x 64]^T,  every 32 elements of an A or B row scaled
//
// A (weight channels) and B (token rows) lie in shared memory as 128-byte rows of codes
// (256 elements, four MMAs deep) in the 128-byte swizzle.  Their scales lie in tensor
// memory: for 128 elements of depth, the four scale bytes of row r as one 32-bit word in
// lane r % 32, column r / 32, the same in all four 32-lane groups; an MMA uses the low or
// the high half of the words, which its instruction descriptor selects.  Warps write them
// there from registers (tcgen05.st): the words then need no particular order in global or
// shared memory beyond one row after the other.
#pragma once
#include "mxfp4.cuh"
#include "tc_common.cuh"

namespace moe {

// Instruction descriptor of kind::mxf4: A and B e2m1, e8m0 scales, M = 128, N in steps of 8.
__device__ __forceinline__ uint32_t mx_idesc(int n) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | (1u << 27);
}
// The scale halves (0: elements 0-63 of the 128, 1: 64-127) an MMA uses.
__device__ __forceinline__ uint32_t mx_idesc_half(uint32_t half) { return (half * 2u) << 4 | (half * 2u) << 29; }

__device__ __forceinline__ void mx_mma(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` once the MMAs issued so far by this thread have completed.
__device__ __forceinline__ void mx_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

template <int kCols>
__device__ __forceinline__ void tmem_alloc(uint32_t* where) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "n"(kCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int kCols>
__device__ __forceinline__ void tmem_dealloc(uint32_t tmem) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols) : "memory");
}

// Columns from the calling warp's 32 lanes (taddr names them): one register per column.
__device__ __forceinline__ void tmem_st1(uint32_t t, uint32_t a) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(t), "r"(a) : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t t, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The MMAs of one 256-deep stage: `steps` (1..4) of 64 elements.  sfa and sfb are the first
// columns of the stage's scales, a plane of 128 elements every sfa_plane / sfb_plane columns.
__device__ __forceinline__ void mx_mma_stage(uint32_t d, uint32_t a_smem, uint32_t b_smem, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfa_plane, uint32_t sfb, uint32_t sfb_plane, int steps,
                                             uint32_t accumulate) {
  const uint64_t a = sw128_desc(a_smem), b = sw128_desc(b_smem);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < steps)
      mx_mma(d, a + 2 * k, b + 2 * k, idesc | mx_idesc_half(k & 1), sfa + (k >> 1) * sfa_plane,
             sfb + (k >> 1) * sfb_plane, k ? 1u : accumulate);
}

// wait_or_abort by a whole warp: every lane gets the same answer, so that no lane leaves a
// sequence of warp-wide instructions alone.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, status));
}

// silu(g) * u in fp32; the fast exponential and division are a few units off in the last
// place, far inside the 4-bit rounding that follows.
__device__ __forceinline__ float mx_swiglu(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// Eight values of one channel (lane) and eight rows (index) -> the MXFP4 block of 32
// channels of each row.  On return lane l holds row l % 8's code word of channels
// 8 (l / 8) .. + 7, and that row's scale byte.  The block maximum is a warp maximum of the
// magnitudes' bits; the codes, nibble i for row i, are transposed among each eight lanes.
__device__ __forceinline__ uint32_t mx_quant_rows8(float (&h)[8], int lane, uint32_t& byte) {
  byte = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = mx_scale_byte(__reduce_max_sync(0xffffffffu, abs_bits(h[i])));
    h[i] = mx_scaled(h[i], mx_multiplier(b), b);
    if ((lane & 7) == i) byte = b;
  }
  uint32_t w = mx_codes8(h);
#pragma unroll
  for (int d = 4; d; d >>= 1) {  // exchange the d-nibble halves of the words between lanes d apart
    const uint32_t mask = d == 4 ? 0x0000ffffu : d == 2 ? 0x00ff00ffu : 0x0f0f0f0fu;
    const uint32_t o = __shfl_xor_sync(0xffffffffu, w, d);
    w = (lane & d) ? ((o >> (4 * d)) & mask) | (w & ~mask) : (w & mask) | ((o & mask) << (4 * d));
  }
  return w;
}

}  // namespace moe
