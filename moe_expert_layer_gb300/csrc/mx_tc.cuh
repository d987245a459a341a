// The block-scaled tcgen05 product of MXFP4 operands: instruction wrappers and the scale
// layout in tensor memory, shared by the grouped product and the few-token layer.
//
//   D[128 x N] (+)= A[128 x 64] * B[N x 64]^T,  every 32 elements of an A or B row scaled
//
// A (weight channels) and B (token rows) lie in shared memory as 128-byte rows of codes
// (256 elements, four MMAs deep) in the 128-byte swizzle.  Their scales lie in tensor
// memory: for 128 elements of depth, the four scale bytes of row r as one 32-bit word in
// lane r % 32, column r / 32, the same in all four 32-lane groups; an MMA uses the low or
// the high half of the words, which its instruction descriptor selects.  In global memory
// and as copied the words stand one row after the other.  The grouped product's warps load them
// from shared memory and store them to tensor memory, each to its 32 lanes; the few-token layer's
// put the 512 bytes of 128 rows into the order of the lanes in place, and tcgen05.cp, issued
// before the MMAs that use them by the same thread, copies them on.
#pragma once
#include "mxfp4.cuh"
#include "tc_common.cuh"

namespace moe {

// Instruction descriptor of kind::mxf4: A and B e2m1, e8m0 scales, M = 128 (a CTA; N in steps
// of 16) or 256 (a pair; N in steps of 32).
__device__ __forceinline__ uint32_t mx_idesc(int m, int n) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27);
}
// The scale half (0: elements 0-63 of the 128, 1: 64-127) an MMA uses.
__device__ __forceinline__ uint32_t mx_idesc_half(uint32_t half) { return (half * 2u) << 4 | (half * 2u) << 29; }

// The warp's number in its CTA, in a form the compiler knows to be the same in all lanes:
// branches on it are uniform.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

// One lane of a converged warp: nonzero there, zero in the others.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(r));
  return r;
}

// MMAs, commits and copies are issued by a whole warp in uniform control flow, each
// instruction predicated on the elected lane, and not by one lane in a branch of its own: the
// operands then stay in uniform registers.  An MMA of 256 x 64 x 64 cost 123 cycles issued by
// a lone lane and 55 this way, one of 256 x 224 x 64 its 112 cycles of tensor-core time
// instead of 147.
//
// PAIR: the MMA of a CTA pair.  Each CTA holds its 128 rows of A and their scales, half of
// B's rows, the scales of all of them, and gets its 128 rows of D.
template <bool PAIR>
__device__ __forceinline__ void mx_mma(uint32_t elected, uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "setp.ne.u32 e, %7, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "setp.ne.u32 e, %7, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(elected)
        : "memory");
}
// Arrive on `bar` (of both CTAs of a pair) once the MMAs issued so far by this thread have
// completed.
template <bool PAIR>
__device__ __forceinline__ void mx_commit(uint32_t elected, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.u32 e, %2, 0;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            bar),
        "h"((uint16_t)3), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.u32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(elected)
        : "memory");
}

// The same on a barrier of this CTA alone.
template <bool PAIR>
__device__ __forceinline__ void mx_commit_local(uint32_t elected, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.u32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(elected)
        : "memory");
  else
    mx_commit<false>(elected, bar);
}

// The copies of common.cuh and the expectation of their bytes, predicated the same way;
// shared-memory operands as addresses.
__device__ __forceinline__ void expect_tx_elect(uint32_t elected, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.u32 e, %2, 0;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void bulk_load_elect(uint32_t elected, uint32_t dst, const void* src, uint32_t bytes,
                                                uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.u32 e, %4, 0;\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_elect(uint32_t elected, uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                                  uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.u32 e, %5, 0;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void tma_gather4_elect(uint32_t elected, uint32_t dst, const void* tmap, int32_t x, int4 y,
                                                  uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.u32 e, %8, 0;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(bar), "r"(elected)
      : "memory");
}
// Orders generic accesses of global memory before and after this point with TMA's.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// A ring of n slots: the current one and the parity of its current use.
struct RingPos {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

template <bool PAIR, int kCols>
__device__ __forceinline__ void tmem_alloc(uint32_t* where) {
  if (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "n"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "n"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <bool PAIR, int kCols>
__device__ __forceinline__ void tmem_dealloc(uint32_t tmem) {
  if (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols) : "memory");
}

// The words of 128 rows at `tile`, read by all lanes (rows l, l + 32, l + 64, l + 96 to lane l),
// and written back as row r's word at byte (r % 32) * 16 + (r / 32) * 4: no bank conflicts either
// way.  Between the two the warp synchronises.
__device__ __forceinline__ uint4 mx_scale_words(const uint8_t* tile, int lane) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(tile) + lane;
  return make_uint4(p[0], p[32], p[64], p[96]);
}
__device__ __forceinline__ void mx_put_scale_words(uint8_t* tile, uint4 w, int lane) {
  reinterpret_cast<uint4*>(tile)[lane] = w;
}

// Eight tensor-memory columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, uint4 a, uint4 b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(a.x), "r"(a.y),
               "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// 512 bytes of arranged scale words -> four tensor-memory columns, in each of the four lane
// groups.
__device__ __forceinline__ void mx_copy_scales(uint32_t elected, uint32_t taddr, uint32_t saddr) {
  // unswizzled: groups of 8 rows of 16 bytes, 128 bytes apart
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.u32 e, %2, 0;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
      "l"(desc), "r"(elected)
      : "memory");
}

// Two MMAs: 128 elements of depth, `half` (0, 1) of a 256-deep stage.
template <bool PAIR>
__device__ __forceinline__ void mx_mma2(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, int half, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  mx_mma<PAIR>(elected, d, a + 4 * half, b + 4 * half, idesc, sfa, sfb, accumulate);
  mx_mma<PAIR>(elected, d, a + 4 * half + 2, b + 4 * half + 2, idesc | mx_idesc_half(1), sfa, sfb, 1u);
}

// wait_or_abort by a whole warp: every lane gets the same answer, so that no lane leaves a
// sequence of warp-wide instructions alone.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, status));
}

// Whether a barrier's phase is complete, without waiting.
__device__ __forceinline__ uint32_t mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok;
}

// h = silu(g) * u of eight channels in fp32; the fast exponential's relative error grows with |g|,
// about 2^-22 |g|, and the division adds 2^-22: far inside the 4-bit rounding that follows.  Below
// -80 the 1 is lost beside exp(-g), and before that leaves fp32 (the division gives 0 past 2^126)
// the power is taken in halves around u, which may be large: right down to -174, where e^(g/2)
// ends.  One look at all eight costs less than one at each (layer at prefill: 13 us).
__device__ __forceinline__ void mx_swiglu8(const float (&g)[8], const float (&u)[8], float (&h)[8]) {
  float least = g[0];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    least = fminf(least, g[i]);
    h[i] = __fdividef(g[i], 1.0f + __expf(-g[i])) * u[i];
  }
  if (least < -80.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float half = __expf(0.5f * g[i]);
      if (g[i] < -80.0f) h[i] = (u[i] * half) * (g[i] * half);
    }
  }
}

// Eight values of a scaled block that four neighbouring lanes hold -> their code word and the
// block's scale byte.  A whole warp enters.
__device__ __forceinline__ uint32_t mx_quant_group8(float (&h)[8], uint32_t& byte) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, abs_bits(h[i]));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
  byte = mx_scale_byte(a);
  const float mult = mx_multiplier(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] *= mult;
  const uint32_t w = mx_codes8(h);
  return byte == 255u ? 0u : w;
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
