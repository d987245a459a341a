// MXFP4 on the device (include/moe_mxfp4.h): block scales, element conversion, the
// weight-block layout and the typed loads and stores its kernels share.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/moe_mxfp4.h"
#include "common.cuh"
#include "mxfp4.h"

namespace moe {

// Bits of |v|: they order as the magnitudes do, infinities above every finite value and
// NaN above infinities, so an integer maximum also finds a block that is not finite.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Scale byte of a block from the largest abs_bits of its elements: floor(log2 a) - 2 + 127
// is the exponent field less 2, held at 0 (which also covers a = 0 and subnormal a); the
// field 255 of an infinity or NaN stays 255.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t f = amax_bits >> 23;
  return f == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}
// 2^(127 - b), what elements are multiplied with (b <= 252; exact, a normal number);
// 0 for the NaN scale, whose codes are 0.
__device__ __forceinline__ float mx_multiplier(uint32_t b) {
  return b == 255u ? 0.0f : __uint_as_float((254u - b) << 23);
}
// 2^(b - 127): 2^-127 is subnormal, 255 is NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fffffffu : (b ? b << 23 : 0x00400000u));
}

// Eight fp32 -> eight e2m1 codes (element i in nibble i), rounded to nearest even and
// saturated at 6 by the conversion instruction.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight e2m1 codes -> fp32, by the conversion instruction to binary16 (exact).
__device__ __forceinline__ void mx_values8(uint32_t w, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// x * 2^(127 - b) for a block that may hold non-finite values (b = 255 -> 0).
__device__ __forceinline__ float mx_scaled(float x, float mult, uint32_t b) { return b == 255u ? 0.0f : x * mult; }

// Launches a kernel as a programmatic dependent of the one before it in the stream: it may start
// when that one's blocks have all asked for dependents or ended, and has to wait
// (griddepcontrol.wait) before it touches anything that earlier work writes or reads.  What earlier
// kernels may still be writing at its launch it reads past the read-only path, which promises
// nothing for data that changes in a kernel's lifetime.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute after;
  after.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  after.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &after;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Byte offset, in its weight block, of 16-byte chunk c of channel row r, and of its scale.
__device__ __forceinline__ int mx_chunk_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }
__device__ __forceinline__ int mx_scale_at(int r, int c) { return kMxCodeBytes + (c >> 2) * 512 + r * 4 + (c & 3); }

// Channel of W that block nb's row r holds (N channels in all).
__device__ __forceinline__ int mx_channel(int nb, int r, int N, bool gate_up) {
  return gate_up ? ((r >> 5) & 1) * (N >> 1) + nb * 64 + (r >> 6) * 32 + (r & 31) : nb * 128 + r;
}

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
// Two values, the first in the low half where a type has 16 bits.
template <typename T> __device__ __forceinline__ void from_f32x2(float a, float b, T* o);
template <> __device__ __forceinline__ void from_f32x2<float>(float a, float b, float* o) {
  o[0] = a;
  o[1] = b;
}
template <> __device__ __forceinline__ void from_f32x2<__half>(float a, float b, __half* o) {
  *reinterpret_cast<__half2*>(o) = f2h2_sat(a, b);
}
template <> __device__ __forceinline__ void from_f32x2<__nv_bfloat16>(float a, float b, __nv_bfloat16* o) {
  *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(a, b);
}
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __low2half(f2h2_sat(v, v)); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

}  // namespace moe
