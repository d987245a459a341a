// Products of 16-bit operands grouped by expert (include/moe_experts16.h): rows times their
// expert's weights, and the two gradients.
//
// A block computes 64 x 64 outputs from 16-deep slices of both operands in shared memory, in fp32.
#include "mxfp4.cuh"
#include "experts16.h"

namespace moe {
namespace {

constexpr int kTile = 64, kDeep = 16, kThreads = 256;

struct Args {
  int R, E, N, D;
  const int32_t* cumsum;
  const void *rows, *rows2, *w;
  void* out;
  int32_t* status;
  bool accumulate;
};

__device__ __forceinline__ int end_of(const Args& a, int e) {
  return e < 0 ? 0 : min(max(__ldcg(a.cumsum + e), 0), a.R);
}

// out[m][n] = sum over k of A(m, k) B(k, n), m < rows, n < cols, k < depth.
template <typename O, typename FA, typename FB>
__device__ __forceinline__ void tile_product(int m0, int n0, int rows, int cols, int depth, FA A, FB B, O* out, int64_t ld,
                                             bool accumulate) {
  __shared__ float sa[kDeep][kTile + 1], sb[kDeep][kTile + 1];
  float acc[4][4] = {};
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  for (int k0 = 0; k0 < depth; k0 += kDeep) {
    for (int i = threadIdx.x; i < kTile * kDeep; i += kThreads) {
      const int k = i % kDeep, r = i / kDeep;
      sa[k][r] = m0 + r < rows && k0 + k < depth ? A(m0 + r, k0 + k) : 0.0f;
      sb[k][r] = n0 + r < cols && k0 + k < depth ? B(k0 + k, n0 + r) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][tm * 4 + i], sb[k][tn * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + tm * 4 + i, n = n0 + tn * 4 + j;
      if (m < rows && n < cols) {
        O* o = out + m * ld + n;
        *o = from_f32<O>(accumulate ? to_f32<O>(*o) + acc[i][j] : acc[i][j]);
      }
    }
}

// blockIdx.x: 64-row tiles, an expert's rounded up (kWeight: channels); blockIdx.y: output columns;
// blockIdx.z: experts (kWeight).
template <typename T, typename O, Gmm16 KIND>
__global__ void __launch_bounds__(kThreads) gmm16_kernel(const Args a) {
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *a.status = 0;
  const T *rows = static_cast<const T*>(a.rows), *rows2 = static_cast<const T*>(a.rows2);
  O* out = static_cast<O*>(a.out);
  const int N = a.N, D = a.D, c0 = blockIdx.y * kTile;
  if constexpr (KIND == Gmm16::kWeight) {
    const int e = blockIdx.z, lo = end_of(a, e - 1), hi = end_of(a, e);
    const T *x = rows + (int64_t)lo * N, *y = rows2 + (int64_t)lo * D;
    tile_product(
        blockIdx.x * kTile, c0, N, D, max(hi - lo, 0), [&](int m, int k) { return to_f32<T>(x[(int64_t)k * N + m]); },
        [&](int k, int n) { return to_f32<T>(y[(int64_t)k * D + n]); }, out + (int64_t)e * N * D, (int64_t)D, a.accumulate);
  } else {
  for (int e = 0, tile = 0; e < a.E; ++e) {
    const int lo = end_of(a, e - 1), hi = end_of(a, e), n = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;
    if ((int)blockIdx.x < tile + n) {
      const int m0 = ((int)blockIdx.x - tile) * kTile;
      const T* w = static_cast<const T*>(a.w) + (int64_t)e * N * D;
      const int depth = KIND == Gmm16::kForward ? D : N, cols = KIND == Gmm16::kForward ? N : D;
      const T* x = rows + (int64_t)lo * depth;
      tile_product(
          m0, c0, hi - lo, cols, depth, [&](int m, int k) { return to_f32<T>(x[(int64_t)m * depth + k]); },
          [&](int k, int n) { return to_f32<T>(KIND == Gmm16::kForward ? w[(int64_t)n * D + k] : w[(int64_t)k * D + n]); },
          out + (int64_t)lo * cols, (int64_t)cols, false);
      return;
    }
    tile += n;
  }
  }
}

template <typename T>
cudaError_t launch(const Gmm16Problem& p, cudaStream_t stream) {
  Args a{p.R, p.E, p.N, p.D, p.cumsum, p.rows, p.rows2, p.w, p.out, p.status, p.accumulate};
  const unsigned tn = (unsigned)(p.N + kTile - 1) / kTile, td = (unsigned)(p.D + kTile - 1) / kTile;
  const unsigned tiles = (unsigned)(p.R / kTile + (p.R < p.E ? p.R : p.E));  // an expert's last tile may be short
  if (p.kind == Gmm16::kForward)
    gmm16_kernel<T, T, Gmm16::kForward><<<dim3(tiles, tn), kThreads, 0, stream>>>(a);
  else if (p.kind == Gmm16::kInput)
    gmm16_kernel<T, T, Gmm16::kInput><<<dim3(tiles, td), kThreads, 0, stream>>>(a);
  else if (p.out_f32)
    gmm16_kernel<T, float, Gmm16::kWeight><<<dim3(tn, td, (unsigned)p.E), kThreads, 0, stream>>>(a);
  else
    gmm16_kernel<T, T, Gmm16::kWeight><<<dim3(tn, td, (unsigned)p.E), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gmm16(const Gmm16Problem& p, cudaStream_t stream) {
  return p.bf16 ? launch<__nv_bfloat16>(p, stream) : launch<__half>(p, stream);
}

}  // namespace moe
