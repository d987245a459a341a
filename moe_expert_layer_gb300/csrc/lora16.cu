// Low-rank adapters of many requests beside a shared projection (include/moe_experts16.h).
//
// Two kernels over the tokens sorted by adapter: v = a[l] x[t] (fp32), then out = base + s b[l] v.
#include "mxfp4.cuh"
#include "experts16.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// The adapter of sorted position i, or -1.
__device__ __forceinline__ int adapter_at(const int32_t* cumsum, int L, int i) {
  if (i >= __ldcg(cumsum + L - 1)) return -1;
  int lo = 0, hi = L - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (i < __ldcg(cumsum + mid)) hi = mid; else lo = mid + 1;
  }
  return lo;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) lora16_shrink_kernel(const Lora16Problem p) {
  const int i = blockIdx.x, t = __ldcg(p.route + i), l = adapter_at(p.cumsum, p.L, i);
  if (l < 0 || (unsigned)t >= (unsigned)p.M) return;
  const T* x = static_cast<const T*>(p.x) + (int64_t)t * p.D;
  for (int r = threadIdx.x / 32; r < p.rank; r += kThreads / 32) {
    const T* a = static_cast<const T*>(p.a) + ((int64_t)l * p.rank + r) * p.D;
    float s = 0.0f;
    for (int k = threadIdx.x % 32; k < p.D; k += 32) s = fmaf(to_f32<T>(x[k]), to_f32<T>(a[k]), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x % 32 == 0) p.v[(int64_t)i * p.rank + r] = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) lora16_expand_kernel(const Lora16Problem p) {
  const int i = blockIdx.x, t = __ldcg(p.route + i), l = adapter_at(p.cumsum, p.L, i);
  if ((unsigned)t >= (unsigned)p.M) return;
  const float scale = l >= 0 && p.scales ? p.scales[l] : 1.0f;
  for (int n = threadIdx.x; n < p.N; n += kThreads) {
    float s = 0.0f;
    if (l >= 0) {
      const T* b = static_cast<const T*>(p.b) + ((int64_t)l * p.N + n) * p.rank;
      for (int r = 0; r < p.rank; ++r) s = fmaf(p.v[(int64_t)i * p.rank + r], to_f32<T>(b[r]), s);
    }
    const int64_t at = (int64_t)t * p.N + n;
    const float y = to_f32<T>(static_cast<const T*>(p.base)[at]);
    static_cast<T*>(p.out)[at] = from_f32<T>(l >= 0 ? fmaf(scale, s, y) : y);
  }
}

}  // namespace

size_t lora16_workspace_bytes(int M, int D, int rank) { return (size_t)M * rank * 4; }

cudaError_t launch_lora16(const Lora16Problem& p, cudaStream_t stream) {
  if (p.bf16) {
    lora16_shrink_kernel<__nv_bfloat16><<<p.M, kThreads, 0, stream>>>(p);
    lora16_expand_kernel<__nv_bfloat16><<<p.M, kThreads, 0, stream>>>(p);
  } else {
    lora16_shrink_kernel<__half><<<p.M, kThreads, 0, stream>>>(p);
    lora16_expand_kernel<__half><<<p.M, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace moe
