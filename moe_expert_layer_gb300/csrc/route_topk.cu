// Top-k router (moe_route_topk in include/moe_mxfp4.h): one warp per token.
//
// The row's logits stay in the lanes' registers (element e in lane e % 32), so the row is
// read once.  The softmax needs the row maximum and the sum of exponentials, two warp
// reductions; a selection is one warp maximum of (key, lowest expert), packed in 64 bits
// so that a single integer comparison orders both.
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

// Order-preserving map of a float (no NaN) to unsigned.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 -> +0: equal keys tie
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint64_t warp_max_u64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, int V>
__global__ void route_topk_kernel(int M, int E, int topK, const T* logits, int64_t stride, const float* bias, int score,
                                  bool renormalise, float scale, int32_t* expert_idx, float* probs) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= M) return;
  const T* row = logits + (int64_t)t * stride;
  constexpr float kMax = 3.402823466e38f;
  float l[V];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    const float v = e < E ? to_f32<T>(row[e]) : -INFINITY;
    l[i] = v != v ? -INFINITY : fminf(v, kMax);
    top = fmaxf(top, l[i]);
  }
  top = warp_max(top);
  float p[V];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (score == MOE_SCORE_SOFTMAX) {
      p[i] = l[i] == -INFINITY ? 0.0f : expf(l[i] - top);
      sum += p[i];
    } else {
      p[i] = l[i] == -INFINITY ? 0.0f : 1.0f / (1.0f + expf(-l[i]));
    }
  }
  const float total = score == MOE_SCORE_SOFTMAX ? warp_sum(sum) : 1.0f;
  uint64_t key[V];  // 0: not to be chosen
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    if (total > 0.0f) p[i] = p[i] / total;
    const float k = bias && e < E ? p[i] + bias[e] : l[i];
    key[i] = l[i] == -INFINITY ? 0ull : ((uint64_t)order_bits(k) << 32) | (uint32_t)(1024 - e);
  }
  float chosen = 0.0f;
  for (int j = 0; j < topK; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = key[i] > best ? key[i] : best;
    best = warp_max_u64(best);
    const int e = best ? 1024 - (int)(uint32_t)best : -1;
    float pe = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (best && key[i] == best) {
        pe = p[i];
        key[i] = 0;
      }
    pe = warp_sum(pe);  // one lane has it
    chosen += pe;
    if (lane == 0) {
      expert_idx[(int64_t)t * topK + j] = e;
      probs[(int64_t)t * topK + j] = pe * scale;
    }
  }
  if (renormalise) {
    __syncwarp();
    for (int j = lane; j < topK; j += 32) {
      float* q = probs + (int64_t)t * topK + j;
      *q = chosen > 0.0f ? *q / chosen : 0.0f;
    }
  }
}

template <typename T>
cudaError_t launch(int M, int E, int topK, const void* logits, int64_t stride, const float* bias, int score,
                   bool renormalise, float scale, int32_t* expert_idx, float* probs, cudaStream_t stream) {
  const int blocks = (M + kWarps - 1) / kWarps;
  const T* x = static_cast<const T*>(logits);
  if (E <= 256)
    route_topk_kernel<T, 8><<<blocks, 32 * kWarps, 0, stream>>>(M, E, topK, x, stride, bias, score, renormalise, scale,
                                                                expert_idx, probs);
  else
    route_topk_kernel<T, 32><<<blocks, 32 * kWarps, 0, stream>>>(M, E, topK, x, stride, bias, score, renormalise, scale,
                                                                 expert_idx, probs);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_topk(int M, int E, int topK, const void* logits, int type, int64_t stride, const float* bias,
                              int score, bool renormalise, float scale, int32_t* expert_idx, float* probs,
                              cudaStream_t stream) {
  switch (type) {
    case MOE_TYPE_F32:
      return launch<float>(M, E, topK, logits, stride, bias, score, renormalise, scale, expert_idx, probs, stream);
    case MOE_TYPE_F16:
      return launch<__half>(M, E, topK, logits, stride, bias, score, renormalise, scale, expert_idx, probs, stream);
    default:
      return launch<__nv_bfloat16>(M, E, topK, logits, stride, bias, score, renormalise, scale, expert_idx, probs,
                                   stream);
  }
}

}  // namespace moe
