// Top-k router (moe_route_topk in include/moe_mxfp4.h): one warp per token, reading its logits
// once.
//
// Lane l holds the keys of the V consecutive experts l * V .. + V - 1, mapped to unsigned
// integers in the floats' order, and the two largest of those not yet chosen.  A selection is
// one warp maximum (redux.sync) of the lanes' largest and the lowest lane that has it: equal
// keys go to the lower expert because lanes and registers are in the experts' order.  Only that
// lane goes on to its second largest, and looks through its keys again when both are spent.
// Each slot's logit is read back from its key.  Where the weights need no sum over the row
// (sigmoid, or softmax made to sum to one over the chosen, which cancels it) only the chosen
// logits go through exp, one to a lane.
// Bound by the integer and comparison pipe (77% busy): 65521 x 256 fp32 logits, 8 chosen, 39 us,
// of which reading them would take 10 (with a search through a lane's keys after each of its
// selections 58 us; with 64-bit keys through shuffles and every logit's exp 140 us).  One row: 2.7
// us between launches as programmatic dependents, 4.1 in order.
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr float kLargest = 3.402823466e38f;

// Order-preserving map of a float (no NaN) to unsigned; -0 as +0.  kNone: that of -infinity, the
// least; a key that is gone is 0.
constexpr uint32_t kNone = 0x007fffffu;
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_order_bits(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct RouteArgs {
  int M, E, topK, score;
  int64_t stride;
  const float* bias;
  bool renormalise;
  float scale;
  int32_t* expert_idx;
  float* probs;
};

// Lane's V logits, masked ones (NaN too) -infinity, +infinity the largest finite value.
template <typename T, int V, bool VEC>
__device__ __forceinline__ void load_logits(const T* row, int E, int lane, float (&l)[V]) {
  if (VEC) {
    constexpr int kBytes = V * sizeof(T);  // 4, 8 or a multiple of 16 per lane
    union {
      T t[V];
      uint32_t u1;
      uint2 u2;
      uint4 u4[kBytes >= 16 ? kBytes / 16 : 1];
    } r;
    const bool in = lane * V < E;  // E is a multiple of V
    if (in) {
      const T* p = row + lane * V;
      if (kBytes == 4) {
        r.u1 = __ldcg(reinterpret_cast<const uint32_t*>(p));
      } else if (kBytes == 8) {
        r.u2 = __ldcg(reinterpret_cast<const uint2*>(p));
      } else {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) r.u4[i] = __ldcg(reinterpret_cast<const uint4*>(p) + i);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = in ? to_f32<T>(r.t[i]) : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = lane * V + i < E ? to_f32<T>(row[lane * V + i]) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = l[i] != l[i] ? -INFINITY : fminf(l[i], kLargest);
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// ALL: every expert's p is needed (a bias on the keys, or softmax weights as they are).
template <typename T, int V, bool VEC, bool ALL>
__global__ void __launch_bounds__(32 * kWarps) route_topk_kernel(const T* logits, const RouteArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.M) return;
  const T* row = logits + (int64_t)t * a.stride;
  float l[V];
  load_logits<T, V, VEC>(row, a.E, lane, l);
  uint32_t key[V];
  float row_top = 0.0f, row_sum = 1.0f;  // of the row's softmax, where it is needed
  if (ALL && a.score == MOE_SCORE_SOFTMAX) {
    row_top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) row_top = fmaxf(row_top, l[i]);
    row_top = warp_max(row_top);
    row_sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) row_sum += l[i] == -INFINITY ? 0.0f : expf(l[i] - row_top);
    row_sum = warp_sum(row_sum);
  }
  // a chosen or keyed expert's p, where ALL
  auto score = [&](float v) { return a.score == MOE_SCORE_SOFTMAX ? expf(v - row_top) / row_sum : sigmoid(v); };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = order_bits(l[i]);
    if (ALL && a.bias && key[i] != kNone) key[i] = order_bits(score(l[i]) + __ldcg(a.bias + lane * V + i));
  }
  // the lane's two largest keys, the first of equals first
  uint32_t best, second;
  uint32_t gone = 0;
  int at, at2;
  bool two;
  auto scan = [&]() {
    best = second = 0;
    at = at2 = 0;
    two = true;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t k = key[i];
      if (k > best) {
        second = best;
        at2 = at;
        best = k;
        at = i;
      } else if (k > second) {
        second = k;
        at2 = i;
      }
    }
  };
  scan();
  const int64_t out = (int64_t)t * a.topK;
  float total = 0.0f, top = 0.0f;  // sum of the chosen p; the largest chosen logit
  // 32 slots at a time: lane s keeps slot s
  for (int j0 = 0; j0 < a.topK; j0 += 32) {
    int mine = -1;
    uint32_t mine_key = 0;
    const int n = min(32, a.topK - j0);
    for (int s = 0; s < n; ++s) {
      const uint32_t win = __reduce_max_sync(0xffffffffu, best);
      if (win <= kNone) break;  // nothing is left
      const int who = __ffs(__ballot_sync(0xffffffffu, best == win)) - 1;
      const int e = __shfl_sync(0xffffffffu, lane * V + at, who);
      if (lane == s) {
        mine = e;
        mine_key = win;
      }
      bool spent = false;
      if (lane == who) {
        gone |= 1u << at;
        best = second;
        at = at2;
        spent = !two;
        two = false;
      }
      if (__any_sync(0xffffffffu, spent)) {
        if (spent) {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if ((gone >> i) & 1u) key[i] = 0;
          scan();
        }
        __syncwarp();
      }
    }
    float val = mine < 0 ? 0.0f : of_order_bits(mine_key), p = 0.0f;
    if (ALL && a.bias && mine >= 0) val = fminf(to_f32<T>(row[mine]), kLargest);  // the key was not the logit
    if (!ALL && j0 == 0) top = __shfl_sync(0xffffffffu, val, 0);
    if (mine >= 0) p = ALL ? score(val) : a.score == MOE_SCORE_SOFTMAX ? expf(val - top) : sigmoid(val);
    if (a.renormalise) total += warp_sum(p);
    if (lane < n) {
      a.expert_idx[out + j0 + lane] = mine;
      // final unless the sum has more slots to come
      a.probs[out + j0 + lane] =
          !a.renormalise || a.topK > 32 ? p * a.scale : total > 0.0f ? p / total * a.scale : 0.0f;
    }
  }
  if (a.renormalise && a.topK > 32) {
    __syncwarp();
    for (int j = lane; j < a.topK; j += 32) {
      float* q = a.probs + out + j;
      *q = total > 0.0f ? *q / total : 0.0f;
    }
  }
}

template <typename T, int V>
cudaError_t launch(const void* logits, const RouteArgs& a, cudaStream_t stream) {
  const int blocks = (a.M + kWarps - 1) / kWarps;
  const T* x = static_cast<const T*>(logits);
  // a lane's logits as whole vectors: every row aligned to them, and none across the row's end
  constexpr int kAlign = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
  const bool vec = kAlign >= 4 && a.stride * sizeof(T) % kAlign == 0 && a.E % V == 0;
  const bool all = a.bias || (a.score == MOE_SCORE_SOFTMAX && !a.renormalise);
  auto* kernel = vec ? (all ? route_topk_kernel<T, V, (kAlign >= 4), true> : route_topk_kernel<T, V, (kAlign >= 4), false>)
                     : (all ? route_topk_kernel<T, V, false, true> : route_topk_kernel<T, V, false, false>);
  return launch_dependent(kernel, (unsigned)blocks, 32 * kWarps, 0, stream, x, a);
}

template <typename T>
cudaError_t launch_type(const void* logits, const RouteArgs& a, cudaStream_t stream) {
  if (a.E <= 64) return launch<T, 2>(logits, a, stream);
  if (a.E <= 128) return launch<T, 4>(logits, a, stream);
  if (a.E <= 256) return launch<T, 8>(logits, a, stream);
  return launch<T, 32>(logits, a, stream);
}

}  // namespace

cudaError_t launch_route_topk(int M, int E, int topK, const void* logits, int type, int64_t stride, const float* bias,
                              int score, bool renormalise, float scale, int32_t* expert_idx, float* probs,
                              cudaStream_t stream) {
  RouteArgs a;
  a.M = M;
  a.E = E;
  a.topK = topK;
  a.score = score;
  a.stride = stride;
  a.bias = bias;
  a.renormalise = renormalise;
  a.scale = scale;
  a.expert_idx = expert_idx;
  a.probs = probs;
  switch (type) {
    case MOE_TYPE_F32: return launch_type<float>(logits, a, stream);
    case MOE_TYPE_F16: return launch_type<__half>(logits, a, stream);
    default: return launch_type<__nv_bfloat16>(logits, a, stream);
  }
}

}  // namespace moe
