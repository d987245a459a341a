// Row operators of the 16-bit experts (include/moe_experts16.h): SwiGLU and its gradient, the
// dispatch of tokens to expert-major rows, the weighted combine, and the combine's gradient.
//
// All are bound by bytes: eight elements (16 bytes) to a lane, arithmetic in fp32, one rounding at
// the store.  Measured (bfloat16; GB/s over the bytes that each call reads and writes):
//   SwiGLU, 48169 rows x 1408           64 us  6360      its gradient                      102 us  6650
//   dispatch, 8192 x 4096 to six rows   72 us  6420      combine                            75 us  6260
//   combine's gradient                 138 us  6230
#include "mxfp4.cuh"
#include "experts16.h"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Eight 16-bit elements.
template <typename T>
union Eight {
  T t[8];
  uint4 u;
};
template <typename T>
__device__ __forceinline__ void load8(const T* p, Eight<T>& r) {
  r.u = __ldcg(reinterpret_cast<const uint4*>(p));
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  Eight<T> r;
#pragma unroll
  for (int i = 0; i < 8; i += 2) from_f32x2<T>(v[i], v[i + 1], &r.t[i]);
  *reinterpret_cast<uint4*>(p) = r.u;
}

// Rows that belong to an expert.
__device__ __forceinline__ int valid_rows(const int32_t* cumsum, int E, int R) {
  return min(max(__ldcg(cumsum + E - 1), 0), R);
}

// g s(g) with s(g) = 1 / (1 + exp(-g)), and s(g).  The exponential's relative error is about
// 2^-22 |g|.  Below -80, where 1 is lost beside exp(-g) and before that leaves fp32, s is e^g taken
// as a product of halves around the other factors (`half` = e^(g/2), 0 elsewhere).
struct Gate {
  float s, half;
};
__device__ __forceinline__ Gate gate_of(float g) {
  Gate r;
  r.s = __fdividef(1.0f, 1.0f + __expf(-g));
  r.half = 0.0f;
  if (g < -80.0f) r.half = __expf(0.5f * g);
  return r;
}
__device__ __forceinline__ float swiglu(float g, float u, const Gate& k) {
  return g < -80.0f ? (u * k.half) * (g * k.half) : g * k.s * u;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) swiglu16_kernel(int R, int E, int I, const T* gu, const int32_t* cumsum,
                                                            T* h) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per = I / 8;
  const int64_t n = (int64_t)valid_rows(cumsum, E, R) * per, step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
    const int64_t d = i / per;
    const T* row = gu + d * 2 * I + (i - d * per) * 8;
    Eight<T> g, u;
    load8(row, g);
    load8(row + I, u);
    float o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = to_f32<T>(g.t[k]);
      o[k] = swiglu(x, to_f32<T>(u.t[k]), gate_of(x));
    }
    store8(h + i * 8, o);
  }
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// dgu may be gu and h may be dh: a thread writes no element but those of a piece that it has read.  AHEAD: where a
// thread has several pieces, copies of its next ones are on their way to its own places in shared memory (no
// thread reads what another has copied) while it is at one.  Two ahead and three blocks to an SM, which is as
// much as the memory likes (48169 x 1408: 102 us; one ahead 105, three 106; two blocks 108, four 113; loads
// to registers by four blocks 113).
constexpr int kGradAhead = 2, kGradBlocks = 3;
constexpr int kGradSmem = (kGradAhead + 1) * 3 * kThreads * 16;
template <typename T, bool AHEAD>
__global__ void __launch_bounds__(kThreads, AHEAD ? kGradBlocks : 4)
    swiglu16_grad_kernel(int R, int E, int I, const T* dh, const T* gu, const int32_t* cumsum, T* dgu, T* h) {
  extern __shared__ __align__(16) uint4 ring[];  // AHEAD: [kGradAhead + 1][g, u, dh][kThreads]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per = I / 8;
  const int64_t n = (int64_t)valid_rows(cumsum, E, R) * per, step = (int64_t)gridDim.x * kThreads;
  const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  int64_t coming = first;
  int to = 0, from = 0;
  auto copy = [&] {
    if (coming < n) {
      const int64_t d = coming / per;
      const T* g = gu + d * 2 * I + (coming - d * per) * 8;
      const uint32_t at = smem_u32(ring + to * 3 * kThreads + threadIdx.x);
      copy16(at, g);
      copy16(at + kThreads * 16, g + I);
      copy16(at + kThreads * 32, dh + coming * 8);
    }
    copies_commit();
    coming += step;
    to = to == kGradAhead ? 0 : to + 1;
  };
  if (AHEAD)
    for (int i = 0; i < kGradAhead; ++i) copy();
  for (int64_t i = first; i < n; i += step) {
    const int64_t d = i / per, at = d * 2 * I + (i - d * per) * 8;
    Eight<T> g8, u8, dh8;
    if (AHEAD) {
      copy();
      copies_wait<kGradAhead>();
      const uint4* x = ring + from * 3 * kThreads + threadIdx.x;
      g8.u = x[0];
      u8.u = x[kThreads];
      dh8.u = x[2 * kThreads];
      from = from == kGradAhead ? 0 : from + 1;
    } else {
      load8(gu + at, g8);
      load8(gu + at + I, u8);
      load8(dh + i * 8, dh8);
    }
    float dg[8], du[8], o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float g = to_f32<T>(g8.t[k]), u = to_f32<T>(u8.t[k]), y = to_f32<T>(dh8.t[k]);
      const Gate s = gate_of(g);
      o[k] = swiglu(g, u, s);
      du[k] = swiglu(g, y, s);
      const float slope = fmaf(g, 1.0f - s.s, 1.0f);
      dg[k] = g < -80.0f ? (u * s.half * (1.0f + g)) * (y * s.half) : y * (s.s * slope) * u;
    }
    store8(dgu + at, dg);
    store8(dgu + at + I, du);
    if (h) store8(h + i * 8, o);
  }
}

// Dispatch and combine: `tpt` threads (a power of two from 32) take a token, or with few tokens a share of
// its channels, eight channels to a thread; the token's rows are looked up once and all read or written
// together.
constexpr int kRoutes = 8;  // at a time
struct Routes {
  int row[kRoutes];
  __device__ __forceinline__ Routes(const int32_t* map, int j, int copies, int rows) {
#pragma unroll
    for (int q = 0; q < kRoutes; ++q) {
      row[q] = j + q < copies ? __ldcg(map + j + q) : -1;
      if ((unsigned)row[q] >= (unsigned)rows) row[q] = -1;
    }
  }
};

template <int DEEP>
__global__ void __launch_bounds__(kThreads) dispatch16_kernel(int M, int D, int copies, int rows, int tpt, int shares,
                                                              const uint4* x, const int32_t* row_map, uint4* out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int group = blockIdx.x / shares, share = blockIdx.x - group * shares, per = D / 8;
  const int t = group * (kThreads / tpt) + threadIdx.x / tpt, lane = threadIdx.x & (tpt - 1);
  if (t >= M) return;
  for (int j = 0; j < copies; j += kRoutes) {
    const Routes r(row_map + (int64_t)t * copies, j, copies, rows);
    for (int c0 = share * tpt + lane; c0 < per; c0 += DEEP * shares * tpt) {
      uint4 v[DEEP];
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        const int c = c0 + d * shares * tpt;
        if (c < per) v[d] = __ldcg(x + (int64_t)t * per + c);
      }
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        const int c = c0 + d * shares * tpt;
#pragma unroll
        for (int q = 0; q < kRoutes; ++q)
          if (r.row[q] >= 0 && c < per) out[(int64_t)r.row[q] * per + c] = v[d];
      }
    }
  }
}

// The sums in order of the routes, in fp32; past eight routes a thread goes on one by one.
template <typename T>
__global__ void __launch_bounds__(kThreads) combine16_kernel(int M, int D, int copies, int rows, int tpt, int shares,
                                                             const T* y, const int32_t* row_map, const float* probs,
                                                             T* out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int group = blockIdx.x / shares, share = blockIdx.x - group * shares, per = D / 8;
  const int t = group * (kThreads / tpt) + threadIdx.x / tpt, lane = threadIdx.x & (tpt - 1);
  if (t >= M) return;
  const int32_t* map = row_map + (int64_t)t * copies;
  const Routes first(map, 0, copies, rows);
  float p[kRoutes];
#pragma unroll
  for (int q = 0; q < kRoutes; ++q) p[q] = first.row[q] >= 0 && probs ? __ldcg(probs + (int64_t)t * copies + q) : 1.0f;
  for (int c = share * tpt + lane; c < per; c += shares * tpt) {
    float acc[8] = {};
    Eight<T> v[kRoutes];
#pragma unroll
    for (int q = 0; q < kRoutes; ++q)
      if (first.row[q] >= 0) load8(y + (int64_t)first.row[q] * D + c * 8, v[q]);
#pragma unroll
    for (int q = 0; q < kRoutes; ++q)
      if (first.row[q] >= 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = fmaf(p[q], to_f32<T>(v[q].t[k]), acc[k]);
      }
    for (int j = kRoutes; j < copies; ++j) {
      const int d = __ldcg(map + j);
      if ((unsigned)d >= (unsigned)rows) continue;
      const float w = probs ? __ldcg(probs + (int64_t)t * copies + j) : 1.0f;
      Eight<T> u;
      load8(y + (int64_t)d * D + c * 8, u);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(w, to_f32<T>(u.t[k]), acc[k]);
    }
    store8(out + (int64_t)t * D + c * 8, acc);
  }
}

// The same for many tokens of up to ROUTES routes: a block goes over its tokens, and while a thread adds up a
// piece, eight channels of a token, copies of its next one are on their way to its own places in shared memory.
// No thread reads what another has copied, so there is nothing to wait for but a thread's own copies.  What is on
// the way at once is what counts, as much as the memory likes and no more (us, of 8192 x 4096, from registers as the
// kernel above: one row 47, two 52, three 57, four 62, six 88; 4096 x 4096 of ten 80):
//   one row, two    four blocks to an SM, three pieces ahead 24, 32; three and four 29, 36; two and six 36, 43
//   three, four     four blocks, one ahead 43, 53; three, one 45, 56; two, two 47, 55; two, three 52, 59
//   six             two blocks, one ahead 75; three blocks 92; two ahead 84, three 129
//   ten             three blocks of half the threads, one ahead 63; two 87
template <int ROUTES>
struct Stream {
  static constexpr int kThreads = ROUTES <= 8 ? 256 : 128, kBlocks = ROUTES <= 4 ? 4 : ROUTES <= 8 ? 2 : 3;
  static constexpr int kAhead = ROUTES <= 2 ? 3 : 1;
  static constexpr int kSmem = (kAhead + 1) * ROUTES * kThreads * 16;
};
template <typename T, int ROUTES>
__global__ void __launch_bounds__(Stream<ROUTES>::kThreads, Stream<ROUTES>::kBlocks)
    combine16_stream_kernel(int M, int D, int copies, int rows, int tpt, const T* y, const int32_t* row_map,
                            const float* probs, T* out) {
  constexpr int kThreads = Stream<ROUTES>::kThreads, kAhead = Stream<ROUTES>::kAhead;
  extern __shared__ __align__(16) uint4 ring[];  // [kAhead + 1][ROUTES][kThreads]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  struct Token {
    int row[ROUTES];
    float p[ROUTES];
  };
  auto look = [&](int t) {
    Token r;
#pragma unroll
    for (int q = 0; q < ROUTES; ++q) {
      const int64_t at = (int64_t)t * copies + q;
      const bool in = t < M && q < copies;
      r.row[q] = in ? __ldcg(row_map + at) : -1;
      r.p[q] = in && probs ? __ldcg(probs + at) : 1.0f;
      if ((unsigned)r.row[q] >= (unsigned)rows) r.row[q] = -1;
    }
    return r;
  };
  const int tokens = kThreads / tpt, per = D / 8, lane = threadIdx.x & (tpt - 1), stride = gridDim.x * tokens;
  int t = blockIdx.x * tokens + threadIdx.x / tpt, c = lane;  // of the next piece to be copied
  if (c >= per) return;
  Token now = look(t), later = look(t + stride);  // its token, and the one behind it
  struct Piece {
    int t, c;
    uint32_t there;
    float p[ROUTES];
  };
  int to_slot = 0, slot = 0;
  auto copy = [&] {
    Piece x;
    x.t = t;
    x.c = c;
    x.there = 0;
    const uint32_t to = smem_u32(ring + to_slot * ROUTES * kThreads + threadIdx.x);
    to_slot = to_slot == kAhead ? 0 : to_slot + 1;
#pragma unroll
    for (int q = 0; q < ROUTES; ++q) {
      x.p[q] = now.p[q];
      if (now.row[q] >= 0) {
        x.there |= 1u << q;
        copy16(to + q * (kThreads * 16), y + (int64_t)now.row[q] * D + c * 8);
      }
    }
    copies_commit();
    c += tpt;
    if (c >= per) {
      c = lane;
      t += stride;
      now = later;
      later = look(t + stride);
    }
    return x;
  };
  Piece coming[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) coming[i] = copy();
  while (coming[0].t < M) {
    const Piece x = coming[0];
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i) coming[i] = coming[i + 1];
    coming[kAhead - 1] = copy();
    copies_wait<kAhead>();
    const uint4* from = ring + slot * ROUTES * kThreads + threadIdx.x;
    slot = slot == kAhead ? 0 : slot + 1;
    float acc[8] = {};
#pragma unroll
    for (int q = 0; q < ROUTES; ++q)
      if (x.there >> q & 1u) {
        Eight<T> v;
        v.u = from[q * kThreads];
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = fmaf(x.p[q], to_f32<T>(v.t[k]), acc[k]);
      }
    store8(out + (int64_t)x.t * D + x.c * 8, acc);
  }
}

// `tpt` threads per token and group of G of its routes, DEEP pieces at a time: dout is read once for the group,
// each y row once, each dy row written, and the products with y summed over the threads in a fixed order.
template <typename T, int G, int DEEP>
__global__ void __launch_bounds__(kThreads) combine16_grad_kernel(int M, int D, int copies, int rows, int tpt,
                                                                  const T* dout, const T* y, const int32_t* row_map,
                                                                  const float* probs, T* dy, float* dprobs) {
  __shared__ float part[kThreads / 32][G];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int groups = (copies + G - 1) / G, tokens = kThreads / tpt;
  const int t0 = blockIdx.x / groups * tokens, j0 = (blockIdx.x % groups) * G;
  const int t = t0 + threadIdx.x / tpt, lane = threadIdx.x & (tpt - 1);
  const int per = D / 8;
  int row[G];
  float p[G], sum[G];
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const int64_t at = (int64_t)t * copies + j0 + q;
    row[q] = t < M && j0 + q < copies ? __ldcg(row_map + at) : -1;
    if ((unsigned)row[q] >= (unsigned)rows) row[q] = -1;
    p[q] = row[q] >= 0 ? __ldcg(probs + at) : 0.0f;
    sum[q] = 0.0f;
  }
  for (int c0 = lane; t < M && c0 < per; c0 += DEEP * tpt) {
    Eight<T> g[DEEP], v[DEEP][G];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      const int c = c0 + d * tpt;
      if (d && c >= per) continue;
      load8(dout + (int64_t)t * D + c * 8, g[d]);
#pragma unroll
      for (int q = 0; q < G; ++q)
        if (row[q] >= 0) load8(y + (int64_t)row[q] * D + c * 8, v[d][q]);
    }
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      const int c = c0 + d * tpt;
      if (d && c >= per) continue;
#pragma unroll
      for (int q = 0; q < G; ++q)
        if (row[q] >= 0) {
          float o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float x = to_f32<T>(g[d].t[k]);
            sum[q] = fmaf(x, to_f32<T>(v[d][q].t[k]), sum[q]);
            o[k] = p[q] * x;
          }
          store8(dy + (int64_t)row[q] * D + c * 8, o);
        }
    }
  }
#pragma unroll
  for (int q = 0; q < G; ++q) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][q] = sum[q];
  }
  __syncthreads();
  const int u = threadIdx.x / G, q = threadIdx.x % G;  // token of the block, route
  if (u < tokens && t0 + u < M && j0 + q < copies) {
    float s = 0.0f;
    for (int w = 0; w < tpt / 32; ++w) s += part[u * (tpt / 32) + w][q];
    dprobs[(int64_t)(t0 + u) * copies + j0 + q] = s;
  }
}

inline unsigned grid_of(int64_t items, int per_sm = 8) {
  const int64_t b = (items + kThreads - 1) / kThreads, most = (int64_t)sm_count() * per_sm;
  return (unsigned)(b < most ? b : most);
}

// Threads to a token: two pieces of eight channels to each at least, where it has as many.
inline int threads_of(int D) {
  int tpt = kThreads;
  while (tpt > 32 && D / 8 < 2 * tpt) tpt /= 2;
  return tpt;
}
// Blocks to `kThreads / tpt` tokens: one, or with few tokens enough for eight blocks on every SM, at most one
// for each piece that their threads take.
inline int shares_of(int groups, int D, int tpt) {
  const int most = (D / 8 + tpt - 1) / tpt, want = (8 * sm_count() + groups - 1) / groups;
  return want < most ? want : most;
}
inline int groups_of(int M, int tpt) { return (M + kThreads / tpt - 1) / (kThreads / tpt); }

template <typename T, bool AHEAD>
cudaError_t swiglu_grad(int R, int E, int I, const void* dh, const void* gu, const int32_t* cumsum, void* dgu, void* h,
                        cudaStream_t stream) {
  const unsigned grid = grid_of((int64_t)R * (I / 8), AHEAD ? kGradBlocks : 8);
  return launch_dependent(swiglu16_grad_kernel<T, AHEAD>, grid, kThreads, AHEAD ? kGradSmem : 0, stream, R, E, I,
                          static_cast<const T*>(dh), static_cast<const T*>(gu), cumsum, static_cast<T*>(dgu),
                          static_cast<T*>(h));
}

template <typename T, int ROUTES>
cudaError_t combine_stream(int M, int D, int copies, int rows, const void* y, const int32_t* row_map,
                           const float* probs, void* out, cudaStream_t stream) {
  using S = Stream<ROUTES>;
  static PerContextOnce set;
  const int dev = current_device();
  if (set.needed(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(combine16_stream_kernel<T, ROUTES>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    set.done(dev);
  }
  const int tpt = threads_of(D) < S::kThreads ? threads_of(D) : S::kThreads, tokens = S::kThreads / tpt;
  const int blocks = (M + tokens - 1) / tokens, most = sm_count() * S::kBlocks;
  return launch_dependent(combine16_stream_kernel<T, ROUTES>, (unsigned)(blocks < most ? blocks : most), S::kThreads,
                          S::kSmem, stream, M, D, copies, rows, tpt, static_cast<const T*>(y), row_map, probs,
                          static_cast<T*>(out));
}

template <typename T, int G, int DEEP>
cudaError_t combine_grad(int M, int D, int copies, int rows, const void* dout, const void* y, const int32_t* row_map,
                         const float* probs, void* dy, float* dprobs, cudaStream_t stream) {
  const int tpt = threads_of(D);
  const unsigned groups = (unsigned)(copies + G - 1) / G;
  return launch_dependent(combine16_grad_kernel<T, G, DEEP>, (unsigned)groups_of(M, tpt) * groups, kThreads, 0, stream,
                          M, D, copies, rows, tpt, static_cast<const T*>(dout), static_cast<const T*>(y), row_map, probs,
                          static_cast<T*>(dy), dprobs);
}

}  // namespace

cudaError_t launch_swiglu16(int R, int E, int I, bool bf16, const void* gu, const int32_t* cumsum, void* h,
                            cudaStream_t stream) {
  const unsigned grid = grid_of((int64_t)R * (I / 8));
  if (bf16)
    return launch_dependent(swiglu16_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, R, E, I,
                            static_cast<const __nv_bfloat16*>(gu), cumsum, static_cast<__nv_bfloat16*>(h));
  return launch_dependent(swiglu16_kernel<__half>, grid, kThreads, 0, stream, R, E, I, static_cast<const __half*>(gu),
                          cumsum, static_cast<__half*>(h));
}

cudaError_t launch_swiglu16_grad(int R, int E, int I, bool bf16, const void* dh, const void* gu, const int32_t* cumsum,
                                 void* dgu, void* h, cudaStream_t stream) {
  // ahead where eight blocks to an SM would have a second round (1024 x 2048, 3.4 blocks: 4.9 us, ahead 5.1,
  // and 0.6 more behind kernels that leave the memory to L1)
  const bool ahead = (int64_t)R * (I / 8) > 8 * (int64_t)sm_count() * kThreads;
  if (bf16)
    return ahead ? swiglu_grad<__nv_bfloat16, true>(R, E, I, dh, gu, cumsum, dgu, h, stream)
                 : swiglu_grad<__nv_bfloat16, false>(R, E, I, dh, gu, cumsum, dgu, h, stream);
  return ahead ? swiglu_grad<__half, true>(R, E, I, dh, gu, cumsum, dgu, h, stream)
               : swiglu_grad<__half, false>(R, E, I, dh, gu, cumsum, dgu, h, stream);
}

cudaError_t launch_dispatch16(int M, int D, int copies, int rows, const void* x, const int32_t* row_map, void* out,
                              cudaStream_t stream) {
  const int tpt = threads_of(D), groups = groups_of(M, tpt), shares = shares_of(groups, D, tpt);
  // a thread that has a token's channels to itself reads two pieces at once (8192 x 4096 to one row: 25.1 and 28.5
  // us, to six 73.0 and 73.8; where they are shared there is one for each: 300 x 4096 to two rows 3.3 and 2.8)
  return launch_dependent(shares == 1 ? dispatch16_kernel<2> : dispatch16_kernel<1>, (unsigned)(groups * shares),
                          kThreads, 0, stream, M, D, copies, rows, tpt, shares, static_cast<const uint4*>(x), row_map,
                          static_cast<uint4*>(out));
}

cudaError_t launch_combine16(int M, int D, int copies, int rows, bool bf16, const void* y, const int32_t* row_map,
                             const float* probs, void* out, cudaStream_t stream) {
  const int tpt = threads_of(D), groups = groups_of(M, tpt), shares = shares_of(groups, D, tpt);
  const unsigned grid = (unsigned)(groups * shares);
  // Pieces of eight channels, as multiples of the threads of a block on every SM (us, streamed and not):
  // 3.4: 4.0 and 4.5 (256 x 4096, six rows), 5.6 and 6.8 (2048 x 512); 2.9: 6.4 and 5.6 (128 x 7168, eight rows);
  // 1.7: 3.8 and 3.0 (128 x 4096).
  if (copies <= 16 && (int64_t)M * (D / 8) > 3 * (int64_t)sm_count() * kThreads) {
    if (copies <= 2)
      return bf16 ? combine_stream<__nv_bfloat16, 2>(M, D, copies, rows, y, row_map, probs, out, stream)
                  : combine_stream<__half, 2>(M, D, copies, rows, y, row_map, probs, out, stream);
    if (copies <= 4)
      return bf16 ? combine_stream<__nv_bfloat16, 4>(M, D, copies, rows, y, row_map, probs, out, stream)
                  : combine_stream<__half, 4>(M, D, copies, rows, y, row_map, probs, out, stream);
    if (copies <= 8)
      return bf16 ? combine_stream<__nv_bfloat16, 8>(M, D, copies, rows, y, row_map, probs, out, stream)
                  : combine_stream<__half, 8>(M, D, copies, rows, y, row_map, probs, out, stream);
    return bf16 ? combine_stream<__nv_bfloat16, 16>(M, D, copies, rows, y, row_map, probs, out, stream)
                : combine_stream<__half, 16>(M, D, copies, rows, y, row_map, probs, out, stream);
  }
  if (bf16)
    return launch_dependent(combine16_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, M, D, copies, rows, tpt, shares,
                            static_cast<const __nv_bfloat16*>(y), row_map, probs, static_cast<__nv_bfloat16*>(out));
  return launch_dependent(combine16_kernel<__half>, grid, kThreads, 0, stream, M, D, copies, rows, tpt, shares,
                          static_cast<const __half*>(y), row_map, probs, static_cast<__half*>(out));
}

cudaError_t launch_combine16_grad(int M, int D, int copies, int rows, bool bf16, const void* dout, const void* y,
                                  const int32_t* row_map, const float* probs, void* dy, float* dprobs,
                                  cudaStream_t stream) {
  // Routes to a group, and pieces read at once.  Few tokens: two and four (61 tokens of eight routes x 7168: 3.4 us;
  // one piece 4.6, eight routes to a group 6.5).  Many: all up to eight, so that dout is read once, as registers
  // for no more leave room for more blocks (8192 x 4096, of one row 44 us, in groups of eight 68; of three 81 and 95;
  // of six 138).
  if (M < 4 * sm_count())
    return bf16 ? combine_grad<__nv_bfloat16, 2, 4>(M, D, copies, rows, dout, y, row_map, probs, dy, dprobs, stream)
                : combine_grad<__half, 2, 4>(M, D, copies, rows, dout, y, row_map, probs, dy, dprobs, stream);
  if (copies <= 2)
    return bf16 ? combine_grad<__nv_bfloat16, 2, 2>(M, D, copies, rows, dout, y, row_map, probs, dy, dprobs, stream)
                : combine_grad<__half, 2, 2>(M, D, copies, rows, dout, y, row_map, probs, dy, dprobs, stream);
  if (copies <= 4)
    return bf16 ? combine_grad<__nv_bfloat16, 4, 1>(M, D, copies, rows, dout, y, row_map, probs, dy, dprobs, stream)
                : combine_grad<__half, 4, 1>(M, D, copies, rows, dout, y, row_map, probs, dy, dprobs, stream);
  return bf16 ? combine_grad<__nv_bfloat16, 8, 1>(M, D, copies, rows, dout, y, row_map, probs, dy, dprobs, stream)
              : combine_grad<__half, 8, 1>(M, D, copies, rows, dout, y, row_map, probs, dy, dprobs, stream);
}

}  // namespace moe
