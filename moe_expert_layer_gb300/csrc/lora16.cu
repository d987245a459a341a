// Low-rank adapters of many requests beside a shared projection (include/moe_experts16.h):
//   v = a[l] x[t],  out[t] = base[t] + s b[l] v
// for the tokens sorted by adapter, in tiles of tokens of one adapter.  Bound by bytes: x, base and
// out once each, and the adapters' weights, which are all there is to read in a decode batch.
//
// Both products are warp-level MMAs (m16n8k16, fp32 sums): with ranks up to 128 they are far too thin
// for tcgen05's 128 rows, and need no shared memory.  An MMA's order of the reduction index is free as
// long as both operands have the same, so each lane takes its operands as 16 bytes straight from a
// row: lane (g, t) holds elements 8 t .. 8 t + 7 of 32, the first four for one MMA and the others for
// the next; a row's 64 bytes come with one load of four lanes.
//
// Shrink: a block per tile and share of D; its warps take 32-deep slices in turn and add up over
// shared memory.  The shares' sums are left in fp32 and added, in order, by the second kernel.
// Expand: a block per tile and share of N.  v goes into the MMA as two 16-bit numbers, v 2^-e = hi +
// lo with e the exponent of the token's largest: 16 significant bits or more, and no rank value
// leaves binary16's range.  The columns of four MMAs are dealt out so that a lane gets eight
// neighbouring channels of a token, 16 bytes of base and out.
#include "experts16.h"
#include "mxfp4.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 32 steps: rows g and g + 8 of A, column g of B, as lane (g, t) holds them.
template <typename T>
__device__ __forceinline__ void mma32(float (&c)[4], const uint4& lo, const uint4& hi, const uint4& b) {
  const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
  mma16<T>(c, a0, b.x, b.y);
  mma16<T>(c, a1, b.z, b.w);
}

// Tile `index` of the tokens sorted by adapter: positions [start, start + rows) of adapter l, or of
// no adapter (l = -1, behind the others).  rows = 0 past the last tile.
struct Tile {
  int l, start, rows;
};
// The whole block enters.  Thread i counts the tiles of adapters 4 i .. 4 i + 3 (L <= 1023).
template <int TOKENS>
__device__ __forceinline__ Tile find_tile(int index, const int32_t* cumsum, int L, int M) {
  __shared__ int s_warp[kWarps];
  __shared__ Tile s_tile;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l0 = threadIdx.x * 4;
  int end[5], count = 0;
#pragma unroll
  for (int i = 0; i < 5; ++i) end[i] = l0 + i - 1 < 0 ? 0 : l0 + i - 1 < L ? min(max(__ldcg(cumsum + l0 + i - 1), 0), M) : -1;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (end[i + 1] > end[i] && end[i] >= 0) count += (end[i + 1] - end[i] + TOKENS - 1) / TOKENS;
  int incl = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) s_warp[warp] = incl;
  if (threadIdx.x == 0) s_tile = Tile{-1, 0, 0};
  __syncthreads();
  int before = incl - count, all = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  if (index >= before && index < before + count) {
    int at = index - before;
    for (int i = 0; i < 4; ++i) {
      const int n = end[i + 1] > end[i] && end[i] >= 0 ? (end[i + 1] - end[i] + TOKENS - 1) / TOKENS : 0;
      if (at < n) {
        s_tile = Tile{l0 + i, end[i] + at * TOKENS, min(TOKENS, end[i + 1] - end[i] - at * TOKENS)};
        break;
      }
      at -= n;
    }
  }
  if (threadIdx.x == 0 && index >= all) {
    const int start = min(max(__ldcg(cumsum + L - 1), 0), M) + (index - all) * TOKENS;
    if (start < M && start >= 0) s_tile = Tile{-1, start, min(TOKENS, M - start)};
  }
  __syncthreads();
  return s_tile;
}

// MMA rows: ranks (MR x 16); columns: tokens (TN x 8).
template <typename T, int MR, int TN>
__global__ void __launch_bounds__(kThreads) lora16_shrink_kernel(const Lora16Problem p, int splits) {
  extern __shared__ __align__(16) float s_part[];  // [kWarps][MR][TN][4][32]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int split = blockIdx.x % splits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Tile tile = find_tile<TN * 8>(blockIdx.x / splits, p.cumsum, p.L, p.M);
  if (tile.rows == 0 || tile.l < 0) return;
  const int D = p.D, chunks = (D + 31) / 32, per = (chunks + splits - 1) / splits;
  const int c1 = min(chunks, (split + 1) * per);
  const T* a = static_cast<const T*>(p.a) + (int64_t)tile.l * p.rank * D;
  const T* x[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int i = j * 8 + g, tok = i < tile.rows ? __ldcg(p.route + tile.start + i) : -1;
    x[j] = (unsigned)tok < (unsigned)p.M ? static_cast<const T*>(p.x) + (int64_t)tok * D : nullptr;
  }
  float c[MR][TN][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int chunk = split * per + warp; chunk < c1; chunk += kWarps) {
    const int k = chunk * 32 + t * 8;
    const bool in = k < D;
    uint4 b[TN], lo[MR], hi[MR];
#pragma unroll
    for (int j = 0; j < TN; ++j) b[j] = in && x[j] ? __ldcg(reinterpret_cast<const uint4*>(x[j] + k)) : zero;
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      const int r = m * 16 + g;
      lo[m] = in && r < p.rank ? __ldcg(reinterpret_cast<const uint4*>(a + (int64_t)r * D + k)) : zero;
      hi[m] = in && r + 8 < p.rank ? __ldcg(reinterpret_cast<const uint4*>(a + (int64_t)(r + 8) * D + k)) : zero;
    }
#pragma unroll
    for (int j = 0; j < TN; ++j)
      if (TN <= 2 || j * 8 < tile.rows) {
#pragma unroll
        for (int m = 0; m < MR; ++m) mma32<T>(c[m][j], lo[m], hi[m], b[j]);
      }
  }
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) s_part[((warp * MR + m) * TN + j) * 128 + q * 32 + lane] = c[m][j][q];
  __syncthreads();
  // element q of lane (g, t): rank 16 m + g + 8 (q / 2), token 8 j + 2 t + q % 2
  float* v = p.v + ((int64_t)split * p.M + tile.start) * p.rank;
  for (int i = threadIdx.x; i < MR * TN * 128; i += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += s_part[w * MR * TN * 128 + i];
    const int l = i & 31, q = (i >> 5) & 3, j = (i >> 7) % TN, m = (i >> 7) / TN;
    const int r = m * 16 + (l >> 2) + 8 * (q >> 1), tok = j * 8 + 2 * (l & 3) + (q & 1);
    if (r < p.rank && tok < tile.rows) v[(int64_t)tok * p.rank + r] = s;
  }
}

// 16-bit conversion that keeps infinities.
template <typename T> __device__ __forceinline__ T to16(float v);
template <> __device__ __forceinline__ __half to16<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 to16<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// MMA rows: tokens (TM x 16); columns: channels, 32 in four MMAs; RC x 32 ranks.
template <typename T, int RC, int TM>
__global__ void __launch_bounds__(kThreads) lora16_expand_kernel(const Lora16Problem p, int splits, int shares) {
  constexpr int kTokens = TM * 16, kPitch = RC * 32 + 8;  // elements: rows 16 bytes past a multiple of 64
  __shared__ __align__(16) T s_hi[kTokens * kPitch], s_lo[kTokens * kPitch];
  __shared__ float s_pow[kTokens];
  __shared__ int s_tok[kTokens];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int share = blockIdx.x % shares, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Tile tile = find_tile<kTokens>(blockIdx.x / shares, p.cumsum, p.L, p.M);
  if (tile.rows == 0 || (tile.l < 0 && p.base == p.out)) return;
  const int N = p.N, strips = (N + 31) / 32, per = (strips + shares - 1) / shares;
  const int last = min(strips, (share + 1) * per);
  const T* base = static_cast<const T*>(p.base);
  T* out = static_cast<T*>(p.out);
  if (threadIdx.x < kTokens) {
    const int tok = (int)threadIdx.x < tile.rows ? __ldcg(p.route + tile.start + threadIdx.x) : -1;
    s_tok[threadIdx.x] = (unsigned)tok < (unsigned)p.M ? tok : -1;
  }
  if (tile.l < 0) {  // no adapter: the base itself
    __syncthreads();
    const int n0 = share * per * 32, n1 = min(N, last * 32);
    for (int i = warp; i < tile.rows; i += kWarps)
      if (s_tok[i] >= 0)
        for (int n = n0 + lane * 8; n < n1; n += 256)
          *reinterpret_cast<uint4*>(out + (int64_t)s_tok[i] * N + n) =
              __ldcg(reinterpret_cast<const uint4*>(base + (int64_t)s_tok[i] * N + n));
    return;
  }
  // a warp per token: its rank values, their largest finite exponent, the two 16-bit parts
  for (int i = warp; i < kTokens; i += kWarps) {
    float v[RC];
    uint32_t most = 0;
#pragma unroll
    for (int q = 0; q < RC; ++q) {
      const int r = q * 32 + lane;
      v[q] = 0.0f;
      if (i < tile.rows && r < p.rank)
        for (int s = 0; s < splits; ++s) v[q] += __ldcg(p.v + ((int64_t)s * p.M + tile.start + i) * p.rank + r);
      const uint32_t f = (__float_as_uint(v[q]) >> 23) & 255u;
      if (f != 255u) most = max(most, f);
    }
    most = max(__reduce_max_sync(0xffffffffu, most), 1u);  // 1 .. 254: 2^(most - 127)
    const float down = most == 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - most) << 23);
#pragma unroll
    for (int q = 0; q < RC; ++q) {
      const float x = v[q] * down;
      const T hi = to16<T>(x);
      const float left = x - to_f32<T>(hi);
      s_hi[i * kPitch + q * 32 + lane] = hi;
      s_lo[i * kPitch + q * 32 + lane] = to16<T>(fabsf(x) < 4.0f ? left : 0.0f);  // infinities and NaN: hi alone
    }
    if (lane == 0) s_pow[i] = __uint_as_float(most << 23);
  }
  __syncthreads();
  const float scale = p.scales ? __ldcg(p.scales + tile.l) : 1.0f;
  const T* b = static_cast<const T*>(p.b) + (int64_t)tile.l * N * p.rank;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int tiles = (tile.rows + 15) / 16;
  for (int strip = share * per + warp; strip < last; strip += kWarps) {
    // column c of MMA j is channel 8 (c / 2) + 2 j + c % 2 of the strip: lane (g, t) then holds channels
    // 8 t .. 8 t + 7 of tokens g and g + 8
    uint4 w[4][RC];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = strip * 32 + (g >> 1) * 8 + j * 2 + (g & 1);
#pragma unroll
      for (int q = 0; q < RC; ++q) {
        const int r = q * 32 + t * 8;
        w[j][q] = n < N && r < p.rank ? __ldcg(reinterpret_cast<const uint4*>(b + (int64_t)n * p.rank + r)) : zero;
      }
    }
    const int n = strip * 32 + t * 8;
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      if (m >= tiles) break;
      int64_t at[2];
      uint4 y[2];
      bool in[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = s_tok[m * 16 + g + 8 * h];
        in[h] = tok >= 0 && n < N;
        at[h] = (int64_t)tok * N + n;
        y[h] = in[h] ? __ldcg(reinterpret_cast<const uint4*>(base + at[h])) : zero;
      }
      float c[4][4] = {};
#pragma unroll
      for (int q = 0; q < RC; ++q) {
        const int s = (m * 16 + g) * kPitch + q * 32 + t * 8;
        const uint4 h0 = *reinterpret_cast<const uint4*>(s_hi + s), h1 = *reinterpret_cast<const uint4*>(s_hi + s + 8 * kPitch);
        const uint4 l0 = *reinterpret_cast<const uint4*>(s_lo + s), l1 = *reinterpret_cast<const uint4*>(s_lo + s + 8 * kPitch);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma32<T>(c[j], l0, l1, w[j][q]);
          mma32<T>(c[j], h0, h1, w[j][q]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (in[h]) {
          const float f = s_pow[m * 16 + g + 8 * h];
          const T* yt = reinterpret_cast<const T*>(&y[h]);
          uint4 o;
          T* ot = reinterpret_cast<T*>(&o);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            from_f32x2<T>(fmaf(scale, c[j][2 * h] * f, to_f32<T>(yt[2 * j])),
                          fmaf(scale, c[j][2 * h + 1] * f, to_f32<T>(yt[2 * j + 1])), ot + 2 * j);
          *reinterpret_cast<uint4*>(out + at[h]) = o;
        }
    }
  }
}

// Shares of D: enough blocks for the device, at most what the workspace holds: max(M, kPartRows)
// rows of fp32 rank values in all.
constexpr int kMaxSplits = 16, kPartRows = 4096;

inline int tiles_of(int M, int groups, int tokens) { return M / tokens + (M < groups ? M : groups); }

template <typename T, int MR, int TN>
cudaError_t shrink(const Lora16Problem& p, int& splits, cudaStream_t stream) {
  const int tiles = tiles_of(p.M, p.L, TN * 8), chunks = (p.D + 31) / 32;
  splits = (2 * sm_count() + tiles - 1) / tiles;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits > kPartRows / p.M) splits = kPartRows / p.M;
  if (splits > chunks / kWarps) splits = chunks / kWarps;
  if (splits < 1) splits = 1;
  const size_t smem = (size_t)kWarps * MR * TN * 128 * 4;
  static PerContextOnce set;
  const int dev = current_device();
  if (smem > 48 * 1024 && set.needed(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(lora16_shrink_kernel<T, MR, TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    set.done(dev);
  }
  return launch_dependent(lora16_shrink_kernel<T, MR, TN>, (unsigned)(tiles * splits), kThreads, smem, stream, p, splits);
}

template <typename T, int RC, int TM>
cudaError_t expand(const Lora16Problem& p, int splits, cudaStream_t stream) {
  const int tiles = tiles_of(p.M, p.L + 1, TM * 16), strips = (p.N + 31) / 32;
  int shares = (4 * sm_count() + tiles - 1) / tiles;
  if (shares > (strips + kWarps - 1) / kWarps) shares = (strips + kWarps - 1) / kWarps;
  return launch_dependent(lora16_expand_kernel<T, RC, TM>, (unsigned)(tiles * shares), kThreads, 0, stream, p, splits,
                          shares);
}

template <typename T>
cudaError_t launch(const Lora16Problem& p, cudaStream_t stream) {
  // tiles of 64 tokens (32 above rank 64, whose sums would not fit the registers) or, for few tokens
  // an adapter, of 16
  const bool few = p.M <= 16 * p.L;
  int splits = 1;
  cudaError_t e;
  if (p.rank <= 16)
    e = few ? shrink<T, 1, 2>(p, splits, stream) : shrink<T, 1, 8>(p, splits, stream);
  else if (p.rank <= 32)
    e = few ? shrink<T, 2, 2>(p, splits, stream) : shrink<T, 2, 8>(p, splits, stream);
  else if (p.rank <= 64)
    e = few ? shrink<T, 4, 2>(p, splits, stream) : shrink<T, 4, 8>(p, splits, stream);
  else
    e = few ? shrink<T, 8, 2>(p, splits, stream) : shrink<T, 8, 4>(p, splits, stream);
  if (e != cudaSuccess) return e;
  if (p.rank <= 32) return few ? expand<T, 1, 1>(p, splits, stream) : expand<T, 1, 4>(p, splits, stream);
  if (p.rank <= 64) return few ? expand<T, 2, 1>(p, splits, stream) : expand<T, 2, 4>(p, splits, stream);
  return few ? expand<T, 4, 1>(p, splits, stream) : expand<T, 4, 4>(p, splits, stream);
}

}  // namespace

size_t lora16_workspace_bytes(int M, int rank) { return (size_t)(M > kPartRows ? M : kPartRows) * rank * 4; }

cudaError_t launch_lora16(const Lora16Problem& p, cudaStream_t stream) {
  return p.bf16 ? launch<__nv_bfloat16>(p, stream) : launch<__half>(p, stream);
}

}  // namespace moe
