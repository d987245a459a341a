// Low-rank adapters of many requests beside a shared projection (include/moe_experts16.h):
//   v = a[l] x[t],  out[t] = base[t] + s b[l] v
// for the tokens sorted by adapter, in tiles of tokens of one adapter.  Bound by bytes: x, base and
// out once each, and the adapters' weights, which are all there is to read in a decode batch.
//
// Both products are warp-level MMAs (m16n8k16, fp32 sums): with ranks up to 128 they are far too thin
// for tcgen05's 128 rows.  An MMA's order of the reduction index is free as long as both operands have
// the same, so a lane can take its operands as 16 bytes straight from a row: lane (g, t) holds elements
// 8 t .. 8 t + 7 of 32, the first four for one MMA and the others for the next; a row's 64 bytes come
// with one load of four lanes.
//
// Many tokens to an adapter, two kernels.  Shrink: a block per tile of 64 tokens and share of D; tokens and
// ranks pass through a ring in shared memory, 64 deep a stage, and the warps divide the outputs.  The shares'
// sums are left in fp32 and added, in order, by the second kernel.  Expand: a block per tile and share
// of N.  It begins, as a programmatic dependent, once every block of the first kernel is past its own
// wait: what that one does not write (tables, weights, base) is read ahead of this one's wait.
// Few tokens: one kernel, a cluster per tile of 16.
//
// Measured (us; GB/s over the bytes of the definition): 128 tokens 7168 -> 4096 on 100 adapters of rank 16
// 10.9 (launch, two chains of loads and the cluster's barrier; 26 MB are 3.9); 8192 tokens 4096 -> 4096,
// 24 adapters, of rank 16 40 (5000), of rank 64 54 (3900): 21 in the first kernel, and there the warp-level
// tensor path is 45% busy.  Above that it bounds: rank 128 93.
//
// v goes into the second MMA as two 16-bit numbers, s v 2^-e = hi + lo with e set by the exponent of the token's
// largest: 16 significant bits or more, and no rank value leaves binary16's range.  The columns of
// four MMAs are dealt out so that a lane gets eight neighbouring channels of a token, 16 bytes of base
// and out.
#include <type_traits>

#include "experts16.h"
#include "mxfp4.cuh"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
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
// The whole block enters.  Thread i counts the tiles of the PER adapters from PER i (L <= 1023).
template <int TOKENS, int THREADS>
__device__ __forceinline__ Tile find_tile(int index, const int32_t* cumsum, int L, int M) {
  constexpr int PER = 1024 / THREADS, WARPS = THREADS / 32;
  __shared__ int s_warp[WARPS];
  __shared__ Tile s_tile;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l0 = threadIdx.x * PER;
  int end[PER + 1], n[PER], count = 0;
#pragma unroll
  for (int i = 0; i <= PER; ++i) {
    const int l = l0 + i - 1;
    end[i] = l < 0 ? 0 : l < L ? min(max(__ldcg(cumsum + l), 0), M) : 0;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    n[i] = l0 + i < L && end[i + 1] > end[i] ? (end[i + 1] - end[i] + TOKENS - 1) / TOKENS : 0;
    count += n[i];
  }
  int incl = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  if (threadIdx.x == 0) s_tile = Tile{-1, 0, 0};
  __syncthreads();
  int before = incl - count, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  int at = index - before;
  if (at >= 0 && at < count) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at >= 0 && at < n[i])
        s_tile = Tile{l0 + i, end[i] + at * TOKENS, min(TOKENS, end[i + 1] - end[i] - at * TOKENS)};
      at -= n[i];
    }
  }
  if (threadIdx.x == 0 && index >= all) {
    const int start = min(max(__ldcg(cumsum + L - 1), 0), M) + (index - all) * TOKENS;
    if (start < M) s_tile = Tile{-1, start, min(TOKENS, M - start)};
  }
  __syncthreads();
  return s_tile;
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Many tokens to an adapter.  MMA rows: tokens, 16 to each of four groups of two warps; columns:
// ranks, MR x 8 to a warp.  A stage is 64 deep: rows of 128 bytes, their 16-byte pieces c at
// c ^ (row % 8).
constexpr int kManyTokens = 64;
// Stages of the rings: more copies under way at low ranks, two blocks of the second kernel to an SM at high ones
// (rank 128, 8192 tokens: four stages 105 us, three 93).
template <int MR>
constexpr int kStagesOf = MR <= 2 ? 6 : MR <= 4 ? 4 : 3;
template <typename T, int MR>
__global__ void __launch_bounds__(kThreads) lora16_shrink_many_kernel(const Lora16Problem p, int splits) {
  constexpr int kXBytes = kManyTokens * 128, kStage = kXBytes + MR * 16 * 128, kStages = kStagesOf<MR>;
  extern __shared__ __align__(128) uint8_t s_ring[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int split = blockIdx.x % splits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Tile tile = find_tile<kManyTokens, kThreads>(blockIdx.x / splits, p.cumsum, p.L, p.M);
  if (tile.rows == 0 || tile.l < 0) return;
  const int D = p.D, chunks = (D + 63) / 64, per = (chunks + splits - 1) / splits;
  const int c0 = split * per, n = max(0, min(chunks - c0, per));
  const int row = threadIdx.x >> 3, piece = threadIdx.x & 7;  // rows 32 apart
  const T* x[2];
  const T* any = static_cast<const T*>(p.x);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int tok = row + 32 * i < tile.rows ? __ldcg(p.route + tile.start + row + 32 * i) : -1;
    x[i] = (unsigned)tok < (unsigned)p.M ? any + (int64_t)tok * D : nullptr;
  }
  const T* a = static_cast<const T*>(p.a) + (int64_t)tile.l * p.rank * D;
  const uint32_t ring = smem_u32(s_ring), swizzled = (uint32_t)((piece ^ (row & 7)) << 4);
  auto load = [&](int chunk, int stage) {
    const int k = (c0 + chunk) * 64 + piece * 8;
    const uint32_t st = ring + stage * kStage;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = x[i] && k < D;
      copy16(st + (row + 32 * i) * 128 + swizzled, in ? x[i] + k : any, in);
    }
#pragma unroll
    for (int r0 = 0; r0 < MR * 16; r0 += 32) {
      const int r = r0 + row;
      const bool in = r < p.rank && k < D;
      if (MR > 1 || r < 16) copy16(st + kXBytes + r * 128 + swizzled, in ? a + (int64_t)r * D + k : any, in);
    }
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (s < n) load(s, s);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const int tg = warp >> 1, half = warp & 1;  // tokens 16 tg .., ranks MR * 8 * half ..
  const int arow = tg * 16 + (lane & 15), brow = half * MR * 8 + (lane & 7) + (MR > 1 ? (lane >> 4) * 8 : 0);
  float c[MR][4] = {};
  for (int i = 0; i < n; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncthreads();  // the stage has landed for all, and all are done with the one that is filled next
    if (i + kStages - 1 < n) load(i + kStages - 1, (i + kStages - 1) % kStages);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const uint32_t st = ring + (i % kStages) * kStage;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t f[4];
      ldmatrix4(f, st + arow * 128 + (((2 * k + (lane >> 4)) ^ (arow & 7)) << 4));
#pragma unroll
      for (int m = 0; m < MR; m += 2) {
        // two columns' tiles of eight ranks (with MR = 1 the second one is the first again)
        uint32_t w[4];
        const int r = brow + m * 8;
        ldmatrix4(w, st + kXBytes + r * 128 + (((2 * k + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
        mma16<T>(c[m], f, w[0], w[1]);
        if (m + 1 < MR) mma16<T>(c[m + 1], f, w[2], w[3]);
      }
    }
  }
  float* v = p.v + ((int64_t)split * p.M + tile.start) * p.rank;
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = tg * 16 + (lane >> 2) + 8 * h, r = half * MR * 8 + m * 8 + (lane & 3) * 2;
      if (tok < tile.rows && r < p.rank)
        *reinterpret_cast<float2*>(v + (int64_t)tok * p.rank + r) = make_float2(c[m][2 * h], c[m][2 * h + 1]);
    }
}

// 16-bit conversion that keeps infinities.
template <typename T> __device__ __forceinline__ T to16(float v);
template <> __device__ __forceinline__ __half to16<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 to16<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// s v of a token as 2^e (hi + lo); a warp enters, lane r with ranks q * 32 + r.  Returns 2^e.  e is the exponent of the
// token's largest finite value, and for bfloat16, whose b may be as large as fp32's numbers, 8 more (held at
// the last one): 128 values below 2^-7 times b stay finite where their sum does.
template <typename T, int RC>
__device__ __forceinline__ float split_ranks(const float (&v)[RC], T* hi, T* lo, int lane) {
  uint32_t most = 0;
#pragma unroll
  for (int q = 0; q < RC; ++q) {
    const uint32_t f = (__float_as_uint(v[q]) >> 23) & 255u;
    if (f != 255u) most = max(most, f);
  }
  most = max(__reduce_max_sync(0xffffffffu, most), 1u);  // 1 .. 254: 2^(most - 127)
  if (!std::is_same<T, __half>::value) most = min(most + 8u, 254u);
  const float down = most == 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - most) << 23);
#pragma unroll
  for (int q = 0; q < RC; ++q) {
    const float x = v[q] * down;
    const T h = to16<T>(x);
    const float left = x - to_f32<T>(h);
    hi[q * 32 + lane] = h;
    lo[q * 32 + lane] = to16<T>(fabsf(x) < 4.0f ? left : 0.0f);  // infinities and NaN: hi alone
  }
  return __uint_as_float(most << 23);
}

// The sums of the shares of the rank values of tokens i, i + STRIDE, .. of a tile, times the adapter's
// scale; four shares of all of them are read together.
template <int RC, int TOKENS, int STRIDE>
__device__ __forceinline__ void load_ranks(const Lora16Problem& p, int splits, const Tile& tile, int i, float scale,
                                           int lane, float (&v)[TOKENS][RC]) {
  const int64_t share = (int64_t)p.M * p.rank;
#pragma unroll
  for (int k = 0; k < TOKENS; ++k)
#pragma unroll
    for (int q = 0; q < RC; ++q) v[k][q] = 0.0f;
  const float* part = p.v + (int64_t)(tile.start + i) * p.rank + lane;
  for (int s = 0; s < splits; s += 4, part += 4 * share) {
    float x[4][TOKENS][RC];
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int k = 0; k < TOKENS; ++k)
#pragma unroll
        for (int q = 0; q < RC; ++q)
          x[d][k][q] = s + d < splits && i + k * STRIDE < tile.rows && q * 32 + lane < p.rank
                           ? __ldcg(part + d * share + k * STRIDE * p.rank + q * 32)
                           : 0.0f;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int k = 0; k < TOKENS; ++k)
#pragma unroll
        for (int q = 0; q < RC; ++q) v[k][q] += x[d][k][q];
  }
#pragma unroll
  for (int k = 0; k < TOKENS; ++k)
#pragma unroll
    for (int q = 0; q < RC; ++q) v[k][q] *= scale;
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Eight neighbouring channels of a token: base + 2^e sums, c[j][0], c[j][1] channels 2 j, 2 j + 1.
template <typename T>
__device__ __forceinline__ uint4 add_base(const uint4& y, const float (&c)[4][4], int h, float f) {
  const T* yt = reinterpret_cast<const T*>(&y);
  uint4 o;
  T* ot = reinterpret_cast<T*>(&o);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    from_f32x2<T>(fmaf(c[j][2 * h], f, to_f32<T>(yt[2 * j])), fmaf(c[j][2 * h + 1], f, to_f32<T>(yt[2 * j + 1])), ot + 2 * j);
  return o;
}

// Tokens without an adapter: the base itself, channels [n0, n1), eight pieces of a thread at a time.
template <typename T, int THREADS>
__device__ __forceinline__ void copy_base(const Lora16Problem& p, const int* tokens, int rows, int n0, int n1) {
  constexpr int DEEP = 8;
  const T* base = static_cast<const T*>(p.base);
  T* out = static_cast<T*>(p.out);
  const int per = max(n1 - n0, 0) / 8, n = rows * per;
  for (int i0 = threadIdx.x; i0 < n; i0 += THREADS * DEEP) {
    uint4 v[DEEP];
    int64_t at[DEEP];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      const int i = i0 + d * THREADS, tok = i < n ? tokens[i / per] : -1;
      at[d] = tok >= 0 ? (int64_t)tok * p.N + n0 + i % per * 8 : -1;
      if (at[d] >= 0) v[d] = __ldcg(reinterpret_cast<const uint4*>(base + at[d]));
    }
#pragma unroll
    for (int d = 0; d < DEEP; ++d)
      if (at[d] >= 0) *reinterpret_cast<uint4*>(out + at[d]) = v[d];
  }
}

// Few tokens to an adapter: both products in one kernel, a cluster of CTAs per tile of 16 tokens.  Each CTA
// takes a share of D: its warps take 32-deep slices straight from memory, DEEP of them under way, and
// add up over its shared memory (MMA rows: ranks, MR x 16; columns: tokens).  Behind the cluster's barrier
// every CTA adds the CTAs' sums, in order, and takes a share of N (MMA rows: tokens; columns: channels, 32 in
// four MMAs); what its first strip needs is on the way meanwhile.  Past 64 ranks two halves of the warps
// divide them, so that two CTAs still fit an SM.
constexpr int kFewTokens = 16;
template <typename T, int MR, int DEEP, int HALVES>
__global__ void __launch_bounds__(kThreads) lora16_few_kernel(const Lora16Problem p, int ctas) {
  constexpr int TN = 2, RC = (MR * HALVES + 1) / 2, kRanks = RC * 32, kPitch = kRanks + 8;  // elements
  constexpr int kSlices = kWarps / HALVES;  // taken at once
  extern __shared__ __align__(16) float s_part[];  // [kWarps][MR][TN][4][32]
  __shared__ float s_sum[kFewTokens][kRanks];
  __shared__ __align__(16) T s_hi[kFewTokens * kPitch], s_lo[kFewTokens * kPitch];
  __shared__ float s_pow[kFewTokens];
  __shared__ int s_tok[kFewTokens];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int share = blockIdx.x % ctas, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Tile tile = find_tile<kFewTokens, kThreads>(blockIdx.x / ctas, p.cumsum, p.L, p.M);  // the cluster's
  if (tile.rows == 0) return;
  const int D = p.D, N = p.N, strips = (N + 31) / 32, per_n = (strips + ctas - 1) / ctas;
  const int last = min(strips, (share + 1) * per_n);
  if (threadIdx.x < kFewTokens) {
    const int tok = (int)threadIdx.x < tile.rows ? __ldcg(p.route + tile.start + threadIdx.x) : -1;
    s_tok[threadIdx.x] = (unsigned)tok < (unsigned)p.M ? tok : -1;
  }
  __syncthreads();
  if (tile.l < 0) {
    if (p.base != p.out) copy_base<T, kThreads>(p, s_tok, tile.rows, share * per_n * 32, min(N, last * 32));
    return;
  }
  const int tok[2] = {s_tok[g], s_tok[g + 8]};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  {
    const int chunks = (D + 31) / 32, per = (chunks + ctas - 1) / ctas, c1 = min(chunks, (share + 1) * per);
    const int rank0 = warp % HALVES * MR * 16, ranks = p.rank - rank0;
    const T* a = static_cast<const T*>(p.a) + ((int64_t)tile.l * p.rank + rank0) * D;
    const T* x[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) x[j] = tok[j] >= 0 ? static_cast<const T*>(p.x) + (int64_t)tok[j] * D : nullptr;
    float c[MR][TN][4] = {};
    for (int chunk = share * per + warp / HALVES; chunk < c1; chunk += kSlices * DEEP) {
      uint4 b[DEEP][TN], lo[DEEP][MR], hi[DEEP][MR];
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        const int k = (chunk + d * kSlices) * 32 + t * 8;
        const bool in = k < D && chunk + d * kSlices < c1;
#pragma unroll
        for (int m = 0; m < MR; ++m) {
          const int r = m * 16 + g;
          lo[d][m] = in && r < ranks ? __ldcg(reinterpret_cast<const uint4*>(a + (int64_t)r * D + k)) : zero;
          hi[d][m] = in && r + 8 < ranks ? __ldcg(reinterpret_cast<const uint4*>(a + (int64_t)(r + 8) * D + k)) : zero;
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) b[d][j] = in && x[j] ? __ldcg(reinterpret_cast<const uint4*>(x[j] + k)) : zero;
      }
#pragma unroll
      for (int d = 0; d < DEEP; ++d)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int m = 0; m < MR; ++m) mma32<T>(c[m][j], lo[d][m], hi[d][m], b[d][j]);
    }
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) s_part[((warp * MR + m) * TN + j) * 128 + q * 32 + lane] = c[m][j][q];
  }
  // a strip of 32 channels: column c of MMA j is channel 8 (c / 2) + 2 j + c % 2, so that lane (g, t)
  // holds channels 8 t .. 8 t + 7 of tokens g and g + 8
  const T* b = static_cast<const T*>(p.b) + (int64_t)tile.l * N * p.rank;
  const T* base = static_cast<const T*>(p.base);
  T* out = static_cast<T*>(p.out);
  uint4 w[4][RC], y[2];
  auto load = [&](int strip) {
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
    for (int h = 0; h < 2; ++h)
      y[h] = tok[h] >= 0 && n < N ? __ldcg(reinterpret_cast<const uint4*>(base + (int64_t)tok[h] * N + n)) : zero;
  };
  int strip = share * per_n + warp;
  if (strip < last) load(strip);
  const float scale = p.scales ? __ldcg(p.scales + tile.l) : 1.0f;
  __syncthreads();
  // element q of lane (g, t): rank 16 m + g + 8 (q / 2), token 8 j + 2 t + q % 2
  for (int i = threadIdx.x; i < HALVES * MR * TN * 128; i += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < kSlices; ++u) s += s_part[u * HALVES * MR * TN * 128 + i];
    const int l = i & 31, q = (i >> 5) & 3, j = (i >> 7) % TN, m = (i >> 7) / TN;
    s_sum[j * 8 + 2 * (l & 3) + (q & 1)][m * 16 + (l >> 2) + 8 * (q >> 1)] = s;
  }
  __syncwarp();
  cluster_sync_all();
#pragma unroll
  for (int k = 0; k < kFewTokens / kWarps; ++k) {
    const int i = warp + k * kWarps;
    float v[RC];
#pragma unroll
    for (int q = 0; q < RC; ++q) {
      v[q] = 0.0f;
      if (q * 32 + lane < p.rank)  // those behind are 0 times x, NaN where x is not finite
        for (int u = 0; u < ctas; ++u) v[q] += ld_cluster(cluster_addr(&s_sum[i][q * 32 + lane], u));
      v[q] *= scale;
    }
    const float f = split_ranks<T, RC>(v, s_hi + i * kPitch, s_lo + i * kPitch, lane);
    if (lane == 0) s_pow[i] = f;
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // done with the other CTAs' sums
  __syncthreads();
  while (strip < last) {
    const int n = strip * 32 + t * 8;
    float c[4][4] = {};
#pragma unroll
    for (int q = 0; q < RC; ++q) {
      const int s = g * kPitch + q * 32 + t * 8;
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
      if (tok[h] >= 0 && n < N)
        *reinterpret_cast<uint4*>(out + (int64_t)tok[h] * N + n) = add_base<T>(y[h], c, h, s_pow[g + 8 * h]);
    strip += kWarps;
    if (strip < last) load(strip);
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // no CTA leaves before the others have read its sums
}

// Many tokens to an adapter: 64, 16 to each of four groups of two warps, which keep their rank values in
// registers; base and the adapter's rows of b pass through a ring in shared memory, 64 channels a stage,
// 32 to a warp.  The rows of b lie there in the order of the MMAs' columns (a row of eight MMA columns after the
// other, 16 bytes past a multiple of 32).
template <typename T, int RK>  // RK x 16 ranks
__global__ void __launch_bounds__(kThreads) lora16_expand_many_kernel(const Lora16Problem p, int splits, int shares) {
  constexpr int RC = (RK + 1) / 2, kPitch = RC * 32 + 8, kRow = RK * 32 + 16;
  constexpr int kBase = kManyTokens * 128, kStage = kBase + 64 * kRow, kStages = kStagesOf<RK>;
  extern __shared__ __align__(128) uint8_t s_mem[];  // the ring, then hi and lo of the rank values
  __shared__ float s_pow[kManyTokens];
  __shared__ int s_tok[kManyTokens];
  T* s_hi = reinterpret_cast<T*>(s_mem + kStages * kStage);
  T* s_lo = s_hi + kManyTokens * kPitch;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int share = blockIdx.x % shares, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Tile tile = find_tile<kManyTokens, kThreads>(blockIdx.x / shares, p.cumsum, p.L, p.M);
  const int N = p.N, strips = (N + 63) / 64, per = (strips + shares - 1) / shares;
  const int first = share * per, n = max(0, min(strips - first, per));
  if (threadIdx.x < kManyTokens) {
    const int tok = (int)threadIdx.x < tile.rows ? __ldcg(p.route + tile.start + threadIdx.x) : -1;
    s_tok[threadIdx.x] = (unsigned)tok < (unsigned)p.M ? tok : -1;
  }
  __syncthreads();
  if (tile.rows == 0 || tile.l < 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tile.rows && p.base != p.out)
      copy_base<T, kThreads>(p, s_tok, tile.rows, first * 64, min(N, (first + n) * 64));
    return;
  }
  const float scale = p.scales ? __ldcg(p.scales + tile.l) : 1.0f;
  const T* b = static_cast<const T*>(p.b) + (int64_t)tile.l * N * p.rank;
  const T* base = static_cast<const T*>(p.base);
  T* out = static_cast<T*>(p.out);
  const uint32_t ring = smem_u32(s_mem);
  // this thread's pieces of a stage: two of base (rows 32 apart, piece c of a row at c ^ (row % 8)) and
  // kB of b, whose channel 8 (c / 2) + 2 j + c % 2 of 32 is column c of MMA j
  constexpr int kB = (RK * 128 + kThreads - 1) / kThreads;
  const int row = threadIdx.x >> 3, piece = threadIdx.x & 7;
  const T *from[2], *bfrom[kB];
  uint32_t to[2], bto[kB];
  int ch[kB];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int tok = s_tok[row + 32 * k];
    from[k] = tok >= 0 ? base + (int64_t)tok * N + first * 64 + piece * 8 : nullptr;
    to[k] = ring + (row + 32 * k) * 128 + ((piece ^ (row & 7)) << 4);
  }
#pragma unroll
  for (int k = 0; k < kB; ++k) {
    const int at = k * kThreads + threadIdx.x, c = at / (RK * 2), q = at % (RK * 2);
    const int r = (c & 32) + ((c >> 1) & 3) * 8 + ((c >> 3) & 3) * 2 + (c & 1);
    ch[k] = at < RK * 128 && q * 8 < p.rank ? first * 64 + c : N;  // N and past it: zeros
    bfrom[k] = b + (int64_t)(first * 64 + c) * p.rank + q * 8;
    bto[k] = ring + kBase + r * kRow + q * 16;
  }
  auto load = [&](int i, int stage) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool in = from[k] && (first + i) * 64 + piece * 8 < N;
      copy16(to[k] + stage * kStage, in ? from[k] + i * 64 : base, in);
    }
#pragma unroll
    for (int k = 0; k < kB; ++k) {
      const bool in = ch[k] + i * 64 < N;
      if (RK > 1 || threadIdx.x < 128) copy16(bto[k] + stage * kStage, in ? bfrom[k] + (int64_t)i * 64 * p.rank : b, in);
    }
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (s < n) load(s, s);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const int tg = warp >> 1, half = warp & 1;
  const int tok[2] = {s_tok[tg * 16 + g], s_tok[tg * 16 + g + 8]};
  T* outs[2] = {out + (int64_t)tok[0] * N, out + (int64_t)tok[1] * N};  // written where tok >= 0
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i0 = warp; i0 < kManyTokens; i0 += 4 * kWarps) {
    float v[4][RC];
    load_ranks<RC, 4, kWarps>(p, splits, tile, i0, scale, lane, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * kWarps;
      const float f = split_ranks<T, RC>(v[k], s_hi + i * kPitch, s_lo + i * kPitch, lane);
      if (lane == 0) s_pow[i] = f;
    }
  }
  __syncthreads();
  uint32_t hi[RK][4], lo[RK][4];
  {
    const int at = (tg * 16 + (lane & 15)) * kPitch + (lane >> 4) * 8;
#pragma unroll
    for (int k = 0; k < RK; ++k) {
      ldmatrix4(hi[k], smem_u32(s_hi + at + k * 16));
      ldmatrix4(lo[k], smem_u32(s_lo + at + k * 16));
    }
  }
  const float f[2] = {s_pow[tg * 16 + g], s_pow[tg * 16 + g + 8]};
  const uint32_t brow = (half * 32 + (lane >> 4) * 8 + (lane & 7)) * kRow + ((lane >> 3) & 1) * 16;
  for (int i = 0; i < n; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncthreads();  // the stage has landed for all, and all are done with the one that is filled next
    if (i + kStages - 1 < n) load(i + kStages - 1, (i + kStages - 1) % kStages);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const uint32_t st = ring + (i % kStages) * kStage + kBase + brow;
    const uint8_t* ys = s_mem + (i % kStages) * kStage;
    float c[4][4] = {};
#pragma unroll
    for (int k = 0; k < RK; ++k) {
      uint32_t w[2][4];
      ldmatrix4(w[0], st + k * 32);
      ldmatrix4(w[1], st + 16 * kRow + k * 32);
#pragma unroll
      for (int j = 0; j < 4; ++j) mma16<T>(c[j], lo[k], w[j >> 1][2 * (j & 1)], w[j >> 1][2 * (j & 1) + 1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) mma16<T>(c[j], hi[k], w[j >> 1][2 * (j & 1)], w[j >> 1][2 * (j & 1) + 1]);
    }
    const int ch = (first + i) * 64 + half * 32 + t * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (tok[h] >= 0 && ch < N) {
        const uint4 y = *reinterpret_cast<const uint4*>(ys + (tg * 16 + g + 8 * h) * 128 + (((half * 4 + t) ^ g) << 4));
        *reinterpret_cast<uint4*>(outs[h] + ch) = add_base<T>(y, c, h, f[h]);
      }
  }
}

// Shares of D: enough blocks for the device, at most what the workspace holds, part_rows(M) rows of
// fp32 rank values in all: eight shares up to 4096 tokens, fewer above.
constexpr int kMaxSplits = 8;
inline int part_rows(int M) {
  const int many = M < 4096 ? kMaxSplits * M : kMaxSplits * 4096;
  return M > many ? M : many;
}

inline int tiles_of(int M, int groups, int tokens) { return M / tokens + (M < groups ? M : groups); }

inline int shrink_splits(const Lora16Problem& p, int tiles, int blocks, int slices) {
  int splits = (blocks + tiles - 1) / tiles;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits > part_rows(p.M) / p.M) splits = part_rows(p.M) / p.M;
  if (splits > slices) splits = slices;
  return splits < 1 ? 1 : splits;
}

// CTAs to a cluster: at most eight, as many as have work for their warps in one of the products, and as the
// device takes at once, about: half of the tiles counted on are there, and two CTAs fit
// an SM (128 tokens on 100 adapters of rank 16: eight CTAs to a tile 15.1 us, four 10.9, two 16.8).
template <typename T, int MR, int DEEP, int HALVES>
cudaError_t few(const Lora16Problem& p, cudaStream_t stream) {
  const int tiles = tiles_of(p.M, p.L + 1, kFewTokens);
  const int work = (p.D > p.N ? p.D : p.N) / (32 * kWarps) + 1;
  int ctas = 8;
  while (ctas > 1 && (tiles * ctas > 4 * sm_count() || ctas >= 2 * work)) ctas /= 2;
  const size_t smem = (size_t)kWarps * MR * 2 * 128 * 4;
  static PerContextOnce set;
  const int dev = current_device();
  if (smem > 16 * 1024 && set.needed(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(lora16_few_kernel<T, MR, DEEP, HALVES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    set.done(dev);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = (unsigned)ctas;
  attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, lora16_few_kernel<T, MR, DEEP, HALVES>, p, ctas);
}

template <typename T, int MR>
cudaError_t shrink_many(const Lora16Problem& p, int& splits, cudaStream_t stream) {
  const int tiles = tiles_of(p.M, p.L, kManyTokens);
  splits = shrink_splits(p, tiles, 3 * sm_count(), (p.D + 255) / 256);
  const size_t smem = (size_t)kStagesOf<MR> * (kManyTokens + MR * 16) * 128;
  static PerContextOnce set;
  const int dev = current_device();
  if (set.needed(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(lora16_shrink_many_kernel<T, MR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    set.done(dev);
  }
  return launch_dependent(lora16_shrink_many_kernel<T, MR>, (unsigned)(tiles * splits), kThreads, smem, stream, p, splits);
}

template <typename T, int RK>
cudaError_t expand_many(const Lora16Problem& p, int splits, cudaStream_t stream) {
  constexpr int RC = (RK + 1) / 2;
  const int tiles = tiles_of(p.M, p.L + 1, kManyTokens), strips = (p.N + 63) / 64;
  // two blocks fit an SM; as many as fill one wave, with adapters' last tiles half full
  const int likely = p.M / kManyTokens + (p.M < p.L ? p.M : p.L) / 2 + 1;
  int shares = 2 * sm_count() / likely;
  if (shares > (strips + 3) / 4) shares = (strips + 3) / 4;
  if (shares < 1) shares = 1;
  const int smem = kStagesOf<RK> * (kManyTokens * 128 + 64 * (RK * 32 + 16)) + 2 * kManyTokens * (RC * 32 + 8) * 2;
  static PerContextOnce set;
  const int dev = current_device();
  if (smem > 48 * 1024 && set.needed(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(lora16_expand_many_kernel<T, RK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    set.done(dev);
  }
  return launch_dependent(lora16_expand_many_kernel<T, RK>, (unsigned)(tiles * shares), kThreads, (size_t)smem, stream, p,
                          splits, shares);
}

template <typename T>
cudaError_t launch(const Lora16Problem& p, cudaStream_t stream) {
  if (p.M <= 16 * p.L)  // few tokens to an adapter
    return p.rank <= 16   ? few<T, 1, 4, 1>(p, stream)
           : p.rank <= 32 ? few<T, 2, 4, 1>(p, stream)
           : p.rank <= 64 ? few<T, 4, 2, 1>(p, stream)
                          : few<T, 4, 2, 2>(p, stream);
  int splits = 1;
  cudaError_t e;
  if (p.rank <= 16) {
    e = shrink_many<T, 1>(p, splits, stream);
    return e != cudaSuccess ? e : expand_many<T, 1>(p, splits, stream);
  }
  if (p.rank <= 32) {
    e = shrink_many<T, 2>(p, splits, stream);
    return e != cudaSuccess ? e : expand_many<T, 2>(p, splits, stream);
  }
  if (p.rank <= 64) {
    e = shrink_many<T, 4>(p, splits, stream);
    return e != cudaSuccess ? e : expand_many<T, 4>(p, splits, stream);
  }
  e = shrink_many<T, 8>(p, splits, stream);
  return e != cudaSuccess ? e : expand_many<T, 8>(p, splits, stream);
}

}  // namespace

size_t lora16_workspace_bytes(int M, int rank) { return (size_t)part_rows(M) * rank * 4; }

cudaError_t launch_lora16(const Lora16Problem& p, cudaStream_t stream) {
  return p.bf16 ? launch<__nv_bfloat16>(p, stream) : launch<__half>(p, stream);
}

}  // namespace moe
