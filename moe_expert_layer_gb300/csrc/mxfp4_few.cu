// The MXFP4 expert layer for a few tokens (include/moe_mxfp4.h) in two kernels:
//   1. gate and up products of every route, SwiGLU, h as MXFP4 rows by route;
//   2. the down products of every route, weighted and summed into the tokens' outputs.
// Up to 32 tokens and 256 routes the layer's time is that of the active experts' weights
// streaming past (17408 bytes per 128 channels x 256 reduction steps), so everything else is
// done beside that stream: each CTA makes the routes' tables itself, x is quantised (and h
// gathered) a 256-deep stage at a time straight into the MMA's operand, and no row is
// dispatched or permuted in memory.
//
// Both kernels are persistent, one CTA per SM, on the same pipeline: warp 0 copies weight
// blocks; warps 4-7 in turn put a stage's weight scales in order and write its token rows;
// warp 1 copies the scales to tensor memory and issues the MMAs, weight channels as rows,
// up to 16 routes of one expert as columns; warps 8-11 take the sums.
//   - Kernel 1 deals out (expert tile, 128-channel block) units.
//   - Kernel 2 cuts the sequence (output block, expert tile, stage) into equal runs of
//     stages, one per CTA: a run's sums add up in shared memory over experts and stages
//     alike.  Where several runs meet in an output block each leaves its sum in the
//     workspace, and the CTA that finishes last adds them in order of the runs.
// Kernel 2 is launched as a programmatic dependent of kernel 1: its CTAs fit beside kernel
// 1's, and its weights are on their way while kernel 1 still runs.
// Every wait is bounded, as in the grouped product.
#include "mx_tc.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kThreads = 384;
constexpr int kWeightWarp = 0, kMmaWarp = 1, kPrepWarp0 = 4, kPrepWarps = 4, kEpiWarp0 = 8;
constexpr int kRows = 16;                                  // routes per tile: the MMA's columns
constexpr int kTokens = kMxBlockBytes;                     // of a stage: the token rows' codes
constexpr int kTokenScales = kTokens + kRows * 128;        // and their scale words, arranged
constexpr int kStageBytes = kTokenScales + 2 * 512;
constexpr int kStages = 5, kSfStages = 4;
constexpr int kSfCols = 16, kSf0 = 2 * kRows, kTmemCols = 128;
static_assert(kStageBytes % 1024 == 0 && kTokens % 1024 == 0, "swizzled rows");
static_assert(kSf0 + kSfStages * kSfCols <= kTmemCols && kSfStages < kStages, "tensor memory");
static_assert(kMxFewRoutes <= 256 && kMxFewRoutes <= kThreads, "a route per thread");

// Shared memory behind the ring: the experts' counts while the tables are made, then kernel
// 1's exchange or kernel 2's output sums.
constexpr int kScratchBytes = 4096;
inline int scratch_bytes(bool down, int M) { return down && M * 512 > kScratchBytes ? M * 512 : kScratchBytes; }
inline int smem_bytes(bool down, int M) { return kStages * kStageBytes + scratch_bytes(down, M) + 1024; }

struct FewArgs {
  int M, K, I, E, topK, R;
  int N, D, KB, NB;            // this kernel's product: channels, depth, stages, blocks
  const __half* x;
  const int32_t* expert_idx;
  const float* probs;
  const uint8_t* w;
  uint8_t* h_codes;            // [R][I / 2]
  uint8_t* h_scales;           // [R][4 * planes(I)]
  float* part;                 // [CTA][2][M][128]
  int32_t* counters;           // [K / 128]
  __half* out;
  int32_t* status;
};

struct Tables {
  int list[kMxFewRoutes];      // routes by expert
  int tile_e[kMxFewRoutes];    // expert tiles: expert,
  int tile_row[kMxFewRoutes];  // first row (of list) | rows << 16
  float prob[kMxFewRoutes];
  int tiles;
};

// A run of stages of one (block, tile): what one accumulation covers.
struct Seg {
  int nb, tile, kb0, kb1;
};

// The runs of kernel 2 (one per CTA, none empty) and where one begins.
__device__ __forceinline__ int runs_of(int64_t total) { return (int)min((int64_t)gridDim.x, total); }
__device__ __forceinline__ int64_t run_begin(int c, int64_t total) { return total * c / max(runs_of(total), 1); }

// The segments of a CTA, in order.
template <bool DOWN>
struct Walk {
  int64_t at, end;
  int step, tiles, NB, KB;
  __device__ __forceinline__ Walk(const FewArgs& a, int tiles_) : tiles(tiles_), NB(a.NB), KB(a.KB) {
    if (DOWN) {
      const int64_t total = (int64_t)NB * tiles * KB;
      const int c = min((int)blockIdx.x, runs_of(total));
      at = run_begin(c, total);
      end = run_begin(min((int)blockIdx.x + 1, runs_of(total)), total);
      step = 0;
    } else {
      at = blockIdx.x;
      end = (int64_t)tiles * NB;
      step = gridDim.x;
    }
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (at >= end) return false;
    if (DOWN) {
      const int per = tiles * KB;
      s.nb = (int)(at / per);
      const int rem = (int)(at - (int64_t)s.nb * per);
      s.tile = rem / KB;
      s.kb0 = rem - s.tile * KB;
      s.kb1 = (int)min((int64_t)KB, s.kb0 + (end - at));
      at += s.kb1 - s.kb0;
    } else {
      s.tile = (int)(at / NB);
      s.nb = (int)(at - (int64_t)s.tile * NB);
      s.kb0 = 0;
      s.kb1 = KB;
      at += step;
    }
    return true;
  }
};

// The routes by expert, in order of the routes, and the tiles of up to 16 of them.
__device__ __forceinline__ void make_tables(const FewArgs& a, Tables& t, int* count, int* wsum) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < a.E; e += kThreads) count[e] = 0;
  __syncthreads();
  int e = -1, pos = 0;
  if (tid < a.R) {
    e = __ldg(a.expert_idx + tid);
    if (e < 0 || e >= a.E) e = -1;
    t.prob[tid] = __ldg(a.probs + tid);
  }
  // a warp at a time, so that an expert's routes keep their order
  for (int w = 0; w * 32 < a.R; ++w) {
    if (warp == w) {
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      if (e >= 0) pos = count[e] + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (e >= 0 && (same >> lane) == 1u) count[e] += __popc(same);
    }
    __syncthreads();
  }
  // first row and first tile of each expert: a scan of rows | tiles << 16
  const int per = (a.E + kThreads - 1) / kThreads;
  const int e0 = min(a.E, tid * per), e1 = min(a.E, e0 + per);
  int sum = 0;
  for (int i = e0; i < e1; ++i) sum += count[i] | ((count[i] + kRows - 1) / kRows) << 16;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < warp; ++w) run += wsum[w];
  for (int i = e0; i < e1; ++i) {
    const int c = count[i], n = (c + kRows - 1) / kRows, row = run & 0xffff, tile = run >> 16;
    for (int k = 0; k < n; ++k) {
      t.tile_e[tile + k] = i;
      t.tile_row[tile + k] = (row + k * kRows) | min(kRows, c - k * kRows) << 16;
    }
    count[i] = row;
    run += c | n << 16;
  }
  if (e0 < a.E && e1 == a.E) t.tiles = run >> 16;
  __syncthreads();
  if (e >= 0) t.list[count[e] + pos] = tid;
  __syncthreads();
}

// One 256-deep stage of a tile's rows, from x: eight elements to a lane, four lanes to a
// scaled block, a row per pass.
__device__ __forceinline__ void put_x_rows(const FewArgs& a, const Tables& t, uint8_t* st, int row0, int rows, int kb,
                                           int lane, const uint4 (&pre)[4]) {
  const int k = kb * 256 + lane * 8;
  for (int c = 0; c < rows; ++c) {
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (c < 4) {
      raw = c == 0 ? pre[0] : c == 1 ? pre[1] : c == 2 ? pre[2] : pre[3];
    } else if (k < a.K) {
      raw = __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)(t.list[row0 + c] / a.topK) * a.K + k));
    }
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
    float v[8];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
      amax = max(amax, max(abs_bits(f.x), abs_bits(f.y)));
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t b = mx_scale_byte(amax);
    const float mult = mx_multiplier(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mx_scaled(v[i], mult, b);
    const int chunk = lane >> 2;
    *reinterpret_cast<uint32_t*>(st + kTokens + mx_chunk_at(c, chunk) + (lane & 3) * 4) = mx_codes8(v);
    if ((lane & 3) == 0) st[kTokenScales + (chunk >> 2) * 512 + c * 16 + (chunk & 3)] = (uint8_t)b;
  }
}

// Whether `ok` holds in all four epilogue warps (named barrier 1).
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// The CTA of kernel 2 whose run holds stage `at` of `total`.
__device__ __forceinline__ int run_of(int64_t at, int64_t total) {
  int c = (int)(at * runs_of(total) / total);
  while (run_begin(c + 1, total) <= at) ++c;
  while (run_begin(c, total) > at) --c;
  return c;
}

template <bool DOWN>
__global__ void __launch_bounds__(kThreads, 1) mx_few_kernel(const FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages], sf_bar[kStages], accfull_bar[2],
      accempty_bar[2], final_bar;
  __shared__ Tables s_t;
  __shared__ int s_wsum[kThreads / 32];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_issued, s_last;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  volatile int* abort_flag = &s_abort;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* ring_g = smem_raw + (ring - smem_u32(smem_raw));
  uint8_t* scratch = ring_g + kStages * kStageBytes;

  if (!DOWN) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    s_abort = 0;
    s_issued = 0;
  }
  if (!DOWN && blockIdx.x == 0) {  // what kernel 2 counts with, and the status word
    for (int i = threadIdx.x; i < a.K / 128; i += kThreads) a.counters[i] = 0;
    if (threadIdx.x == 0) *a.status = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc<false, kTmemCols>(&s_tmem);
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        mbar_init(&full_bar[s], 1);
        mbar_init(&empty_bar[s], 1);
        mbar_init(&sf_bar[s], 1);
      }
      for (int s = 0; s < 2; ++s) {
        mbar_init(&accfull_bar[s], 1);
        mbar_init(&accempty_bar[s], 4);
      }
      mbar_init(&final_bar, 1);
      fence_barrier_init();
    }
    __syncwarp();
    tc_fence_before();
  }
  make_tables(a, s_t, reinterpret_cast<int*>(scratch), s_wsum);
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int tiles = s_t.tiles;

  if (warp == kWeightWarp) {
    const uint32_t elected = elect_one();
    Walk<DOWN> walk(a, tiles);
    Seg s;
    RingPos at;
    int n = 0;
    bool ok = true;
    while (ok && walk.next(s)) {
      const uint8_t* wb = a.w + ((size_t)s_t.tile_e[s.tile] * a.NB + s.nb) * (size_t)a.KB * kMxBlockBytes;
      for (int kb = s.kb0; kb < s.kb1; ++kb, ++n, at.next(kStages)) {
        if (!(ok = warp_wait(&empty_bar[at.slot], at.phase ^ 1u, abort_flag, a.status))) break;
        const uint32_t bar = smem_u32(&full_bar[at.slot]);
        expect_tx_elect(elected, bar, kMxBlockBytes);
        bulk_load_elect(elected, ring + at.slot * kStageBytes, wb + (size_t)kb * kMxBlockBytes, kMxBlockBytes, bar);
      }
    }
    if (lane == 0) s_issued = n;
  } else if (warp == kMmaWarp) {
    const uint32_t elected = elect_one(), t0 = __shfl_sync(0xffffffffu, tmem, 0), idesc = mx_idesc(128, kRows);
    Walk<DOWN> walk(a, tiles);
    Seg s;
    RingPos at, sf;
    int u = 0;
    bool ok = true;
    const int last = (a.D - (a.KB - 1) * 256 + 127) >> 7;  // 128-deep halves of the last stage
    while (ok && walk.next(s)) {
      const int buf = u & 1;
      if (!(ok = warp_wait(&accempty_bar[buf], ((u >> 1) & 1) ^ 1, abort_flag, a.status))) break;
      tc_fence_after();
      const uint32_t d = t0 + buf * kRows;
      for (int kb = s.kb0; kb < s.kb1; ++kb, at.next(kStages), sf.next(kSfStages)) {
        if (!(ok = warp_wait(&sf_bar[at.slot], at.phase, abort_flag, a.status))) break;
        tc_fence_after();
        const uint32_t st = ring + at.slot * kStageBytes, t_sf = t0 + kSf0 + sf.slot * kSfCols;
        const uint64_t da = sw128_desc(st), db = sw128_desc(st + kTokens);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          mx_copy_scales<false>(elected, t_sf + 4 * q, st + kMxCodeBytes + 512 * q);
          mx_copy_scales<false>(elected, t_sf + 8 + 4 * q, st + kTokenScales + 512 * q);
        }
        mx_mma2<false>(elected, d, da, db, 0, idesc, t_sf, t_sf + 8, kb > s.kb0 ? 1u : 0u);
        if (kb < a.KB - 1 || last == 2) mx_mma2<false>(elected, d, da, db, 1, idesc, t_sf + 4, t_sf + 12, 1u);
        mx_commit<false>(elected, smem_u32(&empty_bar[at.slot]));
      }
      if (ok) mx_commit<false>(elected, smem_u32(&accfull_bar[buf]));
      ++u;
    }
    mx_commit<false>(elected, smem_u32(&final_bar));  // every MMA done before tensor memory is freed
    mbar_wait_sleep_bounded(&final_bar, 0);
  } else if (warp >= kPrepWarp0 && warp < kPrepWarp0 + kPrepWarps) {
    if (DOWN) asm volatile("griddepcontrol.wait;" ::: "memory");  // h is kernel 1's
    Walk<DOWN> walk(a, tiles);
    Seg s;
    RingPos at, old;  // old: the stage kSfStages before
    int n = 0;
    bool ok = true;
    while (ok && walk.next(s)) {
      const int row0 = s_t.tile_row[s.tile] & 0xffff, rows = s_t.tile_row[s.tile] >> 16;
      for (int kb = s.kb0; kb < s.kb1; ++kb, ++n, at.next(kStages)) {
        if (n > kSfStages) old.next(kStages);
        if (n % kPrepWarps != warp - kPrepWarp0) continue;
        uint4 pre[4];
        uint32_t words = 0;
        if (DOWN) {  // lane: rows lane / 8 + 4 i, 16-byte chunk lane % 8; one scale word
          const int chunk = kb * 8 + (lane & 7), planes = (a.I + 127) / 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = (lane >> 3) + 4 * i;
            pre[i] = c < rows && chunk * 32 < a.I
                         ? __ldcg(reinterpret_cast<const uint4*>(a.h_codes + (size_t)s_t.list[row0 + c] * (a.I / 2) +
                                                                 chunk * 16))
                         : make_uint4(0, 0, 0, 0);
          }
          const int c = lane & 15, plane = 2 * kb + (lane >> 4);
          if (c < rows && plane < planes)
            words = __ldcg(reinterpret_cast<const uint32_t*>(a.h_scales) + (size_t)s_t.list[row0 + c] * planes + plane);
        } else {
          const int k = kb * 256 + lane * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            pre[i] = i < rows && k < a.K
                         ? __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)(s_t.list[row0 + i] / a.topK) * a.K + k))
                         : make_uint4(0, 0, 0, 0);
        }
        // The stage that used the scale columns is done, and with it the slot's previous use: only
        // then is full_bar known to be in this use's phase (copies complete in any order).
        if (n >= kSfStages && !(ok = warp_wait(&empty_bar[old.slot], old.phase, abort_flag, a.status))) break;
        uint8_t* st = ring_g + at.slot * kStageBytes;
        if (DOWN) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(st + kTokens + mx_chunk_at((lane >> 3) + 4 * i, lane & 7)) = pre[i];
          *reinterpret_cast<uint32_t*>(st + kTokenScales + (lane >> 4) * 512 + (lane & 15) * 16) = words;
        } else {
          put_x_rows(a, s_t, st, row0, rows, kb, lane, pre);
        }
        if (!(ok = warp_wait(&full_bar[at.slot], at.phase, abort_flag, a.status))) break;
        const uint4 w0 = mx_scale_words(st + kMxCodeBytes, lane), w1 = mx_scale_words(st + kMxCodeBytes + 512, lane);
        __syncwarp();
        mx_put_scale_words(st + kMxCodeBytes, w0, lane);
        mx_put_scale_words(st + kMxCodeBytes + 512, w1, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_bar[at.slot]);
      }
    }
  } else if (warp >= kEpiWarp0) {
    const int quarter = warp & 3, ch = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)quarter << 21;
    Walk<DOWN> walk(a, tiles);
    Seg s;
    int u = 0;
    float* sums = reinterpret_cast<float*>(scratch);  // kernel 2: [M][128]
    if (DOWN) {
      for (int t = 0; t < a.M; ++t) sums[t * 128 + ch] = 0.0f;
      if (tiles == 0)  // no route at all
        for (int nb = blockIdx.x; nb < a.NB; nb += gridDim.x)
          for (int t = 0; t < a.M; ++t) a.out[(size_t)t * a.K + nb * 128 + ch] = __float2half(0.0f);
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are kernel 1's
    }
    const int64_t begin = walk.at;
    while (walk.next(s)) {
      const int row0 = s_t.tile_row[s.tile] & 0xffff, rows = s_t.tile_row[s.tile] >> 16, buf = u & 1;
      const bool ok = epi_all(warp_wait(&accfull_bar[buf], (u >> 1) & 1, abort_flag, a.status));
      if (!ok) break;
      tc_fence_after();
      __syncwarp();
      uint32_t v[16];
      tmem_ld16(tmem + lanes + buf * kRows, v);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&accempty_bar[buf]);
      ++u;
      if (!DOWN) {
        // warps in pairs, 32 gate channels and the 32 up channels that multiply them: of 16
        // rows each warp finishes 8, with the other's half through shared memory
        const int pair = quarter >> 1, odd = quarter & 1;
        float* give = reinterpret_cast<float*>(scratch) + pair * 512 + odd * 256 + lane;
        const float* take = reinterpret_cast<float*>(scratch) + pair * 512 + (odd ^ 1) * 256 + lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) give[i * 32] = __uint_as_float(odd ? v[i] : v[8 + i]);
        asm volatile("bar.sync %0, 64;" ::"r"(2 + pair) : "memory");
        float h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = take[i * 32];
          h[i] = odd ? mx_swiglu(o, __uint_as_float(v[8 + i])) : mx_swiglu(__uint_as_float(v[i]), o);
        }
        asm volatile("bar.sync %0, 64;" ::"r"(2 + pair) : "memory");  // both have taken
        uint32_t byte;
        const uint32_t w = mx_quant_rows8(h, lane, byte);
        const int c = odd * 8 + (lane & 7);
        if (c < rows) {
          const int r = s_t.list[row0 + c], k = s.nb * 2 + pair, planes = (a.I + 127) / 128;
          *reinterpret_cast<uint32_t*>(a.h_codes + (size_t)r * (a.I / 2) + k * 16 + (lane >> 3) * 4) = w;
          if (lane < 8) {
            uint8_t* sc = a.h_scales + (size_t)r * planes * 4 + k;
            *sc = (uint8_t)byte;
            if (k == a.I / 32 - 1)  // bytes of the word past the last block
              for (int z = 1; (k + z) & 3; ++z) sc[z] = 0;
          }
        }
        __syncwarp();
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < rows) {
            const int r = s_t.list[row0 + i];
            float* o = sums + (r / a.topK) * 128 + ch;
            *o = fmaf(s_t.prob[r], __uint_as_float(v[i]), *o);
          }
        if (walk.at < walk.end && (s.tile < tiles - 1 || s.kb1 < a.KB)) continue;
        // the run's share of this output block is complete
        const int64_t per = (int64_t)tiles * a.KB, total = per * a.NB, b0 = s.nb * per, b1 = b0 + per;
        const bool whole = begin <= b0 && walk.end >= b1;
        bool write = whole;
        int c0 = 0, c1 = 0;
        if (!whole) {
          float* part = a.part + ((size_t)blockIdx.x * 2 + (s.nb != (int)(begin / per))) * a.M * 128;
          for (int t = 0; t < a.M; ++t) __stcg(part + t * 128 + ch, sums[t * 128 + ch]);
          c0 = run_of(b0, total);
          c1 = run_of(b1 - 1, total);
          __threadfence();
          asm volatile("bar.sync 1, 128;" ::: "memory");
          if (warp == kEpiWarp0 && lane == 0) s_last = atomicAdd(a.counters + s.nb, 1) == c1 - c0;
          asm volatile("bar.sync 1, 128;" ::: "memory");
          write = s_last != 0;
          if (write) __threadfence();
        }
        for (int t = 0; t < a.M; ++t) {
          float acc = sums[t * 128 + ch];
          if (!whole && write) {
            acc = 0.0f;
            for (int c = c0; c <= c1; ++c)
              acc += __ldcg(a.part + ((size_t)c * 2 + (s.nb != (int)(run_begin(c, total) / per))) * a.M * 128 +
                            t * 128 + ch);
          }
          if (write) a.out[(size_t)t * a.K + s.nb * 128 + ch] = from_f32<__half>(acc);
          sums[t * 128 + ch] = 0.0f;
        }
      }
    }
  }

  __syncthreads();
  if (threadIdx.x == 0) {  // copies still in flight (only after an abort) land before shared memory is released
    const int n1 = s_issued;
    for (int n = max(0, n1 - kStages); n < n1; ++n) mbar_wait_bounded(&full_bar[n % kStages], (n / kStages) & 1);
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<false, kTmemCols>(tmem);
  }
}

}  // namespace

size_t mx_few_part_bytes(int M, int K) {
  (void)K;
  return (size_t)sm_count() * 2 * M * 128 * 4;
}

cudaError_t launch_mx_few(const MxFewProblem& p, cudaStream_t stream) {
  static PerContextOnce set;
  const int dev = current_device();
  if (set.needed(dev)) {
    cudaError_t e = cudaFuncSetAttribute(mx_few_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes(false, kMxFewTokens));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(mx_few_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               smem_bytes(true, kMxFewTokens));
    if (e != cudaSuccess) return e;
    set.done(dev);
  }
  FewArgs a;
  a.M = p.M;
  a.K = p.K;
  a.I = p.I;
  a.E = p.E;
  a.topK = p.topK;
  a.R = p.M * p.topK;
  a.N = 2 * p.I;
  a.D = p.K;
  a.KB = mx_depth_blocks(p.K);
  a.NB = p.I / 64;
  a.x = reinterpret_cast<const __half*>(p.x);
  a.expert_idx = p.expert_idx;
  a.probs = p.probs;
  a.w = p.w1;
  a.h_codes = p.h_codes;
  a.h_scales = reinterpret_cast<uint8_t*>(p.h_scales);
  a.part = p.part;
  a.counters = p.counters;
  a.out = reinterpret_cast<__half*>(p.out);
  a.status = p.status;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sm_count());
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(false, p.M);
  cfg.stream = stream;
  cudaError_t e = cudaLaunchKernelEx(&cfg, mx_few_kernel<false>, a);
  if (e != cudaSuccess) return e;
  a.N = p.K;
  a.D = p.I;
  a.KB = mx_depth_blocks(p.I);
  a.NB = p.K / 128;
  a.w = p.w2;
  cudaLaunchAttribute after;
  after.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  after.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &after;
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = smem_bytes(true, p.M);
  return cudaLaunchKernelEx(&cfg, mx_few_kernel<true>, a);
}

}  // namespace moe
