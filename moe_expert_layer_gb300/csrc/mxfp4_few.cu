// The MXFP4 expert layer for a few tokens (include/moe_mxfp4.h) in two kernels:
//   1. x as MXFP4 rows, and the counters of the second kernel cleared;
//   2. everything else: gate and up products of every route, SwiGLU, h as MXFP4 rows by
//      route, down products, weighted sums of the tokens' routes.
// Up to 32 tokens and 256 routes the layer's time is that of the active experts' weights
// streaming past (17408 bytes per 128 channels x 256 reduction steps), so everything else is
// done beside that stream: each CTA makes the routes' tables itself, and no row is
// dispatched or permuted in memory.
// Measured, depth 7168, 2048 channels: one token, 8 of 256 experts, 42 us, where its 187 MB take
// 28 at the measured copy rate; 8 tokens on 16 experts 66 us (55); depth 4096, 1408 channels: 29
// tokens on 64 experts 93 us (82).  The rest is the start, the wait between the two products
// for the last sums of h (its 6 stages in flight cover half of it) and the meeting at the end.
//
// Kernel 2 is persistent, one CTA per SM, with one pipeline for both products, so that the
// down projection's weights are on their way while the last of h is made: warp 0 copies weight
// blocks; warp 2 gathers the token rows and their scales, by tensor copies too (plain loads wait
// behind the ~170 KB of copies that an SM has under way); warps 4-7 in turn put a stage's scales
// in tensor-memory order; warp 1 copies those on and issues the MMAs, weight channels as rows, up
// to 16 routes of one expert as columns; warps 8-11 take the sums.
//   - Of the gate and up product's (expert tile, 128-channel block) units, in this order, the
//     first, as many as do not fill a whole round of the CTAs, are cut into one run of stages per
//     CTA: where runs meet in a unit each leaves its sums in the workspace, and the CTA that
//     finishes last adds them in order.  The others are dealt out whole, in turn, so that the
//     tiles' h come one after the other and the last of them without a meeting.  The CTA that has
//     a unit's sums does the SwiGLU and counts the unit on its tile.  Between one and two rounds
//     of units none is cut: each CTA gets one and takes its next by ticket, when it is ready to
//     load it, because the SMs do not get equal shares of the memory's rate.  (One token, 256
//     units: 45 us cut, 41.4 by tickets; 8 tokens, 512 units: 66 and 72, the last whole units
//     standing alone.)
//   - The down product's stages, in order of (output block, expert tile, stage), are cut into one
//     run per CTA, whose sums add up in shared memory over experts and stages alike and meet the
//     same way.  A run that goes over the end of a block takes the block it ends in first: the
//     tiles whose h is made last come last, and nothing waits for most of h.
// A CTA of kernel 2 waits for others' h, so all of them have to be resident, one per SM: its launch
// is cooperative, which sees to it whatever else runs, and is refused where the stream has fewer
// SMs than the device.  It cannot be a programmatic dependent too (the attribute then changes
// nothing), which costs 3.4 us a call.  Every wait is bounded, as in the grouped product.
#include "mx_tc.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kThreads = 384;
constexpr int kWeightWarp = 0, kMmaWarp = 1, kTokenWarp = 2, kScaleWarp0 = 4, kScaleWarps = 4, kEpiWarp0 = 8;
constexpr int kRows = 16;                                  // routes per tile: the MMA's columns
constexpr int kTokens = kMxBlockBytes;                     // of a stage: the token rows' codes
constexpr int kTokenScales = kTokens + kRows * 128;        // and their scales: 16 bytes a row, four rows
                                                           // to 128, as copied; then arranged
constexpr int kScaleRec = 16;                              // a row's scales of a stage: 8 bytes, padded
constexpr int kStageBytes = kTokenScales + 2 * 512;
constexpr int kStages = 6, kSfStages = 5;
constexpr int kSfCols = 16, kSf0 = 2 * kRows, kTmemCols = 256;
static_assert(kStageBytes % 1024 == 0 && kTokens % 1024 == 0, "swizzled rows");
static_assert(kSf0 + kSfStages * kSfCols <= kTmemCols && kSfStages < kStages, "tensor memory");
static_assert(kMxFewRoutes <= 256 && kMxFewRoutes <= kThreads, "a route per thread");

// Shared memory behind the ring: what the tables are made with, then the gate and up exchange,
// then the output sums.
inline int scratch_bytes(int M) { return M * 512 > 4096 ? M * 512 : 4096; }
inline int smem_bytes(int M) { return kStages * kStageBytes + scratch_bytes(M) + 1024; }

struct FewArgs {
  int M, K, I, E, topK, R;
  const int32_t* expert_idx;
  const float* probs;
  const uint8_t *w1, *w2;
  uint8_t* h_codes;            // [R][I / 2]
  uint8_t* h_scales;           // [R][stages(I)][kScaleRec]
  float* part;                 // [runs][2][rows][128] of h, [runs][2][M][128] of out
  int32_t* counters;           // [R][I / 64] runs of h blocks, [R] blocks of h, [K / 128] runs of out blocks, tickets
  __half* out;
  int32_t* status;
};

// Gathers of rows: codes, 128 bytes of a row, and scales, the stage's record.
struct FewMaps {
  CUtensorMap x_codes, x_scales, h_codes, h_scales;
};

// Where in the counters the tickets are given out: behind the others.
__host__ __device__ inline int counters_of(int M, int K, int I, int topK) {
  return M * topK * (I / 64 + 1) + K / 128 + 1;
}
__device__ __forceinline__ int ticket_at(const FewArgs& a) { return counters_of(a.M, a.K, a.I, a.topK) - 1; }

struct Tables {
  int list[kMxFewRoutes];      // routes by expert,
  int token[kMxFewRoutes];     // and their tokens
  int tile_e[kMxFewRoutes];    // expert tiles: expert,
  int tile_row[kMxFewRoutes];  // first row (of list) | rows << 16
  float prob[kMxFewRoutes];
  int tiles;
};

// A run of stages of one (block, tile): what one accumulation covers.
struct Seg {
  int nb, tile, kb0, kb1;
};

// One of the two products: its blocks of 128 channels, 256-deep stages, and the stages that are
// cut into one run per CTA: all of the down product's, those of the first `head` units of the
// gate and up product.
template <bool DOWN>
struct Product {
  int NB, KB, tiles, units, head, runs;
  bool tickets;
  int cut;  // stages in runs; times the runs below 2^32 (kMxFewStages, and 256 SMs at most)
  __device__ __forceinline__ Product(const FewArgs& a, int tiles_) {
    const int G = gridDim.x;
    tiles = tiles_;
    NB = DOWN ? a.K / 128 : a.I / 64;
    KB = ((DOWN ? a.I : a.K) + 255) / 256;
    units = NB * tiles;
    tickets = !DOWN && units >= G && units < 2 * G;
    head = DOWN ? units : tickets ? 0 : units % G;
    cut = head * KB;
    runs = min(G, cut);  // none empty
  }
  __device__ __forceinline__ int begin_of(int run) const {
    return runs ? (int)((unsigned)cut * (unsigned)min(run, runs) / (unsigned)runs) : 0;
  }
  // The run that holds stage `at`.
  __device__ __forceinline__ int run_of(int at) const {
    int c = (int)((unsigned)at * (unsigned)runs / (unsigned)cut);
    while (begin_of(c + 1) <= at) ++c;
    while (begin_of(c) > at) --c;
    return c;
  }
  // Stages of a block whose sums belong together, and the block that holds stage `at`.
  __device__ __forceinline__ int per() const { return DOWN ? tiles * KB : KB; }
  __device__ __forceinline__ int block_of(int at) const { return at / per(); }
};

// The units that a CTA has got by tickets, for its roles: its i-th (i >= 1) stands in
// unit[(i - 1) % kUnits] once phase (i - 1) / kUnits of its barrier is complete; -1 ends them.  The
// weight warp publishes them and runs a ring of stages ahead of the others at most.
constexpr int kUnits = 32;
static_assert(kUnits > kStages + 4, "no role is that many units behind another");
struct Pipe;
__device__ __forceinline__ bool wait_unit(const Pipe& pp, int i, int& unit);

// The segments of a CTA, in order: those of its run, then its whole units, the i-th by turn or by
// ticket; or for the down product those of its run behind the last block boundary in it, then
// those before.
template <bool DOWN>
struct Walk {
  const Product<DOWN>& p;
  int at, end, begin, mid, i;
  __device__ __forceinline__ Walk(const Product<DOWN>& p_) : p(p_), i(0) {
    begin = at = p.begin_of(blockIdx.x);
    mid = end = p.begin_of(blockIdx.x + 1);
    if (DOWN && end > begin) {
      const int edge = (end - 1) / p.per() * p.per();
      if (edge > begin) at = mid = edge;
    }
  }
  // unit_of(i, unit): the i-th unit's ticket; false if the CTA gives up
  template <typename F>
  __device__ __forceinline__ bool next(Seg& s, F unit_of) {
    if (at == end) {
      if (DOWN) {
        if (mid == end) return false;
        at = begin;
        end = mid;
      } else {
        int unit = p.head + blockIdx.x + i * gridDim.x;
        if (p.tickets && i && !unit_of(i, unit)) return false;
        ++i;
        if (unit < 0 || unit >= p.units) return false;
        at = unit * p.KB;
        end = at + p.KB;
      }
    }
    const int u = at / p.KB;
    s.kb0 = at - u * p.KB;
    s.tile = DOWN ? u % p.tiles : u / p.NB;
    s.nb = DOWN ? u / p.tiles : u % p.NB;
    s.kb1 = min(p.KB, s.kb0 + (end - at));
    at += s.kb1 - s.kb0;
    return true;
  }
  __device__ __forceinline__ bool next(Seg& s, const Pipe& pp) {
    return next(s, [&](int i, int& unit) { return wait_unit(pp, i, unit); });
  }
};

// The routes by expert, in order of the routes, and the tiles of up to 16 of them.  A route's
// place comes from comparing it with all the others, which as many threads share as there are for
// each route (174 routes: 3.5 us by a thread alone, which the first weights wait for); the routes
// that begin a tile are then numbered in the order of the places, by ballots.  `tmp`: 2 *
// kMxFewRoutes words.
__device__ __forceinline__ void make_tables(const FewArgs& a, Tables& t, int* tmp, int* wsum) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int e = -1;
  if (tid < a.R) {
    e = __ldcg(a.expert_idx + tid);
    if (e < 0 || e >= a.E) e = -1;
    t.prob[tid] = __ldcg(a.probs + tid);
  }
  if (tid < kMxFewRoutes) {
    tmp[tid] = e;
    tmp[kMxFewRoutes + tid] = 0;
  }
  __syncthreads();
  // counted for a route, in 10 bits each: routes of lower experts; of its own, before it; in all
  const int R32 = (a.R + 31) & ~31, share = kThreads / R32, who = tid / R32, mine = tid - who * R32;
  const int words = (a.R + 3) >> 2, per = (words + share - 1) / share;
  const int e_mine = who < share ? tmp[mine] : -1;
  if (e_mine >= 0) {
    int count = 0;
    for (int w = who * per; w < min(words, (who + 1) * per); ++w) {
      const int4 o = reinterpret_cast<const int4*>(tmp)[w];
      const int v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        count += v[k] < 0 ? 0 : v[k] < e_mine ? 1 : v[k] > e_mine ? 0 : 4 * w + k < mine ? (1 << 20) + (1 << 10) : 1 << 20;
    }
    if (count) atomicAdd(tmp + kMxFewRoutes + mine, count);
  }
  __syncthreads();
  const int count = tid < kMxFewRoutes ? tmp[kMxFewRoutes + tid] : 0;
  const int before = count >> 10 & 1023, same = count >> 20, place = (count & 1023) + before;
  __syncthreads();
  if (tid < kMxFewRoutes) tmp[kMxFewRoutes + tid] = -1;
  __syncthreads();
  if (e >= 0) {
    t.list[place] = tid;
    t.token[place] = tid / a.topK;
    if (before % kRows == 0) {  // begins a tile
      tmp[place] = place | min(kRows, same - before) << 16;
      tmp[kMxFewRoutes + place] = e;
    }
  }
  __syncthreads();
  const int first = tid < kMxFewRoutes ? tmp[kMxFewRoutes + tid] : -1;
  const uint32_t begins = __ballot_sync(0xffffffffu, first >= 0);
  if (lane == 0) wsum[warp] = __popc(begins);
  __syncthreads();
  int tile = __popc(begins & ((1u << lane) - 1u)), tiles = 0;
  for (int w = 0; w < kMxFewRoutes / 32; ++w) {
    if (w < warp) tile += wsum[w];
    tiles += wsum[w];
  }
  if (first >= 0) {
    t.tile_e[tile] = first;
    t.tile_row[tile] = tmp[tid];
  }
  if (tid == 0) t.tiles = tiles;
  __syncthreads();
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

// Barriers and shared memory of kernel 2's pipeline, and what its roles keep from product to
// product.
struct Pipe {
  uint64_t *full, *empty, *sf, *accfull, *accempty, *unit_bar;
  int* unit;
  uint32_t ring;
  uint8_t* ring_g;
  uint32_t tmem;
  volatile int* abort_flag;
  int32_t* status;
};

__device__ __forceinline__ bool wait_unit(const Pipe& pp, int i, int& unit) {
  --i;
  if (!warp_wait(&pp.unit_bar[i % kUnits], (i / kUnits) & 1, pp.abort_flag, pp.status)) return false;
  unit = *reinterpret_cast<volatile int*>(pp.unit + i % kUnits);
  return true;
}

// The same by the four epilogue warps, who wait for one another below: none goes on, and none
// gives up, alone (one that saw the CTA give up where the others still saw the unit would leave
// them at their next barrier).
__device__ __forceinline__ bool wait_unit_together(const Pipe& pp, int i, int& unit) {
  return epi_all(wait_unit(pp, i, unit));
}

template <bool DOWN>
__device__ __forceinline__ bool load_weights(const FewArgs& a, const Tables& t, const Pipe& pp, const Product<DOWN>& p,
                                             uint32_t elected, int lane, RingPos& at) {
  Walk<DOWN> walk(p);
  Seg s;
  int ticket = 0;  // of the next unit: asked for when a unit is begun, needed when it ends
  auto publish = [&](int i, int& unit) {
    unit = gridDim.x + __shfl_sync(0xffffffffu, ticket, 0);
    if (unit >= p.units) unit = -1;
    if (lane == 0) {
      *reinterpret_cast<volatile int*>(pp.unit + (i - 1) % kUnits) = unit;
      mbar_arrive(&pp.unit_bar[(i - 1) % kUnits]);
    }
    return true;
  };
  while (walk.next(s, publish)) {
    const uint8_t* wb =
        (DOWN ? a.w2 : a.w1) + ((size_t)t.tile_e[s.tile] * p.NB + s.nb) * (size_t)p.KB * kMxBlockBytes;
    for (int kb = s.kb0; kb < s.kb1; ++kb, at.next(kStages)) {
      if (!warp_wait(&pp.empty[at.slot], at.phase ^ 1u, pp.abort_flag, pp.status)) return false;
      const uint32_t bar = smem_u32(&pp.full[at.slot]);
      expect_tx_elect(elected, bar, kMxBlockBytes);
      bulk_load_elect(elected, pp.ring + at.slot * kStageBytes, wb + (size_t)kb * kMxBlockBytes, kMxBlockBytes, bar);
      if (p.tickets && kb == s.kb0) {
        if (lane == 0) ticket = atomicAdd(a.counters + ticket_at(a), 1);
      }
    }
  }
  return true;
}

template <bool DOWN>
__device__ __forceinline__ bool issue_mmas(const FewArgs& a, const Pipe& pp, const Product<DOWN>& p, uint32_t elected,
                                           RingPos& at, RingPos& sf, int& u) {
  const uint32_t t0 = __shfl_sync(0xffffffffu, pp.tmem, 0), idesc = mx_idesc(128, kRows);
  const int last = ((DOWN ? a.I : a.K) - (p.KB - 1) * 256 + 127) >> 7;  // 128-deep halves of the last stage
  Walk<DOWN> walk(p);
  Seg s;
  while (walk.next(s, pp)) {
    const int buf = u & 1;
    if (!warp_wait(&pp.accempty[buf], ((u >> 1) & 1) ^ 1, pp.abort_flag, pp.status)) return false;
    tc_fence_after();
    const uint32_t d = t0 + buf * kRows;
    for (int kb = s.kb0; kb < s.kb1; ++kb, at.next(kStages), sf.next(kSfStages)) {
      if (!warp_wait(&pp.sf[at.slot], at.phase, pp.abort_flag, pp.status)) return false;
      tc_fence_after();
      const uint32_t st = pp.ring + at.slot * kStageBytes, t_sf = t0 + kSf0 + sf.slot * kSfCols;
      const uint64_t da = sw128_desc(st), db = sw128_desc(st + kTokens);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        mx_copy_scales(elected, t_sf + 4 * q, st + kMxCodeBytes + 512 * q);
        mx_copy_scales(elected, t_sf + 8 + 4 * q, st + kTokenScales + 512 * q);
      }
      mx_mma2<false>(elected, d, da, db, 0, idesc, t_sf, t_sf + 8, kb > s.kb0 ? 1u : 0u);
      if (kb < p.KB - 1 || last == 2) mx_mma2<false>(elected, d, da, db, 1, idesc, t_sf + 4, t_sf + 12, 1u);
      mx_commit<false>(elected, smem_u32(&pp.empty[at.slot]));
    }
    mx_commit<false>(elected, smem_u32(&pp.accfull[buf]));
    ++u;
  }
  return true;
}

// Bounded wait until *count >= target, polled closely: a CTA has nothing else to do.
__device__ __forceinline__ bool ready_wait(const int32_t* count, int target) {
  for (int i = 0; i < 4096; ++i)
    if (ld_acquire(count) >= target) return true;
  return count_wait_bounded(count, target);
}

// A stage's token rows: of x by token, or of h by route once all blocks of the tile's h are there.
template <bool DOWN>
__device__ __forceinline__ bool load_tokens(const FewArgs& a, const FewMaps& maps, const Tables& t, const Pipe& pp,
                                            const Product<DOWN>& p, uint32_t elected, int lane, RingPos& at) {
  const int32_t* ready = a.counters + (size_t)a.R * (a.I / 64);
  const int* list = DOWN ? t.list : t.token;
  int seen = -1;  // the last tile whose h was waited for
  Walk<DOWN> walk(p);
  Seg s;
  while (walk.next(s, pp)) {
    if (DOWN && s.tile != seen) {
      const bool ok = *pp.abort_flag == 0 && (lane != 0 || ready_wait(ready + s.tile, a.I / 64));
      if (!__all_sync(0xffffffffu, ok)) {
        if (*pp.abort_flag == 0 && lane == 0) record_status(pp.status, MOE_ERR_TIMEOUT);
        *pp.abort_flag = 1;
        return false;
      }
      // what lane 0 has acquired, for the lane that issues the copies too: a vote orders no memory
      __syncwarp();
      fence_proxy_async_global();
      seen = s.tile;
    }
    const int row0 = t.tile_row[s.tile] & 0xffff, last = (t.tile_row[s.tile] >> 16) - 1, groups = (last + 4) >> 2;
    int4 y[4];
#pragma unroll
    for (int g = 0; g < 4; ++g)
      y[g] = make_int4(list[row0 + min(4 * g, last)], list[row0 + min(4 * g + 1, last)],
                       list[row0 + min(4 * g + 2, last)], list[row0 + min(4 * g + 3, last)]);
    for (int kb = s.kb0; kb < s.kb1; ++kb, at.next(kStages)) {
      if (!warp_wait(&pp.empty[at.slot], at.phase ^ 1u, pp.abort_flag, pp.status)) return false;
      const uint32_t bar = smem_u32(&pp.full[at.slot]), st = pp.ring + at.slot * kStageBytes;
      expect_tx_elect(elected, bar, groups * 4 * (128 + kScaleRec));
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (g < groups) {
          tma_gather4_elect(elected, st + kTokens + g * 512, DOWN ? &maps.h_codes : &maps.x_codes, kb * 128, y[g], bar);
          tma_gather4_elect(elected, st + kTokenScales + g * 128, DOWN ? &maps.h_scales : &maps.x_scales,
                            kb * kScaleRec, y[g], bar);
        }
    }
  }
  return true;
}

// Puts the scales of this warp's stages, every kScaleWarps-th of the CTA's, in order.  n: the
// CTA's stages before this product's, and then with them.
template <bool DOWN>
__device__ __forceinline__ bool arrange_scales(const Pipe& pp, const Product<DOWN>& p, int who, int lane, int& n) {
  Walk<DOWN> walk(p);
  Seg s;
  while (walk.next(s, pp)) {
    for (int kb = s.kb0; kb < s.kb1; ++kb, ++n) {
      if (n % kScaleWarps != who) continue;
      // The stage that used the scale columns is done, and with it the slot's previous use: only
      // then is `full` known to be in this use's phase (copies complete in any order).
      const int old = n - kSfStages, slot = n % kStages;
      if (old >= 0 && !warp_wait(&pp.empty[old % kStages], (old / kStages) & 1, pp.abort_flag, pp.status)) return false;
      if (!warp_wait(&pp.full[slot], (n / kStages) & 1, pp.abort_flag, pp.status)) return false;
      uint8_t* st = pp.ring_g + slot * kStageBytes;
      const uint4 w0 = mx_scale_words(st + kMxCodeBytes, lane), w1 = mx_scale_words(st + kMxCodeBytes + 512, lane);
      uint2 x = make_uint2(0, 0);
      if (lane < kRows)
        x = *reinterpret_cast<const uint2*>(st + kTokenScales + (lane >> 2) * 128 + (lane & 3) * kScaleRec);
      __syncwarp();
      mx_put_scale_words(st + kMxCodeBytes, w0, lane);
      mx_put_scale_words(st + kMxCodeBytes + 512, w1, lane);
      if (lane < kRows) {
        *reinterpret_cast<uint32_t*>(st + kTokenScales + lane * 16) = x.x;
        *reinterpret_cast<uint32_t*>(st + kTokenScales + 512 + lane * 16) = x.y;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pp.sf[slot]);
    }
  }
  return true;
}

// Words of the workspace that hold sums of h, two units to a run, before those of out.
__host__ __device__ inline size_t part_words_of_h(int G, int R) { return (size_t)G * 2 * (R < kRows ? R : kRows) * 128; }

// Adds one to a count of the device.
__device__ __forceinline__ int add_acq_rel(int32_t* count) {
  int before;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(count) : "memory");
  return before;
}
__device__ __forceinline__ void add_release(int32_t* count) {
  asm volatile("red.add.release.gpu.global.s32 [%0], 1;" ::"l"(count) : "memory");
}

// The epilogue warps' barrier.
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// The CTA's sums of a block are in global memory: counts its run, and returns whether all `runs`
// of the block's are there.  The first thread's addition releases and acquires; the barriers carry
// the other threads' writes and reads with it.
__device__ __forceinline__ bool last_run(int32_t* counter, int runs, bool first_thread, int* s_last) {
  epi_sync();
  if (first_thread) *s_last = add_acq_rel(counter) == runs - 1;
  epi_sync();
  return *s_last != 0;
}

// The sums of segment u: 16 columns of this lane's channel.
__device__ __forceinline__ bool take_sums(const Pipe& pp, int u, int quarter, int lane, uint32_t (&v)[16]) {
  const int buf = u & 1;
  if (!epi_all(warp_wait(&pp.accfull[buf], (u >> 1) & 1, pp.abort_flag, pp.status))) return false;
  tc_fence_after();
  __syncwarp();
  tmem_ld16(pp.tmem + ((uint32_t)quarter << 21) + buf * kRows, v);
  tmem_wait_ld();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&pp.accempty[buf]);
  return true;
}

__device__ __forceinline__ bool finish_h(const FewArgs& a, const Tables& t, const Pipe& pp, const Product<false>& p,
                                         float* xchg, int quarter, int lane, int& u, int* s_last) {
  const int pair = quarter >> 1, odd = quarter & 1, ch = quarter * 32 + lane;
  const size_t rec_pitch = (size_t)((a.I + 255) / 256) * kScaleRec;
  float* give = xchg + pair * 512 + odd * 256 + lane;
  const float* take = xchg + pair * 512 + (odd ^ 1) * 256 + lane;
  int32_t* ready = a.counters + (size_t)a.R * (a.I / 64);
  const size_t part_rows = min(kRows, a.R);
  Walk<false> walk(p);
  Seg s;
  auto unit_of = [&](int i, int& unit) { return wait_unit_together(pp, i, unit); };
  while (walk.next(s, unit_of)) {
    const int row0 = t.tile_row[s.tile] & 0xffff, rows = t.tile_row[s.tile] >> 16;
    const int block = s.tile * p.NB + s.nb, run = blockIdx.x;
    int c0 = run, c1 = run;
    if (s.kb1 - s.kb0 < p.KB) {
      c0 = p.run_of(block * p.KB);
      c1 = p.run_of(block * p.KB + p.KB - 1);
    }
    auto part_of = [&](int c) {
      return a.part + ((size_t)c * 2 + (block != p.block_of(p.begin_of(c)))) * part_rows * 128 + ch;
    };
    // The unit's last run, if the others have been counted already, reads their sums while its
    // own MMAs are under way and writes nothing.
    float sum[16] = {};
    auto add = [&](int from, int to) {  // in order; two runs' read at a time
      for (int c = from; c <= to; c += 2) {
        float o[2][16];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float* q = part_of(min(c + k, to));
#pragma unroll
          for (int i = 0; i < 16; ++i) o[k][i] = i < rows ? __ldcg(q + i * 128) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          sum[i] += o[0][i];
          if (c < to) sum[i] += o[1][i];
        }
      }
    };
    bool there = false;
    if (c1 > c0 && run == c1) {
      there = epi_all(ld_acquire(a.counters + block) == c1 - c0);
      if (there) add(c0, c1 - 1);
    }
    uint32_t v[16];
    if (!take_sums(pp, u, quarter, lane, v)) return false;
    ++u;
    if (there) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(sum[i] + __uint_as_float(v[i]));
    } else if (c1 > c0) {
      float* mine = part_of(run);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < rows) __stcg(mine + i * 128, __uint_as_float(v[i]));
      if (!last_run(a.counters + block, c1 - c0 + 1, quarter == 0 && lane == 0, s_last)) continue;
      add(c0, c1);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(sum[i]);
    }
    // warps in pairs, 32 gate channels and the 32 up channels that multiply them: of 16 rows
    // each warp finishes 8, with the other's half through shared memory
#pragma unroll
    for (int i = 0; i < 8; ++i) give[i * 32] = __uint_as_float(odd ? v[i] : v[8 + i]);
    epi_sync();
    float gate[8], up[8], h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = take[i * 32];
      gate[i] = odd ? o : __uint_as_float(v[i]);
      up[i] = odd ? __uint_as_float(v[8 + i]) : o;
    }
    mx_swiglu8(gate, up, h);
    uint32_t byte;
    const uint32_t w = mx_quant_rows8(h, lane, byte);
    const int c = odd * 8 + (lane & 7);
    if (c < rows) {
      const int r = t.list[row0 + c], k = s.nb * 2 + pair;
      *reinterpret_cast<uint32_t*>(a.h_codes + (size_t)r * (a.I / 2) + k * 16 + (lane >> 3) * 4) = w;
      if (lane < 8) {
        uint8_t* sc = a.h_scales + r * rec_pitch + (k >> 3) * kScaleRec + (k & 7);
        *sc = (uint8_t)byte;
        if (k == a.I / 32 - 1)  // bytes of the word past the last block
          for (int z = 1; (k + z) & 3; ++z) sc[z] = 0;
      }
    }
    fence_proxy_async_global();
    epi_sync();  // h is written, and the exchange free
    if (quarter == 0 && lane == 0) add_release(ready + s.tile);
  }
  return true;
}

// out of block nb from the sums of runs c0 .. c1, added in this order: every fourth token to a warp,
// four channels to a lane, and two runs' sums of all its tokens read at a time (29 tokens read one
// after the other took 12 us; four runs of two tokens, for up to 8, no less than this).
__device__ __forceinline__ void add_parts(const FewArgs& a, const Product<true>& p, const float* parts, int nb, int c0, int c1,
                                          __half* out, int quarter, int lane) {
  constexpr int kMine = kMxFewTokens / 4, kRuns = 2;
  float4 acc[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int c = c0; c <= c1; c += kRuns) {
    float4 o[kRuns][kMine];
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int run = min(c + j, c1);
      const float* q = parts + ((size_t)run * 2 + (nb != p.block_of(p.begin_of(run)))) * a.M * 128 + lane * 4;
#pragma unroll
      for (int k = 0; k < kMine; ++k)
        if (quarter + 4 * k < a.M) o[j][k] = __ldcg(reinterpret_cast<const float4*>(q + (quarter + 4 * k) * 128));
    }
#pragma unroll
    for (int j = 0; j < kRuns; ++j)
#pragma unroll
      for (int k = 0; k < kMine; ++k)
        if (c + j <= c1 && quarter + 4 * k < a.M) {
          acc[k].x += o[j][k].x;
          acc[k].y += o[j][k].y;
          acc[k].z += o[j][k].z;
          acc[k].w += o[j][k].w;
        }
  }
#pragma unroll
  for (int k = 0; k < kMine; ++k)
    if (quarter + 4 * k < a.M) {
      uint2 h;
      const __half2 lo = f2h2_sat(acc[k].x, acc[k].y), hi = f2h2_sat(acc[k].z, acc[k].w);
      h.x = *reinterpret_cast<const uint32_t*>(&lo);
      h.y = *reinterpret_cast<const uint32_t*>(&hi);
      *reinterpret_cast<uint2*>(out + (size_t)(quarter + 4 * k) * a.K + lane * 4) = h;
    }
}

__device__ __forceinline__ bool finish_out(const FewArgs& a, const Tables& t, const Pipe& pp, const Product<true>& p,
                                           float* sums, int quarter, int lane, int& u, int* s_last) {
  const int ch = quarter * 32 + lane;
  float* parts = a.part + part_words_of_h(gridDim.x, a.R);
  int32_t* counters = a.counters + (size_t)a.R * (a.I / 64) + a.R;
  Walk<true> walk(p);
  Seg s;
  for (int i = 0; i < a.M; ++i) sums[i * 128 + ch] = 0.0f;
  if (p.tiles == 0)  // no route at all
    for (int nb = blockIdx.x; nb < p.NB; nb += gridDim.x)
      for (int i = 0; i < a.M; ++i) a.out[(size_t)i * a.K + nb * 128 + ch] = __float2half(0.0f);
  while (walk.next(s, pp)) {
    uint32_t v[16];
    if (!take_sums(pp, u, quarter, lane, v)) return false;
    ++u;
    const int row0 = t.tile_row[s.tile] & 0xffff, rows = t.tile_row[s.tile] >> 16;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < rows) {
        const int r = t.list[row0 + i];
        float* o = sums + t.token[row0 + i] * 128 + ch;
        *o = fmaf(t.prob[r], __uint_as_float(v[i]), *o);
      }
    if (walk.at < walk.end && (s.tile < p.tiles - 1 || s.kb1 < p.KB)) continue;
    // the run's share of this output block is complete
    const int b0 = s.nb * p.per(), b1 = b0 + p.per();
    __half* out = a.out + s.nb * 128;
    const int c0 = p.run_of(b0), c1 = p.run_of(b1 - 1);
    if (c0 == c1) {
      for (int i = 0; i < a.M; ++i) {
        out[(size_t)i * a.K + ch] = from_f32<__half>(sums[i * 128 + ch]);
        sums[i * 128 + ch] = 0.0f;
      }
      continue;
    }
    float* part = parts + ((size_t)blockIdx.x * 2 + (s.nb != p.block_of(walk.begin))) * a.M * 128;
    for (int i = 0; i < a.M; ++i) {
      __stcg(part + i * 128 + ch, sums[i * 128 + ch]);
      sums[i * 128 + ch] = 0.0f;
    }
    if (!last_run(counters + s.nb, c1 - c0 + 1, quarter == 0 && lane == 0, s_last)) continue;
    add_parts(a, p, parts, s.nb, c0, c1, out, quarter, lane);
  }
  return true;
}

__global__ void __launch_bounds__(kThreads, 1) mx_few_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages], sf_bar[kStages], accfull_bar[2],
      accempty_bar[2], unit_bar[kUnits], final_bar;
  __shared__ int s_unit[kUnits];
  __shared__ Tables s_t;
  __shared__ int s_wsum[kThreads / 32];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_last;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  Pipe pp;
  pp.full = full_bar;
  pp.empty = empty_bar;
  pp.sf = sf_bar;
  pp.accfull = accfull_bar;
  pp.accempty = accempty_bar;
  pp.unit_bar = unit_bar;
  pp.unit = s_unit;
  pp.ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  pp.ring_g = smem_raw + (pp.ring - smem_u32(smem_raw));
  pp.abort_flag = &s_abort;
  pp.status = a.status;
  uint8_t* scratch = pp.ring_g + kStages * kStageBytes;

  if (threadIdx.x == 0) {
    s_abort = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc<false, kTmemCols>(&s_tmem);
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        mbar_init(&full_bar[s], 2);
        mbar_init(&empty_bar[s], 1);
        mbar_init(&sf_bar[s], 1);
      }
      for (int s = 0; s < 2; ++s) {
        mbar_init(&accfull_bar[s], 1);
        mbar_init(&accempty_bar[s], 4);
      }
      for (int s = 0; s < kUnits; ++s) mbar_init(&unit_bar[s], 1);
      mbar_init(&final_bar, 1);
      fence_barrier_init();
    }
    __syncwarp();
    tc_fence_before();
  }
  make_tables(a, s_t, reinterpret_cast<int*>(scratch), s_wsum);
  tc_fence_after();
  pp.tmem = s_tmem;
  const Product<false> up(a, s_t.tiles);
  const Product<true> down(a, s_t.tiles);

  if (warp == kWeightWarp) {
    const uint32_t elected = elect_one();
    RingPos at;
    if (load_weights<false>(a, s_t, pp, up, elected, lane, at)) load_weights<true>(a, s_t, pp, down, elected, lane, at);
  } else if (warp == kMmaWarp) {
    const uint32_t elected = elect_one();
    RingPos at, sf;
    int u = 0;
    if (issue_mmas<false>(a, pp, up, elected, at, sf, u)) issue_mmas<true>(a, pp, down, elected, at, sf, u);
    __syncwarp();
    mx_commit<false>(elected, smem_u32(&final_bar));  // every MMA done before tensor memory is freed
    mbar_wait_sleep_bounded(&final_bar, 0);
  } else if (warp == kTokenWarp) {
    const uint32_t elected = elect_one();
    RingPos at;
    if (load_tokens<false>(a, maps, s_t, pp, up, elected, lane, at))
      load_tokens<true>(a, maps, s_t, pp, down, elected, lane, at);
  } else if (warp >= kScaleWarp0 && warp < kScaleWarp0 + kScaleWarps) {
    int n = 0;
    if (arrange_scales<false>(pp, up, warp - kScaleWarp0, lane, n)) arrange_scales<true>(pp, down, warp - kScaleWarp0, lane, n);
  } else if (warp >= kEpiWarp0) {
    int u = 0;
    float* shared = reinterpret_cast<float*>(scratch);
    if (finish_h(a, s_t, pp, up, shared, warp & 3, lane, u, &s_last)) {
      epi_sync();  // the exchange becomes the sums
      finish_out(a, s_t, pp, down, shared, warp & 3, lane, u, &s_last);
    }
  }

  // Every copy has been waited for, unless the CTA gave up: then those still under way get the
  // time that they could take before shared memory is released.
  __syncthreads();
  if (s_abort && threadIdx.x == 0)
    for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < kWaitLimitNs / 100;) __nanosleep(1000);
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<false, kTmemCols>(pp.tmem);
  }
}

// Kernel 1: a warp per 256 elements of a token, eight to a lane, four lanes to a scaled block.
constexpr int kXThreads = 256;
__global__ void __launch_bounds__(kXThreads) mx_few_x_kernel(const __half* x, int M, int K, uint8_t* codes, uint8_t* scales,
                                                             int32_t* counters, int n_counters, int32_t* status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // a programmatic dependent of the kernel before
  const int i = blockIdx.x * kXThreads + threadIdx.x;
  for (int c = i; c < n_counters; c += gridDim.x * kXThreads) counters[c] = 0;
  if (i == 0) *status = 0;
  const int per = K / 8;  // lanes of a row; K is a multiple of 128, so four lanes stay together
  const int t = i / per, k = (i - t * per) * 8;
  if (t >= M) return;
  const uint4 raw = __ldcg(reinterpret_cast<const uint4*>(x + (size_t)t * K + k));
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
  float v[8];
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
    amax = max(amax, max(abs_bits(f.x), abs_bits(f.y)));
  }
  const uint32_t mask = 0xfu << (threadIdx.x & 28u);  // M * K / 8 is a multiple of 16: groups of four are whole
  amax = max(amax, __shfl_xor_sync(mask, amax, 1));
  amax = max(amax, __shfl_xor_sync(mask, amax, 2));
  const uint32_t b = mx_scale_byte(amax);
  const float mult = mx_multiplier(b);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = mx_scaled(v[j], mult, b);
  *reinterpret_cast<uint32_t*>(codes + (size_t)t * (K / 2) + k / 2) = mx_codes8(v);
  if ((threadIdx.x & 3) == 0) {
    const int c = k / 32;  // scaled block of the row
    scales[((size_t)t * ((K + 255) / 256) + (c >> 3)) * kScaleRec + (c & 7)] = (uint8_t)b;
  }
}

// Four epilogue warps of a CTA that has given up ask for a ticket that arrives between the first
// warp's look at it and the others'.
__global__ void ticket_probe_kernel(int32_t* answers) {
  __shared__ __align__(8) uint64_t unit_bar[kUnits], asked;
  __shared__ int s_unit[kUnits], s_abort;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(unit_bar, 1);
    mbar_init(&asked, 1);
    fence_barrier_init();
    s_abort = 1;
  }
  __syncthreads();
  if (warp == 4) {
    if (lane == 0) {
      for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000;) __nanosleep(1000);
      s_unit[0] = 0;
      mbar_arrive(unit_bar);
      mbar_arrive(&asked);
    }
    return;
  }
  Pipe pp = {};
  pp.unit_bar = unit_bar;
  pp.unit = s_unit;
  pp.abort_flag = &s_abort;
  if (warp) mbar_wait_bounded(&asked, 0);
  int unit = -1;
  const bool ok = wait_unit_together(pp, 1, unit);
  if (lane == 0) answers[warp] = ok;
}

}  // namespace

cudaError_t launch_mx_ticket_probe(int32_t* answers, cudaStream_t stream) {
  ticket_probe_kernel<<<1, 160, 0, stream>>>(answers);
  return cudaGetLastError();
}

size_t mx_few_part_bytes(int M, int topK) {
  return (part_words_of_h(sm_count(), M * topK) + (size_t)sm_count() * 2 * M * 128) * 4;
}
// Bytes of the scales of `rows` rows of depth D in the records of kernel 2.
size_t mx_few_scale_bytes(int rows, int D) { return (size_t)rows * mx_depth_blocks(D) * kScaleRec; }
size_t mx_few_counter_bytes(int M, int K, int I, int topK) { return (size_t)counters_of(M, K, I, topK) * 4; }

// Whether every CTA of kernel 2 can be resident at once: one per SM.
bool mx_few_resident() {
  static PerContextOnce queried;
  static bool ok[kMaxDevices] = {};
  const int dev = current_device();
  if (queried.needed(dev)) {
    int n = 0;
    // kernel 1 with the same division of L1 as kernel 2, which then need not wait for a change
    ok[dev] = cudaFuncSetAttribute(mx_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   smem_bytes(kMxFewTokens)) == cudaSuccess &&
              cudaFuncSetAttribute(mx_few_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                   cudaSharedmemCarveoutMaxShared) == cudaSuccess &&
              cudaFuncSetAttribute(mx_few_x_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                   cudaSharedmemCarveoutMaxShared) == cudaSuccess &&
              cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, mx_few_kernel, kThreads, smem_bytes(kMxFewTokens)) ==
                  cudaSuccess &&
              n >= 1 && sm_count() <= 256;
    if (!ok[dev]) cudaGetLastError();
    queried.done(dev);
  }
  return ok[dev];
}

cudaError_t launch_mx_few(const MxFewProblem& p, cudaStream_t stream) {
  const int R = p.M * p.topK;
  const uint64_t xs = (uint64_t)mx_depth_blocks(p.K) * kScaleRec, hs = (uint64_t)mx_depth_blocks(p.I) * kScaleRec;
  FewMaps maps;
  if (!encode_tensor_map_rows(&maps.x_codes, p.x_codes, p.K / 2, p.K / 2, p.M, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tensor_map_rows(&maps.h_codes, p.h_codes, p.I / 2, p.I / 2, R, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tensor_map_rows(&maps.x_scales, p.x_scales, xs, xs, p.M, kScaleRec, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode_tensor_map_rows(&maps.h_scales, p.h_scales, hs, hs, R, kScaleRec, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const int n_counters = counters_of(p.M, p.K, p.I, p.topK);
  const unsigned x_blocks = (unsigned)(((size_t)p.M * p.K / 8 + kXThreads - 1) / kXThreads);
  cudaError_t e = launch_dependent(mx_few_x_kernel, x_blocks, kXThreads, 0, stream, reinterpret_cast<const __half*>(p.x), p.M, p.K,
                                   p.x_codes, p.x_scales, p.counters, n_counters, p.status);
  if (e != cudaSuccess) return e;
  FewArgs a;
  a.M = p.M;
  a.K = p.K;
  a.I = p.I;
  a.E = p.E;
  a.topK = p.topK;
  a.R = R;
  a.expert_idx = p.expert_idx;
  a.probs = p.probs;
  a.w1 = p.w1;
  a.w2 = p.w2;
  a.h_codes = p.h_codes;
  a.h_scales = p.h_scales;
  a.part = p.part;
  a.counters = p.counters;
  a.out = reinterpret_cast<__half*>(p.out);
  a.status = p.status;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sm_count());
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(p.M);
  cfg.stream = stream;
  cudaLaunchAttribute together;
  together.id = cudaLaunchAttributeCooperative;
  together.val.cooperative = 1;
  cfg.attrs = &together;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mx_few_kernel, maps, a);
}

}  // namespace moe
