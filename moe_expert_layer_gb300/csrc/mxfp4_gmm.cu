// Grouped MXFP4 product over expert-major rows on the block-scaled tensor cores
// (tcgen05.mma kind::mxf4), with SwiGLU and requantisation behind it where asked, and the
// probability-weighted sum of a token's rows (include/moe_mxfp4.h).
//
// A work item is (expert, channel block, tile of up to NT rows).  The weight channels are the
// MMA's rows (operand A), the token rows its N columns (operand B), so the ragged side is the
// one whose size the instruction takes in steps of 16 (32 for a pair): an expert of cnt rows is
// cut into ceil(cnt / NT) tiles of equal size rounded up to that step.  Items are dealt out expert-major,
// channel blocks innermost, so that CTAs working at the same time share an expert's rows and
// its weights through L2.  Persistent CTAs, one per SM, in two forms:
//   - few rows per expert: single CTAs, 128 channels, tiles of up to 32 rows: the weights
//     stream past (128 tokens x 7168, N = 4096, 256 experts, 8 each: 547 us with the rows'
//     quantisation, the weights at 1.04 of the measured copy rate);
//   - more: CTA pairs (cta_group::2), 256 channels, tiles of up to 192 rows.  Each CTA loads
//     half of the rows: the copies through shared memory, which bound a single CTA's 128 x 208
//     (325 us at 49152 rows, N = 2816, D = 4096, 64 experts, where the pairs take 220), are fewer
//     for each MMA.  The tensor pipe is then 58% busy, L2's path to the SMs 56%: what sets the pace is
//     the turn of the ring, a copy's latency, the scale words' way to tensor memory, the MMAs and
//     their commit, over the six stages that fit (five: 17 us more; tiles of 224 rows and five
//     stages: 17 more; 128 rows and seven: 28 more).
// A tile starts on a multiple of four rows (a 16-byte boundary of the scale words), so an
// expert's first one may begin with up to three rows of the expert before, not stored.
//
// Roles: warp 0 loads, per 256-deep stage, one 17408-byte copy of a weight block with its
// scales and the rows' words of the two scale planes; warp 2 loads the rows' codes, in tensor
// copies of 64, 32 and 16 rows; warps 4-11, two groups in turn, read a stage's scale words and store
// them to tensor memory, each warp to its 32 lanes (one group: 328 us for 265); warp 1 issues the
// MMAs; warps 12-27 are four epilogue groups, two for each of the two accumulators, taking its
// columns in turn.  In a pair the first CTA's MMAs use what the second CTA's scale warps have
// stored: tensor memory, which the tcgen05 fences order across the pair around the barrier.  (Put
// in order in shared memory for tcgen05.cp to copy, the words would need release and acquire at
// cluster scope: 337 us for 255 at 8192 tokens x 4096, N = 2816, 64 experts, six each.)  Every wait
// is bounded: one that gives up records MOE_ERR_TIMEOUT and the CTA winds down.
#include "mx_tc.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kThreads = 896;
constexpr int kWeightWarp = 0, kMmaWarp = 1, kTokenWarp = 2, kScaleWarp0 = 4, kScaleGroups = 2, kEpiWarp0 = 12;
constexpr int kMaxExperts = 1024;
constexpr int kEpiGroups = 4, kEpiBytes = 8192;  // an epilogue group's shared memory

template <int NT, bool PAIR>
struct Cfg {
  static constexpr int kStep = PAIR ? 32 : 16;         // of the MMA's columns
  static constexpr int kCtaRows = PAIR ? NT / 2 : NT;  // token rows in a CTA's shared memory
  static constexpr int kRowTiles = (NT + 127) / 128;      // 128-row tiles of the rows' scale words
  static constexpr int kPlaneWords = 128 * kRowTiles;
  static constexpr int kScales = kMxBlockBytes + kCtaRows * 128;  // of a stage: the rows' scale words
  static constexpr int kStageBytes = kScales + 2 * kPlaneWords * 4;
  static constexpr int kStages = PAIR ? 6 : 8;
  static constexpr int kSfbPlane = 4 * kRowTiles;        // tensor-memory columns per 128 elements of depth
  static constexpr int kSfCols = 8 + 2 * kSfbPlane;      // and of a stage's scales
  // Stages whose scales are in tensor memory.  A slot is written again only when the MMAs of the
  // stage that used it have completed.
  static constexpr int kSfStages = 5;
  static constexpr int kSf0 = 2 * NT;                    // accumulators in columns [0, 2 NT)
  static constexpr int kTmemCols = (kSf0 + kSfStages * kSfCols) <= 128 ? 128 : (kSf0 + kSfStages * kSfCols) <= 256 ? 256 : 512;
  static constexpr int kSmem = kStages * kStageBytes + kEpiGroups * kEpiBytes;
  static_assert(kSfStages < kStages, "a stage's scale columns are waited for after its slot's last use");
  static_assert(NT % kStep == 0 && kSf0 + kSfStages * kSfCols <= 512, "tensor memory");
  static_assert(kMxBlockBytes % 1024 == 0 && kScales % 128 == 0 && kStageBytes % 1024 == 0, "swizzled rows");
  static_assert(kSmem + 9 * 1024 <= 227 * 1024, "shared memory, with ~8.4 KB static");
};

// What becomes of the sums: binary16 rows, fp32 rows, or their SwiGLU as MXFP4 rows.
enum class Out { kHalf, kFloat, kSwiglu };

struct GmmArgs {
  int R, E, N, D, KB, pitch;
  const uint32_t* scales;
  const int32_t* cumsum;
  const uint8_t* w;
  __half* c;
  float* c32;
  uint8_t* h_codes;
  uint8_t* h_scales;
  int32_t* status;
  bool clear;
};

// Tensor maps of the codes, 256 elements x 64, 32 and 16 rows (a CTA's rows of a tile, a
// multiple of 16, are copied as a sum of them), of the scale words, 2 planes x kPlaneWords rows,
// and of the output.
constexpr int kBoxes = 3, kBoxRows = 64;
constexpr int kOutRows = 32;
struct Maps {
  CUtensorMap box[kBoxes], scales, c;  // c: the output, 128 channels x kOutRows rows
};

struct Item {
  int e, cb, row0, rows, skip, n;  // the first `skip` rows are another expert's; n: MMA columns
};

struct WorkList {
  const int* pref;  // first item of each expert; pref[E] = their number
  const int* end;   // last row of each expert + 1
  int CB, E;        // channel blocks (of a CTA or a pair), experts
};

// Row tiles of an expert with rows [start, end), from start rounded down to 4.  With t tiles
// of `size` rows (a multiple of the step, at most NT), (t - 1) * size is less than their number:
// none is empty.
template <int NT>
__device__ __forceinline__ int tiles_of(int start, int end) {
  return end > start ? (end - (start & ~3) + NT - 1) / NT : 0;
}

template <int NT, int STEP>
__device__ __forceinline__ Item decode_item(int j, const WorkList& wl, int& e_hint) {
  // pref[lo] <= j < pref[hi]: mostly the same expert as the item before, or one of the next
  int lo = e_hint, hi = lo + 1, step = 1;
  while (hi < wl.E && wl.pref[hi] <= j) {
    lo = hi;
    hi = min(hi + step, wl.E);
    step *= 2;
  }
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (wl.pref[mid] <= j) lo = mid; else hi = mid;
  }
  e_hint = lo;
  const int start = lo ? wl.end[lo - 1] : 0, end = wl.end[lo], start4 = start & ~3;
  const int t = tiles_of<NT>(start, end), size = ((end - start4 + t - 1) / t + STEP - 1) & -STEP;
  const int local = j - wl.pref[lo], rt = local / wl.CB;
  Item it;
  it.e = lo;
  it.cb = local - rt * wl.CB;
  it.row0 = start4 + rt * size;
  it.rows = min(size, end - it.row0);
  it.skip = max(start - it.row0, 0);
  it.n = (it.rows + STEP - 1) & -STEP;
  return it;
}

// Whether `ok` holds in all four warps of a group (named barrier `id`).
__device__ __forceinline__ bool group_all(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

template <int NT, Out OUT, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gmm_kernel(const __grid_constant__ Maps maps, const GmmArgs a) {
  using C = Cfg<NT, PAIR>;
  constexpr int S = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // swizzled rows: 1024-byte groups
  __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S], sf_bar[S], accfull_bar[2], accempty_bar[2], final_bar;
  __shared__ int s_pref[kMaxExperts + 1], s_end[kMaxExperts], s_wsum[kThreads / 32];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_issued[2];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int E = a.E, NB = a.N / 128, KB = a.KB, CB = PAIR ? (NB + 1) / 2 : NB;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int first = PAIR ? blockIdx.x >> 1 : blockIdx.x, stride = PAIR ? gridDim.x >> 1 : gridDim.x;
  volatile int* abort_flag = &s_abort;

  // ---- work list, barriers, tensor memory.  Launched as a programmatic dependent, which hides the
  // setup (a layer of 128 tokens x 4096, 1408 channels, 64 experts, 6 each: 127 us without, 119
  // with): what the kernels before this one wrote is read behind the wait only.
  {
    if (warp == kMmaWarp) {
      tmem_alloc<PAIR, C::kTmemCols>(&s_tmem);
      if (lane == 0) {
        for (int b = 0; b < kBoxes; ++b) prefetch_tmap(&maps.box[b]);
        prefetch_tmap(&maps.scales);
        if (OUT == Out::kHalf) prefetch_tmap(&maps.c);
        for (int s = 0; s < S; ++s) {
          mbar_init(&full_bar[s], 2);
          mbar_init(&empty_bar[s], 1);
        }
        for (int s = 0; s < S; ++s) mbar_init(&sf_bar[s], PAIR ? 8 : 4);
        for (int s = 0; s < 2; ++s) {
          mbar_init(&accfull_bar[s], 1);
          mbar_init(&accempty_bar[s], PAIR ? 16 : 8);
        }
        mbar_init(&final_bar, 1);
        fence_barrier_init();
      }
      tc_fence_before();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // long before any wait can run out; a memory set of its own took 2 us
    if (a.clear && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    const int per = (E + kThreads - 1) / kThreads;
    const int e0 = min(E, (int)threadIdx.x * per), e1 = min(E, e0 + per);
    int local = 0;
    for (int e = e0; e < e1; ++e) {
      const int hi = min(max(a.cumsum[e], 0), a.R);
      const int lo = e ? min(max(a.cumsum[e - 1], 0), a.R) : 0;
      s_end[e] = hi;
      local += tiles_of<NT>(lo, hi) * CB;
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) s_wsum[warp] = incl;
    if (threadIdx.x == 0) {
      s_abort = 0;
      s_issued[0] = s_issued[1] = 0;
    }
    __syncthreads();
    int run = incl - local;
    for (int w = 0; w < warp; ++w) run += s_wsum[w];
    for (int e = e0; e < e1; ++e) {
      s_pref[e] = run;
      run += tiles_of<NT>(e ? s_end[e - 1] : 0, s_end[e]) * CB;
    }
    if (e0 < E && e1 == E) s_pref[E] = run;
  }
  __syncthreads();
  __syncwarp();
  if (PAIR) cluster_sync_all();  // the peer's barriers and tensor memory are ready
  tc_fence_after();
  WorkList wl;
  wl.pref = s_pref;
  wl.end = s_end;
  wl.CB = CB;
  wl.E = E;
  const int total = s_pref[E];
  const uint32_t tmem = s_tmem;
  const uint32_t ring = smem_u32(smem_raw);
  uint8_t* ring_g = smem_raw;
  // a stage: weight codes at 0, their scales at 16384, token codes at 17408, their scales behind them
  const int planes = (a.D + 127) / 128;

  if (warp == kWeightWarp || warp == kTokenWarp) {
    const uint32_t elected = elect_one();
    RingPos at;
    int n = 0, e_hint = 0;
    bool ok = true;
    for (int j = first; ok && j < total; j += stride) {
      const Item it = decode_item<NT, C::kStep>(j, wl, e_hint);
      // a pair's second block past the last channel reads the last one again (not stored)
      const int nb = PAIR ? min(2 * it.cb + (int)rank, NB - 1) : it.cb;
      const uint8_t* wb = a.w + ((size_t)it.e * NB + nb) * (size_t)KB * kMxBlockBytes;
      const int cta_rows = PAIR ? it.n / 2 : it.n, row0 = it.row0 + (int)rank * cta_rows;
      for (int kb = 0; kb < KB; ++kb, ++n, at.next(S)) {
        if (!(ok = warp_wait(&empty_bar[at.slot], at.phase ^ 1u, abort_flag, a.status))) break;
        const uint32_t st = ring + at.slot * C::kStageBytes, bar = smem_u32(&full_bar[at.slot]);
        if (warp == kWeightWarp) {
          expect_tx_elect(elected, bar, kMxBlockBytes + 2 * C::kPlaneWords * 4);
          bulk_load_elect(elected, st, wb + (size_t)kb * kMxBlockBytes, kMxBlockBytes, bar);
          tma_load_2d_elect(elected, st + C::kScales, &maps.scales, it.row0, 2 * kb, bar);
        } else {
          expect_tx_elect(elected, bar, (uint32_t)cta_rows * 128);
          int r = 0;
#pragma unroll
          for (int b = 0; b < kBoxes; ++b) {
            const int rows = kBoxRows >> b;
            for (; cta_rows - r >= rows; r += rows)
              tma_load_2d_elect(elected, st + kMxBlockBytes + r * 128, &maps.box[b], kb * 128, row0 + r, bar);
          }
        }
      }
    }
    // the next kernel's setup beside the last items
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the last stages' releases: commits arrive in both CTAs of a pair, and neither may leave
    // before an arrival that is still on its way to it
    for (int s = 0; ok && s < S; ++s, at.next(S)) ok = warp_wait(&empty_bar[at.slot], at.phase ^ 1u, abort_flag, a.status);
    if (lane == 0) s_issued[warp == kTokenWarp] = n;
  } else if (warp == kMmaWarp) {
    if (rank == 0) {
      const uint32_t elected = elect_one(), t0 = __shfl_sync(0xffffffffu, tmem, 0);
      RingPos at, sf;
      int e_hint = 0, u = 0;
      bool ok = true;
      // a barrier's answer takes as long as issuing several MMAs: the next stage's is asked for
      // before this one's are issued
      uint32_t there = mbar_test(&sf_bar[0], 0);
      for (int j = first; ok && j < total; j += stride, ++u) {
        const Item it = decode_item<NT, C::kStep>(j, wl, e_hint);
        const int buf = u & 1;
        if (!(ok = warp_wait(&accempty_bar[buf], ((u >> 1) & 1) ^ 1, abort_flag, a.status))) break;
        tc_fence_after();
        const uint32_t idesc = mx_idesc(PAIR ? 256 : 128, it.n), d = t0 + buf * NT;
        const int last = (a.D - (KB - 1) * 256 + 127) >> 7;  // 128-deep halves of the last stage
        for (int kb = 0; kb < KB; ++kb, sf.next(C::kSfStages)) {
          // the scale warps arrive after they have seen the stage's copies complete
          if (!__all_sync(0xffffffffu, there) &&
              !(ok = warp_wait(&sf_bar[at.slot], at.phase, abort_flag, a.status)))
            break;
          tc_fence_after();
          const uint32_t st = ring + at.slot * C::kStageBytes, t_sf = t0 + C::kSf0 + sf.slot * C::kSfCols;
          const uint64_t da = sw128_desc(st), db = sw128_desc(st + kMxBlockBytes);
          const uint32_t done = smem_u32(&empty_bar[at.slot]);
          at.next(S);
          there = mbar_test(&sf_bar[at.slot], at.phase);
          mx_mma2<PAIR>(elected, d, da, db, 0, idesc, t_sf, t_sf + 8, kb ? 1u : 0u);
          if (kb < KB - 1 || last == 2)
            mx_mma2<PAIR>(elected, d, da, db, 1, idesc, t_sf + 4, t_sf + 8 + C::kSfbPlane, 1u);
          mx_commit<PAIR>(elected, done);
        }
        if (ok) mx_commit<PAIR>(elected, smem_u32(&accfull_bar[buf]));
      }
      mx_commit_local<PAIR>(elected, smem_u32(&final_bar));  // every MMA done before tensor memory is freed
      mbar_wait_sleep_bounded(&final_bar, 0);
    }
  } else if (warp >= kScaleWarp0 && warp < kEpiWarp0) {
    // bytes of the last plane past D are no scales
    const uint32_t last_mask = a.D % 128 ? (1u << (a.D % 128 / 4)) - 1u : 0xffffffffu;
    const int group = (warp - kScaleWarp0) >> 2;
    const uint32_t t_sf = tmem + ((uint32_t)(warp & 3) << 21) + C::kSf0;
    RingPos at, old, sf;  // old: the stage kSfStages before
    int n = 0;
    bool ok = true;
    for (int j = first; ok && j < total; j += stride) {
      for (int kb = 0; kb < KB; ++kb, ++n, at.next(S), sf.next(C::kSfStages)) {
        if (n > C::kSfStages) old.next(S);
        if (n % kScaleGroups != group) continue;
        // The scale columns are free once the MMAs of the stage that used them are done.  This wait
        // comes first for another reason too: a warp that takes every second stage has not itself
        // seen the slot's previous copies complete, and copies complete in any order; only after
        // that stage's MMAs is the barrier known to be in this use's phase.
        if (n >= C::kSfStages && !(ok = warp_wait(&empty_bar[old.slot], old.phase, abort_flag, a.status))) break;
        if (!(ok = warp_wait(&full_bar[at.slot], at.phase, abort_flag, a.status))) break;
        tc_fence_after();
        const uint8_t* st = ring_g + at.slot * C::kStageBytes;
        uint4 w[2 + 2 * C::kRowTiles];
#pragma unroll
        for (int i = 0; i < 2 + 2 * C::kRowTiles; ++i) {
          w[i] = mx_scale_words(i < 2 ? st + kMxCodeBytes + 512 * i : st + C::kScales + 512 * (i - 2), lane);
          const int q = (i - 2) / C::kRowTiles;
          if (i >= 2 && 2 * kb + q == planes - 1) {
            w[i].x &= last_mask;
            w[i].y &= last_mask;
            w[i].z &= last_mask;
            w[i].w &= last_mask;
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2 + 2 * C::kRowTiles; i += 2) tmem_st8(t_sf + sf.slot * C::kSfCols + 4 * i, w[i], w[i + 1]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_remote(cluster_addr(&sf_bar[at.slot], 0)); else mbar_arrive(&sf_bar[at.slot]);
        }
      }
    }
  } else if (warp >= kEpiWarp0) {
    const int group = (warp - kEpiWarp0) >> 2, quarter = warp & 3, buf = group & 1;
    const uint32_t lanes = (uint32_t)quarter << 21;  // 32 * quarter in the lane field
    uint8_t* own = ring_g + S * C::kStageBytes + group * kEpiBytes;
    int e_hint = 0;
    for (int u = buf, j = first + buf * stride; j < total; j += 2 * stride, u += 2) {
      const Item it = decode_item<NT, C::kStep>(j, wl, e_hint);
      bool ok = warp_wait(&accfull_bar[buf], (u >> 1) & 1, abort_flag, a.status);
      ok = group_all(9 + group, ok);  // the group's warps wait for one another below
      if (!ok) break;
      tc_fence_after();
      const uint32_t t = tmem + lanes + buf * NT;
      const int nb = PAIR ? 2 * it.cb + (int)rank : it.cb;
      const int rows = nb < NB ? it.rows : 0;  // a pair's block past the last channel stores nothing
      const int skip = it.skip;
      if (OUT == Out::kHalf) {
        // 32 rows x 128 channels of binary16 gathered in shared memory and stored from there by one
        // tensor copy, or, where the tile's first or last rows are not its own, row by row
        for (int c0 = kOutRows * (group >> 1); c0 < it.n; c0 += 2 * kOutRows) {
          uint32_t v[2][16];
          __syncwarp();
          tmem_ld16(t + c0, v[0]);
          if (!PAIR && c0 + 16 >= it.n) {  // a single CTA's tile may end after 16 columns
#pragma unroll
            for (int i = 0; i < 16; ++i) v[1][i] = 0;
          } else {
            tmem_ld16(t + c0 + 16, v[1]);
          }
          if (quarter == 0) bulk_wait_read_all();
          tmem_wait_ld();
          asm volatile("bar.sync %0, 128;" ::"r"(9 + group) : "memory");
          __half* o = reinterpret_cast<__half*>(own) + quarter * 32 + lane;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const __half2 h = f2h2_sat(__uint_as_float(v[i >> 4][i & 15]), __uint_as_float(v[i >> 4][(i & 15) + 1]));
            o[i * 128] = __low2half(h);
            o[i * 128 + 128] = __high2half(h);
          }
          fence_proxy_async_smem();
          asm volatile("bar.sync %0, 128;" ::"r"(9 + group) : "memory");
          if (quarter == 0) {
            if (c0 >= skip && c0 + kOutRows <= rows) {
              if (lane == 0) tma_store_2d(&maps.c, nb * 128, it.row0 + c0, own);
            } else if (c0 + lane >= skip && c0 + lane < rows) {
              bulk_store(a.c + (size_t)(it.row0 + c0 + lane) * a.N + nb * 128, own + lane * 256, 256);
            }
            bulk_commit_group();
          }
        }
      } else if (OUT == Out::kFloat) {
        // a warp's 32 channels of a row are whole 128-byte lines
        for (int c0 = 16 * (group >> 1); c0 < it.n; c0 += 32) {
          uint32_t v[16];
          __syncwarp();
          tmem_ld16(t + c0, v);
          tmem_wait_ld();
          float* o = a.c32 + (size_t)(it.row0 + c0) * a.N + nb * 128 + quarter * 32 + lane;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c0 + i >= skip && c0 + i < rows) o[i * a.N] = __uint_as_float(v[i]);
        }
      } else {
        // Warps in pairs: the even one holds 32 gate channels, the odd one the up channels that
        // multiply them.  16 rows of both go through shared memory to threads that each take
        // eight channels of a row: the scaled block's maximum is then two shuffles, and its
        // scale is found once for eight values (a row at a time across the lanes instead took
        // twice the instructions, and the epilogue longer than the MMAs).  Odd rows have their
        // 16-byte pieces swapped in pairs, which keeps reads off each other's banks.
        const int pair = (warp - kEpiWarp0) >> 1, odd = warp & 1, th = odd * 32 + lane;
        float* x = reinterpret_cast<float*>(own) + (pair & 1) * 1024;  // [16][64]
        const int k = nb * 2 + (quarter >> 1), I = a.N / 2;            // scaled block of h
        const int row = th >> 2, seg = th & 3;
        const float4* gate = reinterpret_cast<const float4*>(x + row * 64 + ((seg * 8) ^ ((row & 1) << 2)));
        const float4* gate2 = reinterpret_cast<const float4*>(x + row * 64 + ((seg * 8 + 4) ^ ((row & 1) << 2)));
        uint8_t* sc = a.h_scales + ((size_t)(k >> 2) * a.pitch + it.row0 + row) * 4;
        uint8_t* co = a.h_codes + (size_t)(it.row0 + row) * (I / 2) + k * 16 + seg * 4;
        const bool tail = k == I / 32 - 1 && (k & 3) != 3;  // bytes of the word past the last block: 0
        for (int c0 = 16 * (group >> 1); c0 < it.n; c0 += 32) {
          uint32_t v[16];
          __syncwarp();
          tmem_ld16(t + c0, v);
          tmem_wait_ld();
          asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");  // both have read the rows before
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i * 64 + (th ^ ((i & 1) << 2))] = __uint_as_float(v[i]);
          asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");
          const float4 g0 = gate[0], g1 = gate2[0], u0 = gate[8], u1 = gate2[8];  // up: 32 floats on
          const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
          const float u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
          float h[8];
          mx_swiglu8(g, u, h);
          uint32_t byte;
          const uint32_t w = mx_quant_group8(h, byte);
          const int r = c0 + row;
          if (r >= skip && r < rows) {
            *reinterpret_cast<uint32_t*>(co + (size_t)c0 * (I / 2)) = w;
            if (seg == 0) {
              if (tail)
                for (int z = (k & 3) + 1; z < 4; ++z) sc[c0 * 4 + z] = 0;
              sc[c0 * 4 + (k & 3)] = (uint8_t)byte;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_remote(cluster_addr(&accempty_bar[buf], 0)); else mbar_arrive(&accempty_bar[buf]);
      }
    }
    if (OUT == Out::kHalf && quarter == 0) bulk_wait_all();  // stores done before shared memory is released
  }

  __syncthreads();
  if (threadIdx.x == 0) {  // copies still in flight (only after an abort) land before shared memory is released
    const int n0 = min(s_issued[0], s_issued[1]), n1 = max(s_issued[0], s_issued[1]);
    for (int n = n0; n < n1; ++n) mbar_arrive(&full_bar[n % S]);  // stages that one of the two loaders never began
    for (int n = max(0, n1 - S); n < n1; ++n) mbar_wait_bounded(&full_bar[n % S], (n / S) & 1);
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (PAIR) cluster_sync_all();  // neither CTA leaves while the pair's MMAs or arrivals may touch it
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<PAIR, C::kTmemCols>(tmem);
  }
}

template <int NT, Out OUT, bool PAIR>
cudaError_t launch_gmm(const MxGemmProblem& p, cudaStream_t stream) {
  using C = Cfg<NT, PAIR>;
  Maps maps;
  const uint64_t half = (uint64_t)p.D / 2, rows = (uint64_t)p.R;
  for (int b = 0; b < kBoxes; ++b)
    if (!encode_tensor_map_2d(&maps.box[b], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.codes, half, rows, 128, (uint32_t)kBoxRows >> b))
      return cudaErrorInvalidValue;
  if (!encode_tensor_map_words(&maps.scales, p.scales, (uint64_t)mx_scale_pitch(p.R), (uint64_t)mx_scale_planes(p.D),
                               C::kPlaneWords, 2))
    return cudaErrorInvalidValue;
  if (OUT == Out::kHalf && !encode_tensor_map_2d(&maps.c, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, p.c, (uint64_t)p.N, rows, 128, kOutRows,
                                       CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  static PerContextOnce set;
  const int dev = current_device();
  if (set.needed(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(mx_gmm_kernel<NT, OUT, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    set.done(dev);
  }
  GmmArgs a;
  a.R = p.R;
  a.E = p.E;
  a.N = p.N;
  a.D = p.D;
  a.KB = mx_depth_blocks(p.D);
  a.pitch = mx_scale_pitch(p.R);
  a.scales = p.scales;
  a.cumsum = p.cumsum;
  a.w = p.w;
  a.c = reinterpret_cast<__half*>(p.c);
  a.c32 = p.c32;
  a.h_codes = p.h_codes;
  a.h_scales = reinterpret_cast<uint8_t*>(p.h_scales);
  a.status = p.status;
  a.clear = p.clear_status;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(PAIR ? sm_count() & ~1 : sm_count()));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = PAIR ? 2 : 1;
  attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, mx_gmm_kernel<NT, OUT, PAIR>, maps, a);
}

// One thread per four channels of a token: each row's 16 bytes, four rows read at a time, then
// the sums in order of the routes, rounded once.  c2 is fp32: a route's row may lie far outside
// binary16 where its weight brings it back, or another route's row cancels it.  Bound by reading
// it: 8192 tokens x 4096, six rows each, 133 us for 864 MB (0.96 of the measured copy rate).
// EARLY: launched as a programmatic dependent of the product, once that one is past its own wait.  Of
// what is read here only c2 is written after this kernel's launch, so c2 is read past the
// read-only path then.
constexpr int kCombineThreads = 256, kCombineBlocks = 6;  // blocks to an SM
template <bool EARLY>
__global__ void __launch_bounds__(kCombineThreads, kCombineBlocks) mx_combine_kernel(const float* c2, const int32_t* expanded,
                                                                     const float* probs, int M, int K, int topK,
                                                                     __half* out) {
  if (EARLY) asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per = K / 4;
  const int64_t i = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x;
  const int t = (int)(i / per), k = (int)(i - (int64_t)t * per);
  if (t >= M) return;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int32_t* rows = expanded + (int64_t)t * topK;
  const float* p = probs + (int64_t)t * topK;
  for (int j = 0; j < topK; j += 4) {
    float4 v[4];
    float w[4];
    bool in[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int d = j + q < topK ? __ldg(rows + j + q) : -1;
      in[q] = d >= 0;
      if (in[q]) {
        const float4* row = reinterpret_cast<const float4*>(c2 + (size_t)d * K) + k;
        v[q] = EARLY ? __ldcg(row) : __ldg(row);
        w[q] = __ldg(p + j + q);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (in[q]) {
        acc.x = fmaf(w[q], v[q].x, acc.x);
        acc.y = fmaf(w[q], v[q].y, acc.y);
        acc.z = fmaf(w[q], v[q].z, acc.z);
        acc.w = fmaf(w[q], v[q].w, acc.w);
      }
  }
  const __half2 lo = f2h2_sat(acc.x, acc.y), hi = f2h2_sat(acc.z, acc.w);
  reinterpret_cast<uint2*>(out)[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

}  // namespace

// Single CTAs up to 32 rows per expert on average, one tile of theirs; us at 16 / 32 / 48 rows of each
// expert (back to back, weights not in L2 but for the second):
//                                     single CTAs          pairs
//   64 experts, D 4096, N 2816     64.4   65.5   77.1   65.3  66.2  67.8
//   8 experts,  D 1408, N 4096      8.4    8.1   11.5    9.5   9.1   9.5
//   256 experts, D 7168, N 4096     575    593    663    565   574   581
// The host knows the average alone: 128 rows on each of 32 of those 256 experts take 166 us here, which
// pairs would take 86 for.
cudaError_t launch_mx_gmm(const MxGemmProblem& p, cudaStream_t stream) {
  if ((double)p.R / p.E <= 32.0)
    return p.h_codes ? launch_gmm<32, Out::kSwiglu, false>(p, stream)
           : p.c32   ? launch_gmm<32, Out::kFloat, false>(p, stream)
                     : launch_gmm<32, Out::kHalf, false>(p, stream);
  return p.h_codes ? launch_gmm<192, Out::kSwiglu, true>(p, stream)
         : p.c32   ? launch_gmm<192, Out::kFloat, true>(p, stream)
                   : launch_gmm<192, Out::kHalf, true>(p, stream);
}

cudaError_t launch_mx_combine(const float* c2, const int32_t* expanded, const float* probs, int M, int K, int topK,
                              uint16_t* out, cudaStream_t stream) {
  const int64_t n = (int64_t)M * (K / 4);
  const unsigned blocks = (unsigned)((n + kCombineThreads - 1) / kCombineThreads);
  __half* o = reinterpret_cast<__half*>(out);
  // early where all blocks fit beside each other: a layer of 64 experts, six each, 200 tokens x 4096
  // (800 blocks) 120.6 us for 121.6 in order, 1024 tokens 166.8 for 166.6, 8192 tokens 598 for 585
  if (blocks <= (unsigned)(kCombineBlocks * sm_count()))
    return launch_dependent(mx_combine_kernel<true>, blocks, kCombineThreads, 0, stream, c2, expanded, probs, M, K, topK, o);
  mx_combine_kernel<false><<<blocks, kCombineThreads, 0, stream>>>(c2, expanded, probs, M, K, topK, o);
  return cudaGetLastError();
}

}  // namespace moe
