// Products of 16-bit operands grouped by expert (include/moe_experts16.h) on the tensor cores
// (tcgen05.mma kind::f16, fp32 accumulators in tensor memory): rows times their expert's weights,
// and the two gradients.
//
//             MMA rows (operand A)             MMA columns (operand B)       reduction
//   kForward  channels n of w[e]               rows of a                     k of D
//   kInput    channels k of w[e] (MN-major)    rows of dc                    n of N
//   kWeight   channels n of dc (MN-major)      channels k of a (MN-major)    rows of the expert
//
// An operand whose reduction index is not the contiguous one is "MN-major": a tensor copy brings
// boxes of 64 channels x 64 steps of the reduction, and the MMA's descriptors name that order, so
// nothing is transposed anywhere.
//
// kForward and kInput: the ragged side, an expert's rows, is the one whose size the instruction
// takes in steps of 16 (32 for a pair): an expert of cnt rows is cut into ceil(cnt / NT) tiles of
// multiples of that step.  Items (expert, row tile, channel block) are dealt out expert-major, channel
// blocks innermost, so that CTAs working at the same time share an expert's rows and its weights
// through L2.  kWeight: items are 256 x 256 blocks of dw[e] (128 x 128 where clusters divide the rows:
// `divide_rows`); the last stage of an expert's rows also brings rows of the next expert, which are
// overwritten with zeros in shared memory (up to the 16 rows that an MMA takes) before the MMAs see
// them: 0 times what they hold could be NaN.
//
// Persistent CTAs, one per SM, in three forms (`choose`, at the end, with what each takes):
//   - single CTAs of 128 channels and tiles of up to 32 rows: the weights stream past few rows.  Where
//     there are too few items for the device, a cluster divides the reduction of each: every CTA leaves
//     its sums in its shared memory, and behind a barrier of the cluster each adds a share of the
//     tile's elements over the CTAs, in order, and stores it.
//   - single CTAs and tiles of up to 128 rows;
//   - CTA pairs (cta_group::2) of 256 channels and tiles of up to 256 rows, of which each CTA loads half.
//
// Measured (bfloat16, GB300; of MEASURED rates 6672 GB/s and 1920 TFLOP/s; weights not in L2):
//   8 experts x 1 row, 7168 -> 4096       70 us   6.7 TB/s: the weights' stream, all there is
//   256 experts x 4, 7168 -> 4096       2030 us   7.4 TB/s (reads alone run faster than a copy)
//   1 expert x 1 row, 4096 -> 4096      10.7 us   3.1 TB/s: launch 3.7, then the stream of a round
//   1 expert x 8192, 4096 -> 4096        138 us   1990 TFLOP/s (the library's product: 142)
//   64 experts x 768, 4096 -> 2816   670-740 us   1530-1690 TFLOP/s alone, tensor pipe 89% busy; back to
//       back for seconds 787, where the power limit holds the clock at 1.45 GHz.  What is left: experts a
//       little past 768 rows take a fourth tile, and 34.2 rounds of items are 35.
//   64 experts x 768, kWeight, 4096 x 1408  460-490 us   1160-1230 TFLOP/s, 1.48 GB written in fp32 (in 16 bits
//       365-400; added to what is there 610)
// At 1.9 GHz a stage of a pair takes its 512 clocks, for every kind; that is 18.4 TB/s from L2, about what
// it has: kWeight's stores and their way on to memory come on top (12 stages and 20 MB of fp32 sums from
// all pairs: 3.24 us without stores, 3.9 while L2 holds them, 5.5 when it writes them back; the same
// stored from registers, or 4 KB contiguous, or with other L2 policies: no faster).  Two pairs to a
// cluster that share their rows by multicast were slower all the same (180 us for 144 at 8192 x 4096 x
// 4096, kWeight 525 for 505): a slot is free only when both are done, and 36 such clusters leave 8 SMs idle.
//
// Roles: warp 0 loads operand A and warp 2 operand B, 64 steps of the reduction a stage, into a ring
// in shared memory (a pair's copies complete the leading CTA's barriers); warp 3 overwrites rows
// (kWeight); warp 1 of the leading CTA issues the MMAs; warps 4-11, two groups, round the
// sums of one accumulator and store them while the MMAs fill the other; a weight gradient of more rows than
// a part has is added up in their registers, which they get from the other warps.  Every wait
// is bounded: one that gives up records MOE_ERR_TIMEOUT and the CTA winds down.
#include <cmath>

#include "experts16.h"
#include "mx_tc.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kThreads = 384;
constexpr int kAWarp = 0, kMmaWarp = 1, kBWarp = 2, kFixWarp = 3, kEpiWarp0 = 4;
constexpr int kMaxExperts = 1024;
constexpr int kABytes = 128 * 128;  // 128 channels x 64 steps
constexpr int kOutRows = 32;        // of an epilogue group's store, x 128 channels
constexpr int kBoxes = 3, kBoxRows = 64;
constexpr int kMaxSplit = 4;
// kWeight, sums in parts: the stages of a part at most (see there), and the registers a thread is launched with and
// goes on with: roles, epilogue.
__host__ __device__ constexpr int part_of(bool bf16, bool out_f32) { return out_f32 ? (bf16 ? 12 : 8) : bf16 ? 512 : 64; }
template <bool BF16, bool OUT_F32>
__device__ __forceinline__ int parts_of(int rows) {
  constexpr int kRows = part_of(BF16, OUT_F32) * 64;
  return (rows + kRows - 1) / kRows;
}
__device__ __forceinline__ int parts_of(bool bf16, bool out_f32, int rows) {  // divided by constants
  if (out_f32) return bf16 ? parts_of<true, true>(rows) : parts_of<false, true>(rows);
  return bf16 ? parts_of<true, false>(rows) : parts_of<false, false>(rows);
}
constexpr int kLaunchRegs = 168, kRoleRegs = 72, kEpiRegs = 216;
static_assert(128 * kRoleRegs + 256 * kEpiRegs <= kThreads * kLaunchRegs, "an increase past the launch's registers never ends");

template <int kLeft>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}
template <uint32_t kRegs>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <uint32_t kRegs>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }

// kWeight: items of few stages, or of many; or either, some of them in parts (`launch_gmm16`).
enum class Sums { kFew, kMany, kFewParts, kParts };

template <Gmm16 KIND, int NT, bool PAIR, Sums SUMS>
struct Cfg {
  static constexpr bool kWeight = KIND == Gmm16::kWeight;
  static constexpr int kStep = PAIR ? 32 : 16;
  static constexpr int kCtaCols = PAIR ? NT / 2 : NT;
  // 64-deep parts of a stage: two where few columns make the MMAs so short that a stage's commit counts
  static constexpr int kParts = !PAIR && NT <= 32 ? 2 : 1, kDeep = 64 * kParts;
  static constexpr int kBBytes = kCtaCols * 128;  // of a part
  static constexpr int kStageBytes = kParts * (kABytes + kBBytes);  // the parts of A, then those of B
  static constexpr bool kFew = SUMS == Sums::kFew || SUMS == Sums::kFewParts;
  static constexpr bool kInParts = SUMS == Sums::kParts || SUMS == Sums::kFewParts;
  static constexpr int kStages = kWeight && (kFew || !PAIR) ? 5 : PAIR || NT > 32 ? 6 : 5;
  // kWeight: pairs' pieces of 4 KB a warp (32 channels x 128 bytes), or a block's sums in fp32; else 8 KB a
  // group, or the sums of a tile of 32 rows
  static constexpr bool kSplits = !PAIR && (kWeight || NT <= 32);
  static constexpr int kPieces = kFew ? 2 : 1;
  static constexpr int kEpiBytes = kWeight ? (PAIR ? 8 * kPieces * 4096 : NT * 512) : 2 * kOutRows * 256;
  static constexpr int kTmemCols = 2 * NT <= 64 ? 64 : 2 * NT <= 256 ? 256 : 512;
  static_assert(!kSplits || kEpiBytes >= NT * 512, "an item's sums");
  static constexpr int kSmem = kStages * kStageBytes + kEpiBytes;
  static_assert(kStageBytes % 1024 == 0 && 2 * NT <= kTmemCols, "swizzled rows, tensor memory");
  static_assert(kSmem + (kWeight ? 1024 : 9 * 1024) <= 227 * 1024, "shared memory");
};

struct Args {
  int R, E, N, D;
  const int32_t* cumsum;
  void* out;
  int32_t* status;
  bool bf16, out_f32, accumulate;
  int split;
};

// a: operand A; b: operand B in boxes of 64, 32 and 16 rows (kWeight: b[0] alone); out.
struct Maps {
  CUtensorMap a, b[kBoxes], out;
};

// Instruction descriptor of kind::f16 with fp32 sums: operands both binary16 or both bfloat16, M =
// 128 (a CTA) or 256 (a pair).
__device__ __forceinline__ uint32_t f16_idesc(bool bf16, bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Descriptor of an MN-major operand in the 128-byte swizzle: boxes of 64 channels (128 bytes) x 64
// steps of the reduction; 8 steps are 1024 bytes, the next 64 channels 8192 bytes on.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(8192 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

template <bool PAIR>
__device__ __forceinline__ void f16_mma(uint32_t elected, uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "setp.ne.u32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "setp.ne.u32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

// Boxes of a tensor map to this CTA's shared memory, completing `bar`: of this CTA or, in a pair, of either.
template <bool PAIR>
__device__ __forceinline__ void load_2d(uint32_t elected, uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                        uint32_t bar) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.u32 e, %5, 0;\n\t"
        "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar), "r"(elected)
        : "memory");
  else
    tma_load_2d_elect(elected, dst, tmap, x, y, bar);
}
template <bool PAIR>
__device__ __forceinline__ void load_3d(uint32_t elected, uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                        int32_t z, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.u32 e, %6, 0;\n\t"
        "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.u32 e, %6, 0;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(elected)
        : "memory");
}
// Tiled store of a 3-D map's box, or its addition (fp32) to what is there.
__device__ __forceinline__ void tma_store_3d(const void* tmap, int32_t x, int32_t y, int32_t z, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void tma_add_3d(const void* tmap, int32_t x, int32_t y, int32_t z, const void* src) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}

// Two sums as a pair of the output's type (lo, hi): bits.
__device__ __forceinline__ uint32_t pack16(bool bf16, uint32_t lo, uint32_t hi) {
  const float a = __uint_as_float(lo), b = __uint_as_float(hi);
  if (bf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = f2h2_sat(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// An arrival on the leading CTA's barrier that publishes what this thread has stored itself, to the
// whole cluster; and the wait for it.  Only stages with overwritten rows pay for these, and never the
// warp that issues MMAs (a wait of cluster scope there took 6% of the weights' gradient).
__device__ __forceinline__ void mbar_arrive_remote_release(uint32_t caddr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}
__device__ __forceinline__ void mbar_acquire_cluster(uint64_t* bar, uint32_t parity) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(parity)
      : "memory");
}

__device__ __forceinline__ float ld_cluster1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void mbar_arrive_twice(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 2;" ::"r"(smem_u32(bar)) : "memory");
}

// kWeight: whether a stage of which `left` rows are the expert's is overwritten behind them: an MMA takes 16.
__device__ __forceinline__ bool fixed(int left) { return left < 64 && (left & 15) != 0; }

struct Item {
  int e, cb;          // expert, block of the MMA's rows (of a CTA or a pair)
  int row0, rows, n;  // kForward, kInput: the tile's rows; MMA columns.  kWeight: the expert's rows
  int col0;           // kWeight: first column
};

struct WorkList {
  const int* pref;  // first item of each expert; pref[E] = their number
  const int* end;   // last row of each expert + 1
  int CB, E;
};

template <int NT>
__device__ __forceinline__ int tiles_of(int start, int end) {
  return end > start ? (end - start + NT - 1) / NT : 0;
}

// An expert's rows are cut into t tiles of two sizes, multiples of the step that differ by it, the larger ones
// first and as few as cover the rows (of one size, 800 rows would be four
// of 224: 16 experts of 800 x 4096 x 2816 198 us for 192).
template <int NT, int STEP>
__device__ __forceinline__ Item tile_item(int j, const WorkList& wl, int& e_hint) {
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
  const int start = lo ? wl.end[lo - 1] : 0, end = wl.end[lo];
  const int t = tiles_of<NT>(start, end), steps = (end - start + STEP - 1) / STEP, less = steps / t, more = steps - less * t;
  const int local = j - wl.pref[lo], rt = local / wl.CB;
  Item it;
  it.e = lo;
  it.cb = local - rt * wl.CB;
  it.row0 = start + (rt * less + min(rt, more)) * STEP;
  it.n = (less + (rt < more ? 1 : 0)) * STEP;
  it.rows = min(it.n, end - it.row0);
  it.col0 = 0;
  return it;
}

__device__ __forceinline__ int end_of(const Args& a, int e) {
  return e < 0 ? 0 : min(max(__ldcg(a.cumsum + e), 0), a.R);
}

// The items that a role of a CTA goes through: the current one, `look` behind its first stage, `next` at its
// end.
template <int NT, int STEP>
struct TileItems {
  WorkList wl;
  int total, stride, j, e_hint = 0;
  Item it;
  __device__ __forceinline__ TileItems(const WorkList& wl_, int total_, int first, int stride_)
      : wl(wl_), total(total_), stride(stride_), j(first) {
    if (j < total) it = tile_item<NT, STEP>(j, wl, e_hint);
  }
  __device__ __forceinline__ bool more() const { return j < total; }
  __device__ __forceinline__ void look() {}
  __device__ __forceinline__ void next() {
    j += stride;
    if (j < total) it = tile_item<NT, STEP>(j, wl, e_hint);
  }
};

// kWeight: blocks of 256 x 256, columns innermost.  There is no room for the prefix in shared memory, and
// its latency in global memory between items left the tensor cores idle (12288 rows x 2816 x 4096 on 16
// experts 192 us, looked up ahead 183).
template <int NT, int STEP>
struct BlockItems {
  const Args& a;
  int total, stride, j, cols, per, de, dl, e, local, lo, hi;  // local: the item within its expert
  Item it;
  __device__ __forceinline__ BlockItems(const Args& a_, int CB, int total_, int first, int stride_)
      : a(a_), total(total_), stride(stride_), j(first) {
    cols = (a.D + NT - 1) / NT;
    per = CB * cols;
    e = j / per;
    local = j - e * per;
    de = stride / per;
    dl = stride - de * per;
    fetch();
    set();
  }
  __device__ __forceinline__ bool more() const { return j < total; }
  __device__ __forceinline__ void fetch() {
    lo = e > 0 && e < a.E ? __ldcg(a.cumsum + e - 1) : 0;
    hi = e < a.E ? __ldcg(a.cumsum + e) : 0;
  }
  __device__ __forceinline__ void look() {
    const int was = e;
    e += de;
    local += dl;
    if (local >= per) {
      local -= per;
      ++e;
    }
    if (e != was) fetch();  // a group that leaves an item to the other has nothing to hide it behind
  }
  __device__ __forceinline__ void set() {
    it.e = e;
    it.cb = local / cols;
    it.col0 = (local - it.cb * cols) * NT;
    it.row0 = min(max(lo, 0), a.R);
    it.rows = max(min(max(hi, 0), a.R) - it.row0, 0);
    it.n = (min(NT, a.D - it.col0) + STEP - 1) & -STEP;
  }
  __device__ __forceinline__ void next() {
    j += stride;
    set();
  }
};

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

template <Gmm16 KIND, int NT, bool PAIR, Sums SUMS>
__global__ void __launch_bounds__(kThreads, 1) gmm16_kernel(const __grid_constant__ Maps maps, const Args a) {
  using C = Cfg<KIND, NT, PAIR, SUMS>;
  constexpr bool PARTS = C::kInParts;
  constexpr int S = C::kStages;
  constexpr bool W = C::kWeight, A_MN = KIND != Gmm16::kForward, FIX = W;
  constexpr bool TURNS = W && PAIR;  // the epilogue's groups have accumulators of their own
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // swizzled rows: 1024-byte groups
  __shared__ __align__(8) uint64_t full_bar[S], tail_bar[W ? S : 1], peer_bar[W ? S : 1], empty_bar[S];
  __shared__ __align__(8) uint64_t accfull_bar[TURNS ? 4 : 2], accempty_bar[TURNS ? 4 : 2], stored_bar[2], final_bar;
  __shared__ __align__(8) uint64_t sums_bar, read_bar;  // of a cluster that divides the reduction
  __shared__ int s_pref[W ? 1 : kMaxExperts + 1], s_end[W ? 1 : kMaxExperts], s_wsum[kThreads / 32];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_issued[2];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int out_rows = KIND == Gmm16::kInput ? a.D : a.N;  // the MMA's rows in all
  const int NB = (out_rows + 127) / 128, CB = PAIR ? (NB + 1) / 2 : NB;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int split = C::kSplits ? a.split : 1, share = C::kSplits ? (int)cluster_ctarank() : 0;  // of the reduction
  const int ctas = PAIR ? 2 : split, first = blockIdx.x / ctas, stride = gridDim.x / ctas;
  volatile int* abort_flag = &s_abort;

  // ---- work list, barriers, tensor memory; what the kernels before this one wrote is read behind
  // the wait only
  if (warp == kMmaWarp) {
    tmem_alloc<PAIR, C::kTmemCols>(&s_tmem);
    if (lane == 0) {
      prefetch_tmap(&maps.a);
      for (int b = 0; b < (W ? 1 : kBoxes); ++b) prefetch_tmap(&maps.b[b]);
      prefetch_tmap(&maps.out);
      for (int s = 0; s < S; ++s) {
        mbar_init(&full_bar[s], 2);
        if (W) {
          mbar_init(&tail_bar[s], 2);
          mbar_init(&peer_bar[s], 1);
        }
        mbar_init(&empty_bar[s], 1);
      }
      for (int s = 0; s < (TURNS ? 4 : 2); ++s) {  // by 2 * group + accumulator
        mbar_init(&accfull_bar[s], 1);
        mbar_init(&accempty_bar[s], (PAIR ? 2 : 1) * (TURNS ? 4 : 8));
      }
      for (int s = 0; s < 2; ++s) mbar_init(&stored_bar[s], 4);
      mbar_init(&final_bar, 1);
      mbar_init(&sums_bar, 8 * split);
      mbar_init(&read_bar, 8 * split);
      fence_barrier_init();
    }
    tc_fence_before();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;  // long before any wait can run out
  if (threadIdx.x == 0) {
    s_abort = 0;
    s_issued[0] = s_issued[1] = 0;
  }
  int total;
  if (W) {
    total = a.E * CB * ((a.D + NT - 1) / NT);
    __syncthreads();
  } else {
    const int E = a.E, per = (E + kThreads - 1) / kThreads;
    const int e0 = min(E, (int)threadIdx.x * per), e1 = min(E, e0 + per);
    int local = 0;
    for (int e = e0; e < e1; ++e) {
      s_end[e] = end_of(a, e);
      local += tiles_of<NT>(end_of(a, e - 1), s_end[e]) * CB;
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) s_wsum[warp] = incl;
    __syncthreads();
    int run = incl - local;
    for (int w = 0; w < warp; ++w) run += s_wsum[w];
    for (int e = e0; e < e1; ++e) {
      s_pref[e] = run;
      run += tiles_of<NT>(e ? s_end[e - 1] : 0, s_end[e]) * CB;
    }
    if (e0 < E && e1 == E) s_pref[E] = run;
    __syncthreads();
    total = s_pref[E];
  }
  __syncwarp();
  if (ctas > 1) cluster_sync_all();  // the other CTAs' barriers and tensor memory are ready
  tc_fence_after();
  const WorkList wl{s_pref, s_end, CB, a.E};
  const uint32_t tmem = s_tmem;
  const uint32_t ring = smem_u32(smem_raw);
  // kForward, kInput: stages of every item
  const int depth = KIND == Gmm16::kForward ? a.D : a.N;
  auto items = [&](int from, int by) {
    if constexpr (W) return BlockItems<NT, C::kStep>(a, CB, total, from, by);
    else return TileItems<NT, C::kStep>(wl, total, from, by);
  };
  auto steps = [&](const Item& it) { return W ? it.rows : depth; };  // of the reduction
  // stages of an item that are this CTA's: [kb0, kb1) of KB (each of a cluster has one at least)
  auto stage0 = [&](int KB) { return split == 1 ? 0 : share * KB / split; };
  auto stage1 = [&](int KB) { return split == 1 ? KB : (share + 1) * KB / split; };

  // An accumulator takes an item's whole sum; of a weight gradient, one of so many rows at most, where it could have
  // more.  The tensor cores add 16 products a step and drop what lies below the sum's last place, always towards zero:
  // two units of it at most, 2^-27 n of the magnitudes of n products.  (Measured, of the norm: n random products
  // 1.3e-9 n in binary16, 1e-9 n in bfloat16; of one sign up to 6e-9 n.)  A longer sum is made in parts,
  // added in registers, or in shared memory where CTAs divide the rows.
  //   16-bit output: 64 stages of binary16, 512 of bfloat16; 2^-27 n is a sixteenth of half a step there.
  //   fp32 output: 8 stages of binary16 (up to 65536 random products 6.7e-7 of the norm, of one sign 2.4e-6), 12 of
  //   bfloat16 (7.4e-7, 6.2e-7).  With 8 for bfloat16 too (4.7e-7) experts of 768 rows would be in two parts: 64 of
  //   them, 4096 x 1408, took 4% more instead of 2.  The additions of the parts round as well: 2^20 random products
  //   8e-7, 2^24 1.7e-6.
  const int most = part_of(a.bf16, a.out_f32);
  auto whole_sum = [&](int n) { return W && (PARTS || !PAIR) ? n <= most * 64 : true; };
  if (warp < kEpiWarp0) {
    if (PARTS) regs_dec<kRoleRegs>();
    if (warp == kAWarp || warp == kBWarp) {
      const uint32_t elected = elect_one();
      const uint32_t full0 = PAIR ? cluster_addr(&full_bar[0], 0) : smem_u32(&full_bar[0]);
      RingPos at;
      int n = 0;
      bool ok = true;
      for (auto list = items(first, stride); ok && list.more(); list.next()) {
        const Item it = list.it;
        list.look();
        const int m0 = (PAIR ? 2 * it.cb + (int)rank : it.cb) * 128;  // past the last: the copies bring zeros
        const int cta_cols = PAIR ? it.n / 2 : it.n, deep = steps(it), KB = (deep + C::kDeep - 1) / C::kDeep;
        const int c0 = (W ? it.col0 : it.row0) + (int)rank * cta_cols;
        for (int kb = stage0(KB), kb1 = stage1(KB); kb < kb1; ++kb, ++n, at.next(S)) {
          if (!(ok = warp_wait(&empty_bar[at.slot], at.phase ^ 1u, abort_flag, a.status))) break;
          const uint32_t st = ring + at.slot * C::kStageBytes;
          const int k0 = kb * C::kDeep, parts = C::kParts == 2 && k0 + 64 < deep ? 2 : 1;
          // The copies of both CTAs of a pair complete the leading one's barrier, which expects the bytes of both;
          // those of a stage whose last rows are overwritten complete each CTA's own.
          const bool fix = W && fixed(deep - k0);
          const uint32_t bar = fix ? smem_u32(&tail_bar[W ? at.slot : 0]) : full0 + at.slot * 8;
          const uint32_t expecting = PAIR && !fix ? (rank == 0 ? elected : 0u) : elected, times = PAIR && !fix ? 2 : 1;
          const uint32_t expected = fix ? bar : smem_u32(&full_bar[at.slot]);
          if (warp == kAWarp) {
            expect_tx_elect(expecting, expected, times * (uint32_t)parts * kABytes);
#pragma unroll
            for (int q = 0; q < C::kParts; ++q) {
              if (q >= parts) break;
              const uint32_t to = st + q * kABytes;
              const int k = k0 + q * 64;
              if (KIND == Gmm16::kForward) {
                load_3d<PAIR>(elected, to, &maps.a, k, m0, it.e, bar);
              } else if (KIND == Gmm16::kInput) {
                load_3d<PAIR>(elected, to, &maps.a, m0, k, it.e, bar);
                load_3d<PAIR>(elected, to + 8192, &maps.a, m0 + 64, k, it.e, bar);
              } else {
                load_2d<PAIR>(elected, to, &maps.a, m0, it.row0 + k, bar);
                load_2d<PAIR>(elected, to + 8192, &maps.a, m0 + 64, it.row0 + k, bar);
              }
            }
          } else if (W) {
            const int boxes = (cta_cols + 63) / 64;
            expect_tx_elect(expecting, expected, times * (uint32_t)boxes * 8192);
            for (int b = 0; b < boxes; ++b)
              load_2d<PAIR>(elected, st + kABytes + b * 8192, &maps.b[0], c0 + b * 64, it.row0 + k0, bar);
          } else {
            expect_tx_elect(expecting, expected, times * (uint32_t)(parts * cta_cols) * 128);
#pragma unroll
            for (int q = 0; q < C::kParts; ++q) {
              if (q >= parts) break;
              int r = 0;
#pragma unroll
              for (int b = 0; b < kBoxes; ++b) {
                const int rows = kBoxRows >> b;
                for (; cta_cols - r >= rows; r += rows)
                  load_2d<PAIR>(elected, st + C::kParts * kABytes + q * C::kBBytes + r * 128, &maps.b[b], k0 + q * 64, c0 + r,
                                bar);
              }
            }
          }
        }
      }
      // the next kernel's setup beside the last items
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      // the last stages' releases: commits arrive in both CTAs of a pair, and neither may leave
      // before an arrival that is still on its way to it
      for (int s = 0; ok && s < S; ++s, at.next(S)) ok = warp_wait(&empty_bar[at.slot], at.phase ^ 1u, abort_flag, a.status);
      if (lane == 0) s_issued[warp == kBWarp] = n;
    } else if (FIX && warp == kFixWarp) {
      if constexpr (FIX) {
        RingPos at;
        uint32_t turn = 0;  // parity of each slot's next use of tail_bar and peer_bar
        bool ok = true;
        for (auto list = items(first, stride); ok && list.more(); list.next()) {
          const Item it = list.it;
          list.look();
          const int KB = (it.rows + 63) / 64;
          for (int kb = stage0(KB), kb1 = stage1(KB); ok && kb < kb1; ++kb, at.next(S)) {
            const int left = it.rows - kb * 64;
            if (!fixed(left)) continue;
            const uint32_t parity = turn >> at.slot & 1u;
            turn ^= 1u << at.slot;
            if (!(ok = warp_wait(&tail_bar[at.slot], parity, abort_flag, a.status))) break;
            // rows of the next expert, in the four boxes of both operands (a row is 128 bytes of each)
            uint8_t* box = smem_raw + at.slot * C::kStageBytes + (lane >> 3) * 8192 + (lane & 7) * 16;
            for (int r = left; r < ((left + 15) & ~15); ++r) *reinterpret_cast<uint4*>(box + r * 128) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (rank == 1) {
              if (lane == 0) mbar_arrive_remote_release(cluster_addr(&peer_bar[at.slot], 0));
            } else {
              if (PAIR) {
                if (!(ok = warp_wait(&peer_bar[at.slot], parity, abort_flag, a.status))) break;
                mbar_acquire_cluster(&peer_bar[at.slot], parity);
                __syncwarp();
              }
              if (lane == 0) mbar_arrive_twice(&full_bar[at.slot]);  // in place of the loaders
            }
          }
        }
      }
    } else if (warp == kMmaWarp) {
      if (rank == 0) {
        const uint32_t elected = elect_one(), t0 = __shfl_sync(0xffffffffu, tmem, 0);
        RingPos at;
        int u = 0;
        uint32_t held = 0, back = 0;  // kWeight: by 2 * group + accumulator, handed over, and its return's parity
        bool ok = true;
        // a barrier's answer takes as long as issuing several MMAs: the next stage's is asked for
        // before this one's are issued
        uint32_t there = mbar_test(&full_bar[0], 0);
        for (auto list = items(first, stride); ok && list.more(); list.next()) {
          const Item it = list.it;
          const int n = steps(it), KB = (n + C::kDeep - 1) / C::kDeep, kb0 = stage0(KB), kb1 = stage1(KB);
          const bool whole = whole_sum(W && !PAIR ? (kb1 - kb0) * 64 : n);
          const uint32_t idesc = f16_idesc(a.bf16, A_MN, W, PAIR ? 256 : 128, it.n);
          int from = kb0;
          do {
            const int buf = u & 1;
            int to = kb1;
            if (!whole && to - from > most) to = to - from > 2 * most ? from + most : (from + to + 1) >> 1;
            if constexpr (TURNS) {  // from those that have it
              for (int i = buf; ok && i < 4; i += 2)
                if (held >> i & 1u) {
                  ok = warp_wait(&accempty_bar[i], back >> i & 1u, abort_flag, a.status);
                  held ^= 1u << i, back ^= 1u << i;
                }
            } else {
              ok = warp_wait(&accempty_bar[buf], ((u >> 1) & 1) ^ 1, abort_flag, a.status);
            }
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = t0 + buf * NT;
            for (int kb = from; kb < to; ++kb) {
              if (!__all_sync(0xffffffffu, there) &&
                  !(ok = warp_wait(&full_bar[at.slot], at.phase, abort_flag, a.status)))
                break;
              tc_fence_after();
              const uint32_t st = ring + at.slot * C::kStageBytes;
              const uint64_t da = A_MN ? sw128_mn_desc(st) : sw128_desc(st);
              const uint64_t db = W ? sw128_mn_desc(st + kABytes) : sw128_desc(st + C::kParts * kABytes);
              const uint32_t done = smem_u32(&empty_bar[at.slot]);
              at.next(S);
              there = mbar_test(&full_bar[at.slot], at.phase);
              const int last = min(4 * C::kParts, (n - kb * C::kDeep + 15) >> 4);  // 16 steps an MMA
#pragma unroll
              for (int k = 0; k < 4 * C::kParts; ++k)
                if (k < last)
                  f16_mma<PAIR>(elected, d, da + (k >> 2) * (kABytes >> 4) + (k & 3) * (A_MN ? 128 : 2),
                                db + (k >> 2) * (C::kBBytes >> 4) + (k & 3) * (W ? 128 : 2), idesc, kb > from || k ? 1u : 0u);
              mx_commit<PAIR>(elected, done);
              if (kb == kb0) list.look();
            }
            if (!ok) break;
            if constexpr (TURNS) {
              const uint32_t who = whole ? 1u << (3 * buf) : 5u << buf;  // the accumulator's group, or both
              for (int i = buf; i < 4; i += 2)
                if (who >> i & 1u) mx_commit<PAIR>(elected, smem_u32(&accfull_bar[i]));
              held |= who;
            } else {
              mx_commit<PAIR>(elected, smem_u32(&accfull_bar[buf]));
            }
            from = to;
            ++u;
          } while (from < kb1);
          if (kb0 == kb1) list.look();
        }
        mx_commit_local<PAIR>(elected, smem_u32(&final_bar));  // every MMA done before tensor memory is freed
        mbar_wait_sleep_bounded(&final_bar, 0);
      }
    }
  } else {
    if (PARTS) regs_inc<kEpiRegs>();
    // Both groups take part in every item, and drain one accumulator while the MMAs fill the other. But
    // those of kWeight take turns at items of one part, an accumulator each: together, their bursts of
    // stores slowed the loads (64 experts x 64 rows, 2816 x 4096: 302 us for 276). Each hears of, and hands
    // back, only what it takes.
    const int group = (warp - kEpiWarp0) >> 2, quarter = warp & 3;
    const uint32_t lanes = (uint32_t)quarter << 21;  // 32 * quarter in the lane field
    constexpr int by = TURNS && !PARTS ? 2 : 1;
    int u = by == 2 ? group : 0;
    int done = 0;     // items of a cluster's sums
    uint32_t at = 0;  // kWeight: the next piece's place
    uint32_t turn = 0;  // kWeight: parity of this group's next turn at each accumulator; from bit 2 on: items in parts
    auto heard = [&](int buf) {
      turn ^= 1u << buf;
      return warp_wait(&accfull_bar[TURNS ? 2 * group + buf : 0], ~turn >> buf & 1u, abort_flag, a.status);
    };
    for (auto list = items(first + u * stride, by * stride); list.more(); list.next(), u += by) {
      const Item it = list.it;
      list.look();
      const int buf = u & 1;
      const bool whole = whole_sum(it.rows);
      if (TURNS && whole && buf != group) continue;
      bool ok = TURNS ? heard(buf) : warp_wait(&accfull_bar[buf], (u >> 1) & 1, abort_flag, a.status);
      // warps that wait for one another below give up together
      if (!C::kSplits || split == 1)
        if (!TURNS) ok = group_all(9 + group, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t = tmem + lanes + buf * NT;
      const int m0 = (PAIR ? 2 * it.cb + (int)rank : it.cb) * 128;
      if constexpr (TURNS) {
        // 32 channels of a warp, 128 bytes of columns at a time, in the 128-byte swizzle of the output's map
        uint8_t* own = smem_raw + S * C::kStageBytes + (warp - kEpiWarp0) * C::kPieces * 4096;
        const int y = m0 + quarter * 32;
        const bool stored = y < a.N && (it.rows || !a.accumulate);
        auto put = [&](int c) {  // the rows are in shared memory
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (a.accumulate) tma_add_3d(&maps.out, it.col0 + c, y, it.e, own + at);
            else tma_store_3d(&maps.out, it.col0 + c, y, it.e, own + at);
            bulk_commit_group();
          }
          if (C::kPieces == 2) at ^= 4096;
        };
        auto row = [&](int i) -> uint4& { return reinterpret_cast<uint4*>(own + at + lane * 128)[i ^ (lane & 7)]; };
        auto release = [&](int n) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(cluster_addr(&accempty_bar[2 * group + n], 0));
        };
        if (whole) {
          const int cols = a.out_f32 ? 32 : 64;
          if (stored) {
            for (int c = 0; c < it.n; c += cols) {
              uint32_t v[4][16];
              __syncwarp();
              if (it.rows) {
                tmem_ld16(t + c, v[0]);
                tmem_ld16(t + c + 16, v[1]);  // a pair's columns come in steps of 32
                if (!a.out_f32 && c + 32 < it.n) {
                  tmem_ld16(t + c + 32, v[2]);
                  tmem_ld16(t + c + 48, v[3]);
                }
                tmem_wait_ld();
              } else {
#pragma unroll
                for (int i = 0; i < 64; ++i) v[i >> 4][i & 15] = 0;
              }
              bulk_wait_read<C::kPieces - 1>();
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                uint4 o;
                if (a.out_f32) {
                  const int k = (i & 3) * 4;
                  o = make_uint4(v[i >> 2][k], v[i >> 2][k + 1], v[i >> 2][k + 2], v[i >> 2][k + 3]);
                } else {
                  const int k = (i & 1) * 8;
                  const uint32_t(&x)[16] = v[i >> 1];
                  o = make_uint4(pack16(a.bf16, x[k], x[k + 1]), pack16(a.bf16, x[k + 2], x[k + 3]),
                                 pack16(a.bf16, x[k + 4], x[k + 5]), pack16(a.bf16, x[k + 6], x[k + 7]));
                }
                row(i) = o;
              }
              put(c);
            }
          }
          release(buf);
          continue;
        }
        // A lane's channel, 128 columns of it to a group: drained into registers, where the parts are added,
        // and the accumulators free again before anything is stored.
        float sum[128] = {};
        const int from = group * 128, parts = parts_of(a.bf16, a.out_f32, it.rows);
        for (int part = 0; part < parts; ++part) {
          if (part) {
            ++u;
            if (!(ok = heard(u & 1))) break;
            tc_fence_after();
          }
#pragma unroll
          for (int c = 0; c < 128; c += 32)
            if (from + c < it.n) {
              uint32_t v[2][16];
              __syncwarp();
              tmem_ld16(tmem + lanes + (u & 1) * NT + from + c, v[0]);
              tmem_ld16(tmem + lanes + (u & 1) * NT + from + c + 16, v[1]);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) sum[c + i] += __uint_as_float(v[i >> 4][i & 15]);
            }
          release(u & 1);
        }
        if (!ok) break;
        // The second group stores behind the first (16 experts x 1536 rows, 2816 x 4096: 373 us for 383). The
        // first is never two items ahead: their parts take the accumulators that the second still has.
        uint64_t* before = &stored_bar[turn >> 2 & 1u];
        const uint32_t parity = turn >> 3 & 1u;
        turn += 4;
        if (group == 1 && !warp_wait(before, parity, abort_flag, a.status)) break;
        if (a.out_f32) {
#pragma unroll
          for (int c = 0; c < 128; c += 32)
            if (stored && from + c < it.n) {
              bulk_wait_read<C::kPieces - 1>();
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                row(i) = make_uint4(__float_as_uint(sum[c + 4 * i]), __float_as_uint(sum[c + 4 * i + 1]),
                                    __float_as_uint(sum[c + 4 * i + 2]), __float_as_uint(sum[c + 4 * i + 3]));
              put(from + c);
            }
        } else {
#pragma unroll
          for (int c = 0; c < 128; c += 64)
            if (stored && from + c < it.n) {
              bulk_wait_read<C::kPieces - 1>();
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                uint32_t x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  x[k] = pack16(a.bf16, __float_as_uint(sum[c + 8 * i + 2 * k]), __float_as_uint(sum[c + 8 * i + 2 * k + 1]));
                row(i) = make_uint4(x[0], x[1], x[2], x[3]);
              }
              put(from + c);
            }
        }
        if (group == 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(before);
        }
        continue;
      } else if (C::kSplits && (W || split > 1)) {
        float* sums = reinterpret_cast<float*>(smem_raw + S * C::kStageBytes);  // [rows][128]
        const int wg = warp - kEpiWarp0, th = wg * 32 + lane, KB = (steps(it) + C::kDeep - 1) / C::kDeep;
        const int own = stage1(KB) - stage0(KB);  // 0: so are its sums
        const int parts = whole_sum(own * 64) ? 1 : parts_of(a.bf16, a.out_f32, own * 64);
        // everybody has read the item before
        if (done > 0 && !warp_wait(&read_bar, (done - 1) & 1, abort_flag, a.status)) break;
        for (int part = 0; part < parts; ++part) {
          if (part) {
            ++u;
            if (!(ok = warp_wait(&accfull_bar[u & 1], (u >> 1) & 1, abort_flag, a.status))) break;
            tc_fence_after();
          }
          for (int c0 = group * 16; c0 < it.n; c0 += 32) {
            uint32_t v[16] = {};
            __syncwarp();
            if (!W || own) {
              tmem_ld16(tmem + lanes + (u & 1) * NT + c0, v);
              tmem_wait_ld();
            }
            float* o = sums + c0 * 128 + quarter * 32 + lane;
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i * 128] = part ? o[i * 128] + __uint_as_float(v[i]) : __uint_as_float(v[i]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&accempty_bar[u & 1]);
        }
        if (!ok) break;
        if (lane < split) mbar_arrive_remote_release(cluster_addr(&sums_bar, lane));
        if (!warp_wait(&sums_bar, done & 1, abort_flag, a.status)) break;
        mbar_acquire_cluster(&sums_bar, done & 1);
        ++done;
        // eight channels of a row to a thread, the tile's pieces dealt out over the cluster
        const int width = min(128, out_rows - m0);
        if constexpr (W) {  // eight columns of a channel
          const int n = it.rows || !a.accumulate ? min(NT, a.D - it.col0) / 8 * 128 : 0;
          for (int i = share * 256 + th; i < n; i += split * 256) {
            const int ch = i & 127, c = (i >> 7) * 8;
            float y[kMaxSplit][8], x[8] = {};
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
              if (q < split)
#pragma unroll
                for (int k = 0; k < 8; ++k) y[q][k] = ld_cluster1(cluster_addr(sums + (c + k) * 128 + ch, q));
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
              if (q < split)
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] += y[q][k];
            if (ch >= width) continue;
            const size_t at = ((size_t)it.e * a.N + m0 + ch) * a.D + it.col0 + c;
            if (a.out_f32) {
              float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
              float4 lo = make_float4(x[0], x[1], x[2], x[3]), hi = make_float4(x[4], x[5], x[6], x[7]);
              if (a.accumulate) {
                const float4 l = o[0], h = o[1];
                lo = make_float4(l.x + lo.x, l.y + lo.y, l.z + lo.z, l.w + lo.w);
                hi = make_float4(h.x + hi.x, h.y + hi.y, h.z + hi.z, h.w + hi.w);
              }
              o[0] = lo;
              o[1] = hi;
            } else {
              uint4 o;
              o.x = pack16(a.bf16, __float_as_uint(x[0]), __float_as_uint(x[1]));
              o.y = pack16(a.bf16, __float_as_uint(x[2]), __float_as_uint(x[3]));
              o.z = pack16(a.bf16, __float_as_uint(x[4]), __float_as_uint(x[5]));
              o.w = pack16(a.bf16, __float_as_uint(x[6]), __float_as_uint(x[7]));
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) = o;
            }
          }
        }
        for (int i = share * 256 + th; !W && i < it.rows * 16; i += split * 256) {
          const int r = i >> 4, c = (i & 15) * 8;
          float4 y[kMaxSplit][2];
#pragma unroll
          for (int q = 0; q < kMaxSplit; ++q)
            if (q < split) {
              const uint32_t from = cluster_addr(sums + r * 128 + c, q);
              y[q][0] = ld_cluster4(from);
              y[q][1] = ld_cluster4(from + 16);
            }
          float x[8] = {};
#pragma unroll
          for (int q = 0; q < kMaxSplit; ++q)
            if (q < split)
#pragma unroll
              for (int k = 0; k < 8; ++k) x[k] += reinterpret_cast<const float*>(y[q])[k];
          if (c < width) {
            uint4 o;
            o.x = pack16(a.bf16, __float_as_uint(x[0]), __float_as_uint(x[1]));
            o.y = pack16(a.bf16, __float_as_uint(x[2]), __float_as_uint(x[3]));
            o.z = pack16(a.bf16, __float_as_uint(x[4]), __float_as_uint(x[5]));
            o.w = pack16(a.bf16, __float_as_uint(x[6]), __float_as_uint(x[7]));
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (size_t)(it.row0 + r) * out_rows + m0 + c) = o;
          }
        }
        __syncwarp();  // what was read has been used: nothing to publish
        if (lane < split) mbar_arrive_remote(cluster_addr(&read_bar, lane));
        continue;
      } else {
        // 32 rows x 128 channels gathered in shared memory and stored from there by one tensor copy,
        // or, where the tile's last rows are not its own, row by row
        uint8_t* own = smem_raw + S * C::kStageBytes + group * (kOutRows * 256);
        const int width = min(128, out_rows - m0);  // channels; none of a pair's block past the last
        const int rows = width > 0 ? it.rows : 0;
        for (int c0 = group * kOutRows; c0 < it.n; c0 += 2 * kOutRows) {
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
          uint16_t* o = reinterpret_cast<uint16_t*>(own) + quarter * 32 + lane;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const uint32_t h = pack16(a.bf16, v[i >> 4][i & 15], v[i >> 4][(i & 15) + 1]);
            o[i * 128] = (uint16_t)h;
            o[i * 128 + 128] = (uint16_t)(h >> 16);
          }
          fence_proxy_async_smem();
          asm volatile("bar.sync %0, 128;" ::"r"(9 + group) : "memory");
          if (quarter == 0) {
            if (c0 + kOutRows <= rows) {
              if (lane == 0) tma_store_2d(&maps.out, m0, it.row0 + c0, own);
            } else if (c0 + lane < rows) {
              bulk_store(static_cast<uint16_t*>(a.out) + (size_t)(it.row0 + c0 + lane) * out_rows + m0, own + lane * 256,
                         (uint32_t)width * 2);
            }
            bulk_commit_group();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_remote(cluster_addr(&accempty_bar[buf], 0)); else mbar_arrive(&accempty_bar[buf]);
      }
    }
    bulk_wait_all();  // stores done before shared memory is released
  }

  __syncthreads();
  // copies still in flight (only after an abort) land before shared memory is released; those of a pair
  // complete the leading CTA's barriers, and the other waits for it below
  if (threadIdx.x == 0 && rank == 0) {
    const int n0 = min(s_issued[0], s_issued[1]), n1 = max(s_issued[0], s_issued[1]);
    for (int n = n0; n < n1; ++n) mbar_arrive(&full_bar[n % S]);  // stages that one of the two loaders never began
    for (int n = max(0, n1 - S); n < n1; ++n) mbar_wait_bounded(&full_bar[n % S], (n / S) & 1);
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (ctas > 1) cluster_sync_all();  // no CTA leaves while the others' MMAs, arrivals or reads may touch it
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<PAIR, C::kTmemCols>(tmem);
  }
}

// 3-D map [e][outer][inner] of `elem`-byte elements in the 128-byte swizzle.
bool encode_tensor_map_3d(CUtensorMap* m, CUtensorMapDataType dt, size_t elem, const void* base, uint64_t inner,
                          uint64_t outer, uint64_t e, uint32_t box_inner, uint32_t box_outer) {
  PFN_encodeTiled fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {inner, outer, e};
  cuuint64_t strides[2] = {inner * elem, inner * outer * elem};
  cuuint32_t box[3] = {box_inner, box_outer, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of this many CTAs, one to an SM, that the device holds at once (GB300: 152, 76 and 36 of 1, 2
// and 4: a cluster of four needs four SMs of one GPC).  CTAs take items whatever their number: where it is another,
// forms are chosen by a wrong count and some CTAs begin when others are done.
inline int resident_clusters(int ctas) {
  const int n = ctas <= 2 ? sm_count() / ctas : sm_count() / 19 * 18 / ctas;
  return n < 1 ? 1 : n;
}

template <Gmm16 KIND, int NT, bool PAIR, Sums SUMS = Sums::kMany>
cudaError_t launch(const Gmm16Problem& p, int split, cudaStream_t stream) {
  using C = Cfg<KIND, NT, PAIR, SUMS>;
  const CUtensorMapDataType t = p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const uint64_t R = p.R, E = p.E, N = p.N, D = p.D;
  Maps maps;
  bool ok;
  if (KIND == Gmm16::kWeight) {
    ok = encode_tensor_map_2d(&maps.a, t, 2, p.rows, N, R, 64, 64) && encode_tensor_map_2d(&maps.b[0], t, 2, p.rows2, D, R, 64, 64) &&
         (p.out_f32 ? encode_tensor_map_3d(&maps.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p.out, D, N, E, 32, 32)
                    : encode_tensor_map_3d(&maps.out, t, 2, p.out, D, N, E, 64, 32));
    maps.b[1] = maps.b[2] = maps.b[0];
  } else {
    const uint64_t depth = KIND == Gmm16::kForward ? D : N, outs = KIND == Gmm16::kForward ? N : D;
    ok = encode_tensor_map_3d(&maps.a, t, 2, p.w, D, N, E, 64, KIND == Gmm16::kForward ? 128 : 64) &&
         encode_tensor_map_2d(&maps.out, t, 2, p.out, outs, R, 128, kOutRows, CU_TENSOR_MAP_SWIZZLE_NONE);
    for (int b = 0; ok && b < kBoxes; ++b)
      ok = encode_tensor_map_2d(&maps.b[b], t, 2, p.rows, depth, R, 64, (uint32_t)kBoxRows >> b);
  }
  if (!ok) return cudaErrorInvalidValue;
  static PerContextOnce set;
  const int dev = current_device();
  if (set.needed(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(gmm16_kernel<KIND, NT, PAIR, SUMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (C::kInParts) {
      // launched with other registers than its split counts on, it would wait for them: the build refuses such a
      // kernel (build.py), and so does this
      cudaFuncAttributes fa;
      const cudaError_t q = cudaFuncGetAttributes(&fa, gmm16_kernel<KIND, NT, PAIR, SUMS>);
      if (q != cudaSuccess) return q;
      if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
    }
    set.done(dev);
  }
  Args a{p.R, p.E, p.N, p.D, p.cumsum, p.out, p.status, p.bf16, p.out_f32, p.accumulate, split};
  cudaLaunchConfig_t cfg = {};
  const int ctas = PAIR ? 2 : split;
  cfg.gridDim = dim3((unsigned)(resident_clusters(ctas) * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = (unsigned)ctas;
  attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gmm16_kernel<KIND, NT, PAIR, SUMS>, maps, a);
}

// What a form takes, in clocks: rounds of its items over the clusters that work at once, each the item's stages
// and what an item costs besides.  The host knows the rows per expert on average only.  Both sides, us
// (forward / gradient for the rows; `32 x 4` is the first form divided by four):
//                                          32      32 x 2     32 x 4      128        pairs
//   1 expert x 1, 4096 -> 4096            13.1      11.3       10.8       15.9        18.4
//   1 expert x 128                        13.7      17.1       22.1       18.1        20.3
//   1 expert x 512                                                        18.8        24.9
//   1 expert x 1024                                                       32.0        25.8
//   8 experts x 40, 4096 -> 2816       41 / 39   39 / 40    48 / 54    41 / 34     44 / 36
//   8 experts x 128                    51 / 50   55 / 59    81 / 101   44 / 36     46 / 37
//   64 experts x 64                   267 / 238 252 / 265  337 / 397  232 / 224   240 / 228
//   32 experts x 200, 2048 -> 1024     60 / 65   79 / 123  143 / 261   40 / 37     35 / 34
struct Form {
  int nt, split;  // columns of a tile; 256: pairs
  double stage;   // clocks of 64 steps of the reduction
};
Form choose(const Gmm16Problem& p) {
  const Form forms[] = {{32, 1, 290}, {32, 2, 290}, {32, kMaxSplit, 290}, {128, 1, 420}, {256, 1, 520}};
  const int outs = p.kind == Gmm16::kForward ? p.N : p.D, depth = p.kind == Gmm16::kForward ? p.D : p.N;
  const int experts = p.R < p.E ? p.R : p.E, KB = (depth + 63) / 64;
  const double rows = (double)p.R / experts;
  Form best{};
  double least = 0.0;
  for (const Form& f : forms) {
    if (f.split > 1 && KB < 4 * kMaxSplit) continue;  // each CTA of a cluster has a stage at least
    const int ctas = f.nt == 256 ? 2 : f.split, width = f.nt == 256 ? 256 : 128;
    const double items = experts * ceil(rows / f.nt) * ((outs + width - 1) / width);
    const double clocks =
        ceil(items / resident_clusters(ctas)) * ((KB + f.split - 1) / f.split * f.stage + (f.split > 1 ? 3000 : 800));
    if (!best.nt || clocks < least) {
      best = f;
      least = clocks;
    }
  }
  return best;
}

// kWeight of few blocks and many rows: blocks of 128 x 128, clusters of up to four CTAs that divide the rows of each
// (0: pairs after all), by the same count; larger clusters have not been measured.  Both sides, us (16 bits / fp32):            pairs      divided
//   1 expert x 16384 rows, 512 x 512                                      73 / 75      22 / 22
//   1 x 8192, 1024 x 1024                                                 40 / 41      22 / 23
//   4 x 2868, 72 x 928                                                    19 / 21      13 / 13
//   3 x 1400, 408 x 152                                                   14 / 15      10 / 10
//   2 x 653, 448 x 632                                                   9.3 / 10.7   8.7 / 9.2
int divide_rows(const Gmm16Problem& p) {
  const int experts = p.R < p.E ? p.R : p.E, KB = (p.R / experts + 63) / 64;
  auto blocks = [&](int m, int n) { return (double)experts * ((p.N + m - 1) / m) * ((p.D + n - 1) / n); };
  double least = ceil(blocks(256, 256) / resident_clusters(2)) * (KB * 520.0 + 1500);
  int best = 0;
  for (int split = 2; split <= kMaxSplit; split *= 2) {
    const double clocks = ceil(blocks(128, 128) / resident_clusters(split)) * ((KB + split - 1) / split * 420.0 + 3000);
    if (clocks < least) {
      best = split;
      least = clocks;
    }
  }
  return best;
}

template <Gmm16 KIND>
cudaError_t launch_rows(const Gmm16Problem& p, cudaStream_t stream) {
  const Form f = choose(p);
  return f.nt == 32    ? launch<KIND, 32, false>(p, f.split, stream)
         : f.nt == 128 ? launch<KIND, 128, false>(p, f.split, stream)
                       : launch<KIND, 256, true>(p, 1, stream);
}

}  // namespace

cudaError_t launch_gmm16(const Gmm16Problem& p, cudaStream_t stream) {
  if (p.kind == Gmm16::kWeight) {
    if (const int split = divide_rows(p)) return launch<Gmm16::kWeight, 128, false>(p, split, stream);
    // Shared memory of one of six stages for a second piece of a warp's sums, where an item has about as few stages
    // as pieces (us, with and without; 16 bits): 1 expert x 128 rows, 4096 x 4096 10.8 and 11.4, 8 x 75, 1416 x
    // 1024 10.3 and 10.7 (fp32 13.7 and 14.5; 64 x 75, 2816 x 4096 519 and 530), 8 x 256, 2816 x 4096 44.6 and 43.8,
    // 16 x 768 93.7 and 90.6.  In parts, if an expert could have more rows than one: the host knows only how
    // many there are in all.
    const int experts = p.R < p.E ? p.R : p.E;
    const bool few = p.R <= 192 * (int64_t)experts, parts = p.R > part_of(p.bf16, p.out_f32) * 64;
    if (parts)
      return few ? launch<Gmm16::kWeight, 256, true, Sums::kFewParts>(p, 1, stream)
                 : launch<Gmm16::kWeight, 256, true, Sums::kParts>(p, 1, stream);
    return few ? launch<Gmm16::kWeight, 256, true, Sums::kFew>(p, 1, stream)
               : launch<Gmm16::kWeight, 256, true, Sums::kMany>(p, 1, stream);
  }
  return p.kind == Gmm16::kForward ? launch_rows<Gmm16::kForward>(p, stream) : launch_rows<Gmm16::kInput>(p, stream);
}

}  // namespace moe
