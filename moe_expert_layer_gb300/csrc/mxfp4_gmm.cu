// Grouped MXFP4 product over expert-major rows on the block-scaled tensor cores
// (tcgen05.mma kind::mxf4), with SwiGLU and requantisation behind it where asked, and the
// probability-weighted sum of a token's rows (include/moe_mxfp4.h).
//
// A work item is (expert, 128-channel block, tile of up to NT rows).  The weight channels
// are the MMA's 128 rows (operand A), the token rows its N columns (operand B), so the
// ragged side is the one whose size the instruction takes in steps of 16: an expert of cnt
// rows is cut into ceil(cnt / NT) tiles of equal size rounded up to 16.  One persistent CTA
// per SM; items are dealt out expert-major, channel blocks innermost, so that CTAs working
// at the same time share an expert's rows and its weights through L2.
//
// Roles: warp 0 loads, per 256-deep stage, one 17408-byte copy of a weight block with its
// scales and the rows' words of the two scale planes; warp 2 loads the rows' codes, in tensor
// copies of 128, 64 and 32 rows; warp 1 issues the MMAs; warps 4-7 move the stage's scales from
// shared into tensor memory; warps 8-15 are two epilogue groups, each owning one of the two
// accumulators.  A copy instruction holds its thread 65-90 cycles, a stage's MMAs take 600 at
// 208 rows: few copies, from two threads.  (Product of 49152 rows, N = 2816, D = 4096, 64
// experts: all copies from one warp in boxes of 32 rows 402 us; scale words read from global
// memory by the scale warps 1754 us.)
// Every wait is bounded:
// one that gives up records MOE_ERR_TIMEOUT and the CTA winds down.
#include "mx_tc.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWeightWarp = 0, kMmaWarp = 1, kTokenWarp = 2, kScaleWarp0 = 4, kEpiWarp0 = 8;
constexpr int kMaxExperts = 1024;
constexpr int kXchgBytes = 4 * 4 * 2 * 8 * 32 * 4 / 2;  // 4 warp pairs x 2 buffers x 2 directions of [8][32] fp32

template <int NT>
struct Cfg {
  // words of a scale plane: NT rows from a row rounded down to 4 (a 16-byte boundary)
  static constexpr int kPlaneWords = (NT + 31) / 32 * 32 + 4;
  static constexpr int kScales = kMxBlockBytes + NT * 128;  // of a stage: the planes' words
  static constexpr int kStageBytes = kScales + (2 * kPlaneWords * 4 + 1023) / 1024 * 1024;
  static constexpr int kStages = NT <= 32 ? 8 : 4;
  static constexpr int kSfbPlane = NT > 128 ? 8 : 4;     // columns per 128 elements of depth
  static constexpr int kSfCols = 8 + 2 * kSfbPlane;      // tensor-memory columns of a stage's scales
  // stages whose scales are in tensor memory at once: a stage's commit arrives ~500 cycles
  // after its last MMA is issued, and putting the next scales there takes ~250 more
  static constexpr int kSfStages = 4;
  static constexpr int kSf0 = 2 * NT;                    // accumulators in columns [0, 2 NT)
  static constexpr int kTmemCols = (kSf0 + kSfStages * kSfCols) <= 128 ? 128 : (kSf0 + kSfStages * kSfCols) <= 256 ? 256 : 512;
  static constexpr int kSmem = kStages * kStageBytes + kXchgBytes + 1024;
  static_assert(NT % 16 == 0 && kSf0 + kSfStages * kSfCols <= 512, "tensor memory");
  static_assert(kStageBytes % 1024 == 0 && kSmem + 10 * 1024 <= 227 * 1024, "shared memory");
};

struct GmmArgs {
  int R, E, N, D, KB, pitch;
  const uint32_t* scales;
  const int32_t* cumsum;
  const uint8_t* w;
  __half* c;
  uint8_t* h_codes;
  uint8_t* h_scales;
  int32_t* status;
};

// Tensor maps of the codes, 256 elements x 128, 64, 32 and 16 rows (a tile's rows, a multiple
// of 16, are copied as a sum of them), and of the scale words, 2 planes x kPlaneWords rows.
constexpr int kBoxes = 4;
struct Maps {
  CUtensorMap box[kBoxes], scales;
};

struct Item {
  int e, nb, row0, rows, n;  // n: MMA columns, rows rounded up to 16
};

struct WorkList {
  const int* pref;  // first item of each expert; pref[E] = their number
  const int* end;   // last row of each expert + 1
  int NB, E;
};

// Row tiles of an expert of cnt rows, and their size.  (t - 1) * size < cnt: none is empty.
template <int NT>
__device__ __forceinline__ int tiles_of(int cnt) { return (cnt + NT - 1) / NT; }

template <int NT>
__device__ __forceinline__ Item decode_item(int j, const WorkList& wl, int& e_hint) {
  int lo = e_hint, hi = wl.E;  // pref[lo] <= j < pref[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (wl.pref[mid] <= j) lo = mid; else hi = mid;
  }
  e_hint = lo;
  const int start = lo ? wl.end[lo - 1] : 0, cnt = wl.end[lo] - start;
  const int t = tiles_of<NT>(cnt), size = ((cnt + t - 1) / t + 15) & ~15;
  const int local = j - wl.pref[lo], rt = local / wl.NB;
  Item it;
  it.e = lo;
  it.nb = local - rt * wl.NB;
  it.row0 = start + rt * size;
  it.rows = min(size, cnt - rt * size);
  it.n = (it.rows + 15) & ~15;
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

template <int NT, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gmm_kernel(const __grid_constant__ Maps maps, const GmmArgs a) {
  using C = Cfg<NT>;
  constexpr int S = C::kStages, SF = C::kSfStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S], sf_bar[SF], accfull_bar[2], accempty_bar[2], final_bar;
  __shared__ int s_pref[kMaxExperts + 1], s_end[kMaxExperts], s_wsum[kThreads / 32];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_issued[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, NB = a.N / 128, KB = a.KB;
  volatile int* abort_flag = &s_abort;

  // ---- work list, barriers, tensor memory
  {
    const int per = (E + kThreads - 1) / kThreads;
    const int e0 = min(E, (int)threadIdx.x * per), e1 = min(E, e0 + per);
    int local = 0;
    for (int e = e0; e < e1; ++e) {
      const int hi = min(max(__ldg(a.cumsum + e), 0), a.R);
      const int lo = e ? min(max(__ldg(a.cumsum + e - 1), 0), a.R) : 0;
      s_end[e] = hi;
      local += tiles_of<NT>(max(hi - lo, 0)) * NB;
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
    if (warp == kMmaWarp) {
      tmem_alloc<C::kTmemCols>(&s_tmem);
      if (lane == 0) {
        for (int b = 0; b < kBoxes; ++b) prefetch_tmap(&maps.box[b]);
        prefetch_tmap(&maps.scales);
        for (int s = 0; s < S; ++s) {
          mbar_init(&full_bar[s], 2);
          mbar_init(&empty_bar[s], 1);
        }
        for (int s = 0; s < SF; ++s) mbar_init(&sf_bar[s], 4);
        for (int s = 0; s < 2; ++s) {
          mbar_init(&accfull_bar[s], 1);
          mbar_init(&accempty_bar[s], 4);
        }
        mbar_init(&final_bar, 1);
        fence_barrier_init();
      }
      tc_fence_before();
    }
    __syncthreads();
    int run = incl - local;
    for (int w = 0; w < warp; ++w) run += s_wsum[w];
    for (int e = e0; e < e1; ++e) {
      s_pref[e] = run;
      run += tiles_of<NT>(max(s_end[e] - (e ? s_end[e - 1] : 0), 0)) * NB;
    }
    if (e0 < E && e1 == E) s_pref[E] = run;
  }
  __syncthreads();
  tc_fence_after();
  WorkList wl;
  wl.pref = s_pref;
  wl.end = s_end;
  wl.NB = NB;
  wl.E = E;
  const int total = s_pref[E];
  const uint32_t tmem = s_tmem;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* ring_g = smem_raw + (ring - smem_u32(smem_raw));
  // a stage: weight codes at 0, their scales at 16384, token codes at 17408, their scales behind them
  const int planes = (a.D + 127) / 128;

  if (warp == kWeightWarp || warp == kTokenWarp) {
    if (lane == 0) {
      int n = 0, e_hint = 0;
      bool ok = true;
      for (int j = blockIdx.x; ok && j < total; j += gridDim.x) {
        const Item it = decode_item<NT>(j, wl, e_hint);
        const uint8_t* wb = a.w + ((size_t)it.e * NB + it.nb) * (size_t)KB * kMxBlockBytes;
        for (int kb = 0; kb < KB; ++kb, ++n) {
          const int slot = n % S;
          if (!(ok = wait_or_abort(&empty_bar[slot], ((n / S) & 1) ^ 1, abort_flag, a.status))) break;
          uint8_t* st = ring_g + slot * C::kStageBytes;
          uint64_t* bar = &full_bar[slot];
          if (warp == kWeightWarp) {
            mbar_arrive_expect_tx(bar, kMxBlockBytes + 2 * C::kPlaneWords * 4);
            bulk_load(st, wb + (size_t)kb * kMxBlockBytes, kMxBlockBytes, bar);
            tma_load_2d(st + C::kScales, &maps.scales, it.row0 & ~3, 2 * kb, bar);
          } else {
            mbar_arrive_expect_tx(bar, (uint32_t)it.n * 128);
            int r = 0;
#pragma unroll
            for (int b = 0; b < kBoxes; ++b) {
              const int rows = 128 >> b;
              for (; it.n - r >= rows; r += rows)
                tma_load_2d(st + kMxBlockBytes + r * 128, &maps.box[b], kb * 128, it.row0 + r, bar);
            }
          }
        }
      }
      s_issued[warp == kTokenWarp] = n;
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      int n = 0, e_hint = 0, u = 0;
      bool ok = true;
      for (int j = blockIdx.x; ok && j < total; j += gridDim.x, ++u) {
        const Item it = decode_item<NT>(j, wl, e_hint);
        const int buf = u & 1;
        if (!(ok = wait_or_abort(&accempty_bar[buf], ((u >> 1) & 1) ^ 1, abort_flag, a.status))) break;
        tc_fence_after();
        const uint32_t idesc = mx_idesc(it.n), d = tmem + buf * NT;
        for (int kb = 0; kb < KB; ++kb, ++n) {
          const int slot = n % S, sf = n % SF;
          // the scale warps arrive after they have seen the stage's copies complete
          if (!(ok = wait_or_abort(&sf_bar[sf], (n / SF) & 1, abort_flag, a.status))) break;
          tc_fence_after();
          const uint32_t st = ring + slot * C::kStageBytes, t_sf = tmem + C::kSf0 + sf * C::kSfCols;
          mx_mma_stage(d, st, st + kMxBlockBytes, idesc, t_sf, 4, t_sf + 8, C::kSfbPlane,
                       min(4, (a.D - kb * 256 + 63) >> 6), kb ? 1u : 0u);
          mx_commit(&empty_bar[slot]);
        }
        if (ok) mx_commit(&accfull_bar[buf]);
      }
      mx_commit(&final_bar);  // every MMA done before tensor memory is freed
      mbar_wait_sleep_bounded(&final_bar, 0);
    }
  } else if (warp >= kScaleWarp0 && warp < kScaleWarp0 + 4) {
    constexpr int J = (NT + 31) / 32;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 * (warp % 4) in the lane field
    const uint32_t last_mask = a.D % 128 ? (1u << (a.D % 128 / 4)) - 1u : 0xffffffffu;  // bytes past D are no scales
    int n = 0, e_hint = 0;
    bool ok = true;
    for (int j = blockIdx.x; ok && j < total; j += gridDim.x) {
      const Item it = decode_item<NT>(j, wl, e_hint);
      const int skew = it.row0 & 3;
      for (int kb = 0; kb < KB; ++kb, ++n) {
        const int slot = n % S, sf = n % SF;
        if (!(ok = warp_wait(&full_bar[slot], (n / S) & 1, abort_flag, a.status))) break;
        const uint8_t* st = ring_g + slot * C::kStageBytes;
        const uint32_t* ws = reinterpret_cast<const uint32_t*>(st + kMxCodeBytes) + lane;
        const uint32_t* xs = reinterpret_cast<const uint32_t*>(st + C::kScales) + skew + lane;
        uint32_t av[8], bv[2][C::kSfbPlane] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) av[i] = ws[32 * i];
        // words past the item's rows scale columns whose sums are never read
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < J; ++i) {
            bv[q][i] = xs[q * C::kPlaneWords + 32 * i];
            if (2 * kb + q == planes - 1) bv[q][i] &= last_mask;
          }
        // the scale columns are free once the MMAs of stage n - SF are done
        if (n >= SF) {
          const int m = n - SF;
          if (!(ok = warp_wait(&empty_bar[m % S], (m / S) & 1, abort_flag, a.status))) break;
          tc_fence_after();
        }
        const uint32_t t = tmem + lanes + C::kSf0 + sf * C::kSfCols;
        tmem_st8(t, av);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (C::kSfbPlane == 8) tmem_st8(t + 8 + q * C::kSfbPlane, bv[q]);
          else if (J == 1) tmem_st1(t + 8 + q * C::kSfbPlane, bv[q][0]);
          else tmem_st4(t + 8 + q * C::kSfbPlane, bv[q]);
        }
        tmem_wait_st();
        tc_fence_before();
        if (lane == 0) mbar_arrive(&sf_bar[sf]);
      }
    }
  } else if (warp >= kEpiWarp0) {
    const int group = (warp - kEpiWarp0) >> 2, quarter = warp & 3;
    const uint32_t lanes = (uint32_t)quarter << 21;
    int e_hint = 0;
    for (int u = group, j = blockIdx.x + group * gridDim.x; j < total; j += 2 * gridDim.x, u += 2) {
      const Item it = decode_item<NT>(j, wl, e_hint);
      bool ok = warp_wait(&accfull_bar[group], (u >> 1) & 1, abort_flag, a.status);
      if (SWIGLU) ok = group_all(1 + group, ok);  // the group's warps wait for one another below
      if (!ok) break;
      tc_fence_after();
      const uint32_t t = tmem + lanes + group * NT;
      if (!SWIGLU) {
        __half* out = a.c + (size_t)it.row0 * a.N + it.nb * 128 + quarter * 32 + lane;
        for (int c0 = 0; c0 < it.n; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(t + c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c0 + i < it.rows) out[(size_t)(c0 + i) * a.N] = from_f32<__half>(__uint_as_float(v[i]));
        }
      } else {
        // warps in pairs: the even one holds 32 gate channels, the odd one the up channels
        // that multiply them.  Of 16 rows each finishes 8, with the other's half through
        // shared memory (double-buffered: one pair barrier per 16 rows).
        const int pair = (warp - kEpiWarp0) >> 1, odd = warp & 1;
        float* x = reinterpret_cast<float*>(ring_g + S * C::kStageBytes) + pair * (2 * 2 * 256);
        const int k = it.nb * 2 + ((quarter >> 1) & 1), I = a.N / 2;  // scaled block of h
        for (int c0 = 0, p = 0; c0 < it.n; c0 += 16, p ^= 1) {
          uint32_t v[16];
          tmem_ld16(t + c0, v);
          tmem_wait_ld();
          float* give = x + p * 512 + odd * 256;
          const float* take = x + p * 512 + (odd ^ 1) * 256;
#pragma unroll
          for (int i = 0; i < 8; ++i) give[i * 32 + lane] = __uint_as_float(odd ? v[i] : v[8 + i]);
          asm volatile("bar.sync %0, 64;" ::"r"(3 + pair) : "memory");
          float h[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float o = take[i * 32 + lane];
            h[i] = odd ? mx_swiglu(o, __uint_as_float(v[8 + i])) : mx_swiglu(__uint_as_float(v[i]), o);
          }
          uint32_t byte;
          const uint32_t w = mx_quant_rows8(h, lane, byte);
          const int r = c0 + odd * 8 + (lane & 7);
          if (r < it.rows) {
            const size_t row = (size_t)it.row0 + r;
            *reinterpret_cast<uint32_t*>(a.h_codes + row * (I / 2) + k * 16 + (lane >> 3) * 4) = w;
            if (lane < 8) {
              uint8_t* sc = a.h_scales + ((size_t)(k >> 2) * a.pitch + row) * 4;
              sc[k & 3] = (uint8_t)byte;
              if (k == I / 32 - 1)
                for (int z = (k & 3) + 1; z < 4; ++z) sc[z] = 0;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&accempty_bar[group]);
    }
  }

  __syncthreads();
  if (threadIdx.x == 0) {  // copies still in flight (only after an abort) land before shared memory is released
    const int n0 = min(s_issued[0], s_issued[1]), n1 = max(s_issued[0], s_issued[1]);
    for (int n = n0; n < n1; ++n) mbar_arrive(&full_bar[n % S]);  // stages that one of the two loaders never began
    for (int n = max(0, n1 - S); n < n1; ++n) mbar_wait_bounded(&full_bar[n % S], (n / S) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<C::kTmemCols>(tmem);
  }
}

template <int NT, bool SWIGLU>
cudaError_t launch_gmm(const MxGemmProblem& p, cudaStream_t stream) {
  using C = Cfg<NT>;
  Maps maps;
  const uint64_t half = (uint64_t)p.D / 2, rows = (uint64_t)p.R;
  for (int b = 0; b < kBoxes; ++b)
    if (!encode_tensor_map_2d(&maps.box[b], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.codes, half, rows, 128, 128u >> b))
      return cudaErrorInvalidValue;
  if (!encode_tensor_map_words(&maps.scales, p.scales, (uint64_t)mx_scale_pitch(p.R), (uint64_t)mx_scale_planes(p.D),
                               C::kPlaneWords, 2))
    return cudaErrorInvalidValue;
  static PerContextOnce set;
  const int dev = current_device();
  if (set.needed(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(mx_gmm_kernel<NT, SWIGLU>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
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
  a.h_codes = p.h_codes;
  a.h_scales = reinterpret_cast<uint8_t*>(p.h_scales);
  a.status = p.status;
  mx_gmm_kernel<NT, SWIGLU><<<sm_count(), kThreads, C::kSmem, stream>>>(maps, a);
  return cudaGetLastError();
}

__global__ void mx_combine_kernel(const __half* c2, const int32_t* expanded, const float* probs, int K, int topK,
                                  __half* out) {
  const size_t t = blockIdx.x;
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    float acc = 0.0f;
    for (int j = 0; j < topK; ++j) {
      const int d = expanded[t * topK + j];
      if (d >= 0) acc = fmaf(probs[t * topK + j], __half2float(c2[(size_t)d * K + k]), acc);
    }
    out[t * K + k] = from_f32<__half>(acc);
  }
}

}  // namespace

cudaError_t launch_mx_gmm(const MxGemmProblem& p, cudaStream_t stream) {
  if ((double)p.R / p.E <= 32.0)
    return p.h_codes ? launch_gmm<32, true>(p, stream) : launch_gmm<32, false>(p, stream);
  return p.h_codes ? launch_gmm<208, true>(p, stream) : launch_gmm<208, false>(p, stream);
}

cudaError_t launch_mx_combine(const uint16_t* c2, const int32_t* expanded, const float* probs, int M, int K, int topK,
                              uint16_t* out, cudaStream_t stream) {
  mx_combine_kernel<<<M, 256, 0, stream>>>(reinterpret_cast<const __half*>(c2), expanded, probs, K, topK,
                                           reinterpret_cast<__half*>(out));
  return cudaGetLastError();
}

}  // namespace moe
