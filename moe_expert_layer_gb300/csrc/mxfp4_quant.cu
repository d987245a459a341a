// MXFP4 quantisation of rows and weights, its inverse, and the packing of MXFP4 weights
// into blocks (include/moe_mxfp4.h).
//
// Bound by bytes: eight elements to a lane, so that a warp reads 512 bytes (16-bit types) and
// writes 128 bytes of codes of one row at a time, and a scaled block of 32 is four neighbouring
// lanes, whose maximum is two shuffles.  A thread takes kItems such pieces at a time, a grid
// apart, and reads them all first: one read of 16 bytes to a thread keeps too few under way.
// Instructions are not far behind: magnitudes of 16-bit types are compared two to an
// instruction, on their bits.
// 90112 x 4096 bfloat16: 168 us and, back, 155, for 934 MB each (0.82 and 0.89 of the measured
// copy rate); the integer pipe is 69% busy in the first.
#include "mxfp4.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kItems = 4;

// Blocks for `items` threads' worth of work, at most as many as the device can hold, `per_sm` to
// an SM: the kernels go on in strides.
inline int grid_of(size_t items, int per_sm = 8) {
  const size_t b = (items + kThreads - 1) / kThreads, most = (size_t)sm_count() * per_sm;
  return (int)(b < most ? b : most);
}

// The pieces of a thread: piece `c` of row `t`, `per` to a row, a grid apart, without a division
// after the first.
struct Pieces {
  int t, c, per, dt, dc;
  __device__ __forceinline__ Pieces(int per_) : per(per_) {
    const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
    t = (int)(first / per);
    c = (int)(first - (int64_t)t * per);
    dt = (int)(step / per);
    dc = (int)(step - (int64_t)dt * per);
  }
  __device__ __forceinline__ void next() {
    t += dt;
    c += dc;
    if (c >= per) {
      c -= per;
      ++t;
    }
  }
};

// Eight elements at p (VEC: p aligned to 16 bytes).
template <typename T>
union Eight {
  T t[8];
  uint4 u[sizeof(T) / 2];
};
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, Eight<T>& r) {
  if (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = __ldcg(reinterpret_cast<const uint4*>(p) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.t[i] = p[i];
  }
}

// abs_bits of the largest magnitude of eight elements and of the other three lanes' of an
// aligned group of four.  16-bit types order by their magnitude bits as fp32 does, infinities
// above finite values and NaN above infinities.
__device__ __forceinline__ uint32_t group_max(const Eight<float>& r) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, abs_bits(r.t[i]));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  return max(a, __shfl_xor_sync(0xffffffffu, a, 2));
}
__device__ __forceinline__ uint32_t group_max16(const uint4& u) {
  uint32_t a = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
  a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, 2));
  return max(a >> 16, a & 0xffffu);
}
__device__ __forceinline__ uint32_t group_max(const Eight<__half>& r) {
  return abs_bits(__half2float(__ushort_as_half((unsigned short)group_max16(r.u[0]))));
}
__device__ __forceinline__ uint32_t group_max(const Eight<__nv_bfloat16>& r) { return group_max16(r.u[0]) << 16; }

// The codes of this lane's eight elements and the scale byte of the block of its four lanes; a
// whole warp enters.
template <typename T>
__device__ __forceinline__ uint32_t quant8(const Eight<T>& r, uint32_t& b) {
  b = mx_scale_byte(group_max(r));
  const float mult = mx_multiplier(b);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(r.t[i]) * mult;
  const uint32_t w = mx_codes8(v);
  return b == 255u ? 0u : w;
}

// One thread per eight elements of a row of x, the row rounded up to 128 elements, whose last
// word of scale bytes is written whole (0 past D).  MAP: rows go where row_map says.
constexpr int kQuantBlocks = 6;  // to an SM: as many as fit together (8, in two waves, took 4% longer)
template <typename T, bool VEC, bool MAP>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(int M, int D, const T* x, int64_t stride,
                                                              const int32_t* row_map, int copies, int rows,
                                                              uint8_t* codes, uint8_t* scales, int pitch) {
  // a programmatic dependent of the kernel before, and the product's setup beside the last rows
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Pieces at((D + 127) / 128 * 16);
  while (__any_sync(0xffffffffu, at.t < M)) {
    Eight<T> r[kItems];
    int t[kItems], c[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k, at.next()) {
      t[k] = at.t;
      c[k] = at.c;
      if (t[k] < M && c[k] * 8 < D) {
        load8<T, VEC>(x + (int64_t)t[k] * stride + c[k] * 8, r[k]);
      } else {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r[k].u[i] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      uint32_t b;
      const uint32_t w = quant8<T>(r[k], b);
      const bool in = c[k] * 8 < D;
      auto put = [&](int d) {
        if (in) *reinterpret_cast<uint32_t*>(codes + (size_t)d * (D / 2) + c[k] * 4) = w;
        if ((c[k] & 3) == 0) scales[((size_t)(c[k] >> 4) * pitch + d) * 4 + ((c[k] >> 2) & 3)] = (uint8_t)b;
      };
      if (t[k] < M) {
        if (MAP) {
          const int32_t* to = row_map + (int64_t)t[k] * copies;
          for (int j = 0; j < copies; j += 4) {
            int d[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q] = j + q < copies ? to[j + q] : -1;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (d[q] >= 0 && d[q] < rows) put(d[q]);
          }
        } else {
          put(t[k]);
        }
      }
    }
  }
}

// The dispatch of many rows to several places each: one warp per row, which makes the row's codes
// and scale words in shared memory and sends them off whole, the codes by one bulk copy per
// place (from lane j to place j), the words a plane to a lane.  The kernel above computes every
// address and stores every word once per place: 8192 x 4096 binary16 rows to 6 places each 58 us,
// here 36 us; but a warp per row takes longer to get through a few long rows (one row of 7168,
// eight places: 9 us against 5).
constexpr int kRowWarps = 4;
template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kRowWarps) quant_dispatch_kernel(int M, int D, const T* x, int64_t stride,
                                                                        const int32_t* row_map, int copies, int rows,
                                                                        uint8_t* codes, uint32_t* scales, int pitch) {
  extern __shared__ __align__(128) uint8_t s_rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int planes = (D + 127) / 128, row_bytes = D / 2;  // a multiple of 16
  uint8_t* s_codes = s_rows + (size_t)warp * (row_bytes + planes * 4 + 15 & ~15);
  uint8_t* s_scales = s_codes + row_bytes;
  for (int t = blockIdx.x * kRowWarps + warp; t < M; t += gridDim.x * kRowWarps) {
    const T* row = x + (int64_t)t * stride;
    bulk_wait_read_all();  // the row before has left
    __syncwarp();
    for (int e0 = 0; e0 < planes * 128; e0 += 256 * kItems) {
      Eight<T> r[kItems];
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int e = e0 + 256 * k + lane * 8;
        if (e < D) {
          load8<T, VEC>(row + e, r[k]);
        } else {
#pragma unroll
          for (int i = 0; i < (int)sizeof(T) / 2; ++i) r[k].u[i] = make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int e = e0 + 256 * k + lane * 8;
        uint32_t b;
        const uint32_t w = quant8<T>(r[k], b);
        if (e < D) *reinterpret_cast<uint32_t*>(s_codes + e / 2) = w;
        if ((lane & 3) == 0 && e < planes * 128) s_scales[e / 32] = (uint8_t)b;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    const int32_t* to = row_map + (int64_t)t * copies;
    for (int j0 = 0; j0 < copies; j0 += 32) {
      int d = j0 + lane < copies ? to[j0 + lane] : -1;
      if (d >= rows) d = -1;
      if (d >= 0) bulk_store(codes + (size_t)d * row_bytes, s_codes, (uint32_t)row_bytes);
      for (int j = 0; j < min(32, copies - j0); ++j) {
        const int dj = __shfl_sync(0xffffffffu, d, j);
        if (dj < 0) continue;
        for (int q = lane; q < planes; q += 32)
          scales[(size_t)q * pitch + dj] = reinterpret_cast<const uint32_t*>(s_scales)[q];
      }
    }
    bulk_commit_group();
  }
  bulk_wait_all();
}

// One thread per eight elements.
constexpr int kDequantBlocks = 4;  // to an SM
template <typename T>
__global__ void __launch_bounds__(kThreads) dequant_rows_kernel(int rows, int D, const uint8_t* codes,
                                                                const uint32_t* scales, int pitch, T* out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Pieces at(D / 8);
  while (at.t < rows) {
    uint32_t w[kItems], sw[kItems];
    size_t i[kItems];
    int t[kItems], c[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k, at.next()) {
      t[k] = at.t;
      c[k] = at.c;
      i[k] = (size_t)t[k] * (D / 8) + c[k];
      if (t[k] < rows) {
        w[k] = __ldcg(reinterpret_cast<const uint32_t*>(codes) + i[k]);
        sw[k] = __ldcg(scales + (size_t)(c[k] >> 4) * pitch + t[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (t[k] >= rows) break;
      const float s = mx_scale_value((sw[k] >> (8 * ((c[k] >> 2) & 3))) & 255u);
      float v[8];
      mx_values8(w[k], v);
      Eight<T> o;
#pragma unroll
      for (int q = 0; q < 8; q += 2) from_f32x2<T>(v[q] * s, v[q + 1] * s, o.t + q);
#pragma unroll
      for (int q = 0; q < (int)sizeof(T) / 2; ++q) reinterpret_cast<uint4*>(out)[i[k] * (sizeof(T) / 2) + q] = o.u[q];
    }
  }
}

// Chunk c (32 elements) of row r of weight block `blk`, and its source row.
struct BlockItem {
  size_t blk, row;
  int r, c, k;  // k: scaled block along D
};
__device__ __forceinline__ BlockItem block_item(size_t i, int N, int KB, bool gate_up) {
  BlockItem it;
  it.blk = i >> 10;
  it.r = (int)(i >> 3) & 127;
  it.c = (int)i & 7;
  const int kb = (int)(it.blk % KB);
  const size_t eb = it.blk / KB;
  const int NB = N / 128;
  const int nb = (int)(eb % NB);
  it.row = (eb / NB) * N + mx_channel(nb, it.r, N, gate_up);
  it.k = kb * 8 + it.c;
  return it;
}

// Four threads to a chunk.
template <typename T>
__global__ void __launch_bounds__(kThreads) quant_weights_kernel(int N, int D, int KB, bool gate_up, size_t items,
                                                                 const T* w, uint8_t* blocks) {
  const size_t n = items * 4, step = (size_t)gridDim.x * kThreads;  // n: a multiple of 4096
  for (size_t i0 = (size_t)blockIdx.x * kThreads + threadIdx.x; i0 < n; i0 += kItems * step) {
    Eight<T> r[kItems];
    BlockItem it[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const size_t i = i0 + k * step;
      if (i >= n) break;
      it[k] = block_item(i >> 2, N, KB, gate_up);
      if (it[k].k * 32 < D) {
        load8<T, true>(w + it[k].row * D + it[k].k * 32 + (i & 3) * 8, r[k]);
      } else {
#pragma unroll
        for (int q = 0; q < (int)sizeof(T) / 2; ++q) r[k].u[q] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const size_t i = i0 + k * step;
      if (i >= n) break;
      uint32_t b;
      const uint32_t c = quant8<T>(r[k], b);
      uint8_t* blk = blocks + it[k].blk * kMxBlockBytes;
      *reinterpret_cast<uint32_t*>(blk + mx_chunk_at(it[k].r, it[k].c) + (i & 3) * 4) = c;
      if ((i & 3) == 0) blk[mx_scale_at(it[k].r, it[k].c)] = (uint8_t)b;
    }
  }
}

__global__ void __launch_bounds__(kThreads) pack_weights_kernel(int N, int D, int KB, bool gate_up, size_t items,
                                                                const uint8_t* codes, const uint8_t* scales,
                                                                uint8_t* blocks) {
  const size_t step = (size_t)gridDim.x * kThreads;
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < items; i += step) {
    const BlockItem it = block_item(i, N, KB, gate_up);
    uint8_t b = 0;
    uint4 c = make_uint4(0, 0, 0, 0);
    if (it.k * 32 < D) {
      c = __ldcg(reinterpret_cast<const uint4*>(codes + it.row * (D / 2) + it.k * 16));
      b = scales[it.row * (D / 32) + it.k];
    }
    uint8_t* blk = blocks + it.blk * kMxBlockBytes;
    *reinterpret_cast<uint4*>(blk + mx_chunk_at(it.r, it.c)) = c;
    blk[mx_scale_at(it.r, it.c)] = b;
  }
}

template <typename T>
cudaError_t quant_rows(int M, int D, const void* x, int64_t stride, const int32_t* row_map, int copies, int rows,
                       uint8_t* codes, uint32_t* scales, cudaStream_t stream) {
  const int grid = grid_of((size_t)M * mx_scale_planes(D) * 16, kQuantBlocks), pitch = mx_scale_pitch(rows);
  const T* p = static_cast<const T*>(x);
  uint8_t* sc = reinterpret_cast<uint8_t*>(scales);
  const bool vec = stride * sizeof(T) % 16 == 0;  // else rows that do not start on 16 bytes
  // a warp per row from about as many rows on as it takes to gain (1024 rows of 7168 to 8 places: 15 us, above 17; 64: 11 and 7)
  if (row_map && M >= sm_count() * 8) {
    const size_t smem = (size_t)kRowWarps * ((D / 2 + mx_scale_planes(D) * 4 + 15) & ~15);  // at most 34 KB
    const int blocks = (M + kRowWarps - 1) / kRowWarps;
    if (vec)
      quant_dispatch_kernel<T, true><<<blocks, 32 * kRowWarps, smem, stream>>>(M, D, p, stride, row_map, copies, rows, codes, scales, pitch);
    else
      quant_dispatch_kernel<T, false><<<blocks, 32 * kRowWarps, smem, stream>>>(M, D, p, stride, row_map, copies, rows, codes, scales, pitch);
    return cudaGetLastError();
  }
  auto* kernel = vec ? (row_map ? quant_rows_kernel<T, true, true> : quant_rows_kernel<T, true, false>)
                     : (row_map ? quant_rows_kernel<T, false, true> : quant_rows_kernel<T, false, false>);
  return launch_dependent(kernel, (unsigned)grid, kThreads, 0, stream, M, D, p, stride, row_map, copies, rows, codes, sc, pitch);
}

template <typename T>
cudaError_t dequant_rows(int rows, int D, const uint8_t* codes, const uint32_t* scales, void* out,
                         cudaStream_t stream) {
  return launch_dependent(dequant_rows_kernel<T>, (unsigned)grid_of((size_t)rows * (D / 8), kDequantBlocks), kThreads, 0, stream,
                          rows, D, codes, scales, mx_scale_pitch(rows), static_cast<T*>(out));
}

template <typename T>
cudaError_t quant_weights(int E, int N, int D, bool gate_up, const void* w, uint8_t* blocks, cudaStream_t stream) {
  const size_t items = mx_weights_bytes(E, N, D) / kMxBlockBytes * 1024;
  quant_weights_kernel<T><<<grid_of(items * 4), kThreads, 0, stream>>>(N, D, mx_depth_blocks(D), gate_up, items,
                                                                       static_cast<const T*>(w), blocks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_quant(int M, int D, const void* x, int type, int64_t stride, const int32_t* row_map, int copies,
                            int rows, uint8_t* codes, uint32_t* scales, cudaStream_t stream) {
  switch (type) {
    case MOE_TYPE_F32: return quant_rows<float>(M, D, x, stride, row_map, copies, rows, codes, scales, stream);
    case MOE_TYPE_F16: return quant_rows<__half>(M, D, x, stride, row_map, copies, rows, codes, scales, stream);
    default: return quant_rows<__nv_bfloat16>(M, D, x, stride, row_map, copies, rows, codes, scales, stream);
  }
}

cudaError_t launch_mx_dequant(int rows, int D, const uint8_t* codes, const uint32_t* scales, void* out, int type,
                              cudaStream_t stream) {
  switch (type) {
    case MOE_TYPE_F32: return dequant_rows<float>(rows, D, codes, scales, out, stream);
    case MOE_TYPE_F16: return dequant_rows<__half>(rows, D, codes, scales, out, stream);
    default: return dequant_rows<__nv_bfloat16>(rows, D, codes, scales, out, stream);
  }
}

cudaError_t launch_mx_quant_weights(int E, int N, int D, bool gate_up, const void* w, int type, uint8_t* blocks,
                                    cudaStream_t stream) {
  switch (type) {
    case MOE_TYPE_F32: return quant_weights<float>(E, N, D, gate_up, w, blocks, stream);
    case MOE_TYPE_F16: return quant_weights<__half>(E, N, D, gate_up, w, blocks, stream);
    default: return quant_weights<__nv_bfloat16>(E, N, D, gate_up, w, blocks, stream);
  }
}

cudaError_t launch_mx_pack_weights(int E, int N, int D, bool gate_up, const uint8_t* codes, const uint8_t* scales,
                                   uint8_t* blocks, cudaStream_t stream) {
  const size_t items = mx_weights_bytes(E, N, D) / kMxBlockBytes * 1024;
  pack_weights_kernel<<<grid_of(items), kThreads, 0, stream>>>(N, D, mx_depth_blocks(D), gate_up, items, codes, scales,
                                                               blocks);
  return cudaGetLastError();
}

}  // namespace moe
