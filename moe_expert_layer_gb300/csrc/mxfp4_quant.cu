// MXFP4 quantisation of rows and weights, its inverse, and the packing of MXFP4 weights
// into blocks (include/moe_mxfp4.h).
//
// Bound by bytes: eight elements to a lane, so that a warp reads 512 bytes (16-bit types) and
// writes 128 bytes of codes of one row at a time, and a scaled block of 32 is four neighbouring
// lanes, whose maximum is two shuffles.  The four scale bytes of 128 elements are put together
// by shuffles too and written as one word.  A thread takes kItems such pieces at a time, a grid
// apart, and reads them all first: one read of 16 bytes to a thread keeps too few under way.
#include "mxfp4.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kItems = 4;

// Blocks for `items` threads' worth of work, at most a few for each the device can hold: the
// kernels go on in strides.
inline int grid_of(size_t items) {
  const size_t b = (items + kThreads - 1) / kThreads, most = (size_t)sm_count() * 8;
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
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.t[i] = p[i];
  }
}

// The codes of this lane's eight elements and the scale byte of the block of its four lanes
// (an aligned group of four lanes enters together).
template <typename T>
__device__ __forceinline__ uint32_t quant8(const Eight<T>& r, uint32_t& b) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(r.t[i]);
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, abs_bits(v[i]));
  const uint32_t group = 0xfu << (threadIdx.x & 28u);
  a = max(a, __shfl_xor_sync(group, a, 1));
  a = max(a, __shfl_xor_sync(group, a, 2));
  b = mx_scale_byte(a);
  const float mult = mx_multiplier(b);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = mx_scaled(v[i], mult, b);
  return mx_codes8(v);
}

// One thread per eight elements of a row of x, the row rounded up to 128 elements (16 lanes, so
// that a word of four scale bytes is made by lanes of one warp; zero bytes past D).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(int M, int D, const T* x, int64_t stride,
                                                              const int32_t* row_map, int copies, int rows,
                                                              uint8_t* codes, uint32_t* scales, int pitch) {
  Pieces at((D + 127) / 128 * 16);
  while (at.t < M) {
    Eight<T> r[kItems];
    int t[kItems], c[kItems];  // t: M or more past the end; D is a multiple of 32: groups of four agree
#pragma unroll
    for (int k = 0; k < kItems; ++k, at.next()) {
      t[k] = at.t;
      c[k] = at.c;
      if (t[k] < M && c[k] * 8 < D) load8<T, VEC>(x + (int64_t)t[k] * stride + c[k] * 8, r[k]);
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (t[k] >= M) break;  // the pieces after it too; 16 lanes agree
      uint32_t b = 0, w = 0;
      if (c[k] * 8 < D) w = quant8<T>(r[k], b);
      // bytes of lanes 0, 4, 8, 12 of the 16
      const uint32_t half = 0xffffu << (threadIdx.x & 16u);
      uint32_t word = b << (8 * ((c[k] >> 2) & 3));
      word |= __shfl_xor_sync(half, word, 4);
      word |= __shfl_xor_sync(half, word, 8);
      for (int j = 0; j < copies; ++j) {
        const int d = row_map ? __ldg(row_map + (int64_t)t[k] * copies + j) : t[k];
        if (d < 0 || d >= rows) continue;
        if (c[k] * 8 < D) *reinterpret_cast<uint32_t*>(codes + (size_t)d * (D / 2) + c[k] * 4) = w;
        if ((c[k] & 15) == 0) scales[(size_t)(c[k] >> 4) * pitch + d] = word;
      }
    }
  }
}

// One thread per eight elements.
template <typename T>
__global__ void __launch_bounds__(kThreads) dequant_rows_kernel(int rows, int D, const uint8_t* codes,
                                                                const uint32_t* scales, int pitch, T* out) {
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
        w[k] = __ldg(reinterpret_cast<const uint32_t*>(codes) + i[k]);
        sw[k] = __ldg(scales + (size_t)(c[k] >> 4) * pitch + t[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (t[k] >= rows) break;
      const float s = mx_scale_value((sw[k] >> (8 * ((c[k] >> 2) & 3))) & 255u);
      Eight<T> o;
#pragma unroll
      for (int q = 0; q < 8; ++q) o.t[q] = from_f32<T>(mx_value((w[k] >> (4 * q)) & 15u) * s);
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
  const size_t n = items * 4, step = (size_t)gridDim.x * kThreads;
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
    const BlockItem it = block_item(i >> 2, N, KB, gate_up);
    const int part = (int)i & 3;
    uint32_t b = 0, c = 0;
    if (it.k * 32 < D) {
      Eight<T> r;
      load8<T, true>(w + it.row * D + it.k * 32 + part * 8, r);
      c = quant8<T>(r, b);
    }
    uint8_t* blk = blocks + it.blk * kMxBlockBytes;
    *reinterpret_cast<uint32_t*>(blk + mx_chunk_at(it.r, it.c) + part * 4) = c;
    if (part == 0) blk[mx_scale_at(it.r, it.c)] = (uint8_t)b;
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
      c = __ldg(reinterpret_cast<const uint4*>(codes + it.row * (D / 2) + it.k * 16));
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
  const int grid = grid_of((size_t)M * mx_scale_planes(D) * 16), pitch = mx_scale_pitch(rows);
  const T* p = static_cast<const T*>(x);
  if (stride * sizeof(T) % 16 == 0)
    quant_rows_kernel<T, true><<<grid, kThreads, 0, stream>>>(M, D, p, stride, row_map, copies, rows, codes, scales,
                                                              pitch);
  else  // rows that do not start on 16 bytes
    quant_rows_kernel<T, false><<<grid, kThreads, 0, stream>>>(M, D, p, stride, row_map, copies, rows, codes, scales,
                                                               pitch);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dequant_rows(int rows, int D, const uint8_t* codes, const uint32_t* scales, void* out,
                         cudaStream_t stream) {
  dequant_rows_kernel<T><<<grid_of((size_t)rows * (D / 8)), kThreads, 0, stream>>>(
      rows, D, codes, scales, mx_scale_pitch(rows), static_cast<T*>(out));
  return cudaGetLastError();
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
