// MXFP4 quantisation of rows and weights, its inverse, and the packing of MXFP4 weights
// into blocks (include/moe_mxfp4.h).  One thread per scaled block of 32 elements.
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

inline int grid_of(size_t items) {
  const size_t b = (items + kThreads - 1) / kThreads;
  return (int)(b < ((size_t)1 << 30) ? b : ((size_t)1 << 30));
}

// The block of 32 at p: its code chunk and scale byte.
template <typename T>
__device__ __forceinline__ uint4 quant_block(const T* p, uint32_t& b) {
  float v[32];
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = to_f32<T>(p[i]);
    a = max(a, abs_bits(v[i]));
  }
  b = mx_scale_byte(a);
  const float mult = mx_multiplier(b);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = mx_scaled(v[8 * k + i], mult, b);
    w[k] = mx_codes8(s);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__global__ void quant_rows_kernel(int M, int D, const T* x, int64_t stride, const int32_t* row_map, int copies, int rows,
                                  uint8_t* codes, uint8_t* scales, int pitch) {
  const int nblk = (D + 127) / 128 * 4;  // blocks of a row, those past D included (scale 0)
  const size_t n = (size_t)M * nblk;
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (size_t)gridDim.x * kThreads) {
    const int t = (int)(i / nblk), k = (int)(i % nblk);
    uint32_t b = 0;
    uint4 c = make_uint4(0, 0, 0, 0);
    if (k * 32 < D) c = quant_block<T>(x + (int64_t)t * stride + k * 32, b);
    for (int j = 0; j < copies; ++j) {
      const int d = row_map ? row_map[(size_t)t * copies + j] : t;
      if (d < 0 || d >= rows) continue;
      if (k * 32 < D) *reinterpret_cast<uint4*>(codes + (size_t)d * (D / 2) + k * 16) = c;
      scales[((size_t)(k >> 2) * pitch + d) * 4 + (k & 3)] = (uint8_t)b;
    }
  }
}

template <typename T>
__global__ void dequant_rows_kernel(int rows, int D, const uint8_t* codes, const uint8_t* scales, int pitch, T* out) {
  const int nblk = D / 32;
  const size_t n = (size_t)rows * nblk;
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (size_t)gridDim.x * kThreads) {
    const size_t r = i / nblk;
    const int k = (int)(i % nblk);
    const float s = mx_scale_value(scales[((size_t)(k >> 2) * pitch + r) * 4 + (k & 3)]);
    const uint8_t* c = codes + r * (D / 2) + k * 16;
    T* o = out + r * D + k * 32;
    for (int j = 0; j < 16; ++j) {
      o[2 * j] = from_f32<T>(mx_value(c[j] & 15u) * s);
      o[2 * j + 1] = from_f32<T>(mx_value(c[j] >> 4) * s);
    }
  }
}

// Item i -> chunk c of row r of block `blk` (nb, kb of expert e), and its source row.
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

template <typename T>
__global__ void quant_weights_kernel(int N, int D, int KB, bool gate_up, size_t items, const T* w, uint8_t* blocks) {
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < items; i += (size_t)gridDim.x * kThreads) {
    const BlockItem it = block_item(i, N, KB, gate_up);
    uint32_t b = 0;
    uint4 c = make_uint4(0, 0, 0, 0);
    if (it.k * 32 < D) c = quant_block<T>(w + it.row * D + it.k * 32, b);
    uint8_t* blk = blocks + it.blk * kMxBlockBytes;
    *reinterpret_cast<uint4*>(blk + mx_chunk_at(it.r, it.c)) = c;
    blk[mx_scale_at(it.r, it.c)] = (uint8_t)b;
  }
}

__global__ void pack_weights_kernel(int N, int D, int KB, bool gate_up, size_t items, const uint8_t* codes,
                                    const uint8_t* scales, uint8_t* blocks) {
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < items; i += (size_t)gridDim.x * kThreads) {
    const BlockItem it = block_item(i, N, KB, gate_up);
    uint8_t b = 0;
    uint4 c = make_uint4(0, 0, 0, 0);
    if (it.k * 32 < D) {
      c = *reinterpret_cast<const uint4*>(codes + it.row * (D / 2) + it.k * 16);
      b = scales[it.row * (D / 32) + it.k];
    }
    uint8_t* blk = blocks + it.blk * kMxBlockBytes;
    *reinterpret_cast<uint4*>(blk + mx_chunk_at(it.r, it.c)) = c;
    blk[mx_scale_at(it.r, it.c)] = b;
  }
}

}  // namespace

cudaError_t launch_mx_quant(int M, int D, const void* x, int type, int64_t stride, const int32_t* row_map, int copies,
                            int rows, uint8_t* codes, uint32_t* scales, cudaStream_t stream) {
  const int grid = grid_of((size_t)M * mx_scale_planes(D) * 4), pitch = mx_scale_pitch(rows);
  uint8_t* sc = reinterpret_cast<uint8_t*>(scales);
  if (type == MOE_TYPE_F32)
    quant_rows_kernel<float><<<grid, kThreads, 0, stream>>>(M, D, static_cast<const float*>(x), stride, row_map, copies,
                                                            rows, codes, sc, pitch);
  else if (type == MOE_TYPE_F16)
    quant_rows_kernel<__half><<<grid, kThreads, 0, stream>>>(M, D, static_cast<const __half*>(x), stride, row_map,
                                                             copies, rows, codes, sc, pitch);
  else
    quant_rows_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(M, D, static_cast<const __nv_bfloat16*>(x), stride,
                                                                    row_map, copies, rows, codes, sc, pitch);
  return cudaGetLastError();
}

cudaError_t launch_mx_dequant(int rows, int D, const uint8_t* codes, const uint32_t* scales, void* out, int type,
                              cudaStream_t stream) {
  const int grid = grid_of((size_t)rows * (D / 32)), pitch = mx_scale_pitch(rows);
  const uint8_t* sc = reinterpret_cast<const uint8_t*>(scales);
  if (type == MOE_TYPE_F32)
    dequant_rows_kernel<float><<<grid, kThreads, 0, stream>>>(rows, D, codes, sc, pitch, static_cast<float*>(out));
  else if (type == MOE_TYPE_F16)
    dequant_rows_kernel<__half><<<grid, kThreads, 0, stream>>>(rows, D, codes, sc, pitch, static_cast<__half*>(out));
  else
    dequant_rows_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(rows, D, codes, sc, pitch,
                                                                      static_cast<__nv_bfloat16*>(out));
  return cudaGetLastError();
}

cudaError_t launch_mx_quant_weights(int E, int N, int D, bool gate_up, const void* w, int type, uint8_t* blocks,
                                    cudaStream_t stream) {
  const int KB = mx_depth_blocks(D);
  const size_t items = mx_weights_bytes(E, N, D) / kMxBlockBytes * 1024;
  const int grid = grid_of(items);
  if (type == MOE_TYPE_F32)
    quant_weights_kernel<float><<<grid, kThreads, 0, stream>>>(N, D, KB, gate_up, items, static_cast<const float*>(w),
                                                               blocks);
  else if (type == MOE_TYPE_F16)
    quant_weights_kernel<__half><<<grid, kThreads, 0, stream>>>(N, D, KB, gate_up, items,
                                                                static_cast<const __half*>(w), blocks);
  else
    quant_weights_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(N, D, KB, gate_up, items,
                                                                       static_cast<const __nv_bfloat16*>(w), blocks);
  return cudaGetLastError();
}

cudaError_t launch_mx_pack_weights(int E, int N, int D, bool gate_up, const uint8_t* codes, const uint8_t* scales,
                                   uint8_t* blocks, cudaStream_t stream) {
  const size_t items = mx_weights_bytes(E, N, D) / kMxBlockBytes * 1024;
  pack_weights_kernel<<<grid_of(items), kThreads, 0, stream>>>(N, D, mx_depth_blocks(D), gate_up, items, codes, scales,
                                                               blocks);
  return cudaGetLastError();
}

}  // namespace moe
