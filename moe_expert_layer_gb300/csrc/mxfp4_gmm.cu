// Grouped MXFP4 product over expert-major rows, with SwiGLU and requantisation behind it
// where asked, and the probability-weighted sum of a token's rows (include/moe_mxfp4.h).
// One CTA per (128-channel block, tile of rows of one expert), one thread per channel.
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int kRows = 8;  // rows per tile

struct GmmArgs {
  int R, E, N, D, KB, pitch, h_pitch;
  const uint8_t* codes;
  const uint32_t* scales;
  const int32_t* cumsum;
  const uint8_t* w;
  __half* c;
  uint8_t* h_codes;
  uint8_t* h_scales;
};

__device__ __forceinline__ int bound_row(const int32_t* cumsum, int e, int R) {
  return e < 0 ? 0 : min(max(__ldg(cumsum + e), 0), R);
}

__global__ void mx_gmm_kernel(const GmmArgs a) {
  const int e = blockIdx.y, nb = blockIdx.x, r = threadIdx.x;
  const int lo = bound_row(a.cumsum, e - 1, a.R), hi = bound_row(a.cumsum, e, a.R);
  const uint8_t* blocks = a.w + ((size_t)e * (a.N / 128) + nb) * (size_t)a.KB * kMxBlockBytes;
  __shared__ float s_x[kRows][32];
  __shared__ float s_y[kRows][128];
  for (int row0 = lo; row0 < hi; row0 += kRows) {
    float acc[kRows] = {};
    for (int k = 0; k < a.D / 32; ++k) {
      __syncthreads();
      for (int i = threadIdx.x; i < kRows * 32; i += 128) {
        const int row = row0 + i / 32, el = i % 32;
        float v = 0.0f;
        if (row < hi) {
          const uint32_t byte = a.codes[(size_t)row * (a.D / 2) + k * 16 + el / 2];
          const uint32_t sw = a.scales[(size_t)(k >> 2) * a.pitch + row];
          v = mx_value((el & 1) ? byte >> 4 : byte & 15u) * mx_scale_value((sw >> (8 * (k & 3))) & 255u);
        }
        s_x[i / 32][el] = v;
      }
      __syncthreads();
      const uint8_t* blk = blocks + (size_t)(k >> 3) * kMxBlockBytes;
      const uint4 c4 = *reinterpret_cast<const uint4*>(blk + mx_chunk_at(r, k & 7));
      const float s = mx_scale_value(blk[mx_scale_at(r, k & 7)]);
      const uint32_t cw[4] = {c4.x, c4.y, c4.z, c4.w};
      float part[kRows] = {};
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float w = mx_value((cw[i / 8] >> (4 * (i % 8))) & 15u);
#pragma unroll
        for (int m = 0; m < kRows; ++m) part[m] = fmaf(w, s_x[m][i], part[m]);
      }
#pragma unroll
      for (int m = 0; m < kRows; ++m) acc[m] = fmaf(part[m], s, acc[m]);
    }
    const int rows = min(kRows, hi - row0);
    if (!a.h_codes) {
      for (int m = 0; m < rows; ++m) a.c[(size_t)(row0 + m) * a.N + nb * 128 + r] = from_f32<__half>(acc[m]);
      continue;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kRows; ++m) s_y[m][r] = acc[m];
    __syncthreads();
    // one thread per (row, scaled block of 32 h): gate channels 64 q .. +31, up 64 q + 32 ..
    const int m = r >> 1, q = r & 1;
    if (r < 2 * kRows && m < rows) {
      float h[32];
      uint32_t amax = 0;
      for (int i = 0; i < 32; ++i) {
        const float g = s_y[m][64 * q + i], u = s_y[m][64 * q + 32 + i];
        h[i] = g / (1.0f + expf(-g)) * u;
        amax = max(amax, abs_bits(h[i]));
      }
      const uint32_t b = mx_scale_byte(amax);
      const float mult = mx_multiplier(b);
      const int I = a.N / 2, row = row0 + m, k = nb * 2 + q;
      uint32_t* out = reinterpret_cast<uint32_t*>(a.h_codes + (size_t)row * (I / 2) + k * 16);
      for (int j = 0; j < 4; ++j) {
        float v[8];
        for (int i = 0; i < 8; ++i) v[i] = mx_scaled(h[8 * j + i], mult, b);
        out[j] = mx_codes8(v);
      }
      a.h_scales[((size_t)(k >> 2) * a.h_pitch + row) * 4 + (k & 3)] = (uint8_t)b;
      if (k == I / 32 - 1)  // scale bytes past the row's end
        for (int j = (k & 3) + 1; j < 4; ++j) a.h_scales[((size_t)(k >> 2) * a.h_pitch + row) * 4 + j] = 0;
    }
  }
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
  GmmArgs a;
  a.R = p.R;
  a.E = p.E;
  a.N = p.N;
  a.D = p.D;
  a.KB = mx_depth_blocks(p.D);
  a.pitch = mx_scale_pitch(p.R);
  a.h_pitch = mx_scale_pitch(p.R);
  a.codes = p.codes;
  a.scales = p.scales;
  a.cumsum = p.cumsum;
  a.w = p.w;
  a.c = reinterpret_cast<__half*>(p.c);
  a.h_codes = p.h_codes;
  a.h_scales = reinterpret_cast<uint8_t*>(p.h_scales);
  mx_gmm_kernel<<<dim3(p.N / 128, p.E), 128, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_mx_combine(const uint16_t* c2, const int32_t* expanded, const float* probs, int M, int K, int topK,
                              uint16_t* out, cudaStream_t stream) {
  mx_combine_kernel<<<M, 256, 0, stream>>>(reinterpret_cast<const __half*>(c2), expanded, probs, K, topK,
                                           reinterpret_cast<__half*>(out));
  return cudaGetLastError();
}

}  // namespace moe
