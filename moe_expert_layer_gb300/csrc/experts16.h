// Internal launch interface of the 16-bit experts' kernels (host side).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

constexpr int kMax16Size = 65536, kMax16Rank = 128;

// Products grouped by expert (gmm16.cu).  kForward: out [R][N] = rows [R][D] times w; kInput:
// out [R][D] = rows [R][N] times w; kWeight: out [E][N][D] = rows [R][N] by rows2 [R][D].
enum class Gmm16 { kForward, kInput, kWeight };
struct Gmm16Problem {
  Gmm16 kind;
  int R, E, N, D;
  bool bf16, out_f32, accumulate;
  const void* rows;
  const void* rows2;
  const void* w;
  const int32_t* cumsum;
  void* out;
  int32_t* status;
};
cudaError_t launch_gmm16(const Gmm16Problem& p, cudaStream_t stream);

// rows16.cu
cudaError_t launch_swiglu16(int R, int E, int I, bool bf16, const void* gu, const int32_t* cumsum, void* h,
                            cudaStream_t stream);
cudaError_t launch_swiglu16_grad(int R, int E, int I, bool bf16, const void* dh, const void* gu, const int32_t* cumsum,
                                 void* dgu, void* h, cudaStream_t stream);
cudaError_t launch_dispatch16(int M, int D, int copies, int rows, const void* x, const int32_t* row_map, void* out,
                              cudaStream_t stream);
cudaError_t launch_combine16(int M, int D, int copies, int rows, bool bf16, const void* y, const int32_t* row_map,
                             const float* probs, void* out, cudaStream_t stream);
cudaError_t launch_combine16_grad(int M, int D, int copies, int rows, bool bf16, const void* dout, const void* y,
                                  const int32_t* row_map, const float* probs, void* dy, float* dprobs,
                                  cudaStream_t stream);

// lora16.cu
struct Lora16Problem {
  int M, N, D, rank, L;
  bool bf16;
  const void* x;
  const int32_t* route;
  const int32_t* cumsum;
  const void* a;
  const void* b;
  const float* scales;
  const void* base;
  void* out;
  float* v;  // workspace
};
size_t lora16_workspace_bytes(int M, int rank);
cudaError_t launch_lora16(const Lora16Problem& p, cudaStream_t stream);

}  // namespace moe
