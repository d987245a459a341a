// Internal launch interface of the router and the MXFP4 kernels (host side).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

// Weight blocks (include/moe_mxfp4.h): 128 channels x 256 reduction steps.
constexpr int kMxCodeBytes = 128 * 128;
constexpr int kMxBlockBytes = kMxCodeBytes + 2 * 512;
constexpr int kMxMaxDepth = 16384, kMxMaxN = 65536, kMxMaxE = 1023;
inline int mx_depth_blocks(int D) { return (D + 255) / 256; }
inline size_t mx_weights_bytes(int E, int N, int D) {
  return (size_t)E * (size_t)(N / 128) * (size_t)mx_depth_blocks(D) * kMxBlockBytes;
}
// Words per plane of the scales of `rows` MXFP4 rows, and planes of depth D.
inline int mx_scale_pitch(int rows) { return (rows + 3) & ~3; }
inline int mx_scale_planes(int D) { return (D + 127) / 128; }

// route_topk.cu
cudaError_t launch_route_topk(int M, int E, int topK, const void* logits, int type, int64_t stride, const float* bias,
                              int score, bool renormalise, float scale, int32_t* expert_idx, float* probs,
                              cudaStream_t stream);

// mxfp4_quant.cu
cudaError_t launch_mx_quant(int M, int D, const void* x, int type, int64_t stride, const int32_t* row_map, int copies,
                            int rows, uint8_t* codes, uint32_t* scales, cudaStream_t stream);
cudaError_t launch_mx_dequant(int rows, int D, const uint8_t* codes, const uint32_t* scales, void* out, int type,
                              cudaStream_t stream);
cudaError_t launch_mx_quant_weights(int E, int N, int D, bool gate_up, const void* w, int type, uint8_t* blocks,
                                    cudaStream_t stream);
cudaError_t launch_mx_pack_weights(int E, int N, int D, bool gate_up, const uint8_t* codes, const uint8_t* scales,
                                   uint8_t* blocks, cudaStream_t stream);

// Grouped product over expert-major MXFP4 rows (mxfp4_gmm.cu).  h_codes null: c gets the sums
// rounded to binary16, or c32 the sums themselves; else N = 2 I channels in gate_up order, and
// the SwiGLU of the sums is written as MXFP4 rows of depth N / 2.
struct MxGemmProblem {
  int R, E, N, D;
  const uint8_t* codes;    // [R][D / 2]
  const uint32_t* scales;  // [planes(D)][pitch(R)]
  const int32_t* cumsum;   // [E]
  const uint8_t* w;        // blocks
  uint16_t* c;             // [R][N] or null
  float* c32;              // [R][N] or null
  uint8_t* h_codes;        // [R][N / 4] or null
  uint32_t* h_scales;      // [planes(N / 2)][pitch(R)]
  int32_t* status;
  bool clear_status;       // the call's first product
};
cudaError_t launch_mx_gmm(const MxGemmProblem& p, cudaStream_t stream);

// The layer for a few tokens in two kernels (mxfp4_few.cu).
constexpr int kMxFewTokens = 32, kMxFewRoutes = 256;
constexpr int kMxFewStages = 1 << 24;  // 256-deep stages of a product: times the SMs, its kernel's 32 bits hold them
inline bool mx_few(int M, int K, int I, int topK) {
  return M <= kMxFewTokens && M * topK <= kMxFewRoutes &&
         (int64_t)M * topK * (I / 64) * ((K + 255) / 256) <= kMxFewStages &&
         (int64_t)M * topK * (K / 128) * ((I + 255) / 256) <= kMxFewStages;
}
bool mx_few_resident();  // whether its second kernel's CTAs, which wait for one another, fit the device at once
struct MxFewProblem {
  int M, K, I, E, topK;
  const uint16_t* x;
  const int32_t* expert_idx;
  const float* probs;
  const uint8_t *w1, *w2;
  uint8_t* x_codes;    // [M][K / 2]
  uint8_t* x_scales;   // mx_few_scale_bytes(M, K)
  uint8_t* h_codes;    // [M * topK][I / 2]
  uint8_t* h_scales;   // mx_few_scale_bytes(M * topK, I)
  float* part;         // mx_few_part_bytes
  int32_t* counters;   // mx_few_counter_bytes
  uint16_t* out;
  int32_t* status;
};
size_t mx_few_part_bytes(int M, int topK);
size_t mx_few_scale_bytes(int rows, int D);
size_t mx_few_counter_bytes(int M, int K, int I, int topK);
// cudaErrorCooperativeLaunchTooLarge where the stream may use fewer SMs than the device has.
cudaError_t launch_mx_few(const MxFewProblem& p, cudaStream_t stream);
cudaError_t launch_mx_ticket_probe(int32_t* answers, cudaStream_t stream);

// out[t] = sum over j of probs[t][j] * c2[expanded[t * topK + j]] (entries < 0 skipped)
cudaError_t launch_mx_combine(const float* c2, const int32_t* expanded, const float* probs, int M, int K, int topK,
                              uint16_t* out, cudaStream_t stream);

}  // namespace moe
