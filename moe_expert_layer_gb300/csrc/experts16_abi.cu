// C entry points of the 16-bit experts (include/moe_experts16.h): host-side checks.
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/moe_experts16.h"
#include "abi_checks.h"
#include "experts16.h"

namespace {

using moe::all_aligned16;
using moe::check_device;
using moe::launch_status;

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int kMaxExperts = 1023;
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

bool type_ok(int32_t t) { return t == MOE_TYPE_F16 || t == MOE_TYPE_BF16; }
bool rows_ok(int64_t rows) { return rows >= 1 && rows < kMaxRows; }
bool experts_ok(int32_t E) { return E >= 1 && E <= kMaxExperts; }
bool size_ok(int32_t n, int32_t most) { return n >= 8 && n <= most && n % 8 == 0; }
bool gmm_ok(int32_t R, int32_t E, int32_t N, int32_t D) {
  return rows_ok(R) && experts_ok(E) && size_ok(N, moe::kMax16Size) && size_ok(D, moe::kMax16Size);
}
bool swiglu_ok(int32_t R, int32_t E, int32_t I, int32_t type) {
  return rows_ok(R) && experts_ok(E) && size_ok(I, moe::kMax16Size / 2) && type_ok(type);
}
bool map_ok(int32_t M, int32_t D, int32_t copies, int32_t rows, int32_t type) {
  return rows_ok(M) && rows_ok(rows) && copies >= 1 && (int64_t)M * copies < kMaxRows && size_ok(D, moe::kMax16Size) &&
         type_ok(type);
}

size_t gmm_workspace_bytes() { return kAlign; }

int32_t run_gmm(moe::Gmm16Problem& p, const void* workspace, size_t bytes, void* stream) {
  if (!p.rows || !p.cumsum || !p.out || !workspace || (p.kind == moe::Gmm16::kWeight ? !p.rows2 : !p.w))
    return MOE_ERR_NULL;
  if (!all_aligned16({p.rows, p.rows2, p.w, p.cumsum, p.out}) || !aligned256(workspace)) return MOE_ERR_ALIGN;
  if (bytes < gmm_workspace_bytes()) return MOE_ERR_WORKSPACE;
  const int32_t rc = check_device();
  if (rc != MOE_OK) return rc;
  return launch_status(moe::launch_gmm16(p, static_cast<cudaStream_t>(stream)));
}

moe::Gmm16Problem problem(moe::Gmm16 kind, int32_t R, int32_t E, int32_t N, int32_t D, int32_t type,
                          const int32_t* cumsum, void* out, void* workspace) {
  moe::Gmm16Problem p{};
  p.kind = kind;
  p.R = R;
  p.E = E;
  p.N = N;
  p.D = D;
  p.bf16 = type == MOE_TYPE_BF16;
  p.cumsum = cumsum;
  p.out = out;
  p.status = static_cast<int32_t*>(workspace);
  return p;
}

}  // namespace

extern "C" {

size_t moe_gmm16_workspace_size(int32_t R, int32_t E, int32_t N, int32_t D) {
  return gmm_ok(R, E, N, D) ? gmm_workspace_bytes() : 0;
}

int32_t moe_gmm16(int32_t R, int32_t E, int32_t N, int32_t D, int32_t type, const void* a, const int32_t* cumsum,
                  const void* w, void* c, void* workspace, size_t workspace_bytes, void* stream) {
  if (!gmm_ok(R, E, N, D) || !type_ok(type)) return MOE_ERR_SHAPE;
  moe::Gmm16Problem p = problem(moe::Gmm16::kForward, R, E, N, D, type, cumsum, c, workspace);
  p.rows = a;
  p.w = w;
  return run_gmm(p, workspace, workspace_bytes, stream);
}

int32_t moe_gmm16_input_grad(int32_t R, int32_t E, int32_t N, int32_t D, int32_t type, const void* dc,
                             const int32_t* cumsum, const void* w, void* da, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (!gmm_ok(R, E, N, D) || !type_ok(type)) return MOE_ERR_SHAPE;
  moe::Gmm16Problem p = problem(moe::Gmm16::kInput, R, E, N, D, type, cumsum, da, workspace);
  p.rows = dc;
  p.w = w;
  return run_gmm(p, workspace, workspace_bytes, stream);
}

int32_t moe_gmm16_weight_grad(int32_t R, int32_t E, int32_t N, int32_t D, int32_t type, const void* dc, const void* a,
                              const int32_t* cumsum, void* dw, int32_t dw_type, int32_t accumulate, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!gmm_ok(R, E, N, D) || !type_ok(type) || (dw_type != type && dw_type != MOE_TYPE_F32) ||
      (accumulate && dw_type != MOE_TYPE_F32))
    return MOE_ERR_SHAPE;
  moe::Gmm16Problem p = problem(moe::Gmm16::kWeight, R, E, N, D, type, cumsum, dw, workspace);
  p.rows = dc;
  p.rows2 = a;
  p.out_f32 = dw_type == MOE_TYPE_F32;
  p.accumulate = accumulate != 0;
  return run_gmm(p, workspace, workspace_bytes, stream);
}

int32_t moe_swiglu16(int32_t R, int32_t E, int32_t I, int32_t type, const void* gu, const int32_t* cumsum, void* h,
                     void* stream) {
  if (!swiglu_ok(R, E, I, type)) return MOE_ERR_SHAPE;
  if (!gu || !cumsum || !h) return MOE_ERR_NULL;
  if (!all_aligned16({gu, cumsum, h})) return MOE_ERR_ALIGN;
  const int32_t rc = check_device();
  if (rc != MOE_OK) return rc;
  return launch_status(
      moe::launch_swiglu16(R, E, I, type == MOE_TYPE_BF16, gu, cumsum, h, static_cast<cudaStream_t>(stream)));
}

int32_t moe_swiglu16_grad(int32_t R, int32_t E, int32_t I, int32_t type, const void* dh, const void* gu,
                          const int32_t* cumsum, void* dgu, void* h, void* stream) {
  if (!swiglu_ok(R, E, I, type)) return MOE_ERR_SHAPE;
  if (!dh || !gu || !cumsum || !dgu) return MOE_ERR_NULL;
  if (!all_aligned16({dh, gu, cumsum, dgu, h})) return MOE_ERR_ALIGN;
  const int32_t rc = check_device();
  if (rc != MOE_OK) return rc;
  return launch_status(moe::launch_swiglu16_grad(R, E, I, type == MOE_TYPE_BF16, dh, gu, cumsum, dgu, h,
                                                 static_cast<cudaStream_t>(stream)));
}

int32_t moe_dispatch16(int32_t M, int32_t D, int32_t copies, int32_t rows, int32_t type, const void* x,
                       const int32_t* row_map, void* out, void* stream) {
  if (!map_ok(M, D, copies, rows, type)) return MOE_ERR_SHAPE;
  if (!x || !row_map || !out) return MOE_ERR_NULL;
  if (!all_aligned16({x, row_map, out})) return MOE_ERR_ALIGN;
  const int32_t rc = check_device();
  if (rc != MOE_OK) return rc;
  return launch_status(
      moe::launch_dispatch16(M, D, copies, rows, x, row_map, out, static_cast<cudaStream_t>(stream)));
}

int32_t moe_combine16(int32_t M, int32_t D, int32_t copies, int32_t rows, int32_t type, const void* y,
                      const int32_t* row_map, const float* probs, void* out, void* stream) {
  if (!map_ok(M, D, copies, rows, type)) return MOE_ERR_SHAPE;
  if (!y || !row_map || !out) return MOE_ERR_NULL;
  if (!all_aligned16({y, row_map, probs, out})) return MOE_ERR_ALIGN;
  const int32_t rc = check_device();
  if (rc != MOE_OK) return rc;
  return launch_status(moe::launch_combine16(M, D, copies, rows, type == MOE_TYPE_BF16, y, row_map, probs, out,
                                             static_cast<cudaStream_t>(stream)));
}

int32_t moe_combine16_grad(int32_t M, int32_t D, int32_t copies, int32_t rows, int32_t type, const void* dout,
                           const void* y, const int32_t* row_map, const float* probs, void* dy, float* dprobs,
                           void* stream) {
  if (!map_ok(M, D, copies, rows, type)) return MOE_ERR_SHAPE;
  if (!dout || !y || !row_map || !probs || !dy || !dprobs) return MOE_ERR_NULL;
  if (!all_aligned16({dout, y, row_map, probs, dy, dprobs})) return MOE_ERR_ALIGN;
  const int32_t rc = check_device();
  if (rc != MOE_OK) return rc;
  return launch_status(moe::launch_combine16_grad(M, D, copies, rows, type == MOE_TYPE_BF16, dout, y, row_map, probs,
                                                  dy, dprobs, static_cast<cudaStream_t>(stream)));
}

size_t moe_lora16_workspace_size(int32_t M, int32_t N, int32_t D, int32_t rank) {
  if (!rows_ok(M) || !size_ok(N, moe::kMax16Size) || !size_ok(D, moe::kMax16Size) || !size_ok(rank, moe::kMax16Rank))
    return 0;
  return (moe::lora16_workspace_bytes(M, rank) + kAlign - 1) & ~(kAlign - 1);
}

int32_t moe_lora16(int32_t M, int32_t N, int32_t D, int32_t rank, int32_t L, int32_t type, const void* x,
                   const int32_t* route, const int32_t* cumsum, const void* a, const void* b, const float* scales,
                   const void* base, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  const size_t bytes = moe_lora16_workspace_size(M, N, D, rank);
  if (!bytes || !experts_ok(L) || !type_ok(type)) return MOE_ERR_SHAPE;
  if (!x || !route || !cumsum || !a || !b || !base || !out || !workspace) return MOE_ERR_NULL;
  if (!all_aligned16({x, route, cumsum, a, b, scales, base, out}) || !aligned256(workspace)) return MOE_ERR_ALIGN;
  if (workspace_bytes < bytes) return MOE_ERR_WORKSPACE;
  const int32_t rc = check_device();
  if (rc != MOE_OK) return rc;
  moe::Lora16Problem p{};
  p.M = M;
  p.N = N;
  p.D = D;
  p.rank = rank;
  p.L = L;
  p.bf16 = type == MOE_TYPE_BF16;
  p.x = x;
  p.route = route;
  p.cumsum = cumsum;
  p.a = a;
  p.b = b;
  p.scales = scales;
  p.base = base;
  p.out = out;
  p.v = static_cast<float*>(workspace);
  return launch_status(moe::launch_lora16(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
