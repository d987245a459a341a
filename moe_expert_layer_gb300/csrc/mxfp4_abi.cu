// C entry points of the router and the MXFP4 operators (include/moe_mxfp4.h): host-side
// checks, workspace carving and the layer's launch sequence.
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/moe_mxfp4.h"
#include "abi_checks.h"
#include "kernels.h"
#include "mxfp4.h"

namespace {

using moe::aligned16;
using moe::all_aligned16;
using moe::check_device;
using moe::check_shape;
using moe::launch_status;

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = (int64_t)1 << 24;
inline size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

bool type_ok(int32_t t) { return t == MOE_TYPE_F32 || t == MOE_TYPE_F16 || t == MOE_TYPE_BF16; }
bool rows_ok(int64_t rows, int32_t D) {
  return rows >= 1 && rows < kMaxRows && D >= 32 && D <= moe::kMxMaxDepth && D % 32 == 0;
}
bool weights_ok(int32_t E, int32_t N, int32_t D) {
  return E >= 1 && E <= moe::kMxMaxE && N >= 128 && N <= moe::kMxMaxN && N % 128 == 0 && rows_ok(1, D);
}

size_t gmm_workspace_bytes() { return kAlign; }

// The layer's workspace.
struct Layout {
  // a few tokens: status, part, counters, the scale records, a_codes (x) and h_codes; and what the other path uses
  size_t status, sorted, expanded, tpe, cumsum, sort_ws, a_codes, a_scales, h_codes, h_scales, c2, part, counters, x_rec, h_rec, total;
};
Layout layout_of(const moe_dims_t* d) {
  const size_t M = d->M, K = d->K, I = d->I, E = d->E, R = M * d->topK;
  Layout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes);
    return at;
  };
  L.status = take(gmm_workspace_bytes());
  const bool few = moe::mx_few(d->M, d->K, d->I, d->topK);
  if (few) {
    L.part = take(moe::mx_few_part_bytes((int)M, d->topK));
    L.counters = take(moe::mx_few_counter_bytes((int)M, (int)K, (int)I, d->topK));
    L.x_rec = take(moe::mx_few_scale_bytes((int)M, (int)K));
    L.h_rec = take(moe::mx_few_scale_bytes((int)R, (int)I));
  }
  L.sorted = take(R * 4);
  L.expanded = take(R * 4);
  L.tpe = take(E * 4);
  L.cumsum = take(E * 4);
  L.sort_ws = take(moe::route_sort_workspace_bytes((int)R, (int)E));
  L.a_codes = take(R * (K / 2));
  L.a_scales = take(moe_mxfp4_scale_words((int64_t)R, (int32_t)K) * 4);
  L.h_codes = take(R * (I / 2));
  L.h_scales = take(moe_mxfp4_scale_words((int64_t)R, (int32_t)I) * 4);
  L.c2 = take(R * K * 4);
  L.total = off;
  return L;
}

template <typename P>
P* at(void* base, size_t off) {
  return reinterpret_cast<P*>(static_cast<uint8_t*>(base) + off);
}

int32_t run_layer(const moe_dims_t* d, const uint16_t* x, const int32_t* expert_idx, const float* probs,
                  const uint8_t* w1, const uint8_t* w2, uint16_t* out, void* ws, const Layout& L, cudaStream_t st) {
  const int M = d->M, K = d->K, I = d->I, E = d->E, topK = d->topK, R = M * topK;
  cudaError_t e;
  if (moe::mx_few(M, K, I, topK) && moe::mx_few_resident()) {
    moe::MxFewProblem p;
    p.M = M;
    p.K = K;
    p.I = I;
    p.E = E;
    p.topK = topK;
    p.x = x;
    p.expert_idx = expert_idx;
    p.probs = probs;
    p.w1 = w1;
    p.w2 = w2;
    p.x_codes = at<uint8_t>(ws, L.a_codes);
    p.x_scales = at<uint8_t>(ws, L.x_rec);
    p.h_codes = at<uint8_t>(ws, L.h_codes);
    p.h_scales = at<uint8_t>(ws, L.h_rec);
    p.part = at<float>(ws, L.part);
    p.counters = at<int32_t>(ws, L.counters);
    p.out = out;
    p.status = at<int32_t>(ws, L.status);
    e = moe::launch_mx_few(p, st);
    if (e != cudaErrorCooperativeLaunchTooLarge) return launch_status(e);
    cudaGetLastError();  // not an error of this call, which goes on with the other path
  }
  int32_t* expanded = at<int32_t>(ws, L.expanded);
  int32_t* cumsum = at<int32_t>(ws, L.cumsum);
  if ((e = moe::launch_route_sort(expert_idx, R, E, at<int32_t>(ws, L.sorted), expanded, at<int32_t>(ws, L.tpe), cumsum,
                                  at<void>(ws, L.sort_ws), st)) != cudaSuccess)
    return launch_status(e);
  if ((e = moe::launch_mx_quant(M, K, x, MOE_TYPE_F16, K, expanded, topK, R, at<uint8_t>(ws, L.a_codes),
                                at<uint32_t>(ws, L.a_scales), st)) != cudaSuccess)
    return launch_status(e);
  moe::MxGemmProblem g{};
  g.R = R;
  g.E = E;
  g.N = 2 * I;
  g.D = K;
  g.codes = at<uint8_t>(ws, L.a_codes);
  g.scales = at<uint32_t>(ws, L.a_scales);
  g.cumsum = cumsum;
  g.w = w1;
  g.h_codes = at<uint8_t>(ws, L.h_codes);
  g.h_scales = at<uint32_t>(ws, L.h_scales);
  g.status = at<int32_t>(ws, L.status);
  g.clear_status = true;
  if ((e = moe::launch_mx_gmm(g, st)) != cudaSuccess) return launch_status(e);
  g.codes = g.h_codes;
  g.scales = g.h_scales;
  g.N = K;
  g.D = I;
  g.w = w2;
  g.c32 = at<float>(ws, L.c2);
  g.h_codes = nullptr;
  g.h_scales = nullptr;
  g.clear_status = false;
  if ((e = moe::launch_mx_gmm(g, st)) != cudaSuccess) return launch_status(e);
  return launch_status(moe::launch_mx_combine(g.c32, expanded, probs, M, K, topK, out, st));
}

}  // namespace

extern "C" {

int32_t moe_route_topk(int32_t M, int32_t E, int32_t topK, const void* logits, int32_t type, int64_t stride,
                       const float* bias, int32_t score, int32_t renormalise, float scale, int32_t* expert_idx,
                       float* probs, void* stream) {
  if (M < 1 || topK < 1 || E < topK || E > moe::kMxMaxE || (int64_t)M * topK >= kMaxRows || stride < E ||
      !type_ok(type) || (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID))
    return MOE_ERR_SHAPE;
  if (!logits || !expert_idx || !probs) return MOE_ERR_NULL;
  if (!all_aligned16({logits, bias, expert_idx, probs})) return MOE_ERR_ALIGN;
  int32_t rc;
  if ((rc = check_device()) != MOE_OK) return rc;
  return launch_status(moe::launch_route_topk(M, E, topK, logits, type, stride, bias, score, renormalise != 0, scale,
                                              expert_idx, probs, static_cast<cudaStream_t>(stream)));
}

size_t moe_mxfp4_scale_words(int64_t rows, int32_t D) {
  if (!rows_ok(rows, D)) return 0;
  return (size_t)moe::mx_scale_planes(D) * (size_t)moe::mx_scale_pitch((int)rows);
}

int32_t moe_mxfp4_quant(int32_t M, int32_t D, const void* x, int32_t type, int64_t stride, const int32_t* row_map,
                        int32_t copies, int32_t rows, uint8_t* codes, uint32_t* scales, void* stream) {
  if (!rows_ok(M, D) || !rows_ok(rows, D) || stride < D || copies < 1 || !type_ok(type) ||
      (int64_t)M * copies >= kMaxRows || (!row_map && (copies != 1 || rows != M)))
    return MOE_ERR_SHAPE;
  if (!x || !codes || !scales) return MOE_ERR_NULL;
  if (!all_aligned16({x, row_map, codes, scales})) return MOE_ERR_ALIGN;
  int32_t rc;
  if ((rc = check_device()) != MOE_OK) return rc;
  return launch_status(moe::launch_mx_quant(M, D, x, type, stride, row_map, copies, rows, codes, scales,
                                            static_cast<cudaStream_t>(stream)));
}

int32_t moe_mxfp4_dequant(int32_t rows, int32_t D, const uint8_t* codes, const uint32_t* scales, void* out,
                          int32_t type, void* stream) {
  if (!rows_ok(rows, D) || !type_ok(type)) return MOE_ERR_SHAPE;
  if (!codes || !scales || !out) return MOE_ERR_NULL;
  if (!all_aligned16({codes, scales, out})) return MOE_ERR_ALIGN;
  int32_t rc;
  if ((rc = check_device()) != MOE_OK) return rc;
  return launch_status(
      moe::launch_mx_dequant(rows, D, codes, scales, out, type, static_cast<cudaStream_t>(stream)));
}

size_t moe_mxfp4_weights_bytes(int32_t E, int32_t N, int32_t D) {
  return weights_ok(E, N, D) ? moe::mx_weights_bytes(E, N, D) : 0;
}

int32_t moe_mxfp4_quant_weights(int32_t E, int32_t N, int32_t D, int32_t gate_up, const void* w, int32_t type,
                                uint8_t* blocks, void* stream) {
  if (!weights_ok(E, N, D) || !type_ok(type)) return MOE_ERR_SHAPE;
  if (!w || !blocks) return MOE_ERR_NULL;
  if (!all_aligned16({w, blocks})) return MOE_ERR_ALIGN;
  int32_t rc;
  if ((rc = check_device()) != MOE_OK) return rc;
  return launch_status(moe::launch_mx_quant_weights(E, N, D, gate_up != 0, w, type, blocks,
                                                    static_cast<cudaStream_t>(stream)));
}

int32_t moe_mxfp4_pack_weights(int32_t E, int32_t N, int32_t D, int32_t gate_up, const uint8_t* codes,
                               const uint8_t* scales, uint8_t* blocks, void* stream) {
  if (!weights_ok(E, N, D)) return MOE_ERR_SHAPE;
  if (!codes || !scales || !blocks) return MOE_ERR_NULL;
  if (!all_aligned16({codes, scales, blocks})) return MOE_ERR_ALIGN;
  int32_t rc;
  if ((rc = check_device()) != MOE_OK) return rc;
  return launch_status(moe::launch_mx_pack_weights(E, N, D, gate_up != 0, codes, scales, blocks,
                                                   static_cast<cudaStream_t>(stream)));
}

size_t moe_mxfp4_gmm_workspace_size(int32_t R, int32_t E, int32_t N, int32_t D) {
  return rows_ok(R, D) && weights_ok(E, N, D) ? gmm_workspace_bytes() : 0;
}

int32_t moe_mxfp4_gmm(int32_t R, int32_t E, int32_t N, int32_t D, const uint8_t* codes, const uint32_t* scales,
                      const int32_t* cumsum, const uint8_t* w, uint16_t* c, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (!rows_ok(R, D) || !weights_ok(E, N, D)) return MOE_ERR_SHAPE;
  if (!codes || !scales || !cumsum || !w || !c || !workspace) return MOE_ERR_NULL;
  if (!all_aligned16({codes, scales, cumsum, w, c}) || !aligned256(workspace)) return MOE_ERR_ALIGN;
  if (workspace_bytes < gmm_workspace_bytes()) return MOE_ERR_WORKSPACE;
  int32_t rc;
  if ((rc = check_device()) != MOE_OK) return rc;
  moe::MxGemmProblem p{};
  p.R = R;
  p.E = E;
  p.N = N;
  p.D = D;
  p.codes = codes;
  p.scales = scales;
  p.cumsum = cumsum;
  p.w = w;
  p.c = c;
  p.status = static_cast<int32_t*>(workspace);
  p.clear_status = true;
  return launch_status(moe::launch_mx_gmm(p, static_cast<cudaStream_t>(stream)));
}

int32_t moe_mxfp4_gmm_swiglu(int32_t R, int32_t E, int32_t I, int32_t D, const uint8_t* codes, const uint32_t* scales,
                             const int32_t* cumsum, const uint8_t* w, uint8_t* h_codes, uint32_t* h_scales,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (I < 64 || I > 8192 || I % 64 || !rows_ok(R, D) || !weights_ok(E, 2 * I, D)) return MOE_ERR_SHAPE;
  if (!codes || !scales || !cumsum || !w || !h_codes || !h_scales || !workspace) return MOE_ERR_NULL;
  if (!all_aligned16({codes, scales, cumsum, w, h_codes, h_scales}) || !aligned256(workspace)) return MOE_ERR_ALIGN;
  if (workspace_bytes < gmm_workspace_bytes()) return MOE_ERR_WORKSPACE;
  int32_t rc;
  if ((rc = check_device()) != MOE_OK) return rc;
  moe::MxGemmProblem p{};
  p.R = R;
  p.E = E;
  p.N = 2 * I;
  p.D = D;
  p.codes = codes;
  p.scales = scales;
  p.cumsum = cumsum;
  p.w = w;
  p.h_codes = h_codes;
  p.h_scales = h_scales;
  p.status = static_cast<int32_t*>(workspace);
  p.clear_status = true;
  return launch_status(moe::launch_mx_gmm(p, static_cast<cudaStream_t>(stream)));
}

size_t moe_mxfp4_layer_workspace_size(const moe_dims_t* d) {
  if (check_shape(d) != MOE_OK) return 0;
  // the few-token path asks for more than some larger batches do, and a workspace of d serves fewer tokens too
  moe_dims_t few = *d;
  if (few.M > moe::kMxFewTokens) few.M = moe::kMxFewTokens;
  while (few.M > 1 && !moe::mx_few(few.M, few.K, few.I, few.topK)) --few.M;
  const size_t own = layout_of(d).total, fewer = layout_of(&few).total;
  return own > fewer ? own : fewer;
}

int32_t moe_mxfp4_layer_fwd(const moe_dims_t* d, const uint16_t* x, const int32_t* expert_idx, const float* probs,
                            const uint8_t* w1, const uint8_t* w2, uint16_t* out, void* workspace,
                            size_t workspace_bytes, void* stream) {
  int32_t rc = check_shape(d);
  if (rc != MOE_OK) return rc;
  if (!x || !expert_idx || !probs || !w1 || !w2 || !out || !workspace) return MOE_ERR_NULL;
  if (!all_aligned16({x, expert_idx, probs, w1, w2, out}) || !aligned256(workspace)) return MOE_ERR_ALIGN;
  const Layout L = layout_of(d);
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  if ((rc = check_device()) != MOE_OK) return rc;
  return run_layer(d, x, expert_idx, probs, w1, w2, out, workspace, L, static_cast<cudaStream_t>(stream));
}

int32_t moe_selftest_mxfp4_tickets(int32_t* answers, void* stream) {
  if (!answers) return MOE_ERR_NULL;
  if (!aligned16(answers)) return MOE_ERR_ALIGN;
  int32_t rc;
  if ((rc = check_device()) != MOE_OK) return rc;
  return launch_status(moe::launch_mx_ticket_probe(answers, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
