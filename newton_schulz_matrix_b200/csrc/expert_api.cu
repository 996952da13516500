// C ABI of the expert-layer operators (include/muon.h): argument checks and
// dispatch.  The kernels are in expert_route.cu (sort, gather, combine),
// expert_tc.cu (products on the tensor cores) and expert_simt.cu (products on
// the CUDA cores).
#include <stdint.h>

#include "../../include/muon.h"
#include "common.cuh"
#include "expert.h"
#include "internal.h"
#include "profile.h"

using namespace muon;

namespace {

bool dtype_ok(int d) { return d == MUON_BF16 || d == MUON_FP16 || d == MUON_FP32; }

bool element_aligned(const void* p, int dtype) {
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)dtype_size(dtype) == 0;
}

// A matrix argument: present, aligned to its elements, rows that do not overlap.
bool matrix_ok(const void* p, long long ld, long long cols, int dtype) {
  return p != nullptr && element_aligned(p, dtype) && ld >= cols && ld <= (1LL << 40);
}

// Rows, columns and assignments of one call: kernels step through them with
// 32-bit indices that must not wrap on the last step.
constexpr long long kMaxRows = 1LL << 30;

// Sizes shared by the gather, the combine and its gradients.
int check_route(const int* slot, int tokens, int topk, int cols, long long rows, int dtype, const void* weights,
                int w_dtype) {
  if (tokens < 0 || topk <= 0 || cols <= 0 || cols > kMaxRows || rows < 0 || rows > kMaxRows) return MUON_ERR_INVALID;
  if ((long long)tokens * topk > kMaxRows) return MUON_ERR_INVALID;
  if (!dtype_ok(dtype) || (weights != nullptr && !dtype_ok(w_dtype))) return MUON_ERR_UNSUPPORTED;
  if (tokens == 0) return MUON_OK;
  if (slot == nullptr || !element_aligned(slot, MUON_FP32)) return MUON_ERR_INVALID;
  if (weights != nullptr && !element_aligned(weights, w_dtype)) return MUON_ERR_INVALID;
  return MUON_OK;
}

RouteArgs route(const int* slot, int tokens, int topk, int cols, long long rows, int dtype) {
  RouteArgs a{};
  a.slot = slot;
  a.tokens = tokens; a.topk = topk; a.cols = cols; a.rows = rows; a.dtype = dtype;
  return a;
}

int check_product(const int* offsets, int experts, long long rows, int inner, int outer, int dtype) {
  if (experts <= 0 || experts > kMaxExperts || rows < 0 || rows > kMaxRows || inner <= 0 || outer <= 0 ||
      inner > kMaxRows || outer > kMaxRows || (long long)experts * outer > (1LL << 34))
    return MUON_ERR_INVALID;
  if (!dtype_ok(dtype)) return MUON_ERR_UNSUPPORTED;
  if (offsets == nullptr || !element_aligned(offsets, MUON_FP32)) return MUON_ERR_INVALID;
  return MUON_OK;
}

int run_product(const ExpertDesc& g, void* ws, size_t ws_bytes, cudaStream_t s) {
  if (g.status != nullptr && (!element_aligned(g.status, MUON_FP32) || cudaMemsetAsync(g.status, 0, sizeof(int), s) != cudaSuccess))
    return MUON_ERR_INVALID;
  if (g.rows == 0 && (g.kind != kWeightGrad || g.accumulate)) return MUON_OK;
  const double flops = 2.0 * g.rows * g.inner * (double)g.outer;
  const double es = dtype_size(g.dtype);
  const double bytes = (double)g.rows * (g.inner + g.outer) * es +
                       (double)g.experts * g.inner * g.outer * (g.kind == kWeightGrad ? dtype_size(g.d_dtype) : es);
  const bool tc = g.rows > 0 && expert_tc_ok(g);
  const size_t pack = g.rows > 0 ? expert_pack_bytes(g) : 0;
  const bool packed = !tc && pack > 0 && ws != nullptr && ws_bytes >= pack;
  ProfScope ps(tc || packed ? kProfExpertProduct : kProfExpertSimt, flops, bytes, s);
  const int rc = tc ? expert_tc(g, s) : packed ? expert_tc_packed(g, ws, s) : expert_simt(g, s);
  return rc == 0 ? MUON_OK : MUON_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t muon_expert_sort_workspace_size(int tokens, int topk, int experts) {
  if (tokens < 0 || topk <= 0 || experts <= 0 || experts > kMaxExperts || (long long)tokens * topk > kMaxRows) return 0;
  return 256 + expert_sort_ws_bytes(tokens, topk, experts);
}

int muon_expert_sort(const void* ids, int id_bytes, long long ld_ids, int tokens, int topk, int experts, int* offsets,
                     int* slot, int* source, void* ws, size_t ws_bytes, void* stream) {
  if (tokens < 0 || topk <= 0 || experts <= 0 || experts > kMaxExperts || (long long)tokens * topk > kMaxRows)
    return MUON_ERR_INVALID;
  if (id_bytes != 4 && id_bytes != 8) return MUON_ERR_UNSUPPORTED;
  if (offsets == nullptr || !element_aligned(offsets, MUON_FP32)) return MUON_ERR_INVALID;
  if (tokens > 0 && (ids == nullptr || slot == nullptr || source == nullptr || ld_ids < topk || ld_ids > (1LL << 40) ||
                     reinterpret_cast<uintptr_t>(ids) % (uintptr_t)id_bytes != 0 || !element_aligned(slot, MUON_FP32) ||
                     !element_aligned(source, MUON_FP32)))
    return MUON_ERR_INVALID;
  const size_t need = expert_sort_ws_bytes(tokens, topk, experts);
  if (need > 0) {
    if (ws == nullptr || !element_aligned(ws, MUON_FP32)) return MUON_ERR_INVALID;
    if (ws_bytes < need) return MUON_ERR_WORKSPACE;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const SortArgs a{ids, id_bytes == 8, ld_ids, tokens, topk, experts, offsets, slot, source};
  ProfScope ps(kProfExpertSort, 0.0, (double)tokens * topk * (id_bytes + 8) + 4.0 * (experts + 1), s);
  return launch_expert_sort(a, reinterpret_cast<int*>(ws), s) == 0 ? MUON_OK : MUON_ERR_CUDA;
}

int muon_expert_gather(const void* x, long long ld_x, const int* slot, int tokens, int topk, int cols, int dtype,
                       void* xs, long long ld_xs, long long rows, void* stream) {
  const int rc = check_route(slot, tokens, topk, cols, rows, dtype, nullptr, 0);
  if (rc != MUON_OK) return rc;
  if (tokens == 0 || rows == 0) return MUON_OK;
  if (!matrix_ok(x, ld_x, cols, dtype) || !matrix_ok(xs, ld_xs, cols, dtype)) return MUON_ERR_INVALID;
  RouteArgs a = route(slot, tokens, topk, cols, rows, dtype);
  a.by_token = x; a.ld_token = ld_x;
  a.out_row = xs; a.ld_out_row = ld_xs;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(kProfExpertGather, 0.0, (double)tokens * (topk + 1) * cols * dtype_size(dtype), s);
  return launch_expert_gather(a, s) == 0 ? MUON_OK : MUON_ERR_CUDA;
}

int muon_expert_combine(const void* ys, long long ld_ys, long long rows, const int* slot, const void* weights,
                        int w_dtype, int tokens, int topk, int cols, int dtype, void* y, long long ld_y, void* stream) {
  const int rc = check_route(slot, tokens, topk, cols, rows, dtype, weights, w_dtype);
  if (rc != MUON_OK) return rc;
  if (tokens == 0) return MUON_OK;
  if ((rows > 0 && !matrix_ok(ys, ld_ys, cols, dtype)) || !matrix_ok(y, ld_y, cols, dtype)) return MUON_ERR_INVALID;
  RouteArgs a = route(slot, tokens, topk, cols, rows, dtype);
  a.weights = weights; a.w_dtype = w_dtype;
  a.by_row = ys; a.ld_row = ld_ys;
  a.out_token = y; a.ld_out_token = ld_y;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(kProfExpertCombine, 2.0 * tokens * topk * cols, (double)tokens * (topk + 1) * cols * dtype_size(dtype), s);
  return launch_expert_combine(a, s) == 0 ? MUON_OK : MUON_ERR_CUDA;
}

int muon_expert_combine_backward(const void* dy, long long ld_dy, const void* ys, long long ld_ys, long long rows,
                                 const int* slot, const void* weights, int w_dtype, int tokens, int topk, int cols,
                                 int dtype, void* dys, long long ld_dys, void* dweights, void* stream) {
  const int rc = check_route(slot, tokens, topk, cols, rows, dtype, weights, w_dtype);
  if (rc != MUON_OK) return rc;
  if (dweights != nullptr && !dtype_ok(w_dtype)) return MUON_ERR_UNSUPPORTED;
  if (tokens == 0) return MUON_OK;
  if (!matrix_ok(dy, ld_dy, cols, dtype)) return MUON_ERR_INVALID;
  if (rows > 0 && (!matrix_ok(dys, ld_dys, cols, dtype) || (dweights != nullptr && !matrix_ok(ys, ld_ys, cols, dtype))))
    return MUON_ERR_INVALID;
  if (dweights != nullptr && !element_aligned(dweights, w_dtype)) return MUON_ERR_INVALID;
  RouteArgs a = route(slot, tokens, topk, cols, rows, dtype);
  a.weights = weights; a.w_dtype = w_dtype;
  a.by_token = dy; a.ld_token = ld_dy;
  a.by_row = ys; a.ld_row = ld_ys;
  a.out_row = dys; a.ld_out_row = ld_dys;
  a.dweights = dweights;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(kProfExpertCombineBackward, 3.0 * tokens * topk * cols,
               (double)tokens * (topk * (dweights ? 2 : 1) + 1) * cols * dtype_size(dtype), s);
  return launch_expert_combine_backward(a, s) == 0 ? MUON_OK : MUON_ERR_CUDA;
}

size_t muon_expert_workspace_size(int kind, const void* a, long long ld_a, const void* b, long long ld_b,
                                  long long stride_b, int experts, long long rows, int inner, int outer, int dtype) {
  if (kind < MUON_EXPERT_PRODUCT || kind > MUON_EXPERT_WEIGHT_GRAD || experts <= 0 || experts > kMaxExperts || rows <= 0 ||
      rows > kMaxRows || inner <= 0 || outer <= 0 || inner > kMaxRows || outer > kMaxRows || !dtype_ok(dtype))
    return 0;
  const ExpertDesc g{kind, nullptr, experts, rows, inner, outer, dtype, a, ld_a, b, ld_b, stride_b, nullptr, 0, 0, dtype, 0,
                     nullptr};
  return expert_pack_bytes(g);
}

int muon_expert_product(const void* xs, long long ld_xs, const void* w, long long ld_w, long long stride_w,
                        const int* offsets, int experts, long long rows, int inner, int outer, int dtype, void* y,
                        long long ld_y, void* ws, size_t ws_bytes, int* status, void* stream) {
  const int rc = check_product(offsets, experts, rows, inner, outer, dtype);
  if (rc != MUON_OK) return rc;
  if (rows > 0 && (!matrix_ok(xs, ld_xs, inner, dtype) || !matrix_ok(w, ld_w, inner, dtype) ||
                   !matrix_ok(y, ld_y, outer, dtype) || stride_w < 0))
    return MUON_ERR_INVALID;
  ExpertDesc g{kForward, offsets, experts, rows, inner, outer, dtype, xs, ld_xs, w, ld_w, stride_w, y, ld_y, 0, dtype, 0, status};
  return run_product(g, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

int muon_expert_input_grad(const void* dys, long long ld_dys, const void* w, long long ld_w, long long stride_w,
                           const int* offsets, int experts, long long rows, int inner, int outer, int dtype, void* dxs,
                           long long ld_dxs, void* ws, size_t ws_bytes, int* status, void* stream) {
  const int rc = check_product(offsets, experts, rows, inner, outer, dtype);
  if (rc != MUON_OK) return rc;
  if (rows > 0 && (!matrix_ok(dys, ld_dys, outer, dtype) || !matrix_ok(w, ld_w, inner, dtype) ||
                   !matrix_ok(dxs, ld_dxs, inner, dtype) || stride_w < 0))
    return MUON_ERR_INVALID;
  ExpertDesc g{kInputGrad, offsets, experts, rows, inner, outer, dtype, dys, ld_dys, w, ld_w, stride_w, dxs, ld_dxs, 0,
               dtype, 0, status};
  return run_product(g, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

int muon_expert_weight_grad(const void* dys, long long ld_dys, const void* xs, long long ld_xs, const int* offsets,
                            int experts, long long rows, int inner, int outer, int dtype, void* dw, long long ld_dw,
                            long long stride_dw, int dw_dtype, int accumulate, void* ws, size_t ws_bytes, int* status,
                            void* stream) {
  const int rc = check_product(offsets, experts, rows, inner, outer, dtype);
  if (rc != MUON_OK) return rc;
  // the result's type: the operands' or fp32; sums over several calls are held in fp32
  if (dw_dtype != dtype && dw_dtype != MUON_FP32) return MUON_ERR_UNSUPPORTED;
  if (accumulate && dw_dtype != MUON_FP32) return MUON_ERR_UNSUPPORTED;
  if (!matrix_ok(dw, ld_dw, inner, dw_dtype) || stride_dw < 0 || (experts > 1 && stride_dw < inner)) return MUON_ERR_INVALID;
  if (rows > 0 && (!matrix_ok(dys, ld_dys, outer, dtype) || !matrix_ok(xs, ld_xs, inner, dtype))) return MUON_ERR_INVALID;
  ExpertDesc g{kWeightGrad, offsets, experts, rows, inner, outer, dtype, dys, ld_dys, xs, ld_xs, 0, dw, ld_dw, stride_dw,
               dw_dtype, accumulate ? 1 : 0, status};
  return run_product(g, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
