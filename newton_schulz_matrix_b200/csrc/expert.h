// Internal launchers of the expert-layer operators (the C ABI around them is
// expert_api.cu).  All return 0 or a CUDA error code.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace muon {

// ---------------------------------------------------------------- routing (expert_route.cu)
constexpr int kMaxExperts = 1024;

struct SortArgs {
  const void* ids; int wide;   // int32, or int64 when wide
  long long ld;                // row pitch of ids
  int tokens, topk, experts;
  int* offsets; int* slot; int* source;
};
size_t expert_sort_ws_bytes(int tokens, int topk, int experts);
int launch_expert_sort(const SortArgs& a, int* ws, cudaStream_t s);

struct RouteArgs {
  const int* slot;             // tokens x topk: sorted row or negative
  int tokens, topk, cols;
  long long rows;              // rows of the sorted matrices; slots outside [0, rows) are skipped
  int dtype;
  const void* weights; int w_dtype;   // tokens x topk, or null for ones
  const void* by_token; long long ld_token;    // x or dy (read)
  const void* by_row; long long ld_row;        // ys (read)
  void* out_token; long long ld_out_token;     // y (written)
  void* out_row; long long ld_out_row;         // xs or dys (written)
  void* dweights;              // tokens x topk of w_dtype, or null
};
int launch_expert_gather(const RouteArgs& a, cudaStream_t s);
int launch_expert_combine(const RouteArgs& a, cudaStream_t s);
int launch_expert_combine_backward(const RouteArgs& a, cudaStream_t s);

// ---------------------------------------------------------------- products
// Which of the three products of an expert layer (W[e] is outer x inner):
//   kForward     Y[p] = W[e] X[p]           a = X, b = W, d = Y
//   kInputGrad   dX[p] = W[e]^T dY[p]       a = dY, b = W, d = dX
//   kWeightGrad  dW[e] = sum_p dY[p] X[p]^T a = dY, b = X, d = dW (+ dW if accumulate)
// for the rows p in [offsets[e], offsets[e+1]), clamped to [0, rows).
enum ExpertKind { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };
struct ExpertDesc {
  int kind;
  const int* offsets; int experts; long long rows;
  int inner, outer;
  int dtype;                   // of a and b, and of d except for kWeightGrad
  const void* a; long long ld_a;
  const void* b; long long ld_b, stride_b;   // stride_b: one expert's W (kForward, kInputGrad)
  void* d; long long ld_d, stride_d;         // stride_d: one expert's dW (kWeightGrad)
  int d_dtype; int accumulate;               // kWeightGrad only
  int* status;                 // device word for MUON_STATUS_TIMEOUT, or null
};
bool expert_tc_ok(const ExpertDesc& g);   // whether expert_tc takes it: 16-bit operands that TMA can address
int expert_tc(const ExpertDesc& g, cudaStream_t s);     // tensor cores (expert_tc.cu)
size_t expert_pack_bytes(const ExpertDesc& g);          // workspace with which expert_tc_packed takes it; 0: it does not
int expert_tc_packed(const ExpertDesc& g, void* ws, cudaStream_t s);   // after copying operands into aligned rows
int expert_simt(const ExpertDesc& g, cudaStream_t s);   // any type, alignment and pitch (expert_simt.cu)

}  // namespace muon
