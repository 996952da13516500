// The three products of an expert layer on the CUDA cores: any of the storage
// types (fp32 math), any pitch and alignment.  It carries fp32 operands, whose
// products the tensor cores would round to TF32, and 16-bit ones that TMA
// cannot address (a base, pitch or stride that is no multiple of 16 bytes).
//
// 64 x 64 output tiles, 16-deep k steps through shared memory, a 4 x 4 block
// of sums per thread.  The tile list is read from the offsets on the device:
// a block walks the experts' tiles of its own index and stride, so nothing
// waits for the counts on the host.
#include <algorithm>

#include "common.cuh"
#include "expert.h"
#include "internal.h"

namespace muon {
namespace {

constexpr int kTB = 64;
constexpr int kTK = 16;

// Element (i, k) of an operand at p + i * si + k * sk.
struct Operand {
  const void* p;
  long long si, sk;
  int rows, depth;
};

__device__ void load_tile(const Operand& o, int dt, int i0, int k0, float (*s)[kTB + 4]) {
  // consecutive threads along the operand's contiguous direction
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = threadIdx.x + 256 * q;
    const int i = o.sk == 1 ? e >> 4 : e & 63, k = o.sk == 1 ? e & 15 : e >> 6;
    const bool in = i0 + i < o.rows && k0 + k < o.depth;
    s[k][i] = in ? load_any(o.p, (i0 + i) * o.si + (k0 + k) * o.sk, dt) : 0.f;
  }
}

__global__ void __launch_bounds__(256)
expert_simt_kernel(const ExpertDesc g) {
  __shared__ __align__(16) float As[kTK][kTB + 4];
  __shared__ __align__(16) float Bs[kTK][kTB + 4];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int es = dtype_size(g.dtype);
  long long next = blockIdx.x;  // this block's next tile, counted over all experts
  long long first = 0;          // tiles of the experts before e
  for (int e = 0; e < g.experts; ++e) {
    const long long lo = min(max((long long)g.offsets[e], 0LL), g.rows);
    const long long hi = min(max((long long)g.offsets[e + 1], lo), g.rows);
    const int count = (int)(hi - lo);
    const int M = g.kind == kWeightGrad ? g.outer : count;
    const int N = g.kind == kInputGrad || g.kind == kWeightGrad ? g.inner : g.outer;
    const int K = g.kind == kForward ? g.inner : g.kind == kInputGrad ? g.outer : count;
    const long long tn = (N + kTB - 1) / kTB, tiles = ((M + kTB - 1) / kTB) * tn;
    for (; next < first + tiles; next += gridDim.x) {
      const int i0 = (int)((next - first) / tn) * kTB, j0 = (int)((next - first) % tn) * kTB;
      const char* a = reinterpret_cast<const char*>(g.a) + lo * g.ld_a * es;
      const char* b = reinterpret_cast<const char*>(g.b) + (g.kind == kWeightGrad ? lo * g.ld_b : e * g.stride_b) * es;
      const Operand A = g.kind == kWeightGrad ? Operand{a, 1, g.ld_a, M, K} : Operand{a, g.ld_a, 1, M, K};
      const Operand B = g.kind == kForward ? Operand{b, g.ld_b, 1, N, K} : Operand{b, 1, g.ld_b, N, K};
      float acc[4][4] = {};
      for (int k0 = 0; k0 < K; k0 += kTK) {
        load_tile(A, g.dtype, i0, k0, As);
        load_tile(B, g.dtype, j0, k0, Bs);
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kTK; ++kk) {
          const float4 a4 = *reinterpret_cast<const float4*>(&As[kk][ty * 4]);
          const float4 b4 = *reinterpret_cast<const float4*>(&Bs[kk][tx * 4]);
          const float av[4] = {a4.x, a4.y, a4.z, a4.w};
          const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        __syncthreads();
      }
      const long long base = g.kind == kWeightGrad ? e * g.stride_d : lo * g.ld_d;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = i0 + ty * 4 + i, c = j0 + tx * 4 + j;
          if (r >= M || c >= N) continue;
          const long long at = base + r * g.ld_d + c;
          store_any(g.d, at, g.d_dtype, g.accumulate ? load_any(g.d, at, g.d_dtype) + acc[i][j] : acc[i][j]);
        }
    }
    first += tiles;
  }
}

}  // namespace

int expert_simt(const ExpertDesc& g, cudaStream_t s) {
  expert_simt_kernel<<<4 * num_sms(), 256, 0, s>>>(g);
  return (int)cudaGetLastError();
}

}  // namespace muon
