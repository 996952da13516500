// The three products of an expert layer on the CUDA cores: any of the storage
// types (fp32 math), any pitch and alignment.  It carries fp32 operands, whose
// products the tensor cores would round to TF32, and 16-bit ones that TMA
// cannot address (a base, pitch or stride that is no multiple of 16 bytes).
//
// 64 x 64 output tiles, 32-deep k steps through shared memory (the next step's
// elements are loaded into registers while this one is multiplied: with few
// tiles the loads' latency is what counts), a 4 x 4 block of sums per thread.
// The tile list is read from the offsets on the device:
// a block walks the experts' tiles of its own index and stride, so nothing
// waits for the counts on the host.
#include <algorithm>

#include "common.cuh"
#include "expert.h"
#include "internal.h"

namespace muon {
namespace {

constexpr int kTB = 64;
constexpr int kTK = 32;
constexpr int kLoads = kTB * kTK / 256;  // elements of a tile per thread

// Element (i, k) of an operand at p + i * si + k * sk.
struct Operand {
  const void* p;
  long long si, sk;
  int rows, depth;
};

// This thread's elements of a tile: consecutive threads along the operand's
// contiguous direction.
__device__ __forceinline__ int tile_i(const Operand& o, int e) { return o.sk == 1 ? e / kTK : e % kTB; }
__device__ __forceinline__ int tile_k(const Operand& o, int e) { return o.sk == 1 ? e % kTK : e / kTB; }
__device__ __forceinline__ void fetch(const Operand& o, int dt, int i0, int k0, float (&r)[kLoads]) {
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    const int e = threadIdx.x + 256 * q;
    const int i = i0 + tile_i(o, e), k = k0 + tile_k(o, e);
    r[q] = i < o.rows && k < o.depth ? load_any(o.p, i * o.si + k * o.sk, dt) : 0.f;
  }
}
__device__ __forceinline__ void put(const Operand& o, const float (&r)[kLoads], float (*s)[kTB + 4]) {
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    const int e = threadIdx.x + 256 * q;
    s[tile_k(o, e)][tile_i(o, e)] = r[q];
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
      float ra[kLoads], rb[kLoads];
      fetch(A, g.dtype, i0, 0, ra);
      fetch(B, g.dtype, j0, 0, rb);
      for (int k0 = 0; k0 < K; k0 += kTK) {
        put(A, ra, As);
        put(B, rb, Bs);
        __syncthreads();
        if (k0 + kTK < K) {
          fetch(A, g.dtype, i0, k0 + kTK, ra);
          fetch(B, g.dtype, j0, k0 + kTK, rb);
        }
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
