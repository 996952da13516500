// The three products of an expert layer on the CUDA cores: any of the storage
// types (fp32 math), any pitch and alignment.  It carries fp32 operands, whose
// products the tensor cores would round to TF32, and 16-bit ones that TMA
// cannot address (a base, pitch or stride that is no multiple of 16 bytes).
//
// 64 x 64 output tiles with a 4 x 4 block of sums per thread, or 32 x 32 with
// 2 x 2 where the larger ones cannot occupy the SMs; 32-deep k steps through
// shared memory (the next step's elements are loaded into registers while this
// one is multiplied: with few tiles the loads' latency is what counts).  The
// three products of 301 rows over 7 experts, 333 to 130 wide: 135 us with
// 16-deep steps and one load at a time, 73 with 64 x 64 tiles as here, 39 with
// 32 x 32.  The tile list is read from the offsets on the device:
// a block walks the experts' tiles of its own index and stride, so nothing
// waits for the counts on the host.
#include <algorithm>

#include "common.cuh"
#include "expert.h"
#include "internal.h"

namespace muon {
namespace {

constexpr int kTK = 32;

// Element (i, k) of an operand at p + i * si + k * sk.
struct Operand {
  const void* p;
  long long si, sk;
  int rows, depth;
};

// This thread's elements of a tile: consecutive threads along the operand's
// contiguous direction.
template <int TB>
__device__ __forceinline__ int tile_i(const Operand& o, int e) { return o.sk == 1 ? e / kTK : e % TB; }
template <int TB>
__device__ __forceinline__ int tile_k(const Operand& o, int e) { return o.sk == 1 ? e % kTK : e / TB; }
template <int TB>
__device__ __forceinline__ void fetch(const Operand& o, int dt, int i0, int k0, float (&r)[TB * kTK / 256]) {
#pragma unroll
  for (int q = 0; q < TB * kTK / 256; ++q) {
    const int e = threadIdx.x + 256 * q;
    const int i = i0 + tile_i<TB>(o, e), k = k0 + tile_k<TB>(o, e);
    r[q] = i < o.rows && k < o.depth ? load_any(o.p, i * o.si + k * o.sk, dt) : 0.f;
  }
}
template <int TB>
__device__ __forceinline__ void put(const Operand& o, const float (&r)[TB * kTK / 256], float (*s)[TB + 4]) {
#pragma unroll
  for (int q = 0; q < TB * kTK / 256; ++q) {
    const int e = threadIdx.x + 256 * q;
    s[tile_k<TB>(o, e)][tile_i<TB>(o, e)] = r[q];
  }
}

template <int TB>
__global__ void __launch_bounds__(256)
expert_simt_kernel(const ExpertDesc g) {
  __shared__ __align__(16) float As[kTK][TB + 4];
  __shared__ __align__(16) float Bs[kTK][TB + 4];
  constexpr int S = TB / 16;  // sums per thread and direction
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
    const long long tn = (N + TB - 1) / TB, tiles = ((M + TB - 1) / TB) * tn;
    for (; next < first + tiles; next += gridDim.x) {
      const int i0 = (int)((next - first) / tn) * TB, j0 = (int)((next - first) % tn) * TB;
      const char* a = reinterpret_cast<const char*>(g.a) + lo * g.ld_a * es;
      const char* b = reinterpret_cast<const char*>(g.b) + (g.kind == kWeightGrad ? lo * g.ld_b : e * g.stride_b) * es;
      const Operand A = g.kind == kWeightGrad ? Operand{a, 1, g.ld_a, M, K} : Operand{a, g.ld_a, 1, M, K};
      const Operand B = g.kind == kForward ? Operand{b, g.ld_b, 1, N, K} : Operand{b, 1, g.ld_b, N, K};
      float acc[S][S] = {};
      float ra[TB * kTK / 256], rb[TB * kTK / 256];
      fetch<TB>(A, g.dtype, i0, 0, ra);
      fetch<TB>(B, g.dtype, j0, 0, rb);
      for (int k0 = 0; k0 < K; k0 += kTK) {
        put<TB>(A, ra, As);
        put<TB>(B, rb, Bs);
        __syncthreads();
        if (k0 + kTK < K) {
          fetch<TB>(A, g.dtype, i0, k0 + kTK, ra);
          fetch<TB>(B, g.dtype, j0, k0 + kTK, rb);
        }
#pragma unroll
        for (int kk = 0; kk < kTK; ++kk) {
          float av[S], bv[S];
#pragma unroll
          for (int i = 0; i < S; ++i) {
            av[i] = As[kk][ty * S + i];
            bv[i] = Bs[kk][tx * S + i];
          }
#pragma unroll
          for (int i = 0; i < S; ++i)
#pragma unroll
            for (int j = 0; j < S; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        __syncthreads();
      }
      const long long base = g.kind == kWeightGrad ? e * g.stride_d : lo * g.ld_d;
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < S; ++j) {
          const int r = i0 + ty * S + i, c = j0 + tx * S + j;
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
  // the most 64 x 64 tiles that the launch can have
  const long long tn = ((g.kind == kForward ? g.outer : g.inner) + 63) / 64;
  const long long tiles = tn * (g.kind == kWeightGrad ? (long long)g.experts * ((g.outer + 63) / 64)
                                                      : std::min<long long>(g.rows, g.rows / 64 + g.experts));
  if (tiles < 2 * num_sms()) expert_simt_kernel<32><<<4 * num_sms(), 256, 0, s>>>(g);
  else expert_simt_kernel<64><<<4 * num_sms(), 256, 0, s>>>(g);
  return (int)cudaGetLastError();
}

}  // namespace muon
