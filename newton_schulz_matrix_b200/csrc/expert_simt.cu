// The three products of an expert layer on the CUDA cores: any of the storage
// types (fp32 math), any pitch and alignment.  It carries fp32 operands, whose
// products the tensor cores would round to TF32, and small 16-bit ones that TMA
// cannot address (a base, pitch or stride that is no multiple of 16 bytes).
//
// 128 x 128 output tiles with an 8 x 8 block of sums per thread (16384 fp32 rows
// over 16 experts of 1408 x 2048: 35 TFLOP/s, bound by the FMA pipe and the
// shared-memory reads beside it; 64 x 64 tiles 23), 64 x 64 with 4 x 4 or 32 x 32
// with 2 x 2 where larger ones cannot occupy the SMs: the three products of 301
// rows over 7 experts, 333 to 130 wide, take 39 us with 32 x 32 tiles and 73 with
// 64 x 64.  The k steps go through shared memory, the next step's elements being
// loaded into registers while this one is multiplied.  The tile list is read
// from the offsets on the device: a block walks the experts' tiles of its own
// index and stride, so nothing waits for the counts on the host.
#include <algorithm>

#include "common.cuh"
#include "expert.h"
#include "internal.h"

namespace muon {
namespace {

// Element (i, k) of an operand at p + i * si + k * sk.
struct Operand {
  const void* p;
  long long si, sk;
  int rows, depth;
};

// This thread's elements of a TB x TK tile: consecutive threads along the
// operand's contiguous direction.
template <int TB, int TK>
__device__ __forceinline__ int tile_i(const Operand& o, int e) { return o.sk == 1 ? e / TK : e % TB; }
template <int TB, int TK>
__device__ __forceinline__ int tile_k(const Operand& o, int e) { return o.sk == 1 ? e % TK : e / TB; }
template <typename T, int TB, int TK>
__device__ __forceinline__ void fetch(const Operand& o, int i0, int k0, float (&r)[TB * TK / 256]) {
  const T* p = reinterpret_cast<const T*>(o.p);
#pragma unroll
  for (int q = 0; q < TB * TK / 256; ++q) {
    const int e = threadIdx.x + 256 * q;
    const int i = i0 + tile_i<TB, TK>(o, e), k = k0 + tile_k<TB, TK>(o, e);
    r[q] = i < o.rows && k < o.depth ? to_f32(p[i * o.si + k * o.sk]) : 0.f;
  }
}
template <int TB, int TK>
__device__ __forceinline__ void put(const Operand& o, const float (&r)[TB * TK / 256], float (*s)[TB + 4]) {
#pragma unroll
  for (int q = 0; q < TB * TK / 256; ++q) {
    const int e = threadIdx.x + 256 * q;
    s[tile_k<TB, TK>(o, e)][tile_i<TB, TK>(o, e)] = r[q];
  }
}
// S consecutive values of a row of a tile.
template <int S>
__device__ __forceinline__ void take(const float* s, float (&v)[S]) {
#pragma unroll
  for (int i = 0; i < S; i += S < 4 ? 2 : 4) {
    if constexpr (S < 4) {
      const float2 f = *reinterpret_cast<const float2*>(s + i);
      v[i] = f.x; v[i + 1] = f.y;
    } else {
      const float4 f = *reinterpret_cast<const float4*>(s + i);
      v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
    }
  }
}

template <typename T, int TB, int TK>
__global__ void __launch_bounds__(256, TB > 64 ? 2 : 1)
expert_simt_kernel(const ExpertDesc g) {
  __shared__ __align__(16) float As[TK][TB + 4];
  __shared__ __align__(16) float Bs[TK][TB + 4];
  constexpr int S = TB / 16;  // sums per thread and direction
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const T* ga = reinterpret_cast<const T*>(g.a);
  const T* gb = reinterpret_cast<const T*>(g.b);
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
      const T* a = ga + lo * g.ld_a;
      const T* b = gb + (g.kind == kWeightGrad ? lo * g.ld_b : e * g.stride_b);
      const Operand A = g.kind == kWeightGrad ? Operand{a, 1, g.ld_a, M, K} : Operand{a, g.ld_a, 1, M, K};
      const Operand B = g.kind == kForward ? Operand{b, g.ld_b, 1, N, K} : Operand{b, 1, g.ld_b, N, K};
      float acc[S][S] = {};
      float ra[TB * TK / 256], rb[TB * TK / 256];
      fetch<T, TB, TK>(A, i0, 0, ra);
      fetch<T, TB, TK>(B, j0, 0, rb);
      for (int k0 = 0; k0 < K; k0 += TK) {
        put<TB, TK>(A, ra, As);
        put<TB, TK>(B, rb, Bs);
        __syncthreads();
        if (k0 + TK < K) {
          fetch<T, TB, TK>(A, i0, k0 + TK, ra);
          fetch<T, TB, TK>(B, j0, k0 + TK, rb);
        }
#pragma unroll (TB > 64 ? 8 : TK)
        for (int kk = 0; kk < TK; ++kk) {
          float av[S], bv[S];
          take<S>(&As[kk][ty * S], av);
          take<S>(&Bs[kk][tx * S], bv);
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

template <typename T>
int launch(const ExpertDesc& g, cudaStream_t s) {
  // the most tiles of edge t that the launch can have
  auto tiles = [&](int t) {
    const long long tn = ((g.kind == kForward ? g.outer : g.inner) + t - 1) / t;
    return tn * (g.kind == kWeightGrad ? (long long)g.experts * ((g.outer + t - 1) / t)
                                       : std::min<long long>(g.rows, g.rows / t + g.experts));
  };
  const int sms = num_sms();
  if (tiles(64) < 2 * sms) expert_simt_kernel<T, 32, 32><<<4 * sms, 256, 0, s>>>(g);
  else if (tiles(128) < 2 * sms) expert_simt_kernel<T, 64, 32><<<4 * sms, 256, 0, s>>>(g);
  else expert_simt_kernel<T, 128, 16><<<2 * sms, 256, 0, s>>>(g);
  return (int)cudaGetLastError();
}

}  // namespace

int expert_simt(const ExpertDesc& g, cudaStream_t s) {
  switch (g.dtype) {
    case kBF16: return launch<__nv_bfloat16>(g, s);
    case kFP16: return launch<__half>(g, s);
    default: return launch<float>(g, s);
  }
}

}  // namespace muon
