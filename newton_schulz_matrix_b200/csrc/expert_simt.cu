// The three products of an expert layer on the CUDA cores: any of the storage
// types (fp32 math), any pitch and alignment.  It carries fp32 operands, whose
// products the tensor cores would round to TF32, and small 16-bit ones that TMA
// cannot address (a base, pitch or stride that is no multiple of 16 bytes).
//
// 128 x 128 output tiles with an 8 x 8 block of sums per thread (16384 fp32 rows
// over 16 experts of 1408 x 2048: 35 TFLOP/s, bound by the FMA pipe and the
// shared-memory reads beside it; 64 x 64 tiles 23), 64 x 64 with 4 x 4 or 32 x 32
// with 2 x 2 where larger ones cannot occupy the SMs (15 rows over 2 experts, 1946
// to 848 wide, forward: 62 us with 32 x 32 tiles, 140 with 64 x 64; 1610 rows over
// 25 experts, 144 to 304 wide: 31 and 22) or the segments cannot fill them (2000
// rows over 1024 experts, 64 to 64 wide: 56 us with 32 x 32, 78 with 128 x 128).
// The k steps go through shared memory, the next step's elements being
// loaded into registers while this one is multiplied.  The tile list comes from
// the offsets on the device: every block keeps the segments and a running count
// of tiles in shared memory, takes the tiles of its own index and stride and
// finds their experts by bisection, so nothing waits for the counts on the host.
// (Walking the offsets in memory instead cost each block a fifth of a microsecond
// per expert: those 2000 rows 245 us, 203 rows over 64 experts 49 us for 19 now.)
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
__global__ void __launch_bounds__(256, 1)
expert_simt_kernel(const ExpertDesc g) {
  __shared__ __align__(16) float As[TK][TB + 4];
  __shared__ __align__(16) float Bs[TK][TB + 4];
  __shared__ int seg_lo[kMaxExperts], seg_len[kMaxExperts], rows_before[kMaxExperts + 1];
  constexpr int S = TB / 16;  // sums per thread and direction
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const T* ga = reinterpret_cast<const T*>(g.a);
  const T* gb = reinterpret_cast<const T*>(g.b);
  const bool wg = g.kind == kWeightGrad;
  const int N = g.kind == kForward ? g.outer : g.inner;
  const long long tn = (N + TB - 1) / TB;
  for (int e = threadIdx.x; e < g.experts; e += blockDim.x) {
    const int lo = (int)min(max((long long)g.offsets[e], 0LL), g.rows);
    seg_lo[e] = lo;
    seg_len[e] = (int)min(max((long long)g.offsets[e + 1], (long long)lo), g.rows) - lo;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    // running counts of tile rows, 32 experts at a time
    const int lane = threadIdx.x;
    int sum = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 32) {
      const int e = e0 + lane;
      int incl = e < g.experts ? ((wg ? g.outer : seg_len[e]) + TB - 1) / TB : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < g.experts) rows_before[e + 1] = sum + incl;
      sum += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) rows_before[0] = 0;
  }
  __syncthreads();
  const long long total = rows_before[g.experts] * tn;
#pragma unroll 1
  for (long long next = blockIdx.x; next < total; next += gridDim.x) {
    const int tile_row = (int)(next / tn);
    // its expert: the last one with rows_before[e] <= tile_row (empty ones repeat a count)
    int e = 0;
    for (int past = g.experts; past - e > 1;) {
      const int mid = (e + past) >> 1;
      if (rows_before[mid] <= tile_row) e = mid; else past = mid;
    }
    const int M = wg ? g.outer : seg_len[e];
    const int K = g.kind == kForward ? g.inner : g.kind == kInputGrad ? g.outer : seg_len[e];
    const int i0 = (tile_row - rows_before[e]) * TB, j0 = (int)(next % tn) * TB;
    const T* a = ga + seg_lo[e] * g.ld_a;
    const T* b = gb + (wg ? seg_lo[e] * g.ld_b : e * g.stride_b);
    const Operand A = wg ? Operand{a, 1, g.ld_a, M, K} : Operand{a, g.ld_a, 1, M, K};
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
#pragma unroll (TB > 64 ? 4 : TK)
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
    const long long base = wg ? e * g.stride_d : seg_lo[e] * g.ld_d;
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
}

template <typename T>
int launch(const ExpertDesc& g, cudaStream_t s) {
  // the most tiles of edge t that the launch can have
  auto tiles = [&](int t) {
    const long long tn = ((g.kind == kForward ? g.outer : g.inner) + t - 1) / t;
    return tn * (g.kind == kWeightGrad ? (long long)g.experts * ((g.outer + t - 1) / t)
                                       : std::min<long long>(g.rows, g.rows / t + g.experts));
  };
  // and the average length of a segment in the direction that the tiles cut
  const long long fill = g.kind == kWeightGrad ? g.outer : g.rows / g.experts;
  const int sms = num_sms();
  if (tiles(64) < sms || fill <= 32) expert_simt_kernel<T, 32, 32><<<4 * sms, 256, 0, s>>>(g);
  else if (tiles(128) < 2 * sms || fill <= 64) expert_simt_kernel<T, 64, 32><<<4 * sms, 256, 0, s>>>(g);
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
