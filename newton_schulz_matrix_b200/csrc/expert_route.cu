// Routing of an expert layer: the stable counting sort of token assignments
// by expert, the gather of the tokens' rows into expert order, and the
// weighted combine back to the tokens with its gradients.  All of them move
// bytes (or, below ~1e5 assignments, wait for latency); none needs the tensor
// cores.
//
//   sort     slot[t, j] = offsets[e] + #{assignments to e before (t, j)},  e = ids[t, j]
//   gather   xs[slot[t, j]] = x[t]
//   combine  y[t] = sum_j w[t, j] ys[slot[t, j]]
//   its gradients  dys[slot[t, j]] = w[t, j] dy[t],  dw[t, j] = <dy[t], ys[slot[t, j]]>
//
// The order of every floating-point sum is fixed (j ascending; a fixed tree
// over the columns), so results do not change from run to run.  Nothing is
// computed from a row that no assignment names: a dropped assignment is
// skipped rather than multiplied by zero, so Inf and NaN behind it stay out.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "expert.h"
#include "internal.h"

namespace muon {
namespace {

// ----------------------------------------------------------------------------
// sort
// ----------------------------------------------------------------------------
// A block ranks a run of consecutive assignments in two passes over them, its
// 32 warps taking consecutive pieces: pass 1 counts each warp's keys (lanes of
// equal key found by votes, one add per distinct key), a prefix over the
// warps and the experts turns the counts into first positions, and pass 2
// walks the same pieces again and hands positions out in order, so equal keys
// keep their order and no atomic decides a position.  A warp loads kKeys groups
// of 32 keys at once and, where its piece is no longer, keeps them for pass 2:
// one group at a time waits for memory at every group (131072 x 8 ids to 64
// experts: 26.3 us, 24.6 with groups of eight; 18 with votes in place of
// match_any and the early start below).
//
// Up to kSortOneBlock assignments run as one block and one launch (2048 to 64
// experts 6.6 us, two launches 6.9; 4096: 9.0 and 6.8); beyond, a first launch counts the keys of up
// to one run per SM, and every block of the second launch sums the counts of the
// runs before its own.  The second launch counts its own warps' keys while the
// first still runs (programmatic dependent launch).
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortOneBlock = 2048;
constexpr int kSortMinRun = 1024;
constexpr int kKeys = 8;
constexpr int kSortOwnSm = 120 * 1024;

__device__ __forceinline__ int key_of(const SortArgs& a, int i) {
  const long long at = a.ld == a.topk ? (long long)i : (long long)(i / a.topk) * a.ld + i % a.topk;
  const long long id = a.wide ? reinterpret_cast<const long long*>(a.ids)[at] : reinterpret_cast<const int*>(a.ids)[at];
  return id >= 0 && id < a.experts ? (int)id : a.experts;  // bucket `experts`: no expert
}

// The lanes of this warp that hold the same key, by one vote per bit of the keys.
__device__ __forceinline__ unsigned lanes_of(int key, int bits) {
  unsigned same = 0xffffffffu;
  for (int i = 0; i < bits; ++i) {
    const bool on = (key >> i) & 1;
    const unsigned votes = __ballot_sync(0xffffffffu, on);
    same &= on ? votes : ~votes;
  }
  return same;
}

__global__ void __launch_bounds__(kSortThreads)
expert_count_kernel(const SortArgs a, int n, int run, int* __restrict__ counts) {
  extern __shared__ int hist[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int e = threadIdx.x; e <= a.experts; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * run, last = min(n, first + run);
  for (int i0 = first + (int)threadIdx.x; i0 < last; i0 += kKeys * kSortThreads) {
    int key[kKeys];
#pragma unroll
    for (int q = 0; q < kKeys; ++q) {
      const int i = i0 + q * kSortThreads;
      key[q] = i < last ? key_of(a, i) : -1;
    }
#pragma unroll
    for (int q = 0; q < kKeys; ++q)
      if (key[q] >= 0) atomicAdd(&hist[key[q]], 1);
  }
  __syncthreads();
  int* out = counts + (long long)blockIdx.x * (a.experts + 1);
  for (int e = threadIdx.x; e <= a.experts; e += kSortThreads) out[e] = hist[e];
}

__global__ void __launch_bounds__(kSortThreads)
expert_rank_kernel(const SortArgs a, int n, int run, int warps, const int* __restrict__ counts) {
  extern __shared__ int smem[];
  const int E = a.experts, buckets = E + 1;
  int* hist = smem;                       // [warps][buckets]
  int* total = hist + warps * buckets;    // [buckets] whole-batch counts, then first positions
  int* before = total + buckets;          // [buckets] counts of the runs before this block's
  __shared__ int warp_sum[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x * run, last = min(n, first + run);

  for (int e = threadIdx.x; e < (warps + 2) * buckets; e += kSortThreads) smem[e] = 0;
  __syncthreads();

  // this warp's piece: whole groups of 32 consecutive assignments
  const int piece = ((last - first + warps - 1) / warps + 31) / 32 * 32;
  const int p0 = first + warp * piece, p1 = warp < warps ? min(last, p0 + piece) : p0;
  int* mine = hist + warp * buckets;
  const int bits = 32 - __clz(buckets);  // of keys 0 .. buckets (no assignment)
  int key[kKeys];
  auto load = [&](int i0) {
#pragma unroll
    for (int q = 0; q < kKeys; ++q) {
      const int i = i0 + q * 32 + lane;
      key[q] = i < p1 ? key_of(a, i) : buckets;
    }
  };
  for (int i0 = p0; i0 < p1; i0 += 32 * kKeys) {
    load(i0);
#pragma unroll
    for (int q = 0; q < kKeys; ++q) {
      if (i0 + q * 32 >= p1) break;
      const unsigned same = lanes_of(key[q], bits);
      if (key[q] < buckets && lane == __ffs(same) - 1) mine[key[q]] += __popc(same);
      __syncwarp();
    }
  }
  if (gridDim.x > 1) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the counts are complete
    // groups of threads share a bucket's column of counts; integer sums, so
    // their order does not matter
    const int groups = max(1, kSortThreads / buckets), g = (int)threadIdx.x / buckets;
    for (int e = threadIdx.x - g * buckets; e < buckets && g < groups; e += groups > 1 ? buckets : kSortThreads) {
      int all = 0, upto = 0;
#pragma unroll 8
      for (int b = g; b < (int)gridDim.x; b += groups) {
        const int c = counts[b * buckets + e];
        all += c;
        upto += b < (int)blockIdx.x ? c : 0;
      }
      atomicAdd(&total[e], all);
      atomicAdd(&before[e], upto);
    }
  }
  __syncthreads();
  const int e = threadIdx.x;              // experts <= kSortThreads: one per thread
  int all = 0;
  if (e < E) {
    if (gridDim.x > 1) {
      all = total[e];
    } else {
      for (int w = 0; w < warps; ++w) all += hist[w * buckets + e];
    }
  }
  int incl = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    warp_sum[lane] = v;
  }
  __syncthreads();
  if (warp > 0) incl += warp_sum[warp - 1];
  if (e < E) total[e] = incl - all;
  if (e == 0) total[E] = warp_sum[kSortWarps - 1];
  __syncthreads();
  if (blockIdx.x == 0)
    for (int k = threadIdx.x; k < buckets; k += kSortThreads) a.offsets[k] = total[k];
  // first position of every warp's keys
  for (int k = threadIdx.x; k < buckets; k += kSortThreads) {
    int at = total[k] + before[k];
    for (int w = 0; w < warps; ++w) {
      const int c = hist[w * buckets + k];
      hist[w * buckets + k] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int i0 = p0; i0 < p1; i0 += 32 * kKeys) {
    if (p1 - p0 > 32 * kKeys) load(i0);
#pragma unroll
    for (int q = 0; q < kKeys; ++q) {
      if (i0 + q * 32 >= p1) break;
      const int i = i0 + q * 32 + lane;
      const unsigned same = lanes_of(key[q], bits);
      const int leader = __ffs(same) - 1;
      int at = 0;
      if (key[q] < buckets && lane == leader) {
        at = mine[key[q]];
        mine[key[q]] = at + __popc(same);
      }
      at = __shfl_sync(0xffffffffu, at, leader);
      at += __popc(same & ((1u << lane) - 1u));
      if (i < p1) {
        a.slot[i] = key[q] < E ? at : -1;
        if (at < n) a.source[at] = i;  // ids that change under the sort write nothing out of range
      }
      __syncwarp();
    }
  }
}

struct SortPlan {
  int n, blocks, run, warps;
};
SortPlan sort_plan(int tokens, int topk) {
  SortPlan p{};
  p.n = tokens * topk;
  if (p.n <= kSortOneBlock) {
    p.blocks = 1;
    p.run = p.n;
  } else {
    const int most = (p.n + kSortMinRun - 1) / kSortMinRun;
    p.blocks = std::min(most, 148);
    p.run = (int)(((long long)p.n + p.blocks - 1) / p.blocks);
    p.blocks = (int)(((long long)p.n + p.run - 1) / p.run);
  }
  p.warps = std::max(1, std::min(kSortWarps, (p.run + 31) / 32));
  return p;
}

// ----------------------------------------------------------------------------
// gather, combine and its gradients
// ----------------------------------------------------------------------------
constexpr int kRouteThreads = 256;

// Threads along a row of `units` loads, and rows per block: a power of two
// that covers the row in one go where it is short, so that short rows share a
// block.
dim3 route_block(long long units) {
  int x = 8;
  while (x < kRouteThreads && x < units) x *= 2;
  return dim3(x, kRouteThreads / x);
}

template <int BYTES> struct Unit;
template <> struct Unit<16> { using T = uint4; };
template <> struct Unit<8> { using T = uint2; };
template <> struct Unit<4> { using T = unsigned; };
template <> struct Unit<2> { using T = unsigned short; };

// One token per blockDim.x threads: its row is read once (up to four units of
// a thread in flight) and written to every row its assignments name.
template <int BYTES>
__global__ void __launch_bounds__(kRouteThreads)
expert_gather_kernel(const RouteArgs a, int units, int es) {
  using U = typename Unit<BYTES>::T;
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.tokens) return;
  const U* src = reinterpret_cast<const U*>(reinterpret_cast<const char*>(a.by_token) + t * a.ld_token * es);
  const int* slot = a.slot + t * a.topk;
  for (int c0 = blockIdx.y * 4 * blockDim.x + threadIdx.x; c0 < units; c0 += gridDim.y * 4 * blockDim.x) {
    U v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c0 + q * (int)blockDim.x < units) v[q] = src[c0 + q * blockDim.x];
    for (int j = 0; j < a.topk; ++j) {
      const int s = slot[j];
      if (s < 0 || s >= a.rows) continue;
      U* dst = reinterpret_cast<U*>(reinterpret_cast<char*>(a.out_row) + (long long)s * a.ld_out_row * es);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c0 + q * (int)blockDim.x < units) dst[c0 + q * blockDim.x] = v[q];
    }
  }
}

// N elements of type T as one load.
template <typename T, int N> struct Pack;
template <typename T> struct Pack<T, 1> {
  T v;
  __device__ void get(float* f) const { f[0] = to_f32(v); }
  __device__ void set(const float* f) { v = from_f32<T>(f[0]); }
};
template <typename T> struct Pack<T, 16 / sizeof(T)> {
  uint4 v;
  __device__ void get(float* f) const {
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(T)); ++i) f[i] = to_f32(e[i]);
  }
  __device__ void set(const float* f) {
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(T)); ++i) e[i] = from_f32<T>(f[i]);
  }
};

// Combine and its gradients give a token to `wpt` neighbouring warps of a
// block, which walk its columns together: one warp where there are tokens
// enough to fill the GPU (no block-wide sum, and a warp's loads of one column
// step overlap the next's), more where there are few.  Up to kGroup
// assignments are read at once, their rows and weights kept in registers over
// the columns; more go in groups of kGroup.
constexpr int kGroup = 8;

struct Taken {  // up to kGroup assignments of a token
  int row[kGroup];
  float w[kGroup];
};
__device__ __forceinline__ Taken taken(const RouteArgs& a, long long t, int j0) {
  Taken r;
#pragma unroll
  for (int q = 0; q < kGroup; ++q) {
    const int j = j0 + q;
    const int s = j < a.topk ? a.slot[t * a.topk + j] : -1;
    r.row[q] = s < a.rows ? s : -1;
    r.w[q] = r.row[q] >= 0 && a.weights != nullptr ? load_any(a.weights, t * a.topk + j, a.w_dtype) : 1.f;
  }
  return r;
}

// The rows are added in the order of the assignments; fp32 sum, rounded once.
// A thread has U steps of columns in flight: one of 16 bytes (two take the
// registers of other warps, which hide more), four of one element.
// MORE: more than kGroup assignments a token (they are then looked up again at
// every step; kept apart, since the two loops together spill).
template <typename T, int N, int U, bool MORE>
__global__ void __launch_bounds__(256)
expert_combine_kernel(const RouteArgs a, int units, int wpt) {
  using P = Pack<T, N>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long t = ((long long)blockIdx.x * (blockDim.x >> 5) + warp) / wpt;
  if (t >= a.tokens) return;
  const int next = 32 * wpt * gridDim.y, step = next * U;
  const int first = (blockIdx.y * wpt + warp % wpt) * 32 + lane;
  const T* ys = reinterpret_cast<const T*>(a.by_row);
  const Taken head = taken(a, t, 0);
  for (int c = first; c < units; c += step) {
    float acc[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[u][i] = 0.f;
    auto add = [&](const Taken& k) {
      P v[U][kGroup];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < kGroup; ++q)
          if (k.row[q] >= 0 && c + u * next < units)
            v[u][q] = reinterpret_cast<const P*>(ys + (long long)k.row[q] * a.ld_row)[c + u * next];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < kGroup; ++q) {
          if (k.row[q] < 0) continue;
          float f[N];
          v[u][q].get(f);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[u][i] = fmaf(k.w[q], f[i], acc[u][i]);
        }
    };
    add(head);
    if constexpr (MORE) {
#pragma unroll 1
      for (int j0 = kGroup; j0 < a.topk; j0 += kGroup) add(taken(a, t, j0));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u * next >= units) break;
      P out;
      out.set(acc[u]);
      reinterpret_cast<P*>(reinterpret_cast<T*>(a.out_token) + t * a.ld_out_token)[c + u * next] = out;
    }
  }
}

// dy is read once per kGroup assignments, each row of ys once, and every row
// of dys is written once; the dot products go through a fixed tree (a lane's
// columns, lanes, then the token's warps in order).
template <typename T, int N, int U>
__global__ void __launch_bounds__(512)
expert_combine_backward_kernel(const RouteArgs a, int units, int wpt) {
  using P = Pack<T, N>;
  __shared__ float part[16][kGroup];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % wpt;
  const long long t = ((long long)blockIdx.x * (blockDim.x >> 5) + warp) / wpt;
  const bool live = t < a.tokens;
  const T* dy = reinterpret_cast<const T*>(a.by_token) + (live ? t : 0) * a.ld_token;
  const T* ys = reinterpret_cast<const T*>(a.by_row);
  T* dys = reinterpret_cast<T*>(a.out_row);
  const bool dots = a.dweights != nullptr;
  for (int j0 = 0; j0 < a.topk; j0 += kGroup) {
    float dot[kGroup];
#pragma unroll
    for (int q = 0; q < kGroup; ++q) dot[q] = 0.f;
    if (live) {
      const Taken k = taken(a, t, j0);
      const int next = 32 * wpt;
      for (int c = sub * 32 + lane; c < units; c += next * U) {
        P d[U], v[U][kGroup];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (c + u * next >= units) break;
          d[u] = reinterpret_cast<const P*>(dy)[c + u * next];
          if (dots) {
#pragma unroll
            for (int q = 0; q < kGroup; ++q)
              if (k.row[q] >= 0) v[u][q] = reinterpret_cast<const P*>(ys + (long long)k.row[q] * a.ld_row)[c + u * next];
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (c + u * next >= units) break;
          float g[N];
          d[u].get(g);
#pragma unroll
          for (int q = 0; q < kGroup; ++q) {
            if (k.row[q] < 0) continue;
            float f[N];
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = k.w[q] * g[i];
            P out;
            out.set(f);
            reinterpret_cast<P*>(dys + (long long)k.row[q] * a.ld_out_row)[c + u * next] = out;
            if (dots) {
              v[u][q].get(f);
#pragma unroll
              for (int i = 0; i < N; ++i) dot[q] = fmaf(g[i], f[i], dot[q]);
            }
          }
        }
      }
    }
    if (!dots) continue;
    float mine = 0.f;  // lane q: assignment j0 + q
#pragma unroll
    for (int q = 0; q < kGroup; ++q) {
      float s = dot[q];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == q) mine = s;
    }
    if (wpt > 1) {
      if (lane < kGroup) part[warp][lane] = mine;
      __syncthreads();
      if (sub == 0 && lane < kGroup)
        for (int k = 1; k < wpt; ++k) mine += part[warp + k][lane];
      __syncthreads();
    }
    if (live && sub == 0 && lane < kGroup && j0 + lane < a.topk)
      store_any(a.dweights, t * a.topk + j0 + lane, a.w_dtype, mine);
  }
}

// Warps per token: enough to give every SM 32 warps, no more than the row has
// steps of 32 units, at most 16.
int warps_per_token(int tokens, int units) {
  const int steps = (units + 31) / 32;
  int w = 1;
  while (w < 16 && w < steps && (long long)tokens * w < 32LL * num_sms()) w *= 2;
  return w;
}

bool on16(const void* p, long long ld, int es) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * es % 16 == 0;
}

// Calls f with a value of the element type and the elements of a unit: 16
// bytes where every row starts on 16 bytes and the width is whole units, one
// element otherwise.
template <typename F>
int with_type(int dtype, bool vec, F f) {
  switch (dtype) {
    case kBF16: return vec ? f(__nv_bfloat16{}, std::integral_constant<int, 8>{}) : f(__nv_bfloat16{}, std::integral_constant<int, 1>{});
    case kFP16: return vec ? f(__half{}, std::integral_constant<int, 8>{}) : f(__half{}, std::integral_constant<int, 1>{});
    default: return vec ? f(0.f, std::integral_constant<int, 4>{}) : f(0.f, std::integral_constant<int, 1>{});
  }
}

// Column blocks for calls with few tokens: enough blocks for the SMs.
int column_blocks(long long token_blocks, long long units, int per_block) {
  const long long most = (units + per_block - 1) / per_block;
  const long long want = (4LL * num_sms() + token_blocks - 1) / token_blocks;
  return (int)std::max(1LL, std::min(most, want));
}

}  // namespace

size_t expert_sort_ws_bytes(int tokens, int topk, int experts) {
  const SortPlan p = sort_plan(tokens, topk);
  return p.blocks > 1 ? (size_t)p.blocks * (experts + 1) * sizeof(int) : 0;
}

int launch_expert_sort(const SortArgs& a, int* ws, cudaStream_t s) {
  const SortPlan p = sort_plan(a.tokens, a.topk);
  // more than half an SM's shared memory where there is a block per SM: blocks
  // that start early would otherwise pair up on the first SMs that have room
  // (131072 x 8 to 64 experts: 27 us, 19 without the early start, 18 so)
  size_t smem = (size_t)(p.warps + 2) * (a.experts + 1) * sizeof(int);
  if (p.blocks > 1) smem = std::max(smem, (size_t)kSortOwnSm);
  if (smem > 48 * 1024) {
    static std::atomic<int> opted[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return (int)cudaErrorInvalidDevice;
    if (!opted[dev].load(std::memory_order_acquire)) {
      const int most = std::max((kSortWarps + 2) * (kMaxExperts + 1) * (int)sizeof(int), kSortOwnSm);
      const cudaError_t e = cudaFuncSetAttribute(expert_rank_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return (int)e;
      opted[dev].store(1, std::memory_order_release);
    }
  }
  if (p.blocks > 1) {
    expert_count_kernel<<<p.blocks, kSortThreads, (a.experts + 1) * sizeof(int), s>>>(a, p.n, p.run, ws);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.blocks);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = p.blocks > 1 ? 1 : 0;
  return (int)cudaLaunchKernelEx(&cfg, expert_rank_kernel, a, p.n, p.run, p.warps, (const int*)ws);
}

int launch_expert_gather(const RouteArgs& a, cudaStream_t s) {
  if (a.tokens == 0 || a.cols == 0) return 0;
  const int es = dtype_size(a.dtype);
  // the widest unit that every row's start and the width allow
  const uintptr_t mix = reinterpret_cast<uintptr_t>(a.by_token) | reinterpret_cast<uintptr_t>(a.out_row) |
                        (uintptr_t)(a.ld_token * es) | (uintptr_t)(a.ld_out_row * es) | (uintptr_t)((long long)a.cols * es);
  const int bytes = mix % 16 == 0 ? 16 : mix % 8 == 0 ? 8 : mix % 4 == 0 ? 4 : 2;
  const long long units = (long long)a.cols * es / bytes;
  const dim3 block = route_block(units);
  dim3 grid((a.tokens + block.y - 1) / block.y);
  grid.y = column_blocks(grid.x, units, 4 * block.x);
  switch (bytes) {
    case 16: expert_gather_kernel<16><<<grid, block, 0, s>>>(a, (int)units, es); break;
    case 8: expert_gather_kernel<8><<<grid, block, 0, s>>>(a, (int)units, es); break;
    case 4: expert_gather_kernel<4><<<grid, block, 0, s>>>(a, (int)units, es); break;
    default: expert_gather_kernel<2><<<grid, block, 0, s>>>(a, (int)units, es); break;
  }
  return (int)cudaGetLastError();
}

int launch_expert_combine(const RouteArgs& a, cudaStream_t s) {
  if (a.tokens == 0 || a.cols == 0) return 0;
  const int es = dtype_size(a.dtype);
  const bool vec = on16(a.by_row, a.ld_row, es) && on16(a.out_token, a.ld_out_token, es) && (long long)a.cols * es % 16 == 0;
  return with_type(a.dtype, vec, [&](auto type, auto n) {
    using T = decltype(type);
    constexpr int N = decltype(n)::value, U = N == 1 ? 4 : 1;
    const int units = a.cols / N, wpt = std::min(8, warps_per_token(a.tokens, units));
    dim3 grid((unsigned)(((long long)a.tokens * wpt + 7) / 8));
    grid.y = column_blocks(grid.x, units, 32 * wpt * U);
    if (a.topk <= kGroup) expert_combine_kernel<T, N, U, false><<<grid, 256, 0, s>>>(a, units, wpt);
    else expert_combine_kernel<T, N, 1, true><<<grid, 256, 0, s>>>(a, units, wpt);
    return (int)cudaGetLastError();
  });
}

int launch_expert_combine_backward(const RouteArgs& a, cudaStream_t s) {
  if (a.tokens == 0) return 0;
  const int es = dtype_size(a.dtype);
  const bool vec = on16(a.by_token, a.ld_token, es) && on16(a.out_row, a.ld_out_row, es) &&
                   (a.dweights == nullptr || on16(a.by_row, a.ld_row, es)) && (long long)a.cols * es % 16 == 0;
  return with_type(a.dtype, vec, [&](auto type, auto n) {
    const int units = a.cols / n, wpt = warps_per_token(a.tokens, units);
    const int warps = std::max(8, wpt);
    const unsigned grid = (unsigned)(((long long)a.tokens * wpt + warps - 1) / warps);
    constexpr int N = decltype(n)::value, U = N == 1 ? 4 : 2;
    expert_combine_backward_kernel<decltype(type), N, U><<<grid, 32 * warps, 0, s>>>(a, units, wpt);
    return (int)cudaGetLastError();
  });
}

}  // namespace muon
