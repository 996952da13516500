// The whole Newton-Schulz chain and update of small blocks in one launch: n <= 128
// rows (the heads of an attention projection), up to 4096 columns, 16-bit
// storage, the standard form.
//
//   A = f^2 X X^T,  B = b A + c A A,  X <- f (a X + B X)   K times,
//   then W <- decay W - step X
//
// (f = 1 / (||U|| + eps) in the first iteration of a chain that starts from the
// raw U, 1 otherwise.)  As separate launches these products cannot fill the
// GPU: X X^T of a 128 x 2048 block is one output tile with a 2048-deep sum,
// A A one tile with a 128-deep one, and X makes two trips through L2 an
// iteration (44 us an iteration on 64 blocks, of which the arithmetic is 4).
//
// Here a cluster of C CTAs (1, 2, 4 or 8) owns a block and keeps X in shared
// memory from the first product to the update: each CTA holds all rows of a
// slice of at most 512 columns, as 64-column blocks of 128 rows in the 128-byte
// swizzle.  The same bytes are both operands of X X^T (rows contiguous along
// the sum) and the B operand of B X (columns contiguous, rows along the sum), so
// nothing is transposed.
//   X X^T   each CTA sums its slice's columns into TMEM; the partial sums (fp32)
//           go to shared memory, CTA r adds rows [128 r / C, 128 (r + 1) / C) of
//           all CTAs over distributed shared memory in rank order, and stores
//           them, rounded once, into every CTA's A
//   A A     in every CTA (one 128 x 128 x 128 product), B over A in place
//   B X     each CTA its own columns, 128 at a time: a column chunk of X is
//           overwritten by its epilogue once that chunk's product is done
// A, B and X are rounded to the chain's type where the separate products store
// them; X X^T is summed in another order, so results differ from theirs by
// roundings.  W is brought into L2 while the chain runs, and updated at the end
// from shared memory.
//
// Bounded by latency: of the 16 thousand cycles of an iteration (four CTAs, 512
// columns each) the tensor cores work 4.6; X X^T takes 3.0 thousand, the sum over
// the CTAs and its barriers 6.8, B 1.6, B X and its epilogue 4.6.  64 blocks of
// 128 x 2048 take 118 us in two waves of 37 clusters.
//
// Waits on mbarriers are bounded; on expiry a CTA raises its abort flag, skips
// its further waits and still takes part in every cluster barrier, so that none
// is left waiting, then reports through the error word.
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "tc_common.cuh"

namespace muon {
namespace tc {
namespace blk {

constexpr int EPI_WARPS = 16;
constexpr int THREADS = 32 * EPI_WARPS + 32;         // and one warp that issues the loads and MMAs
constexpr int ROWS = 128;
constexpr int BLOCK_BYTES = ROWS * 128;              // 128 rows x 64 columns
constexpr int MOST_SLICE = 512;
constexpr int X_BYTES = MOST_SLICE / 64 * BLOCK_BYTES;
constexpr int GRAM_BYTES = 2 * BLOCK_BYTES;          // A, then B
constexpr int PART_BYTES = ROWS * ROWS * 4;          // partial sums; at the end the update's staging boxes
constexpr int SMEM = X_BYTES + GRAM_BYTES + PART_BYTES + 256 + 1024;
static_assert(SMEM <= 232448 && EPI_WARPS * STAGE_TILE_BYTES <= PART_BYTES, "shared memory");

struct BParams {
  int n, m, slice, iters, raw;
  const float* inv;
  int* err;
  long long timeout_ns;
  float coeffs[3 * kBlockChainMaxIters];
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// Byte of 16-byte chunk c (8 columns) of a row in a 64-column block.
__device__ __forceinline__ uint32_t at16(int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); }

// Two values of the chain's type in a word (one conversion instruction each way
// per pair: the epilogues are bound by their instructions).
template <int IN_FMT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (IN_FMT) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <int IN_FMT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (IN_FMT) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Four 16-byte chunks (32 values) of a row: x <- s * acc + c * x, rounded.
template <int IN_FMT>
__device__ __forceinline__ void blend32(uint8_t* block, int row, int chunk, const uint32_t (&acc)[32], float s, float c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4* at = reinterpret_cast<uint4*>(block + at16(row, chunk + i));
    uint4 w = *at;
    uint32_t* e = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = unpack2<IN_FMT>(e[k]);
      const float a0 = __uint_as_float(acc[8 * i + 2 * k]), a1 = __uint_as_float(acc[8 * i + 2 * k + 1]);
      e[k] = pack2<IN_FMT>(fmaf(c, x.x, s * a0), fmaf(c, x.y, s * a1));
    }
    *at = w;
  }
}

// What a warp needs of one 32 x 32 box of O for the update: where the box lies in
// W (in W's own orientation), and W's segments, loaded ahead.
struct Box {
  char* base;
  long long ld;
  int rows, cols, r0, c0;  // of W that exist; first row and column of X
  uint4 w[4];
};
// Box k of this warp's share of the slice (64 columns of X at a time).
__device__ __forceinline__ void locate(Box& x, const BParams& p, const UpdateSlots& u, int b, int col0, int k) {
  const int boxes_down = (p.n + 31) >> 5;
  x.r0 = k % boxes_down * 32;
  x.c0 = k / boxes_down * 32;
  const unsigned kind = u.kind[b];
  const int es = ((kind >> 1) & 3) == kFP32 ? 4 : 2;
  x.ld = u.ld[b];
  const int gr = x.r0, gc = col0 + x.c0;
  char* W = reinterpret_cast<char*>(u.w[b]);
  if (kind & 1u) {  // stored m x n: the box's rows are X's columns
    x.base = W + (gc * x.ld + gr) * es;
    x.rows = min(32, p.m - gc);
    x.cols = min(32, p.n - gr);
  } else {
    x.base = W + (gr * x.ld + gc) * es;
    x.rows = min(32, p.n - gr);
    x.cols = min(32, p.m - gc);
  }
}
// Lane l takes row 8 i + l / 4 and the 8 columns from 8 (l % 4), i = 0..3.
__device__ __forceinline__ bool box_vec(const Box& x, unsigned kind, int i, int lane) {
  return (kind & 8u) && ((kind >> 1) & 3) != kFP32 && i * 8 + (lane >> 2) < x.rows && (lane & 3) * 8 + 8 <= x.cols;
}
__device__ __forceinline__ void load_box(Box& x, unsigned kind, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (box_vec(x, kind, i, lane))
      x.w[i] = *reinterpret_cast<const uint4*>(x.base + ((i * 8 + (lane >> 2)) * x.ld + (lane & 3) * 8) * 2);
}

template <int IN_FMT, int CL>
__global__ void __launch_bounds__(THREADS, 1)
ns_block_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ BParams p,
                const __grid_constant__ UpdateSlots u) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* X = smem;
  uint8_t* A = X + X_BYTES;
  uint8_t* part = A + GRAM_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(part + PART_BYTES);
  uint64_t* load_bar = bars;       // X has arrived
  uint64_t* gram_bar = bars + 1;   // X X^T
  uint64_t* sq_bar = bars + 2;     // A A
  uint64_t* up_bar = bars + 3;     // [4] B X, 128 columns each
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 7);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool issuer = warp == EPI_WARPS;     // the warp that issues loads and MMAs
  const int q = warp & 3, quarter = warp >> 2;  // TMEM lane quarter; which 32 of 128 columns
  const int row = q * 32 + lane;
  const uint32_t rank = cluster_rank();
  const int b = blockIdx.x / CL;
  const int col0 = (int)rank * p.slice;
  const int blocks = p.slice / 64, chunks = p.slice / 128;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 7; ++i) mbar_init(smem_u32(&bars[i]), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (issuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  const uint32_t lanes = (uint32_t)(q * 32) << 16;
  constexpr uint32_t idesc_kk = make_idesc(IN_FMT, 0, ROWS, 128), idesc_mn = make_idesc(IN_FMT, 1, ROWS, 128);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!*abort_flag) mbar_wait(smem_u32(bar), parity, abort_flag, p.timeout_ns);
    __syncwarp();
    tc_fence_after();
  };
  // product of K-major A (over this CTA's A) and itself or X, eight k-steps
  auto gram_desc = [&](int k) {
    return smem_desc(smem_u32(A + (k >> 2) * BLOCK_BYTES) + (k & 3) * (UMMA_K * 2), 16, 1024);
  };

  const unsigned kind = u.kind[b];
  const int boxes = ((p.n + 31) >> 5) * (p.slice / 32);
  if (issuer) {
    if (lane == 0) {
      // columns past m and rows past n arrive as zeros
      mbar_expect_tx(smem_u32(load_bar), blocks * BLOCK_BYTES);
      for (int k = 0; k < blocks; ++k)
        tma_load_3d(smem_u32(X + k * BLOCK_BYTES), &tmap_x, smem_u32(load_bar), col0 + k * 64, 0, b);
      // this CTA's own copies: waited for whatever the other roles met
      volatile int never = 0;
      if (!mbar_wait(smem_u32(load_bar), 0, &never, p.timeout_ns)) *abort_flag = 1;
    }
    __syncwarp();
  } else {
    // W is read at the end: bring it into L2 under the iterations
    for (int k = warp; k < boxes; k += EPI_WARPS) {
      Box x;
      locate(x, p, u, b, col0, k);
      const int es = ((kind >> 1) & 3) == kFP32 ? 4 : 2;
      if (lane < x.rows && x.cols > 0)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(x.base + lane * x.ld * es));
    }
    wait(load_bar, 0);
  }

  uint32_t sq_parity = 0;  // of the next A A: iterations without that term skip it
  for (int it = 0; it < p.iters; ++it) {
    const uint32_t parity = it & 1;
    const float a = p.coeffs[3 * it], bb = p.coeffs[3 * it + 1], cc = p.coeffs[3 * it + 2];
    const float f = it == 0 && p.raw ? p.inv[b] : 1.f;

    // ---- A = f^2 X X^T
    if (issuer) {
      if (lane == 0) {
        for (int k = 0; k < blocks * 4; ++k) {
          const uint64_t d = smem_desc(smem_u32(X + (k >> 2) * BLOCK_BYTES) + (k & 3) * (UMMA_K * 2), 16, 1024);
          tc_mma(tmem, d, d, idesc_kk, k > 0);
        }
        tc_commit(smem_u32(gram_bar));
      }
      __syncwarp();
    } else {
      wait(gram_bar, parity);
      uint32_t r[32];
      tmem_ld32(tmem + lanes + quarter * 32, r);
      if constexpr (CL == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack2<IN_FMT>(f * f * __uint_as_float(r[8 * i + 2 * k]), f * f * __uint_as_float(r[8 * i + 2 * k + 1]));
          *reinterpret_cast<uint4*>(A + (quarter >> 1) * BLOCK_BYTES + at16(row, (quarter & 1) * 4 + i)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
        // partial sums: row r, 16-byte chunk k at r * 512 + ((k ^ (r & 31)) << 4)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = quarter * 8 + i;
          *reinterpret_cast<uint4*>(part + row * 512 + ((k ^ (row & 31)) << 4)) =
              make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
      }
      tc_fence_before();
    }
    if constexpr (CL > 1) {
      cluster_sync();  // every CTA's partial sums are there
      if (!issuer) {
        // this CTA's rows of all CTAs, every load in flight at once
        constexpr int PER = ROWS / CL / EPI_WARPS > 0 ? ROWS / CL / EPI_WARPS : 1;
        const uint32_t part0 = smem_u32(part), a0 = smem_u32(A);
        float4 v[PER][CL];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int r = ROWS / CL * (int)rank + i * EPI_WARPS + warp;
          const uint32_t off = part0 + r * 512 + ((lane ^ (r & 31)) << 4);
#pragma unroll
          for (int c = 0; c < CL; ++c) v[i][c] = ld_cluster4(mapa(off, c));
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int r = ROWS / CL * (int)rank + i * EPI_WARPS + warp;
          float4 s = v[i][0];
#pragma unroll
          for (int c = 1; c < CL; ++c) {
            s.x += v[i][c].x; s.y += v[i][c].y; s.z += v[i][c].z; s.w += v[i][c].w;
          }
          const uint32_t lo = pack2<IN_FMT>(f * f * s.x, f * f * s.y), hi = pack2<IN_FMT>(f * f * s.z, f * f * s.w);
          // columns 4 lane .. 4 lane + 3: half of a 16-byte chunk
          const uint32_t to = a0 + (lane >> 4) * BLOCK_BYTES + at16(r, (lane & 15) >> 1) + (lane & 1) * 8;
#pragma unroll
          for (int c = 0; c < CL; ++c) st_cluster2(mapa(to, c), lo, hi);
        }
        asm volatile("fence.proxy.async;" ::: "memory");  // the MMAs of every CTA read A through the async proxy
      }
      cluster_sync();  // A is complete everywhere
    } else {
      fence_async_smem();
      __syncthreads();
    }
    tc_fence_after();

    // ---- B = b A + c A A, over A
    float scale = bb;  // of the product below: B X, or b A X without an A A term
    if (cc != 0.f) {
      scale = 1.f;
      if (issuer) {
        if (lane == 0) {
          fence_async_smem();
          for (int k = 0; k < 8; ++k) tc_mma(tmem + 128, gram_desc(k), gram_desc(k), idesc_kk, k > 0);
          tc_commit(smem_u32(sq_bar));
        }
        __syncwarp();
      } else {
        wait(sq_bar, sq_parity);
        uint32_t r[32];
        tmem_ld32(tmem + lanes + 128 + quarter * 32, r);
        blend32<IN_FMT>(A + (quarter >> 1) * BLOCK_BYTES, row, (quarter & 1) * 4, r, cc, bb);
        fence_async_smem();
        tc_fence_before();
      }
      sq_parity ^= 1u;
      __syncthreads();
      tc_fence_after();
    }

    // ---- X <- f (a X + B X), 128 columns at a time (256 took the same time)
    if (issuer) {
      if (lane == 0) {
        fence_async_smem();
        for (int j = 0; j < chunks; ++j) {
          for (int k = 0; k < 8; ++k) {
            const uint64_t bd = smem_desc(smem_u32(X + 2 * j * BLOCK_BYTES) + k * (UMMA_K * 128), BLOCK_BYTES, 1024);
            tc_mma(tmem + j * 128, gram_desc(k), bd, idesc_mn, k > 0);
          }
          tc_commit(smem_u32(&up_bar[j]));
        }
      }
      __syncwarp();
    } else {
#pragma unroll 1
      for (int j = 0; j < chunks; ++j) {
        wait(&up_bar[j], parity);
        uint32_t r[32];
        tmem_ld32(tmem + lanes + j * 128 + quarter * 32, r);
        blend32<IN_FMT>(X + (2 * j + (quarter >> 1)) * BLOCK_BYTES, row, (quarter & 1) * 4, r, f * scale, f * a);
      }
      fence_async_smem();
      tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
  }

  // ---- W <- decay W - step X, in W's orientation, 32 x 32 boxes per warp with
  // the next box's W on its way
  if (!issuer) {
    uint8_t* S = part + warp * STAGE_TILE_BYTES;
    const int wdt = (int)(kind >> 1) & 3, es = wdt == kFP32 ? 4 : 2;
    int bad = 0;
    Box now, next;
    if (warp < boxes) {
      locate(next, p, u, b, col0, warp);
      load_box(next, kind, lane);
    }
    for (int k = warp; k < boxes; k += EPI_WARPS) {
      now = next;
      if (k + EPI_WARPS < boxes) {
        locate(next, p, u, b, col0, k + EPI_WARPS);
        load_box(next, kind, lane);
      }
      if (now.rows <= 0 || now.cols <= 0) continue;  // past m: warp-uniform
      const uint8_t* x = X + (now.c0 >> 6) * BLOCK_BYTES;
      const int ch = (now.c0 & 63) >> 3;  // first 16-byte chunk of the box's rows
      if (kind & 1u) {
        // rows of W are columns of X: turn the box through the staging box
        uint32_t m[4][4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(m[g][0]), "=r"(m[g][1]), "=r"(m[g][2]), "=r"(m[g][3])
                       : "r"(smem_u32(x) + at16(now.r0 + lane, ch + g))
                       : "memory");
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 4; ++g)
          asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                           smem_u32(S) + sw64(g * 8 + (lane & 7), lane >> 3)),
                       "r"(m[g][0]), "r"(m[g][1]), "r"(m[g][2]), "r"(m[g][3])
                       : "memory");
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), c = (lane & 3) * 8;
        if (r >= now.rows || c >= now.cols) continue;
        const uint4 seg = *reinterpret_cast<const uint4*>((kind & 1u) ? S + sw64(r, lane & 3) : x + at16(now.r0 + r, ch + (lane & 3)));
        const int valid = min(8, now.cols - c);
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (IN_FMT) o[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(&seg)[e]);
          else o[e] = __half2float(reinterpret_cast<const __half*>(&seg)[e]);
          bad |= e < valid && !isfinite(o[e]);
        }
        update8(now.base + (r * now.ld + c) * es, wdt, o, valid, valid == 8 && (kind & 8u), u.decay, u.step,
                box_vec(now, kind, i, lane), now.w[i]);
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0 && u.status != nullptr) atomicOr(u.status + u.status_idx[b], kStatusNonFinite);
  }

  __syncthreads();
  if (issuer) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  if (threadIdx.x == 0 && *abort_flag && p.err != nullptr) atomicOr(p.err, kStatusTimeout);
}

static int cluster_for(int m) {
  int c = 1;
  while (c * MOST_SLICE < m) c *= 2;
  return c;
}

template <int IN_FMT, int CL>
static int launch(const CUtensorMap& map, const BParams& p, const UpdateSlots& u, int count, cudaStream_t s) {
  static std::atomic<int> opted[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return (int)cudaErrorInvalidDevice;
  auto kern = ns_block_kernel<IN_FMT, CL>;
  if (!opted[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return (int)e;
    opted[dev].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(count * CL));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = programmatic_launch() ? 2 : 1;
  return (int)cudaLaunchKernelEx(&cfg, kern, map, p, u);
}

}  // namespace blk
}  // namespace tc

bool ns_block_ok(int n, int m, int iters) {
  return n <= tc::blk::ROWS && m <= 8 * tc::blk::MOST_SLICE && iters <= kBlockChainMaxIters;
}

int launch_ns_block(const BlockChainArgs& a, const UpdateSlots& u, cudaStream_t s) {
  using namespace tc;
  using namespace tc::blk;
  BParams p{};
  p.n = a.n; p.m = a.m; p.iters = a.iters; p.raw = a.raw;
  const int cluster = cluster_for(a.m);
  p.slice = ((a.m + cluster - 1) / cluster + 127) / 128 * 128;
  p.inv = a.inv; p.err = a.err;
  p.timeout_ns = wait_timeout_ns();
  for (int i = 0; i < 3 * a.iters; ++i) p.coeffs[i] = a.coeffs[i];
  CUtensorMap map;
  if (!encode_map(&map, a.dtype, a.x, a.m, a.n, a.count, a.ld_x, a.x_bs, 64, ROWS)) return (int)cudaErrorInvalidValue;
  const bool bf = a.dtype == kBF16;
  switch (cluster) {
    case 1: return bf ? launch<1, 1>(map, p, u, a.count, s) : launch<0, 1>(map, p, u, a.count, s);
    case 2: return bf ? launch<1, 2>(map, p, u, a.count, s) : launch<0, 2>(map, p, u, a.count, s);
    case 4: return bf ? launch<1, 4>(map, p, u, a.count, s) : launch<0, 4>(map, p, u, a.count, s);
    default: return bf ? launch<1, 8>(map, p, u, a.count, s) : launch<0, 8>(map, p, u, a.count, s);
  }
}

}  // namespace muon
