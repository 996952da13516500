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
// roundings.  Bounded by latency: per iteration three dependent tensor-core
// phases, two cluster barriers and their epilogues.
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

constexpr int THREADS = 256;
constexpr int ROWS = 128;
constexpr int BLOCK_BYTES = ROWS * 128;              // 128 rows x 64 columns
constexpr int MOST_SLICE = 512;
constexpr int X_BYTES = MOST_SLICE / 64 * BLOCK_BYTES;
constexpr int GRAM_BYTES = 2 * BLOCK_BYTES;          // A, then B
constexpr int PART_BYTES = ROWS * ROWS * 4;          // partial sums; at the end the update's staging boxes
constexpr int SMEM = X_BYTES + GRAM_BYTES + PART_BYTES + 256 + 1024;
static_assert(SMEM <= 232448 && THREADS / 32 * STAGE_TILE_BYTES <= PART_BYTES, "shared memory");

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

__device__ __forceinline__ uint32_t pack2(float a, float b, int dt) {
  return (uint32_t)to_bits(a, dt) | ((uint32_t)to_bits(b, dt) << 16);
}

template <int IN_FMT>
__global__ void __launch_bounds__(THREADS, 1)
ns_block_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ BParams p,
                const __grid_constant__ UpdateSlots u) {
  constexpr int DT = IN_FMT ? kBF16 : kFP16;
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
  const int q = warp & 3, half = warp >> 2;   // TMEM lane quarter; which 64 of 128 columns
  const int row = q * 32 + lane;
  uint32_t cluster;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cluster));
  const uint32_t rank = cluster_rank();
  const int b = blockIdx.x / cluster;
  const int col0 = (int)rank * p.slice;
  const int blocks = p.slice / 64, chunks = p.slice / 128;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 7; ++i) mbar_init(smem_u32(&bars[i]), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
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
    tc_fence_after();
  };

  if (threadIdx.x == 0) {
    // columns past m and rows past n arrive as zeros
    mbar_expect_tx(smem_u32(load_bar), blocks * BLOCK_BYTES);
    for (int k = 0; k < blocks; ++k)
      tma_load_3d(smem_u32(X + k * BLOCK_BYTES), &tmap_x, smem_u32(load_bar), col0 + k * 64, 0, b);
  }
  {
    // this CTA's own copies: waited for whatever the other roles met
    volatile int never = 0;
    if (!mbar_wait(smem_u32(load_bar), 0, &never, p.timeout_ns)) *abort_flag = 1;
  }

  uint32_t sq_parity = 0;  // of the next A A: iterations without that term skip it
  for (int it = 0; it < p.iters; ++it) {
    const uint32_t parity = it & 1;
    const float a = p.coeffs[3 * it], bb = p.coeffs[3 * it + 1], cc = p.coeffs[3 * it + 2];
    const float f = it == 0 && p.raw ? p.inv[b] : 1.f;

    // ---- X X^T of this slice
    if (threadIdx.x == 0) {
      for (int k = 0; k < blocks * 4; ++k) {
        const uint64_t d = smem_desc(smem_u32(X + (k >> 2) * BLOCK_BYTES) + (k & 3) * (UMMA_K * 2), 16, 1024);
        tc_mma(tmem, d, d, idesc_kk, k > 0);
      }
      tc_commit(smem_u32(gram_bar));
    }
    wait(gram_bar, parity);
    if (cluster == 1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[32];
        tmem_ld32(tmem + lanes + half * 64 + h * 32, r);
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = f * f * __uint_as_float(r[j]);
        uint4 o[4];
        pack_row32(v, DT, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(A + half * BLOCK_BYTES + at16(row, h * 4 + i)) = o[i];
      }
      fence_async_smem();
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
    } else {
      // partial sums: row r, 16-byte chunk k at r * 512 + ((k ^ (r & 31)) << 4)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[32];
        tmem_ld32(tmem + lanes + half * 64 + h * 32, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = half * 16 + h * 8 + i;
          *reinterpret_cast<uint4*>(part + row * 512 + ((k ^ (row & 31)) << 4)) =
              make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
      }
      tc_fence_before();
      cluster_sync();  // every CTA's partial sums are there
      tc_fence_after();
      const int r0 = ROWS / (int)cluster * (int)rank, count = ROWS / (int)cluster * 32;
      const uint32_t part0 = smem_u32(part), a0 = smem_u32(A);
      for (int i = threadIdx.x; i < count; i += THREADS) {
        const int r = r0 + (i >> 5), k = i & 31;
        const uint32_t off = part0 + r * 512 + ((k ^ (r & 31)) << 4);
        float4 s = ld_cluster4(mapa(off, 0));
        for (uint32_t c = 1; c < cluster; ++c) {
          const float4 v = ld_cluster4(mapa(off, c));
          s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        const uint32_t lo = pack2(f * f * s.x, f * f * s.y, DT), hi = pack2(f * f * s.z, f * f * s.w, DT);
        // columns 4 k .. 4 k + 3: half of a 16-byte chunk
        const uint32_t to = a0 + (k >> 4) * BLOCK_BYTES + at16(r, (k & 15) >> 1) + (k & 1) * 8;
        for (uint32_t c = 0; c < cluster; ++c) st_cluster2(mapa(to, c), lo, hi);
      }
      asm volatile("fence.proxy.async;" ::: "memory");  // the MMAs of every CTA read A through the async proxy
      cluster_sync();  // A is complete everywhere
      fence_async_smem();
      __syncthreads();
    }

    // ---- B = b A + c A A, over A
    float scale = bb;  // of the product below: B X, or b A X without an A A term
    if (cc != 0.f) {
      scale = 1.f;
      if (threadIdx.x == 0) {
        for (int k = 0; k < 8; ++k) {
          const uint64_t d = smem_desc(smem_u32(A + (k >> 2) * BLOCK_BYTES) + (k & 3) * (UMMA_K * 2), 16, 1024);
          tc_mma(tmem + 128, d, d, idesc_kk, k > 0);
        }
        tc_commit(smem_u32(sq_bar));
      }
      wait(sq_bar, sq_parity);
      sq_parity ^= 1u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[32];
        tmem_ld32(tmem + lanes + 128 + half * 64 + h * 32, r);
        uint4 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = *reinterpret_cast<const uint4*>(A + half * BLOCK_BYTES + at16(row, h * 4 + i));
        float v[32];
        cvt_row32(o, DT, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = cc * __uint_as_float(r[j]) + bb * v[j];
        pack_row32(v, DT, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(A + half * BLOCK_BYTES + at16(row, h * 4 + i)) = o[i];
      }
      fence_async_smem();
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
    }

    // ---- X <- f (a X + B X), 128 columns at a time
    if (threadIdx.x == 0) {
      for (int j = 0; j < chunks; ++j) {
        for (int k = 0; k < 8; ++k) {
          const uint64_t ad = smem_desc(smem_u32(A + (k >> 2) * BLOCK_BYTES) + (k & 3) * (UMMA_K * 2), 16, 1024);
          const uint64_t bd = smem_desc(smem_u32(X + 2 * j * BLOCK_BYTES) + k * (UMMA_K * 128), BLOCK_BYTES, 1024);
          tc_mma(tmem + j * 128, ad, bd, idesc_mn, k > 0);
        }
        tc_commit(smem_u32(&up_bar[j]));
      }
    }
    const bool last = it == p.iters - 1;
    Params e{};  // of the update's epilogue: O = f (scale acc + a X)
    e.M = p.n; e.N = p.m;
    e.d_dtype = DT; e.c_dtype = DT;
    e.C = X;     // present; the values are handed over in registers
    e.c_acc = scale; e.c_in = a;
    const Tile tl{b, 0, 0};
#pragma unroll 1
    for (int j = 0; j < chunks; ++j) {
      const int chunk = (col0 + j * 128 + half * 64) >> 5;  // 32-column chunk of the block
      WPrefetch pf[2];
      if (last) {
        pf[0] = prefetch_w(e, u, tl, q, lane, chunk);
        pf[1] = prefetch_w(e, u, tl, q, lane, chunk + 1);
      }
      wait(&up_bar[j], parity);
      uint8_t* x = X + (2 * j + half) * BLOCK_BYTES;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[32];
        tmem_ld32(tmem + lanes + j * 128 + half * 64 + h * 32, r);
        uint4 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = *reinterpret_cast<const uint4*>(x + at16(row, h * 4 + i));
        if (last) {
          update_chunk(e, u, tl, q, lane, chunk + h, r, o, true, f, part + warp * STAGE_TILE_BYTES, pf[h]);
        } else {
          float v[32];
          cvt_row32(o, DT, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = f * (scale * __uint_as_float(r[i]) + a * v[i]);
          pack_row32(v, DT, o);
#pragma unroll
          for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(x + at16(row, h * 4 + i)) = o[i];
        }
      }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }

  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  if (threadIdx.x == 0 && *abort_flag && p.err != nullptr) atomicOr(p.err, kStatusTimeout);
}

static int cluster_for(int m) {
  int c = 1;
  while (c * MOST_SLICE < m) c *= 2;
  return c;
}

template <int IN_FMT>
static int launch(const CUtensorMap& map, const BParams& p, const UpdateSlots& u, int count, cudaStream_t s) {
  static std::atomic<int> opted[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return (int)cudaErrorInvalidDevice;
  auto kern = ns_block_kernel<IN_FMT>;
  if (!opted[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return (int)e;
    opted[dev].store(1, std::memory_order_release);
  }
  const int cluster = cluster_for(p.m);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(count * cluster));
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
  return a.dtype == kBF16 ? launch<1>(map, p, u, a.count, s) : launch<0>(map, p, u, a.count, s);
}

}  // namespace muon
