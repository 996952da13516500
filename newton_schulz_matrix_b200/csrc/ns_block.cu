// The whole Muon step of small blocks in one launch: n <= 128 rows (the heads of an
// attention projection), up to 4096 columns, 16-bit storage, the standard form.
//
//   M <- mu M + (1 - mu) G,  U = M or (1 - mu) G + mu M
//   X = U / (||U|| + eps)
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
//   U       each warp turns 32 x 32 boxes of its CTA's slice; G and M come by
//           asynchronous copies, half a box ahead, through the memory that X
//           takes later.  U waits in TMEM, in fp32, until the cluster has added
//           up its squares, so G and M are read once although X is rounded only
//           after the norm is known (a pass for the norm and one that stores X
//           read both twice: 52 of the 183 us that the step below then took)
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
// 128 x 2048 take 156 us in two waves of 37 clusters, of which U is about 35 (HBM:
// 26 for G, M and the new M).  Pushing the partial sums to the CTA that adds them
// instead of reading them from there: 159 us, 166 with 16-byte stores to rows.
// Blocks whose rows start anywhere load element by element, whole pieces at a time:
// 64 of 127 x 2047 take 225 us (297 with one load after the other).
//
// Every block that fits takes this launch.  Steps by separate products and here, us
// (bf16 W and G, dense blocks that each are a tensor): 64 of 128 x 2048 317 and 170,
// one 165 and 76; 64 of 128 x 4096 (clusters of eight) 515 and 401, 16 264 and 150,
// 64 of 64 x 4096 384 and 355; 256 of 128 x 512 302 and 121; few rows, padded to 128:
// 512 of 8 x 256 267 and 122, 512 of 16 x 1024 634 and 407, 128 of 32 x 2048 331 and
// 262, 64 of 64 x 640 140 and 60.
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
constexpr int THREADS = 32 * EPI_WARPS + 32;         // and one warp that issues the MMAs
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
  float mu, eps;
  int nesterov;
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
// Up to `count` elements of es bytes, `stride` bytes apart, as bits: the type is
// looked at once, so that all the loads are in flight together.
template <int N>
__device__ __forceinline__ void load_bits(uint32_t (&v)[N], const char* p, long long stride, int count, int es) {
  if (es == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < count ? *reinterpret_cast<const uint32_t*>(p + i * stride) : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < count ? *reinterpret_cast<const uint16_t*>(p + i * stride) : 0u;
  }
}
__device__ __forceinline__ float value_of(uint32_t bits, int dt) {
  if (dt == kFP32) return __uint_as_float(bits);
  return dt == kBF16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half((unsigned short)bits));
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

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void cp_async(uint32_t to, const void* from, int bytes) {
  if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}

// The momentum of one block as its warps see it: 32 x 32 boxes of G and M in W's
// orientation, two halves of 16 rows each.  Lane l takes rows 4 i + l / 8 of a
// half and the 4 columns from 4 (l % 8), i = 0..3.
struct Momentum {
  const char* src;
  float* mom;
  long long ld_g, ld_m;
  int dt, es;
  bool vec, turned;
  uint8_t* ring;   // this warp's 8 KB: half h of M at 2048 h, of G at 4096 + 2048 h
  uint8_t* stage;  // and 4 KB for a box of U
};
struct MBox {
  long long row, col;  // in W's orientation
  int rows, cols;      // that exist
};
__device__ __forceinline__ MBox mbox(const Momentum& t, const BParams& p, int r0, int gc) {
  return t.turned ? MBox{gc, r0, p.m - gc, p.n - r0} : MBox{r0, gc, p.n - r0, p.m - gc};
}
// A half that exists whole, of rows that start on 16 bytes, comes by asynchronous
// copies; others are loaded when they are used.
__device__ __forceinline__ bool copied(const Momentum& t, const MBox& x, int h) {
  return t.vec && x.rows >= h * 16 + 16 && x.cols >= 32;
}
__device__ __forceinline__ void fetch_half(const Momentum& t, const MBox& x, int h, int lane) {
  if (copied(t, x, h)) {
    const int c = 4 * (lane & 7);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = h * 16 + 4 * i + (lane >> 3);
      const uint32_t at = smem_u32(t.ring) + 2048 * h + (32 * i + lane) * 16;
      cp_async(at, t.mom + (x.row + r) * t.ld_m + x.col + c, 16);
      const char* g = t.src + ((x.row + r) * t.ld_g + x.col + c) * t.es;
      if (t.es == 4) cp_async(at + 4096, g, 16);
      else cp_async(smem_u32(t.ring) + 4096 + 2048 * h + (32 * i + lane) * 8, g, 8);
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// M <- mu M + (1 - mu) G of four elements: ms and the sum of squares on, U to the staging box.
__device__ __forceinline__ void momentum4(const BParams& p, const float (&gs)[4], float (&ms)[4], float& ssq, uint8_t* to) {
  float us[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    ms[e] = p.mu * ms[e] + (1.f - p.mu) * gs[e];
    us[e] = p.nesterov ? (1.f - p.mu) * gs[e] + p.mu * ms[e] : ms[e];
    ssq += us[e] * us[e];
  }
  *reinterpret_cast<float4*>(to) = make_float4(us[0], us[1], us[2], us[3]);
}
// The momentum of a half, stored; U left in the staging box (row r, 16-byte chunk k
// at r * 128 + ((k ^ (r & 7)) << 4)).  Returns this lane's sum of squares.  A lane
// reads only what it copied itself, so no other lane is waited for.
__device__ __forceinline__ float momentum_half(const Momentum& t, const MBox& x, const BParams& p, int h, int lane) {
  const int c = 4 * (lane & 7);
  float ssq = 0.f;
  auto stage = [&](int r) { return t.stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4); };
  asm volatile("cp.async.wait_group 1;" ::: "memory");
  if (copied(t, x, h)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = h * 16 + 4 * i + (lane >> 3);
      const uint8_t* from = t.ring + 2048 * h + (32 * i + lane) * 16;
      const float4 m = *reinterpret_cast<const float4*>(from);
      float gs[4], ms[4] = {m.x, m.y, m.z, m.w};
      if (t.es == 4) {
        const float4 g = *reinterpret_cast<const float4*>(from + 4096);
        gs[0] = g.x; gs[1] = g.y; gs[2] = g.z; gs[3] = g.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(t.ring + 4096 + 2048 * h + (32 * i + lane) * 8);
        const float2 lo = t.dt == kBF16 ? unpack2<1>(w.x) : unpack2<0>(w.x);
        const float2 hi = t.dt == kBF16 ? unpack2<1>(w.y) : unpack2<0>(w.y);
        gs[0] = lo.x; gs[1] = lo.y; gs[2] = hi.x; gs[3] = hi.y;
      }
      momentum4(p, gs, ms, ssq, stage(r));
      *reinterpret_cast<float4*>(t.mom + (x.row + r) * t.ld_m + x.col + c) = make_float4(ms[0], ms[1], ms[2], ms[3]);
    }
    return ssq;
  }
#pragma unroll 1
  for (int k = 0; k < 4; k += 2) {
    // eight rows: every load before the first store
    uint32_t gb[2][4], mb[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = h * 16 + 4 * (k + i) + (lane >> 3);
      const int valid = r < x.rows ? min(x.cols - c, 4) : 0;
      load_bits<4>(gb[i], t.src + ((x.row + r) * t.ld_g + x.col + c) * t.es, t.es, valid, t.es);
      load_bits<4>(mb[i], reinterpret_cast<const char*>(t.mom + (x.row + r) * t.ld_m + x.col + c), 4, valid, 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = h * 16 + 4 * (k + i) + (lane >> 3);
      float* at = t.mom + (x.row + r) * t.ld_m + x.col + c;
      float gs[4], ms[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        gs[e] = value_of(gb[i][e], t.dt);
        ms[e] = __uint_as_float(mb[i][e]);
      }
      momentum4(p, gs, ms, ssq, stage(r));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r < x.rows && c + e < x.cols) at[e] = ms[e];
    }
  }
  return ssq;
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
ns_block_kernel(const __grid_constant__ BParams p, const __grid_constant__ PackSlots g,
                const __grid_constant__ UpdateSlots u) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* X = smem;
  uint8_t* A = X + X_BYTES;
  uint8_t* part = A + GRAM_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(part + PART_BYTES);
  uint64_t* gram_bar = bars;       // X X^T
  uint64_t* sq_bar = bars + 1;     // A A
  uint64_t* up_bar = bars + 2;     // [4] B X, 128 columns each
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool issuer = warp == EPI_WARPS;     // the warp that issues the MMAs
  const int q = warp & 3, quarter = warp >> 2;  // TMEM lane quarter; which 32 of 128 columns
  const int row = q * 32 + lane;
  const uint32_t rank = cluster_rank();
  const int b = blockIdx.x / CL;
  const int col0 = (int)rank * p.slice;
  const int blocks = p.slice / 64, chunks = p.slice / 128;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 6; ++i) mbar_init(smem_u32(&bars[i]), 1);
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

  float inv;  // 1 / (||U|| + eps)
  const unsigned kind = u.kind[b];
  const int boxes = ((p.n + 31) >> 5) * (p.slice / 32);

  // ---- M <- mu M + (1 - mu) G, X = U / (||U|| + eps) (or U, for a chain that takes
  // the norm as f).  U waits in TMEM, in fp32, for the norm: 128 rows x 512 columns
  // are exactly all of it, and the chain has not begun.
  {
    double* sums = reinterpret_cast<double*>(A);  // per warp, then this CTA's
    const int width = p.slice / 4;                // columns of this warp
    if (!issuer) {
      const unsigned gk = g.kind[b];
      const Momentum t{reinterpret_cast<const char*>(g.src[b]), g.mom[b], g.ld_src[b], g.ld_mom[b], (int)gk & 3,
                       (gk & 3) == kFP32 ? 4 : 2, (gk & 4u) != 0, (kind & 1u) != 0, X + warp * 8192, part + warp * 4096};
      const uint8_t* S = t.stage;
      const int first = quarter * width, past = first + width;
      float ssq = 0.f;
      MBox now = mbox(t, p, q * 32, col0 + first);
      fetch_half(t, now, 0, lane);
      fetch_half(t, now, 1, lane);
#pragma unroll 1
      for (int c0 = first; c0 < past; c0 += 32) {
        // the next box's halves are on their way as soon as this one's have been read
        MBox next = mbox(t, p, q * 32, col0 + c0 + 32);
        if (c0 + 32 >= past) next.rows = 0;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          ssq += momentum_half(t, now, p, h, lane);
          fetch_half(t, next, h, lane);
        }
        now = next;
        __syncwarp();
        uint32_t v[32];
        if (t.turned) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = *reinterpret_cast<const uint32_t*>(S + i * 128 + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(S + lane * 128 + ((i ^ (lane & 7)) << 4));
            v[4 * i] = w.x; v[4 * i + 1] = w.y; v[4 * i + 2] = w.z; v[4 * i + 3] = w.w;
          }
        }
        tmem_st32(tmem + lanes + c0, v);
        __syncwarp();
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ssq += __shfl_down_sync(0xffffffffu, ssq, o);
      if (lane == 0) sums[warp] = (double)ssq;
      // W is read at the end: bring it into L2 under the iterations
      for (int k = warp; k < boxes; k += EPI_WARPS) {
        Box x;
        locate(x, p, u, b, col0, k);
        const int es = ((kind >> 1) & 3) == kFP32 ? 4 : 2;
        if (lane < x.rows && x.cols > 0)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(x.base + lane * x.ld * es));
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      double t = 0.0;
      for (int i = 0; i < EPI_WARPS; ++i) t += sums[i];
      sums[EPI_WARPS] = t;
    }
    if constexpr (CL > 1) cluster_sync();
    else __syncthreads();
    double total = 0.0;
#pragma unroll
    for (int c = 0; c < CL; ++c)
      total += CL > 1 ? ld_cluster_f64(mapa(smem_u32(sums + EPI_WARPS), c)) : sums[EPI_WARPS];
    inv = (float)(1.0 / (sqrt(total) + (double)p.eps));
    if (!issuer) {
      const float scale = p.raw ? 1.f : inv;
#pragma unroll 1
      for (int c0 = quarter * width; c0 < (quarter + 1) * width; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(tmem + lanes + c0, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack2<IN_FMT>(scale * __uint_as_float(r[8 * i + 2 * k]), scale * __uint_as_float(r[8 * i + 2 * k + 1]));
          *reinterpret_cast<uint4*>(X + (c0 >> 6) * BLOCK_BYTES + at16(row, ((c0 & 63) >> 3) + i)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_async_smem();
      tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
  }

  uint32_t sq_parity = 0;  // of the next A A: iterations without that term skip it
  for (int it = 0; it < p.iters; ++it) {
    const uint32_t parity = it & 1;
    const float a = p.coeffs[3 * it], bb = p.coeffs[3 * it + 1], cc = p.coeffs[3 * it + 2];
    const float f = it == 0 && p.raw ? inv : 1.f;

    // ---- A = f^2 X X^T
    if (issuer) {
      if (lane == 0) {
        fence_async_smem();
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
      if (!(kind & 8u)) {
        // rows of W that start anywhere: a lane per column, sixteen rows in flight
#pragma unroll 1
        for (int r0 = 0; r0 < now.rows; r0 += 16) {
          uint32_t v[16];
          load_bits<16>(v, now.base + (r0 * now.ld + lane) * es, now.ld * es, lane < now.cols ? now.rows - r0 : 0, es);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int r = r0 + e;
            if (r >= now.rows || lane >= now.cols) continue;
            const uint16_t* at = reinterpret_cast<const uint16_t*>(
                (kind & 1u) ? S + sw64(r, lane >> 3) : x + at16(now.r0 + r, ch + (lane >> 3))) + (lane & 7);
            const float o = load_any(at, 0, IN_FMT ? kBF16 : kFP16);
            bad |= !isfinite(o);
            store_any(now.base + r * now.ld * es, lane, wdt, weight_update(value_of(v[e], wdt), o, u.decay, u.step));
          }
        }
        continue;
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
        update8(now.base + (r * now.ld + c) * es, wdt, o, valid, valid == 8, u.decay, u.step,
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
static int launch(const BParams& p, const PackSlots& g, const UpdateSlots& u, int count, cudaStream_t s) {
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
  return (int)cudaLaunchKernelEx(&cfg, kern, p, g, u);
}

}  // namespace blk
}  // namespace tc

bool ns_block_ok(int n, int m, int iters) {
  return n <= tc::blk::ROWS && m <= 8 * tc::blk::MOST_SLICE && iters <= kBlockChainMaxIters;
}

int launch_ns_block(const BlockChainArgs& a, const PackSlots& g, const UpdateSlots& u, cudaStream_t s) {
  using namespace tc;
  using namespace tc::blk;
  BParams p{};
  p.n = a.n; p.m = a.m; p.iters = a.iters; p.raw = a.raw;
  const int cluster = cluster_for(a.m);
  p.slice = ((a.m + cluster - 1) / cluster + 127) / 128 * 128;
  p.mu = a.mu; p.eps = a.eps; p.nesterov = a.nesterov; p.err = a.err;
  p.timeout_ns = wait_timeout_ns();
  for (int i = 0; i < 3 * a.iters; ++i) p.coeffs[i] = a.coeffs[i];
  const bool bf = a.dtype == kBF16;
  switch (cluster) {
    case 1: return bf ? launch<1, 1>(p, g, u, a.count, s) : launch<0, 1>(p, g, u, a.count, s);
    case 2: return bf ? launch<1, 2>(p, g, u, a.count, s) : launch<0, 2>(p, g, u, a.count, s);
    case 4: return bf ? launch<1, 4>(p, g, u, a.count, s) : launch<0, 4>(p, g, u, a.count, s);
    default: return bf ? launch<1, 8>(p, g, u, a.count, s) : launch<0, 8>(p, g, u, a.count, s);
  }
}

}  // namespace muon
