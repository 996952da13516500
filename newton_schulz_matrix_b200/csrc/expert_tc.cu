// The three products of an expert layer on the tensor cores (tcgen05, TMEM,
// TMA), bf16 and fp16 operands, fp32 accumulators.
//
//   forward      Y[p] = W[e] X[p]          D = W[e] (256 features) x X^T (tokens)
//   input grad   dX[p] = W[e]^T dY[p]      D = W[e]^T (256 features) x dY^T (tokens)
//   weight grad  dW[e] = dY_e^T X_e        D = dY_e^T (256 rows) x X_e (256 columns)
//
// A pair of CTAs owns one output tile of 256 rows (cta_group::2: 128 TMEM lanes
// each) and up to 256 columns, as in gemm_tc2.cu (or one CTA a tile of 128 x 128,
// where there are few tokens an expert); what differs is where tiles come from
// and how their ragged edges are handled.
//
// Tiles.  An expert's rows are a segment [lo, hi) that only the device knows.
// Every CTA reads the offsets at its start, clamps them to the matrix, and
// keeps the segments and a running count of tiles in shared memory; tile t of
// the launch then belongs to the expert whose range holds it, and pair k takes
// tiles k, k + pairs, ...  No count reaches the host and no list is built in
// global memory.
//
// Forward and input gradient put the weights on the 256-row side (A) and the
// tokens on the column side (B): the MMA's column count is a run-time value
// (a multiple of 32), so an expert with 3 tokens runs N = 32 and one with 300
// runs two tiles of 160, where tokens on the row side would cost 256 rows each.
// With few tokens an expert the launch streams the weights once and is bound by
// HBM; with many it is bound by the tensor cores.  The tile comes out
// transposed (a TMEM lane is a feature); each 32 x 32 box is turned in shared
// memory by ldmatrix.trans / stmatrix and stored by TMA, or row by row where
// the expert's tokens end inside the box.
//
// A TMA store clips in whole 16 bytes: the last box of a row whose width is no
// multiple of that would write up to 7 elements behind the row, into whatever a
// result with a larger pitch has there.  Such boxes are stored element by element.
//
// The weight gradient's contraction runs over the segment's tokens, so its last
// k-block may end inside the next expert's rows.  MMAs cover whole groups of 16
// tokens; the rows of the last group beyond the segment are zeroed in shared
// memory in both operands (0 * NaN is NaN), after the TMA load and before the
// MMA: that block's load reports to a barrier of its own CTA, on which one more
// warp waits, and once that warp of both CTAs has zeroed its rows and arrived,
// the leader's "full" barrier opens.  The producers meanwhile go on to the next
// tiles (waiting for that load in the producer itself emptied the ring at every
// tile and took a tenth longer).  49152 rows over 64 experts of 1408 x 2048, bf16:
// forward 254, input gradient 244, weight gradient 291 us each after a rest, at the full
// clock of 1965 MHz; 295, 281 and 330 us over seconds under the power cap, which
// leaves 1.39 to 1.53 GHz (a dense library product of the forward's size there: 238).
//
// fp32 weight gradients.  The tensor cores truncate when they add to an fp32
// accumulator, a bias that grows with the length of the sum (relative error of one
// sum 1.3e-6 at 1024 tokens, 4.9e-6 at 4096, 1.9e-5 at 16384).  Where the result is
// stored in fp32 a tile is therefore summed in runs of 512 tokens, each in a
// fresh accumulator (two in TMEM), and the epilogue warps add the runs in
// registers with round-to-nearest, 128 sums a thread, while the next run's MMAs
// go on: 6.5e-7 in fp16 and 4.8e-7 in bf16 at every length to 16384 (fp32 operands on
// the CUDA cores 5.7e-7 at 1024 tokens, 2.3e-6 at 16384), at 277 us where the 16-bit
// result takes 250 (8192 rows, 8 experts of 2048 x 7168, under the power cap).
// Sixteen epilogue warps of 64 sums leave room for five stages only, and took 15 %
// longer.
//
// Waits are bounded as in the other product kernels.
#include <algorithm>
#include <atomic>

#include "expert.h"
#include "tc_common.cuh"

namespace muon {
namespace tc {
namespace expk {

constexpr int NSTAGES = 6;
constexpr int EPI = NUM_EPI_WARPS;
// producer, MMA, epilogue and, for weight gradients, the zeroing warp
constexpr int threads_of(bool wg) { return 64 + 32 * EPI + (wg ? 32 : 0); }
constexpr double PACK_FLOPS = 2e8;                // least product whose operands are copied into aligned rows
constexpr int SINGLE_TOKENS = 48;                 // tokens per expert up to which single CTAs run
constexpr int FOLD_KB = 8;                        // k-blocks of a run of an fp32 weight gradient: 512 tokens
constexpr int HALF_BYTES = 128 * BK * 2;          // one operand of a stage in one CTA: 16 KB
constexpr int STAGE2 = 2 * HALF_BYTES;
constexpr int BOX_BYTES = STAGE_TILE_BYTES;       // one staging box per epilogue warp
constexpr int TABLE_INTS = 3 * kMaxExperts + 8;   // segment starts, lengths, first tiles
constexpr int BAR_BYTES = 256;
constexpr int SMEM = NSTAGES * STAGE2 + EPI * BOX_BYTES + TABLE_INTS * 4 + BAR_BYTES + 1024;
static_assert(SMEM <= 232448, "shared memory of one CTA");
static_assert((3 * NSTAGES + 5) * 8 + 8 <= BAR_BYTES, "barrier area");

struct EParams {
  const int* offsets;
  int experts, rows;
  int F;                 // rows of D: outer (forward, weight grad) or inner (input grad)
  int C;                 // columns of D (weight grad): inner
  int K;                 // contraction of forward (inner) and input grad (outer)
  int tiles_f, tiles_c;
  void* D; long long ldd, stride_d;
  int d_vec;             // 1: D's rows start on 16 bytes (TMA and 16-byte stores); 0: element by element
  int accumulate;
  int* err;
  long long timeout_ns;
};

// Tensor maps: the weights or dY (a), the tokens in boxes of 16, 32, 64 and
// 128 rows or X (b[0]), the output (d).
struct EMaps {
  CUtensorMap a, b[4], d;
};

__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster, int x, int y,
                                              int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void mma2(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                     uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// The segments and tiles of a launch, in shared memory.
struct Table {
  int* lo;      // [experts] first row
  int* len;     // [experts] rows
  int* first;   // [experts + 1] tiles of the experts before
};
// A role's place in the table: it meets tiles in increasing order.
struct Cursor {
  int e = 0;
};
struct ETile {
  int e, lo, len;   // the expert and its segment
  int f;            // 256-row tile of D
  int c;            // weight grad: 256-column tile of D
  int t0, tokens;   // forward, input grad: first token (of the segment) and count
};
// Rows of D per tile and most tokens per tile: of a pair of CTAs, or of one.
__host__ __device__ constexpr int tile_rows(bool pair) { return pair ? 256 : 128; }
__host__ __device__ constexpr int tile_tokens(bool pair) { return pair ? 256 : 128; }
template <bool PAIR>
__device__ __forceinline__ int token_tiles(int len) { return (len + tile_tokens(PAIR) - 1) / tile_tokens(PAIR); }

template <int KIND, bool PAIR>
__device__ __forceinline__ ETile find_tile(const EParams& p, const Table& tb, Cursor& cur, int t) {
  while (t >= tb.first[cur.e + 1]) ++cur.e;
  ETile r;
  r.e = cur.e;
  r.lo = tb.lo[r.e];
  r.len = tb.len[r.e];
  const int q = t - tb.first[r.e];
  if (KIND == kWeightGrad) {
    r.f = q / p.tiles_c;
    r.c = q - r.f * p.tiles_c;
    r.t0 = 0;
    r.tokens = r.len;
  } else {
    // the token tiles of one feature tile follow each other: they share its weights
    const int nt = token_tiles<PAIR>(r.len);
    r.f = q / nt;
    r.c = 0;
    // equal tiles, in whole groups of 32 tokens (the MMA's column granularity)
    const int size = ((r.len + nt - 1) / nt + 31) & ~31;
    r.t0 = (q - r.f * nt) * size;
    r.tokens = min(size, r.len - r.t0);
  }
  return r;
}

template <int KIND, int IN_FMT, bool OUT32, bool PAIR>
__global__ void __launch_bounds__(threads_of(KIND == kWeightGrad), 1)
expert_kernel(const __grid_constant__ EMaps maps, const __grid_constant__ EParams p) {
  static_assert(KIND == kWeightGrad || !OUT32, "fp32 results: weight gradients only");
  static_assert(KIND != kWeightGrad || PAIR, "single CTAs: forward and input gradient only");
  constexpr int CTAS = PAIR ? 2 : 1;
  constexpr bool WG = KIND == kWeightGrad;
  constexpr bool A_MN = KIND != kForward;   // A is read along its columns
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + NSTAGES * STAGE2;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + EPI * BOX_BYTES);
  uint64_t* full_bar = bars;                     // [NSTAGES] (used in the leader)
  uint64_t* empty_bar = bars + NSTAGES;          // [NSTAGES] (both CTAs)
  uint64_t* tfull_bar = bars + 2 * NSTAGES;      // [2]       (both CTAs)
  uint64_t* tempty_bar = bars + 2 * NSTAGES + 2; // [2]       (used in the leader)
  uint64_t* drain_bar = bars + 2 * NSTAGES + 4;  // [1]
  uint64_t* tail_bar = bars + 2 * NSTAGES + 5;   // [NSTAGES] (both CTAs; weight grad)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * NSTAGES + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* table = reinterpret_cast<int*>(staging + EPI * BOX_BYTES + BAR_BYTES);
  const Table tb{table, table + kMaxExperts, table + 2 * kMaxExperts};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0;  // 0 = leader, 1 = peer
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NSTAGES; ++s) {
      mbar_init(smem_u32(&full_bar[s]), WG ? 2 : 1);  // weight grad: both CTAs arrive
      mbar_init(smem_u32(&empty_bar[s]), 1);
      mbar_init(smem_u32(&tail_bar[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull_bar[a]), 1);
      mbar_init(smem_u32(&tempty_bar[a]), CTAS * EPI);
    }
    mbar_init(smem_u32(drain_bar), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.d)) : "memory");
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(TMEM_COLS)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(TMEM_COLS)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  if (warp == 2) {
    // segments and running tile counts, 32 experts at a time
    int tiles = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + lane;
      int n = 0;
      if (e < p.experts) {
        const int lo = min(max(p.offsets[e], 0), p.rows);
        const int len = min(max(p.offsets[e + 1], lo), p.rows) - lo;
        tb.lo[e] = lo;
        tb.len[e] = len;
        if (WG) n = p.accumulate && len == 0 ? 0 : p.tiles_f * p.tiles_c;
        else n = token_tiles<PAIR>(len) * p.tiles_f;
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < p.experts) tb.first[e + 1] = tiles + incl;
      tiles += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) tb.first[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = tb.first[p.experts];
  const int pair = (int)blockIdx.x / CTAS, pairs = (int)gridDim.x / CTAS;
  const uint32_t leader_full = PAIR ? mapa(smem_u32(full_bar), 0) : smem_u32(full_bar);
  const uint32_t leader_tempty = PAIR ? mapa(smem_u32(tempty_bar), 0) : 0;
  auto load = [](uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    if constexpr (PAIR) tma_load_pair(dst, map, bar, x, y, z);
    else tma_load_3d(dst, map, bar, x, y, z);
  };
  // arrives, once the MMAs so far are done, on this barrier of the tile's CTAs
  auto commit = [](uint64_t* bar) {
    if constexpr (PAIR) commit_pair(smem_u32(bar), 0x3);
    else tc_commit(smem_u32(bar));
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- producers (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      Cursor cur;
      for (int t = pair; t < total && ok; t += pairs) {
        const ETile tl = find_tile<KIND, PAIR>(p, tb, cur, t);
        const int f0 = tl.f * tile_rows(PAIR) + (int)rank * 128;  // this CTA's rows of D
        if (!WG) {
          const int half = ((tl.tokens + 31) & ~31) / CTAS;  // this CTA's tokens
          const int size = half > 64 ? 3 : half > 32 ? 2 : half > 16 ? 1 : 0;
          const CUtensorMap* mb = &maps.b[size];
          const uint32_t b_bytes = (16u << size) * 128u;
          const int row0 = tl.lo + tl.t0 + (int)rank * half;
          const int num_kb = (p.K + BK - 1) / BK;
          for (int kb = 0; kb < num_kb; ++kb) {
            if (!mbar_wait(smem_u32(&empty_bar[stage]), phase ^ 1u, abort_flag, p.timeout_ns)) { ok = false; break; }
            if (leader) mbar_expect_tx(smem_u32(&full_bar[stage]), CTAS * (HALF_BYTES + b_bytes));
            const uint32_t fb = leader_full + stage * 8;
            const uint32_t sa = smem_u32(smem + stage * STAGE2);
            if (A_MN) {
              load(sa, &maps.a, fb, f0, kb * BK, tl.e);
              load(sa + BK * 128, &maps.a, fb, f0 + 64, kb * BK, tl.e);
            } else {
              load(sa, &maps.a, fb, kb * BK, f0, tl.e);
            }
            load(sa + HALF_BYTES, mb, fb, kb * BK, row0, 0);
            if (++stage == NSTAGES) { stage = 0; phase ^= 1u; }
          }
        } else {
          const bool narrow = p.C - tl.c * 256 <= 128;
          const int c0 = tl.c * 256 + (int)rank * (narrow ? 64 : 128);  // this CTA's columns of D
          const uint32_t bytes = HALF_BYTES + (narrow ? HALF_BYTES / 2 : HALF_BYTES);
          const int num_kb = (tl.len + BK - 1) / BK;
          const int tail_kb = (tl.len & 15) ? num_kb - 1 : num_kb;  // the k-block that the zeroing warp finishes
          for (int kb = 0; kb < num_kb; ++kb) {
            if (!mbar_wait(smem_u32(&empty_bar[stage]), phase ^ 1u, abort_flag, p.timeout_ns)) { ok = false; break; }
            const uint32_t sa = smem_u32(smem + stage * STAGE2);
            const int row = tl.lo + kb * BK;
            if (kb != tail_kb) {
              const uint32_t fb = leader_full + stage * 8;
              if (leader) mbar_expect_tx(smem_u32(&full_bar[stage]), 2 * bytes);
              else remote_arrive_cta(fb);
              tma_load_pair(sa, &maps.a, fb, f0, row, 0);
              tma_load_pair(sa + BK * 128, &maps.a, fb, f0 + 64, row, 0);
              tma_load_pair(sa + HALF_BYTES, &maps.b[0], fb, c0, row, 0);
              if (!narrow) tma_load_pair(sa + HALF_BYTES + BK * 128, &maps.b[0], fb, c0 + 64, row, 0);
            } else {
              const uint32_t tbar = smem_u32(&tail_bar[stage]);
              mbar_expect_tx(tbar, bytes);
              tma_load_3d(sa, &maps.a, tbar, f0, row, 0);
              tma_load_3d(sa + BK * 128, &maps.a, tbar, f0 + 64, row, 0);
              tma_load_3d(sa + HALF_BYTES, &maps.b[0], tbar, c0, row, 0);
              if (!narrow) tma_load_3d(sa + HALF_BYTES + BK * 128, &maps.b[0], tbar, c0 + 64, row, 0);
            }
            if (++stage == NSTAGES) { stage = 0; phase ^= 1u; }
          }
        }
      }
      // no drain needed where all went well: the leader's MMAs consume every
      // issued stage, and the final cluster barrier keeps this CTA resident
      // until then.  After an abort, stages may be on their way that nothing
      // waits for: copies land within microseconds, so both CTAs stay 1 ms.
      if (!ok) {
        const uint64_t t0 = global_timer();
        for (uint32_t i = 0; i < (1u << 24) && global_timer() - t0 < 1000000ull; ++i) {
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (leader only)
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;  // accumulators begun
      bool ok = true;
      Cursor cur;
      for (int t = pair; t < total && ok; t += pairs) {
        const ETile tl = find_tile<KIND, PAIR>(p, tb, cur, t);
        const int N = WG ? (p.C - tl.c * 256 <= 128 ? 128 : 256) : (tl.tokens + 31) & ~31;
        const uint32_t idesc = make_idesc(IN_FMT, WG ? 1 : 0, tile_rows(PAIR), N) | (A_MN ? 1u << 15 : 0u);
        const int K = WG ? tl.len : p.K;
        const int num_kb = (K + BK - 1) / BK;
        const int run = OUT32 ? FOLD_KB : num_kb;  // k-blocks per accumulator
        int kb = 0;
        do {
          const int acc = it & 1;
          const uint32_t aph = (uint32_t)(it >> 1) & 1u;
          ++it;
          if (!mbar_wait(smem_u32(&tempty_bar[acc]), aph ^ 1u, abort_flag, p.timeout_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
          const int first = kb, end = min(num_kb, kb + run);
          for (; kb < end; ++kb) {
            const bool got = WG ? mbar_wait_cluster(smem_u32(&full_bar[stage]), phase, abort_flag, p.timeout_ns)
                                : mbar_wait(smem_u32(&full_bar[stage]), phase, abort_flag, p.timeout_ns);
            if (!got) { ok = false; break; }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * STAGE2);
            const uint32_t sb = sa + HALF_BYTES;
            // groups of 16 that hold a token (weight grad); elsewhere TMA zero-fills the ends of K
            const int steps = WG ? min(BK / UMMA_K, (K - kb * BK + UMMA_K - 1) / UMMA_K) : BK / UMMA_K;
#pragma unroll
            for (int k = 0; k < BK / UMMA_K; ++k) {
              if (k >= steps) break;
              const uint64_t ad = A_MN ? smem_desc(sa + k * (UMMA_K * 128), BK * 128, 1024)
                                       : smem_desc(sa + k * (UMMA_K * 2), 16, 1024);
              const uint64_t bd = WG ? smem_desc(sb + k * (UMMA_K * 128), BK * 128, 1024)
                                     : smem_desc(sb + k * (UMMA_K * 2), 16, 1024);
              if constexpr (PAIR) mma2(d_tmem, ad, bd, idesc, kb > first || k > 0);
              else tc_mma(d_tmem, ad, bd, idesc, kb > first || k > 0);
            }
            commit(&empty_bar[stage]);  // stage free
            if (++stage == NSTAGES) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          commit(&tfull_bar[acc]);      // accumulator ready
        } while (kb < num_kb);
      }
      if constexpr (PAIR) commit_pair(smem_u32(drain_bar), 0x1);
      else tc_commit(smem_u32(drain_bar));
      volatile int never = 0;
      mbar_wait(smem_u32(drain_bar), 0, &never, p.timeout_ns);
    }
  } else if (WG && warp == 2 + EPI) {
    // ---------------------------------------------------------------- zeroing of the segments' ends (both CTAs)
    int stage = 0;
    uint32_t seen = 0;  // per stage: parity of its next tail load
    Cursor cur;
    for (int t = pair; t < total; t += pairs) {
      const ETile tl = find_tile<KIND, PAIR>(p, tb, cur, t);
      const int num_kb = (tl.len + BK - 1) / BK;
      if (tl.len & 15) {
        const int s = (stage + num_kb - 1) % NSTAGES;
        int ok = 1;
        if (lane == 0) ok = mbar_wait(smem_u32(&tail_bar[s]), (seen >> s) & 1u, abort_flag, p.timeout_ns);
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        __syncwarp();
        seen ^= 1u << s;
        // rows [rem, rem rounded up to 16) of the four 64-column boxes: 128 bytes
        // each, so the 32 lanes clear one row of all four per step
        uint8_t* sm = smem + s * STAGE2 + (lane >> 3) * (BK * 128) + (lane & 7) * 16;
        const int rem = tl.len & (BK - 1), upto = (rem + 15) & ~15;
        for (int r = rem; r < upto; ++r) *reinterpret_cast<uint4*>(sm + r * 128) = make_uint4(0, 0, 0, 0);
        fence_async_smem();  // the MMA reads these rows through the async proxy
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(smem_u32(&full_bar[s]));
          else remote_arrive(leader_full + s * 8);
        }
      }
      stage = (stage + num_kb) % NSTAGES;
    }
  } else if (OUT32) {
    // ---------------------------------------------------------------- fp32 epilogue (both CTAs): runs added in registers
    const int q = warp & 3;         // TMEM lane quarter
    constexpr int COLS = 128;       // columns of a warp
    const int c0 = ((warp - 2) >> 2) * COLS;
    uint8_t* S = staging + (warp - 2) * BOX_BYTES;
    const uint32_t s0 = smem_u32(S);
    int it = 0;
    int ok = 1;
    Cursor cur;
    for (int t = pair; t < total && ok; t += pairs) {
      const ETile tl = find_tile<KIND, PAIR>(p, tb, cur, t);
      const int fi = tl.f * 256 + (int)rank * 128 + q * 32;  // first row of D of this warp
      const int gj = tl.c * 256 + c0;
      const bool mine = fi < p.F && gj < p.C;
      const int runs = max(1, (tl.len + FOLD_KB * BK - 1) / (FOLD_KB * BK));
      float sum[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) sum[j] = 0.f;
      for (int run = 0; run < runs; ++run, ++it) {
        const int acc = it & 1;
        const uint32_t aph = (uint32_t)(it >> 1) & 1u;
        if (lane == 0) ok = mbar_wait(smem_u32(&tfull_bar[acc]), aph, abort_flag, p.timeout_ns);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        tc_fence_after();
        if (mine && tl.len > 0) {
          const uint32_t tbase = tmem_base + (uint32_t)(acc * BN + c0) + ((uint32_t)(q * 32) << 16);
#pragma unroll
          for (int h = 0; h < COLS / 16; ++h) {
            uint32_t r[16];
            tmem_ld16(tbase + h * 16, r);
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[h * 16 + j] += __uint_as_float(r[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(smem_u32(&tempty_bar[acc]));
          else remote_arrive_cta(leader_tempty + acc * 8);
        }
      }
      if (!ok || !mine) continue;
      // boxes of 16 columns
#pragma unroll
      for (int h = 0; h < COLS / 16; ++h) {
        if (gj + h * 16 >= p.C) break;
        if (lane == 0) bulk_wait_read0();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float4*>(S + sw64(lane, k)) =
              make_float4(sum[h * 16 + k * 4], sum[h * 16 + k * 4 + 1], sum[h * 16 + k * 4 + 2], sum[h * 16 + k * 4 + 3]);
        if (!p.d_vec || ((p.C & 3) && gj + h * 16 + 16 > p.C)) {
          __syncwarp();
          const int col = gj + h * 16 + (lane & 15);
          float* d = reinterpret_cast<float*>(p.D) + tl.e * p.stride_d + col;
          for (int r = lane >> 4; r < min(32, p.F - fi); r += 2) {
            if (col >= p.C) continue;
            const float v = *reinterpret_cast<const float*>(S + sw64(r, (lane & 15) >> 2) + (lane & 3) * 4);
            float* at = d + (fi + r) * p.ldd;
            *at = p.accumulate ? *at + v : v;
          }
          continue;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (p.accumulate) tma_add_3d(&maps.d, s0, gj + h * 16, fi, tl.e);
          else tma_store_3d(&maps.d, s0, gj + h * 16, fi, tl.e);
          bulk_commit();
        }
      }
    }
    __syncwarp();
    if (lane == 0) bulk_wait_all0();  // this warp's output stores have completed
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    const int q = warp & 3;            // TMEM lane quarter
    const int half = (warp - 2) >> 2;  // even or odd 32-column chunks
    uint8_t* S = staging + (warp - 2) * BOX_BYTES;
    const uint32_t s0 = smem_u32(S);
    int it = 0;
    Cursor cur;
    for (int t = pair; t < total; t += pairs, ++it) {
      const ETile tl = find_tile<KIND, PAIR>(p, tb, cur, t);
      const int acc = it & 1;
      const uint32_t aph = (uint32_t)(it >> 1) & 1u;
      int ok = 1;
      if (lane == 0) ok = mbar_wait(smem_u32(&tfull_bar[acc]), aph, abort_flag, p.timeout_ns);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (uint32_t)(acc * BN) + ((uint32_t)(q * 32) << 16);
      const int fi = tl.f * tile_rows(PAIR) + (int)rank * 128 + q * 32;  // first row of D of this warp
      const int cols = WG ? min(256, p.C - tl.c * 256) : tl.tokens;
      const int chunks = fi < p.F ? (cols + 31) >> 5 : 0;
      bool released = false;
      for (int c = half; c < chunks; c += 2) {
        uint32_t r[32];
        tmem_ld32(tbase + (uint32_t)(c * 32), r);
        if (c + 2 >= chunks) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (leader) mbar_arrive(smem_u32(&tempty_bar[acc]));
            else remote_arrive_cta(leader_tempty + acc * 8);
          }
          released = true;
        }
        if (WG && tl.len == 0) {  // no MMA wrote the accumulator: an expert without rows
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0;
        }
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        uint4 dq[4];
        pack_row32(v, IN_FMT ? kBF16 : kFP16, dq);
        if (lane == 0) bulk_wait_read0();  // the box is free once the previous store has read it
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(S + sw64(lane, k)) = dq[k];
        if (WG && (!p.d_vec || ((p.C & 7) && tl.c * 256 + c * 32 + 32 > p.C))) {
          __syncwarp();
          const int col = tl.c * 256 + c * 32 + lane;
          uint16_t* d = reinterpret_cast<uint16_t*>(p.D) + tl.e * p.stride_d + col;
          for (int k = 0; k < min(32, p.F - fi); ++k)
            if (col < p.C) d[(fi + k) * p.ldd] = *reinterpret_cast<const uint16_t*>(S + sw64(k, lane >> 3) + (lane & 7) * 2);
        } else if (WG) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&maps.d, s0, tl.c * 256 + c * 32, fi, tl.e);
            bulk_commit();
          }
        } else {
          // rows of the box are features: turn it in place, then its rows are tokens
          __syncwarp();
          uint32_t m[4][4];
#pragma unroll
          for (int g = 0; g < 4; ++g)
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(m[g][0]), "=r"(m[g][1]), "=r"(m[g][2]), "=r"(m[g][3])
                         : "r"(s0 + sw64(lane, g))
                         : "memory");
          __syncwarp();
#pragma unroll
          for (int g = 0; g < 4; ++g)
            asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                             s0 + sw64(g * 8 + (lane & 7), lane >> 3)),
                         "r"(m[g][0]), "r"(m[g][1]), "r"(m[g][2]), "r"(m[g][3])
                         : "memory");
          const int valid = tl.tokens - c * 32;         // tokens of this box that are the expert's
          const int row = tl.lo + tl.t0 + c * 32;
          if (!p.d_vec) {
            __syncwarp();
            uint16_t* d = reinterpret_cast<uint16_t*>(p.D) + fi + lane;
            for (int k = 0; k < min(32, valid); ++k)
              if (fi + lane < p.F)
                d[(row + k) * p.ldd] = *reinterpret_cast<const uint16_t*>(S + sw64(k, lane >> 3) + (lane & 7) * 2);
          } else if (valid >= 32 && (!(p.F & 7) || fi + 32 <= p.F)) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&maps.d, s0, fi, row, 0);    // clips the features past F (whole 8s)
              bulk_commit();
            }
          } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tr = i * 8 + (lane >> 2), f = fi + (lane & 3) * 8;
              if (tr >= valid || f >= p.F) continue;
              const uint4 v8 = *reinterpret_cast<const uint4*>(S + sw64(tr, lane & 3));
              uint16_t* dst = reinterpret_cast<uint16_t*>(p.D) + (long long)(row + tr) * p.ldd + f;
              if (f + 8 <= p.F) {
                *reinterpret_cast<uint4*>(dst) = v8;
              } else {
                const uint16_t* e = reinterpret_cast<const uint16_t*>(&v8);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  if (f + k < p.F) dst[k] = e[k];
              }
            }
          }
        }
      }
      if (!released) {  // no chunk of this tile is this warp's
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(smem_u32(&tempty_bar[acc]));
          else remote_arrive_cta(leader_tempty + acc * 8);
        }
      }
    }
    if (lane == 0) bulk_wait_all0();  // this warp's output stores have completed
    __syncwarp();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the leader's MMAs into this CTA's TMEM are drained
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
  }
  if (threadIdx.x == 0 && *abort_flag && p.err != nullptr) atomicOr(p.err, kStatusTimeout);
}

template <int KIND, int IN_FMT, bool OUT32 = false, bool PAIR = true>
static int launch(const EMaps& maps, const EParams& p, long long tiles, cudaStream_t s) {
  // per device: shared-memory opt-in done and how many CTAs or pairs fit at once
  static std::atomic<int> max_pairs_of[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return (int)cudaErrorInvalidDevice;
  constexpr int CTAS = PAIR ? 2 : 1;
  auto kern = expert_kernel<KIND, IN_FMT, OUT32, PAIR>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CTAS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(threads_of(KIND == kWeightGrad));
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int max_pairs = max_pairs_of[dev].load(std::memory_order_acquire);
  if (max_pairs <= 0) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return (int)e;
    cfg.gridDim = dim3(CTAS * (num_sms() / CTAS));
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess || n <= 0) n = num_sms() / CTAS;
    max_pairs = n;
    max_pairs_of[dev].store(n, std::memory_order_release);
  }
  cfg.gridDim = dim3(CTAS * (unsigned)std::min<long long>(tiles, max_pairs));
  return (int)cudaLaunchKernelEx(&cfg, kern, maps, p);
}

static bool on16(const void* p, long long ld, int es) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * es % 16 == 0;
}

// Rows of any alignment (per > 0: matrices of `per` rows, `stride` apart) into
// rows of `units` 16-byte units, zeros behind the columns.
__global__ void __launch_bounds__(256)
expert_pack_kernel(const uint16_t* __restrict__ src, long long ld, long long stride, int per, long long rows, int cols,
                   int units, uint4* __restrict__ dst) {
  for (long long r = (long long)blockIdx.x * blockDim.y + threadIdx.y; r < rows; r += (long long)gridDim.x * blockDim.y) {
    const uint16_t* from = src + (per > 0 ? r / per * stride + r % per * ld : r * ld);
    for (int k = threadIdx.x; k < units; k += blockDim.x) {
      uint4 v;
      uint16_t* e = reinterpret_cast<uint16_t*>(&v);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = k * 8 + i < cols ? from[k * 8 + i] : (uint16_t)0;
      dst[r * units + k] = v;
    }
  }
}

}  // namespace expk
}  // namespace tc

// Forward and input gradient with few tokens an expert run on single CTAs: their
// 128-row tiles of the weights, which then are all that counts, spread more
// evenly over the SMs.  64 experts of 1408 x 2048, forward / input gradient, single
// CTAs against pairs: 16 tokens an expert 65.6 / 61.6 against 73.8 / 62.1 us, 32
// 66.6 / 63.0 against 75.4 / 63.6, 64 68.3 / 71.2 against 76.9 / 65.9, 128 86.5 /
// 105.7 against 82.3 / 77.0 (the host knows the mean only).
static bool use_pairs(const ExpertDesc& g) {
  return g.kind == kWeightGrad || g.rows > (long long)tc::expk::SINGLE_TOKENS * g.experts;
}

// The most tiles a launch can have, whatever the offsets say.
static long long most_tiles(const ExpertDesc& g, int tiles_f, int tiles_c) {
  if (g.kind == kWeightGrad) return (long long)tiles_f * tiles_c * g.experts;
  return tiles_f * std::min<long long>(g.rows, g.rows / tc::expk::tile_tokens(use_pairs(g)) + g.experts);
}

// Whether TMA can address an operand: 16-byte base and pitch, and an expert
// stride that is a 16-byte multiple and not zero (shared weights).
static bool tma_a(const ExpertDesc& g) { return tc::expk::on16(g.a, g.ld_a, 2); }
static bool tma_b(const ExpertDesc& g) {
  return tc::expk::on16(g.b, g.ld_b, 2) &&
         (g.kind == kWeightGrad || g.experts == 1 || (g.stride_b * 2 % 16 == 0 && g.stride_b > 0));
}

// Packed copies: rows of a multiple of 8 elements.
static long long packed_ld(int cols) { return (cols + 7) / 8 * 8; }
static size_t packed_bytes(long long rows, int cols) { return (size_t)((rows * packed_ld(cols) * 2 + 255) / 256 * 256); }
static int cols_a(const ExpertDesc& g) { return g.kind == kForward ? g.inner : g.outer; }
static long long rows_b(const ExpertDesc& g) { return g.kind == kWeightGrad ? g.rows : (long long)g.experts * g.outer; }

// Operands that TMA cannot address are copied into rows that it can, where the
// product is large enough to pay for it.  Against the CUDA cores: 0.13 GFLOP (256
// rows over 4 experts, 511 to 509 wide) 31 us against 40 (forward) and 21 (weight
// gradient), 0.27 GFLOP 26 against 43 and 34, 137 GFLOP (32768 rows over 32
// experts, 2047 to 1021) 219 against 9681.
size_t expert_pack_bytes(const ExpertDesc& g) {
  if ((g.dtype != kBF16 && g.dtype != kFP16) || (tma_a(g) && tma_b(g))) return 0;
  if (2.0 * g.rows * g.inner * (double)g.outer < tc::expk::PACK_FLOPS) return 0;
  size_t n = 0;
  if (!tma_a(g)) n += packed_bytes(g.rows, cols_a(g));
  if (!tma_b(g)) n += packed_bytes(rows_b(g), g.inner);
  return n + 256;
}

static int pack_rows(const void* src, long long ld, long long stride, int per, long long rows, int cols, void* dst,
                     cudaStream_t s) {
  const int units = (int)(packed_ld(cols) / 8);
  dim3 block(32, 8);
  while ((int)block.x < units && block.x < 256) { block.x *= 2; block.y /= 2; }
  const unsigned grid = (unsigned)std::min<long long>((rows + block.y - 1) / block.y, 148LL * 32);
  tc::expk::expert_pack_kernel<<<grid, block, 0, s>>>(reinterpret_cast<const uint16_t*>(src), ld, stride, per, rows, cols,
                                                      units, reinterpret_cast<uint4*>(dst));
  return (int)cudaGetLastError();
}

int expert_tc_packed(const ExpertDesc& g, void* ws, cudaStream_t s) {
  ExpertDesc d = g;
  char* at = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws) + 255) & ~uintptr_t(255));
  int rc = 0;
  if (!tma_a(g)) {
    if ((rc = pack_rows(g.a, g.ld_a, 0, 0, g.rows, cols_a(g), at, s))) return rc;
    d.a = at;
    d.ld_a = packed_ld(cols_a(g));
    at += packed_bytes(g.rows, cols_a(g));
  }
  if (!tma_b(g)) {
    const bool weights = g.kind != kWeightGrad;
    if ((rc = pack_rows(g.b, g.ld_b, weights ? g.stride_b : 0, weights ? g.outer : 0, rows_b(g), g.inner, at, s))) return rc;
    d.b = at;
    d.ld_b = packed_ld(g.inner);
    d.stride_b = g.outer * d.ld_b;
  }
  return expert_tc(d, s);
}

bool expert_tc_ok(const ExpertDesc& g) {
  using namespace tc::expk;
  if (g.dtype != kBF16 && g.dtype != kFP16) return false;
  if (!tma_a(g) || !tma_b(g)) return false;
  const int F = g.kind == kInputGrad ? g.inner : g.outer;
  const int rows = tile_rows(use_pairs(g));
  return most_tiles(g, (F + rows - 1) / rows, (g.inner + 255) / 256) <= (1LL << 30);
}

int expert_tc(const ExpertDesc& g, cudaStream_t s) {
  using namespace tc;
  using namespace tc::expk;
  EParams p{};
  p.offsets = g.offsets; p.experts = g.experts; p.rows = (int)g.rows;
  p.F = g.kind == kInputGrad ? g.inner : g.outer;
  p.C = g.inner;
  p.K = g.kind == kForward ? g.inner : g.outer;
  const bool pairs = use_pairs(g);
  p.tiles_f = (p.F + tile_rows(pairs) - 1) / tile_rows(pairs);
  p.tiles_c = (p.C + 255) / 256;
  p.D = g.d; p.ldd = g.ld_d; p.stride_d = g.stride_d;
  const int des = dtype_size(g.d_dtype);
  p.d_vec = on16(g.d, g.ld_d, des) && (g.kind != kWeightGrad || g.experts == 1 || (g.stride_d * des % 16 == 0 && g.stride_d > 0));
  p.accumulate = g.accumulate;
  p.err = g.status;
  p.timeout_ns = wait_timeout_ns();
  const long long tiles = most_tiles(g, p.tiles_f, p.tiles_c);
  EMaps m;
  bool ok = true;
  if (g.kind == kWeightGrad) {
    // both operands are read along their columns: 64-column boxes of 64 rows
    ok = ok && encode_map(&m.a, g.dtype, g.a, g.outer, g.rows, 1, g.ld_a, g.ld_a, 64, BK);
    ok = ok && encode_map(&m.b[0], g.dtype, g.b, g.inner, g.rows, 1, g.ld_b, g.ld_b, 64, BK);
    for (int i = 1; i < 4; ++i) m.b[i] = m.b[0];
    if (p.d_vec)
      ok = ok && encode_map(&m.d, g.d_dtype, g.d, g.inner, g.outer, g.experts, g.ld_d, g.experts > 1 ? g.stride_d : g.ld_d,
                            g.d_dtype == kFP32 ? 16 : 32, 32, kTmaSw64);
    else m.d = m.a;  // not used
  } else {
    const long long stride = g.experts > 1 ? g.stride_b : g.ld_b;
    ok = ok && (g.kind == kForward ? encode_map(&m.a, g.dtype, g.b, g.inner, g.outer, g.experts, g.ld_b, stride, BK, BM)
                                   : encode_map(&m.a, g.dtype, g.b, g.inner, g.outer, g.experts, g.ld_b, stride, 64, BK));
    for (int i = 0; i < 4; ++i) ok = ok && encode_map(&m.b[i], g.dtype, g.a, p.K, g.rows, 1, g.ld_a, g.ld_a, BK, 16 << i);
    if (p.d_vec) ok = ok && encode_map(&m.d, g.d_dtype, g.d, p.F, g.rows, 1, g.ld_d, g.ld_d, 32, 32, kTmaSw64);
    else m.d = m.a;  // not used
  }
  if (!ok) return (int)cudaErrorInvalidValue;
  const bool bf = g.dtype == kBF16;
  switch (g.kind) {
    case kForward:
      if (!pairs) return bf ? launch<kForward, 1, false, false>(m, p, tiles, s) : launch<kForward, 0, false, false>(m, p, tiles, s);
      return bf ? launch<kForward, 1>(m, p, tiles, s) : launch<kForward, 0>(m, p, tiles, s);
    case kInputGrad:
      if (!pairs) return bf ? launch<kInputGrad, 1, false, false>(m, p, tiles, s) : launch<kInputGrad, 0, false, false>(m, p, tiles, s);
      return bf ? launch<kInputGrad, 1>(m, p, tiles, s) : launch<kInputGrad, 0>(m, p, tiles, s);
    default:
      if (g.d_dtype == kFP32) return bf ? launch<kWeightGrad, 1, true>(m, p, tiles, s) : launch<kWeightGrad, 0, true>(m, p, tiles, s);
      return bf ? launch<kWeightGrad, 1>(m, p, tiles, s) : launch<kWeightGrad, 0>(m, p, tiles, s);
  }
}

}  // namespace muon
