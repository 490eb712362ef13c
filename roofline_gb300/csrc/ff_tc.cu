// The products of the gated feed-forward block on the tcgen05 tensor cores.
//
// One persistent kernel for all of them (FfProduct in ff_tc.cuh).  Operands
// are BF16 planes read by TMA as they are stored, K-major or MN-major; the
// sums stay in tensor memory in FP32 and every epilogue (act, the product of
// the two sums, rounding) runs on them there.
//
// A FP32 product is the sum of the six products of planes x_i y_j with
// i + j <= 2; what is left out is below 2^-26 of |x||y|.  Each MMA rounds the
// sum it adds to towards zero, which over thousands of steps would shift the
// result by far more than FP32's own rounding (measured at K = 2048 with one
// accumulator for all six: 4e-5 of the result).  So x_0 y_0 gathers in one
// accumulator for kFlush K blocks only, is then added to a sum in registers
// with ordinary rounding, and starts again; the five small products, whose
// sum is 2^-8 of the result and its rounding as much smaller, gather in a
// second accumulator over the whole of K.  The small products of a K block
// take five times as long as x_0 y_0, and the registers are updated
// meanwhile, so the MMAs never wait for it.
#include <cstdlib>
#include <mutex>

#include "ff_tc.cuh"
#include "tc_common.cuh"

namespace gg {

using namespace tc;

namespace {

__device__ int g_ff_status;  // 0 = ok, else a GEMM_ERR_* code

// warp 0: TMA, warp 1: MMA, warps 2..9: epilogue, two for each 32 rows
constexpr int kThreadsFF = 320;
constexpr int kEpiWarps = 8;
constexpr int kFlush = 2;

struct FfParams {
  int64_t M, N;        // output extents (of one matrix)
  int kb, segs;        // K blocks of one segment, segments (concat: 2)
  int tiles_m, tiles_n, batches, group_n;
  int a_seg, a_batch, b_seg, b_batch;  // operand = segment * x_seg + batch * x_batch
  int a_mn, b_mn;      // operands stored MN-major
  int act;
  void *c[2];
  int64_t ldc[2];
  float *g, *u;
  int64_t ldg, ldu;
  uint64_t wait_ns;
  int stall_producer;  // test hook: the producer issues nothing
};

// CG: CTAs that share one tile of CG * 128 rows (a pair splits the columns of
// B between its two shared memories).  BN: accumulator columns of a tile; the
// gated form gives half of them to each of its two sums.  P: planes.
template <int P, int CG, int BN, bool GATED>
struct FfCfg {
  static constexpr int BK = 64;                     // 128 bytes of K, one swizzle line
  static constexpr int B_ROWS = BN / CG;            // columns of B in this CTA
  static constexpr int A_BYTES = 128 * BK * 2;      // one plane
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE_BYTES = P * (A_BYTES + B_BYTES);
  static constexpr int EPI_BYTES = kEpiWarps * 32 * 128;  // 32 rows x 128 bytes per warp
  static constexpr int BUDGET = 227 * 1024 - 1024 - 256 - EPI_BYTES;
  static constexpr int FIT = BUDGET / STAGE_BYTES;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 256 + EPI_BYTES;
  // two accumulators: one plane, one is filled while the other is drained;
  // three planes, the large and the small products
  static constexpr int ACCS = 2;
  static constexpr int TMEM_COLS = ACCS * BN;
  static constexpr int OUT_COLS = GATED ? BN / 2 : BN;
  // columns of B one load brings: the gated form takes each half of a single
  // CTA's columns, or all of one CTA of a pair, from one of the two matrices
  static constexpr int B_LOAD = GATED && CG == 1 ? BN / 2 : B_ROWS;
  static_assert(TMEM_COLS <= 512 && STAGES >= 2, "");
};

// Waits for the phase of `bar` with the given parity, at most ns; gives up at
// once when another role of the CTA has.
__device__ __forceinline__ bool ff_wait(uint64_t *bar, uint32_t parity, uint64_t ns,
                                        volatile int *abort_flag) {
  uint64_t deadline = 0;
  uint32_t spins = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++spins & 63u) == 0) {
      if (*abort_flag) return false;
      const uint64_t t = globaltimer();
      if (deadline == 0)
        deadline = t + ns;
      else if (t > deadline)
        return false;
    }
  }
  return true;
}

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The shared::cluster address of a shared-memory address in CTA `rank`.
__device__ __forceinline__ uint32_t map_to_cta(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

template <int CG>
__device__ __forceinline__ void arrive_leader(uint64_t *bar) {
  if constexpr (CG == 1)
    mbar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                     map_to_cta(smem_u32(bar), 0))
                 : "memory");
}

// A box of the map at (x, y, plane z) into this CTA's shared memory; its bytes
// count on the leader's barrier (address `bar` in shared::cluster for a pair).
template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                         int32_t x, int32_t y, int32_t z) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// One plane of an operand tile of `rows` (along M or N) x 64 (along K) from
// row r0 and K index k0.  K-major: one box of rows x 64.  MN-major: boxes of
// 64 K rows x 64, one for each 64 of the tile's rows.
template <int CG>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                          int mn, int rows, int32_t r0, int32_t k0, int plane) {
  if (!mn) {
    load_box<CG>(dst, map, bar, k0, r0, plane);
  } else {
    for (int r = 0; r < rows; r += 64) load_box<CG>(dst + r * 128, map, bar, r0 + r, k0, plane);
  }
}

// Descriptor of a 128-byte-swizzled operand tile.  K-major: rows of 128 bytes,
// 8-row groups 1024 bytes apart; MN-major: 8-deep K groups 1024 bytes apart
// (SBO), 64-wide blocks 64 * 128 bytes apart (LBO).  Fields as smem_desc.
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr, int mn) {
  return smem_desc(saddr, 1024, 2) + (mn ? ((uint64_t)((8192 >> 4) - 1) << 16) : 0);
}

template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on `bar` (in both CTAs of a pair) once the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if constexpr (CG == 1)
    mma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void ff_tmem_alloc(uint32_t *slot, uint32_t cols) {
  if constexpr (CG == 1) {
    tmem_alloc(slot, cols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}

template <int CG>
__device__ __forceinline__ void ff_tmem_dealloc(uint32_t taddr, uint32_t cols) {
  if constexpr (CG == 1)
    tmem_dealloc(taddr, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15])
      : "r"(taddr));
}

// Stores a warp's 32 x 32 block: lane r holds row r.  dst is row 0, column 0
// of it, rows and cols what lies inside the matrix.  The block goes through
// the warp's shared memory in 16-byte pieces, swizzled so that neither side
// has bank conflicts, and leaves as whole rows of 64 (BF16) or 128 bytes; a
// clipped or unaligned block leaves element by element.
template <typename T>
__device__ __forceinline__ void store_block(uint8_t *st, const float (&v)[32], T *dst, int64_t ld,
                                            int rows, int cols, bool vec) {
  constexpr int PER = 16 / sizeof(T);      // values of a piece
  constexpr int PIECES = 32 / PER;         // pieces of a row: 4 or 8
  constexpr int ROW = 32 * sizeof(T);
  const int lane = threadIdx.x & 31;
  auto at = [](int r, int k) {
    return r * ROW + ((k ^ (PIECES == 8 ? r & 7 : (r >> 1) & 3)) * 16);
  };
#pragma unroll
  for (int k = 0; k < PIECES; ++k) {
    __align__(16) T t[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) t[i] = from_f32<T>(v[k * PER + i]);
    *reinterpret_cast<uint4 *>(st + at(lane, k)) = *reinterpret_cast<const uint4 *>(t);
  }
  __syncwarp();
  if (vec && cols >= 32) {
#pragma unroll
    for (int it = 0; it < PIECES; ++it) {
      const int r = it * (32 / PIECES) + lane / PIECES, k = lane % PIECES;
      if (r < rows)
        *reinterpret_cast<uint4 *>(dst + r * ld + k * PER) =
            *reinterpret_cast<const uint4 *>(st + at(r, k));
    }
  } else if (lane < cols) {
#pragma unroll 4
    for (int r = 0; r < rows; ++r)
      dst[r * ld + lane] =
          *reinterpret_cast<const T *>(st + at(r, lane / PER) + (lane % PER) * sizeof(T));
  }
  __syncwarp();
}

struct TileAt {
  int64_t m, n;
  int batch;
};
// Tiles are numbered batch by batch, each in bands of group_n tile columns
// walked down their rows, so that the tiles worked on at one time cover a
// compact block of the output and share their operands through L2.
__device__ __forceinline__ TileAt tile_at(const FfParams &p, int64_t t) {
  const int64_t per = (int64_t)p.tiles_m * p.tiles_n;
  const int batch = (int)(t / per);
  t -= batch * per;
  const int64_t band_tiles = (int64_t)p.group_n * p.tiles_m, band = t / band_tiles;
  const int64_t first = band * p.group_n, left = p.tiles_n - first;
  const int64_t width = left < p.group_n ? left : p.group_n, local = t - band * band_tiles;
  return {local / width, first + local % width, batch};
}

template <int P, int CG, int BN, bool GATED>
__global__ void __launch_bounds__(kThreadsFF, 1)
ff_tc_kernel(const __grid_constant__ CUtensorMap ma0, const __grid_constant__ CUtensorMap ma1,
             const __grid_constant__ CUtensorMap mb0, const __grid_constant__ CUtensorMap mb1,
             const FfParams p) {
  using Cfg = FfCfg<P, CG, BN, GATED>;
  using T = typename std::conditional<P == 1, bf16, float>::type;
  constexpr int STAGES = Cfg::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + STAGES * Cfg::STAGE_BYTES);
  uint64_t *empty = full + STAGES;
  uint64_t *acc_full = empty + STAGES;      // [ACCS]
  uint64_t *acc_empty = acc_full + Cfg::ACCS;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + Cfg::ACCS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  uint8_t *epi = reinterpret_cast<uint8_t *>(full) + 256;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : cta_rank();
  const int64_t worker = blockIdx.x / CG, workers = gridDim.x / CG;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * p.batches;
  const int kbs = p.kb * p.segs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < Cfg::ACCS; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], CG * kEpiWarps);  // every epilogue warp of the tile
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) ff_tmem_alloc<CG>(tmem_slot, Cfg::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  bool ok = true;
  if (warp == 0) {
    // ---------------- producer: this CTA's rows of A and columns of B
    uint32_t issued = 0;
    if (lane == 0 && !p.stall_producer) {
      for (int64_t t = worker; ok && t < tiles; t += workers) {
        const TileAt at = tile_at(p, t);
        const int32_t m0 = (int32_t)(at.m * (CG * 128) + rank * 128);
        const int32_t n0 = (int32_t)(at.n * Cfg::OUT_COLS);
        for (int kb = 0; kb < kbs; ++kb, ++issued) {
          const uint32_t s = issued % STAGES;
          if (!ff_wait(&empty[s], ((issued / STAGES) & 1u) ^ 1u, p.wait_ns,
                       abort_flag)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_expect_tx(&full[s], CG * Cfg::STAGE_BYTES);
          const uint32_t bar =
              CG == 1 ? smem_u32(&full[s]) : map_to_cta(smem_u32(&full[s]), 0);
          const int seg = kb >= p.kb;
          const int32_t k0 = (kb - seg * p.kb) * Cfg::BK;
          const CUtensorMap *ma = seg * p.a_seg + at.batch * p.a_batch ? &ma1 : &ma0;
          const CUtensorMap *mb = seg * p.b_seg + at.batch * p.b_batch ? &mb1 : &mb0;
          const uint32_t a = smem_u32(smem + s * Cfg::STAGE_BYTES), b = a + P * Cfg::A_BYTES;
#pragma unroll
          for (int q = 0; q < P; ++q) {
            load_tile<CG>(a + q * Cfg::A_BYTES, ma, bar, p.a_mn, 128, m0, k0, q);
            const uint32_t bq = b + q * Cfg::B_BYTES;
            if constexpr (!GATED) {
              load_tile<CG>(bq, mb, bar, p.b_mn, Cfg::B_ROWS, n0 + (int)rank * Cfg::B_ROWS, k0, q);
            } else if constexpr (CG == 2) {
              load_tile<CG>(bq, rank ? &mb1 : &mb0, bar, p.b_mn, Cfg::B_ROWS, n0, k0, q);
            } else {
              load_tile<CG>(bq, &mb0, bar, p.b_mn, BN / 2, n0, k0, q);
              load_tile<CG>(bq + BN / 2 * 128, &mb1, bar, p.b_mn, BN / 2, n0, k0, q);
            }
          }
        }
      }
      // Every stage handed back: no load is in flight and no arrival from the
      // pair's MMAs still on its way here.
      for (uint32_t it = issued > STAGES ? issued - STAGES : 0; ok && it < issued; ++it)
        if (!ff_wait(&empty[it % STAGES], (it / STAGES) & 1u, p.wait_ns, abort_flag))
          ok = false;
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (of the pair)
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)p.a_mn << 15) |
                             ((uint32_t)p.b_mn << 16) | ((uint32_t)(BN >> 3) << 17) |
                             ((uint32_t)((CG * 128) >> 4) << 24);
      // 16 along K: 32 bytes of a K-major line, two 8-deep groups MN-major
      const uint64_t astep = p.a_mn ? 2048 >> 4 : 32 >> 4, bstep = p.b_mn ? 2048 >> 4 : 32 >> 4;
      uint32_t it = 0, used[2] = {0, 0};  // K blocks; times each accumulator was filled
      // Before accumulator i is filled anew, the epilogue has read it.
      auto take = [&](int i) {
        ok = ff_wait(&acc_empty[i], (used[i]++ & 1u) ^ 1u, p.wait_ns, abort_flag);
        tc_fence_after();
        return ok;
      };
      int done = 0;
      for (int64_t t = worker; ok && t < tiles; t += workers, ++done) {
        const int acc = P == 1 ? done & 1 : 0;
        if (P == 1 && !take(acc)) break;
        const uint32_t d = tmem_base + (uint32_t)(acc * BN);
        for (int kb = 0; kb < kbs; ++kb, ++it) {
          const uint32_t s = it % STAGES;
          if (!ff_wait(&full[s], (it / STAGES) & 1u, p.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + s * Cfg::STAGE_BYTES), b = a + P * Cfg::A_BYTES;
          const uint64_t da = tile_desc(a, p.a_mn), db = tile_desc(b, p.b_mn);
          if (P == 3 && kb % kFlush == 0 && !take(0)) break;
          const bool first = P == 1 ? kb == 0 : kb % kFlush == 0;
#pragma unroll
          for (int kk = 0; kk < Cfg::BK / 16; ++kk)
            mma_bf16<CG>(d, da + kk * astep, db + kk * bstep, idesc, first && kk == 0 ? 0u : 1u);
          if constexpr (P == 3) {
            if (kb % kFlush == kFlush - 1 || kb == kbs - 1) commit<CG>(&acc_full[0]);
            if (kb == 0 && !take(1)) break;
#pragma unroll
            for (int kk = 0; kk < Cfg::BK / 16; ++kk) {
#pragma unroll
              for (int sum = P - 1; sum >= 1; --sum) {
#pragma unroll
                for (int i = 0; i <= sum; ++i)
                  mma_bf16<CG>(d + BN, da + kk * astep + (uint64_t)(i * (Cfg::A_BYTES >> 4)),
                               db + kk * bstep + (uint64_t)((sum - i) * (Cfg::B_BYTES >> 4)),
                               idesc, (kb > 0 || kk > 0 || sum < P - 1 || i > 0) ? 1u : 0u);
              }
            }
          }
          commit<CG>(&empty[s]);
        }
        if (ok) commit<CG>(&acc_full[P == 1 ? acc : 1]);
      }
    }
  } else {
    // ---------------- epilogue: a warp has 32 rows (the tensor-memory lanes
    // 32 (w & 3) on) and half the columns of the tile
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    constexpr int COLS = Cfg::OUT_COLS / 2;
    uint8_t *st = epi + (warp - 2) * (32 * 128);
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    auto aligned = [](const void *q, int64_t ld, int64_t size) {
      return ((reinterpret_cast<uintptr_t>(q) | (uintptr_t)(ld * size)) & 15) == 0;
    };
    const bool vec_c = aligned(p.c[0], p.ldc[0], sizeof(T)) &&
                       aligned(p.c[1], p.ldc[1], sizeof(T));
    const bool vec_g = aligned(p.g, p.ldg, 4), vec_u = aligned(p.u, p.ldu, 4);
    uint32_t used[2] = {0, 0};
    // tcgen05.ld is warp-collective: the warp proceeds or stops as one
    auto wait_full = [&](int i) {
      ok = __all_sync(0xffffffffu, ff_wait(&acc_full[i], used[i]++ & 1u, p.wait_ns, abort_flag));
      tc_fence_after();
      return ok;
    };
    auto release = [&](int i) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader<CG>(&acc_empty[i]);
    };
    int done = 0;
    for (int64_t t = worker; ok && t < tiles; t += workers, ++done) {
      const TileAt at = tile_at(p, t);
      const int64_t r0 = at.m * (CG * 128) + rank * 128 + quarter * 32;
      const int64_t c0 = at.n * Cfg::OUT_COLS + half * COLS;
      const int rows = (int)(p.M - r0 < 32 ? (p.M - r0 > 0 ? p.M - r0 : 0) : 32);
      T *c = static_cast<T *>(p.c[at.batch]);
      const int64_t ldc = p.ldc[at.batch];
      // 32 columns from c0 + j on: v the sums (of the gate), w those of b1
      auto finish = [&](int j, float (&v)[32], const float (&w)[32]) {
        const int64_t left = p.N - c0 - j;
        if (left <= 0 || rows == 0) return;
        const int cols = left < 32 ? (int)left : 32;
        if constexpr (GATED) {
          if (p.g) {
            store_block<float>(st, v, p.g + r0 * p.ldg + c0 + j, p.ldg, rows, cols, vec_g);
            store_block<float>(st, w, p.u + r0 * p.ldu + c0 + j, p.ldu, rows, cols, vec_u);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = act_value<P == 1>(v[i], p.act) * w[i];
        }
        if (c) store_block<T>(st, v, c + r0 * ldc + c0 + j, ldc, rows, cols, vec_c);
      };
      if constexpr (P == 1) {
        const int acc = done & 1;
        if (!wait_full(acc)) break;
        const uint32_t base = lane_base + (uint32_t)(acc * BN + half * COLS);
#pragma unroll 1
        for (int j = 0; j < COLS; j += 32) {
          float v[32], w[32];
          tmem_ld32(base + (uint32_t)j, reinterpret_cast<uint32_t(&)[32]>(v));
          if constexpr (GATED)
            tmem_ld32(base + (uint32_t)(BN / 2 + j), reinterpret_cast<uint32_t(&)[32]>(w));
          tmem_ld_wait();
          if (j + 32 >= COLS) release(acc);
          finish(j, v, w);
        }
      } else {
        constexpr int BLOCKS = (GATED ? 2 : 1) * COLS / 32;
        float sum[BLOCKS][32];
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
          for (int k = 0; k < 32; ++k) sum[i][k] = 0.0f;
        // the accumulator columns of block i
        auto col = [&](int i) {
          const int j = 32 * i;
          return (uint32_t)(GATED && j >= COLS ? BN / 2 + half * COLS + j - COLS
                                               : half * COLS + j);
        };
        const int parts = (kbs + kFlush - 1) / kFlush + 1;
        for (int part = 0; part < parts; ++part) {
          const int acc = part == parts - 1;
          if (!wait_full(acc)) break;
#pragma unroll
          for (int i = 0; i < 2 * BLOCKS; ++i) {
            float x[16];
            tmem_ld16(lane_base + (uint32_t)(acc * BN) + col(i / 2) + (i & 1) * 16, x);
            tmem_ld_wait();
            if (i == 2 * BLOCKS - 1) release(acc);
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[i / 2][(i & 1) * 16 + k] += x[k];
          }
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < COLS / 32; ++i)
          finish(32 * i, sum[i], sum[GATED ? i + COLS / 32 : i]);
      }
    }
  }

  if (!ok) {
    *abort_flag = 1;
    atomicExch(&g_ff_status, GEMM_ERR_DEVICE_TIMEOUT);
    // copies and MMAs still in flight land within microseconds: 1 ms, then out
    const uint64_t until = globaltimer() + 1000000ull;
    while (globaltimer() < until) __nanosleep(1000);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the pair's MMAs read both shared memories
  tc_fence_after();
  if (warp == 1) ff_tmem_dealloc<CG>(tmem_base, Cfg::TMEM_COLS);
}

// ------------------------------------------------------------------ host side

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool get_encoder() {
  std::call_once(g_encode_once, [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    else
      cudaGetLastError();
  });
  return g_encode != nullptr;
}

// Map of an operand's planes whose box is 64 contiguous values x `rows` rows.
bool encode(CUtensorMap *m, const FfOperand &o, int planes, int rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2,
                                 (cuuint64_t)(planes > 1 ? o.plane : o.ld * o.outer) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1}, estr[3] = {1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16 *>(o.p), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint64_t env_u64(const char *name, uint64_t dflt) {
  const char *v = std::getenv(name);
  return v && *v ? std::strtoull(v, nullptr, 10) : dflt;
}

template <int P, int CG, int BN, bool GATED>
int launch_cfg(const FfProduct &q, const DeviceProps &dp, cudaStream_t s) {
  using Cfg = FfCfg<P, CG, BN, GATED>;
  FfParams p{};
  p.M = q.M;
  p.N = q.N;
  p.kb = (int)ceil_div(q.K, Cfg::BK);
  p.segs = q.kind == kFfConcat ? 2 : 1;
  p.batches = q.kind == kFfBatch ? 2 : 1;
  p.a_seg = p.b_seg = q.kind == kFfConcat;
  p.a_batch = q.kind == kFfBatch && q.a_two;
  p.b_batch = q.kind == kFfBatch && q.b_two;
  p.a_mn = q.a[0].mn_major;
  p.b_mn = q.b[0].mn_major;
  p.act = q.act;
  p.c[0] = q.c[0];
  p.c[1] = q.c[1];
  p.ldc[0] = q.ldc;
  p.ldc[1] = q.ldc2;
  p.g = q.g;
  p.u = q.u;
  p.ldg = q.ldg;
  p.ldu = q.ldu;
  p.wait_ns = env_u64("GEMM_DEBUG_WAIT_LIMIT_NS", 2000000000ull);
  p.stall_producer = (int)env_u64("GEMM_DEBUG_STALL_PRODUCER", 0);
  p.tiles_m = (int)ceil_div(q.M, CG * 128);
  p.tiles_n = (int)ceil_div(q.N, Cfg::OUT_COLS);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * p.batches;
  int64_t workers = dp.sm_count / CG;
  if (workers > tiles) workers = tiles;
  p.group_n = p.tiles_n < 8 ? p.tiles_n : 8;

  CUtensorMap ma[2], mb[2];
  for (int i = 0; i < 2; ++i) {
    const FfOperand &a = q.a[i].p ? q.a[i] : q.a[0], &b = q.b[i].p ? q.b[i] : q.b[0];
    if (!encode(&ma[i], a, P, a.mn_major ? 64 : 128) ||
        !encode(&mb[i], b, P, b.mn_major ? 64 : Cfg::B_LOAD))
      return GEMM_ERR_UNSUPPORTED;
  }
  auto kern = ff_tc_kernel<P, CG, BN, GATED>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) !=
      cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(workers * CG));
  lc.blockDim = dim3(kThreadsFF);
  lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, kern, ma[0], ma[1], mb[0], mb[1], p) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

template <int P, bool GATED>
int launch_any(const FfProduct &q, const DeviceProps &dp, cudaStream_t s) {
  // Tiles of 256 x 256 by pairs of CTAs once they fill the GPU, 128 x 128 by
  // single ones otherwise.
  const int64_t out = GATED ? 128 : 256;
  const int64_t big = ceil_div(q.M, 256) * ceil_div(q.N, out) * (q.kind == kFfBatch ? 2 : 1);
  if (big >= dp.sm_count / 2) return launch_cfg<P, 2, 256, GATED>(q, dp, s);
  return launch_cfg<P, 1, 128, GATED>(q, dp, s);
}

}  // namespace

int launch_ff_product(const FfProduct &q, const DeviceProps &dp, cudaStream_t s) {
  if (!tc_supported(dp)) return GEMM_ERR_UNSUPPORTED;
  if (!get_encoder()) return GEMM_ERR_CUDA;
  if (q.planes == 1)
    return q.kind == kFfGated ? launch_any<1, true>(q, dp, s) : launch_any<1, false>(q, dp, s);
  return q.kind == kFfGated ? launch_any<3, true>(q, dp, s) : launch_any<3, false>(q, dp, s);
}

// Called on a synchronised stream.
int ff_read_and_clear_status() {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_ff_status, sizeof(int)) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_ff_status, &zero, sizeof(int)) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_CUDA;
    }
  }
  return v;
}

}  // namespace gg
