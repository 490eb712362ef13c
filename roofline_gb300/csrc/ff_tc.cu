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
// meanwhile, so the MMAs never wait for it.  A BF16 product's sum is one
// accumulator's up to 32768 of K; longer ones are added up in parts (kLong).
//
// GB300 (a dense BF16 GEMM reaches 1920 TFLOP/s in a burst, 1725 sustained):
// BF16 4096 x 4096 x 14336, 0.96 TFLOP, 507-524 us, the tensor pipe busy 87 %
// of it; 1 x 4096 x 11008, 180 MB, 32.9 us (5.5 TB/s).  FP32 2048 x 1024 x 2816
// with GELU: the block 125 us with the tensor pipe 60 % busy (142 GFLOP of BF16
// products: 74 us), its gradients 165 us, 86 % busy.
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
constexpr int kFlush = 4;
// K blocks of one part of a long BF16 sum.  The rounding towards zero takes up
// to 1.6 x 2^-24 of a sum of one sign for every 16 of K: 1.5e-4 over a part's
// 32768, a thirteenth of BF16's own rounding, but 6e-3 over a million tokens.
constexpr int kLong = 512;

// One product of a launch.
struct FfParams {
  int64_t M, N;        // output extents (of one matrix)
  int64_t tiles;
  int kb, segs;        // K blocks of one segment, segments (concat: 2)
  int tiles_m, tiles_n, group_n;
  int a_seg, a_batch, b_seg, b_batch;  // operand = segment * x_seg + batch * x_batch
  int a_mn, b_mn;      // operands stored MN-major
  int bn, out_cols;    // a tile's accumulator and output columns
  int a_bytes, b_bytes;  // one plane of a stage: A's rows and B's columns in this CTA
  int act;
  void *c[2];
  int64_t ldc[2];
  float *g, *u;
  int64_t ldg, ldu;
};

// A launch: one product, or the two of a backward pass, whose tiles the
// workers (CTAs or pairs) take as one list (Walk).
struct FfLaunch {
  CUtensorMap map[2][4];  // of a product: A, A', B, B'
  FfParams p[2];          // the second without tiles if there is one product
  int stages, stage_bytes;
  int64_t early_from, early;
  uint64_t wait_ns;
  int stall_producer;  // test hook: the producer issues nothing
};

// A worker's tiles: those of the first product in turn; then, for the workers
// from early_from on, which got one fewer of them, as many of the second as
// that one takes the time of (early); then the rest of the second in turn.
struct Walk {
  const FfLaunch &l;
  int64_t worker, workers, first, done = 0, second;
  __device__ __forceinline__ Walk(const FfLaunch &launch, int64_t w, int64_t n)
      : l(launch), worker(w), workers(n), first(w),
        second((n - launch.early_from) * launch.early + w) {}
  __device__ __forceinline__ bool next(int &product, int64_t &tile) {
    if (first < l.p[0].tiles) {
      product = 0;
      tile = first;
      first += workers;
      return true;
    }
    product = 1;
    if (worker >= l.early_from && done < l.early) {
      tile = (worker - l.early_from) * l.early + done++;
      if (tile < l.p[1].tiles) return true;
      done = l.early;
    }
    tile = second;
    second += workers;
    return tile < l.p[1].tiles;
  }
};

constexpr int kLine = 128;       // bytes of one row of a stage: 64 of K, a swizzle line
constexpr int kBlockK = 64;
constexpr int kMaxStages = 12;
constexpr int kEpiBytes = kEpiWarps * 4096;  // 32 x 16 values, twice, per warp
constexpr int kStageBudget = 227 * 1024 - 1024 - 256 - kEpiBytes;
constexpr int kTmemCols = 512;

// The accumulators of a tile.  One plane: two, one filled while the other is
// drained.  Three planes: one or, where they fit, two for the large products
// (the second is filled while the first is added to the registers), and one
// for the small ones.
template <int P, int BN>
struct Acc {
  static constexpr int COLS = P == 1 ? 256 : BN;
  static constexpr int LARGE = P == 1 || 3 * BN <= kTmemCols ? 2 : 1;
  static constexpr int SMALL = LARGE;  // index of the small products' accumulator
  static constexpr int COUNT = P == 1 ? 2 : LARGE + 1;
  static_assert(COUNT * COLS <= kTmemCols, "");
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

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&r)[16]) {
  uint32_t v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(r[i]);
  tmem_st<16>(taddr, v);
}

// What a warp's blocks of 32 rows x 16 columns become: c = v, or (gated)
// act(v) * w with v and w themselves to g and u if given.
template <typename T, bool GATED>
struct Writer {
  uint8_t *st;  // the warp's 4 KB of shared memory: v, then w
  T *c;
  float *g, *u;  // row 0 of the warp's rows, column 0 of the matrix
  int64_t ldc, ldg, ldu, N;
  int rows, act;
  bool vec_c, vec_gu;  // every row of c, of g and u, starts on a 16-byte boundary

  // Row r's 16-byte piece k: swizzled so that a quarter warp that writes one
  // piece of 8 rows, or reads the 4 of 2 rows, meets each bank once.
  __device__ __forceinline__ static int piece(int r, int k) {
    return r * 64 + ((k ^ ((r >> 1) & 3)) * 16);
  }

  // act(x) * y for eight values at once: one choice of the activation, and
  // eight chains of arithmetic in flight in a warp that has few neighbours.
  __device__ __forceinline__ void combine(float (&x)[8], const float (&y)[8]) const {
    with_act(act, [&](auto a) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = act_of<T, decltype(a)::value>(x[i]) * y[i];
    });
  }

  // Columns [col, col + 16): lane r holds row r.  The values go through shared
  // memory and are finished where they leave: four of a row to a lane, or one
  // of a row in a clipped or unaligned block, so that rows leave in whole
  // sectors.
  __device__ __forceinline__ void block(int64_t col, const float *v, const float *w) const {
    const int lane = threadIdx.x & 31;
    if (rows <= 0 || col >= N) return;
    const int cols = N - col < 16 ? (int)(N - col) : 16;
    const uint8_t *sw = st + 2048;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      *reinterpret_cast<float4 *>(st + piece(lane, k)) =
          make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      if (GATED)
        *reinterpret_cast<float4 *>(st + 2048 + piece(lane, k)) =
            make_float4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
    __syncwarp();
    if (GATED && g) {
      if (vec_gu && cols == 16) {
        const int k = lane & 3;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int r = it * 8 + (lane >> 2);
          if (r >= rows) continue;
          *reinterpret_cast<float4 *>(g + r * ldg + col + 4 * k) =
              *reinterpret_cast<const float4 *>(st + piece(r, k));
          *reinterpret_cast<float4 *>(u + r * ldu + col + 4 * k) =
              *reinterpret_cast<const float4 *>(sw + piece(r, k));
        }
      } else {
        const int j = lane & 15, off = (j & 3) * 4;
#pragma unroll 4
        for (int r = lane >> 4; r < 32; r += 2) {
          if (j >= cols || r >= rows) continue;
          g[r * ldg + col + j] = *reinterpret_cast<const float *>(st + piece(r, j >> 2) + off);
          u[r * ldu + col + j] = *reinterpret_cast<const float *>(sw + piece(r, j >> 2) + off);
        }
      }
    }
    float x[8], y[8];
    if (!c) {
    } else if (vec_c && cols == 16) {
      const int k = lane & 3;
      const int64_t at = col + 4 * k;
#pragma unroll 1
      for (int r0 = lane >> 2; r0 < 32; r0 += 16) {  // rows r0 and r0 + 8
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 f = *reinterpret_cast<const float4 *>(st + piece(r0 + 8 * h, k));
          x[4 * h] = f.x, x[4 * h + 1] = f.y, x[4 * h + 2] = f.z, x[4 * h + 3] = f.w;
          if (GATED) {
            const float4 e = *reinterpret_cast<const float4 *>(sw + piece(r0 + 8 * h, k));
            y[4 * h] = e.x, y[4 * h + 1] = e.y, y[4 * h + 2] = e.z, y[4 * h + 3] = e.w;
          }
        }
        if (GATED) combine(x, y);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = r0 + 8 * h;
          __align__(16) T t[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = from_f32<T>(x[4 * h + i]);
          if (r < rows) {
            if constexpr (sizeof(T) == 4)
              *reinterpret_cast<float4 *>(c + r * ldc + at) = *reinterpret_cast<float4 *>(t);
            else
              *reinterpret_cast<uint2 *>(c + r * ldc + at) = *reinterpret_cast<uint2 *>(t);
          }
        }
      }
    } else {
      const int j = lane & 15, off = (j & 3) * 4, last = j < cols ? rows : 0;
#pragma unroll 1
      for (int r0 = lane >> 4; r0 < 32; r0 += 16) {  // rows r0, r0 + 2, ..., r0 + 14
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          x[h] = *reinterpret_cast<const float *>(st + piece(r0 + 2 * h, j >> 2) + off);
          if (GATED)
            y[h] = *reinterpret_cast<const float *>(sw + piece(r0 + 2 * h, j >> 2) + off);
        }
        if (GATED) combine(x, y);
#pragma unroll
        for (int h = 0; h < 8; ++h)
          if (r0 + 2 * h < last) c[(r0 + 2 * h) * ldc + col + j] = from_f32<T>(x[h]);
      }
    }
    __syncwarp();  // the block's place is written again
  }
};

// One part of a long sum: the columns of this warp's blocks (every second 16 from
// j0 on, gated: of both sums) at `from`, with those at `sum` if they are to be
// added, to `to`.
template <bool GATED>
__device__ __forceinline__ void gather_part(uint32_t from, uint32_t sum, uint32_t to, bool add,
                                         int out_cols, int j0) {
#pragma unroll 1
  for (int j = j0; j < out_cols; j += 32) {
#pragma unroll
    for (int side = 0; side < (GATED ? 2 : 1); ++side) {
      const uint32_t at = (uint32_t)(side * out_cols + j);
      float v[16], w[16];
      tmem_ld16(from + at, v);
      if (add) tmem_ld16(sum + at, w);
      tmem_ld_wait();
      if (add) {
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] += w[k];
      }
      tmem_st16(to + at, v);
    }
  }
  tmem_st_wait();
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

// CG: CTAs that share one tile of CG * 128 rows (a pair splits the columns of
// B between its two shared memories).  BN: accumulator columns of a tile, of
// which the gated form gives half to each of its two sums; with one plane it
// is chosen at run time (BN = 0).  P: planes.  LONG: one plane, sums over more
// than kLong blocks among the launch's; apart, because what they need in the
// issuing thread's and the epilogue's loops slows the other sums down by 2 %
// (4096 x 4096 x 14336 590 -> 602 us, 1025 x 777 x 1341 trained 52.8 -> 54.0).
template <int P, int CG, int BN, bool GATED, bool LONG>
__global__ void __launch_bounds__(kThreadsFF, 1)
ff_tc_kernel(const __grid_constant__ FfLaunch l) {
  static_assert((P == 1) == (BN == 0) && (P == 1 || !LONG), "");
  using T = typename std::conditional<P == 1, bf16, float>::type;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  const uint32_t stages = (uint32_t)l.stages, stage_bytes = (uint32_t)l.stage_bytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + stages * stage_bytes);
  uint64_t *empty = full + kMaxStages;
  using A = Acc<P, BN>;
  uint64_t *acc_full = empty + kMaxStages;  // [A::COUNT]
  uint64_t *acc_empty = acc_full + 3;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 3);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  uint8_t *epi = reinterpret_cast<uint8_t *>(full) + 256;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : cta_rank();
  const int64_t worker = blockIdx.x / CG, workers = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < A::COUNT; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], CG * kEpiWarps);  // every epilogue warp of the tile
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane < 4) prefetch_tmap(&l.map[0][lane]);
  if (warp == 1) ff_tmem_alloc<CG>(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // operands come from the passes before it in the stream
  grid_dependency_wait();
  grid_launch_dependents();

  bool ok = true;
  if (warp == 0) {
    // ---------------- producer: this CTA's rows of A and columns of B
    if (lane == 0 && !l.stall_producer) {
      uint32_t s = 0, ph = 1;
      auto take = [&] {
        ok = ff_wait(&empty[s], ph, l.wait_ns, abort_flag);
        return ok;
      };
      auto next = [&] {
        if (++s == stages) s = 0, ph ^= 1;
      };
      // A product's parameters and maps at addresses that the compiler knows:
      // issuing a copy through a pointer that it does not took longer than the
      // tensor core takes for the K block (8192 x 4096 x 11008, MN-major
      // operands in BF16: 2.1 ms for both products, 1.66 this way).
      auto load = [&](auto which, int64_t t) {
        constexpr int product = decltype(which)::value;
        const FfParams &p = l.p[product];
        const int kbs = p.kb * p.segs, b_rows = p.b_bytes / kLine;
        const TileAt at = tile_at(p, t);
        const int32_t m0 = (int32_t)(at.m * (CG * 128) + rank * 128);
        const int32_t n0 = (int32_t)(at.n * p.out_cols);
        for (int kb = 0; kb < kbs && take(); ++kb, next()) {
          if (rank == 0) mbar_expect_tx(&full[s], CG * P * (uint32_t)(p.a_bytes + p.b_bytes));
          const uint32_t bar =
              CG == 1 ? smem_u32(&full[s]) : map_to_cta(smem_u32(&full[s]), 0);
          const int seg = kb >= p.kb;
          const int32_t k0 = (kb - seg * p.kb) * kBlockK;
          const CUtensorMap *ma =
              seg * p.a_seg + at.batch * p.a_batch ? &l.map[product][1] : &l.map[product][0];
          const CUtensorMap *mb =
              seg * p.b_seg + at.batch * p.b_batch ? &l.map[product][3] : &l.map[product][2];
          const uint32_t a = smem_u32(smem) + s * stage_bytes, b = a + P * (uint32_t)p.a_bytes;
#pragma unroll
          for (int q = 0; q < P; ++q) {
            load_tile<CG>(a + q * p.a_bytes, ma, bar, p.a_mn, 128, m0, k0, q);
            const uint32_t bq = b + q * p.b_bytes;
            if constexpr (!GATED) {
              load_tile<CG>(bq, mb, bar, p.b_mn, b_rows, n0 + (int)rank * b_rows, k0, q);
            } else if constexpr (CG == 2) {
              load_tile<CG>(bq, rank ? &l.map[product][3] : &l.map[product][2], bar, p.b_mn,
                            b_rows, n0, k0, q);
            } else {
              load_tile<CG>(bq, &l.map[product][2], bar, p.b_mn, b_rows / 2, n0, k0, q);
              load_tile<CG>(bq + p.b_bytes / 2, &l.map[product][3], bar, p.b_mn, b_rows / 2, n0,
                            k0, q);
            }
          }
        }
      };
      Walk walk(l, worker, workers);
      int product;
      int64_t t;
      while (ok && walk.next(product, t)) {
        if (GATED || product == 0)
          load(std::integral_constant<int, 0>(), t);
        else
          load(std::integral_constant<int, 1>(), t);
      }
      // Every stage handed back: no load is in flight and no arrival from the
      // pair's MMAs still on its way here.  All stages in turn, from the next one
      // on: of one that was never filled the wait passes at once, and the last one
      // filled is the last one waited for.
      for (uint32_t i = 0; i < stages && ok; ++i) {
        take();
        next();
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (of the pair)
    if (lane == 0 && rank == 0) {
      uint32_t s = 0, ph = 0;  // stage and its phase
      uint32_t filled = 0;     // bit i: the parity of accumulator i's fillings
      // Before accumulator i is filled anew, the epilogue has read it.
      auto take = [&](int i) {
        ok = ff_wait(&acc_empty[i], ((filled >> i) & 1u) ^ 1u, l.wait_ns, abort_flag);
        filled ^= 1u << i;
        tc_fence_after();
        return ok;
      };
      int acc = A::LARGE - 1;  // the accumulator in use, of those taken in turn
      Walk walk(l, worker, workers);
      int product;
      int64_t t;
      while (ok && walk.next(product, t)) {
        const FfParams &p = l.p[product];
        const int bn = P == 1 ? p.bn : BN, a_mn = p.a_mn, b_mn = p.b_mn, kbs = p.kb * p.segs;
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) |
                               ((uint32_t)b_mn << 16) | ((uint32_t)(bn >> 3) << 17) |
                               ((uint32_t)((CG * 128) >> 4) << 24);
        // 16 along K: 32 bytes of a K-major line, two 8-deep groups MN-major
        const uint64_t astep = a_mn ? 2048 >> 4 : 32 >> 4, bstep = b_mn ? 2048 >> 4 : 32 >> 4;
        const uint32_t a_plane = (uint32_t)p.a_bytes, b_plane = (uint32_t)p.b_bytes;
        if (P == 1) {
          acc ^= 1;
          if (!take(acc)) break;
        }
        for (int kb = 0; kb < kbs; ++kb) {
          if (LONG && kb > 0 && kb % kLong == 0) {
            commit<CG>(&acc_full[acc]);
            if (!take(acc)) break;
          }
          if (!ff_wait(&full[s], ph, l.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem) + s * stage_bytes, b = a + P * a_plane;
          const uint64_t da = tile_desc(a, a_mn), db = tile_desc(b, b_mn);
          if (P == 3 && kb % kFlush == 0) {
            if (A::LARGE == 2) acc ^= 1;
            if (!take(acc)) break;
          }
          const uint32_t d = tmem_base + (uint32_t)(acc * A::COLS);
          const bool first = LONG ? kb % kLong == 0 : P == 1 ? kb == 0 : kb % kFlush == 0;
#pragma unroll
          for (int kk = 0; kk < kBlockK / 16; ++kk)
            mma_bf16<CG>(d, da + kk * astep, db + kk * bstep, idesc, first && kk == 0 ? 0u : 1u);
          if constexpr (P == 3) {
            if (kb % kFlush == kFlush - 1 || kb == kbs - 1) commit<CG>(&acc_full[acc]);
            if (kb == 0 && !take(A::SMALL)) break;
#pragma unroll
            for (int kk = 0; kk < kBlockK / 16; ++kk) {
#pragma unroll
              for (int sum = P - 1; sum >= 1; --sum) {
#pragma unroll
                for (int i = 0; i <= sum; ++i)
                  mma_bf16<CG>(tmem_base + (uint32_t)(A::SMALL * A::COLS),
                               da + kk * astep + (uint64_t)(i * (a_plane >> 4)),
                               db + kk * bstep + (uint64_t)((sum - i) * (b_plane >> 4)), idesc,
                               (kb > 0 || kk > 0 || sum < P - 1 || i > 0) ? 1u : 0u);
              }
            }
          }
          commit<CG>(&empty[s]);
          if (++s == stages) s = 0, ph ^= 1;
        }
        if (ok) commit<CG>(&acc_full[P == 1 ? acc : A::SMALL]);
        if (LONG && kbs > kLong) acc ^= 1;  // the other one holds the sum of the parts
      }
    }
  } else {
    // ---------------- epilogue: a warp has 32 rows (the tensor-memory lanes
    // 32 (w & 3) on) and every second 16 columns of the tile
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint8_t *st = epi + (warp - 2) * 4096;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    auto aligned = [](const void *q, int64_t ld, int64_t size) {
      return ((reinterpret_cast<uintptr_t>(q) | (uintptr_t)(ld * size)) & 15) == 0;
    };
    Writer<T, GATED> out;
    out.st = st;
    uint32_t drained = 0;  // bit i: the parity of accumulator i's drainings
    int acc = A::LARGE - 1;
    // tcgen05.ld is warp-collective: the warp proceeds or stops as one
    auto wait_full = [&](int i) {
      ok = __all_sync(0xffffffffu,
                      ff_wait(&acc_full[i], (drained >> i) & 1u, l.wait_ns, abort_flag));
      drained ^= 1u << i;
      tc_fence_after();
      return ok;
    };
    auto release = [&](int i) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader<CG>(&acc_empty[i]);
    };
    Walk walk(l, worker, workers);
    int product;
    int64_t t;
    while (ok && walk.next(product, t)) {
      const FfParams &p = l.p[product];
      const int out_cols = p.out_cols;
      out.N = p.N;
      out.act = p.act;
      out.ldg = p.ldg;
      out.ldu = p.ldu;
      const TileAt at = tile_at(p, t);
      const int64_t r0 = at.m * (CG * 128) + rank * 128 + quarter * 32;
      const int64_t c0 = at.n * out_cols;
      out.rows = (int)(p.M - r0 < 32 ? p.M - r0 : 32);
      out.ldc = p.ldc[at.batch];
      out.c = static_cast<T *>(p.c[at.batch]);
      out.vec_c = aligned(out.c, out.ldc, sizeof(T));
      out.vec_gu = aligned(p.g, p.ldg, 4) && aligned(p.u, p.ldu, 4);
      if (out.c) out.c += r0 * out.ldc;
      out.g = p.g ? p.g + r0 * p.ldg : nullptr;
      out.u = p.u ? p.u + r0 * p.ldu : nullptr;
      if constexpr (P == 1) {
        acc ^= 1;
        const uint32_t base = lane_base + (uint32_t)(acc * A::COLS);
        // A long sum comes in parts, which gather in the place of the accumulator
        // that the tile before this one had: this warp has read its share of it,
        // and the MMAs go on in the one that it reads last here.
        const int parts = LONG ? (p.kb * p.segs + kLong - 1) / kLong : 1;
        if (!wait_full(acc)) break;
        if constexpr (LONG) {
          const uint32_t sum = lane_base + (uint32_t)((acc ^ 1) * A::COLS);
          for (int part = 0; parts > 1; ++part) {
            const bool last = part == parts - 1;
            gather_part<GATED>(base, sum, last ? base : sum, part > 0, out_cols, 16 * half);
            if (last) break;
            release(acc);
            if (!wait_full(acc)) break;
          }
          if (!ok) break;
        }
        int j = 16 * half;
        if (j >= out_cols) release(acc);
#pragma unroll 1
        for (; j < out_cols; j += 32) {
          float v[16], w[16];
          tmem_ld16(base + (uint32_t)j, v);
          if constexpr (GATED) tmem_ld16(base + (uint32_t)(out_cols + j), w);
          tmem_ld_wait();
          if (j + 32 >= out_cols) release(acc);
          out.block(c0 + j, v, w);
        }
        if (LONG && parts > 1) acc ^= 1;
      } else {
        constexpr int COLS = GATED ? BN / 4 : BN / 2;  // output columns of a warp
        constexpr int BLOCKS = BN / 32;                // 16 columns of the sums each
        float sum[BLOCKS][16];
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
          for (int k = 0; k < 16; ++k) sum[i][k] = 0.0f;
        const int parts = (p.kb * p.segs + kFlush - 1) / kFlush + 1;
        for (int part = 0; part < parts; ++part) {
          const bool small = part == parts - 1;
          if (A::LARGE == 2 && !small) acc ^= 1;
          const int from = small ? A::SMALL : acc;
          if (!wait_full(from)) break;
#pragma unroll
          for (int i = 0; i < BLOCKS; ++i) {
            float x[16];
            tmem_ld16(lane_base + (uint32_t)(from * A::COLS + 16 * half + 32 * i), x);
            tmem_ld_wait();
            if (i == BLOCKS - 1) release(from);
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[i][k] += x[k];
          }
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < COLS / 16; ++i)
          out.block(c0 + 16 * half + 32 * i, sum[i], sum[GATED ? i + COLS / 16 : i]);
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
  if (warp == 1) ff_tmem_dealloc<CG>(tmem_base, kTmemCols);
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
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint64_t env_u64(const char *name, uint64_t dflt) {
  const char *v = std::getenv(name);
  return v && *v ? std::strtoull(v, nullptr, 10) : dflt;
}

// A tile: the CTAs that share it, its accumulator columns and the rows of A
// that each CTA loads.  Of a tile with few rows only those are loaded; the MMA
// reads what lies behind them in place of the others, which ends in rows of
// the accumulator that nothing reads.
struct Choice {
  int cg, bn, a_rows;
};

int stage_bytes_of(const Choice &c, int planes) {
  return planes * (c.a_rows + c.bn / c.cg) * kLine;
}

FfParams params_of(const FfProduct &q, const Choice &ch) {
  FfParams p{};
  p.M = q.M;
  p.N = q.N;
  p.kb = (int)ceil_div(q.K, kBlockK);
  p.segs = q.kind == kFfConcat ? 2 : 1;
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
  p.bn = ch.bn;
  p.out_cols = q.kind == kFfGated ? ch.bn / 2 : ch.bn;
  p.a_bytes = ch.a_rows * kLine;
  p.b_bytes = ch.bn / ch.cg * kLine;
  p.tiles_m = (int)ceil_div(q.M, ch.cg * 128);
  p.tiles_n = (int)ceil_div(q.N, p.out_cols);
  p.group_n = p.tiles_n < 8 ? p.tiles_n : 8;
  p.tiles = (int64_t)p.tiles_m * p.tiles_n * (q.kind == kFfBatch ? 2 : 1);
  return p;
}

// Estimated clocks of one tile.  An MMA (16 along K) takes bn / 2 clocks, or
// what shared memory needs at 128 bytes a clock for its reads (128 rows of A
// and all the tile's columns of B, those of the pair's other CTA too) and for
// the copies' writes, which serve the one or six products of their planes.
// (GB300, clocks a K block, modelled / measured: one plane 256 x 256 by pairs
// 640 / 640; three planes 256 x 256 3072 / 3360, 256 x 128 2112 / 2208, 128 x
// 128 2304 / 2200.)  A CTA's loads come at about 55 bytes a clock with the
// ring full of requests (one token, 128 KB in flight: 28 bytes with half of
// that).
double tile_clocks(const FfProduct &q, const Choice &c) {
  const double kbs = (double)ceil_div(q.K, kBlockK) * (q.kind == kFfConcat ? 2 : 1);
  const double products = q.planes == 1 ? 1 : 6, rows = 128 + c.bn;
  const double mma = 4 * products * c.bn / 2.0;
  const double smem = 4 * products * rows * 32 / 128 + stage_bytes_of(c, q.planes) / 128.0;
  const double load = stage_bytes_of(c, q.planes) / 55.0;
  const double most = mma > smem ? mma : smem;
  return kbs * (most > load ? most : load);
}

int64_t tiles_of(const FfProduct &q, const Choice &c) {
  return ceil_div(q.M, c.cg * 128) * ceil_div(q.N, q.kind == kFfGated ? c.bn / 2 : c.bn) *
         (q.kind == kFfBatch ? 2 : 1);
}

// Whether the product's operands can be cut into such tiles.  Three planes
// come in a few sizes, one plane in every width that the operands' storage
// lets TMA cut: blocks of 16 output columns, MN-major ones of 64, from one
// matrix or one half.
bool tile_fits(const FfProduct &q, int cg, int bn) {
  const bool gated = q.kind == kFfGated;
  const int parts = gated || cg == 2 ? 2 : 1;  // loads that share the columns
  const int unit = q.b[0].mn_major ? 64 * parts : gated || cg == 2 ? 32 : 16;
  if (bn % unit != 0) return false;
  if (q.planes == 1) return true;
  return cg == 2 ? bn == 256 || bn == 128 : bn == 128 || (bn == 64 && !gated);
}

Choice choice_of(const FfProduct &q, int cg, int bn) {
  const bool few = cg == 1 && !q.a[0].mn_major && q.M < 128;
  return {cg, bn, few ? (int)ceil_div(q.M, 8) * 8 : 128};
}

// The tiles of n products (one, or two of one launch) with the least
// estimated time.  One product: whole waves of its tiles and an epilogue that
// nothing hides, about 30 clocks a column.  Two, whose tiles are one list:
// all work spread evenly and one more tile of the second product, but no less
// than the first one's waves.  Two products share the CTAs of a tile, and
// with three planes the kernel's columns.
void choose(const FfProduct *q, int n, int sms, Choice *best) {
  struct Candidate {
    Choice c;
    double clocks, waves, even;  // of a tile; of all tiles, whole and spread
  };
  double least = 0.0;
  for (int cg = 2; cg >= 1; --cg) {
    const int64_t workers = sms / cg;
    Candidate list[2][16];
    int count[2] = {0, 0};
    for (int i = 0; i < n; ++i)
      for (int bn = 256; bn >= 32; bn -= 16) {
        if (!tile_fits(q[i], cg, bn)) continue;
        const Choice c = choice_of(q[i], cg, bn);
        const double clocks = tile_clocks(q[i], c);
        const int64_t tiles = tiles_of(q[i], c);
        list[i][count[i]++] = {c, clocks, clocks * (double)ceil_div(tiles, workers),
                               clocks * (double)tiles / (double)workers};
      }
    for (int i = 0; i < count[0]; ++i) {
      const Candidate &x = list[0][i];
      for (int j = 0; j < (n == 2 ? count[1] : 1); ++j) {
        double t = x.waves + 30.0 * x.c.bn;
        if (n == 2) {
          const Candidate &y = list[1][j];
          if (q[0].planes == 3 && x.c.bn != y.c.bn) continue;
          const double even = x.even + y.even + y.clocks + 15.0 * (x.c.bn + y.c.bn);
          if (even > t) t = even;
        }
        if (least == 0.0 || t < least) {
          least = t;
          best[0] = x.c;
          if (n == 2) best[1] = list[1][j].c;
        }
      }
    }
  }
}

template <int P, int CG, int BN, bool GATED, bool LONG>
int launch_cfg(const FfProduct *q, int n, const Choice *ch, const DeviceProps &dp,
               cudaStream_t s) {
  FfLaunch l{};
  int64_t workers = dp.sm_count / CG, tiles = 0;
  double clocks[2] = {0.0, 0.0};
  for (int i = 0; i < n; ++i) {
    l.p[i] = params_of(q[i], ch[i]);
    tiles += l.p[i].tiles;
    clocks[i] = tile_clocks(q[i], ch[i]);
    const int stage = stage_bytes_of(ch[i], P);
    if (stage > l.stage_bytes) l.stage_bytes = stage;
    // columns of B one load brings: the gated form takes each half of a single
    // CTA's columns, or all of one CTA of a pair, from one of the two matrices
    const int b_load = GATED && CG == 1 ? ch[i].bn / 2 : ch[i].bn / CG;
    for (int k = 0; k < 2; ++k) {
      const FfOperand &a = q[i].a[k].p ? q[i].a[k] : q[i].a[0];
      const FfOperand &b = q[i].b[k].p ? q[i].b[k] : q[i].b[0];
      if (!encode(&l.map[i][k], a, P, a.mn_major ? 64 : ch[i].a_rows) ||
          !encode(&l.map[i][2 + k], b, P, b.mn_major ? 64 : b_load))
        return GEMM_ERR_UNSUPPORTED;
    }
  }
  if (workers > tiles) workers = tiles;
  l.stages = kStageBudget / l.stage_bytes < kMaxStages ? kStageBudget / l.stage_bytes : kMaxStages;
  l.early_from = l.p[0].tiles % workers;
  if (n == 2 && l.early_from > 0) {
    const int64_t share = ceil_div(l.p[1].tiles, workers - l.early_from);
    l.early = (int64_t)(clocks[0] / clocks[1]);
    if (l.early > share) l.early = share;
  }
  // The epilogue's one wait is for a whole sum, 0.3 us a block of K in BF16 (2 s
  // alone would end sums over 4.7e8 tokens), and the pair's other CTA may be a
  // block of FP32, 2 us, behind: the limit grows with the sum.
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t k = (int64_t)l.p[i].kb * l.p[i].segs;
    if (k > blocks) blocks = k;
  }
  l.wait_ns = env_u64("GEMM_DEBUG_WAIT_LIMIT_NS", 2000000000ull) + (uint64_t)blocks * 8000;
  l.stall_producer = (int)env_u64("GEMM_DEBUG_STALL_PRODUCER", 0);

  auto kern = ff_tc_kernel<P, CG, BN, GATED, LONG>;
  static Once once;
  if (allow_shared_memory(once, kern, 227 * 1024, dp.device) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(workers * CG));
  lc.blockDim = dim3(kThreadsFF);
  lc.dynamicSmemBytes = l.stages * l.stage_bytes + 1024 + 256 + kEpiBytes;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 2;
  if (cudaLaunchKernelEx(&lc, kern, l) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

template <int P, bool GATED>
int launch_any(const FfProduct *q, int n, const DeviceProps &dp, cudaStream_t s) {
  Choice c[2];
  choose(q, n, dp.sm_count, c);
  if constexpr (P == 1) {
    bool is_long = false;
    for (int i = 0; i < n; ++i)
      is_long = is_long || ceil_div(q[i].K, kBlockK) * (q[i].kind == kFfConcat ? 2 : 1) > kLong;
    if (is_long)
      return c[0].cg == 2 ? launch_cfg<1, 2, 0, GATED, true>(q, n, c, dp, s)
                          : launch_cfg<1, 1, 0, GATED, true>(q, n, c, dp, s);
    return c[0].cg == 2 ? launch_cfg<1, 2, 0, GATED, false>(q, n, c, dp, s)
                        : launch_cfg<1, 1, 0, GATED, false>(q, n, c, dp, s);
  } else {
    if (c[0].cg == 2)
      return c[0].bn == 256 ? launch_cfg<3, 2, 256, GATED, false>(q, n, c, dp, s)
                            : launch_cfg<3, 2, 128, GATED, false>(q, n, c, dp, s);
    if constexpr (!GATED)
      if (c[0].bn == 64) return launch_cfg<3, 1, 64, false, false>(q, n, c, dp, s);
    return launch_cfg<3, 1, 128, GATED, false>(q, n, c, dp, s);
  }
}

}  // namespace

int launch_ff_products(const FfProduct *q, int n, const DeviceProps &dp, cudaStream_t s) {
  if (!tc_supported(dp)) return GEMM_ERR_UNSUPPORTED;
  if (!get_encoder()) return GEMM_ERR_CUDA;
  if (q[0].planes == 1)
    return q[0].kind == kFfGated ? launch_any<1, true>(q, n, dp, s)
                                 : launch_any<1, false>(q, n, dp, s);
  return q[0].kind == kFfGated ? launch_any<3, true>(q, n, dp, s)
                               : launch_any<3, false>(q, n, dp, s);
}

int ff_read_and_clear_status(cudaStream_t s) {
  int v = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_ff_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(g_ff_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) !=
            cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_CUDA;
    }
  }
  return v;
}

}  // namespace gg
