// Products with 4-bit weights for a few tokens (include/gb300_gemm.h,
// q4_matmul and q4_gated).
//
// Y^T = W X^T on mma.sync tiles of 16 weight rows x 8 columns of X^T, BF16 in,
// FP32 sums.  What bounds the product itself is reading the codes once (N K / 2
// bytes).  So each warp copies its own rows' codes to shared memory ahead of
// their use, asynchronously, 128 bytes of a row at a time, with no barrier between
// warps; and the arithmetic per code is kept small: a 32-bit word of eight codes becomes four BF16 pairs
// 128 + q, exact, by 3 shifts and 4 three-input logic operations that mask and
// or in the exponent of 128 (integers put under the exponent of a float whose
// last place is 1; Kim et al., "Who Says Elephants Can't Run", 2022, have it for
// 4-bit weights).
//
// GB300, from cold caches, BF16, groups of 128: 1 token by 2 x 14336 x 4096
// (60.6 MB) 20.7 us, 2.9 TB/s, the ALU pipe 50 % and the issue slots 49 %
// busy: what the codes' conversion costs, with the ramp of a short kernel on
// both sides.  16 tokens by 8192 x 28672 (132 MB) 61.5 us, 2.1 TB/s: without
// the copies 49, without x's loads 55, the copies alone 29; the arithmetic is
// no faster with 16 warps (MMA and ALU work add up).  1 token by 4096 x 4096 (8.7 MB) 6.2
// us: one pass of latency, and a launch that does not overlap the kernel before.
//
// Scales multiply the FP32 sums of one group, from which (128 + z) sum x is
// taken first, with the sums of x from MMAs whose weights are ones; that
// difference costs about 5 of FP32's 24 bits, which a BF16 result does not
// show.  With FP32 X the pairs are made q - 8 instead (exact, one paired
// subtraction each) and only (z - 8) sum x is taken off.
//
// An MMA sums 16 values of k in any order, so a thread's eight codes of one
// word are the k that it feeds to two MMAs, and X is loaded to match.  All k
// of an MMA belong to one group: the four threads of a row take 32 W values of
// k, W = 1, 2, 4 words each for groups of 32, 64, 128 (or 256).
//
// FP32 X is split into three BF16 (24 bits) that take three columns of an MMA
// each token, so a tile holds 2 tokens, and 8 in BF16.  4 tokens by 4096 x
// 14336 take 28.7 us; the step from planes that are rounded to planes that are
// cut took the same from 93 to 31.
//
// A CTA has one block of rows and its warps split k; their sums meet in shared
// memory in a fixed order.  Where the blocks of rows are few and long, a
// cluster of up to 8 CTAs shares one, and reads one another's sums: 1 token by
// 512 x 16384 8.3 us, 14.4 with one CTA a block.
//
// Rows that do not start on 16-byte boundaries are copied by the aligned
// pieces that they lie in and shifted in shared memory (3 tokens by 2 x 758 x
// 21645, group 32: 37 us; 82 with loads through registers and no clusters).
#include "ff.cuh"

namespace gg {
namespace {

struct Q4Side {
  const uint8_t *q;
  int64_t ldq;
  const void *s, *z;
};
struct Q4Args {
  int64_t M, N, K, ldx, ldy, groups;
  int act, group;
  const void *x;
  void *y;
  Q4Side w[2];
  uint32_t mask;    // 0x000f000f
  int group_shift;  // group = 1 << group_shift
  int vec_x;        // rows of X start on 16-byte boundaries
  int aligned, scales_aligned;  // rows of codes on 16 bytes; a step's scales on theirs
  int split;                    // CTAs (a cluster) that share a block of rows, each a part of k
};

constexpr int kMaxWarps = 16;  // of a CTA: its parts of k

__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, int bytes) {
  if (bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else if (bytes == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// The first `bytes` of 16, zeros for the rest.
__device__ __forceinline__ void cp_async_part(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Of a launch without clusters: 0 and blockIdx.x.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_id() {
  uint32_t r;
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive;\nbarrier.cluster.wait;" ::: "memory");
}
// A float of the shared memory of the cluster's CTA `rank`, at `p` in this one's.
__device__ __forceinline__ float load_of(const float *p, uint32_t rank) {
  float v;
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n"
               " ld.shared::cluster.f32 %0, [a];\n}"
               : "=f"(v)
               : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank)
               : "memory");
  return v;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from a sum of zero.
__device__ __forceinline__ void mma_16816_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                                uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Codes i and i + 4 of a word as the BF16 pair 128 + q or (EXACT) q - 8.
// `mask` is 0x000f000f out of a register: mask and exponent as two immediates
// would take two instructions.
template <bool EXACT, int I>
__device__ __forceinline__ uint32_t codes(uint32_t w, uint32_t mask) {
  uint32_t u;
  asm("lop3.b32 %0, %1, %2, 0x43004300, 0xea;" : "=r"(u) : "r"(w >> (4 * I)), "r"(mask));
  if (!EXACT) return u;
  __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162 *>(&u);
  h = __hsub2(h, __nv_bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308)));
  return *reinterpret_cast<uint32_t *>(&h);
}

// The column `g` of X^T that a lane feeds: token and plane (FP32: three a token).
template <typename T>
__device__ __forceinline__ int column_token(int g) {
  return sizeof(T) == 4 ? g / 3 : g;
}
template <typename T>
constexpr int kTileTokens = sizeof(T) == 4 ? 2 : 8;

// Eight values of x as they come: 16 bytes of BF16 or 32 of FP32.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};

// The pairs (x_i, x_i+4), i = 0..3, of plane `plane`.  FP32 is cut, not
// rounded, into its planes, which cannot overflow and takes four operations a
// value: the first two 8 bits of the fraction with their leading one, the last
// what is left, 8 bits too.  An Inf leaves NaN in its second and third, for
// which formula_sums() answers.
__device__ __forceinline__ void pairs(const Raw8<bf16> &r, int, uint32_t (&b)[4]) {
  const uint4 v = r.v[0];
  b[0] = __byte_perm(v.x, v.z, 0x5410);
  b[1] = __byte_perm(v.x, v.z, 0x7632);
  b[2] = __byte_perm(v.y, v.w, 0x5410);
  b[3] = __byte_perm(v.y, v.w, 0x7632);
}
__device__ __forceinline__ uint32_t plane_of(float x, int plane) {
  const uint32_t first = plane > 0 ? 0xffff0000u : 0u, second = plane > 1 ? 0xffff0000u : 0u;
  x -= __uint_as_float(__float_as_uint(x) & first);
  x -= __uint_as_float(__float_as_uint(x) & second);
  return __float_as_uint(x);
}
__device__ __forceinline__ void pairs(const Raw8<float> &r, int plane, uint32_t (&b)[4]) {
  const float *f = reinterpret_cast<const float *>(r.v);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    b[i] = __byte_perm(plane_of(f[i], plane), plane_of(f[i + 4], plane), 0x7632);
}

// W: words of codes that a thread takes of a row and group (a group is 32 W
// values of k, or twice that).  TI: 16-row tiles of a warp (gated: half of
// each matrix).  NT: tiles of columns.
template <typename T, int W, int TI, int NT, bool GATED>
struct Q4Cfg {
  static constexpr int STEP = 256;                  // k of one step: 128 bytes of codes a row
  static constexpr int PARTS = STEP / (32 * W);     // groups of a step
  static constexpr int COLS = NT * 8;
  static constexpr int TILES = GATED ? TI / 2 : TI; // of one matrix
  static constexpr int ROWS = TILES * 16;
  static constexpr int STAGES = 2;
  static constexpr int SCALES = TI * 16 * PARTS * (int)sizeof(T);  // bytes, one stage
  static constexpr int SLOT = TI * 16 * 128 + 2 * SCALES;          // codes, scales, zero points
  // unaligned rows: one 16-byte piece more of each, behind all the rings
  static constexpr int TAIL = TI * 16 * 16, WARP_TAILS = STAGES * TAIL;
  static_assert(!GATED || TI % 2 == 0, "");
  // the ring of a warp, or its share of the sums
  static constexpr int RING = STAGES * SLOT, RED = TI * 16 * COLS * 4;
  static constexpr int WARP_BYTES = RING > RED ? RING : RED;
  // Warps that an SM holds.  With four tiles 8 run faster than 12 (16 x 8192 x
  // 28672: 68 against 78 us when they were chosen, 61.5 with 8 now): what shared memory they leave is L1 for x.  With
  // two and two of columns of large groups 12, by their registers (16 x 2048 x
  // 8192: 12.4 us, with 16 warps 16.5), and 8 in FP32 (4 x 4096 x 14336: 28.7
  // us, with 12 32.7).
  static constexpr int BY_SMEM = 226 * 1024 / WARP_BYTES,
                       BY_REGS = TI == 4 ? 8 : NT == 2 && W == 4 ? (sizeof(T) == 4 ? 8 : 12) : 16;
  static constexpr int SM_WARPS = BY_SMEM < BY_REGS ? BY_SMEM / 4 * 4 : BY_REGS;
  static constexpr int MAX_WARPS = SM_WARPS < kMaxWarps ? SM_WARPS : kMaxWarps;
};

// Eight values of x from k on, zeros from K on.
template <typename T>
__device__ __forceinline__ void load_x(const Q4Args &p, const T *x, int64_t k, float (&v)[8]) {
  __align__(16) T t[8];
  if (p.vec_x && k + 8 <= p.K) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4 *>(t)[i] = __ldg(reinterpret_cast<const uint4 *>(x + k) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = k + i < p.K ? x[k + i] : from_f32<T>(0.0f);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
}

// Whether token m has a NaN, by one warp.
template <typename T>
__device__ __noinline__ bool has_nan(const Q4Args &p, int64_t m) {
  const T *x = static_cast<const T *>(p.x) + m * p.ldx;
  bool nan = false;
#pragma unroll 4
  for (int64_t k = (threadIdx.x & 31) * 8; k < p.K; k += 256) {
    float v[8];
    load_x(p, x, k, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) nan = nan || v[i] != v[i];
  }
  return __any_sync(0xffffffffu, nan);
}

// sum_k x(m,k) W(n + i,k), i = 0..7, of one matrix again, by the formula, by one
// warp: for the sums that the tiles' arithmetic leaves Inf or NaN.  Those
// include an Inf of X (which leaves NaN there) and sums that are finite: in BF16
// a group's 128 + q and in FP32 its q - 8 can pass FP32's range where s (q - z)
// x does not.  Eight codes' products in FP32, scaled by 2^-16 where an x is
// beyond 2^112, so that none of them and no sum of them overflows for any zero
// point below 2^9; the scales and the sum in 64 bits, which hold every product.
// Lane i gets row i's sum; rows that the matrix does not have stand for its last.
// What costs here is latency: 16 tokens by 8192 x 28672 take 61 us, 1.1 ms where
// one token has an Inf and 0.1 where it has a NaN, for which has_nan() answers.
template <typename T>
__device__ __noinline__ float formula_sums(const Q4Args &p, int side, int64_t m, int64_t n) {
  constexpr int R = 8;
  const int lane = threadIdx.x & 31;
  const Q4Side &w = p.w[side];
  const T *x = static_cast<const T *>(p.x) + m * p.ldx;
  double sum[R];
#pragma unroll
  for (int j = 0; j < R; ++j) sum[j] = 0.0;
  for (int64_t k = lane * 8; k < p.K; k += 256) {
    float v[8], most = 0.0f;
    load_x(p, x, k, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i]));
    const bool large = most >= 0x1p112f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = large ? v[i] * 0x1p-16f : v[i];
    const int there = (int)(p.K - k < 8 ? p.K - k : 8);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t row = n + j < p.N ? n + j : p.N - 1, at = row * p.groups + (k >> p.group_shift);
      const uint8_t *q = w.q + row * w.ldq + k / 2;
      const float zero = w.z ? to_f32(static_cast<const T *>(w.z)[at]) : 8.0f;
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < there) part = fmaf((float)(q[i / 2] >> (i % 2 * 4) & 15) - zero, v[i], part);
      sum[j] = fma((double)to_f32(static_cast<const T *>(w.s)[at]),
                   (double)part * (large ? 0x1p16 : 1.0), sum[j]);
    }
  }
  float mine = 0.0f;
#pragma unroll
  for (int j = 0; j < R; ++j) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
    if (lane == j) mine = (float)sum[j];
  }
  return mine;
}

template <typename T, int W, int TI, int NT, bool GATED>
__global__ void __launch_bounds__(Q4Cfg<T, W, TI, NT, GATED>::SM_WARPS * 32, 1)
q4_kernel(const Q4Args p) {
  using Cfg = Q4Cfg<T, W, TI, NT, GATED>;
  constexpr int STEP = Cfg::STEP, PARTS = Cfg::PARTS, STAGES = Cfg::STAGES, RW = TI * 16;
  constexpr int COLS = Cfg::COLS, TILES = Cfg::TILES, ROWS = Cfg::ROWS;
  constexpr bool EXACT = sizeof(T) == 4;
  extern __shared__ __align__(128) uint8_t shared[];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int warps = blockDim.x >> 5, rank = (int)cluster_rank();
  const int part_of_k = rank * warps + warp, parts_of_k = p.split * warps;
  uint8_t *ring = shared + warp * Cfg::WARP_BYTES;
  uint8_t *tails = shared + warps * Cfg::WARP_BYTES + warp * Cfg::WARP_TAILS;
  const bool has_z = p.w[0].z != nullptr;
  const uint32_t mask = p.mask;
  const int64_t m0 = (int64_t)blockIdx.y * (kTileTokens<T> * NT);
  const int64_t n0 = (int64_t)cluster_id() * ROWS;
  const int left = (int)(p.N - n0 < ROWS ? p.N - n0 : ROWS);
  const int steps = (int)((p.K + STEP - 1) / STEP);
  const int mine = steps > part_of_k ? (steps - part_of_k + parts_of_k - 1) / parts_of_k : 0;
  const int64_t row_bytes = (p.K + 1) / 2;
  // Rows that the matrix does not have stand for its last one: what is
  // computed of them is not stored.
  auto weight_row = [&](int r) { return n0 + (r < left ? r : left - 1); };

  // Row r's 16-byte piece c, placed so that the four threads of a row and its
  // neighbours meet every bank once, whether they read 4, 8 or 16 bytes each.
  auto piece = [](int r, int c) {
    return r * 128 + ((c ^ ((r & 1) << 2 | (r & 2) | ((r >> 2) & 1))) * 16);
  };

  // Where this lane's copies begin: 16 bytes of every fourth row.
  const int lr = lane >> 3, lc = lane & 7;
  const uint8_t *from[GATED ? 2 : 1];
#pragma unroll
  for (int k = 0; k < (GATED ? 2 : 1); ++k) from[k] = p.w[k].q + n0 * p.w[k].ldq + lc * 16;
  const int to[2] = {piece(lr, lc), piece(4 + lr, lc) - 512};

  // Step `c`'s codes, scales and zero points of all the warp's rows, to slot `st`.
  auto copy = [&](int c, int st) {
    uint8_t *slot = ring + st * Cfg::SLOT, *tail = tails + st * Cfg::TAIL;
    const int64_t at = (int64_t)c * (STEP / 2);
    auto source = [&](int i) {  // of rows 4 i on
      const int k = i * 4 / ROWS, r = i * 4 % ROWS + lr;
      return from[k] + at + (uint64_t)(uint32_t)(r < left ? r : left - 1) * (uint32_t)p.w[k].ldq;
    };
    if (p.aligned && at + STEP / 2 <= row_bytes) {
      const uint32_t dst = (uint32_t)__cvta_generic_to_shared(slot);
#pragma unroll
      for (int i = 0; i < RW / 4; ++i) cp_async(dst + to[i & 1] + i * 512, source(i), 16);
    } else {
      // unaligned rows, and the ends of the rows: the aligned 16 bytes that a
      // piece begins in (realign() shifts them), without what lies outside the
      // matrix; x is zero where the codes then are
      auto fetch = [&](int k, uint8_t *to_byte, const uint8_t *src) {
        const uint8_t *first = p.w[k].q, *end = first + (p.N - 1) * p.w[k].ldq + row_bytes;
        if (src >= first) {
          const int64_t bytes = end - src;
          if (bytes <= 0) src = end - 1 - (reinterpret_cast<uintptr_t>(end - 1) & 15);
          cp_async_part((uint32_t)__cvta_generic_to_shared(to_byte), src,
                        bytes >= 16 ? 16 : bytes > 0 ? (int)bytes : 0);
        } else {
          for (int b = 0; b < 16; ++b)
            to_byte[b] = src + b >= first && src + b < end ? src[b] : (uint8_t)0;
        }
      };
#pragma unroll 4
      for (int i = 0; i < RW / 4; ++i) {
        const uint8_t *src = source(i);
        fetch(i * 4 / ROWS, slot + i * 512 + to[i & 1], src - (reinterpret_cast<uintptr_t>(src) & 15));
      }
#pragma unroll
      for (int i = 0; i < RW; i += 32) {
        const int e = i + lane, k = e / ROWS, r = e % ROWS;
        const uint8_t *src = p.w[k].q + at + weight_row(r) * p.w[k].ldq;
        const int off = (int)(reinterpret_cast<uintptr_t>(src) & 15);
        if (off) fetch(k, tail + e * 16, src - off + 128);
      }
    }
    // scales and zero points: PARTS a row, in the order of k
    const int64_t grp = ((int64_t)c * STEP) >> p.group_shift;
    T *ds = reinterpret_cast<T *>(slot + RW * 128);
    constexpr int BYTES = PARTS * (int)sizeof(T), PIECE = BYTES < 16 ? BYTES : 16;
    constexpr int PER = BYTES / PIECE;  // pieces of a row
    if (p.scales_aligned && grp + PARTS <= p.groups) {
#pragma unroll
      for (int i = 0; i < RW * PER / 32; ++i) {
        const int e = i * 32 + lane, r = e / PER, k = r / ROWS, o = e % PER * (PIECE / (int)sizeof(T));
        const Q4Side &w = p.w[GATED ? k : 0];
        const int64_t from = weight_row(r - k * ROWS) * p.groups + grp + o;
        T *dst = ds + r * PARTS + o;
        cp_async((uint32_t)__cvta_generic_to_shared(dst), static_cast<const T *>(w.s) + from, PIECE);
        if (has_z)
          cp_async((uint32_t)__cvta_generic_to_shared(dst + RW * PARTS),
                   static_cast<const T *>(w.z) + from, PIECE);
      }
    } else {
      // four loads at a time, then their stores: one wait for all four
      auto gather = [&](bool zero, T *dst) {
        constexpr int EACH = RW * PARTS / 32, AT_ONCE = EACH < 4 ? EACH : 4;
#pragma unroll 1
        for (int i = 0; i < EACH; i += AT_ONCE) {
          T v[AT_ONCE];
#pragma unroll
          for (int j = 0; j < AT_ONCE; ++j) {
            const int e = (i + j) * 32 + lane, r = e / PARTS, k = r / ROWS;
            const int64_t gr = ((int64_t)c * STEP + e % PARTS * (32 * W)) >> p.group_shift;
            const Q4Side &w = p.w[GATED ? k : 0];
            const T *from = static_cast<const T *>(zero ? w.z : w.s);
            v[j] = gr < p.groups ? from[weight_row(r - k * ROWS) * p.groups + gr] : from_f32<T>(0.0f);
          }
#pragma unroll
          for (int j = 0; j < AT_ONCE; ++j) dst[(i + j) * 32 + lane] = v[j];
        }
      };
      gather(false, ds);
      if (has_z) gather(true, ds + RW * PARTS);
    }
  };
  // Shifts the rows of a slot to where aligned ones lie: a row's codes begin
  // its address's last four bits into its first piece, in every step alike.
  auto realign = [&](int st) {
    uint8_t *slot = ring + st * Cfg::SLOT;
    const uint8_t *tail = tails + st * Cfg::TAIL;
#pragma unroll 2
    for (int i = 0; i < RW / 4; ++i) {
      const int k = i * 4 / ROWS, r = i * 4 % ROWS + lr, e = i * 4 + lr;
      const uint32_t off = ((uint32_t)reinterpret_cast<uintptr_t>(p.w[k].q) +
                            (uint32_t)weight_row(r) * (uint32_t)p.w[k].ldq) & 15;
      uint4 *here = reinterpret_cast<uint4 *>(slot + i * 512 + to[i & 1]);
      const uint4 a = *here;
      const uint4 b = *reinterpret_cast<const uint4 *>(
          lc < 7 ? slot + piece(e, lc + 1) : tail + e * 16);
      uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 6; ++j) v[j] = off & 8 ? v[j + 2] : v[j];
#pragma unroll
      for (int j = 0; j < 5; ++j) v[j] = off & 4 ? v[j + 1] : v[j];
      __syncwarp();
      *here = make_uint4(__funnelshift_r(v[0], v[1], 8 * (off & 3)),
                         __funnelshift_r(v[1], v[2], 8 * (off & 3)),
                         __funnelshift_r(v[2], v[3], 8 * (off & 3)),
                         __funnelshift_r(v[3], v[4], 8 * (off & 3)));
    }
    __syncwarp();
  };

  // This lane's column of each tile of X^T.  A column without a token stands
  // for another one; its sums are not stored.
  const int plane = sizeof(T) == 4 ? g % 3 : 0;
  const T *xrow[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int64_t m = m0 + nt * kTileTokens<T> + column_token<T>(g);
    xrow[nt] = static_cast<const T *>(p.x) + (m < p.M ? m : p.M - 1) * p.ldx + t * (8 * W);
  }
  // The x of the group that begins at k0: loaded a group ahead
  Raw8<T> raw[NT][W];
  auto fetch_x = [&](int64_t k0) {
    if (p.vec_x != 0 && k0 + 32 * W <= p.K) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
          for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            raw[nt][j].v[i] =
                __ldg(reinterpret_cast<const uint4 *>(xrow[nt] + k0) + j * (sizeof(T) / 2) + i);
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const int64_t n = p.K - k0 - t * (8 * W) - 8 * j;
          __align__(16) T v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = i < n ? xrow[nt][k0 + 8 * j + i] : from_f32<T>(0.0f);
#pragma unroll
          for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            raw[nt][j].v[i] = reinterpret_cast<const uint4 *>(v)[i];
        }
    }
  };

#pragma unroll 1
  for (int st = 0; st < STAGES - 1; ++st) {
    if (st < mine) copy(part_of_k + st * parts_of_k, st);
    cp_async_commit();
  }
  float acc[TI][NT][4];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.0f;

  if (mine > 0) fetch_x((int64_t)part_of_k * STEP);
#pragma unroll 1
  for (int it = 0; it < mine; ++it) {
    const int c = part_of_k + it * parts_of_k, st = it % STAGES;
    cp_async_wait<STAGES - 2>();
    __syncwarp();  // this step is here, and every lane is done with the one before
    if (it + STAGES - 1 < mine) copy(c + (STAGES - 1) * parts_of_k, (it + STAGES - 1) % STAGES);
    cp_async_commit();
    const uint8_t *slot = ring + st * Cfg::SLOT;
    if (!p.aligned) realign(st);
    const T *ds = reinterpret_cast<const T *>(slot + RW * 128);
#pragma unroll 1
    for (int part = 0; part < PARTS; ++part) {
      uint32_t b[NT][W][4];  // as the MMAs take it
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < W; ++j) pairs(raw[nt][j], plane, b[nt][j]);
      if (part + 1 < PARTS)
        fetch_x((int64_t)c * STEP + (part + 1) * (32 * W));
      else if (it + 1 < mine)
        fetch_x((int64_t)(c + parts_of_k) * STEP);
      float xs[NT][4];
      if (!EXACT || has_z) {
        constexpr uint32_t one = 0x3f803f80u;
#pragma unroll
        for (int j = 0; j < 2 * W; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t b0 = b[nt][j / 2][j % 2 * 2], b1 = b[nt][j / 2][j % 2 * 2 + 1];
            if (j == 0)
              mma_16816_first(xs[nt], one, one, one, one, b0, b1);
            else
              mma_16816(xs[nt], one, one, one, one, b0, b1);
          }
      }
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        uint32_t w[2][W];
        float s[2], z[2];  // scales; what is taken off of each code still
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = i * 16 + 8 * h + g;
          const uint8_t *src = slot + piece(r, (part * 4 * W + t * W) / 4) + t * W % 4 * 4;
          if constexpr (W == 4)
            *reinterpret_cast<uint4 *>(w[h]) = *reinterpret_cast<const uint4 *>(src);
          else if constexpr (W == 2)
            *reinterpret_cast<uint2 *>(w[h]) = *reinterpret_cast<const uint2 *>(src);
          else
            w[h][0] = *reinterpret_cast<const uint32_t *>(src);
          s[h] = to_f32(ds[r * PARTS + part]);
          z[h] = (EXACT ? 8.0f : -128.0f) - (has_z ? to_f32(ds[(RW + r) * PARTS + part]) : 8.0f);
        }
        // two sums a tile: an MMA that adds to the one before it waits 31 clocks
        // for it, and one can begin every 9
        float d[NT][4], d2[NT][4];
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t a0 = codes<EXACT, 0>(w[0][j], mask), a1 = codes<EXACT, 0>(w[1][j], mask),
                         a2 = codes<EXACT, 1>(w[0][j], mask), a3 = codes<EXACT, 1>(w[1][j], mask),
                         a4 = codes<EXACT, 2>(w[0][j], mask), a5 = codes<EXACT, 2>(w[1][j], mask),
                         a6 = codes<EXACT, 3>(w[0][j], mask), a7 = codes<EXACT, 3>(w[1][j], mask);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (j == 0)
              mma_16816_first(d[nt], a0, a1, a2, a3, b[nt][j][0], b[nt][j][1]);
            else
              mma_16816(d[nt], a0, a1, a2, a3, b[nt][j][0], b[nt][j][1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (j == 0)
              mma_16816_first(d2[nt], a4, a5, a6, a7, b[nt][j][2], b[nt][j][3]);
            else
              mma_16816(d2[nt], a4, a5, a6, a7, b[nt][j][2], b[nt][j][3]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = d[nt][e] + d2[nt][e];
            if (!EXACT || has_z) v = fmaf(z[e >> 1], xs[nt][e], v);
            acc[i][nt][e] = fmaf(s[e >> 1], v, acc[i][nt][e]);
          }
      }
    }
  }

  // The warps' sums, added in order; then, FP32, the planes.  They take the
  // place of the rings, which every warp has emptied.
  cp_async_wait<0>();
  __syncthreads();
  float *red = reinterpret_cast<float *>(shared);  // [warp][tile row][column]
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2 *>(red + ((warp * TI + i) * 16 + 8 * h + g) * COLS + nt * 8 +
                                    2 * t) = make_float2(acc[i][nt][2 * h], acc[i][nt][2 * h + 1]);
  __syncthreads();
  if (p.split > 1) {
    // this CTA's sums, in place of its first warp's, for the cluster to read
    for (int e = tid; e < RW * COLS; e += blockDim.x) {
      float v = 0.0f;
#pragma unroll 4
      for (int w = 0; w < warps; ++w) v += red[w * RW * COLS + e];
      red[e] = v;
    }
    cluster_sync();
  }
  constexpr int TOKENS = kTileTokens<T> * NT;
  auto total = [&](int r, int m) {
    float v = 0.0f;
    constexpr int PLANES = sizeof(T) == 4 ? 3 : 1;
    const int col = m / kTileTokens<T> * 8 + m % kTileTokens<T> * PLANES;
#pragma unroll
    for (int q = PLANES - 1; q >= 0; --q)
      if (p.split > 1) {
        for (int cta = 0; cta < p.split; ++cta) v += load_of(red + r * COLS + col + q, cta);
      } else {
#pragma unroll 4
        for (int w = 0; w < warps; ++w) v += red[(w * RW + r) * COLS + col + q];
      }
    return v;
  };
  const int tokens = (int)(p.M - m0 < TOKENS ? p.M - m0 : TOKENS), all = ROWS * tokens;
  // a warp's 32 outputs at a time: all its lanes take part in formula_sums(),
  // which has eight rows of one token
  for (int e0 = rank * (int)blockDim.x + tid - lane; e0 < all; e0 += p.split * (int)blockDim.x) {
    const int e = e0 + lane, r = e % ROWS, m = e / ROWS;
    const bool here = e < all && r < left;
    float y = 0.0f, u = 0.0f;
    if (here) {
      y = total(r, m);
      if constexpr (GATED) u = total(ROWS + r, m);
    }
    const bool bad = !isfinite(y) || !isfinite(u);
    const uint32_t again = __ballot_sync(0xffffffffu, bad);
    for (int of = 0; again != 0 && of < 32; of += 8) {
      if ((again >> of & 0xffu) == 0) continue;
      const int64_t om = m0 + (e0 + of) / ROWS, on = n0 + (e0 + of) % ROWS;
      float v[2] = {__int_as_float(0x7fc00000), __int_as_float(0x7fc00000)};
      if (!has_nan<T>(p, om)) {
#pragma unroll
        for (int k = 0; k < (GATED ? 2 : 1); ++k) v[k] = formula_sums<T>(p, k, om, on);
      }
#pragma unroll
      for (int k = 0; k < (GATED ? 2 : 1); ++k)
        v[k] = __shfl_sync(0xffffffffu, v[k], lane & 7);
      if (bad && lane >= of && lane < of + 8) y = v[0], u = GATED ? v[1] : 0.0f;
    }
    if (!here) continue;
    if constexpr (GATED)
      with_act(p.act, [&](auto a) { y = act_of<T, decltype(a)::value>(y) * u; });
    static_cast<T *>(p.y)[(m0 + m) * p.ldy + n0 + r] = from_f32<T>(y);
  }
  if (p.split > 1) cluster_sync();  // the others have read this CTA's sums
}

template <typename T, int W, int TI, int NT, bool GATED>
cudaError_t launch_q4(Q4Args p, cudaStream_t s, const DeviceProps &dp) {
  using Cfg = Q4Cfg<T, W, TI, NT, GATED>;
  constexpr int MOST = (Cfg::WARP_BYTES + Cfg::WARP_TAILS) * Cfg::MAX_WARPS;
  static_assert(MOST <= 227 * 1024 && Cfg::MAX_WARPS >= 4, "");
  auto kern = q4_kernel<T, W, TI, NT, GATED>;
  static Once once;
  const cudaError_t e = allow_shared_memory(once, kern, MOST, dp.device);
  if (e != cudaSuccess) return e;
  // Warps: as many as fill the SMs, but no more than there are steps.  Blocks
  // of rows that leave SMs idle are split along k, while that gives a warp
  // fewer steps.
  const int64_t passes = ceil_div(p.M, kTileTokens<T> * NT);
  const int64_t ctas = ceil_div(p.N, Cfg::ROWS), steps = ceil_div(p.K, Cfg::STEP);
  int64_t warps = (int64_t)Cfg::SM_WARPS * dp.sm_count / ctas;
  warps = warps < 4 ? 4 : warps > Cfg::MAX_WARPS ? Cfg::MAX_WARPS : warps;
  int split = 1;
  while (split < 8 && 2 * split * ctas * passes <= dp.sm_count && steps > split * warps) split *= 2;
  if (warps * split > steps) warps = steps < 1 ? 1 : ceil_div(steps, split);
  p.split = split;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(ctas * split), (unsigned)passes);
  lc.blockDim = dim3((unsigned)warps * 32);
  lc.dynamicSmemBytes = (Cfg::WARP_BYTES + (p.aligned ? 0 : Cfg::WARP_TAILS)) * warps;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = split > 1;
  return cudaLaunchKernelEx(&lc, kern, p);
}

// One tile of columns: two tiles of rows.  Two tiles of columns: four, which
// load x half as often, where they are faster: a block of four takes about 20/13
// of a block of two, and an SM runs one of either at a time.  GB300, 16
// tokens, us with two / four: 4096 x 4096 10.3 / 12.4, 1341 x 2050 11 / 22.6,
// 5000 x 4096 20.5 / 14.3, 8192 x 28672 82 / 61.5, 2 x 5504 x 4096 23.8 / 30.8.
template <typename T, int W, bool GATED>
cudaError_t pick_tiles(Q4Args p, cudaStream_t s, const DeviceProps &dp) {
  constexpr int parts = 8 / W, bytes = parts * (int)sizeof(T) < 16 ? parts * (int)sizeof(T) : 16;
  uintptr_t q = 0, sc = (uintptr_t)p.groups * sizeof(T);
  for (int k = 0; k < (GATED ? 2 : 1); ++k) {
    q |= reinterpret_cast<uintptr_t>(p.w[k].q) | (p.N > 1 ? (uintptr_t)p.w[k].ldq : 0);
    sc |= reinterpret_cast<uintptr_t>(p.w[k].s) | reinterpret_cast<uintptr_t>(p.w[k].z);
  }
  p.aligned = q % 16 == 0;
  p.scales_aligned = p.group == 32 * W && sc % bytes == 0 && bytes >= 4;
  if (p.M <= kTileTokens<T>) return launch_q4<T, W, 2, 1, GATED>(p, s, dp);
  const int64_t passes = ceil_div(p.M, kTileTokens<T> * 2);
  auto waves = [&](int rows) { return ceil_div(ceil_div(p.N, rows) * passes, dp.sm_count); };
  return 13 * waves(GATED ? 16 : 32) < 20 * waves(GATED ? 32 : 64)
             ? launch_q4<T, W, 2, 2, GATED>(p, s, dp)
             : launch_q4<T, W, 4, 2, GATED>(p, s, dp);
}

template <typename T, bool GATED>
cudaError_t pick_group(const Q4Args &p, cudaStream_t s, const DeviceProps &dp) {
  return p.group == 32   ? pick_tiles<T, 1, GATED>(p, s, dp)
         : p.group == 64 ? pick_tiles<T, 2, GATED>(p, s, dp)
                         : pick_tiles<T, 4, GATED>(p, s, dp);
}

bool side_ok(const Q4Side &w, const Q4Args &p, int dtype) {
  const uintptr_t mask = dtype_size(dtype) - 1;
  if (w.ldq < (p.K + 1) / 2 || w.ldq >= ((int64_t)1 << 32)) return false;
  if (p.M == 0 || p.N == 0 || p.K == 0) return true;
  return w.q && w.s && !(reinterpret_cast<uintptr_t>(w.s) & mask) &&
         !(reinterpret_cast<uintptr_t>(w.z) & mask);
}

int run_q4(int dtype, int sides, Q4Args p, cudaStream_t stream) {
  constexpr int64_t lim = ((int64_t)1 << 31) - 512;
  if (!dtype_known(dtype) || !act_known(p.act)) return GEMM_ERR_INVALID_ARG;
  if (p.M < 0 || p.N < 0 || p.K < 0) return GEMM_ERR_INVALID_ARG;
  if (p.group != 32 && p.group != 64 && p.group != 128 && p.group != 256)
    return GEMM_ERR_INVALID_ARG;
  if (p.M > lim || p.N > lim || p.K > lim) return GEMM_ERR_UNSUPPORTED;
  if (p.ldx < (p.K > 1 ? p.K : 1) || p.ldy < (p.N > 1 ? p.N : 1)) return GEMM_ERR_INVALID_ARG;
  for (int k = 0; k < sides; ++k)
    if (!side_ok(p.w[k], p, dtype)) return GEMM_ERR_INVALID_ARG;
  if (sides == 2 && (p.w[0].z == nullptr) != (p.w[1].z == nullptr)) return GEMM_ERR_INVALID_ARG;
  if (p.M == 0 || p.N == 0) return GEMM_OK;
  const uintptr_t size = dtype_size(dtype), mask = size - 1;
  if (!p.y || (reinterpret_cast<uintptr_t>(p.y) & mask) ||
      (p.K > 0 && (!p.x || (reinterpret_cast<uintptr_t>(p.x) & mask))))
    return GEMM_ERR_INVALID_ARG;
  if (ceil_div(p.M, kTileTokens<float> * 2) > 65535) return GEMM_ERR_UNSUPPORTED;
  int dev = -1;
  const int st = current_device(&dev);
  if (st != GEMM_OK) return st;
  const DeviceProps &dp = props_of(dev);
  p.mask = 0x000f000f;
  p.group_shift = p.group == 32 ? 5 : p.group == 64 ? 6 : p.group == 128 ? 7 : 8;
  p.vec_x = ((reinterpret_cast<uintptr_t>(p.x) | (p.M > 1 ? (uintptr_t)p.ldx * size : 0)) & 15) == 0;
  cudaError_t e;
  if (dtype == GEMM_DT_F32)
    e = sides == 2 ? pick_group<float, true>(p, stream, dp)
                   : pick_group<float, false>(p, stream, dp);
  else
    e = sides == 2 ? pick_group<bf16, true>(p, stream, dp)
                   : pick_group<bf16, false>(p, stream, dp);
  return to_status(e);
}

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

int q4_matmul(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
              const void *Q, int64_t ldq, const void *S, const void *Z, int group, void *Y,
              int64_t ldy, cudaStream_t stream) {
  Q4Args p{M, N, K, ldx, ldy, group > 0 ? ceil_div(K, group) : 0, GEMM_ACT_SILU, group, X, Y, {}};
  p.w[0] = {static_cast<const uint8_t *>(Q), ldq, S, Z};
  return run_q4(dtype, 1, p, stream);
}

int q4_gated(int dtype, int act, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
             const void *Qg, int64_t ldqg, const void *Sg, const void *Zg, const void *Qu,
             int64_t ldqu, const void *Su, const void *Zu, int group, void *H, int64_t ldh,
             cudaStream_t stream) {
  Q4Args p{M, N, K, ldx, ldh, group > 0 ? ceil_div(K, group) : 0, act, group, X, H, {}};
  p.w[0] = {static_cast<const uint8_t *>(Qg), ldqg, Sg, Zg};
  p.w[1] = {static_cast<const uint8_t *>(Qu), ldqu, Su, Zu};
  return run_q4(dtype, 2, p, stream);
}

}  // extern "C"
