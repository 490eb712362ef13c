// Products with 4-bit weights for a few tokens (include/gb300_gemm.h,
// q4_matmul and q4_gated).
//
// Y^T = W X^T on mma.sync tiles of 16 weight rows x 8 columns of X^T, BF16 in,
// FP32 sums.  What bounds it is reading the codes once (N K / 2 bytes), so
// each thread copies the codes that it alone will use to shared memory ahead
// of time, asynchronously and a ring of stages deep, and the arithmetic per
// code is kept under what that leaves: a 32-bit word of eight codes becomes
// four BF16 pairs 128 + q, exact, by 3 shifts and 4 three-input logic
// operations that mask and or in the exponent of 128.  The ALU pipe, which
// runs these at half the issue rate, is what the kernel is nearest to.
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
// each token, so a tile holds 2 tokens, and 8 in BF16.
//
// A CTA has one block of rows and its warps split k; their sums meet in shared
// memory in a fixed order.
#include <cstdlib>

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
  int group_shift;  // group = 1 << group_shift
  int vec_x;        // rows of X start on 16-byte boundaries
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
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
template <bool EXACT, int I>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
  const uint32_t u = ((w >> (4 * I)) & 0x000f000fu) | 0x43004300u;
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

// The pairs (x_i, x_i+4), i = 0..3, of plane `plane`.
__device__ __forceinline__ void pairs(const Raw8<bf16> &r, int, uint32_t (&b)[4]) {
  const uint4 v = r.v[0];
  b[0] = __byte_perm(v.x, v.z, 0x5410);
  b[1] = __byte_perm(v.x, v.z, 0x7632);
  b[2] = __byte_perm(v.y, v.w, 0x5410);
  b[3] = __byte_perm(v.y, v.w, 0x7632);
}
__device__ __forceinline__ uint32_t plane_of(float x, int plane) {
  bf16 h = __float2bfloat16_rn(x);
  const bool fin = (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u;
  if (fin && (__bfloat16_as_ushort(h) & 0x7f80u) == 0x7f80u) h = __float2bfloat16_rz(x);
  if (plane > 0) {
    const float r = fin ? x - __bfloat162float(h) : 0.0f;
    h = __float2bfloat16_rn(r);
    if (plane > 1) h = __float2bfloat16_rn(r - __bfloat162float(h));
  }
  return __bfloat16_as_ushort(h);
}
__device__ __forceinline__ void pairs(const Raw8<float> &r, int plane, uint32_t (&b)[4]) {
  const float *f = reinterpret_cast<const float *>(r.v);
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = plane_of(f[i], plane) | (plane_of(f[i + 4], plane) << 16);
}

// W: words of codes of a thread, row and step.  TI: 16-row tiles of a warp
// (gated: half of each matrix).  NT: tiles of columns.  VEC: every row of codes
// starts on a boundary of 4 W bytes; otherwise the aligned words around a
// thread's bytes are copied, one more, and shifted when used.
template <typename T, int W, int TI, int NT, bool GATED, bool VEC>
struct Q4Cfg {
  static constexpr int WW = VEC ? W : W + 1;
  static constexpr int STEP = 32 * W;                 // k of one step
  static constexpr int SLOT = TI * 2 * WW;            // words of a stage for each thread
  // warps that an SM holds, by registers: 24 with two tiles, 16 with four
  static constexpr int SM_WARPS = TI == 4 ? 16 : 24;
  static constexpr int DEEP = 227 * 1024 / (SM_WARPS * 128) / SLOT;
  static constexpr int STAGES = DEEP > 8 ? 8 : DEEP;
  static_assert(STAGES >= 2, "");
  static constexpr int COLS = NT * 8;
  static constexpr int TILES = GATED ? TI / 2 : TI;   // of one matrix
  static constexpr int ROWS = TILES * 16;
  static_assert(!GATED || TI % 2 == 0, "");
  // the ring of a thread, or its warp's share of the sums
  static constexpr int RING = STAGES * SLOT * 32, RED = TI * 16 * COLS;
  static constexpr int WARP_BYTES = (RING > RED ? RING : RED) * 4;
};

template <typename T, int W, int TI, int NT, bool GATED, bool VEC>
__global__ void __launch_bounds__(Q4Cfg<T, W, TI, NT, GATED, VEC>::SM_WARPS * 32, 1)
q4_kernel(const Q4Args p) {
  using Cfg = Q4Cfg<T, W, TI, NT, GATED, VEC>;
  constexpr int WW = Cfg::WW, STEP = Cfg::STEP, SLOT = Cfg::SLOT, STAGES = Cfg::STAGES;
  constexpr int COLS = Cfg::COLS, TILES = Cfg::TILES, SIDES = GATED ? 2 : 1;
  constexpr bool EXACT = sizeof(T) == 4;
  extern __shared__ __align__(16) uint32_t shared[];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int warps = blockDim.x >> 5;
  // this thread's ring: word w of a slot at ring[w * 32], or 4 W bytes together
  uint32_t *ring = shared + warp * (Cfg::WARP_BYTES / 4) + (VEC ? lane * W : lane);
  const bool has_z = p.w[0].z != nullptr;
  const int64_t m0 = (int64_t)blockIdx.y * (kTileTokens<T> * NT);
  const int64_t n0 = (int64_t)blockIdx.x * Cfg::ROWS;
  const int left = (int)(p.N - n0 < Cfg::ROWS ? p.N - n0 : Cfg::ROWS);
  const int steps = (int)((p.K + STEP - 1) / STEP);
  const int mine = steps > warp ? (steps - warp + warps - 1) / warps : 0;
  const int64_t row_bytes = (p.K + 1) / 2;

  // Weight rows of the halves of the tiles.  Rows that the matrix does not
  // have stand for its last one: what is computed of them is not stored.
  uint32_t row[TILES][2];
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = i * 16 + 8 * h + g;
      row[i][h] = (uint32_t)(r < left ? r : left - 1);
    }
  const uint8_t *base[SIDES];
  const T *sbase[SIDES], *zbase[SIDES];
#pragma unroll
  for (int k = 0; k < SIDES; ++k) {
    base[k] = p.w[k].q + n0 * p.w[k].ldq + t * (4 * W);
    sbase[k] = static_cast<const T *>(p.w[k].s) + n0 * p.groups;
    zbase[k] = static_cast<const T *>(p.w[k].z) + (has_z ? n0 * p.groups : 0);
  }

  // The codes of this thread in step `c`, to slot `st`.
  auto copy = [&](int c, int st) {
    const int64_t at = (int64_t)c * (STEP / 2);
    // A step inside the rows is copied as it is.  Words copied for unaligned
    // rows begin and end in other rows, of which the matrix's ends have none.
    bool inside = at + STEP / 2 <= row_bytes;
    if (!VEC && ((n0 == 0 && c == 0) || (n0 + left == p.N && c + 2 >= steps))) inside = false;
    uint32_t *slot = ring + st * (SLOT * 32);
    auto each = [&](auto f) {
#pragma unroll
      for (int k = 0; k < SIDES; ++k)
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t *src = base[k] + at + (uint64_t)row[i][h] * (uint32_t)p.w[k].ldq;
            if (!VEC) src -= reinterpret_cast<uintptr_t>(src) & 3;
            f(src, slot + ((k * TILES + i) * 2 + h) * WW * 32, k);
          }
    };
    auto issue = [&](const uint8_t *src, uint32_t *dst) {
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
      if constexpr (VEC) {
        cp_async(to, src, 4 * W);
      } else {
#pragma unroll
        for (int j = 0; j < WW; ++j) cp_async(to + j * 128, src + 4 * j, 4);
      }
    };
    if (inside) {
      each([&](const uint8_t *src, uint32_t *dst, int) { issue(src, dst); });
    } else {
      each([&](const uint8_t *src, uint32_t *dst, int k) {
        const uint8_t *first = p.w[k].q, *end = first + (p.N - 1) * p.w[k].ldq + row_bytes;
        if (src >= first && src + 4 * WW <= end) {
          issue(src, dst);
          return;
        }
        // at the ends of the matrix: code 8 beyond it
#pragma unroll 1
        for (int j = 0; j < WW; ++j, src += 4) {
          uint32_t v = 0x88888888u;
          if (src >= first && src + 4 <= end) {
            v = *reinterpret_cast<const uint32_t *>(src);
          } else if (src < end && src + 4 > first) {
            v = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b)
              v |= (uint32_t)(src + b >= first && src + b < end ? src[b] : 0x88) << (8 * b);
          }
          dst[VEC ? j : j * 32] = v;
        }
      });
    }
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
  // The scales are loaded a step ahead, x at the step's start
  Raw8<T> raw[NT][W];
  T sraw[SIDES][TILES][2], zraw[SIDES][TILES][2];
  auto fetch_x = [&](int c) {
    const int64_t k0 = (int64_t)c * STEP;
    if (p.vec_x != 0 && k0 + STEP <= p.K) {
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
  auto fetch_s = [&](int c) {
    const int64_t grp = (int64_t)c * STEP >> p.group_shift;
#pragma unroll
    for (int k = 0; k < SIDES; ++k)
#pragma unroll
      for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t at = (uint64_t)row[i][h] * (uint32_t)p.groups;
          sraw[k][i][h] = (sbase[k] + grp)[at];
          if (has_z) zraw[k][i][h] = (zbase[k] + grp)[at];
        }
  };

#pragma unroll
  for (int st = 0; st < STAGES - 1; ++st) {
    if (st < mine) copy(warp + st * warps, st);
    cp_async_commit();
  }
  float acc[TI][NT][4];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.0f;
  if (mine > 0) fetch_s(warp);

  int st = 0;
#pragma unroll 1
  for (int it = 0; it < mine; ++it) {
    const int c = warp + it * warps;
    fetch_x(c);
    uint32_t b[NT][W][4];
    float s[TI][2], z[TI][2];  // scales; what is taken off of each code still
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s[i][h] = to_f32(sraw[i / TILES][i % TILES][h]);
        z[i][h] = (EXACT ? 8.0f : -128.0f) - (has_z ? to_f32(zraw[i / TILES][i % TILES][h]) : 8.0f);
      }
    if (it + 1 < mine) fetch_s(c + warps);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < W; ++j) pairs(raw[nt][j], plane, b[nt][j]);
    float xs[NT][4];
    if (!EXACT || has_z) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        constexpr uint32_t one = 0x3f803f80u;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          if (j == 0)
            mma_16816_first(xs[nt], one, one, one, one, b[nt][j][0], b[nt][j][1]);
          else
            mma_16816(xs[nt], one, one, one, one, b[nt][j][0], b[nt][j][1]);
          mma_16816(xs[nt], one, one, one, one, b[nt][j][2], b[nt][j][3]);
        }
      }
    }
    cp_async_wait<STAGES - 2>();  // this step's codes are here (each thread reads its own)
    const uint32_t *slot = ring + st * (SLOT * 32);
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      uint32_t w[2][W];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t *src = slot + (i * 2 + h) * WW * 32;
        if constexpr (VEC) {
          if constexpr (W == 4)
            *reinterpret_cast<uint4 *>(w[h]) = *reinterpret_cast<const uint4 *>(src);
          else if constexpr (W == 2)
            *reinterpret_cast<uint2 *>(w[h]) = *reinterpret_cast<const uint2 *>(src);
          else
            w[h][0] = src[0];
        } else {
          const Q4Side &sd = p.w[i / TILES];
          const int shift = 8 * (((uint32_t)reinterpret_cast<uintptr_t>(base[i / TILES]) +
                                  row[i % TILES][h] * (uint32_t)sd.ldq) & 3);
          uint32_t lo = src[0];
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const uint32_t hi = src[(j + 1) * 32];
            w[h][j] = __funnelshift_r(lo, hi, shift);
            lo = hi;
          }
        }
      }
      float d[NT][4];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t a0 = codes<EXACT, 0>(w[0][j]), a1 = codes<EXACT, 0>(w[1][j]),
                       a2 = codes<EXACT, 1>(w[0][j]), a3 = codes<EXACT, 1>(w[1][j]),
                       a4 = codes<EXACT, 2>(w[0][j]), a5 = codes<EXACT, 2>(w[1][j]),
                       a6 = codes<EXACT, 3>(w[0][j]), a7 = codes<EXACT, 3>(w[1][j]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (j == 0)
            mma_16816_first(d[nt], a0, a1, a2, a3, b[nt][j][0], b[nt][j][1]);
          else
            mma_16816(d[nt], a0, a1, a2, a3, b[nt][j][0], b[nt][j][1]);
          mma_16816(d[nt], a4, a5, a6, a7, b[nt][j][2], b[nt][j][3]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = d[nt][e];
          if (!EXACT || has_z) v = fmaf(z[i][e >> 1], xs[nt][e], v);
          acc[i][nt][e] = fmaf(s[i][e >> 1], v, acc[i][nt][e]);
        }
    }
    // the slot that the step before freed
    if (it + STAGES - 1 < mine) copy(c + (STAGES - 1) * warps, st == 0 ? STAGES - 1 : st - 1);
    cp_async_commit();
    if (++st == STAGES) st = 0;
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
  constexpr int TOKENS = kTileTokens<T> * NT;
  auto total = [&](int r, int m) {
    float v = 0.0f;
    constexpr int PLANES = sizeof(T) == 4 ? 3 : 1;
    const int col = m / kTileTokens<T> * 8 + m % kTileTokens<T> * PLANES;
#pragma unroll
    for (int q = PLANES - 1; q >= 0; --q)
#pragma unroll 4
      for (int w = 0; w < warps; ++w) v += red[(w * TI * 16 + r) * COLS + col + q];
    return v;
  };
  const int tokens = (int)(p.M - m0 < TOKENS ? p.M - m0 : TOKENS);
  for (int e = tid; e < Cfg::ROWS * tokens; e += blockDim.x) {
    const int r = e % Cfg::ROWS, m = e / Cfg::ROWS;
    if (r >= left) continue;
    float y = total(r, m);
    if constexpr (GATED) {
      const float u = total(Cfg::ROWS + r, m);
      with_act(p.act, [&](auto a) { y = act_of<sizeof(T) == 2, decltype(a)::value>(y) * u; });
    }
    static_cast<T *>(p.y)[(m0 + m) * p.ldy + n0 + r] = from_f32<T>(y);
  }
}

template <typename T, int W, int TI, int NT, bool GATED, bool VEC>
cudaError_t launch_q4(const Q4Args &p, cudaStream_t s, int warps) {
  using Cfg = Q4Cfg<T, W, TI, NT, GATED, VEC>;
  static_assert(Cfg::WARP_BYTES * kMaxWarps <= 227 * 1024, "");
  auto kern = q4_kernel<T, W, TI, NT, GATED, VEC>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg::WARP_BYTES * kMaxWarps);
  if (e != cudaSuccess) return e;
  kern<<<dim3((unsigned)ceil_div(p.N, Cfg::ROWS), (unsigned)ceil_div(p.M, kTileTokens<T> * NT)),
         warps * 32, Cfg::WARP_BYTES * warps, s>>>(p);
  return cudaGetLastError();
}

// Tiles and warps: two tiles for one tile of columns, so that six CTAs of four
// warps share an SM; four tiles for two, whose x is then loaded half as often.
template <typename T, int W, bool GATED, bool VEC>
cudaError_t pick_tiles(const Q4Args &p, cudaStream_t s, int sms) {
  const int steps = (int)ceil_div(p.K, 32 * W);
  const bool wide = p.M > kTileTokens<T>;
  const int tiles = wide ? 4 : 2;
  const int64_t ctas = ceil_div(p.N, tiles * 16 / (GATED ? 2 : 1));
  const int most = wide ? 16 : 24;  // warps that an SM holds
  int warps = (int)(most * sms / ctas);
  warps = warps < 4 ? 4 : warps > kMaxWarps ? kMaxWarps : warps;
  if (warps > steps) warps = steps < 1 ? 1 : steps;
  if (const char *e = std::getenv("Q4_WARPS")) warps = std::atoi(e);
  return wide ? launch_q4<T, W, 4, 2, GATED, VEC>(p, s, warps)
              : launch_q4<T, W, 2, 1, GATED, VEC>(p, s, warps);
}

template <typename T, int W, bool GATED>
cudaError_t pick_vec(const Q4Args &p, cudaStream_t s, int sms) {
  uintptr_t bits = 0;
  for (int k = 0; k < (GATED ? 2 : 1); ++k)
    bits |= reinterpret_cast<uintptr_t>(p.w[k].q) | (p.N > 1 ? (uintptr_t)p.w[k].ldq : 0);
  return bits % (4 * W) == 0 ? pick_tiles<T, W, GATED, true>(p, s, sms)
                             : pick_tiles<T, W, GATED, false>(p, s, sms);
}

template <typename T, bool GATED>
cudaError_t pick_group(const Q4Args &p, cudaStream_t s, int sms) {
  return p.group == 32   ? pick_vec<T, 1, GATED>(p, s, sms)
         : p.group == 64 ? pick_vec<T, 2, GATED>(p, s, sms)
                         : pick_vec<T, 4, GATED>(p, s, sms);
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
  const int sms = props_of(dev).sm_count;
  p.group_shift = p.group == 32 ? 5 : p.group == 64 ? 6 : p.group == 128 ? 7 : 8;
  p.vec_x = ((reinterpret_cast<uintptr_t>(p.x) | (p.M > 1 ? (uintptr_t)p.ldx * size : 0)) & 15) == 0;
  cudaError_t e;
  if (dtype == GEMM_DT_F32)
    e = sides == 2 ? pick_group<float, true>(p, stream, sms)
                   : pick_group<float, false>(p, stream, sms);
  else
    e = sides == 2 ? pick_group<bf16, true>(p, stream, sms)
                   : pick_group<bf16, false>(p, stream, sms);
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
