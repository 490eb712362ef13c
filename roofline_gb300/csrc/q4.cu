// Products with 4-bit weights for a few tokens (include/gb300_gemm.h,
// q4_matmul and q4_gated).
//
// Y^T = W X^T on mma.sync tiles of 16 weight rows x 8 columns of X^T, BF16 in,
// FP32 sums.  What bounds it is reading the codes once (N K / 2 bytes), so
// each thread copies the codes that it alone will use to shared memory ahead
// of time, asynchronously and a ring of stages deep, and the arithmetic per
// code is kept under what that leaves: a 32-bit word of eight codes becomes
// four pairs of BF16 by 3 shifts, 4 three-input logic operations (mask, and
// or in the exponent of 128: 128 + q is exact) and 4 paired subtractions of
// 136, which leave q - 8, exact too.  Scales multiply the FP32 sums of one
// group; a zero point z other than 8 adds s (8 - z) sum x, with the sums of x
// from one more MMA whose weights are ones.
//
// An MMA sums 16 values of k in any order, so a thread's eight codes of one
// word are the k that it feeds to two MMAs, and X is loaded to match.  All k
// of an MMA belong to one group: the four threads of a row take 32 W values of
// k, W = 1, 2, 4 words each for groups of 32, 64, 128 (or 256).
//
// FP32 X is split into three BF16 (24 bits) that take three columns of an MMA
// each token, so a tile holds 2 tokens, and 8 in BF16.
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
  int rows, blocks;  // weight rows of one block (of each matrix), blocks
  int vec_x;         // rows of X start on 16-byte boundaries
};

constexpr int kQ4Threads = 256, kQ4Warps = kQ4Threads / 32;
constexpr int kTiles = 4;              // 16-row tiles of a warp (gated: two of each matrix)
constexpr int kStageWords = 20480;     // shared memory of the code ring: 160 KB at W = 4

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

// Codes i and i + 4 of a word, as the BF16 pair (q - 8, q - 8).
template <int I>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
  const uint32_t u = ((w >> (4 * I)) & 0x000f000fu) | 0x43004300u;
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

template <typename T>
__device__ __forceinline__ void load_x(Raw8<T> &r, const T *row, int64_t k, int64_t K, bool vec) {
  if (vec && k + 8 <= K) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      r.v[i] = __ldg(reinterpret_cast<const uint4 *>(row + k) + i);
  } else {
    __align__(16) T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = k + i < K ? row[k + i] : from_f32<T>(0.0f);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const uint4 *>(t)[i];
  }
}

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

// W: words of codes of a thread, row and step.  NT: tiles of columns.  VEC:
// every row of codes starts on a boundary of 4 W bytes; otherwise the aligned
// words around a thread's bytes are copied, one more, and shifted when used.
template <typename T, int W, int NT, bool GATED, bool VEC>
__global__ void __launch_bounds__(kQ4Threads, 1) q4_kernel(const Q4Args p) {
  constexpr int WW = VEC ? W : W + 1;
  constexpr int STEP = 32 * W;                           // k of one step
  constexpr int SLOT = kTiles * 2 * WW * kQ4Threads;     // words of one stage
  constexpr int STAGES = kStageWords * 2 / SLOT > 10 ? 10 : kStageWords * 2 / SLOT;
  constexpr int COLS = NT * 8;
  constexpr int SIDE_TILES = GATED ? kTiles / 2 : kTiles;
  extern __shared__ __align__(16) uint32_t ring[];
  float *red = reinterpret_cast<float *>(ring + STAGES * SLOT);  // [warp][tile row][column]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int64_t m0 = (int64_t)blockIdx.y * (kTileTokens<T> * NT);
  const int steps = (int)((p.K + STEP - 1) / STEP);
  const int mine = steps > warp ? (steps - warp + kQ4Warps - 1) / kQ4Warps : 0;
  const int64_t row_bytes = (p.K + 1) / 2;

  // The codes of this thread in step `c` of block `blk`, to slot `st`.
  auto copy = [&](int blk, int c, int st) {
    const int64_t n0 = (int64_t)blk * p.rows;
    const int left = (int)(p.N - n0 < p.rows ? p.N - n0 : p.rows);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const Q4Side &w = p.w[GATED && i >= SIDE_TILES];
      const uint8_t *end = w.q + (p.N - 1) * w.ldq + row_bytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = (i % SIDE_TILES) * 16 + 8 * h + g;
        uint32_t *dst = ring + st * SLOT + (i * 2 + h) * WW * kQ4Threads;
        if ((i % SIDE_TILES) * 16 >= left) continue;  // the whole tile: never read
        const uint8_t *src = w.q + (n0 + r) * w.ldq + (int64_t)c * (STEP / 2) + t * (4 * W);
        if constexpr (VEC) {
          dst += tid * W;
          if (r < left && src + 4 * W <= end) {
            cp_async((uint32_t)__cvta_generic_to_shared(dst), src, 4 * W);
            continue;
          }
        } else {
          src -= reinterpret_cast<uintptr_t>(src) & 3;
          if (r < left && src >= w.q && src + 4 * WW <= end) {
#pragma unroll
            for (int j = 0; j < WW; ++j)
              cp_async((uint32_t)__cvta_generic_to_shared(dst + j * kQ4Threads + tid), src + 4 * j,
                       4);
            continue;
          }
        }
        // at the ends of the matrix byte by byte; code 8 where there is none
        for (int j = 0; j < WW; ++j) {
          uint32_t v = r < left ? 0 : 0x88888888u;
          for (int b = 0; b < 4 && r < left; ++b) {
            const uint8_t *at = src + 4 * j + b;
            v |= (uint32_t)(at >= w.q && at < end ? *at : 0x88) << (8 * b);
          }
          dst[VEC ? j : j * kQ4Threads + tid] = v;
        }
      }
    }
  };

  // This lane's column of each tile of X^T
  const int col_token = column_token<T>(g), plane = sizeof(T) == 4 ? g % 3 : 0;
  const T *xrow[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int64_t m = m0 + nt * kTileTokens<T> + col_token;
    xrow[nt] = col_token < kTileTokens<T> && m < p.M ? static_cast<const T *>(p.x) + m * p.ldx
                                                     : nullptr;
  }
  auto fetch_x = [&](int c, Raw8<T> (&r)[NT][W]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if (xrow[nt] != nullptr) {
          load_x(r[nt][j], xrow[nt], (int64_t)c * STEP + t * (8 * W) + 8 * j, p.K, p.vec_x != 0);
        } else {
#pragma unroll
          for (int i = 0; i < (int)sizeof(T) / 2; ++i) r[nt][j].v[i] = make_uint4(0, 0, 0, 0);
        }
      }
  };

  // The copies run ahead of the arithmetic, over the ends of blocks too.
  int cb = blockIdx.x, ci = 0;  // block and own step to copy next
  auto copy_next = [&](int st) {
    if (cb < p.blocks && mine > 0) {
      copy(cb, warp + ci * kQ4Warps, st);
      if (++ci == mine) {
        ci = 0;
        cb += gridDim.x;
      }
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int st = 0; st < STAGES - 1; ++st) copy_next(st);

  int st = 0;
  for (int blk = blockIdx.x; blk < p.blocks; blk += gridDim.x) {
    const int64_t n0 = (int64_t)blk * p.rows;
    const int left = (int)(p.N - n0 < p.rows ? p.N - n0 : p.rows);
    float acc[kTiles][NT][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.0f;

    // x and the scales are loaded a step ahead
    Raw8<T> raw[NT][W];
    T sraw[kTiles][2], zraw[kTiles][2];
    auto fetch_s = [&](int c) {
      const int64_t grp = (int64_t)c * STEP / p.group;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const Q4Side &w = p.w[GATED && i >= SIDE_TILES];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = (i % SIDE_TILES) * 16 + 8 * h + g;
          const int64_t at = (n0 + r) * p.groups + grp;
          sraw[i][h] = r < left ? static_cast<const T *>(w.s)[at] : from_f32<T>(0.0f);
          zraw[i][h] = r < left && w.z ? static_cast<const T *>(w.z)[at] : from_f32<T>(8.0f);
        }
      }
    };
    if (mine > 0) {
      fetch_x(warp, raw);
      fetch_s(warp);
    }
#pragma unroll 1
    for (int it = 0; it < mine; ++it) {
      const int c = warp + it * kQ4Warps;
      float s[kTiles][2], z[kTiles][2];  // scales; 8 less the zero points
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s[i][h] = to_f32(sraw[i][h]);
          z[i][h] = 8.0f - to_f32(zraw[i][h]);
        }
      uint32_t b[NT][W][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < W; ++j) pairs(raw[nt][j], plane, b[nt][j]);
      if (it + 1 < mine) {
        fetch_x(c + kQ4Warps, raw);
        fetch_s(c + kQ4Warps);
      }

      cp_async_wait<STAGES - 2>();  // this step's codes are here (each thread reads its own)
      const uint32_t *slot = ring + st * SLOT;
      float xs[NT][4];
      if (p.w[0].z != nullptr) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          xs[nt][0] = xs[nt][1] = xs[nt][2] = xs[nt][3] = 0.0f;
          constexpr uint32_t one = 0x3f803f80u;
#pragma unroll
          for (int j = 0; j < W; ++j) {
            mma_16816(xs[nt], one, one, one, one, b[nt][j][0], b[nt][j][1]);
            mma_16816(xs[nt], one, one, one, one, b[nt][j][2], b[nt][j][3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        if ((i % SIDE_TILES) * 16 >= left) continue;
        uint32_t w[2][W];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t *src = slot + (i * 2 + h) * WW * kQ4Threads;
          if constexpr (VEC) {
            src += tid * W;
            if constexpr (W == 4)
              *reinterpret_cast<uint4 *>(w[h]) = *reinterpret_cast<const uint4 *>(src);
            else if constexpr (W == 2)
              *reinterpret_cast<uint2 *>(w[h]) = *reinterpret_cast<const uint2 *>(src);
            else
              w[h][0] = src[0];
          } else {
            const Q4Side &sd = p.w[GATED && i >= SIDE_TILES];
            const int r = (i % SIDE_TILES) * 16 + 8 * h + g;
            const int shift = 8 * (int)((reinterpret_cast<uintptr_t>(sd.q) + (n0 + r) * sd.ldq) & 3);
            uint32_t lo = src[tid];
#pragma unroll
            for (int j = 0; j < W; ++j) {
              const uint32_t hi = src[(j + 1) * kQ4Threads + tid];
              w[h][j] = __funnelshift_r(lo, hi, shift);
              lo = hi;
            }
          }
        }
        float d[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t a0 = codes<0>(w[0][j]), a1 = codes<0>(w[1][j]), a2 = codes<1>(w[0][j]),
                         a3 = codes<1>(w[1][j]), a4 = codes<2>(w[0][j]), a5 = codes<2>(w[1][j]),
                         a6 = codes<3>(w[0][j]), a7 = codes<3>(w[1][j]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816(d[nt], a0, a1, a2, a3, b[nt][j][0], b[nt][j][1]);
            mma_16816(d[nt], a4, a5, a6, a7, b[nt][j][2], b[nt][j][3]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = d[nt][e];
            if (p.w[0].z != nullptr) v = fmaf(z[i][e >> 1], xs[nt][e], v);
            acc[i][nt][e] = fmaf(s[i][e >> 1], v, acc[i][nt][e]);
          }
      }
      copy_next(st == 0 ? STAGES - 1 : st - 1);  // the slot that the step before freed
      if (++st == STAGES) st = 0;
    }

    // The warps' sums over their steps, added in order; then, FP32, the planes.
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2 *>(red + ((warp * kTiles + i) * 16 + 8 * h + g) * COLS + nt * 8 +
                                      2 * t) =
              make_float2(acc[i][nt][2 * h], acc[i][nt][2 * h + 1]);
    __syncthreads();
    constexpr int ROWS = SIDE_TILES * 16, TOKENS = kTileTokens<T> * NT;
    auto total = [&](int row, int m) {
      float v = 0.0f;
      constexpr int PLANES = sizeof(T) == 4 ? 3 : 1;
      const int col = m / kTileTokens<T> * 8 + m % kTileTokens<T> * PLANES;
#pragma unroll
      for (int q = PLANES - 1; q >= 0; --q)
#pragma unroll
        for (int w = 0; w < kQ4Warps; ++w)
          v += red[(w * kTiles * 16 + row) * COLS + col + q];
      return v;
    };
    for (int e = tid; e < ROWS * TOKENS; e += kQ4Threads) {
      const int r = e % ROWS, m = e / ROWS;
      if (r >= left || m0 + m >= p.M) continue;
      float y = total(r, m);
      if constexpr (GATED) {
        const float u = total(ROWS + r, m);
        with_act(p.act, [&](auto a) { y = act_of<sizeof(T) == 2, decltype(a)::value>(y) * u; });
      }
      static_cast<T *>(p.y)[(m0 + m) * p.ldy + n0 + r] = from_f32<T>(y);
    }
    __syncthreads();  // red is written again
  }
  cp_async_wait<0>();
}

template <typename T, int W, int NT, bool GATED, bool VEC>
cudaError_t launch_q4(const Q4Args &p, cudaStream_t s, int sms) {
  constexpr int SLOT = kTiles * 2 * (VEC ? W : W + 1) * kQ4Threads;
  constexpr int STAGES = kStageWords * 2 / SLOT > 10 ? 10 : kStageWords * 2 / SLOT;
  constexpr int smem = (STAGES * SLOT + kQ4Warps * kTiles * 16 * NT * 8) * 4;
  static_assert(smem <= 227 * 1024 && STAGES >= 3, "");
  auto kern = q4_kernel<T, W, NT, GATED, VEC>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t ty = ceil_div(p.M, kTileTokens<T> * NT);
  kern<<<dim3((unsigned)(p.blocks < sms ? p.blocks : sms), (unsigned)ty), kQ4Threads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int W, bool GATED, bool VEC>
cudaError_t pick_nt(const Q4Args &p, cudaStream_t s, int sms) {
  return p.M <= kTileTokens<T> ? launch_q4<T, W, 1, GATED, VEC>(p, s, sms)
                               : launch_q4<T, W, 2, GATED, VEC>(p, s, sms);
}

template <typename T, int W, bool GATED>
cudaError_t pick_vec(const Q4Args &p, cudaStream_t s, int sms) {
  uintptr_t bits = 0;
  for (int k = 0; k < (GATED ? 2 : 1); ++k)
    bits |= reinterpret_cast<uintptr_t>(p.w[k].q) | (p.N > 1 ? (uintptr_t)p.w[k].ldq : 0);
  return bits % (4 * W) == 0 ? pick_nt<T, W, GATED, true>(p, s, sms)
                             : pick_nt<T, W, GATED, false>(p, s, sms);
}

template <typename T, bool GATED>
cudaError_t pick_group(const Q4Args &p, cudaStream_t s, int sms) {
  return p.group == 32   ? pick_vec<T, 1, GATED>(p, s, sms)
         : p.group == 64 ? pick_vec<T, 2, GATED>(p, s, sms)
                         : pick_vec<T, 4, GATED>(p, s, sms);
}

bool side_ok(const Q4Side &w, const Q4Args &p, int dtype) {
  const uintptr_t mask = dtype_size(dtype) - 1;
  if (w.ldq < (p.K + 1) / 2) return false;
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
  // Blocks of equal rows, as many for each SM, at most what a warp's tiles hold.
  const int sms = props_of(dev).sm_count;
  const int64_t most = kTiles * 16 / sides, rounds = ceil_div(p.N, most * sms);
  p.rows = (int)ceil_div(p.N, rounds * sms);
  p.blocks = (int)ceil_div(p.N, p.rows);
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
