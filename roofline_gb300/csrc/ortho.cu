// Updates orthogonalised by Newton-Schulz products on the tcgen05 tensor
// cores (include/gb300_gemm.h, orthogonalize).
//
// X0 = G / (|G| + eps), then `steps` times, on the smaller side of X (m x n,
// m <= n; G is transposed on the way in and out if it is taller than wide):
//     A = X X^T       X <- a X + (b A + c A A) X.
// With any t, and U = A - t I, the same step is
//     D = (b + 2 c t) I + c U      B = U D      X <- (a + b t + c t t) X + B X.
// t is the mean of A's spectrum, |X|^2 / m, so that U and B are small where X
// is nearly orthogonal already and their rounding with them: rounded to 11
// bits (FP16) and with t = 0, products of BF16 updates end 2.4e-3 off the
// result, with this t 0.5e-3 (512 x 1408, normal values), less than the
// result's own rounding to BF16 (1.7e-3).  X itself stays in FP32 and its first
// term is added in FP32: what a step loses is a part of B X, which lies in the
// directions that X has, and is not blown up in those that it hardly has (the
// steps multiply these by a each).
//
// So the products' factors are FP16 values scaled by powers of two: one plane
// (11 bits) for BF16 updates and two, x0 + x1 (22 bits, three products), for
// FP32 ones.  A and B are symmetric: only tiles on and above the diagonal are
// computed, and their epilogue writes both.  A step is three launches of one
// persistent kernel; TMA brings the operands (X for B X as it lies, MN-major),
// the sums stay in tensor memory, and the epilogues make U, D, B and X of
// them.  Products of few tiles split K over a cluster, whose CTAs add their
// sums up through distributed shared memory in a fixed order.
//
// Each MMA rounds the sum it adds to towards zero, 2^-24 of it or so.  FP32's
// large products therefore gather for kFlush K blocks only before they are
// added to sums in registers, and the small ones apart (as in ff_tc.cu); BF16's
// gather over the whole of K, which takes 2e-4 off a sum of one sign over 32768
// at the most (2048 MMAs, each up to 1.6 * 2^-24: an eighth of the result's own
// rounding), and beyond that two planes are taken.
#include <atomic>
#include <cmath>

#include "ortho.cuh"

namespace gg {

using namespace tc;

namespace {

__device__ int g_ortho_status;  // 0 = ok, else a GEMM_ERR_* code
// Whether this process has launched (or captured) the kernels that write it: each word
// that gemm_check_status reads takes it 10 us.
std::atomic<bool> g_ortho_ran{false};

// X is kept in FP32 in the order in which the apply step's warps hold it: for
// 32 rows and 16 columns, the first 8 columns row by row, then the others, so
// that a warp reads and writes 1 KB at a time.  (As a matrix, every access of a
// warp touched 32 lines, and the apply step of 8 x 777 x 1341 took 51 us.)
__host__ __device__ __forceinline__ int64_t x32_rows(int64_t m) { return (m + 31) / 32 * 32; }
__device__ __forceinline__ int64_t x32_at(int64_t ldx, int64_t i, int64_t j) {
  return (i >> 5) * 32 * ldx + (j >> 3) * 256 + (i & 31) * 8 + (j & 7);
}

// ------------------------------------------------------------------ on the way in

constexpr int kPrepThreads = 256;
constexpr int kPrepTile = 64;

struct PrepParams {
  const void *g;
  int64_t ldg, stride;  // of G's rows and matrices, in elements
  int64_t rows, cols;   // of G as it is stored
  int64_t m, n, ldx;    // of X
  int transposed;       // X = G^T
  double eps;
  double *partial;      // [batch][blocks]
  float *x32;           // [batch][x32_rows][ldx]
  __half *x16;          // [batch][planes][m][ldx]
  float *sumsq;         // [batch]: |X|^2
};

// A thread's place in a tile of 64 rows x 64 columns: 8 columns of 2 rows, a
// warp's 8 rows of 64 (BF16) or 128 bytes.
__device__ __forceinline__ int prep_row() { return (threadIdx.x & 31) / 4 + 8 * (threadIdx.x >> 6); }
__device__ __forceinline__ int prep_col() {
  return 8 * ((threadIdx.x & 3) + ((threadIdx.x >> 5) & 1) * 4);
}

// 16 values of a tile of G from (r0, c0) on, zeros beyond the matrix.  VEC (rows
// on 16-byte boundaries): those of the thread's place.  Else columns lane and
// lane + 32 of every eighth row.
template <typename T, bool VEC>
__device__ __forceinline__ void load_part(const PrepParams &p, const T *g, int64_t r0, int64_t c0,
                                          float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] = 0.0f;
  if constexpr (VEC) {
    const int64_t c = c0 + prep_col();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = r0 + prep_row() + 32 * i;
      if (r >= p.rows) continue;
      const T *from = g + r * p.ldg + c;
      if (c + 8 <= p.cols) {
        __align__(16) T t[8];
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
          reinterpret_cast<uint4 *>(t)[k] = __ldg(reinterpret_cast<const uint4 *>(from) + k);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[8 * i + k] = to_f32(t[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < p.cols) x[8 * i + k] = to_f32(from[k]);
      }
    }
  } else {
    const int64_t c = c0 + (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + (threadIdx.x >> 5) + 8 * i;
      if (r >= p.rows) continue;
      const T *from = g + r * p.ldg + c;
      if (c < p.cols) x[2 * i] = to_f32(from[0]);
      if (c + 32 < p.cols) x[2 * i + 1] = to_f32(from[32]);
    }
  }
}

// Sums of squares.  A warp takes 4 KB of a row at a time (contiguous matrices are one
// row), as 16-byte vectors from the first boundary on: their squares in FP32 where
// they neither over- nor underflow, then in FP64.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads)
ortho_norm_kernel(const PrepParams p) {
  constexpr int VE = 16 / sizeof(T), kVecs = 8, kWarps = kPrepThreads / 32;
  __shared__ double part[kWarps];
  const T *g = static_cast<const T *>(p.g) + blockIdx.y * p.stride;
  const bool whole = p.ldg == p.cols || p.rows == 1;
  const int64_t rows = whole ? 1 : p.rows, length = whole ? p.rows * p.cols : p.cols;
  const int64_t pieces = (length / VE + 32 * kVecs - 1) / (32 * kVecs) + 1;  // one for the ends
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  double sum = 0.0;
  for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < rows * pieces;
       item += (int64_t)gridDim.x * kWarps) {
    const int64_t r = item / pieces, piece = item - r * pieces;
    const T *row = g + r * p.ldg;
    int64_t head = (int64_t)(-reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T);
    if (head > length) head = length;
    const int64_t vecs = (length - head) / VE, tail = head + vecs * VE;
    if (piece == pieces - 1) {  // fewer than VE values on either side
      float x = 0.0f;
      if (lane < head) x = to_f32(row[lane]);
      if (lane >= 16 && tail + lane - 16 < length) x = to_f32(row[tail + lane - 16]);
      sum += squares([&](float scale) { return x * scale * (x * scale); });
      continue;
    }
    uint4 v[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int64_t at = (piece * kVecs + k) * 32 + lane;
      v[k] = at < vecs ? __ldg(reinterpret_cast<const uint4 *>(row + head) + at)
                       : make_uint4(0, 0, 0, 0);
    }
    sum += squares([&](float scale) {
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        __align__(16) T t[VE];
        *reinterpret_cast<uint4 *>(t) = v[k];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float y = to_f32(t[e]) * scale;
          s[e & 1] = fmaf(y, y, s[e & 1]);
        }
      }
      return s[0] + s[1];
    });
  }
  sum = warp_sum(sum);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    for (int w = 0; w < kWarps; ++w) sum += part[w];
    p.partial[blockIdx.y * (int64_t)gridDim.x + blockIdx.x] = sum;
  }
}

// Row i of X from column j on, eight values, to both its forms.
template <int P>
__device__ __forceinline__ void store_x(const PrepParams &p, float *x32, __half *x16, int64_t i,
                                        int64_t j, float *x) {
  if (i >= p.m || j >= p.ldx) return;
  store32(x32 + x32_at(p.ldx, i, j), x);
#pragma unroll
  for (int q = 0; q < P; ++q) {
    uint4 v;
    uint32_t *u = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      if (q == 0) x[k] *= kScaleX, x[k + 1] *= kScaleX;
      const __half a = __float2half_rn(x[k]), b = __float2half_rn(x[k + 1]);
      x[k] -= __half2float(a), x[k + 1] -= __half2float(b);
      u[k / 2] = pack_half(a, b);
    }
    *reinterpret_cast<uint4 *>(x16 + (q * p.m + i) * p.ldx + j) = v;
  }
}

// X0 in FP32 and in planes; `parts` blocks made the sums.
template <typename T, bool VEC, int P>
__global__ void __launch_bounds__(kPrepThreads)
ortho_scale_kernel(const PrepParams p, int parts) {
  __shared__ float tile[kPrepTile][kPrepTile + 1];
  __shared__ double factor;
  const int64_t z = blockIdx.y;
  const T *g = static_cast<const T *>(p.g) + z * p.stride;
  const int64_t across = (p.cols + kPrepTile - 1) / kPrepTile;
  const int64_t tiles = across * ((p.rows + kPrepTile - 1) / kPrepTile);
  const int row = prep_row(), col = prep_col();
  grid_dependency_wait();
  grid_launch_dependents();
  if (threadIdx.x < 32) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += 32) sum += p.partial[z * parts + i];
    sum = warp_sum(sum);
    if (threadIdx.x == 0) {
      const double norm = sqrt(sum);
      factor = 1.0 / (norm + p.eps);
      if (blockIdx.x == 0) p.sumsq[z] = (float)(norm * factor * norm * factor);
    }
  }
  __syncthreads();
  const double inv = factor;
  const float f = (float)inv;
  // beyond FP32's normal range the factor is applied in FP64
  const bool plain = (f >= 0x1p-126f && f <= 0x1p126f) || !(inv > 0.0 && inv < INFINITY);
  float *x32 = p.x32 + z * x32_rows(p.m) * p.ldx;
  __half *x16 = p.x16 + z * P * p.m * p.ldx;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t r0 = t / across * kPrepTile, c0 = t % across * kPrepTile;
    float x[16];
    load_part<T, VEC>(p, g, r0, c0, x);
    if (plain) {
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] *= f;
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = (float)((double)x[k] * inv);
    }
    // columns from n to ldx become zeros, as G's end there
    if (VEC && !p.transposed) {
#pragma unroll
      for (int i = 0; i < 2; ++i) store_x<P>(p, x32, x16, r0 + row + 32 * i, c0 + col, x + 8 * i);
      continue;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int r = VEC ? row + 32 * (k >> 3) : (threadIdx.x >> 5) + 8 * (k >> 1);
      const int c = VEC ? col + (k & 7) : (threadIdx.x & 31) + 32 * (k & 1);
      if (p.transposed)
        tile[c][r] = x[k];
      else
        tile[r][c] = x[k];
    }
    __syncthreads();
    const int64_t i0 = p.transposed ? c0 : r0, j0 = p.transposed ? r0 : c0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = tile[row + 32 * i][col + k];
      store_x<P>(p, x32, x16, i0 + row + 32 * i, j0 + col, x);
    }
  }
}

// ------------------------------------------------------------------ the products

// warp 0: TMA, warp 1: MMA, the others: epilogue, four or two for each 32 rows.  One
// plane: 16 warps, whose blocks hide one another's latency.  Two planes: 8, whose
// registers hold a tile's sums (with 16 of 96 registers, 256 x 768 took 117 us instead
// of 111, 1024 x 2816 294 instead of 285).
constexpr int epi_warps(int planes) { return planes == 1 ? 16 : 8; }
constexpr int threads_of(int planes) { return 64 + 32 * epi_warps(planes); }
constexpr int kFlush = 4;
constexpr int kMaxStages = 12;
constexpr int kEpiStage = 2048;  // 32 x 16 values, per warp
constexpr int epi_bytes(int planes) { return epi_warps(planes) * kEpiStage; }
constexpr int stage_budget(int planes) { return 227 * 1024 - 1024 - 256 - epi_bytes(planes); }
constexpr int kMaxSplit = 8;
constexpr int kExchange = 128 * 128 * 4;  // split K: the parts of the columns that a CTA finishes
constexpr int64_t kOnePlaneK = 32768;

// What a launch computes: U and D from X X^T, B from U D, or X from B X.
enum NsStep { kGram, kPoly, kApply };

struct NsParams {
  CUtensorMap a, b;     // planes of all matrices: z = matrix * planes + plane
  int64_t M, N;         // of the output
  int64_t tiles;        // of all matrices
  int per, tiles_m, tiles_n, group_n;
  int kb, split;        // K blocks, and the CTAs of a cluster that share them
  int stages;
  float unscale;        // what the factors' scales make of the sums
  float ca, cb, cc;     // the step's coefficients
  float *t;             // [matrix]
  const float *sums;    // [matrix][sum_count]: parts of |X|^2
  int sum_count;
  float *sums_out;      // apply: the next step's, [matrix][tile][epilogue warps of all its CTAs]
  __half *p0, *p1;      // gram: U and D, poly: B, apply: X; [matrix][plane][M][ld]
  int64_t ld;
  float *x32;           // [matrix][x32_rows][ld], read and (but for the last step) written
  void *out;            // the last step's result, or null
  int64_t ldo, out_stride;
  int out_t, out_bf16;
  uint64_t wait_ns;
  int stall_producer;   // test hook: the producer issues nothing
};

// The accumulators of a tile.  One plane: two, one filled while the other is
// read.  Two planes: one or, where they fit, two for the large products, one
// for the small ones, and a place for the tile's sums: of its own, or that of the
// small products, which the next tile's wait for (KEEP).
template <int P, int BN>
struct Acc {
  static constexpr int LARGE = P == 1 || 4 * BN <= 512 ? 2 : 1;
  static constexpr int SMALL = LARGE;
  static constexpr bool KEEP = P == 2 && 4 * BN > 512;
  static constexpr int SUMS = KEEP ? SMALL : SMALL + 1;
  static constexpr int BARS = P == 1 ? 2 : SMALL + 1;
  static constexpr int COUNT = P == 1 ? 2 : SUMS + 1;
  static constexpr int COLS = COUNT * BN <= 256 ? 256 : 512;
  static_assert(COUNT * BN <= COLS, "");
};

struct TileAt {
  int m, n;
  int64_t matrix;
};

// SYM: the tiles (i, j), j >= i, row by row.  Else bands of group_n tile
// columns walked down their rows, so that the tiles worked on at one time
// share their operands through L2.
template <bool SYM>
__device__ __forceinline__ TileAt tile_at(const NsParams &p, int64_t tile) {
  const int64_t matrix = tile / p.per;
  int t = (int)(tile - matrix * p.per);
  if (SYM) {
    int i = 0;
    while (t >= p.tiles_m - i) t -= p.tiles_m - i++;
    return {i, i + t, matrix};
  }
  const int band_tiles = p.group_n * p.tiles_m, band = t / band_tiles, first = band * p.group_n;
  const int left = p.tiles_n - first, width = left < p.group_n ? left : p.group_n;
  t -= band * band_tiles;
  return {t / width, first + t % width, matrix};
}

// Columns [c, c + 16) of the warp's rows, lane i's r0 + i, to the planes at `p` and
// (mirror) turned to rows c on.  Rows are padded to 16 columns.  They are turned
// by ldmatrix, from rows 48 bytes apart in `stage`: matrix j of eight columns
// takes rows 8 q + 2 j and 8 q + 2 j + 1 for each q < 4, so that lane 4 i + q holds
// rows 8 q to 8 q + 7 of column i, 16 bytes.  (Turned by stores of one value a lane,
// an off-diagonal tile took 2 to 5 us more than a diagonal one.)
template <int P>
__device__ __forceinline__ void store_planes(__half *p, int64_t plane, int64_t ld, int64_t rows,
                                             int64_t r0, int64_t c, float (&x)[16], bool mirror,
                                             uint8_t *stage) {
  constexpr int kRow = 48;
  const int lane = threadIdx.x & 31;
  const uint32_t from = smem_u32(stage) +
                        (uint32_t)((8 * ((lane & 7) >> 1) + 2 * (lane >> 3) + (lane & 1)) * kRow);
#pragma unroll
  for (int q = 0; q < P; ++q, p += plane) {
    uint32_t u[8];
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const __half2 h = __floats2half2_rn(x[k], x[k + 1]);
      if (q + 1 < P) {
        const float2 f = __half22float2(h);
        x[k] -= f.x, x[k + 1] -= f.y;
      }
      u[k / 2] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if (r0 + lane < rows) store32(p + (r0 + lane) * ld + c, u);
    if (!mirror) continue;
    uint4 *own = reinterpret_cast<uint4 *>(stage + lane * kRow);
    own[0] = make_uint4(u[0], u[1], u[2], u[3]);
    own[1] = make_uint4(u[4], u[5], u[6], u[7]);
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // eight columns
      uint4 v;
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(from + 16 * h)
                   : "memory");
      const int64_t to = c + 8 * h + (lane >> 2), at = r0 + 8 * (lane & 3);
      if (to < rows && at < ld) *reinterpret_cast<uint4 *>(p + to * ld + at) = v;
    }
    __syncwarp();
  }
}

// The sum of a matrix's parts of |X|^2, in a fixed order, in every lane.
__device__ __forceinline__ float sum_parts(const float *parts, int count) {
  float s = 0.0f;
  for (int i = threadIdx.x & 31; i < count; i += 32) s += parts[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// What becomes of a tile's sums, 16 columns of 32 rows at a time.
template <int P, NsStep STEP>
struct Finish {
  const NsParams &p;
  float *stage;
  int64_t r0, matrix;
  bool mirror;
  float t, q0, sumsq;

  // Apply: requests X of the block at column c; nothing waits for it yet.
  __device__ __forceinline__ void request(float (&x32)[16], int64_t c) const {
    const int64_t r = r0 + (threadIdx.x & 31);
    if (STEP != kApply) return;
#pragma unroll
    for (int k = 0; k < 16; ++k) x32[k] = 0.0f;
    if (c >= p.ld || r >= p.M) return;
    const float *from = p.x32 + matrix * x32_rows(p.M) * p.ld + x32_at(p.ld, r, c);
    load32(from, x32);
    load32(from + 256, x32 + 8);
  }

  __device__ __forceinline__ void begin(const TileAt &at, int64_t row, bool first_warp) {
    if (STEP == kGram && at.matrix != matrix) {
      t = sum_parts(p.sums + at.matrix * p.sum_count, p.sum_count) / (float)p.M;
      // every tile's warps find the same t; the apply step reads it
      if (first_warp && at.m == 0 && at.n == 0 && (threadIdx.x & 31) == 0) p.t[at.matrix] = t;
    }
    if (STEP == kApply) {
      t = p.t[at.matrix];
      q0 = fmaf(fmaf(p.cc, t, p.cb), t, p.ca);
      sumsq = 0.0f;
    }
    matrix = at.matrix;
    r0 = row;
    mirror = at.m != at.n;
  }

  // The block at column c, whose X is in x32, where that of the one at column `next`
  // (none: at least ld) is requested.
  __device__ __forceinline__ void block(float (&x32)[16], int64_t c, int64_t next,
                                        const float (&v)[16]) {
    const int64_t r = r0 + (threadIdx.x & 31), plane = p.M * p.ld;
    if (c >= p.ld) return;  // warp-uniform
    if (STEP == kApply) {
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = fmaf(q0, x32[k], v[k] * p.unscale);
      request(x32, next);
      if (p.out) {
        const OrthoOut to{p.M, p.N, p.ldo, p.out_t};
        if (p.out_bf16)
          store_out<bf16>(to, static_cast<bf16 *>(p.out) + matrix * p.out_stride, stage, r0, c, x);
        else
          store_out<float>(to, static_cast<float *>(p.out) + matrix * p.out_stride, stage, r0, c, x);
      } else {
        float *to = p.x32 + matrix * x32_rows(p.M) * p.ld + x32_at(p.ld, r, c);
        if (r < p.M) {
          store32(to, x);
          store32(to + 256, x + 8);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          sumsq = fmaf(x[k], x[k], sumsq);  // 0 in rows and columns behind the matrix
          x[k] *= kScaleX;
        }
        store_planes<P>(p.p0 + matrix * P * plane, plane, p.ld, p.M, r0, c, x, false, nullptr);
      }
    } else {
      uint8_t *turn = reinterpret_cast<uint8_t *>(stage);
      float x[16], d[16];
      const float scale = p.unscale * (STEP == kGram ? kScaleU : kScaleB);
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = v[k] * scale;
      if (STEP == kGram) {
        const float to_d = p.cc * (kScaleD / kScaleU);
        const bool diagonal = c < r0 + 32 && r0 < c + 16;  // some of these values are
        if (diagonal) {
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] -= r == c + k ? t * kScaleU : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) d[k] = x[k] * to_d;
        if (diagonal) {
          const float more = kScaleD * fmaf(2.0f * p.cc, t, p.cb);
#pragma unroll
          for (int k = 0; k < 16; ++k) d[k] += r == c + k ? more : 0.0f;
        }
      }
      store_planes<P>(p.p0 + matrix * P * plane, plane, p.ld, p.M, r0, c, x, mirror, turn);
      if (STEP == kGram)
        store_planes<P>(p.p1 + matrix * P * plane, plane, p.ld, p.M, r0, c, d, mirror, turn);
    }
  }

  // `slot`: this warp's among the sums of the matrix
  __device__ __forceinline__ void end(int slot, int count) {
    if (STEP != kApply || p.out) return;
    float s = sumsq;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) p.sums_out[matrix * count + slot] = s;
  }
};

// CG: CTAs that share one tile of CG * 128 rows (a pair splits the columns of
// B between its two shared memories).  BN: a tile's columns.  P: planes.
// Single CTAs may be in a cluster of p.split that shares a tile's K.
template <int P, int CG, int BN, NsStep STEP>
__global__ void __launch_bounds__(threads_of(P), 1)
ortho_kernel(const __grid_constant__ NsParams p) {
  constexpr bool SYM = STEP != kApply;
  constexpr int kRowsB = BN / CG, kABytes = 128 * kLine, kBBytes = kRowsB * kLine;
  constexpr uint32_t kStage = P * (kABytes + kBBytes);
  constexpr int kEpiWarps = epi_warps(P), kGroups = kEpiWarps / 4;  // those of the same rows
  constexpr int BLOCKS = BN / 16 / kGroups;  // of 16 columns of a warp
  using A = Acc<P, BN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  const uint32_t stages = (uint32_t)p.stages;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + stages * kStage);
  uint64_t *empty = full + kMaxStages;
  uint64_t *acc_full = empty + kMaxStages;  // [A::BARS]
  uint64_t *acc_empty = acc_full + 3;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 3);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  float *epi = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(full) + 256);
  uint8_t *exchange = reinterpret_cast<uint8_t *>(full) + 256 + epi_bytes(P);  // kExchange, if split

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int shared_by = CG == 2 ? 2 : p.split;  // CTAs of a tile
  const uint32_t rank = shared_by == 1 ? 0 : cta_rank();
  const uint32_t pair_rank = CG == 2 ? rank : 0, part = CG == 2 ? 0 : rank;
  const int64_t worker = blockIdx.x / shared_by, workers = gridDim.x / shared_by;
  // this CTA's K blocks, one at least
  const int kb0 = (int)((int64_t)p.kb * part / p.split);
  const int kbs = (int)((int64_t)p.kb * (part + 1) / p.split) - kb0;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < A::BARS; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], CG * kEpiWarps);  // every epilogue warp of the tile
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&p.a);
    prefetch_tmap(&p.b);
  }
  if (warp == 1) pair_tmem_alloc<CG>(tmem_slot, A::COLS);
  tc_fence_before();
  __syncthreads();
  if (shared_by > 1) cluster_sync();  // the others' shared memory is written from here on
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // operands come from the passes before it in the stream
  grid_dependency_wait();
  grid_launch_dependents();
  fence_async_global();
  bool ok = true;
  bool exchanged = CG == 2 || shared_by == 1;  // the sums of a tile whose K is split
  if (warp == 0) {
    // ---------------- producer: this CTA's rows of A and columns of B
    if (lane == 0 && !p.stall_producer) {
      uint32_t s = 0, ph = 1;
      auto take = [&] {
        ok = role_wait(&empty[s], ph, p.wait_ns, abort_flag);
        return ok;
      };
      auto next = [&] {
        if (++s == stages) s = 0, ph ^= 1;
      };
      for (int64_t tile = worker; ok && tile < p.tiles; tile += workers) {
        const TileAt at = tile_at<SYM>(p, tile);
        const int32_t m0 = at.m * (CG * 128) + (int32_t)pair_rank * 128;
        const int32_t n0 = at.n * BN + (int32_t)pair_rank * kRowsB;
        const int z = (int)at.matrix * P;
        for (int kb = 0; kb < kbs && take(); ++kb, next()) {
          if (pair_rank == 0) mbar_expect_tx(&full[s], CG * kStage);
          const uint32_t bar = CG == 1 ? smem_u32(&full[s]) : map_to_cta(smem_u32(&full[s]), 0);
          const int32_t k0 = (kb0 + kb) * kBlockK;
          const uint32_t a = smem_u32(smem) + s * kStage, b = a + P * kABytes;
#pragma unroll
          for (int q = 0; q < P; ++q) {
            load_tile<CG>(a + q * kABytes, &p.a, bar, 0, 128, m0, k0, z + q);
            load_tile<CG>(b + q * kBBytes, &p.b, bar, !SYM, kRowsB, n0, k0, z + q);
          }
        }
      }
      // Every stage handed back: no load is in flight and no arrival from the
      // pair's MMAs still on its way here (see ff_tc.cu).
      for (uint32_t i = 0; i < stages && ok; ++i) {
        take();
        next();
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (of the pair)
    if (lane == 0 && pair_rank == 0) {
      // FP16 operands, FP32 sums; B of the apply step MN-major
      constexpr uint32_t idesc = (1u << 4) | ((uint32_t)!SYM << 16) | ((uint32_t)(BN >> 3) << 17) |
                                 ((uint32_t)((CG * 128) >> 4) << 24);
      constexpr uint64_t astep = 32 >> 4, bstep = SYM ? 32 >> 4 : 2048 >> 4;
      uint32_t s = 0, ph = 0, filled = 0;
      auto take = [&](int i) {
        ok = role_wait(&acc_empty[i], ((filled >> i) & 1u) ^ 1u, p.wait_ns, abort_flag);
        filled ^= 1u << i;
        tc_fence_after();
        return ok;
      };
      int acc = A::LARGE - 1;
      for (int64_t tile = worker; ok && tile < p.tiles; tile += workers) {
        if (P == 1) {
          acc ^= 1;
          if (!take(acc)) break;
        }
        for (int kb = 0; kb < kbs; ++kb) {
          if (!role_wait(&full[s], ph, p.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem) + s * kStage, b = a + P * kABytes;
          const uint64_t da = tile_desc(a, 0), db = tile_desc(b, !SYM);
          if (P == 2 && kb % kFlush == 0) {
            if (A::LARGE == 2) acc ^= 1;
            if (!take(acc)) break;
          }
          const uint32_t d = tmem_base + (uint32_t)(acc * BN);
          const bool first = P == 1 ? kb == 0 : kb % kFlush == 0;
#pragma unroll
          for (int kk = 0; kk < kBlockK / 16; ++kk)
            mma_16bit<CG>(d, da + kk * astep, db + kk * bstep, idesc, first && kk == 0 ? 0u : 1u);
          if constexpr (P == 2) {
            if (kb % kFlush == kFlush - 1 || kb == kbs - 1) commit<CG>(&acc_full[acc]);
            if (kb == 0 && !take(A::SMALL)) break;
            const uint32_t e = tmem_base + (uint32_t)(A::SMALL * BN);
#pragma unroll
            for (int kk = 0; kk < kBlockK / 16; ++kk) {
              mma_16bit<CG>(e, da + kk * astep, db + kk * bstep + (kBBytes >> 4), idesc,
                            kb > 0 || kk > 0 ? 1u : 0u);
              mma_16bit<CG>(e, da + kk * astep + (kABytes >> 4), db + kk * bstep, idesc, 1u);
            }
          }
          commit<CG>(&empty[s]);
          if (++s == stages) s = 0, ph ^= 1;
        }
        if (ok) commit<CG>(&acc_full[P == 1 ? acc : A::SMALL]);
      }
    }
  } else {
    // ---------------- epilogue: a warp has 32 rows (the tensor-memory lanes
    // 32 (w & 3) on) and every kGroups-th 16 columns of the tile
    const int quarter = warp & 3, group = (warp - 2) >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const int warp_slot = (int)rank * kEpiWarps + warp - 2, slots = shared_by * kEpiWarps;
    Finish<P, STEP> out{p, epi + (warp - 2) * (kEpiStage / 4), 0, -1, false, 0.0f, 0.0f, 0.0f};
    uint32_t drained = 0;
    int acc = A::LARGE - 1;
    // tcgen05.ld is warp-collective: the warp proceeds or stops as one
    auto wait_full = [&](int i) {
      ok = __all_sync(0xffffffffu,
                      role_wait(&acc_full[i], (drained >> i) & 1u, p.wait_ns, abort_flag));
      drained ^= 1u << i;
      tc_fence_after();
      return ok;
    };
    auto release = [&](int i) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader<CG>(&acc_empty[i]);
    };
    // Split K: of the tile's blocks of 16 columns each CTA finishes `share`, in turn.
    // Block b of these rows goes there, to the place of this CTA: [source][block of
    // the owner][4 values][row].
    const int share = BN / 16 / (CG == 1 ? shared_by : 1), row = quarter * 32 + lane;
    auto send = [&](int b, const float (&v)[16]) {
      const uint32_t to = map_to_cta(smem_u32(exchange), (uint32_t)(b / share));
      const uint32_t at = to + (uint32_t)((((int)rank * share + b % share) * 4 * 128 + row) * 16);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        cluster_store(at + k * 128 * 16,
                      make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
    };
    for (int64_t tile = worker; ok && tile < p.tiles; tile += workers) {
      const TileAt at = tile_at<SYM>(p, tile);
      const bool split = CG == 1 && shared_by > 1;  // one tile a cluster
      // this warp's blocks of 16 columns: group, group + kGroups, ... of the CTA's
      const int first = split ? (int)rank * share : 0;
      const int own = split ? (share - group + kGroups - 1) / kGroups : BLOCKS;
      const int64_t c0 = (int64_t)at.n * BN + 16 * (first + group);
      out.begin(at, (int64_t)at.m * (CG * 128) + pair_rank * 128 + quarter * 32, warp_slot == 0);
      auto column = [&](int i) { return i < own ? c0 + 16 * kGroups * i : p.ld; };
      float x32[16];  // apply: X of the next block (of two or four, with two planes, no faster)
      // The tile's sums, where they stay in tensor memory.
      uint32_t sums;
      if constexpr (P == 1) {
        out.request(x32, column(0));
        acc ^= 1;
        if (!wait_full(acc)) break;
        sums = lane_base + (uint32_t)(acc * BN + 16 * group);
        if (split) {
#pragma unroll 1
          for (int i = 0; i < BLOCKS; ++i) {
            float v[16];
            tmem_ld16(sums + 16 * kGroups * i, v);
            tmem_ld_wait();
            send(group + kGroups * i, v);
          }
        }
      } else {
        float sum[BLOCKS][16];
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
          for (int k = 0; k < 16; ++k) sum[i][k] = 0.0f;
        const int gathers = (kbs + kFlush - 1) / kFlush + 1;
        for (int g = 0; g < gathers; ++g) {
          const bool small = g == gathers - 1;
          if (A::LARGE == 2 && !small) acc ^= 1;
          const int from = small ? A::SMALL : acc;
          if (!wait_full(from)) break;
#pragma unroll
          for (int i = 0; i < BLOCKS; ++i) {
            float x[16];
            tmem_ld16(lane_base + (uint32_t)(from * BN + 16 * (group + kGroups * i)), x);
            tmem_ld_wait();
            if (i == BLOCKS - 1 && !(A::KEEP && small)) release(from);
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[i][k] += x[k];
          }
        }
        if (!ok) break;
        // Back to tensor memory: what follows is a loop over blocks then (unrolled for
        // sums in registers, 8 blocks of it are 40 KB of code, and took 1 us each).
        sums = lane_base + (uint32_t)(A::SUMS * BN + 16 * group);
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i) {
          if (split)
            send(group + kGroups * i, sum[i]);
          else
            tmem_st16(sums + 16 * kGroups * i, sum[i]);
        }
        tmem_st_wait();
        out.request(x32, column(0));
      }
      if (split) {
        cluster_sync();
        exchanged = true;
      }
      const float4 *got = reinterpret_cast<const float4 *>(exchange) + row;
#pragma unroll 1
      for (int i = 0; i < own; ++i) {
        float v[16];
        if (split) {
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = 0.0f;
          for (int src = 0; src < shared_by; ++src) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 f = got[((src * share + group + kGroups * i) * 4 + k) * 128];
              v[4 * k] += f.x, v[4 * k + 1] += f.y, v[4 * k + 2] += f.z, v[4 * k + 3] += f.w;
            }
          }
        } else {
          tmem_ld16(sums + 16 * kGroups * i, v);
          tmem_ld_wait();
          if (i == BLOCKS - 1) {
            if (P == 1) release(acc);
            if (A::KEEP) release(A::SMALL);
          }
        }
        out.block(x32, column(i), column(i + 1), v);
      }
      out.end((int)(tile - at.matrix * p.per) * slots + warp_slot, p.per * slots);
    }
  }

  if (!ok) {
    *abort_flag = 1;
    atomicExch(&g_ortho_status, GEMM_ERR_DEVICE_TIMEOUT);
    // copies and MMAs still in flight land within microseconds: 1 ms, then out
    const uint64_t until = globaltimer() + 1000000ull;
    while (globaltimer() < until) __nanosleep(1000);
  }
  if (!exchanged) cluster_sync();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the pair's MMAs read both shared memories
  tc_fence_after();
  if (warp == 1) pair_tmem_dealloc<CG>(tmem_base, A::COLS);
}

// ------------------------------------------------------------------ host side

uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }
int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

// A tile: the CTAs that share its rows, its columns, the CTAs that share its K.
struct Choice {
  int cg, bn, split;
};

// Rows, columns and K of a step's product.
void extents(const OrthoSizes &q, NsStep step, int64_t *M, int64_t *N, int64_t *K) {
  *M = q.m;
  *N = step == kApply ? q.n : q.m;
  *K = step == kGram ? q.n : q.m;
}

int64_t tiles_per(const OrthoSizes &q, NsStep step, const Choice &c) {
  int64_t M, N, K;
  extents(q, step, &M, &N, &K);
  const int64_t tm = ceil_div(M, c.cg * 128), tn = ceil_div(N, c.bn);
  return step == kApply ? tm * tn : tm * (tm + 1) / 2;
}

int stage_bytes_of(int planes, const Choice &c) { return planes * (128 + c.bn / c.cg) * kLine; }

// The tile with the least estimated time, in clocks.  A K block takes what the
// MMAs, shared memory's reads and writes or the loads take (as in ff_tc.cu).  A
// tile's epilogue moves 8 + 2 P bytes a value of X, 8 P of U and D and 4 P of B, at
// 32 a clock (16 with two planes' 8 warps) with all SMs at it (L2 then gives 9
// TB/s); it runs beside the next tile's sums, but for a tile that keeps their
// place, and the last one's is not hidden.  A cluster that shares a tile's K
// exchanges sums in about 2000.  (Tiles of 256 x 128 by pairs, for X, were never
// faster than both of these by more than a hundredth.)
Choice choose(const OrthoSizes &q, NsStep step, int sms) {
  static const Choice all[] = {{2, 256, 1}, {1, 128, 1}, {1, 128, 2}, {1, 128, 4}, {1, 128, 8}};
  Choice best{};
  double least = 0.0;
  int64_t M, N, K;
  extents(q, step, &M, &N, &K);
  const int64_t blocks = ceil_div(K, kBlockK);
  const double P = q.planes, products = q.planes == 1 ? 1 : 3;
  for (const Choice &c : all) {
    const int64_t tiles = q.batch * tiles_per(q, step, c);
    if (c.split > 1 && (tiles > clusters_at_once(c.split) || blocks < c.split)) continue;
    const double mma = 4 * products * c.bn / 2.0;
    const double smem = 4 * products * (128 + c.bn) * 32 / 128.0 + stage_bytes_of(q.planes, c) / 128.0;
    const double load = stage_bytes_of(q.planes, c) / 50.0;
    double clocks = mma > smem ? mma : smem;
    if (load > clocks) clocks = load;
    const int64_t ctas = tiles * c.cg * c.split;
    const double busy = ctas < sms ? (double)ctas / sms : 1.0;
    double finish = 128.0 * c.bn / c.split / (q.planes == 1 ? 32.0 : 16.0) *
                    (busy > 0.5 ? busy : 0.5) *
                    (step == kApply ? 8 + 2 * P : step == kGram ? 8 * P : 4 * P);
    const double sum = (double)ceil_div(blocks, c.split) * clocks;
    const double waves = c.split > 1 ? 1.0 : (double)ceil_div(tiles, sms / c.cg);
    const bool keep = q.planes == 2 && c.bn == 256;
    const double t = (keep ? waves * (sum + finish) : waves * (sum > finish ? sum : finish) + finish) +
                     (c.split > 1 ? 2000.0 : 0.0);
    if (least == 0.0 || t < least) {
      least = t;
      best = c;
    }
  }
  return best;
}

template <int P, int CG, int BN, NsStep STEP>
int launch_step(NsParams &l, const Choice &c, const DeviceProps &dp, cudaStream_t s) {
  const int stage = stage_bytes_of(P, c);
  int64_t workers = dp.sm_count / (c.cg > 1 ? c.cg : c.split);
  if (c.split > 1 || workers > l.tiles) workers = l.tiles;
  const int cluster = c.cg > 1 ? c.cg : c.split;
  const int extra = c.split > 1 ? kExchange : 0;
  l.stages = (stage_budget(P) - extra) / stage;
  if (l.stages > kMaxStages) l.stages = kMaxStages;
  auto kern = ortho_kernel<P, CG, BN, STEP>;
  static Once once;
  if (allow_shared_memory(once, kern, 227 * 1024, dp.device) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(workers * cluster));
  lc.blockDim = dim3(threads_of(P));
  lc.dynamicSmemBytes = (size_t)l.stages * stage + 1024 + 256 + epi_bytes(P) + extra;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 2;
  if (cudaLaunchKernelEx(&lc, kern, l) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

template <int P, NsStep STEP>
int launch_tile(NsParams &l, const Choice &c, const DeviceProps &dp, cudaStream_t s) {
  return c.cg == 2 ? launch_step<P, 2, 256, STEP>(l, c, dp, s)
                   : launch_step<P, 1, 128, STEP>(l, c, dp, s);
}

template <NsStep STEP>
int launch(NsParams &l, int planes, const Choice &c, const DeviceProps &dp, cudaStream_t s) {
  return planes == 1 ? launch_tile<1, STEP>(l, c, dp, s) : launch_tile<2, STEP>(l, c, dp, s);
}

// The buffers of a call, one after the other in its workspace.
struct Layout {
  int64_t ldx, ldm, blocks, sums;  // blocks of the norm for each matrix; most parts of |X|^2
  uint64_t x32, x16[2], u, d, b, partial, part[2], t, end;
};

Layout layout_of(const OrthoSizes &q, int sms) {
  Layout y{};
  y.ldx = round16(q.n);
  y.ldm = round16(q.m);
  const int64_t tiles = ceil_div(q.m, kPrepTile) * ceil_div(q.n, kPrepTile);
  const int64_t most = ceil_div((int64_t)sms * 4, q.batch);  // the norm's
  y.blocks = tiles < most ? tiles : most;
  // the apply step's smallest tiles, and every warp of their clusters
  y.sums = ceil_div(q.m, 128) * ceil_div(q.n, 128) * kMaxSplit * epi_warps(q.planes);
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t a = at;
    at += align256(bytes);
    return a;
  };
  const uint64_t xs = (uint64_t)q.batch * q.m * y.ldx, ms = (uint64_t)q.batch * q.m * y.ldm;
  y.x32 = take((uint64_t)q.batch * x32_rows(q.m) * y.ldx * 4);
  for (uint64_t &x : y.x16) x = take(xs * 2 * q.planes);
  y.u = take(ms * 2 * q.planes);
  y.d = take(ms * 2 * q.planes);
  y.b = take(ms * 2 * q.planes);
  y.partial = take((uint64_t)q.batch * y.blocks * 8);
  for (uint64_t &x : y.part) x = take((uint64_t)q.batch * y.sums * 4);
  y.t = take((uint64_t)q.batch * 4);
  y.end = at;
  return y;
}

OrthoSizes sizes_of(int dtype, int64_t batch, int64_t M, int64_t N) {
  const int64_t m = M < N ? M : N, n = M < N ? N : M;
  return {dtype == GEMM_DT_F32 || n > kOnePlaneK ? 2 : 1, batch, m, n};
}

// Whether the singular values, from 1 at most, and what the steps make of them
// stay where the FP16 factors hold them: X up to s, U up to l = s s (t is at most the
// largest eigenvalue), D up to |b| + 2 |c| t + |c| l, and B, which is b x + c x x at an
// eigenvalue less that at t.
bool in_range(int steps, const float *abc) {
  double s = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double a = abc[3 * i], b = abc[3 * i + 1], c = abc[3 * i + 2], l = s * s;
    // b x + c x x over [0, l]
    double lo = 0.0, hi = 0.0;
    auto see = [&](double x) {
      if (!(x > 0.0 && x <= l)) return;
      const double v = (b + c * x) * x;
      lo = v < lo ? v : lo;
      hi = v > hi ? v : hi;
    };
    see(l);
    if (c != 0.0) see(-b / (2.0 * c));
    if (!(s <= kMostX && l <= kMostU && std::fabs(b) + 3.0 * std::fabs(c) * l <= kMostD &&
          hi - lo <= kMostB))
      return false;
    // |a x + b x^3 + c x^5| over [0, s]: at s, and where a + 3 b y + 5 c y^2 = 0, y = x^2
    double most = std::fabs(((c * l + b) * l + a) * s);
    auto turn = [&](double y) {
      if (!(y > 0.0 && y < l)) return;
      const double v = std::fabs(((c * y + b) * y + a) * std::sqrt(y));
      most = v > most ? v : most;
    };
    if (c != 0.0) {
      const double disc = 9.0 * b * b - 20.0 * a * c;
      if (disc >= 0.0) {
        turn((-3.0 * b + std::sqrt(disc)) / (10.0 * c));
        turn((-3.0 * b - std::sqrt(disc)) / (10.0 * c));
      }
    } else if (b != 0.0) {
      turn(-a / (3.0 * b));
    }
    s = 1.001 * most;
  }
  return s < 1e30;
}

constexpr int64_t kMaxExtent = ((int64_t)1 << 31) - 512;
constexpr int64_t kMaxLd = (int64_t)1 << 36;

int check_sizes(int dtype, int64_t batch, int64_t M, int64_t N) {
  if (!dtype_known(dtype) || batch < 0 || M < 0 || N < 0) return GEMM_ERR_INVALID_ARG;
  const int64_t m = M < N ? M : N, n = M < N ? N : M;
  // tiles of a launch and rows of the matrices' planes count in 32 bits
  if (n > kMaxExtent || m > ((int64_t)1 << 20) || batch > 65535) return GEMM_ERR_UNSUPPORTED;
  if (m > 0 && ceil_div(m, 128) * ceil_div(n, 128) > ((int64_t)1 << 24) / (batch > 0 ? batch : 1))
    return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

// Whether no two of `batch` M x N matrices share an element, whose rows are ldo and
// which themselves are `stride` elements apart: one after the other, or row by row
// side by side.
bool results_apart(int64_t batch, int64_t M, int64_t N, int64_t ldo, int64_t stride) {
  if (stride < N) return batch < 2 || M == 0 || N == 0;
  int64_t at = 0;  // where matrix d begins, in the first one's rows
  for (int64_t d = 1; d < batch; ++d) {
    if (at > INT64_MAX - stride) return true;
    at += stride;
    const int64_t row = at / ldo, col = at % ldo;
    if (row >= M || (row == M - 1 && col >= N)) return true;  // behind it, as are all others
    if (col < N || (row + 1 < M && ldo - col < N)) return false;
  }
  return true;
}

template <typename... Params, typename... Args>
cudaError_t launch_prep(void (*kern)(Params...), dim3 grid, cudaStream_t s, const Args &...args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(kPrepThreads);
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kern, Params(args)...);
}

template <typename T, bool VEC>
cudaError_t prepare(const PrepParams &p, int planes, int64_t batch, int blocks, int64_t tiles,
                    int sms, cudaStream_t s) {
  cudaError_t e = launch_prep(ortho_norm_kernel<T>, dim3(blocks, (unsigned)batch), s, p);
  if (e != cudaSuccess) return e;
  const int64_t most = ceil_div((int64_t)sms * 8, batch);
  const dim3 grid((unsigned)(tiles < most ? tiles : most), (unsigned)batch);
  if constexpr (std::is_same<T, bf16>::value)  // FP32 always has two planes
    if (planes == 1) return launch_prep(ortho_scale_kernel<T, VEC, 1>, grid, s, p, blocks);
  return launch_prep(ortho_scale_kernel<T, VEC, 2>, grid, s, p, blocks);
}

}  // namespace

int ortho_read_and_clear_status(cudaStream_t s) {
  int v = 0;
  if (!g_ortho_ran.load(std::memory_order_relaxed)) return ortho_small_read_and_clear_status(s);
  if (cudaMemcpyFromSymbolAsync(&v, g_ortho_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(g_ortho_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice,
                                s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_CUDA;
    }
  }
  return v != GEMM_OK ? v : ortho_small_read_and_clear_status(s);
}

}  // namespace gg

using namespace gg;

extern "C" {

int orthogonalize_workspace(int dtype, int64_t batch, int64_t M, int64_t N, uint64_t *bytes) {
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  const int st = check_sizes(dtype, batch, M, N);
  if (st != GEMM_OK) return st;
  *bytes = 0;
  if (batch == 0 || M == 0 || N == 0) return GEMM_OK;
  const OrthoSizes q = sizes_of(dtype, batch, M, N);
  const int sms = current_props().sm_count;
  if (!ortho_small_fits({q.planes, batch, q.m, q.n})) *bytes = layout_of(q, sms).end;
  return GEMM_OK;
}

int orthogonalize(int dtype, int64_t batch, int64_t M, int64_t N, const void *G, int64_t ldg,
                  int64_t stride_g, void *O, int64_t ldo, int64_t stride_o, int steps,
                  const float *coefficients, double eps, void *workspace, size_t ws_bytes,
                  cudaStream_t stream) {
  int st = check_sizes(dtype, batch, M, N);
  if (st != GEMM_OK) return st;
  if (steps < 1 || !coefficients || !(eps >= 0.0) || std::isinf(eps)) return GEMM_ERR_INVALID_ARG;
  if (steps > kOrthoMaxSteps) return GEMM_ERR_UNSUPPORTED;
  for (int i = 0; i < 3 * steps; ++i)
    if (!std::isfinite(coefficients[i])) return GEMM_ERR_INVALID_ARG;
  const uintptr_t mask = dtype_size(dtype) - 1;
  const int64_t width = N > 1 ? N : 1;
  if (ldg < width || ldo < width || ldg > kMaxLd || ldo > kMaxLd) return GEMM_ERR_INVALID_ARG;
  if (batch > 1 && (stride_g < 0 || stride_o < 0)) return GEMM_ERR_INVALID_ARG;
  if (!results_apart(batch, M, N, ldo, stride_o)) return GEMM_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return GEMM_ERR_INVALID_ARG;
  if (batch > 0 && M > 0 && N > 0 &&
      (!G || !O || ((reinterpret_cast<uintptr_t>(G) | reinterpret_cast<uintptr_t>(O)) & mask)))
    return GEMM_ERR_INVALID_ARG;
  if (!in_range(steps, coefficients)) return GEMM_ERR_UNSUPPORTED;
  if (batch == 0 || M == 0 || N == 0) return GEMM_OK;
  int dev = -1;
  st = current_device(&dev);
  if (st != GEMM_OK) return st;
  const DeviceProps &dp = props_of(dev);
  if (!tc_supported(dp)) return GEMM_ERR_UNSUPPORTED;
  if (!tensor_map_encoder()) return GEMM_ERR_CUDA;

  const OrthoSizes q = sizes_of(dtype, batch, M, N);
  if (ortho_small_fits({q.planes, batch, q.m, q.n}))
    return launch_ortho_small({q.planes, batch, q.m, q.n}, {dtype, M, N, G, ldg,
                                                            batch > 1 ? stride_g : 0, O, ldo,
                                                            batch > 1 ? stride_o : 0, steps,
                                                            coefficients, eps},
                              dp, stream);
  const Layout y = layout_of(q, dp.sm_count);
  void *given = workspace;
  if (workspace && ws_bytes < y.end) return GEMM_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace) {
    st = library_workspace(dev, (size_t)y.end, &given);
    if (st != GEMM_OK) return st;
  }
  g_ortho_ran.store(true, std::memory_order_relaxed);
  uint8_t *ws = static_cast<uint8_t *>(given);
  auto at = [&](uint64_t offset) { return static_cast<void *>(ws + offset); };

  const int64_t size = (int64_t)dtype_size(dtype);
  PrepParams pp{};
  pp.g = G;
  pp.ldg = ldg;
  pp.stride = batch > 1 ? stride_g : 0;
  pp.rows = M;
  pp.cols = N;
  pp.m = q.m;
  pp.n = q.n;
  pp.ldx = y.ldx;
  pp.transposed = M > N;
  pp.eps = eps;
  pp.partial = static_cast<double *>(at(y.partial));
  pp.x32 = static_cast<float *>(at(y.x32));
  pp.x16 = static_cast<__half *>(at(y.x16[0]));
  pp.sumsq = static_cast<float *>(at(y.part[0]));
  const bool vec = ((reinterpret_cast<uintptr_t>(G) | (uintptr_t)(ldg * size) |
                     (uintptr_t)(pp.stride * size)) & 15) == 0;
  const int64_t tiles = ceil_div(q.m, kPrepTile) * ceil_div(q.n, kPrepTile);
  cudaError_t e;
  if (dtype == GEMM_DT_F32)
    e = vec ? prepare<float, true>(pp, q.planes, batch, (int)y.blocks, tiles, dp.sm_count, stream)
            : prepare<float, false>(pp, q.planes, batch, (int)y.blocks, tiles, dp.sm_count, stream);
  else
    e = vec ? prepare<bf16, true>(pp, q.planes, batch, (int)y.blocks, tiles, dp.sm_count, stream)
            : prepare<bf16, false>(pp, q.planes, batch, (int)y.blocks, tiles, dp.sm_count, stream);
  if (e != cudaSuccess) return to_status(e);

  const auto f16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int64_t planes = q.planes * batch, xp = q.m * y.ldx, mp = q.m * y.ldm;
  const Choice cg = choose(q, kGram, dp.sm_count), cp = choose(q, kPoly, dp.sm_count),
               ca = choose(q, kApply, dp.sm_count);
  int sum_count = 1;
  for (int i = 0; i < steps; ++i) {
    const int in = i & 1;
    // Parameters of one product, and the maps of its operands.
    auto params = [&](NsStep step, const Choice &c, uint64_t a, uint64_t b, bool &fine) {
      NsParams l{};
      int64_t K;
      extents(q, step, &l.M, &l.N, &K);
      l.tiles_m = (int)ceil_div(l.M, c.cg * 128);
      l.tiles_n = (int)ceil_div(l.N, c.bn);
      l.per = (int)tiles_per(q, step, c);
      l.tiles = l.per * batch;
      l.group_n = l.tiles_n < 8 ? l.tiles_n : 8;
      l.kb = (int)ceil_div(K, kBlockK);
      l.split = c.split;
      l.ca = coefficients[3 * i];
      l.cb = coefficients[3 * i + 1];
      l.cc = coefficients[3 * i + 2];
      l.t = static_cast<float *>(at(y.t));
      l.sums = static_cast<const float *>(at(y.part[in]));
      l.sum_count = sum_count;
      l.sums_out = static_cast<float *>(at(y.part[in ^ 1]));
      l.ld = step == kApply ? y.ldx : y.ldm;
      l.wait_ns = env_u64("GEMM_DEBUG_WAIT_LIMIT_NS", 2000000000ull) + (uint64_t)l.kb * 8000;
      l.stall_producer = (int)env_u64("GEMM_DEBUG_STALL_PRODUCER", 0);
      const bool x_rows = step == kGram;
      fine = encode_planes(&l.a, f16, at(a), x_rows ? q.n : q.m, q.m, x_rows ? y.ldx : y.ldm,
                           planes, x_rows ? xp : mp, 128) &&
             (step == kApply
                  ? encode_planes(&l.b, f16, at(b), q.n, q.m, y.ldx, planes, xp, 64)
                  : encode_planes(&l.b, f16, at(b), x_rows ? q.n : q.m, q.m,
                                  x_rows ? y.ldx : y.ldm, planes, x_rows ? xp : mp,
                                  c.bn / c.cg));
      return l;
    };
    bool fine = true;
    NsParams l = params(kGram, cg, y.x16[in], y.x16[in], fine);
    if (!fine) return GEMM_ERR_UNSUPPORTED;
    l.unscale = 1.0f / (kScaleX * kScaleX);
    l.p0 = static_cast<__half *>(at(y.u));
    l.p1 = static_cast<__half *>(at(y.d));
    st = launch<kGram>(l, q.planes, cg, dp, stream);
    if (st != GEMM_OK) return st;

    l = params(kPoly, cp, y.u, y.d, fine);
    if (!fine) return GEMM_ERR_UNSUPPORTED;
    l.unscale = 1.0f / (kScaleU * kScaleD);
    l.p0 = static_cast<__half *>(at(y.b));
    st = launch<kPoly>(l, q.planes, cp, dp, stream);
    if (st != GEMM_OK) return st;

    l = params(kApply, ca, y.b, y.x16[in], fine);
    if (!fine) return GEMM_ERR_UNSUPPORTED;
    l.unscale = 1.0f / (kScaleB * kScaleX);
    l.x32 = static_cast<float *>(at(y.x32));
    l.p0 = static_cast<__half *>(at(y.x16[in ^ 1]));
    if (i == steps - 1) {
      l.out = O;
      l.ldo = ldo;
      l.out_stride = batch > 1 ? stride_o : 0;
      l.out_t = M > N;
      l.out_bf16 = dtype == GEMM_DT_BF16;
    }
    st = launch<kApply>(l, q.planes, ca, dp, stream);
    if (st != GEMM_OK) return st;
    sum_count = l.per * (ca.cg > 1 ? ca.cg : ca.split) * epi_warps(q.planes);
  }
  return GEMM_OK;
}

}  // extern "C"
