// Orthogonalised updates of matrices whose smaller side m is at most 128, on chip.
// The steps and their planes are those of ortho.cu; D alone is rounded otherwise: it is
// made of U as its planes hold it, there of the sums before they are rounded to them.
//
// The general kernels spend 15 launches of 5 to 8 us on such a matrix, whatever
// its size.  Here a cluster of up to 16 CTAs holds it for all steps: each CTA has
// nc columns of X, in FP32 in tensor memory and as FP16 planes in shared memory,
// and a step is
//   X X^T of its columns (one MMA tile of 128 x 128), drained and sent, 128 / C rows
//     to each of the C CTAs, through distributed shared memory;
//   U, of those rows, added up in a fixed order and copied to all;
//   D from U, B = U D and B X (every CTA makes B for itself: 128 x 128 x 128 is
//     less than what its exchange would take).
// Both operands of a product are read from shared memory as they lie: the same
// planes of X are K-major for X X^T and MN-major for B X.
// Times at ortho_small_fits.
#include <atomic>
#include <cmath>

#include "ortho.cuh"

namespace gg {

using namespace tc;

namespace {

__device__ int g_small_status;           // 0 = ok, else a GEMM_ERR_* code
std::atomic<bool> g_small_ran{false};    // as g_ortho_ran

constexpr int kThreads = 512;  // 16 warps: four for each 32 rows
constexpr int kWarps = kThreads / 32, kStep = 16 * kWarps / 4;  // columns of all warps' blocks
constexpr int kSide = 128;     // rows of X and of U, with those behind m
constexpr int kPlane = kSide * kSide * 2;  // bytes of a plane of U, D or B
constexpr int kXBytes = 65536, kExchange = kSide * kSide * 4;
constexpr int kMaxCluster = 16;
// X's columns in tensor memory, and the accumulators: two planes' small products in the
// upper half of theirs
constexpr uint32_t kAcc = 256, kSmall = 128;

struct SmallParams {
  const void *g;
  int64_t ldg, stride_g;
  void *o;
  int64_t ldo, stride_o;
  int m, n, nc;  // nc: columns of a CTA, a multiple of 64
  int transposed, vec;
  int steps;
  double eps;
  uint64_t wait_ns;
  int stall;     // test hook: no MMA is issued
  float abc[3 * kOrthoMaxSteps];
};

// Shared memory: planes of X; of U, then B; of D (two planes: in the place of the
// exchange); the exchange; and small things.
template <int P>
constexpr int smem_bytes() {
  return 1024 + kXBytes + P * kPlane + (P == 1 ? kPlane + kExchange : P * kPlane) + 1024;
}

struct SmallShared {
  uint64_t bar, u_bar;  // the MMAs; the other CTAs' rows of U
  uint32_t tmem;
  int abort;
  double part[kWarps], norm2[kMaxCluster], inv;
  float warp_sum[kWarps], sum[kMaxCluster];  // |X|^2 of each CTA's columns
};

// The byte of element (r, c), c a multiple of 4, in a plane of 128-byte-swizzled
// blocks of 64 columns.
__device__ __forceinline__ uint32_t at_plane(int r, int c) {
  return (uint32_t)((c >> 6) * (kSide * kLine) + r * kLine + (((((c & 63) >> 3) ^ (r & 7)) << 4) |
                                                              ((c & 4) << 1)));
}

// N floats as FP16 planes: u[q][i] holds values 2 i and 2 i + 1 of plane q.
template <int P, int N>
__device__ __forceinline__ void split_planes(float (&x)[N], uint32_t (&u)[P][N / 2]) {
#pragma unroll
  for (int q = 0; q < P; ++q)
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const __half2 h = __floats2half2_rn(x[k], x[k + 1]);
      if (q + 1 < P) {
        const float2 f = __half22float2(h);
        x[k] -= f.x, x[k + 1] -= f.y;
      }
      u[q][k / 2] = *reinterpret_cast<const uint32_t *>(&h);
    }
}

// 16 values of row r from column c on (a multiple of 16) to planes at `to`.
template <int P>
__device__ __forceinline__ void store16(uint8_t *to, int plane, int r, int c, float (&x)[16]) {
  uint32_t u[P][8];
  split_planes<P, 16>(x, u);
#pragma unroll
  for (int q = 0; q < P; ++q)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint4 *>(to + q * plane + at_plane(r, c + 8 * h)) =
          make_uint4(u[q][4 * h], u[q][4 * h + 1], u[q][4 * h + 2], u[q][4 * h + 3]);
}

// Shared memory to another CTA's, counted on a barrier there.
__device__ __forceinline__ void cluster_copy(uint32_t to, uint32_t from, uint32_t bytes,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(to),
      "r"(from), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void cluster_store_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_store_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// 16 values of row i of X from column j on, 0 behind the matrix.
template <typename T>
__device__ __forceinline__ void load_row(const SmallParams &p, const T *g, int i, int j,
                                         float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] = 0.0f;
  if (i >= p.m) return;
  if (p.transposed) {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (j + k < p.n) x[k] = to_f32(g[(int64_t)(j + k) * p.ldg + i]);
  } else if (p.vec && j + 16 <= p.n) {
    __align__(16) T t[16];
    const uint4 *from = reinterpret_cast<const uint4 *>(g + (int64_t)i * p.ldg + j);
#pragma unroll
    for (int k = 0; k < (int)sizeof(T); ++k) reinterpret_cast<uint4 *>(t)[k] = __ldg(from + k);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = to_f32(t[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (j + k < p.n) x[k] = to_f32(g[(int64_t)i * p.ldg + j + k]);
  }
}

// D(tmem) = A B over `steps` times 16 of K, 4 of them a block of A: both K-major
// (b_mn = 0), or B MN-major.  Two planes: the large products at d, the small ones at
// d + small.
template <int P>
__device__ __forceinline__ void multiply(uint32_t d, uint32_t small, uint32_t a, uint32_t a_plane,
                                         uint32_t b, uint32_t b_plane, int steps, int b_mn, int N) {
  const uint32_t idesc = (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
                         ((uint32_t)(kSide >> 4) << 24);
  constexpr uint32_t kBlock = kSide * kLine;  // of 64 columns
  for (int k = 0; k < steps; ++k) {
    const uint32_t ka = (uint32_t)(k >> 2) * kBlock + (uint32_t)(k & 3) * 32;
    const uint32_t kb = b_mn ? (uint32_t)k * 2048 : ka;
    auto da = [&](int q) { return smem_desc(a + q * a_plane + ka, 1024, 2); };
    auto db = [&](int q) {
      return smem_desc(b + q * b_plane + kb, 1024, 2) +
             (b_mn ? (uint64_t)((kBlock >> 4) - 1) << 16 : 0);
    };
    const uint32_t more = k > 0;
    mma_16bit<1>(d, da(0), db(0), idesc, more);
    if constexpr (P == 2) {
      mma_16bit<1>(d + small, da(0), db(1), idesc, more);
      mma_16bit<1>(d + small, da(1), db(0), idesc, 1u);
    }
  }
}

template <int P, typename T>
__global__ void __launch_bounds__(kThreads, 1)
ortho_small_kernel(const __grid_constant__ SmallParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *xs = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                            ~uintptr_t(1023));
  uint8_t *us = xs + kXBytes, *ds = us + P * kPlane;
  uint8_t *exchange = P == 1 ? ds + kPlane : ds;
  SmallShared &sh = *reinterpret_cast<SmallShared *>(P == 1 ? exchange + kExchange
                                                            : ds + P * kPlane);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quarter = warp & 3, group = warp >> 2, row = quarter * 32 + lane;
  const int x_plane = (p.nc >> 6) * kSide * kLine;
  int rank, C;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const int64_t matrix = blockIdx.x / C;
  const T *g = static_cast<const T *>(p.g) + matrix * p.stride_g;
  const int j0 = rank * p.nc;  // the first of this CTA's columns

  if (tid == 0) {
    mbar_init(&sh.bar, 1);
    mbar_init(&sh.u_bar, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) pair_tmem_alloc<1>(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the others' shared memory is written from here on
  tc_fence_after();
  const uint32_t tmem = sh.tmem, lanes = tmem + ((uint32_t)(quarter * 32) << 16);
  grid_dependency_wait();
  grid_launch_dependents();

  bool ok = true;
  uint32_t phase = 0;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (ok) ok = role_wait(bar, parity, p.wait_ns, &sh.abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) sh.abort = 1;
  };
  // Everything that the warps wrote to shared memory is there for the MMAs, which
  // thread 0 issues; all wait for them.
  auto products = [&](auto issue) {
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && !p.stall) {
      issue();
      mma_commit(&sh.bar);
    }
    __syncwarp();
    wait(&sh.bar, phase);
    phase ^= 1;
    tc_fence_after();
  };
  // The sums of 16 columns from c on: of the large and the small products.
  auto sums = [&](uint32_t c, uint32_t small, float (&v)[16]) {
    tmem_ld16(lanes + kAcc + c, v);
    if constexpr (P == 2) {
      float w[16];
      tmem_ld16(lanes + kAcc + small + c, w);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] += w[k];
    } else {
      tmem_ld_wait();
    }
  };
  auto remote = [&](const void *local, int to) { return map_to_cta(smem_u32(local), (uint32_t)to); };

  // G's columns to tensor memory, and the norm: 16 squares in FP32 where they neither
  // over- nor underflow, then in FP64
  double sum = 0.0;
  for (int c = 16 * group; c < p.nc; c += kStep) {
    float x[16];
    load_row<T>(p, g, row, j0 + c, x);
    sum += squares([&](float scale) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float y = x[k] * scale;
        s = fmaf(y, y, s);
      }
      return s;
    });
    tmem_st16(lanes + (uint32_t)c, x);
  }
  tmem_st_wait();
  sum = warp_sum(sum);
  if (lane == 0) sh.part[warp] = sum;
  __syncthreads();
  if (tid < C) {
    double all = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += sh.part[w];
    cluster_store_f64(remote(&sh.norm2[rank], tid), all);
  }
  cluster_sync();
  if (tid == 0) {
    double all = 0.0;
    for (int c = 0; c < C; ++c) all += sh.norm2[c];
    const double norm = sqrt(all);
    sh.inv = 1.0 / (norm + p.eps);
    sh.sum[0] = (float)(norm * sh.inv * norm * sh.inv);
    for (int c = 1; c < C; ++c) sh.sum[c] = 0.0f;
  }
  __syncthreads();
  {
    const double inv = sh.inv;
    const float f = (float)inv;
    // beyond FP32's normal range the factor is applied in FP64
    const bool plain = (f >= 0x1p-126f && f <= 0x1p126f) || !(inv > 0.0 && inv < INFINITY);
    for (int c = 16 * group; c < p.nc; c += kStep) {
      float x[16];
      tmem_ld16(lanes + (uint32_t)c, x);
      tmem_ld_wait();
      if (plain) {
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] *= f;
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = (float)((double)x[k] * inv);
      }
      // rows and columns behind the matrix stay 0 (0 times an Inf is not)
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (row >= p.m || j0 + c + k >= p.n) x[k] = 0.0f;
      tmem_st16(lanes + (uint32_t)c, x);
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] *= kScaleX;
      store16<P>(xs, x_plane, row, c, x);
    }
    tmem_st_wait();
  }

  const int chunk = kSide / C;  // rows of U that this CTA adds up, from rank * chunk on
  for (int step = 0; step < p.steps; ++step) {
    const float ca = p.abc[3 * step], cb = p.abc[3 * step + 1], cc = p.abc[3 * step + 2];
    // ---------------- X X^T of these columns, sent to the CTAs that add them up
    products([&] {
      multiply<P>(tmem + kAcc, kSmall, smem_u32(xs), (uint32_t)x_plane, smem_u32(xs),
                  (uint32_t)x_plane, p.nc / 16, 0, kSide);
    });
    if (P == 2 && step > 0) cluster_wait();  // all are done with D, where the sums go
    for (int c = 16 * group; c < kSide; c += kStep) {
      float v[16];
      sums((uint32_t)c, kSmall, v);
#pragma unroll
      for (int k = 0; k < 16; k += 4)
        cluster_store(remote(exchange, row / chunk) +
                          (uint32_t)(((rank * 32 + (c + k) / 4) * chunk + row % chunk) * 16),
                      make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]));
    }
    cluster_sync();
    float t = 0.0f;
    for (int c = 0; c < C; ++c) t += sh.sum[c];
    t /= (float)p.m;
    for (int u = tid; u < chunk * 32; u += kThreads) {  // four columns of a row
      const int r = rank * chunk + u % chunk, c = u / chunk * 4;
      const float4 *from = reinterpret_cast<const float4 *>(exchange) + u;
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int src = 0; src < C; ++src) {
        const float4 f = from[src * chunk * 32];
        x[0] += f.x, x[1] += f.y, x[2] += f.z, x[3] += f.w;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] *= kScaleU / (kScaleX * kScaleX);
        if (r == c + k && r < p.m) x[k] -= t * kScaleU;
      }
      uint32_t w[P][2];
      split_planes<P, 4>(x, w);
#pragma unroll
      for (int q = 0; q < P; ++q)
        *reinterpret_cast<uint2 *>(us + q * kPlane + at_plane(r, c)) = make_uint2(w[q][0], w[q][1]);
    }
    // These rows, 128 bytes of each block of 64 columns, go to the others' planes as they
    // lie (a multiple of 8 rows keeps its swizzle).
    fence_async_smem();
    __syncthreads();
    if (tid == 0) mbar_expect_tx(&sh.u_bar, (uint32_t)(P * kPlane - P * kPlane / C));
    if (warp < C && warp != rank && lane < 2 * P) {
      uint8_t *at = us + (lane >> 1) * kPlane + (lane & 1) * (kSide * kLine) + rank * chunk * kLine;
      cluster_copy(remote(at, warp), smem_u32(at), (uint32_t)(chunk * kLine),
                   remote(&sh.u_bar, warp));
    }
    wait(&sh.u_bar, (uint32_t)step & 1);
    cluster_arrive();  // U is here; waited for before B takes its place
    // ---------------- D, from the planes of U
    {
      const float to_d = cc * (kScaleD / kScaleU), diagonal = kScaleD * fmaf(2.0f * cc, t, cb);
      for (int c = 16 * group; c < kSide; c += kStep) {
        float x[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = at_plane(row, c + 8 * h);
          uint4 v[P];
#pragma unroll
          for (int q = 0; q < P; ++q)
            v[q] = *reinterpret_cast<const uint4 *>(us + q * kPlane + at);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 f = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int q = P - 1; q >= 0; --q) {
              const uint32_t w = (&v[q].x)[k];
              const float2 part = __half22float2(*reinterpret_cast<const __half2 *>(&w));
              f.x += part.x, f.y += part.y;
            }
            x[8 * h + 2 * k] = f.x * to_d, x[8 * h + 2 * k + 1] = f.y * to_d;
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (row == c + k) x[k] += diagonal;
        store16<P>(ds, kPlane, row, c, x);
      }
    }
    // ---------------- B = U D, in the place of U
    products([&] {
      multiply<P>(tmem + kAcc, kSmall, smem_u32(us), kPlane, smem_u32(ds), kPlane, kSide / 16, 0,
                  kSide);
    });
    cluster_wait();  // U's rows have reached all others
    if (P == 2 && step + 1 < p.steps) cluster_arrive();  // D may be written over
    for (int c = 16 * group; c < kSide; c += kStep) {
      float v[16];
      sums((uint32_t)c, kSmall, v);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] *= kScaleB / (kScaleU * kScaleD);
      store16<P>(us, kPlane, row, c, v);
    }
    // ---------------- X <- (a + b t + c t t) X + B X
    products([&] {
      multiply<P>(tmem + kAcc, (uint32_t)p.nc, smem_u32(us), kPlane, smem_u32(xs),
                  (uint32_t)x_plane, kSide / 16, 1, p.nc);
    });
    const float q0 = fmaf(fmaf(cc, t, cb), t, ca);
    const bool last = step + 1 == p.steps;
    float sumsq = 0.0f;
    for (int c = 16 * group; c < p.nc; c += kStep) {
      float v[16], x[16];
      tmem_ld16(lanes + (uint32_t)c, x);
      sums((uint32_t)c, (uint32_t)p.nc, v);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        x[k] = fmaf(q0, x[k], v[k] * (1.0f / (kScaleB * kScaleX)));
        sumsq = fmaf(x[k], x[k], sumsq);
      }
      if (last) {
        // (B has been read: its place is free)
        const OrthoOut to{p.m, p.n, p.ldo, p.transposed};
        store_out<T>(to, static_cast<T *>(p.o) + matrix * p.stride_o,
                     reinterpret_cast<float *>(us + warp * 2048), quarter * 32, j0 + c, x);
      } else {
        tmem_st16(lanes + (uint32_t)c, x);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] *= kScaleX;
        store16<P>(xs, x_plane, row, c, x);
      }
    }
    if (last) break;
    tmem_st_wait();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sumsq += __shfl_xor_sync(0xffffffffu, sumsq, o);
    if (lane == 0) sh.warp_sum[warp] = sumsq;
    __syncthreads();
    if (tid < C) {
      float all = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) all += sh.warp_sum[w];
      cluster_store_f32(remote(&sh.sum[rank], tid), all);
    }
  }

  if (!ok) {
    if (tid == 0) atomicExch(&g_small_status, GEMM_ERR_DEVICE_TIMEOUT);
    // MMAs still in flight end within microseconds: 1 ms, then out
    const uint64_t until = globaltimer() + 1000000ull;
    while (globaltimer() < until) __nanosleep(1000);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) pair_tmem_dealloc<1>(tmem, 512);
}

// The clusters of one call: CTAs of each, columns of a CTA.
struct Shape {
  int cluster, nc;
};
// The clusters that take the least time: waves of them, each of 8 and another one for
// every 64 columns of a plane that a CTA has (us, one wave: BF16 40 with 64 columns and 8
// CTAs, 44 with 16, 47 with 128, 56 with 256; FP32 58 with 64, 63 with 16 CTAs, 69 with 128).
Shape shape_of(const OrthoSizes &q, int64_t *waves) {
  Shape best{};
  int64_t least = 0;
  for (int C = 1; C <= kMaxCluster; C *= 2) {
    const int64_t nc = ceil_div(q.n, 64 * C) * 64;
    const int at_once = clusters_at_once(C);
    if (nc * q.planes > 256 || at_once == 0) continue;
    const int64_t w = ceil_div(q.batch, at_once), t = w * (8 + nc * q.planes / 64);
    if (least != 0 && t >= least) continue;
    least = t;
    best = {C, (int)nc};
    *waves = w;
  }
  return best;
}

template <int P, typename T>
cudaError_t allow(int dev) {
  static Once smem_once, cluster_once;
  auto kern = ortho_small_kernel<P, T>;
  cudaError_t e = allow_shared_memory(smem_once, kern, smem_bytes<P>(), dev);
  const bool known = dev >= 0 && dev < 64;
  if (e != cudaSuccess || (known && cluster_once.done[dev].load(std::memory_order_relaxed)))
    return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && known) cluster_once.done[dev].store(true, std::memory_order_relaxed);
  return e;
}

// A launch of clusters of `size` CTAs.
struct Launch {
  cudaLaunchAttribute attr[2] = {};
  cudaLaunchConfig_t config = {};
  Launch(int size, int64_t clusters, int smem, cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    config.gridDim = dim3((unsigned)(clusters * size));
    config.blockDim = dim3(kThreads);
    config.dynamicSmemBytes = (size_t)smem;
    config.stream = s;
    config.attrs = attr;
    config.numAttrs = 2;
  }
};

template <int P, typename T>
int launch(int64_t batch, const SmallParams &p, int cluster, const DeviceProps &dp,
           cudaStream_t s) {
  cudaError_t e = allow<P, T>(dp.device);
  const Launch l(cluster, batch, smem_bytes<P>(), s);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&l.config, ortho_small_kernel<P, T>, p);
  if (e != cudaSuccess) cudaGetLastError();
  return to_status(e);
}

}  // namespace

int clusters_at_once(int size) {
  // GPCs of 16 to 20 SMs, not all of which have 16 left: a GB300's numbers, asked of it once
  static const int usual[5] = {152, 76, 36, 15, 7};
  static std::atomic<int> known[64][5];  // and one
  int i = 0, dev = -1;
  while ((1 << i) < size) ++i;
  if (current_device(&dev) != GEMM_OK || dev >= 64) return usual[i];
  int n = known[dev][i].load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  const Launch l(size, 1, smem_bytes<1>(), nullptr);
  if (allow<1, bf16>(dev) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, ortho_small_kernel<1, bf16>, &l.config) != cudaSuccess) {
    cudaGetLastError();
    return usual[i];
  }
  known[dev][i].store(n + 1, std::memory_order_relaxed);
  return n;
}

// Matrices of up to 128 x 4096 (BF16) or 128 x 2048 (FP32), if their clusters run in one
// wave, or in two from 10 matrices on, by the general kernels / here, us, back to back.  One
// wave: 32 x 64 FP32 71 / 55, 128 x 512 FP32 105 / 58 and BF16 87 / 40, 128 x 2000 116 / 69 and
// 94 / 47, 128 x 4000 BF16 100 / 56, 8 of 64 x 1024 FP32 102 / 65, 32 of 128 x 512 134 / 68 and
// 104 / 46.  Two: 10 of 128 x 2000 FP32 157 / 141, 10 of 128 x 4096 BF16 150 / 111, 20 of 128 x
// 1000 FP32 156 / 132, 50 of 128 x 512 166 / 131, 100 of 128 x 512 BF16 153 / 104, 300 of 64 x 64
// FP32 124 / 113; of fewer, 8 of 64 x 2048 FP32 109 / 137.  Three: 40 of 128 x 1024 FP32 200 /
// 210.
bool ortho_small_fits(const OrthoSizes &q) {
  if (q.m > kSide || q.n > kMaxCluster * 256 / q.planes) return false;
  int64_t waves = 0;
  return shape_of(q, &waves).cluster > 0 && waves <= (q.batch < 10 ? 1 : 2);
}

int launch_ortho_small(const OrthoSizes &q, const OrthoCall &call, const DeviceProps &dp,
                       cudaStream_t s) {
  int64_t waves;
  const Shape shape = shape_of(q, &waves);
  g_small_ran.store(true, std::memory_order_relaxed);
  SmallParams p{};
  p.g = call.g;
  p.ldg = call.ldg;
  p.stride_g = call.stride_g;
  p.o = call.o;
  p.ldo = call.ldo;
  p.stride_o = call.stride_o;
  p.m = (int)q.m;
  p.n = (int)q.n;
  p.nc = shape.nc;
  p.transposed = call.rows > call.cols;
  const int64_t size = (int64_t)dtype_size(call.dtype);
  p.vec = ((reinterpret_cast<uintptr_t>(call.g) | (uintptr_t)(call.ldg * size) |
            (uintptr_t)(call.stride_g * size)) & 15) == 0;
  p.steps = call.steps;
  p.eps = call.eps;
  p.wait_ns = env_u64("GEMM_DEBUG_WAIT_LIMIT_NS", 2000000000ull);
  p.stall = (int)env_u64("GEMM_DEBUG_STALL_PRODUCER", 0);
  for (int i = 0; i < 3 * call.steps; ++i) p.abc[i] = call.abc[i];
  if (call.dtype == GEMM_DT_F32) return launch<2, float>(q.batch, p, shape.cluster, dp, s);
  return launch<1, bf16>(q.batch, p, shape.cluster, dp, s);
}

int ortho_small_read_and_clear_status(cudaStream_t s) {
  int v = 0;
  if (!g_small_ran.load(std::memory_order_relaxed)) return GEMM_OK;
  if (cudaMemcpyFromSymbolAsync(&v, g_small_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(g_small_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) !=
            cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_CUDA;
    }
  }
  return v;
}

}  // namespace gg
