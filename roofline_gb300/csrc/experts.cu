// A mixture layer's tokens sorted by expert, gathered into rows and brought
// back with weights, and the gradients (include/gb300_gemm.h, expert_sort to
// expert_combine_backward).
//
// expert_sort is a counting sort in one launch: a block, or a cluster of them,
// whose warps own consecutive choices.  A warp counts its choices of each
// expert in its own row of shared memory (one lane
// of those with the same expert adds for all, so no two write to one counter and
// the order is that of the input), the counts become first rows by a scan over warps,
// blocks and experts, and the warps pass over their choices again.
//
// The other three move rows and are bound by HBM.  All go token by token: a
// token's row is read once, whatever the number of its choices, and its
// choices' rows, the larger part, are written or read in whole lines.  GB300, 8192
// tokens of 4096 BF16 values: gathered to 8 of 64 experts 98 us (604 MB, 6.2 TB/s), the
// sort before it 9 us (one choice a lane, 16 SMs; 524,288 choices of 256 experts 50 us);
// 8 rows of each added up 107 us (605 MB, 5.7 TB/s); gradients of 2 rows of each 58 us
// (336 MB, 5.8 TB/s).  A copy on the same device moves 6.8 TB/s.  Rows that begin
// anywhere are moved in the widest pieces that all of them allow (1025 x 777 FP32, 4
// bytes: 3 rows of each added up 6.5 us, gradients 7.3 us).
#include "ff.cuh"
#include "tc_common.cuh"

namespace gg {
namespace {

// ------------------------------------------------------------------ the sort

constexpr int kSortWarps = 32;
constexpr int kSortCluster = 16;

struct SortParams {
  const void *ids;
  int64_t ld, n;     // choices
  int64_t per_warp;  // choices of one warp, a multiple of 32
  int k, experts, bits, warps;  // bits of an expert
  int32_t *place, *offsets, *order;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ int cluster_load(const int *p, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Calls f(choice, expert, lanes with the same expert) for this warp's choices,
// 32 at a time and in order; expert -1 where it is none of the experts.  Equal
// experts are found bit by bit, a ballot for each (by match.any 65,536 choices of 64
// experts took 12.9 us instead of 9.2, 524,288 of 256 72 instead of 50).
template <typename Id, typename F>
__device__ __forceinline__ void for_choices(const SortParams &p, int64_t first, int64_t last,
                                            F f) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31;
  for (int64_t i0 = first; i0 < last; i0 += 32 * kAhead) {
    Id id[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int64_t i = i0 + 32 * a + lane;
      id[a] = -1;
      if (i < last) {
        int64_t at = i;
        if (p.ld != p.k) {
          const uint32_t t = (uint32_t)i / (uint32_t)p.k;
          at = t * p.ld + ((uint32_t)i - t * (uint32_t)p.k);
        }
        id[a] = __ldg(static_cast<const Id *>(p.ids) + at);
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int64_t i = i0 + 32 * a + lane;
      if (i - lane >= last) break;
      const int e = id[a] >= 0 && id[a] < p.experts ? (int)id[a] : -1;
      uint32_t same = __ballot_sync(0xffffffffu, e >= 0);
      if (e < 0) same = ~same;
      for (int b = 0; b < p.bits; ++b) {
        const bool one = (e >> b) & 1;
        const uint32_t ones = __ballot_sync(0xffffffffu, one);
        same &= one ? ones : ~ones;
      }
      f(i, e, same);
    }
  }
}

template <typename Id>
__global__ void __launch_bounds__(32 * kSortWarps)
expert_sort_kernel(const SortParams p) {
  extern __shared__ int sort_smem[];
  __shared__ int warp_sum[kSortWarps], routed;
  const int E = p.experts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int *count = sort_smem;              // [warps][E]: then the warp's next row, from first[e] on
  int *total = count + p.warps * E;    // [E]: this block's choices
  int *first = total + E;              // [E]: the block's first row
  const uint32_t rank = cluster_rank(), blocks = cluster_size();
  const uint32_t below = (1u << lane) - 1;

  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  for (int i = tid; i < p.warps * E; i += blockDim.x) count[i] = 0;
  __syncthreads();
  const int64_t from = min(p.n, ((int64_t)rank * p.warps + warp) * p.per_warp);
  const int64_t to = warp < p.warps ? min(p.n, from + p.per_warp) : from;
  int *mine = count + warp * E;
  for_choices<Id>(p, from, to, [&](int64_t, int e, uint32_t same) {
    if (e >= 0 && (same & below) == 0) mine[e] += __popc(same);
    __syncwarp();
  });
  __syncthreads();
  if (tid < E) {
    int run = 0;
    for (int w0 = 0; w0 < p.warps; w0 += 8) {
      int c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = w0 + w < p.warps ? count[(w0 + w) * E + tid] : 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w0 + w < p.warps) count[(w0 + w) * E + tid] = run;
        run += c[w];
      }
    }
    total[tid] = run;
  }
  // the experts' totals over all blocks, and their sum over the blocks before this one
  int all = 0, before = 0;
  if (blocks > 1) {
    cluster_arrive();
    cluster_wait();
    if (tid < E) {
#pragma unroll 8
      for (uint32_t r = 0; r < blocks; ++r) {
        const int c = cluster_load(&total[tid], r);
        if (r < rank) before += c;
        all += c;
      }
    }
    cluster_arrive();  // waited for at the end: this block's totals have been read
  } else if (tid < E) {
    all = total[tid];
  }
  int scan = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) scan += w < warp ? warp_sum[w] : 0;
  if (tid < E) {
    first[tid] = scan - all + before;
    if (rank == 0) p.offsets[tid] = scan - all;
    if (tid == E - 1) {
      routed = scan;
      if (rank == 0) p.offsets[E] = scan;
    }
  }
  __syncthreads();
  for_choices<Id>(p, from, to, [&](int64_t i, int e, uint32_t same) {
    int row = -1;
    if (e >= 0) row = first[e] + mine[e] + __popc(same & below);
    __syncwarp();
    if (e >= 0 && (same & below) == 0) mine[e] += __popc(same);
    __syncwarp();
    if (i < to) {
      p.place[i] = row;
      if (row >= 0 && p.order) p.order[row] = (int32_t)i;
    }
  });
  if (p.order)
    for (int64_t r = routed + (int64_t)rank * blockDim.x + tid; r < p.n;
         r += (int64_t)blocks * blockDim.x)
      p.order[r] = -1;
  if (blocks > 1) cluster_wait();
}

// ------------------------------------------------------------------ the rows

constexpr int kRowThreads = 128;

// A vector of VB bytes of T, as floats.
template <int VB>
struct VecOf;
template <>
struct VecOf<16> { using type = uint4; };
template <>
struct VecOf<8> { using type = uint2; };
template <>
struct VecOf<4> { using type = uint32_t; };
template <>
struct VecOf<2> { using type = uint16_t; };

template <typename T, int VB>
__device__ __forceinline__ void vec_unpack(const typename VecOf<VB>::type &v,
                                           float (&x)[VB / sizeof(T)]) {
  __align__(16) T t[VB / sizeof(T)];
  *reinterpret_cast<typename VecOf<VB>::type *>(t) = v;
#pragma unroll
  for (int i = 0; i < (int)(VB / sizeof(T)); ++i) x[i] = to_f32(t[i]);
}
template <typename T, int VB>
__device__ __forceinline__ typename VecOf<VB>::type vec_pack(const float (&x)[VB / sizeof(T)]) {
  __align__(16) T t[VB / sizeof(T)];
#pragma unroll
  for (int i = 0; i < (int)(VB / sizeof(T)); ++i) t[i] = from_f32<T>(x[i]);
  return *reinterpret_cast<typename VecOf<VB>::type *>(t);
}

// What the three kernels share.  A block's threads are `lanes` columns wide
// (a power of two) and take kRowThreads / lanes tokens at once.
struct RowParams {
  int64_t T, rows;            // tokens; rows of the sorted buffers
  int k, vecs, lanes, parts;  // vectors of a row; gather, combine: parts that blocks share
  const uint8_t *x;           // tokens' rows: X (gather), dO (backward)
  uint8_t *o;                 // tokens' rows: O (combine)
  const uint8_t *y;           // sorted rows that are read
  uint8_t *dy;                // sorted rows that are written
  int64_t ldx, ldo, ldy, lddy;  // in bytes
  const int32_t *place, *routed;
  const void *w;              // weights, or null: 1
  void *dw;
  int64_t ldw, lddw;
  int w_bf16;
};

// The sorted row of choice j of token t, -1 for none: places from elsewhere
// than the sort stay inside the buffers.
__device__ __forceinline__ int row_of(const RowParams &p, int64_t t, int j) {
  const int r = __ldg(p.place + t * p.k + j);
  return (uint32_t)r < (uint64_t)p.rows ? r : -1;
}
__device__ __forceinline__ float weight_of(const RowParams &p, int64_t t, int j) {
  if (!p.w) return 1.0f;
  return p.w_bf16 ? to_f32(static_cast<const bf16 *>(p.w)[t * p.ldw + j])
                  : static_cast<const float *>(p.w)[t * p.ldw + j];
}

// Rows behind the routed ones: zero.
template <int VB>
__device__ __forceinline__ void zero_rest(const RowParams &p) {
  using V = typename VecOf<VB>::type;
  const int64_t routed = *p.routed;
  for (int64_t r = (routed > 0 ? routed : 0) + blockIdx.x; r < p.rows; r += gridDim.x)
    for (int v = threadIdx.x; v < p.vecs; v += kRowThreads)
      reinterpret_cast<V *>(p.dy + r * p.lddy)[v] = V{};
}

// Four vectors of a token's row, eight of its places at a time.
template <int VB>
__global__ void __launch_bounds__(kRowThreads)
gather_kernel(const RowParams p) {
  using V = typename VecOf<VB>::type;
  constexpr int kVecs = 4, kRows = 8;
  const int tx = threadIdx.x & (p.lanes - 1), ty = threadIdx.x / p.lanes;
  const int64_t tokens = kRowThreads / p.lanes, groups = (p.T + tokens - 1) / tokens;
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  for (int64_t item = blockIdx.x; item < groups * p.parts; item += gridDim.x) {
    const int64_t t = item / p.parts * tokens + ty;
    if (t >= p.T) continue;
    const V *x = reinterpret_cast<const V *>(p.x + t * p.ldx);
    for (int v0 = (int)(item % p.parts) * p.lanes + tx; v0 < p.vecs;
         v0 += kVecs * p.parts * p.lanes) {
      V r[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int v = v0 + i * p.parts * p.lanes;
        if (v < p.vecs) r[i] = x[v];
      }
      for (int j0 = 0; j0 < p.k; j0 += kRows) {
        int row[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) row[j] = j0 + j < p.k ? row_of(p, t, j0 + j) : -1;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          if (row[j] < 0) continue;
          V *y = reinterpret_cast<V *>(p.dy + row[j] * p.lddy);
#pragma unroll
          for (int i = 0; i < kVecs; ++i) {
            const int v = v0 + i * p.parts * p.lanes;
            if (v < p.vecs) y[v] = r[i];
          }
        }
      }
    }
  }
  zero_rest<VB>(p);
}

// The loads of a thread at a time: VV vectors of KR choices' rows, 8 in all.  (One
// vector whatever the number of choices: 2 rows of 8192 x 4096 added up 67 us instead of
// 37, their gradients 105 instead of 57.)
constexpr int kLoads = 8;

// O = sum over the choices of w Y, in FP32 in the choices' order.
template <typename T, int VB, int KR>
__global__ void __launch_bounds__(kRowThreads)
combine_kernel(const RowParams p) {
  using V = typename VecOf<VB>::type;
  constexpr int VE = VB / sizeof(T), VV = kLoads / KR;
  const int tx = threadIdx.x & (p.lanes - 1), ty = threadIdx.x / p.lanes;
  const int step = p.parts * p.lanes;
  const int64_t tokens = kRowThreads / p.lanes, groups = (p.T + tokens - 1) / tokens;
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  for (int64_t item = blockIdx.x; item < groups * p.parts; item += gridDim.x) {
    const int64_t t = item / p.parts * tokens + ty;
    if (t >= p.T) continue;
    for (int v0 = (int)(item % p.parts) * p.lanes + tx; v0 < p.vecs; v0 += VV * step) {
      float sum[VV][VE];
#pragma unroll
      for (int u = 0; u < VV; ++u)
#pragma unroll
        for (int i = 0; i < VE; ++i) sum[u][i] = 0.0f;
      for (int j0 = 0; j0 < p.k; j0 += KR) {
        int row[KR];
        float w[KR];
        V y[KR][VV];
#pragma unroll
        for (int j = 0; j < KR; ++j) {
          row[j] = j0 + j < p.k ? row_of(p, t, j0 + j) : -1;
          w[j] = row[j] >= 0 ? weight_of(p, t, j0 + j) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < KR; ++j)
#pragma unroll
          for (int u = 0; u < VV; ++u)
            if (row[j] >= 0 && v0 + u * step < p.vecs)
              y[j][u] = __ldg(reinterpret_cast<const V *>(p.y + row[j] * p.ldy) + v0 + u * step);
#pragma unroll
        for (int j = 0; j < KR; ++j) {
          if (row[j] < 0) continue;
#pragma unroll
          for (int u = 0; u < VV; ++u) {
            float x[VE];
            vec_unpack<T, VB>(y[j][u], x);
#pragma unroll
            for (int i = 0; i < VE; ++i) sum[u][i] = fmaf(w[j], x[i], sum[u][i]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < VV; ++u)
        if (v0 + u * step < p.vecs)
          reinterpret_cast<V *>(p.o + t * p.ldo)[v0 + u * step] = vec_pack<T, VB>(sum[u]);
    }
  }
}

// dY = w dO for every choice, dw = <dO, Y>.  A token's dO and the rows of up to
// KR choices are read side by side; the sums of a token's lanes meet in a
// fixed order, in the warp and then in shared memory.
template <typename T, int VB, int KR>
__global__ void __launch_bounds__(kRowThreads)
combine_backward_kernel(const RowParams p) {
  using V = typename VecOf<VB>::type;
  constexpr int VE = VB / sizeof(T), VV = kLoads / KR, kWarps = kRowThreads / 32;
  __shared__ float part[kWarps][KR];
  const int tx = threadIdx.x & (p.lanes - 1), ty = threadIdx.x / p.lanes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int token_warps = p.lanes / 32;  // 0: less than one
  const int64_t tokens = kRowThreads / p.lanes, groups = (p.T + tokens - 1) / tokens;
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  for (int64_t item = blockIdx.x; item < groups; item += gridDim.x) {
    const int64_t t = item * tokens + ty;
    const bool on = t < p.T;
    const V *x = reinterpret_cast<const V *>(p.x + t * p.ldx);
    for (int j0 = 0; j0 < p.k; j0 += KR) {
      int row[KR];
      float w[KR], dot[KR];
#pragma unroll
      for (int j = 0; j < KR; ++j) {
        row[j] = on && j0 + j < p.k ? row_of(p, t, j0 + j) : -1;
        w[j] = row[j] >= 0 ? weight_of(p, t, j0 + j) : 0.0f;
        dot[j] = 0.0f;
      }
      for (int v0 = tx; on && v0 < p.vecs; v0 += VV * p.lanes) {
        V xv[VV], y[KR][VV];
#pragma unroll
        for (int u = 0; u < VV; ++u) {
          const int v = v0 + u * p.lanes;
          if (v >= p.vecs) continue;
          xv[u] = x[v];
          if (!p.dw) continue;
#pragma unroll
          for (int j = 0; j < KR; ++j)
            if (row[j] >= 0) y[j][u] = __ldg(reinterpret_cast<const V *>(p.y + row[j] * p.ldy) + v);
        }
#pragma unroll
        for (int u = 0; u < VV; ++u) {
          const int v = v0 + u * p.lanes;
          if (v >= p.vecs) continue;
          float d[VE];
          vec_unpack<T, VB>(xv[u], d);
#pragma unroll
          for (int j = 0; j < KR; ++j) {
            if (row[j] < 0) continue;
            float r[VE];
            if (p.dw) {
              vec_unpack<T, VB>(y[j][u], r);
#pragma unroll
              for (int i = 0; i < VE; ++i) dot[j] = fmaf(d[i], r[i], dot[j]);
            }
            if (p.dy) {
#pragma unroll
              for (int i = 0; i < VE; ++i) r[i] = w[j] * d[i];
              reinterpret_cast<V *>(p.dy + row[j] * p.lddy)[v] = vec_pack<T, VB>(r);
            }
          }
        }
      }
      if (!p.dw) continue;
      auto store = [&](float sum) {
        if (p.w_bf16)
          static_cast<bf16 *>(p.dw)[t * p.lddw + j0 + tx] = from_f32<bf16>(sum);
        else
          static_cast<float *>(p.dw)[t * p.lddw + j0 + tx] = sum;
      };
      const bool mine = on && tx < KR && j0 + tx < p.k;  // lanes are no fewer than KR
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < KR; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (o < p.lanes) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        if (tx == j) sum = dot[j];
      }
      if (token_warps <= 1) {
        if (mine) store(sum);
        continue;
      }
#pragma unroll
      for (int j = 0; j < KR; ++j)
        if (lane == j) part[warp][j] = dot[j];
      __syncthreads();
      if (mine) {
        sum = 0.0f;
        for (int q = 0; q < token_warps; ++q) sum += part[ty * token_warps + q][tx];
        store(sum);
      }
      __syncthreads();
    }
  }
  if (p.dy) zero_rest<VB>(p);
}

// ------------------------------------------------------------------ host side

template <typename... Params, typename... Args>
cudaError_t launch(void (*kern)(Params...), int64_t grid, int threads, int smem, int cluster,
                   cudaStream_t s, const Args &...args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = (size_t)smem;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&lc, kern, Params(args)...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

// Lets the kernel have its shared memory and clusters of kSortCluster, once for each
// device.
template <typename Id>
cudaError_t allow_sort(int dev) {
  static Once smem_once, cluster_once;
  auto kern = expert_sort_kernel<Id>;
  const int most = (kSortWarps + 2) * GEMM_MAX_EXPERTS * (int)sizeof(int);
  cudaError_t e = allow_shared_memory(smem_once, kern, most, dev);
  const bool known = dev >= 0 && dev < 64;
  if (e != cudaSuccess || (known && cluster_once.done[dev].load(std::memory_order_relaxed)))
    return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && known) cluster_once.done[dev].store(true, std::memory_order_relaxed);
  return e;
}

template <typename Id>
cudaError_t launch_sort(SortParams p, int dev, cudaStream_t s) {
  const cudaError_t e = allow_sort<Id>(dev);
  if (e != cudaSuccess) return e;
  int blocks = 1;
  while (blocks < kSortCluster && p.n > (int64_t)blocks * 4096) blocks *= 2;
  if (blocks == kSortCluster && clusters_at_once(kSortCluster) == 0) blocks /= 2;
  const int64_t warps = ceil_div(ceil_div(p.n, blocks), 32);
  p.warps = (int)(warps < 1 ? 1 : warps > kSortWarps ? kSortWarps : warps);
  p.per_warp = ceil_div(ceil_div(p.n, (int64_t)blocks * p.warps), 32) * 32;
  int threads = 32 * p.warps;
  if (threads < p.experts) threads = (int)ceil_div(p.experts, 32) * 32;
  const int smem = (p.warps + 2) * p.experts * (int)sizeof(int);
  return launch(expert_sort_kernel<Id>, blocks, threads, smem, blocks, s, p);
}

constexpr int64_t kMaxChoices = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxWidth = (int64_t)1 << 28;
constexpr int64_t kMaxLd = (int64_t)1 << 36;

// Sizes of a call on tokens and their choices; `rows` of the sorted buffer.
int check_sizes(int64_t T, int64_t k, int64_t D, int64_t rows) {
  if (T < 0 || k < 0 || D < 0 || rows < 0) return GEMM_ERR_INVALID_ARG;
  if (T > kMaxChoices || k > kMaxChoices || T * k > kMaxChoices || D > kMaxWidth ||
      rows > kMaxChoices)
    return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

bool aligned(const void *p, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}
bool rows_ok(const void *p, int64_t ld, int64_t rows, int64_t cols, int64_t size) {
  if (ld < (cols > 1 ? cols : 1) || ld > kMaxLd) return false;
  return rows == 0 || cols == 0 || (p != nullptr && aligned(p, size));
}

// The widest vector that all rows (base, stride in bytes) and the width allow.
struct Strided {
  const void *p;
  int64_t ld;
};
int vector_bytes(int64_t width, std::initializer_list<Strided> all) {
  uint64_t bits = (uint64_t)width | 16;
  for (const Strided &m : all)
    if (m.p) bits |= reinterpret_cast<uintptr_t>(m.p) | (uint64_t)m.ld;
  return (int)(bits & (~bits + 1));
}

// Threads along a row: enough for its vectors.  Rows of few tokens are cut into
// parts, until there are so many blocks.
void shape_rows(RowParams &p, int64_t blocks) {
  p.lanes = 8;
  while (p.lanes < kRowThreads && p.lanes < p.vecs) p.lanes *= 2;
  p.parts = 1;
  const int64_t groups = ceil_div(p.T, kRowThreads / p.lanes);
  while (p.parts * p.lanes < p.vecs && groups * p.parts < blocks) p.parts *= 2;
}
// Blocks for the tokens, or as many as there are rows that no choice can have and that
// zero_rest clears, if those are more (512 MB behind one token's 8 rows, us: gather 2034
// by the token's own four blocks, 80 with this, gradients 8122 by one and 81).
int64_t grid_of(const RowParams &p, int sms) {
  int64_t blocks = ceil_div(p.T, kRowThreads / p.lanes) * p.parts;
  const int64_t behind = p.dy ? p.rows - p.T * p.k : 0, most = (int64_t)sms * 16;
  if (blocks < behind) blocks = behind;
  return blocks < most ? (blocks > 0 ? blocks : 1) : most;
}

// The kernel of a type, vector and number of choices: make(type, bytes of a vector,
// choices at once).
template <typename T, int VB, typename F>
auto for_choices_of(int64_t k, F make) {
  using B = std::integral_constant<int, VB>;
  return k <= 2   ? make(T(), B(), std::integral_constant<int, 2>())
         : k <= 4 ? make(T(), B(), std::integral_constant<int, 4>())
                  : make(T(), B(), std::integral_constant<int, 8>());
}
template <typename F>
auto for_rows(int dtype, int vb, int64_t k, F make) {
  if (dtype == GEMM_DT_F32)
    return vb == 16  ? for_choices_of<float, 16>(k, make)
           : vb == 8 ? for_choices_of<float, 8>(k, make)
                     : for_choices_of<float, 4>(k, make);
  return vb == 16  ? for_choices_of<bf16, 16>(k, make)
         : vb == 8 ? for_choices_of<bf16, 8>(k, make)
         : vb == 4 ? for_choices_of<bf16, 4>(k, make)
                   : for_choices_of<bf16, 2>(k, make);
}

int device_of(int *dev, int *sms) {
  const int st = current_device(dev);
  if (st == GEMM_OK) *sms = props_of(*dev).sm_count;
  return st;
}

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

int expert_sort(int id_bytes, int64_t T, int64_t k, int64_t experts, const void *ids, int64_t ldi,
                int32_t *place, int32_t *offsets, int32_t *order, cudaStream_t stream) {
  if (id_bytes != 4 && id_bytes != 8) return GEMM_ERR_INVALID_ARG;
  int st = check_sizes(T, k, 0, 0);
  if (st != GEMM_OK) return st;
  if (experts < 1 || !offsets || !aligned(offsets, 4)) return GEMM_ERR_INVALID_ARG;
  if (experts > GEMM_MAX_EXPERTS) return GEMM_ERR_UNSUPPORTED;
  if (!rows_ok(ids, ldi, T, k, id_bytes) || !rows_ok(place, k > 1 ? k : 1, T, k, 4) ||
      (order && !aligned(order, 4)))
    return GEMM_ERR_INVALID_ARG;
  int dev = -1, sms = 0;
  st = device_of(&dev, &sms);
  if (st != GEMM_OK) return st;
  SortParams p{};
  p.ids = ids;
  p.ld = ldi;
  p.n = T * k;
  p.k = k > 0 ? (int)k : 1;
  p.experts = (int)experts;
  while ((1 << p.bits) < experts) ++p.bits;
  p.place = place;
  p.offsets = offsets;
  p.order = order;
  return to_status(id_bytes == 8 ? launch_sort<int64_t>(p, dev, stream)
                                 : launch_sort<int32_t>(p, dev, stream));
}

int expert_gather(int dtype, int64_t T, int64_t k, int64_t D, const void *X, int64_t ldx,
                  const int32_t *place, const int32_t *routed, int64_t rows, void *Y, int64_t ldy,
                  cudaStream_t stream) {
  if (!dtype_known(dtype)) return GEMM_ERR_INVALID_ARG;
  int st = check_sizes(T, k, D, rows);
  if (st != GEMM_OK) return st;
  const int64_t size = (int64_t)dtype_size(dtype);
  if (!rows_ok(X, ldx, k ? T : 0, D, size) || !rows_ok(Y, ldy, rows, D, size) ||
      !rows_ok(place, k > 1 ? k : 1, T, k, 4) || !routed || !aligned(routed, 4))
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || D == 0) return GEMM_OK;
  int dev = -1, sms = 0;
  st = device_of(&dev, &sms);
  if (st != GEMM_OK) return st;
  RowParams p{};
  p.T = k ? T : 0;
  p.rows = rows;
  p.k = (int)k;
  p.x = static_cast<const uint8_t *>(X);
  p.dy = static_cast<uint8_t *>(Y);
  p.ldx = ldx * size;
  p.lddy = ldy * size;
  p.place = place;
  p.routed = routed;
  const int vb = vector_bytes(D * size, {{X, p.ldx}, {Y, p.lddy}});
  p.vecs = (int)(D * size / vb);
  shape_rows(p, 4 * sms);
  const int64_t grid = grid_of(p, sms);
  auto kern = vb == 16 ? gather_kernel<16> : vb == 8 ? gather_kernel<8>
              : vb == 4 ? gather_kernel<4> : gather_kernel<2>;
  return to_status(launch(kern, grid, kRowThreads, 0, 1, stream, p));
}

int expert_combine(int dtype, int w_dtype, int64_t T, int64_t k, int64_t D, const void *Y,
                   int64_t ldy, int64_t rows, const int32_t *place, const void *W, int64_t ldw,
                   void *O, int64_t ldo, cudaStream_t stream) {
  if (!dtype_known(dtype) || !dtype_known(w_dtype)) return GEMM_ERR_INVALID_ARG;
  int st = check_sizes(T, k, D, rows);
  if (st != GEMM_OK) return st;
  const int64_t size = (int64_t)dtype_size(dtype);
  if (!rows_ok(Y, ldy, rows, D, size) || !rows_ok(O, ldo, T, D, size) ||
      !rows_ok(place, k > 1 ? k : 1, T, k, 4) ||
      (W && !rows_ok(W, ldw, T, k, (int64_t)dtype_size(w_dtype))))
    return GEMM_ERR_INVALID_ARG;
  if (T == 0 || D == 0) return GEMM_OK;
  int dev = -1, sms = 0;
  st = device_of(&dev, &sms);
  if (st != GEMM_OK) return st;
  RowParams p{};
  p.T = T;
  p.rows = rows;
  p.k = (int)k;
  p.o = static_cast<uint8_t *>(O);
  p.y = static_cast<const uint8_t *>(Y);
  p.ldo = ldo * size;
  p.ldy = ldy * size;
  p.place = place;
  p.w = W;
  p.ldw = ldw;
  p.w_bf16 = w_dtype == GEMM_DT_BF16;
  const int vb = vector_bytes(D * size, {{O, p.ldo}, {rows ? Y : nullptr, p.ldy}});
  p.vecs = (int)(D * size / vb);
  shape_rows(p, 16 * sms);
  const int64_t grid = grid_of(p, sms);
  auto kern = for_rows(dtype, vb, k, [](auto type, auto bytes, auto rows_at_once) {
    return combine_kernel<decltype(type), decltype(bytes)::value, decltype(rows_at_once)::value>;
  });
  return to_status(launch(kern, grid, kRowThreads, 0, 1, stream, p));
}

int expert_combine_backward(int dtype, int w_dtype, int64_t T, int64_t k, int64_t D,
                            const void *dO, int64_t lddo, const void *Y, int64_t ldy, int64_t rows,
                            const int32_t *place, const int32_t *routed, const void *W, int64_t ldw,
                            void *dY, int64_t lddy, void *dW, int64_t lddw, cudaStream_t stream) {
  if (!dtype_known(dtype) || !dtype_known(w_dtype)) return GEMM_ERR_INVALID_ARG;
  int st = check_sizes(T, k, D, rows);
  if (st != GEMM_OK) return st;
  const int64_t size = (int64_t)dtype_size(dtype), wsize = (int64_t)dtype_size(w_dtype);
  if (!dY && !dW && T > 0 && k > 0 && D > 0) return GEMM_ERR_INVALID_ARG;
  if (!rows_ok(dO, lddo, k ? T : 0, D, size) || !rows_ok(place, k > 1 ? k : 1, T, k, 4) ||
      (W && !rows_ok(W, ldw, T, k, wsize)))
    return GEMM_ERR_INVALID_ARG;
  if (dY && (!rows_ok(dY, lddy, rows, D, size) || !routed || !aligned(routed, 4)))
    return GEMM_ERR_INVALID_ARG;
  if (dW && (!rows_ok(dW, lddw, T, k, wsize) || !rows_ok(Y, ldy, rows, D, size)))
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || D == 0) dY = nullptr;
  if (T == 0 || k == 0) dW = nullptr;
  if (!dY && !dW) return GEMM_OK;
  int dev = -1, sms = 0;
  st = device_of(&dev, &sms);
  if (st != GEMM_OK) return st;
  RowParams p{};
  p.T = k ? T : 0;
  p.rows = rows;
  p.k = (int)k;
  p.x = static_cast<const uint8_t *>(dO);
  p.y = static_cast<const uint8_t *>(Y);
  p.dy = static_cast<uint8_t *>(dY);
  p.ldx = lddo * size;
  p.ldy = ldy * size;
  p.lddy = lddy * size;
  p.place = place;
  p.routed = routed;
  p.w = W;
  p.ldw = ldw;
  p.w_bf16 = w_dtype == GEMM_DT_BF16;
  p.dw = dW;
  p.lddw = lddw;
  const int vb = vector_bytes(D * size, {{D ? dO : nullptr, p.ldx},
                                         {dW && rows ? Y : nullptr, p.ldy}, {dY, p.lddy}});
  p.vecs = (int)(D * size / vb);
  shape_rows(p, 1);
  const int64_t grid = grid_of(p, sms);
  auto kern = for_rows(dtype, vb, k, [](auto type, auto bytes, auto rows_at_once) {
    return combine_backward_kernel<decltype(type), decltype(bytes)::value,
                                   decltype(rows_at_once)::value>;
  });
  return to_status(launch(kern, grid, kRowThreads, 0, 1, stream, p));
}

}  // extern "C"
