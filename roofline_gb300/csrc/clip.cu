// The global gradient norm over many tensors, and clipping by it
// (include/gb300_gemm.h, grad_norm_clip).
//
// Two kernels: the sum of squares, and the scaling, which adds the blocks'
// sums in a fixed order first.  Both are bound by HBM: every gradient is read
// twice (a set larger than L2 cannot wait on the chip for the norm) and
// written once.  The tensors are cut into chunks of 32 KB, eight 16-byte loads
// in flight a thread, which the blocks take in turn: first to last in the
// first kernel and last to first in the second, so that it begins with what
// the first one left in L2.  600 M gradients (1.32 GB) on GB300: 626 us, 6.3
// TB/s over the three passes; with chunks of 16 KB 688, with a run of
// neighbouring chunks for each block 637.
#include "ff.cuh"
#include "tc_common.cuh"

namespace gg {
namespace {

// The tensors go to the kernels as a launch parameter (32,764 bytes at most):
// no copy to the device, so the call can be captured into a graph.
struct ClipTensor {
  const void *in;
  void *out;
  int64_t n;
  int32_t first, dtype;  // its first chunk among the table's
};
template <int N>
struct ClipTable {
  int count, chunks;
  ClipTensor t[N];
};
constexpr int kClipSmall = 64, kClipTable = 1000;  // tensors of one launch
constexpr int kClipThreads = 256, kClipVectors = 8;
constexpr int kClipChunk = kClipThreads * kClipVectors;  // 16-byte vectors of a chunk
constexpr int kClipBlocksPerSm = 8;

// The elements of a tensor before its first 16-byte boundary.
__host__ __device__ __forceinline__ int64_t clip_head(const void *p, int64_t n, int size) {
  const int64_t head = (16 - (int64_t)(reinterpret_cast<uintptr_t>(p) & 15)) % 16 / size;
  return head < n ? head : n;
}
__host__ __device__ __forceinline__ int64_t clip_vectors(const void *p, int64_t n, int size) {
  return (n - clip_head(p, n, size)) / (16 / size);
}

// The tensor of chunk `c`.
template <int N>
__device__ __forceinline__ int clip_find(const ClipTable<N> &tab, int c) {
  int lo = 0, hi = tab.count - 1;  // the last tensor that begins at or before c
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (tab.t[mid].first <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ void clip_unpack(const uint4 &v, float (&x)[16 / sizeof(T)]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// The block's sum of v, in a fixed order, in every thread.
__device__ double block_sum(double v) {
  __shared__ double part[kClipThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kClipThreads / 32; ++w) v += part[w];
  __syncthreads();
  return v;
}

// Sum of the squares of a thread's values: in FP32 where that neither
// overflows nor underflows, else with the values scaled by a power of two.
template <typename F>
__device__ __forceinline__ double squares(F sum_scaled) {
  const float s = sum_scaled(1.0f);
  if (s >= 0x1p-80f && s <= 0x1p100f) return (double)s;
  if (s < 0x1p-80f) return (double)sum_scaled(0x1p64f) * 0x1p-128;
  return (double)sum_scaled(0x1p-96f) * 0x1p192;  // Inf and NaN stay what they are
}

template <typename T>
__device__ __forceinline__ double clip_chunk_sum(const ClipTensor &t, int64_t v0) {
  constexpr int VE = 16 / sizeof(T);
  const T *in = static_cast<const T *>(t.in);
  const int64_t head = clip_head(in, t.n, sizeof(T)), vectors = (t.n - head) / VE;
  const uint4 *vec = reinterpret_cast<const uint4 *>(in + head);
  uint4 r[kClipVectors];
#pragma unroll
  for (int j = 0; j < kClipVectors; ++j) {
    const int64_t v = v0 + j * kClipThreads + threadIdx.x;
    r[j] = v < vectors ? __ldg(vec + v) : make_uint4(0, 0, 0, 0);
  }
  double sum = squares([&](float scale) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < kClipVectors; ++j) {
      float x[VE];
      clip_unpack<T>(r[j], x);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float y = x[i] * scale;
        s = fmaf(y, y, s);
      }
    }
    return s;
  });
  // the elements before the first vector and behind the last
  if (v0 == 0 && threadIdx.x < head) {
    const double x = to_f32(in[threadIdx.x]);
    sum += x * x;
  }
  const int64_t tail = head + vectors * VE + threadIdx.x;
  if (v0 + kClipChunk >= vectors && tail < t.n) {
    const double x = to_f32(in[tail]);
    sum += x * x;
  }
  return sum;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads)
clip_sum_kernel(const __grid_constant__ ClipTable<N> tab, double *partial) {
  tc::grid_dependency_wait();
  double sum = 0.0;
  int k = clip_find(tab, blockIdx.x);
  for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    while (k + 1 < tab.count && tab.t[k + 1].first <= c) ++k;
    const ClipTensor &t = tab.t[k];
    const int64_t v0 = (int64_t)(c - t.first) * kClipChunk;
    sum += t.dtype == GEMM_DT_F32 ? clip_chunk_sum<float>(t, v0) : clip_chunk_sum<bf16>(t, v0);
  }
  tc::grid_launch_dependents();
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__device__ float clip_norm(const double *partial, int count) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < count; i += kClipThreads) sum += partial[i];
  return (float)sqrt(block_sum(sum));
}

__global__ void __launch_bounds__(kClipThreads)
clip_norm_kernel(const double *partial, int count, float *norm) {
  tc::grid_dependency_wait();
  const float n = clip_norm(partial, count);
  if (threadIdx.x == 0) *norm = n;
}

template <typename T>
__device__ __forceinline__ void clip_chunk_scale(const ClipTensor &t, int64_t v0, float c) {
  constexpr int VE = 16 / sizeof(T);
  const T *in = static_cast<const T *>(t.in);
  T *out = static_cast<T *>(t.out);
  const int64_t head = clip_head(in, t.n, sizeof(T)), vectors = (t.n - head) / VE;
  auto scaled = [&](float x) { return from_f32<T>(x * c); };
  if ((((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0)) {
    const uint4 *vec = reinterpret_cast<const uint4 *>(in + head);
    uint4 *dst = reinterpret_cast<uint4 *>(out + head);
    uint4 r[kClipVectors];
#pragma unroll
    for (int j = 0; j < kClipVectors; ++j) {
      const int64_t v = v0 + j * kClipThreads + threadIdx.x;
      r[j] = v < vectors ? vec[v] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kClipVectors; ++j) {
      const int64_t v = v0 + j * kClipThreads + threadIdx.x;
      float x[VE];
      clip_unpack<T>(r[j], x);
      __align__(16) T y[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) y[i] = scaled(x[i]);
      if (v < vectors) dst[v] = *reinterpret_cast<const uint4 *>(y);
    }
  } else {
    // out is aligned otherwise: element by element
    const int64_t e1 = head + (v0 + kClipChunk < vectors ? v0 + kClipChunk : vectors) * VE;
#pragma unroll 4
    for (int64_t e = head + v0 * VE + threadIdx.x; e < e1; e += kClipThreads)
      out[e] = scaled(to_f32(in[e]));
  }
  if (v0 == 0 && threadIdx.x < head) out[threadIdx.x] = scaled(to_f32(in[threadIdx.x]));
  const int64_t tail = head + vectors * VE + threadIdx.x;
  if (v0 + kClipChunk >= vectors && tail < t.n) out[tail] = scaled(to_f32(in[tail]));
}

template <int N>
__global__ void __launch_bounds__(kClipThreads)
clip_scale_kernel(const __grid_constant__ ClipTable<N> tab, const double *partial, int count,
                  float max_norm, float *norm) {
  tc::grid_dependency_wait();
  const float n = clip_norm(partial, count);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  const float r = max_norm / (n + 1e-6f);
  const float s = r < 1.0f || r != r ? r : 1.0f;
  // the grid is no larger than the number of chunks
  const int last = blockIdx.x + (tab.chunks - 1 - blockIdx.x) / gridDim.x * gridDim.x;
  int k = clip_find(tab, last);
  for (int c = last; c >= 0; c -= gridDim.x) {
    while (tab.t[k].first > c) --k;
    const ClipTensor &t = tab.t[k];
    if (s == 1.0f && t.in == t.out) continue;  // x * 1 is there already
    const int64_t v0 = (int64_t)(c - t.first) * kClipChunk;
    if (t.dtype == GEMM_DT_F32)
      clip_chunk_scale<float>(t, v0, s);
    else
      clip_chunk_scale<bf16>(t, v0, s);
  }
}

// Launched with programmatic dependent launch: each kernel waits for the one
// before it before it touches memory.
template <typename... Params, typename... Args>
cudaError_t clip_launch(void (*kern)(Params...), int grid, cudaStream_t s, const Args &...args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3(kClipThreads);
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kern, Params(args)...);
}

struct ClipCall {
  int64_t count;
  const int *dtypes;
  const void *const *grads;
  void *const *outs;
  const int64_t *sizes;
  int blocks;  // most of one launch
  double *partial;
  float max_norm, *norm;
  cudaStream_t stream;
};

// All launches of a call, up to N tensors in each.
template <int N>
cudaError_t clip_run(const ClipCall &q) {
  static thread_local ClipTable<N> tab;
  // The tensors from `at` on; returns the first that is left.
  auto fill = [&](int64_t at) {
    int64_t chunks = 0;
    tab.count = 0;
    while (at < q.count && tab.count < N) {
      const int size = (int)dtype_size(q.dtypes[at]);
      const int64_t c =
          ceil_div(clip_vectors(q.grads[at], q.sizes[at], size), kClipChunk);
      if (q.sizes[at] > 0) {
        tab.t[tab.count++] = {q.grads[at], q.outs ? q.outs[at] : nullptr, q.sizes[at],
                              (int32_t)chunks, q.dtypes[at]};
        chunks += c > 0 ? c : 1;
      }
      ++at;
    }
    tab.chunks = (int)chunks;
    return at;
  };
  auto grid = [&] { return tab.chunks < q.blocks ? tab.chunks : q.blocks; };
  int partials = 0;
  cudaError_t e = cudaSuccess;
  for (int64_t at = 0; at < q.count && e == cudaSuccess;) {
    at = fill(at);
    if (tab.count == 0) continue;
    e = clip_launch(clip_sum_kernel<N>, grid(), q.stream, tab, q.partial + partials);
    partials += grid();
  }
  if (e != cudaSuccess) return e;
  if (!q.outs || partials == 0)
    return clip_launch(clip_norm_kernel, 1, q.stream, q.partial, partials, q.norm);
  float *norm = q.norm;
  for (int64_t at = 0; at < q.count && e == cudaSuccess;) {
    at = fill(at);
    if (tab.count == 0) continue;
    e = clip_launch(clip_scale_kernel<N>, grid(), q.stream, tab, q.partial, partials, q.max_norm,
                    norm);
    norm = nullptr;  // the first launch writes it
  }
  return e;
}

// Launches of one pass, at most.
int64_t clip_launches(int64_t count) { return count > 0 ? ceil_div(count, kClipTable) : 0; }

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

uint64_t grad_norm_clip_workspace(int64_t count) {
  return (uint64_t)clip_launches(count) * current_props().sm_count * kClipBlocksPerSm *
         sizeof(double);
}

int grad_norm_clip(int64_t count, const int *dtypes, const void *const *grads, void *const *outs,
                   const int64_t *sizes, float max_norm, float *norm, void *workspace,
                   size_t ws_bytes, cudaStream_t stream) {
  if (count < 0 || count > ((int64_t)1 << 24) || !norm ||
      (reinterpret_cast<uintptr_t>(norm) & 3) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return GEMM_ERR_INVALID_ARG;
  if (count > 0 && (!dtypes || !grads || !sizes)) return GEMM_ERR_INVALID_ARG;
  if (outs && !(max_norm >= 0.0f)) return GEMM_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (!dtype_known(dtypes[i]) || sizes[i] < 0 || sizes[i] > ((int64_t)1 << 40))
      return GEMM_ERR_INVALID_ARG;
    const uintptr_t mask = dtype_size(dtypes[i]) - 1;
    if (sizes[i] > 0 && (!grads[i] || (reinterpret_cast<uintptr_t>(grads[i]) & mask)))
      return GEMM_ERR_INVALID_ARG;
    if (outs && sizes[i] > 0 && (!outs[i] || (reinterpret_cast<uintptr_t>(outs[i]) & mask)))
      return GEMM_ERR_INVALID_ARG;
    total += sizes[i];
  }
  // 2^40 elements are more than any device's memory holds, and the chunks of
  // fewer count in 32 bits
  if (total > ((int64_t)1 << 40)) return GEMM_ERR_UNSUPPORTED;
  int dev = -1;
  int st = current_device(&dev);
  if (st != GEMM_OK) return st;
  const uint64_t need = grad_norm_clip_workspace(count);
  void *ws = workspace;
  if (workspace && ws_bytes < need) return GEMM_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace && need) {
    st = library_workspace(dev, (size_t)need, &ws);
    if (st != GEMM_OK) return st;
  }
  const ClipCall q{count,    dtypes, grads, outs, sizes, props_of(dev).sm_count * kClipBlocksPerSm,
                   static_cast<double *>(ws), max_norm, norm, stream};
  return to_status(count <= kClipSmall ? clip_run<kClipSmall>(q) : clip_run<kClipTable>(q));
}

}  // extern "C"
