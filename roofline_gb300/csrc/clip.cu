// The global gradient norm over many tensors, and clipping by it
// (include/gb300_gemm.h, grad_norm_clip).
#include "ff.cuh"

namespace gg {
namespace {

// The tensors go to the kernels as a launch parameter (32,764 bytes at most):
// no copy to the device, so the call can be captured into a graph.
struct ClipTensor {
  const void *in;
  void *out;
  int64_t n;
  int64_t dtype;
};
constexpr int kClipTable = 1000;  // tensors of one launch
struct ClipTable {
  int count;
  ClipTensor t[kClipTable];
};
constexpr int kClipBlocks = 608, kClipThreads = 256;

__device__ __forceinline__ float clip_load(const ClipTensor &t, int64_t i) {
  return t.dtype == GEMM_DT_F32 ? static_cast<const float *>(t.in)[i]
                                : to_f32(static_cast<const bf16 *>(t.in)[i]);
}

// The block's sum of v, in a fixed order, in thread 0.
__device__ double block_sum(double v) {
  __shared__ double part[kClipThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kClipThreads / 32; ++w) v += part[w];
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kClipThreads)
clip_sum_kernel(const __grid_constant__ ClipTable tab, double *partial) {
  double sum = 0.0;
  for (int k = 0; k < tab.count; ++k) {
    const ClipTensor &t = tab.t[k];
    for (int64_t i = blockIdx.x * (int64_t)kClipThreads + threadIdx.x; i < t.n;
         i += (int64_t)kClipBlocks * kClipThreads) {
      const double x = clip_load(t, i);
      sum += x * x;
    }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kClipThreads)
clip_norm_kernel(const double *partial, int64_t n, float *norm) {
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kClipThreads) sum += partial[i];
  sum = block_sum(sum);
  if (threadIdx.x == 0) *norm = (float)sqrt(sum);
}

__global__ void __launch_bounds__(kClipThreads)
clip_scale_kernel(const __grid_constant__ ClipTable tab, const float *norm, float max_norm) {
  const float r = max_norm / (*norm + 1e-6f);
  const float c = r < 1.0f || r != r ? r : 1.0f;
  for (int k = 0; k < tab.count; ++k) {
    const ClipTensor &t = tab.t[k];
    for (int64_t i = blockIdx.x * (int64_t)kClipThreads + threadIdx.x; i < t.n;
         i += (int64_t)kClipBlocks * kClipThreads) {
      const float x = clip_load(t, i) * c;
      if (t.dtype == GEMM_DT_F32)
        static_cast<float *>(t.out)[i] = x;
      else
        static_cast<bf16 *>(t.out)[i] = from_f32<bf16>(x);
    }
  }
}

int64_t clip_launches(int64_t count) { return count > 0 ? ceil_div(count, kClipTable) : 0; }

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

uint64_t grad_norm_clip_workspace(int64_t count) {
  return (uint64_t)(count > 0 ? clip_launches(count) : 0) * kClipBlocks * sizeof(double);
}

int grad_norm_clip(int64_t count, const int *dtypes, const void *const *grads, void *const *outs,
                   const int64_t *sizes, float max_norm, float *norm, void *workspace,
                   size_t ws_bytes, cudaStream_t stream) {
  if (count < 0 || count > ((int64_t)1 << 24) || !norm ||
      (reinterpret_cast<uintptr_t>(norm) & 3) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return GEMM_ERR_INVALID_ARG;
  if (count > 0 && (!dtypes || !grads || !sizes)) return GEMM_ERR_INVALID_ARG;
  if (outs && !(max_norm >= 0.0f)) return GEMM_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    if (!dtype_known(dtypes[i]) || sizes[i] < 0 || sizes[i] > ((int64_t)1 << 46))
      return GEMM_ERR_INVALID_ARG;
    const uintptr_t mask = dtype_size(dtypes[i]) - 1;
    if (sizes[i] > 0 && (!grads[i] || (reinterpret_cast<uintptr_t>(grads[i]) & mask)))
      return GEMM_ERR_INVALID_ARG;
    if (outs && sizes[i] > 0 && (!outs[i] || (reinterpret_cast<uintptr_t>(outs[i]) & mask)))
      return GEMM_ERR_INVALID_ARG;
  }
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
  double *partial = static_cast<double *>(ws);
  static thread_local ClipTable tab;
  cudaError_t e = cudaSuccess;
  for (int pass = 0; pass < (outs ? 2 : 1) && e == cudaSuccess; ++pass) {
    for (int64_t at = 0; at < count && e == cudaSuccess; at += kClipTable) {
      tab.count = (int)(count - at < kClipTable ? count - at : kClipTable);
      for (int k = 0; k < tab.count; ++k)
        tab.t[k] = {grads[at + k], outs ? outs[at + k] : nullptr, sizes[at + k], dtypes[at + k]};
      if (pass == 0)
        clip_sum_kernel<<<kClipBlocks, kClipThreads, 0, stream>>>(
            tab, partial + at / kClipTable * kClipBlocks);
      else
        clip_scale_kernel<<<kClipBlocks, kClipThreads, 0, stream>>>(tab, norm, max_norm);
      e = cudaGetLastError();
    }
    if (pass == 0 && e == cudaSuccess) {
      clip_norm_kernel<<<1, kClipThreads, 0, stream>>>(partial, clip_launches(count) * kClipBlocks,
                                                       norm);
      e = cudaGetLastError();
    }
  }
  return to_status(e);
}

}  // extern "C"
