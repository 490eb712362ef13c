// Shared by the feed-forward operators (ff.cu, q4.cu, clip.cu): element types
// and the activations with their derivatives.
#pragma once

#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"

namespace gg {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x) {
  return __float2bfloat16_rn(x);
}

// 1 / (1 + exp(-x)) with the fast exponential and quotient.  Its relative
// error, 2^-22 and 2^-24 |x|, counts in act(g) times 1 - sigmoid, so what
// reaches the result is under 1e-7 of max(|g|, 1): FP32's own rounding.
__device__ __forceinline__ float sigmoid(float x) {
  return __fdividef(1.0f, 1.0f + __expf(-x));
}

// act(g) (formulas in gb300_gemm.h).
template <int ACT>
__device__ __forceinline__ float act_of(float g) {
  if (ACT == GEMM_ACT_SILU) return g * sigmoid(g);
  if (ACT == GEMM_ACT_RELU) return g > 0.0f ? g : (g != g ? g : 0.0f);
  if (ACT == GEMM_ACT_GELU) return 0.5f * g * (1.0f + erff(g * 0.70710678f));
  // (1 + tanh(u)) / 2 = sigmoid(2u)
  return g * sigmoid(2.0f * 0.79788456f * (g + 0.044715f * g * g * g));
}

// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ void act_both(float g, float &a, float &d) {
  if (ACT == GEMM_ACT_SILU) {
    const float s = sigmoid(g);
    a = g * s;
    d = s * (1.0f + g * (1.0f - s));
  } else if (ACT == GEMM_ACT_RELU) {
    a = act_of<ACT>(g);
    d = g > 0.0f ? 1.0f : 0.0f;
  } else if (ACT == GEMM_ACT_GELU) {
    const float p = 0.5f * (1.0f + erff(g * 0.70710678f));
    a = g * p;
    d = p + g * 0.39894228f * __expf(-0.5f * g * g);
  } else {
    const float s = sigmoid(2.0f * 0.79788456f * (g + 0.044715f * g * g * g));
    a = g * s;
    d = s + 2.0f * g * s * (1.0f - s) * 0.79788456f * (1.0f + 0.134145f * g * g);
  }
}

// f with the activation as a compile-time value: the choice is made once for
// a block of values, not for each (unrolled 32 times, the four branches were
// more code than the instruction cache holds).
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case GEMM_ACT_SILU: f(std::integral_constant<int, GEMM_ACT_SILU>()); break;
    case GEMM_ACT_GELU: f(std::integral_constant<int, GEMM_ACT_GELU>()); break;
    case GEMM_ACT_GELU_TANH: f(std::integral_constant<int, GEMM_ACT_GELU_TANH>()); break;
    default: f(std::integral_constant<int, GEMM_ACT_RELU>()); break;
  }
}

inline bool dtype_known(int d) { return d == GEMM_DT_F32 || d == GEMM_DT_BF16; }
inline bool act_known(int a) { return a >= GEMM_ACT_SILU && a <= GEMM_ACT_RELU; }
inline size_t dtype_size(int d) { return d == GEMM_DT_F32 ? 4 : 2; }

// Lets a kernel use `bytes` of dynamic shared memory on device `dev`.  The
// attribute stays with the kernel, so each launcher keeps one Once for its
// kernel and sets it once for each device: half a microsecond of every later
// call.  (Two threads that set it at once do no harm.)
struct Once {
  std::atomic<bool> done[64] = {};
};
template <typename K>
cudaError_t allow_shared_memory(Once &once, K kern, int bytes, int dev) {
  const bool known = dev >= 0 && dev < 64;
  if (known && once.done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && known) once.done[dev].store(true, std::memory_order_relaxed);
  return e;
}

// abi.cu
int current_device(int *dev);
int library_workspace(int dev, size_t need, void **out);
int to_status(cudaError_t e);

}  // namespace gg
