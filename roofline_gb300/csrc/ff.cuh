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

// The activations are computed in FP32 for results of type T.  FP32 results
// take expf and erfcf (2048 x 1024 x 2816 trained with GELU: 337 us, 328 with
// erff, whose 2^-23 of 1 is all there is of the negative tail at g = -5).  For
// BF16 ones, rounded to 2^-9, the fast exponential (2 + 1.2 |x| units of 2^-23
// off) and 1 + erf are enough.  The quotient, of a divisor from 1 to 2, is the
// fast one in both, 2 units of 2^-23 off (rounded, 1023 x 777 x 1025 in FP32
// takes 28.8 us instead of 27.2).
template <typename T>
__device__ __forceinline__ float exp_for(float x) {
  return std::is_same<T, float>::value ? expf(x) : __expf(x);
}

// s = 1 / (1 + exp(-x)) and c = 1 - s, each with the relative accuracy of the
// exponential, by e = exp(-|x|) <= 1: neither tail cancels or leaves the range
// before the result itself does.
struct Logistic {
  float s, c;
};
template <typename T>
__device__ __forceinline__ Logistic logistic(float x) {
  const float e = exp_for<T>(-fabsf(x));
  const float r = __fdividef(1.0f, 1.0f + e);
  return x >= 0.0f ? Logistic{r, e * r} : Logistic{e * r, r};
}

// (1 + erf(g / sqrt(2))) / 2.  In FP32 by erfc, which keeps the negative tail.
template <typename T>
__device__ __forceinline__ float normal_cdf(float g) {
  return std::is_same<T, float>::value ? 0.5f * erfcf(g * -0.70710678f)
                                       : 0.5f * (1.0f + erff(g * 0.70710678f));
}

// (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u)), u as in the header's GELU_TANH.
template <typename T>
__device__ __forceinline__ Logistic tanh_gate(float g) {
  return logistic<T>(2.0f * 0.79788456f * (g + 0.044715f * g * g * g));
}

// act(g) (formulas in gb300_gemm.h).
template <typename T, int ACT>
__device__ __forceinline__ float act_of(float g) {
  if (ACT == GEMM_ACT_SILU) return g * logistic<T>(g).s;
  if (ACT == GEMM_ACT_RELU) return g > 0.0f ? g : (g != g ? g : 0.0f);
  if (ACT == GEMM_ACT_GELU) return g * normal_cdf<T>(g);
  return g * tanh_gate<T>(g).s;
}

// act(g) and act'(g).
template <typename T, int ACT>
__device__ __forceinline__ void act_both(float g, float &a, float &d) {
  if (ACT == GEMM_ACT_SILU) {
    const Logistic l = logistic<T>(g);
    a = g * l.s;
    d = l.s * (1.0f + g * l.c);
  } else if (ACT == GEMM_ACT_RELU) {
    a = act_of<T, ACT>(g);
    d = g > 0.0f ? 1.0f : 0.0f;
  } else if (ACT == GEMM_ACT_GELU) {
    const float p = normal_cdf<T>(g);
    a = g * p;
    d = p + g * 0.39894228f * exp_for<T>(-0.5f * g * g);
  } else {
    const Logistic l = tanh_gate<T>(g);
    a = g * l.s;
    // s c is 0 long before g g leaves FP32's range, where their product would be NaN
    d = l.s + l.s * l.c * (1.59576912f * (1.0f + 0.134145f * fminf(g * g, 1e30f))) * g;
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
