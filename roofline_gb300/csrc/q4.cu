// Products with 4-bit weights for a few tokens (include/gb300_gemm.h,
// q4_matmul and q4_gated).
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
};

// One warp computes one output row n for every token, one byte a lane and step.
template <typename T>
__device__ float q4_dot(const Q4Args &p, const Q4Side &w, int64_t m, int64_t n) {
  const int lane = threadIdx.x & 31;
  const T *x = static_cast<const T *>(p.x) + m * p.ldx;
  float acc = 0.0f;
  for (int64_t b = lane; 2 * b < p.K; b += 32) {
    const int64_t g = 2 * b / p.group;
    const float s = to_f32(static_cast<const T *>(w.s)[n * p.groups + g]);
    const float z = w.z ? to_f32(static_cast<const T *>(w.z)[n * p.groups + g]) : 8.0f;
    const int code = w.q[n * w.ldq + b];
    acc = fmaf(s * ((float)(code & 15) - z), to_f32(x[2 * b]), acc);
    if (2 * b + 1 < p.K) acc = fmaf(s * ((float)(code >> 4) - z), to_f32(x[2 * b + 1]), acc);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  return acc;
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(128) q4_kernel(Q4Args p) {
  const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (n >= p.N) return;
  for (int64_t m = 0; m < p.M; ++m) {
    float y = q4_dot<T>(p, p.w[0], m, n);
    if (GATED) {
      const float u = q4_dot<T>(p, p.w[1], m, n);
      with_act(p.act, [&](auto a) { y = act_of<false, decltype(a)::value>(y) * u; });
    }
    if ((threadIdx.x & 31) == 0) static_cast<T *>(p.y)[m * p.ldy + n] = from_f32<T>(y);
  }
}

bool side_ok(const Q4Side &w, const Q4Args &p, int dtype) {
  const uintptr_t mask = dtype_size(dtype) - 1;
  if (w.ldq < (p.K + 1) / 2) return false;
  if (p.M == 0 || p.N == 0 || p.K == 0) return true;
  return w.q && w.s && !(reinterpret_cast<uintptr_t>(w.s) & mask) &&
         !(reinterpret_cast<uintptr_t>(w.z) & mask);
}

int run_q4(int dtype, int sides, const Q4Args &p, cudaStream_t stream) {
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
  const uintptr_t mask = dtype_size(dtype) - 1;
  if (!p.y || (reinterpret_cast<uintptr_t>(p.y) & mask) ||
      (p.K > 0 && (!p.x || (reinterpret_cast<uintptr_t>(p.x) & mask))))
    return GEMM_ERR_INVALID_ARG;
  int dev = -1;
  const int st = current_device(&dev);
  if (st != GEMM_OK) return st;
  const unsigned grid = (unsigned)ceil_div(p.N, 4);
  if (dtype == GEMM_DT_F32) {
    if (sides == 2)
      q4_kernel<float, true><<<grid, 128, 0, stream>>>(p);
    else
      q4_kernel<float, false><<<grid, 128, 0, stream>>>(p);
  } else {
    if (sides == 2)
      q4_kernel<bf16, true><<<grid, 128, 0, stream>>>(p);
    else
      q4_kernel<bf16, false><<<grid, 128, 0, stream>>>(p);
  }
  return to_status(cudaGetLastError());
}

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

int q4_matmul(int dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
              const void *Q, int64_t ldq, const void *S, const void *Z, int group, void *Y,
              int64_t ldy, cudaStream_t stream) {
  const Q4Args p{M, N, K, ldx, ldy, group > 0 ? ceil_div(K, group) : 0, GEMM_ACT_SILU, group, X,
                 Y, {{static_cast<const uint8_t *>(Q), ldq, S, Z}, {nullptr, 0, nullptr, nullptr}}};
  return run_q4(dtype, 1, p, stream);
}

int q4_gated(int dtype, int act, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
             const void *Qg, int64_t ldqg, const void *Sg, const void *Zg, const void *Qu,
             int64_t ldqu, const void *Su, const void *Zu, int group, void *H, int64_t ldh,
             cudaStream_t stream) {
  const Q4Args p{M, N, K, ldx, ldh, group > 0 ? ceil_div(K, group) : 0, act, group, X, H,
                 {{static_cast<const uint8_t *>(Qg), ldqg, Sg, Zg},
                  {static_cast<const uint8_t *>(Qu), ldqu, Su, Zu}}};
  return run_q4(dtype, 2, p, stream);
}

}  // extern "C"
