// The gated feed-forward block and its gradients: argument checks, workspace
// and the launches (include/gb300_gemm.h, gated_ff and gated_ff_backward).
#include "ff.cuh"

namespace gg {
namespace {

// C(i,j) = sum_k A(i,k) B(k,j) (+ sum_k A2(i,k) B2(k,j)); GATED: act of the
// first sum times the second, whose A is the first's.  Element strides.
struct Operand {
  const void *p;
  int64_t rs, cs;
};
struct SimpleArgs {
  int64_t M, N, K;
  int act;
  Operand a, b, a2, b2;
  void *c;
  float *g, *u;
  int64_t ldc, ldg, ldu;
};

// One 16 x 16 tile of C per block through shared memory, one value a thread.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256) ff_simple_kernel(SimpleArgs p) {
  __shared__ float sa[16][17], sb[16][17], sb2[16][17];
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int64_t i = (int64_t)blockIdx.y * 16 + ty, j = (int64_t)blockIdx.x * 16 + tx;
  float s = 0.0f, s2 = 0.0f;
  const int parts = !GATED && p.a2.p != nullptr ? 2 : 1;
  for (int part = 0; part < parts; ++part) {
    const Operand &A = part ? p.a2 : p.a, &B = part ? p.b2 : p.b;
    for (int64_t k0 = 0; k0 < p.K; k0 += 16) {
      const int64_t ka = k0 + tx, kb = k0 + ty;
      sa[ty][tx] = i < p.M && ka < p.K
                       ? to_f32(static_cast<const T *>(A.p)[i * A.rs + ka * A.cs])
                       : 0.0f;
      sb[ty][tx] = j < p.N && kb < p.K
                       ? to_f32(static_cast<const T *>(B.p)[kb * B.rs + j * B.cs])
                       : 0.0f;
      if (GATED)
        sb2[ty][tx] = j < p.N && kb < p.K
                          ? to_f32(static_cast<const T *>(p.b2.p)[kb * p.b2.rs + j * p.b2.cs])
                          : 0.0f;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        s = fmaf(sa[ty][k], sb[k][tx], s);
        if (GATED) s2 = fmaf(sa[ty][k], sb2[k][tx], s2);
      }
      __syncthreads();
    }
  }
  if (i >= p.M || j >= p.N) return;
  if (GATED) {
    if (p.g) p.g[i * p.ldg + j] = s;
    if (p.u) p.u[i * p.ldu + j] = s2;
    s = act_value<false>(s, p.act) * s2;
  }
  if (p.c) static_cast<T *>(p.c)[i * p.ldc + j] = from_f32<T>(s);
}

template <typename T, bool GATED>
cudaError_t launch_simple(const SimpleArgs &p, cudaStream_t s) {
  if (p.M == 0 || p.N == 0) return cudaSuccess;
  ff_simple_kernel<T, GATED><<<dim3((unsigned)ceil_div(p.N, 16), (unsigned)ceil_div(p.M, 16)),
                               dim3(16, 16), 0, s>>>(p);
  return cudaGetLastError();
}

// dG = dH * U * act'(G), dU = dH * act(G), each M x F, contiguous.
template <typename T>
__global__ void __launch_bounds__(256)
ff_dgate_kernel(int64_t M, int64_t F, int act, const T *dH, int64_t lddh, const float *G,
                int64_t ldg, const float *U, int64_t ldu, T *dG, T *dU) {
  const int64_t n = M * F;
  for (int64_t e = blockIdx.x * 256ll + threadIdx.x; e < n; e += gridDim.x * 256ll) {
    const int64_t i = e / F, j = e - i * F;
    const float h = to_f32(dH[i * lddh + j]);
    float a, d;
    act_both<false>(G[i * ldg + j], act, a, d);
    dG[e] = from_f32<T>(h * U[i * ldu + j] * d);
    dU[e] = from_f32<T>(h * a);
  }
}

bool ld_ok(int64_t ld, int64_t width) { return ld >= (width > 1 ? width : 1); }
uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

// The extents that every kernel takes: 32-bit tile coordinates.
constexpr int64_t kMaxExtent = ((int64_t)1 << 31) - 512;
constexpr int64_t kMaxLd = (int64_t)1 << 36;

int check_sizes(int dtype, int act, int op_w, int64_t M, int64_t D, int64_t F) {
  if (!dtype_known(dtype) || !act_known(act) || (op_w != GEMM_OP_N && op_w != GEMM_OP_T))
    return GEMM_ERR_INVALID_ARG;
  if (M < 0 || D < 0 || F < 0) return GEMM_ERR_INVALID_ARG;
  if (M > kMaxExtent || D > kMaxExtent || F > kMaxExtent) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

// A matrix argument: its pointer aligned to its elements and, unless the
// matrix is empty, not null; its leading dimension no less than a row.
bool matrix_ok(const void *p, int64_t ld, int64_t rows, int64_t cols, int dtype) {
  if (!ld_ok(ld, cols) || ld > kMaxLd) return false;
  if (rows == 0 || cols == 0) return true;
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (dtype_size(dtype) - 1)) == 0;
}

Operand weight(const void *w, int64_t ld, int op_w) {  // as the D x F matrix
  return op_w == GEMM_OP_N ? Operand{w, ld, 1} : Operand{w, 1, ld};
}

uint64_t backward_bytes(int dtype, int64_t M, int64_t F) {
  return 2 * align256((uint64_t)M * (uint64_t)F * dtype_size(dtype));
}

// The caller's workspace, or the library's.
int take_workspace(int dev, uint64_t need, void *workspace, size_t ws_bytes, void **out) {
  *out = nullptr;
  if (need == 0) return GEMM_OK;
  if (workspace == nullptr) return library_workspace(dev, (size_t)need, out);
  if (ws_bytes < need) return GEMM_ERR_WORKSPACE_TOO_SMALL;
  *out = workspace;
  return GEMM_OK;
}

template <typename T>
int run_forward(const SimpleArgs &p, cudaStream_t stream) {
  return to_status(launch_simple<T, true>(p, stream));
}

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

int gated_ff_workspace(int backward, int dtype, int op_w, int64_t M, int64_t D, int64_t F,
                       int aligned, uint64_t *bytes) {
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  const int st = check_sizes(dtype, GEMM_ACT_SILU, op_w, M, D, F);
  if (st != GEMM_OK) return st;
  (void)aligned;
  *bytes = backward ? backward_bytes(dtype, M, F) : 0;
  return GEMM_OK;
}

int gated_ff(int dtype, int act, int op_w, int64_t M, int64_t D, int64_t F, const void *X,
             int64_t ldx, const void *Wg, int64_t ldwg, const void *Wu, int64_t ldwu, void *H,
             int64_t ldh, float *G, int64_t ldg, float *U, int64_t ldu, void *workspace,
             size_t ws_bytes, cudaStream_t stream) {
  int st = check_sizes(dtype, act, op_w, M, D, F);
  if (st != GEMM_OK) return st;
  const int64_t wr = op_w == GEMM_OP_N ? D : F, wc = op_w == GEMM_OP_N ? F : D;
  const bool none = M == 0 || F == 0;
  if (!matrix_ok(X, ldx, none ? 0 : M, D, dtype) || !matrix_ok(Wg, ldwg, none ? 0 : wr, wc, dtype) ||
      !matrix_ok(Wu, ldwu, none ? 0 : wr, wc, dtype))
    return GEMM_ERR_INVALID_ARG;
  if ((G == nullptr) != (U == nullptr) || (H == nullptr && G == nullptr && !none))
    return GEMM_ERR_INVALID_ARG;
  if ((H && !matrix_ok(H, ldh, M, F, dtype)) || (G && !matrix_ok(G, ldg, M, F, GEMM_DT_F32)) ||
      (U && !matrix_ok(U, ldu, M, F, GEMM_DT_F32)))
    return GEMM_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return GEMM_ERR_INVALID_ARG;
  if (none) return GEMM_OK;
  int dev = -1;
  st = current_device(&dev);
  if (st != GEMM_OK) return st;
  (void)ws_bytes;
  SimpleArgs p{M, F, D, act, {X, ldx, 1}, weight(Wg, ldwg, op_w), {nullptr, 0, 0},
               weight(Wu, ldwu, op_w), H, G, U, ldh, ldg, ldu};
  return dtype == GEMM_DT_F32 ? run_forward<float>(p, stream) : run_forward<bf16>(p, stream);
}

}  // extern "C"

namespace gg {
namespace {

template <typename T>
int run_backward(int act, int op_w, int64_t M, int64_t D, int64_t F, const void *dH, int64_t lddh,
                 const void *X, int64_t ldx, const void *Wg, int64_t ldwg, const void *Wu,
                 int64_t ldwu, const float *G, int64_t ldg, const float *U, int64_t ldu, void *dX,
                 int64_t lddx, void *dWg, int64_t lddwg, void *dWu, int64_t lddwu, void *ws,
                 cudaStream_t s) {
  T *dG = static_cast<T *>(ws);
  T *dU = reinterpret_cast<T *>(static_cast<uint8_t *>(ws) +
                                align256((uint64_t)M * (uint64_t)F * sizeof(T)));
  cudaError_t e = cudaSuccess;
  if (M > 0 && F > 0) {
    const int64_t blocks = ceil_div(M * F, 256);
    ff_dgate_kernel<T><<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(
        M, F, act, static_cast<const T *>(dH), lddh, G, ldg, U, ldu, dG, dU);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && dX) {
    Operand wg = weight(Wg, ldwg, op_w), wu = weight(Wu, ldwu, op_w);
    SimpleArgs p{M, D, F, act, {dG, F, 1}, {wg.p, wg.cs, wg.rs}, {dU, F, 1},
                 {wu.p, wu.cs, wu.rs}, dX, nullptr, nullptr, lddx, 0, 0};
    e = launch_simple<T, false>(p, s);
  }
  for (int k = 0; k < 2 && e == cudaSuccess && dWg; ++k) {
    void *dW = k ? dWu : dWg;
    const int64_t ld = k ? lddwu : lddwg;
    const T *d = k ? dU : dG;
    const Operand none{nullptr, 0, 0};
    SimpleArgs p = op_w == GEMM_OP_N
                       ? SimpleArgs{D, F, M, act, {X, 1, ldx}, {d, F, 1}, none, none, dW,
                                    nullptr, nullptr, ld, 0, 0}
                       : SimpleArgs{F, D, M, act, {d, 1, F}, {X, ldx, 1}, none, none, dW,
                                    nullptr, nullptr, ld, 0, 0};
    e = launch_simple<T, false>(p, s);
  }
  return to_status(e);
}

}  // namespace
}  // namespace gg

extern "C" int gated_ff_backward(int dtype, int act, int op_w, int64_t M, int64_t D, int64_t F,
                                 const void *dH, int64_t lddh, const void *X, int64_t ldx,
                                 const void *Wg, int64_t ldwg, const void *Wu, int64_t ldwu,
                                 const float *G, int64_t ldg, const float *U, int64_t ldu, void *dX,
                                 int64_t lddx, void *dWg, int64_t lddwg, void *dWu,
                                 int64_t lddwu, void *workspace, size_t ws_bytes,
                                 cudaStream_t stream) {
  int st = check_sizes(dtype, act, op_w, M, D, F);
  if (st != GEMM_OK) return st;
  const int64_t wr = op_w == GEMM_OP_N ? D : F, wc = op_w == GEMM_OP_N ? F : D;
  if ((dWg == nullptr) != (dWu == nullptr)) return GEMM_ERR_INVALID_ARG;
  if (dX == nullptr && dWg == nullptr && D > 0 && (M > 0 || F > 0)) return GEMM_ERR_INVALID_ARG;
  if (!matrix_ok(dH, lddh, M, F, dtype) || !matrix_ok(G, ldg, M, F, GEMM_DT_F32) ||
      !matrix_ok(U, ldu, M, F, GEMM_DT_F32))
    return GEMM_ERR_INVALID_ARG;
  if (dX && (!matrix_ok(dX, lddx, M, D, dtype) || !matrix_ok(Wg, ldwg, M ? wr : 0, wc, dtype) ||
             !matrix_ok(Wu, ldwu, M ? wr : 0, wc, dtype)))
    return GEMM_ERR_INVALID_ARG;
  if (dWg && (!matrix_ok(dWg, lddwg, wr, wc, dtype) || !matrix_ok(dWu, lddwu, wr, wc, dtype) ||
              !matrix_ok(X, ldx, F ? M : 0, D, dtype)))
    return GEMM_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return GEMM_ERR_INVALID_ARG;
  if (D == 0 || (M == 0 && F == 0)) return GEMM_OK;
  int dev = -1;
  st = current_device(&dev);
  if (st != GEMM_OK) return st;
  void *ws = nullptr;
  st = take_workspace(dev, backward_bytes(dtype, M, F), workspace, ws_bytes, &ws);
  if (st != GEMM_OK) return st;
  return dtype == GEMM_DT_F32
             ? run_backward<float>(act, op_w, M, D, F, dH, lddh, X, ldx, Wg, ldwg, Wu, ldwu, G,
                                   ldg, U, ldu, dX, lddx, dWg, lddwg, dWu, lddwu, ws, stream)
             : run_backward<bf16>(act, op_w, M, D, F, dH, lddh, X, ldx, Wg, ldwg, Wu, ldwu, G, ldg,
                                  U, ldu, dX, lddx, dWg, lddwg, dWu, lddwu, ws, stream);
}
