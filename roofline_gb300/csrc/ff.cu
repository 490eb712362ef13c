// The gated feed-forward block and its gradients: argument checks, workspace
// and the launches (include/gb300_gemm.h, gated_ff and gated_ff_backward).
#include "ff_few.cuh"
#include "ff_tc.cuh"

namespace gg {
namespace {

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

// A stored matrix and, once laid out, the operand made of it.
struct Stored {
  const void *p;
  int64_t rows, cols, ld;
};

int64_t round8(int64_t x) { return (x + 7) / 8 * 8; }
int planes_of(int dtype) { return dtype == GEMM_DT_F32 ? 3 : 1; }
uint64_t plane_bytes(int dtype, int64_t rows, int64_t cols) {
  return align256((uint64_t)planes_of(dtype) * (uint64_t)rows * (uint64_t)round8(cols) * 2);
}

// BF16 rows that TMA reads where they are: 16-byte aligned, or only one.
bool direct(int dtype, const Stored &m) {
  return dtype == GEMM_DT_BF16 && (reinterpret_cast<uintptr_t>(m.p) & 15) == 0 &&
         ((m.ld & 7) == 0 || m.rows == 1);
}

uint64_t pack_bytes(int dtype, const Stored &m) {
  return direct(dtype, m) ? 0 : plane_bytes(dtype, m.rows, m.cols);
}

// Collects the matrices of a call: each is used where it is or gets a place
// in the workspace and a job of the packing pass.
struct Layout {
  int dtype;
  uint8_t *ws;
  PackJob jobs[kPackJobs];
  int n = 0;

  // mn_major: the summed index runs down the rows
  FfOperand operand(const Stored &m, int mn_major) {
    if (direct(dtype, m))
      return {static_cast<const bf16 *>(m.p), m.cols, m.rows,
              m.rows == 1 ? round8(m.cols) : m.ld, 0, mn_major};
    FfOperand o{reinterpret_cast<const bf16 *>(ws), m.cols, m.rows, round8(m.cols),
                m.rows * round8(m.cols), mn_major};
    jobs[n++] = {m.p, m.rows, m.cols, m.ld, reinterpret_cast<bf16 *>(ws), o.ld, o.plane};
    ws += plane_bytes(dtype, m.rows, m.cols);
    return o;
  }
};

Stored weight(const void *w, int64_t ld, int op_w, int64_t D, int64_t F) {
  return op_w == GEMM_OP_N ? Stored{w, D, F, ld} : Stored{w, F, D, ld};
}

cudaError_t zero(void *p, int64_t ld, int64_t rows, int64_t cols, size_t size, cudaStream_t s) {
  if (!p || rows == 0 || cols == 0) return cudaSuccess;
  return cudaMemset2DAsync(p, ld * size, 0, cols * size, rows, s);
}

// FP32 calls that the CUDA cores take (ff_few.cu).  GB300, 4096 x 11008, us by
// the tensor cores / the CUDA cores, for 1, 8 and 16 tokens; weights D x F:
// block 297/94, 297/270, 298/504, gradients 808/167, 807/277, 814/451; weights
// F x D: block 302/86, 301/137, 300/228, gradients 801/168, 801/427, 808/745.
bool few_tokens(int dtype, int64_t M, bool backward, int op_w) {
  return dtype == GEMM_DT_F32 && M <= (backward || op_w == GEMM_OP_T ? kFewTokens : kFewTokens / 2);
}

// dG and dU as floats, then the sums of dX's parts.
uint64_t few_gate_bytes(int64_t M, int64_t F) {
  return align256((uint64_t)M * (uint64_t)round8(F) * 4);
}
uint64_t few_backward_bytes(int op_w, int64_t M, int64_t D, int64_t F, int sms) {
  return 2 * few_gate_bytes(M, F) + few_bytes(M, D, F, op_w == GEMM_OP_N, sms);
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

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

int gated_ff_workspace(int backward, int dtype, int op_w, int64_t M, int64_t D, int64_t F,
                       int aligned, uint64_t *bytes) {
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  const int st = check_sizes(dtype, GEMM_ACT_SILU, op_w, M, D, F);
  if (st != GEMM_OK) return st;
  if (few_tokens(dtype, M, backward != 0, op_w)) {
    *bytes = backward ? few_backward_bytes(op_w, M, D, F, current_props().sm_count)
                      : few_bytes(M, F, D, op_w == GEMM_OP_T, current_props().sm_count);
    return GEMM_OK;
  }
  const bool packed = dtype == GEMM_DT_F32 || !aligned;
  *bytes = packed ? plane_bytes(dtype, M, D) + 2 * plane_bytes(dtype, op_w == GEMM_OP_N ? D : F,
                                                               op_w == GEMM_OP_N ? F : D)
                  : 0;
  if (backward) *bytes += 2 * plane_bytes(dtype, M, F);
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
  const DeviceProps &dp = props_of(dev);
  if (D == 0) {
    cudaError_t e = zero(H, ldh, M, F, dtype_size(dtype), stream);
    if (e == cudaSuccess) e = zero(G, ldg, M, F, 4, stream);
    if (e == cudaSuccess) e = zero(U, ldu, M, F, 4, stream);
    return to_status(e);
  }
  const Stored x{X, M, D, ldx}, wg = weight(Wg, ldwg, op_w, D, F), wu = weight(Wu, ldwu, op_w, D, F);
  void *ws = nullptr;
  if (few_tokens(dtype, M, false, op_w)) {
    st = take_workspace(dev, few_bytes(M, F, D, op_w == GEMM_OP_T, dp.sm_count), workspace, ws_bytes,
                        &ws);
    if (st != GEMM_OK) return st;
    FewArgs p{};
    p.M = M;
    p.N = F;
    p.K = D;
    p.gated = 1;
    p.act = act;
    p.rows_are_outputs = op_w == GEMM_OP_T;
    p.a[0] = p.a[1] = static_cast<const float *>(X);
    p.lda = ldx;
    p.b[0] = static_cast<const float *>(Wg);
    p.b[1] = static_cast<const float *>(Wu);
    p.ldb[0] = ldwg;
    p.ldb[1] = ldwu;
    p.c = static_cast<float *>(H);
    p.ldc = ldh;
    p.g = G;
    p.u = U;
    p.ldg = ldg;
    p.ldu = ldu;
    return to_status(launch_few(p, ws, dp.sm_count, stream));
  }
  st = take_workspace(dev, pack_bytes(dtype, x) + pack_bytes(dtype, wg) + pack_bytes(dtype, wu),
                      workspace, ws_bytes, &ws);
  if (st != GEMM_OK) return st;
  Layout lay{dtype, static_cast<uint8_t *>(ws)};
  FfProduct p{};
  p.kind = kFfGated;
  p.planes = planes_of(dtype);
  p.act = act;
  p.M = M;
  p.N = F;
  p.K = D;
  p.a[0] = lay.operand(x, 0);
  p.b[0] = lay.operand(wg, op_w == GEMM_OP_N);
  p.b[1] = lay.operand(wu, op_w == GEMM_OP_N);
  p.c[0] = H;
  p.ldc = ldh;
  p.g = G;
  p.u = U;
  p.ldg = ldg;
  p.ldu = ldu;
  const cudaError_t e = launch_pack(lay.jobs, lay.n, dtype, dp.sm_count, stream);
  return e == cudaSuccess ? launch_ff_products(&p, 1, dp, stream) : to_status(e);
}

}  // extern "C"

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
  const DeviceProps &dp = props_of(dev);
  const size_t size = dtype_size(dtype);
  // an empty sum: zeros
  if (M == 0 || F == 0) {
    cudaError_t e = zero(dX, lddx, M, D, size, stream);
    if (e == cudaSuccess) e = zero(dWg, lddwg, wr, wc, size, stream);
    if (e == cudaSuccess) e = zero(dWu, lddwu, wr, wc, size, stream);
    return to_status(e);
  }
  const Stored x{X, M, D, ldx}, wg = weight(Wg, ldwg, op_w, D, F), wu = weight(Wu, ldwu, op_w, D, F);
  if (few_tokens(dtype, M, true, op_w)) {
    void *few = nullptr;
    st = take_workspace(dev, few_backward_bytes(op_w, M, D, F, dp.sm_count), workspace, ws_bytes, &few);
    if (st != GEMM_OK) return st;
    const uint64_t part = few_gate_bytes(M, F);
    uint8_t *at = static_cast<uint8_t *>(few);
    const float *dg = reinterpret_cast<float *>(at), *du = reinterpret_cast<float *>(at + part);
    const DgateArgs gate{M, F, act, dH, lddh, G, U, ldg, ldu, reinterpret_cast<bf16 *>(at),
                         reinterpret_cast<bf16 *>(at + part), round8(F), 0};
    cudaError_t e = launch_dgate_f32(gate, dp.sm_count, stream);
    if (e == cudaSuccess && dX) {
      FewArgs p{};
      p.M = M;
      p.N = D;
      p.K = F;
      p.rows_are_outputs = op_w == GEMM_OP_N;
      p.a[0] = dg;
      p.a[1] = du;
      p.lda = round8(F);
      p.b[0] = static_cast<const float *>(Wg);
      p.b[1] = static_cast<const float *>(Wu);
      p.ldb[0] = ldwg;
      p.ldb[1] = ldwu;
      p.c = static_cast<float *>(dX);
      p.ldc = lddx;
      e = launch_few(p, at + 2 * part, dp.sm_count, stream);
    }
    if (e == cudaSuccess && dWg) {
      // stored D x F: rows of X by columns of dG; stored F x D the other way
      const float *x = static_cast<const float *>(X), *d[2] = {dg, du};
      OuterArgs p{};
      p.M = M;
      p.R = wr;
      p.N = wc;
      for (int i = 0; i < 2; ++i) {
        p.q[i] = op_w == GEMM_OP_N ? x : d[i];
        p.ldq[i] = op_w == GEMM_OP_N ? ldx : round8(F);
        p.x[i] = op_w == GEMM_OP_N ? d[i] : x;
        p.ldx[i] = op_w == GEMM_OP_N ? round8(F) : ldx;
        p.c[i] = static_cast<float *>(i ? dWu : dWg);
        p.ldc[i] = i ? lddwu : lddwg;
      }
      e = launch_outer(p, stream);
    }
    return to_status(e);
  }
  const uint64_t part = plane_bytes(dtype, M, F);
  uint64_t need = 2 * part;
  if (dX) need += pack_bytes(dtype, wg) + pack_bytes(dtype, wu);
  if (dWg) need += pack_bytes(dtype, x);
  void *ws = nullptr;
  st = take_workspace(dev, need, workspace, ws_bytes, &ws);
  if (st != GEMM_OK) return st;
  uint8_t *at = static_cast<uint8_t *>(ws);
  Layout lay{dtype, at + 2 * part};
  bf16 *dg = reinterpret_cast<bf16 *>(at), *du = reinterpret_cast<bf16 *>(at + part);
  const int64_t ld = round8(F);
  const DgateArgs gate{M, F, act, dH, lddh, G, U, ldg, ldu, dg, du, ld, M * ld};
  // dG and dU as an operand whose summed index is the width F (dX) or the token (dW)
  auto grad = [&](const bf16 *p, int mn_major) {
    return FfOperand{p, F, M, ld, M * ld, mn_major};
  };
  FfProduct px{}, pw{};
  px.planes = pw.planes = planes_of(dtype);
  if (dX) {
    px.kind = kFfConcat;
    px.M = M;
    px.N = D;
    px.K = F;
    px.a[0] = grad(dg, 0);
    px.a[1] = grad(du, 0);
    px.b[0] = lay.operand(wg, op_w == GEMM_OP_T);
    px.b[1] = lay.operand(wu, op_w == GEMM_OP_T);
    px.c[0] = dX;
    px.ldc = lddx;
  }
  if (dWg) {
    // stored D x F: X^T dG; stored F x D: dG^T X
    const FfOperand ox = lay.operand(x, 1);
    pw.kind = kFfBatch;
    pw.M = wr;
    pw.N = wc;
    pw.K = M;
    pw.a[0] = op_w == GEMM_OP_N ? ox : grad(dg, 1);
    pw.b[0] = op_w == GEMM_OP_N ? grad(dg, 1) : ox;
    pw.a_two = op_w == GEMM_OP_T;
    pw.b_two = op_w == GEMM_OP_N;
    (op_w == GEMM_OP_N ? pw.b : pw.a)[1] = grad(du, 1);
    pw.c[0] = dWg;
    pw.c[1] = dWu;
    pw.ldc = lddwg;
    pw.ldc2 = lddwu;
  }
  const cudaError_t e = launch_dgate(gate, lay.jobs, lay.n, dtype, dp.sm_count, stream);
  if (e != cudaSuccess) return to_status(e);
  if (!dX || !dWg) return launch_ff_products(dX ? &px : &pw, 1, dp, stream);
  // Both in one launch, always: the tiles that do not fill a wave of one product
  // are followed by the other's, which pays in all of these but one.  Apart / merged with the gate's pass, us: BF16
  // 2048 x 1024 x 2816 91 / 55, 1024 x 1024 x 2816 62 / 57, 4096 x 4096 x 11008
  // 1112 / 1035, 8192 x 4096 x 11008 2137 / 2069, 1024 x 4096 x 11008 (weights
  // D x F) 299 / 319; FP32 2048 x 1024 x 2816 271 / 199.
  const FfProduct both[2] = {2 * F >= M ? px : pw, 2 * F >= M ? pw : px};
  return launch_ff_products(both, 2, dp, stream);
}
