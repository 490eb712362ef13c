// The tensor-core products of the gated feed-forward block (ff_tc.cu) and the
// passes that lay their operands out (ff_pack.cu).
#pragma once

#include "ff.cuh"

namespace gg {

// A BF16 operand of one product: `planes` matrices of `outer` rows of `inner`
// contiguous elements, rows `ld` and planes `plane` elements apart.  A FP32
// matrix x is three planes x0 + x1 + x2, each the BF16 nearest to what the
// ones before it leave: 24 bits.  mn_major = 0: inner is the summed extent K
// and the rows are rows of A or columns of B; 1: the other way round.
struct FfOperand {
  const bf16 *p;
  int64_t inner, outer, ld, plane;
  int mn_major;
};

// Products of M x K and K x N operands, BF16 planes in, FP32 sums:
//   gated:  c0 = act(a0 b0) * (a0 b1), with the sums to g and u if given
//   concat: c0 = a0 b0 + a1 b1
//   batch:  c0 = a0 b0, c1 = a[a_two] b[b_two]
// Outputs are BF16 for one plane and FP32 for three.
enum FfKind { kFfGated, kFfConcat, kFfBatch };
struct FfProduct {
  FfKind kind;
  int planes, act;
  int64_t M, N, K;
  FfOperand a[2], b[2];
  int a_two, b_two;  // batch: which operands the second product takes
  void *c[2];
  int64_t ldc, ldc2;  // of c0 and c1
  float *g, *u;
  int64_t ldg, ldu;
};
// Enqueues n products in one launch: one, or two that are not gated and of as
// many planes, the one with longer sums first.  Returns a GEMM_* status.
int launch_ff_products(const FfProduct *p, int n, const DeviceProps &dp, cudaStream_t s);
int ff_read_and_clear_status(cudaStream_t s);

// Lays one matrix (rows x cols, row stride ld, FP32 or BF16) out as BF16
// planes whose rows TMA can read: ld_out a multiple of 8, 16-byte aligned.
struct PackJob {
  const void *src;
  int64_t rows, cols, ld;
  bf16 *dst;
  int64_t ld_out, plane;
};
constexpr int kPackJobs = 3;
cudaError_t launch_pack(const PackJob *jobs, int n, int dtype, int sms, cudaStream_t s);

// dG = dH * U * act'(G) and dU = dH * act(G), M x F (neither 0), as such
// planes; launch_dgate: and the jobs, in the same launch.
struct DgateArgs {
  int64_t M, F;
  int act;
  const void *dh;
  int64_t lddh;
  const float *g, *u;
  int64_t ldg, ldu;
  bf16 *dg, *du;
  int64_t ld_out, plane;
};
// The same as M x ld_out floats at dg and du, from FP32.
cudaError_t launch_dgate_f32(const DgateArgs &p, int sms, cudaStream_t s);
cudaError_t launch_dgate(const DgateArgs &p, const PackJob *jobs, int n, int dtype, int sms,
                         cudaStream_t s);

}  // namespace gg
