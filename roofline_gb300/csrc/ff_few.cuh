// The gated block and its gradients for a few tokens in FP32 (ff_few.cu).
#pragma once

#include "ff.cuh"

namespace gg {

constexpr int kFewTokens = 16;  // at most

// Two products of M (up to kFewTokens) rows: s_i = a_i b_i with a_i M x K.
//   gated: c = act(s_0) * s_1 (a_0 = a_1), s_0 and s_1 to g and u if given
//   else:  c = s_0 + s_1
// rows_are_outputs: b_i is stored as N rows of K, else as K rows of N.
struct FewArgs {
  int64_t M, N, K;
  int gated, act, rows_are_outputs;
  const float *a[2];
  int64_t lda;
  const float *b[2];
  int64_t ldb[2];
  float *c, *g, *u;
  int64_t ldc, ldg, ldu;
};
uint64_t few_bytes(int64_t M, int64_t N, int64_t K, bool rows_are_outputs, int sms);
cudaError_t launch_few(const FewArgs &p, void *ws, int sms, cudaStream_t s);

// c_i = q_i^T x_i, R x N, from M rows of q_i (R long) and x_i (N long).
struct OuterArgs {
  int64_t M, R, N;
  const float *q[2];
  int64_t ldq[2];
  const float *x[2];
  int64_t ldx[2];
  float *c[2];
  int64_t ldc[2];
};
cudaError_t launch_outer(const OuterArgs &p, cudaStream_t s);

}  // namespace gg
