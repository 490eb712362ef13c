// The gated block and its gradients for a few tokens in FP32, on the CUDA
// cores.
//
// With M tokens each weight takes M multiply-adds and 4 bytes, so reading the
// weights is what a few tokens cannot do without; laying them out as BF16
// planes for the tensor cores (4 bytes read, 6 written and 6 read again) takes
// four times that.  These kernels read FP32 weights once for every 8 tokens
// and add in FP32; the gradients of the weights are sums of M outer products,
// bound by writing them.
//
// Weights with K contiguous: a warp has two rows of each matrix, its lanes
// split K.  Weights with the outputs contiguous: a lane has four outputs, the
// warps and blocks split K and a second pass adds the blocks' sums.  All sums
// are added in a fixed order.  x of all the tokens is loaded ahead of its
// products, and registers are held to two blocks an SM: without the two, 8
// tokens by 4096 x 11008 took 328 us where they now take 137 (rows), 408 and
// 270 (columns).  One token takes 86 and 94 us for 361 MB, 4.2 and 3.8 TB/s
// with the weights out of the L2, and 16 tokens pass over the weights twice.
#include "ff_few.cuh"
#include "tc_common.cuh"

namespace gg {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Four values of a row from column c on; zeros from `cols` on.
template <bool VEC>
__device__ __forceinline__ float4 load4(const float *row, int64_t c, int64_t cols) {
  if (VEC && c + 4 <= cols) return __ldg(reinterpret_cast<const float4 *>(row + c));
  float4 v;
  v.x = c < cols ? row[c] : 0.0f;
  v.y = c + 1 < cols ? row[c + 1] : 0.0f;
  v.z = c + 2 < cols ? row[c + 2] : 0.0f;
  v.w = c + 3 < cols ? row[c + 3] : 0.0f;
  return v;
}

__device__ __forceinline__ float dot4(float s, const float4 &a, const float4 &b) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}

// c (and g, u) from the sums of the two products.
__device__ __forceinline__ void finish(const FewArgs &p, int64_t m, int64_t n, float s0, float s1) {
  if (!p.gated) {
    p.c[m * p.ldc + n] = s0 + s1;
    return;
  }
  if (p.g) {
    p.g[m * p.ldg + n] = s0;
    p.u[m * p.ldu + n] = s1;
  }
  if (p.c) with_act(p.act, [&](auto a) { p.c[m * p.ldc + n] = act_of<float, decltype(a)::value>(s0) * s1; });
}

// b0, b1: N rows of K.  Two rows of each a warp; `split` warps of a block share
// them, taking 128 values of K in turn.
template <int MT, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) few_rows_kernel(const FewArgs p, int split) {
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  __shared__ float red[kWarps][2][2][MT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t m0 = (int64_t)blockIdx.y * MT;
  const int64_t n0 = ((int64_t)blockIdx.x * (kWarps / split) + warp / split) * 2;
  float acc[2][2][MT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[i][r][m] = 0.0f;
  if (n0 < p.N) {
    const float *w[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        w[i][r] = p.b[i] + (n0 + r < p.N ? n0 + r : n0) * p.ldb[i];
#pragma unroll 2
    for (int64_t k = (warp % split) * 128 + lane * 4; k < p.K; k += split * 128) {
      float4 v[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) v[i][r] = load4<VEC>(w[i][r], k, p.K);
      float4 x[MT];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 0 || !p.gated) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int64_t t = m0 + m < p.M ? m0 + m : p.M - 1;  // a token that is not there: unused
            x[m] = load4<VEC>(p.a[i] + t * p.lda, k, p.K);
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < 2; ++r) acc[i][r][m] = dot4(acc[i][r][m], v[i][r], x[m]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float s = acc[i][r][m];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) red[warp][i][r][m] = s;
      }
  __syncthreads();
  for (int e = threadIdx.x; e < kWarps / split * 2 * MT; e += kThreads) {
    const int r = e & 1, m = (e >> 1) % MT, part = (e >> 1) / MT;
    const int64_t n = ((int64_t)blockIdx.x * (kWarps / split) + part) * 2 + r;
    if (n >= p.N || m0 + m >= p.M) continue;
    float s0 = 0.0f, s1 = 0.0f;
    for (int w = part * split; w < (part + 1) * split; ++w) {
      s0 += red[w][0][r][m];
      s1 += red[w][1][r][m];
    }
    finish(p, m0 + m, n, s0, s1);
  }
}

// b0, b1: K rows of N.  A lane has four columns, a block 128; its warps take
// four rows of K in turn, and blockIdx.z parts of K: their sums go to
// partial[part][i][m][n].
template <int MT, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) few_cols_kernel(const FewArgs p, float *partial) {
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  __shared__ float4 red[kWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t m0 = (int64_t)blockIdx.y * MT, n = (int64_t)blockIdx.x * 128 + lane * 4;
  float4 acc[2][MT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  constexpr int R = MT > 4 ? 2 : 4;  // rows at a time: registers for two blocks an SM
  const int64_t step = (int64_t)gridDim.z * kWarps * R;
  for (int64_t k = ((int64_t)blockIdx.z * kWarps + warp) * R; k < p.K; k += step) {
    float4 v[2][R];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j)
        v[i][j] = k + j < p.K ? load4<VEC>(p.b[i] + (k + j) * p.ldb[i], n, p.N)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float x[MT][R];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i == 0 || !p.gated) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int64_t t = m0 + m < p.M ? m0 + m : p.M - 1;
          const float *row = p.a[i] + t * p.lda;
          if (VEC && R == 4 && k + 4 <= p.K) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(row + k));
            x[m][0] = f.x, x[m][1] = f.y, x[m][R - 2] = f.z, x[m][R - 1] = f.w;
          } else {
#pragma unroll
            for (int j = 0; j < R; ++j) x[m][j] = k + j < p.K ? row[k + j] : 0.0f;
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < R; ++j) {
          acc[i][m].x = fmaf(x[m][j], v[i][j].x, acc[i][m].x);
          acc[i][m].y = fmaf(x[m][j], v[i][j].y, acc[i][m].y);
          acc[i][m].z = fmaf(x[m][j], v[i][j].z, acc[i][m].z);
          acc[i][m].w = fmaf(x[m][j], v[i][j].w, acc[i][m].w);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      __syncthreads();
      red[warp][lane] = acc[i][m];
      __syncthreads();
      if (threadIdx.x < 128 && m0 + m < p.M) {
        const int64_t col = (int64_t)blockIdx.x * 128 + threadIdx.x;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          s += reinterpret_cast<const float *>(red[w])[threadIdx.x];
        if (col < p.N) partial[(((int64_t)blockIdx.z * 2 + i) * p.M + m0 + m) * p.N + col] = s;
      }
    }
}

__global__ void __launch_bounds__(kThreads)
few_sum_kernel(const FewArgs p, const float *partial, int parts) {
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x, m = blockIdx.y;
  if (n >= p.N) return;
  float s[2] = {0.0f, 0.0f};
  for (int z = 0; z < parts; ++z)
#pragma unroll
    for (int i = 0; i < 2; ++i) s[i] += partial[(((int64_t)z * 2 + i) * p.M + m) * p.N + n];
  finish(p, m, n, s[0], s[1]);
}

// c_i(r, n) = sum over the tokens of q_i(m, r) x_i(m, n): 32 rows x 1024
// columns a block, four columns a thread.
template <int MT, bool VEC>
__global__ void __launch_bounds__(kThreads) few_outer_kernel(const OuterArgs p) {
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  __shared__ float q[MT][32];
  const int i = blockIdx.z;
  const int64_t across = (p.N + 1023) / 1024;
  const int64_t r0 = blockIdx.x / across * 32, n = blockIdx.x % across * 1024 + threadIdx.x * 4;
  for (int e = threadIdx.x; e < MT * 32; e += kThreads) {
    const int m = e / 32, r = e % 32;
    q[m][r] = m < p.M && r0 + r < p.R ? p.q[i][m * p.ldq[i] + r0 + r] : 0.0f;
  }
  float4 x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    x[m] = m < p.M ? load4<VEC>(p.x[i] + m * p.ldx[i], n, p.N) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __syncthreads();
  if (n >= p.N) return;
  const int rows = (int)(p.R - r0 < 32 ? p.R - r0 : 32);
  for (int r = 0; r < rows; ++r) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float f = q[m][r];
      s.x = fmaf(f, x[m].x, s.x);
      s.y = fmaf(f, x[m].y, s.y);
      s.z = fmaf(f, x[m].z, s.z);
      s.w = fmaf(f, x[m].w, s.w);
    }
    float *c = p.c[i] + (r0 + r) * p.ldc[i] + n;
    if (VEC && n + 4 <= p.N) {
      *reinterpret_cast<float4 *>(c) = s;
    } else {
      const float v[4] = {s.x, s.y, s.z, s.w};
      for (int k = 0; k < 4 && n + k < p.N; ++k) c[k] = v[k];
    }
  }
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kern)(Params...), dim3 grid, cudaStream_t s, const Args &...args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(kThreads);
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kern, Params(args)...);
}

bool aligned16(const float *p, int64_t ld) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * 4)) & 15) == 0;
}

// Parts of K of few_cols_kernel: two blocks for each SM, of no less than 64 of K.
int parts_of(int64_t N, int64_t K, int64_t tokens_y, int sms) {
  const int64_t blocks = ceil_div(N, 128) * tokens_y;
  int64_t parts = ceil_div(2 * sms, blocks);
  if (parts > ceil_div(K, 64)) parts = ceil_div(K, 64);
  return (int)(parts < 1 ? 1 : parts > 64 ? 64 : parts);
}

int tokens_of(int64_t M) { return M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : 8; }

template <int MT, bool VEC>
cudaError_t run_few(const FewArgs &p, void *ws, int sms, cudaStream_t s) {
  const unsigned ty = (unsigned)ceil_div(p.M, MT);
  if (p.rows_are_outputs) {
    // warps enough for every SM's 16, by sharing rows among up to a block's
    int split = 1;
    while (split < kWarps && ceil_div(p.N, 2) * split * ty < (int64_t)sms * 16) split *= 2;
    return launch(few_rows_kernel<MT, VEC>,
                  dim3((unsigned)ceil_div(p.N, 2 * (kWarps / split)), ty), s, p, split);
  }
  const int parts = parts_of(p.N, p.K, ty, sms);
  float *partial = static_cast<float *>(ws);
  const cudaError_t e = launch(few_cols_kernel<MT, VEC>,
                               dim3((unsigned)ceil_div(p.N, 128), ty, (unsigned)parts), s, p, partial);
  if (e != cudaSuccess) return e;
  return launch(few_sum_kernel, dim3((unsigned)ceil_div(p.N, kThreads), (unsigned)p.M), s, p,
                (const float *)partial, parts);
}

template <int MT>
cudaError_t pick_few(const FewArgs &p, void *ws, int sms, cudaStream_t s) {
  const bool vec = aligned16(p.a[0], p.M > 1 ? p.lda : 0) && aligned16(p.a[1], p.M > 1 ? p.lda : 0) &&
                   aligned16(p.b[0], p.ldb[0]) && aligned16(p.b[1], p.ldb[1]);
  return vec ? run_few<MT, true>(p, ws, sms, s) : run_few<MT, false>(p, ws, sms, s);
}

}  // namespace

uint64_t few_bytes(int64_t M, int64_t N, int64_t K, bool rows_are_outputs, int sms) {
  if (rows_are_outputs) return 0;
  return (uint64_t)parts_of(N, K, ceil_div(M, tokens_of(M)), sms) * 2 * M * N * 4;
}

cudaError_t launch_few(const FewArgs &p, void *ws, int sms, cudaStream_t s) {
  switch (tokens_of(p.M)) {
    case 1: return pick_few<1>(p, ws, sms, s);
    case 2: return pick_few<2>(p, ws, sms, s);
    case 4: return pick_few<4>(p, ws, sms, s);
    default: return pick_few<8>(p, ws, sms, s);
  }
}

cudaError_t launch_outer(const OuterArgs &p, cudaStream_t s) {
  bool vec = true;
  for (int i = 0; i < 2; ++i)
    vec = vec && aligned16(p.x[i], p.M > 1 ? p.ldx[i] : 0) && aligned16(p.c[i], p.R > 1 ? p.ldc[i] : 0);
  const dim3 grid((unsigned)(ceil_div(p.N, 1024) * ceil_div(p.R, 32)), 1, 2);
  if (p.M <= 4)
    return vec ? launch(few_outer_kernel<4, true>, grid, s, p)
               : launch(few_outer_kernel<4, false>, grid, s, p);
  return vec ? launch(few_outer_kernel<kFewTokens, true>, grid, s, p)
             : launch(few_outer_kernel<kFewTokens, false>, grid, s, p);
}

}  // namespace gg
