// Passes around the feed-forward products: operands that TMA cannot read (or
// FP32 ones) laid out as BF16 planes, and the gradients of the gate.  Both are
// bound by HBM: eight values a thread, 16-byte loads and stores wherever rows
// allow.  Gate's gradients of 8192 x 11008 in BF16 on GB300, 14 bytes a value:
// 190 us, 6.6 TB/s.
#include "ff_tc.cuh"
#include "tc_common.cuh"

namespace gg {
namespace {

// x as three BF16 values, each the nearest to what is left; x_0 of a finite x
// is kept finite (nearest would round the largest ones up to Inf), so that
// their sum is x exactly while 2^-133, the least BF16, is under its last bit.
// A non-finite x keeps its first plane and leaves zeros.
__device__ __forceinline__ void split3(float x, bf16 (&o)[3]) {
  bf16 h = __float2bfloat16_rn(x);
  const bool fin = (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u;
  if (fin && (__bfloat16_as_ushort(h) & 0x7f80u) == 0x7f80u) h = __float2bfloat16_rz(x);
  const float r = fin ? x - __bfloat162float(h) : 0.0f;
  const bf16 m = __float2bfloat16_rn(r);
  o[0] = h;
  o[1] = m;
  o[2] = __float2bfloat16_rn(r - __bfloat162float(m));
}

template <int P>
__device__ __forceinline__ void store_planes(const float (&v)[8], bf16 *dst, int64_t plane) {
  __align__(16) bf16 o[P][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (P == 3) {
      bf16 t[3];
      split3(v[i], t);
#pragma unroll
      for (int q = 0; q < 3; ++q) o[q][i] = t[q];
    } else {
      o[0][i] = __float2bfloat16_rn(v[i]);
    }
  }
#pragma unroll
  for (int q = 0; q < P; ++q)
    *reinterpret_cast<uint4 *>(dst + q * plane) = *reinterpret_cast<const uint4 *>(o[q]);
}

// Eight values of one row, rounded to P planes, as one 16-byte store each; as
// they are with P = 0 (dst then holds floats).
template <int P>
__device__ __forceinline__ void store8(const float (&v)[8], bf16 *dst, int64_t plane) {
  if constexpr (P == 0) {
    float4 *to = reinterpret_cast<float4 *>(dst);
    to[0] = make_float4(v[0], v[1], v[2], v[3]);
    to[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    store_planes<P>(v, dst, plane);
  }
}

// Eight values from column c on (zeros from `cols` on), 16 bytes at a time
// where every row starts on a 16-byte boundary (vec).
template <typename T>
__device__ __forceinline__ void load8(const T *row, int64_t c, int64_t cols, bool vec,
                                      float (&v)[8]) {
  if (vec && c + 8 <= cols) {
    __align__(16) T t[8];
#pragma unroll
    for (int i = 0; i < 8; i += 16 / sizeof(T))
      *reinterpret_cast<uint4 *>(t + i) = __ldg(reinterpret_cast<const uint4 *>(row + c + i));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_f32(row[c + i]) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ bool rows_aligned(const T *p, int64_t ld) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * (int64_t)sizeof(T))) & 15) == 0;
}

struct PackJobs {
  PackJob j[kPackJobs];
  int64_t first[kPackJobs + 1];  // each job's first group of eight
  int n;
};

// Group e of eight values of the jobs.
template <typename T, int P>
__device__ __forceinline__ void pack_group(const PackJobs &jobs, int64_t e) {
  int k = 0;
  while (e >= jobs.first[k + 1]) ++k;
  const PackJob &j = jobs.j[k];
  const int64_t per_row = j.ld_out / 8, at = e - jobs.first[k];
  const int64_t r = at / per_row, c = (at - r * per_row) * 8;
  const T *src = static_cast<const T *>(j.src);
  float v[8];
  load8(src + r * j.ld, c, j.cols, rows_aligned(src, j.ld), v);
  store8<P>(v, j.dst + r * j.ld_out + c, j.plane);
}

template <typename T, int P>
__global__ void __launch_bounds__(256) ff_pack_kernel(PackJobs jobs) {
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  for (int64_t e = blockIdx.x * 256ll + threadIdx.x; e < jobs.first[jobs.n];
       e += gridDim.x * 256ll)
    pack_group<T, P>(jobs, e);
}

struct GateAndPack {
  DgateArgs gate;
  PackJobs jobs;
};

// The gradients of the gate, and behind them the backward pass's packing,
// which needs nothing of them: one launch, no tail between the two.
// In BF16, dG and dU are rounded to BF16 here: the tensor core takes factors of
// that type, and each further plane of them would cost the backward products
// once more (8192 x 4096 x 11008: 1.9 ms).  The gradients are then 2.35e-3 off
// where rounding them alone makes 1.66e-3.
template <typename T, int P>
__global__ void __launch_bounds__(256) ff_dgate_kernel(GateAndPack q) {
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  const DgateArgs &p = q.gate;
  const int64_t per_row = p.ld_out / 8, n = p.M * per_row, all = n + q.jobs.first[q.jobs.n];
  const T *dh = static_cast<const T *>(p.dh);
  const bool vh = rows_aligned(dh, p.lddh), vg = rows_aligned(p.g, p.ldg),
             vu = rows_aligned(p.u, p.ldu);
  for (int64_t e = blockIdx.x * 256ll + threadIdx.x; e < all; e += gridDim.x * 256ll) {
    if constexpr (P > 0) {
      if (e >= n) {
        pack_group<T, P>(q.jobs, e - n);
        continue;
      }
    }
    const int64_t r = e / per_row, c = (e - r * per_row) * 8;
    float h[8], g[8], u[8], a[8], d[8];
    load8(dh + r * p.lddh, c, p.F, vh, h);
    load8(p.g + r * p.ldg, c, p.F, vg, g);
    load8(p.u + r * p.ldu, c, p.F, vu, u);
    with_act(p.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < 8; ++i) act_both<T, decltype(act)::value>(g[i], a[i], d[i]);
    });
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[i] = h[i] * u[i] * d[i];
      a[i] = h[i] * a[i];
    }
    const int64_t to = (r * p.ld_out + c) * (P == 0 ? 2 : 1);  // in bf16
    store8<P>(d, p.dg + to, p.plane);
    store8<P>(a, p.du + to, p.plane);
  }
}

// Launched with programmatic dependent launch: scheduled while the kernel
// before it drains, for which every thread of it waits first.
template <typename Args>
cudaError_t launch(void (*kern)(Args), int grid, const Args &p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3(256);
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kern, p);
}

int blocks_for(int64_t groups, int sms) {
  const int64_t b = ceil_div(groups, 256), most = (int64_t)sms * 16;
  return (int)(b < most ? b : most);
}

PackJobs listed(const PackJob *jobs, int n) {
  PackJobs p{};
  for (int k = 0; k < n; ++k) {
    p.j[p.n] = jobs[k];
    p.first[p.n + 1] = p.first[p.n] + jobs[k].rows * (jobs[k].ld_out / 8);
    ++p.n;
  }
  return p;
}

}  // namespace

cudaError_t launch_pack(const PackJob *jobs, int n, int dtype, int sms, cudaStream_t s) {
  const PackJobs p = listed(jobs, n);
  if (p.n == 0) return cudaSuccess;
  const int grid = blocks_for(p.first[p.n], sms);
  if (dtype == GEMM_DT_F32) return launch(ff_pack_kernel<float, 3>, grid, p, s);
  return launch(ff_pack_kernel<bf16, 1>, grid, p, s);
}

cudaError_t launch_dgate_f32(const DgateArgs &p, int sms, cudaStream_t s) {
  const GateAndPack q{p, PackJobs{}};
  return launch(ff_dgate_kernel<float, 0>, blocks_for(p.M * (p.ld_out / 8), sms), q, s);
}

cudaError_t launch_dgate(const DgateArgs &p, const PackJob *jobs, int n, int dtype, int sms,
                         cudaStream_t s) {
  const GateAndPack q{p, listed(jobs, n)};
  const int grid = blocks_for(p.M * (p.ld_out / 8) + q.jobs.first[q.jobs.n], sms);
  if (dtype == GEMM_DT_F32) return launch(ff_dgate_kernel<float, 3>, grid, q, s);
  return launch(ff_dgate_kernel<bf16, 1>, grid, q, s);
}

}  // namespace gg
