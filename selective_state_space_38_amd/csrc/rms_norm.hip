// Root-mean-square norm of a row with the residual's addition, its output in
// the activation type or in 8 bits with a scale for every 128 values, and its
// backward, for gfx950.

#include "layer_internal.h"
#include "ssm_device.h"

namespace ssm {

__device__ __forceinline__ float load_as(const void* p, int dtype, int64_t i) {
  return dtype == 0 ? static_cast<const float*>(p)[i] : to_f32(static_cast<const bf16_t*>(p)[i]);
}
__device__ __forceinline__ void store_as(void* p, int dtype, int64_t i, float v) {
  if (dtype == 0)
    static_cast<float*>(p)[i] = v;
  else
    store_act(static_cast<bf16_t*>(p), i, v);
}

// Sum over a workgroup of four waves, returned in every thread.
template <typename F>
__device__ __forceinline__ F block_sum(F v, F* lds) {
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  __syncthreads();
  return v;
}

// One workgroup per row.
template <bool FP8, bool NORM>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs p) {
  __shared__ float lds[4];
  const int64_t row = blockIdx.x, base = row * p.dim;
  const int dim = static_cast<int>(p.dim);
  float ss = 0.0f;
  if (NORM) {
    for (int c = threadIdx.x; c < dim; c += 256) {
      float v = load_as(p.x, p.dtype, base + c);
      if (p.residual) v += load_as(p.residual, p.residual_dtype, base + c);
      ss = fmaf(v, v, ss);
    }
    ss = block_sum(ss, lds);
  }
  const float rstd = NORM ? 1.0f / sqrtf(ss / static_cast<float>(dim) + p.eps) : 1.0f;
  // 256 columns (two groups of 128) at a time, whole for every thread
  for (int c0 = 0; c0 < dim; c0 += 256) {
    const int c = c0 + threadIdx.x;
    float v = 0.0f;
    if (c < dim) {
      v = load_as(p.x, p.dtype, base + c);
      if (NORM && p.residual) {
        v += load_as(p.residual, p.residual_dtype, base + c);
        store_as(p.residual_out, p.residual_dtype, base + c, v);
      }
      if (NORM) v = v * rstd * p.weight[c];
      if (!FP8) store_as(p.y, p.dtype, base + c, v);
    }
    if (FP8) {
      float m = fabsf(v);
      for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
      __syncthreads();
      if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
      __syncthreads();
      const int pair = (threadIdx.x >> 7) * 2;
      m = fmaxf(fmaxf(lds[pair], lds[pair + 1]), kFp8AmaxFloor);
      if (c < dim) {
        const int q = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_ratio(v, m), 0.0f, 0, false);
        p.q[base + c] = static_cast<uint8_t>(q);
        if (c % kFp8Group == 0) p.scale[(c / kFp8Group) * p.rows + row] = m / kFp8Max;
      }
    }
  }
}

// In 64 bits: with few columns the two terms of ds all but cancel (with one
// column they leave eps / s^2 of themselves).
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormArgs p, float* rstds) {
  __shared__ double lds[4];
  const int64_t row = blockIdx.x, base = row * p.dim;
  const int dim = static_cast<int>(p.dim);
  double ss = 0.0, dot = 0.0;
  for (int c = threadIdx.x; c < dim; c += 256) {
    const double v = load_as(p.s, p.residual_dtype, base + c);
    ss = fma(v, v, ss);
    dot = fma(static_cast<double>(load_as(p.dy, p.dtype, base + c)) * p.weight[c], v, dot);
  }
  ss = block_sum(ss, lds);
  dot = block_sum(dot, lds);
  const double var = ss / dim + p.eps;
  const double rstd = 1.0 / sqrt(var);
  const double k = dot / (dim * var);
  for (int c = threadIdx.x; c < dim; c += 256) {
    const double v = load_as(p.s, p.residual_dtype, base + c);
    double g = rstd * (static_cast<double>(load_as(p.dy, p.dtype, base + c)) * p.weight[c] - v * k);
    if (p.dres) g += load_as(p.dres, p.residual_dtype, base + c);
    store_as(p.ds, p.residual_dtype, base + c, static_cast<float>(g));
  }
  if (threadIdx.x == 0) rstds[row] = static_cast<float>(rstd);
}

__global__ __launch_bounds__(64) void norm_dweight_kernel(NormArgs p, const float* rstds) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (c >= p.dim) return;
  float sum = 0.0f;
  for (int64_t row = 0; row < p.rows; ++row)
    sum += load_as(p.dy, p.dtype, row * p.dim + c) *
           load_as(p.s, p.residual_dtype, row * p.dim + c) * rstds[row];
  p.dweight[c] = sum;
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t stream) {
  norm_fwd_kernel<false, true><<<static_cast<unsigned>(a.rows), 256, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_norm_fp8(const NormArgs& a, bool norm, hipStream_t stream) {
  if (norm)
    norm_fwd_kernel<true, true><<<static_cast<unsigned>(a.rows), 256, 0, stream>>>(a);
  else
    norm_fwd_kernel<true, false><<<static_cast<unsigned>(a.rows), 256, 0, stream>>>(a);
  return hipGetLastError();
}

int64_t norm_bwd_work(int, int, int64_t rows, int64_t) { return rows * 4; }

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t stream) {
  float* rstds = static_cast<float*>(a.work);
  norm_bwd_kernel<<<static_cast<unsigned>(a.rows), 256, 0, stream>>>(a, rstds);
  norm_dweight_kernel<<<static_cast<unsigned>(div_up64(a.dim, 64)), 64, 0, stream>>>(a, rstds);
  return hipGetLastError();
}

}  // namespace ssm
