// Root-mean-square norm of a row with the residual's addition, its output in
// the activation type or in 8 bits with a scale for every 128 values, and its
// backward, for gfx950.
//
// All of it streams: a row is read once into registers, reduced there, and
// written once.  Rows of up to 4096 values belong to one wave (no LDS, no
// barrier: lane l holds the runs of 8 values l, l + 64, ..., 16 bytes of
// bfloat16 each), longer ones to the four waves of a workgroup.  A group of 128
// values is then 16 neighbouring lanes' runs, one DPP row.  A wave walks rows a
// grid apart with the weights in registers.  Rows whose length is no multiple
// of 8, or that are not 16-byte aligned, take the plain kernels at the end: a
// workgroup per row, element by element.

#include "layer_device.h"

namespace ssm {

// 8 consecutive values of a row as stored.
template <typename T>
using Run8 = Run<T, 8>;

template <typename T>
__device__ __forceinline__ void put8(void* p, int64_t i, const float (&v)[8]) {
  store_run<T, 8>(static_cast<T*>(p) + i, v, true, 7);
}

// Sum over the WPR waves that share a row, in every thread.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  v = wave_sum(v);
  if constexpr (WPR == 1) {
    return v;
  } else {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    __syncthreads();
    return v;
  }
}

struct None {};  // no residual

// S: the residual's type, or None.  NORM = false: y = x (8-bit output only).
template <typename T, typename S, bool FP8, bool NORM, int NV, int WPR>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormArgs p) {
  constexpr bool kRes = !std::is_same<S, None>::value;
  using RS = Run8<typename std::conditional<kRes, S, T>::type>;
  __shared__ float lds[4];
  constexpr int LANES = 64 * WPR;
  const int lane = threadIdx.x % LANES;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (4 / WPR);
  const int runs = static_cast<int>(p.dim / 8);
  float w[NV][8];
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Run8<float> t;
      const int r = i * LANES + lane;
      t.load_vec(p.weight + (r < runs ? r : runs - 1) * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = t.get(e);
    }
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (4 / WPR) + threadIdx.x / LANES;
       row < p.rows; row += step) {
    const int64_t base = row * p.dim;
    Run8<T> x[NV];
    RS res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int r = i * LANES + lane;
      const int64_t at = base + (r < runs ? r : runs - 1) * 8;
      x[i].load_vec(static_cast<const T*>(p.x) + at);
      if constexpr (kRes) res[i].load_vec(static_cast<const S*>(p.residual) + at);
    }
    float s[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool on = i * LANES + lane < runs;
      float part = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[i][e] = x[i].get(e);
        if constexpr (kRes) s[i][e] += res[i].get(e);
        part = fmaf(s[i][e], s[i][e], part);
      }
      ss += on ? part : 0.0f;
      if constexpr (kRes)
        if (on) put8<S>(p.residual_out, base + (i * LANES + lane) * 8, s[i]);
    }
    float rms = 1.0f, rstd = 1.0f;
    if constexpr (NORM) {
      const float var = row_sum<WPR>(ss, lds) / static_cast<float>(p.dim) + p.eps;
      rms = sqrtf(var);
      rstd = 1.0f / rms;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int r = i * LANES + lane;
      const bool on = r < runs;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = NORM ? s[i][e] * w[i][e] : s[i][e];
      if constexpr (!FP8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= rstd;
        if (on) put8<T>(p.y, base + r * 8, y);
      } else {
        // q = 448 y / max |y| does not need rstd; the scale does
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
        m = fmaxf(row16_max(on ? m : 0.0f), kFp8AmaxFloor * rms);
        const Fp8Scaler to(m);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = to(y[e]);
        if (on)
          *reinterpret_cast<uint2*>(p.q + base + r * 8) =
              make_uint2(pack_fp8x4(y[0], y[1], y[2], y[3]), pack_fp8x4(y[4], y[5], y[6], y[7]));
        if (on && (lane & 15) == 0) p.scale[(r >> 4) * p.rows + row] = m * rstd / kFp8Max;
      }
    }
  }
}

// Backward: ds = rstd (w dy - s rstd^2 mean(w dy s)) + dres.  Every wave keeps
// its rows' sum of dy s rstd in registers; a workgroup's four sums meet in LDS
// and leave as one row of part [workgroups][dim], which a second kernel adds up.
template <typename T, typename S, int NV, int WPR>
__global__ __launch_bounds__(256) void norm_bwd_rows_kernel(NormArgs p, float* part) {
  __shared__ float lds[4];
  __shared__ float s_dw[WPR == 1 ? 64 * NV * 8 : 1];
  constexpr int LANES = 64 * WPR;
  const int lane = threadIdx.x % LANES;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (4 / WPR);
  const int runs = static_cast<int>(p.dim / 8);
  const float inv_dim = 1.0f / static_cast<float>(p.dim);
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    Run8<float> t;
    const int r = i * LANES + lane;
    t.load_vec(p.weight + (r < runs ? r : runs - 1) * 8);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[i][e] = t.get(e);
      dw[i][e] = 0.0f;
    }
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (4 / WPR) + threadIdx.x / LANES;
       row < p.rows; row += step) {
    const int64_t base = row * p.dim;
    Run8<S> s[NV], dres[NV];
    Run8<T> dy[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int r = i * LANES + lane;
      const int64_t at = base + (r < runs ? r : runs - 1) * 8;
      s[i].load_vec(static_cast<const S*>(p.s) + at);
      dy[i].load_vec(static_cast<const T*>(p.dy) + at);
      if (p.dres) dres[i].load_vec(static_cast<const S*>(p.dres) + at);
    }
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool on = i * LANES + lane < runs;
      float a = 0.0f, b = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = s[i].get(e);
        a = fmaf(v, v, a);
        b = fmaf(dy[i].get(e) * w[i][e], v, b);
      }
      ss += on ? a : 0.0f;
      dot += on ? b : 0.0f;
    }
    ss = row_sum<WPR>(ss, lds);
    dot = row_sum<WPR>(dot, lds);
    const float rstd = 1.0f / sqrtf(ss * inv_dim + p.eps);
    const float k = rstd * rstd * (dot * inv_dim);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int r = i * LANES + lane;
      float g[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = s[i].get(e), d = dy[i].get(e);
        dw[i][e] = fmaf(d, v * rstd, dw[i][e]);
        g[e] = rstd * fmaf(-v, k, d * w[i][e]);
        if (p.dres) g[e] += dres[i].get(e);
      }
      if (r < runs) put8<S>(p.ds, base + r * 8, g);
    }
  }
  float* out = part + static_cast<int64_t>(blockIdx.x) * p.dim;
  if constexpr (WPR == 1) {
    for (int k = 0; k < 4; ++k) {
      if (threadIdx.x >> 6 == static_cast<unsigned>(k)) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* t = &s_dw[(e * NV + i) * 64 + lane];
            dw[i][e] = k ? *t + dw[i][e] : dw[i][e];
            *t = dw[i][e];
          }
      }
      __syncthreads();
    }
    if (threadIdx.x < 192) return;  // the last wave holds the sums
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i * LANES + lane < runs) put8<float>(out, (i * LANES + lane) * 8, dw[i]);
}

// ---- any row length and alignment: a workgroup per row ----

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

__global__ __launch_bounds__(256) void norm_any_kernel(NormArgs p) {
  __shared__ float lds[4];
  const int64_t row = blockIdx.x, base = row * p.dim;
  const int dim = static_cast<int>(p.dim);
  float ss = 0.0f;
  for (int c = threadIdx.x; c < dim; c += 256) {
    float v = load_as(p.x, p.dtype, base + c);
    if (p.residual) v += load_as(p.residual, p.residual_dtype, base + c);
    ss = fmaf(v, v, ss);
  }
  ss = block_sum(ss, lds);
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(dim) + p.eps);
  for (int c = threadIdx.x; c < dim; c += 256) {
    float v = load_as(p.x, p.dtype, base + c);
    if (p.residual) {
      v += load_as(p.residual, p.residual_dtype, base + c);
      store_as(p.residual_out, p.residual_dtype, base + c, v);
    }
    store_as(p.y, p.dtype, base + c, v * rstd * p.weight[c]);
  }
}

// In 64 bits: with few columns the two terms of ds all but cancel (with one
// column they leave eps / s^2 of themselves).
__global__ __launch_bounds__(256) void norm_bwd_any_kernel(NormArgs p, float* rstds) {
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

// dweight of a slab of rows: part[slab][c], 4 waves taking every 4th row.
constexpr int kSlab = 256;
__global__ __launch_bounds__(256) void norm_dweight_any_kernel(NormArgs p, const float* rstds,
                                                               float* part) {
  __shared__ float lds[4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kSlab;
  const int64_t r1 = r0 + kSlab < p.rows ? r0 + kSlab : p.rows;
  float sum = 0.0f;
  if (c < p.dim)
    for (int64_t row = r0 + w; row < r1; row += 4)
      sum = fmaf(load_as(p.dy, p.dtype, row * p.dim + c),
                 load_as(p.s, p.residual_dtype, row * p.dim + c) * rstds[row], sum);
  lds[w][lane] = sum;
  __syncthreads();
  if (w == 0 && c < p.dim)
    part[blockIdx.y * p.dim + c] = (lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane]);
}

// ---- host ----

static bool whole_runs(const NormArgs& a) {
  if (a.dim % 8) return false;
  for (const void* q : {a.x, a.residual, static_cast<const void*>(a.weight),
                        static_cast<const void*>(a.y), static_cast<const void*>(a.residual_out),
                        a.dy, a.s, a.dres, static_cast<const void*>(a.ds)})
    if (reinterpret_cast<uintptr_t>(q) & 15) return false;
  return true;
}

static unsigned count(int64_t n, int64_t per, int64_t most) {
  const int64_t k = div_up64(n, per);
  return static_cast<unsigned>(k < most ? k : most);
}

// One wave per row up to 4096 values, four beyond; NV runs of 8 per lane.
#define SSM_NORM_BY_SIZE(LAUNCH)                 \
  do {                                           \
    const int64_t runs = a.dim / 8;              \
    if (runs <= 64) LAUNCH(1, 1);                \
    else if (runs <= 128) LAUNCH(2, 1);          \
    else if (runs <= 192) LAUNCH(3, 1);          \
    else if (runs <= 320) LAUNCH(5, 1);          \
    else if (runs <= 512) LAUNCH(8, 1);          \
    else if (runs <= 768) LAUNCH(3, 4);          \
    else if (runs <= 1024) LAUNCH(4, 4);         \
    else LAUNCH(8, 4);                           \
  } while (0)

template <typename T, typename S, bool FP8, bool NORM>
static void launch_rows(const NormArgs& a, hipStream_t stream) {
#define SSM_LAUNCH(NV, WPR)                                                                 \
  norm_rows_kernel<T, S, FP8, NORM, NV, WPR>                                                \
      <<<count(a.rows, 4 / WPR, 256 * 8), 256, 0, stream>>>(a)
  SSM_NORM_BY_SIZE(SSM_LAUNCH);
#undef SSM_LAUNCH
}

template <bool FP8>
static void launch_rows_typed(const NormArgs& a, hipStream_t stream) {
  if (a.dtype == 0) {
    if (!a.residual) launch_rows<float, None, FP8, true>(a, stream);
    else if (a.residual_dtype == 0) launch_rows<float, float, FP8, true>(a, stream);
    else launch_rows<float, bf16_t, FP8, true>(a, stream);
  } else {
    if (!a.residual) launch_rows<bf16_t, None, FP8, true>(a, stream);
    else if (a.residual_dtype == 0) launch_rows<bf16_t, float, FP8, true>(a, stream);
    else launch_rows<bf16_t, bf16_t, FP8, true>(a, stream);
  }
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t stream) {
  if (whole_runs(a))
    launch_rows_typed<false>(a, stream);
  else
    norm_any_kernel<<<static_cast<unsigned>(a.rows), 256, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_norm_fp8(const NormArgs& a, bool norm, hipStream_t stream) {
  if (norm) launch_rows_typed<true>(a, stream);
  else if (a.dtype == 0) launch_rows<float, None, true, false>(a, stream);
  else launch_rows<bf16_t, None, true, false>(a, stream);
  return hipGetLastError();
}

constexpr int64_t kBwdGroups = 512;  // workgroups of the backward, two per CU

int64_t norm_bwd_work(int, int, int64_t rows, int64_t dim) {
  const int64_t slabs = div_up64(rows, kSlab), groups = rows < kBwdGroups ? rows : kBwdGroups;
  const int64_t any = div_up64(rows, 4) * 16 + slabs * dim * 4;
  return any > groups * dim * 4 ? any : groups * dim * 4;
}

template <typename T, typename S>
static unsigned launch_bwd_rows(const NormArgs& a, float* part, hipStream_t stream) {
  unsigned grid = 0;
#define SSM_LAUNCH(NV, WPR)                                                   \
  (grid = count(a.rows, 4 / WPR, kBwdGroups),                                 \
   norm_bwd_rows_kernel<T, S, NV, WPR><<<grid, 256, 0, stream>>>(a, part))
  SSM_NORM_BY_SIZE(SSM_LAUNCH);
#undef SSM_LAUNCH
  return grid;
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t stream) {
  float* work = static_cast<float*>(a.work);
  if (whole_runs(a)) {
    unsigned rows;
    if (a.dtype == 0)
      rows = a.residual_dtype == 0 ? launch_bwd_rows<float, float>(a, work, stream)
                                   : launch_bwd_rows<float, bf16_t>(a, work, stream);
    else
      rows = a.residual_dtype == 0 ? launch_bwd_rows<bf16_t, float>(a, work, stream)
                                   : launch_bwd_rows<bf16_t, bf16_t>(a, work, stream);
    launch_column_sum(work, rows, a.dim, a.dweight, stream);
  } else {
    float* part = work + div_up64(a.rows, 4) * 4;
    const unsigned slabs = count(a.rows, kSlab, a.rows);
    norm_bwd_any_kernel<<<static_cast<unsigned>(a.rows), 256, 0, stream>>>(a, work);
    norm_dweight_any_kernel<<<dim3(count(a.dim, 64, a.dim), slabs), 256, 0, stream>>>(a, work, part);
    launch_column_sum(part, slabs, a.dim, a.dweight, stream);
  }
  return hipGetLastError();
}

}  // namespace ssm
