// Root-mean-square norm of a row with the residual's addition, its output in
// the activation type or in 8 bits with a scale for every 128 values, and its
// backward, for gfx950.
//
// All of it streams: a row is read once into registers, reduced there, and
// written once.  Rows of up to 4096 values belong to one wave (no LDS, no
// barrier: lane l holds the runs of 8 values l, l + 64, ..., 16 bytes of
// bfloat16 each), longer ones to the four waves of a workgroup.  A group of 128
// values is then 16 neighbouring lanes' runs, one DPP row.  A wave walks rows a
// grid apart with the weights in registers.  32768 rows of 2560 bfloat16 values:
// with a float32 residual and 8-bit output 176 us, the training pair 258 us,
// 5.2 TB/s each, the rate of a large copy.

#include "layer_device.h"

namespace ssm {

// A row's runs of 8 values as a thread holds them: run i LANES + lane for i < NV.
// TAIL: the row's length is no multiple of 8 and its last run is shorter.
template <int LANES, bool TAIL>
struct RowRuns {
  int lane, runs, last;  // last: index of the last run's last value
  __device__ __forceinline__ RowRuns(int64_t dim)
      : lane(threadIdx.x % LANES),
        runs(static_cast<int>((dim + 7) / 8)),
        last(TAIL ? static_cast<int>((dim - 1) % 8) : 7) {}
  __device__ __forceinline__ bool on(int i) const { return i * LANES + lane < runs; }
  // values of run i, at p + at(i); a thread past the row repeats its last run
  __device__ __forceinline__ int at(int i) const {
    const int r = i * LANES + lane;
    return (r < runs ? r : runs - 1) * 8;
  }
  __device__ __forceinline__ bool cut(int i) const {
    return TAIL && i * LANES + lane >= runs - 1;
  }
  __device__ __forceinline__ int last_of(int i) const { return cut(i) ? last : 7; }
  template <typename T>
  __device__ __forceinline__ void load(const T* row, int i, Run8<T>& r) const {
    if (cut(i))
      r.load_elems(row + at(i), last);
    else
      r.load(row + at(i));
  }
  // r's value e, zero past the row's end
  template <typename T>
  __device__ __forceinline__ float get(const Run8<T>& r, int i, int e) const {
    return TAIL && e > last_of(i) ? 0.0f : r.get(e);
  }
};

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
template <typename T, typename S, bool FP8, bool NORM, int NV, int WPR, bool TAIL>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormArgs p) {
  constexpr bool kRes = !std::is_same<S, None>::value;
  using R = typename std::conditional<kRes, S, T>::type;
  __shared__ float lds[4];
  constexpr int LANES = 64 * WPR;
  const RowRuns<LANES, TAIL> q(p.dim);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (4 / WPR);
  float w[NV][8];
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Run8<float> t;
      q.load(p.weight, i, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = t.get(e);
    }
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (4 / WPR) + threadIdx.x / LANES;
       row < p.rows; row += step) {
    const int64_t base = row * p.dim;
    Run8<T> x[NV];
    Run8<R> res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      q.load(static_cast<const T*>(p.x) + base, i, x[i]);
      if constexpr (kRes) q.load(static_cast<const R*>(p.residual) + base, i, res[i]);
    }
    float s[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float part = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[i][e] = q.get(x[i], i, e);
        if constexpr (kRes) s[i][e] += q.get(res[i], i, e);
        part = fmaf(s[i][e], s[i][e], part);
      }
      ss += q.on(i) ? part : 0.0f;
      if constexpr (kRes)
        if (q.on(i)) store8(static_cast<R*>(p.residual_out) + base + q.at(i), s[i], q.last_of(i));
    }
    float rms = 1.0f, rstd = 1.0f;
    if constexpr (NORM) {
      const float var = row_sum<WPR>(ss, lds) / static_cast<float>(p.dim) + p.eps;
      rms = sqrtf(var);
      rstd = 1.0f / rms;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = NORM ? s[i][e] * w[i][e] : s[i][e];
      if constexpr (!FP8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= rstd;
        if (q.on(i)) store8(static_cast<T*>(p.y) + base + q.at(i), y, q.last_of(i));
      } else {
        // q = 448 y / max |y| does not need rstd; the scale does
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
        m = fmaxf(row16_max(q.on(i) ? m : 0.0f), kFp8AmaxFloor * rms);
        const Fp8Scaler to(m);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = to(y[e]);
        const int r = i * LANES + q.lane;
        if (q.on(i))
          *reinterpret_cast<uint2*>(p.q + base + r * 8) =
              make_uint2(pack_fp8x4(y[0], y[1], y[2], y[3]), pack_fp8x4(y[4], y[5], y[6], y[7]));
        if (q.on(i) && (q.lane & 15) == 0) p.scale[(r >> 4) * p.rows + row] = m * rstd / kFp8Max;
      }
    }
  }
}

// Backward: ds = rstd (w dy - s rstd^2 mean(w dy s)) + dres.  Every wave keeps
// its rows' sum of dy s rstd in registers; a workgroup's four sums meet in LDS
// and leave as one row of part [workgroups][dim], which a second kernel adds up.
template <typename T, typename S, int NV, int WPR, bool TAIL>
__global__ __launch_bounds__(256) void norm_bwd_rows_kernel(NormArgs p, float* part) {
  __shared__ float lds[4];
  __shared__ float s_dw[WPR == 1 ? 64 * NV * 8 : 1];
  constexpr int LANES = 64 * WPR;
  const RowRuns<LANES, TAIL> q(p.dim);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (4 / WPR);
  const float inv_dim = 1.0f / static_cast<float>(p.dim);
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    Run8<float> t;
    q.load(p.weight, i, t);
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
      q.load(static_cast<const S*>(p.s) + base, i, s[i]);
      q.load(static_cast<const T*>(p.dy) + base, i, dy[i]);
      if (p.dres) q.load(static_cast<const S*>(p.dres) + base, i, dres[i]);
    }
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a = 0.0f, b = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = q.get(s[i], i, e);
        a = fmaf(v, v, a);
        b = fmaf(dy[i].get(e) * w[i][e], v, b);
      }
      ss += q.on(i) ? a : 0.0f;
      dot += q.on(i) ? b : 0.0f;
    }
    ss = row_sum<WPR>(ss, lds);
    dot = row_sum<WPR>(dot, lds);
    const float rstd = 1.0f / sqrtf(ss * inv_dim + p.eps);
    const float k = rstd * rstd * (dot * inv_dim);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float g[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = s[i].get(e), d = dy[i].get(e);
        dw[i][e] = fmaf(d, v * rstd, dw[i][e]);
        g[e] = rstd * fmaf(-v, k, d * w[i][e]);
        if (p.dres) g[e] += dres[i].get(e);
      }
      if (q.on(i)) store8(static_cast<S*>(p.ds) + base + q.at(i), g, q.last_of(i));
    }
  }
  if constexpr (WPR == 1) {
    for (int k = 0; k < 4; ++k) {
      if (threadIdx.x >> 6 == static_cast<unsigned>(k)) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* t = &s_dw[(e * NV + i) * 64 + q.lane];
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
    if (q.on(i)) store8(part + blockIdx.x * p.dim + q.at(i), dw[i], q.last_of(i));
}

// ---- backward of few columns: a workgroup per row, element by element ----

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

// In 64 bits: with few columns the two terms of ds all but cancel (with one
// column they leave eps / s^2 of themselves).
__global__ __launch_bounds__(256) void norm_bwd_few_kernel(NormArgs p, float* rstds) {
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
__global__ __launch_bounds__(256) void norm_dweight_few_kernel(NormArgs p, const float* rstds,
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

// Backward rows shorter than this go through the kernels for few columns.
constexpr int64_t kFewColumns = 64;

static unsigned count(int64_t n, int64_t per, int64_t most) {
  const int64_t k = div_up64(n, per);
  return static_cast<unsigned>(k < most ? k : most);
}

// One wave per row up to 4096 values, four beyond; NV runs of 8 per lane.
#define SSM_NORM_BY_SIZE(LAUNCH)                 \
  do {                                           \
    const int64_t runs = div_up64(a.dim, 8);     \
    if (runs <= 64) LAUNCH(1, 1);                \
    else if (runs <= 128) LAUNCH(2, 1);          \
    else if (runs <= 192) LAUNCH(3, 1);          \
    else if (runs <= 320) LAUNCH(5, 1);          \
    else if (runs <= 512) LAUNCH(8, 1);          \
    else if (runs <= 768) LAUNCH(3, 4);          \
    else if (runs <= 1024) LAUNCH(4, 4);         \
    else LAUNCH(8, 4);                           \
  } while (0)

template <typename T, typename S, bool FP8, bool NORM, bool TAIL>
static void launch_rows_cut(const NormArgs& a, hipStream_t stream) {
#define SSM_LAUNCH(NV, WPR)                                                                 \
  norm_rows_kernel<T, S, FP8, NORM, NV, WPR, TAIL>                                          \
      <<<count(a.rows, 4 / WPR, 256 * 8), 256, 0, stream>>>(a)
  SSM_NORM_BY_SIZE(SSM_LAUNCH);
#undef SSM_LAUNCH
}

template <typename T, typename S, bool FP8, bool NORM>
static void launch_rows(const NormArgs& a, hipStream_t stream) {
  if constexpr (!FP8) {  // 8-bit rows are whole runs of 16 values
    if (a.dim % 8) return launch_rows_cut<T, S, FP8, NORM, true>(a, stream);
  }
  launch_rows_cut<T, S, FP8, NORM, false>(a, stream);
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
  launch_rows_typed<false>(a, stream);
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

template <typename T, typename S, bool TAIL>
static unsigned launch_bwd_rows_cut(const NormArgs& a, float* part, hipStream_t stream) {
  unsigned grid = 0;
#define SSM_LAUNCH(NV, WPR)                                                         \
  (grid = count(a.rows, 4 / WPR, kBwdGroups),                                       \
   norm_bwd_rows_kernel<T, S, NV, WPR, TAIL><<<grid, 256, 0, stream>>>(a, part))
  SSM_NORM_BY_SIZE(SSM_LAUNCH);
#undef SSM_LAUNCH
  return grid;
}

template <typename T, typename S>
static unsigned launch_bwd_rows(const NormArgs& a, float* part, hipStream_t stream) {
  return a.dim % 8 ? launch_bwd_rows_cut<T, S, true>(a, part, stream)
                   : launch_bwd_rows_cut<T, S, false>(a, part, stream);
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t stream) {
  float* work = static_cast<float*>(a.work);
  if (a.dim >= kFewColumns) {
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
    norm_bwd_few_kernel<<<static_cast<unsigned>(a.rows), 256, 0, stream>>>(a, work);
    norm_dweight_few_kernel<<<dim3(count(a.dim, 64, a.dim), slabs), 256, 0, stream>>>(a, work, part);
    launch_column_sum(part, slabs, a.dim, a.dweight, stream);
  }
  return hipGetLastError();
}

}  // namespace ssm
