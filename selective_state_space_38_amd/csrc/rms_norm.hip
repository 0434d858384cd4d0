// Root-mean-square norm of a row with the residual's addition, its output in
// the activation type or in 8 bits with a scale for every 128 values, and its
// backward, for gfx950.
//
// All of it streams: a row is read once into registers, reduced there, and
// written once.  A row belongs to LANES threads, which hold its runs of 8 values
// l, l + LANES, ... (16 bytes of bfloat16 each): 16 lanes up to 256 values, a
// wave up to some 3000 (neither needs LDS or a barrier), the four waves of a
// workgroup beyond.  A group of 128 values is 16 neighbouring lanes' runs, one DPP row.
// Short rows, such as a head's, by 16 lanes: 200000 x 64 float32 values 32 us
// against 51 a wave each, backward 34 against 72.  A wave walks rows a
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

// Sum over the LANES threads that share a row, in every thread.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  if constexpr (LANES == 16) return row16_sum(v);
  v = wave_sum(v);
  if constexpr (LANES == 256) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    __syncthreads();
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ double row_sum(double v, float*) {
  static_assert(LANES == 16, "short rows only");
#pragma unroll
  for (int d = 8; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

struct None {};  // no residual

// S: the residual's type, or None.  NORM = false: y = x (8-bit output only).
template <typename T, typename S, bool FP8, bool NORM, int NV, int LANES, bool TAIL>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormArgs p) {
  constexpr bool kRes = !std::is_same<S, None>::value;
  using R = typename std::conditional<kRes, S, T>::type;
  __shared__ float lds[4];
  const RowRuns<LANES, TAIL> q(p.dim);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (256 / LANES);
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
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
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
    float rstd = 1.0f;
    if constexpr (NORM)
      rstd = 1.0f / sqrtf(row_sum<LANES>(ss, lds) / static_cast<float>(p.dim) + p.eps);
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
        // q = 448 y / max |y| needs rstd only where the floor decides, or may (the
        // row holds next to nothing, or an infinity, which makes rstd 0): times a
        // small or large rms instead, the floor would underflow or overflow
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
        m = row16_max(q.on(i) ? m : 0.0f);
        const float top = NORM ? m * rstd : m;
        const float most = fmaxf(top, kFp8AmaxFloor);
        const bool plain = m > kFp8AmaxFloor && top >= kFp8AmaxFloor;
        const Fp8Scaler to(NORM && plain ? m : most, NORM && !plain ? rstd : 1.0f);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = to(y[e]);
        const int r = i * LANES + q.lane;
        if (q.on(i))
          *reinterpret_cast<uint2*>(p.q + base + r * 8) =
              make_uint2(pack_fp8x4(y[0], y[1], y[2], y[3]), pack_fp8x4(y[4], y[5], y[6], y[7]));
        if (q.on(i) && (q.lane & 15) == 0) p.scale[(r >> 4) * p.rows + row] = most / kFp8Max;
      }
    }
  }
}

// Backward: ds = rstd (w dy - s rstd^2 mean(w dy s)) + dres.  Every thread keeps
// its rows' sum of dy s rstd in registers; a workgroup's sums meet in LDS and
// leave as one row of part [workgroups][dim], which a second kernel adds up.
//
// F: the row's sums and ds in double where there are few columns, since the two
// terms of ds then all but cancel (with one column they leave eps / s^2 of
// themselves).
template <typename T, typename S, typename F, int NV, int LANES, bool TAIL>
__global__ __launch_bounds__(256) void norm_bwd_rows_kernel(NormArgs p, float* part) {
  __shared__ float lds[4];
  __shared__ float s_dw[LANES <= 64 ? 64 * NV * 8 : 1];
  const RowRuns<LANES, TAIL> q(p.dim);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (256 / LANES);
  const F inv_dim = F(1) / static_cast<F>(p.dim);
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
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
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
    F ss = 0, dot = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      F a = 0, b = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const F v = q.get(s[i], i, e);
        a = fma(v, v, a);
        b = fma(static_cast<F>(dy[i].get(e)) * static_cast<F>(w[i][e]), v, b);
      }
      ss += q.on(i) ? a : F(0);
      dot += q.on(i) ? b : F(0);
    }
    ss = row_sum<LANES>(ss, lds);
    dot = row_sum<LANES>(dot, lds);
    const F rstd = F(1) / sqrt(ss * inv_dim + static_cast<F>(p.eps));
    const F k = rstd * rstd * (dot * inv_dim);
    const float rstd32 = static_cast<float>(rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float g[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const F v = s[i].get(e), d = dy[i].get(e);
        dw[i][e] = fmaf(static_cast<float>(d), static_cast<float>(v) * rstd32, dw[i][e]);
        F t = rstd * fma(-v, k, d * static_cast<F>(w[i][e]));
        if (p.dres) t += static_cast<F>(dres[i].get(e));
        g[e] = static_cast<float>(t);
      }
      if (q.on(i)) store8(static_cast<S*>(p.ds) + base + q.at(i), g, q.last_of(i));
    }
  }
  if constexpr (LANES == 16) {  // the wave's four rows at a time
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[i][e] += __shfl_xor(dw[i][e], 16, 64);
        dw[i][e] += __shfl_xor(dw[i][e], 32, 64);
      }
  }
  if constexpr (LANES <= 64) {
    for (int k = 0; k < 4; ++k) {
      if (threadIdx.x >> 6 == static_cast<unsigned>(k)) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* t = &s_dw[(e * NV + i) * 64 + (threadIdx.x & 63)];
            dw[i][e] = k ? *t + dw[i][e] : dw[i][e];
            *t = dw[i][e];
          }
      }
      __syncthreads();
    }
    if (threadIdx.x < 256 - LANES) return;  // the last wave holds the sums
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (q.on(i)) store8(part + blockIdx.x * p.dim + q.at(i), dw[i], q.last_of(i));
}

// ---- host ----

// Backward rows shorter than this are summed in double.
constexpr int64_t kFewColumns = 64;

static unsigned count(int64_t n, int64_t per, int64_t most) {
  const int64_t k = div_up64(n, per);
  return static_cast<unsigned>(k < most ? k : most);
}

// NV runs of 8 a thread, LANES threads a row; MOST: the longest rows, in runs, of
// a wave.  Forward 448: 16384 rows of 2688 values 98 us against 103 by four waves,
// but 8192 of 4096 81 against 76.  Backward, with twice the registers, 320: 16384
// of 2688 127 us by a wave against 116, 8192 of 4096 100 against 91.
#define SSM_NORM_BY_SIZE(LAUNCH, MOST)           \
  do {                                           \
    const int64_t runs = div_up64(a.dim, 8);     \
    if (runs <= 16) LAUNCH(1, 16);               \
    else if (runs <= 32) LAUNCH(2, 16);          \
    else if (runs <= 64) LAUNCH(1, 64);          \
    else if (runs <= 128) LAUNCH(2, 64);         \
    else if (runs <= 192) LAUNCH(3, 64);         \
    else if (runs <= 320) LAUNCH(5, 64);         \
    else if (runs <= MOST) LAUNCH(MOST / 64, 64); \
    else if (runs <= 512) LAUNCH(2, 256);        \
    else if (runs <= 768) LAUNCH(3, 256);        \
    else if (runs <= 1024) LAUNCH(4, 256);       \
    else LAUNCH(8, 256);                         \
  } while (0)

template <typename T, typename S, bool FP8, bool NORM, bool TAIL>
static void launch_rows_cut(const NormArgs& a, hipStream_t stream) {
#define SSM_LAUNCH(NV, LANES)                                                               \
  norm_rows_kernel<T, S, FP8, NORM, NV, LANES, TAIL>                                        \
      <<<count(a.rows, 256 / LANES, 256 * 8), 256, 0, stream>>>(a)
  SSM_NORM_BY_SIZE(SSM_LAUNCH, 448);
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

int64_t norm_bwd_work(int64_t rows, int64_t dim) {
  return (rows < kBwdGroups ? rows : kBwdGroups) * dim * 4;
}

template <typename T, typename S, bool TAIL>
static unsigned launch_bwd_rows_cut(const NormArgs& a, float* part, hipStream_t stream) {
  unsigned grid = 0;
#define SSM_LAUNCH_AS(F, NV, LANES)                                                     \
  (grid = count(a.rows, 256 / LANES, kBwdGroups),                                       \
   norm_bwd_rows_kernel<T, S, F, NV, LANES, TAIL><<<grid, 256, 0, stream>>>(a, part))
#define SSM_LAUNCH(NV, LANES) SSM_LAUNCH_AS(float, NV, LANES)
  if (a.dim < kFewColumns)
    SSM_LAUNCH_AS(double, 1, 16);
  else
    SSM_NORM_BY_SIZE(SSM_LAUNCH, 320);
#undef SSM_LAUNCH_AS
#undef SSM_LAUNCH
  return grid;
}

template <typename T, typename S>
static unsigned launch_bwd_rows(const NormArgs& a, float* part, hipStream_t stream) {
  return a.dim % 8 ? launch_bwd_rows_cut<T, S, true>(a, part, stream)
                   : launch_bwd_rows_cut<T, S, false>(a, part, stream);
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t stream) {
  float* part = static_cast<float*>(a.work);
  unsigned rows;
  if (a.dtype == 0)
    rows = a.residual_dtype == 0 ? launch_bwd_rows<float, float>(a, part, stream)
                                 : launch_bwd_rows<float, bf16_t>(a, part, stream);
  else
    rows = a.residual_dtype == 0 ? launch_bwd_rows<bf16_t, float>(a, part, stream)
                                 : launch_bwd_rows<bf16_t, bf16_t>(a, part, stream);
  launch_column_sum(part, rows, a.dim, a.dweight, stream);
  return hipGetLastError();
}

}  // namespace ssm
