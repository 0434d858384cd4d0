// Tokens into the experts' order and back, for gfx950:
//   xs[r] = x[token[r]],  out[t] = residual[t] + sum_j w_tj y[slot_tj],
// and the gradient of the second (the first's is the second without weights).

#include "feed_internal.h"
#include "layer_device.h"

namespace ssm {

// Runs of 8 values.  L lanes hold a row, each every L-th run of it; WHOLE: rows are
// a whole number of runs.  Memory bounds all three, and a wave a row (16 lanes up to 128
// values) keeps eight or more loads of 16 bytes in flight a lane: 32768 tokens' 4 rows each of 2560 bfloat16
// into the order 195 us (168 MB read four times, three of them from the caches, 671 MB written:
// 163 us at a copy's rate), back onto float32 246 to 269 us by card (1.34 GB: 260), gradient of
// 8191 x 2 x 1536 float32 56 (253 MB: 49).

template <typename T, bool WHOLE>
__device__ __forceinline__ void load8(Run8<T>& run, const T* p, int left) {
  if (WHOLE || left >= 8) run.load(p);
  else run.load_elems(p, left - 1);
}

__device__ __forceinline__ void clear(Run8<float>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r.w[i] = 0;
}
__device__ __forceinline__ void clear(Run8<bf16_t>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = 0;
}

// Copies: the values move as stored.
template <typename T>
__device__ __forceinline__ void put8(T* p, const Run8<T>& r, int left) {
  if (left >= 8) {
    u32x4_any* q = reinterpret_cast<u32x4_any*>(p);
#pragma unroll
    for (int i = 0; i < Run<T, 8>::NW / 4; ++i)
      q[i] = u32x4{r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]};
    return;
  }
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < left) {
      if constexpr (sizeof(T) == 4) p[k] = __uint_as_float(r.w[k]);
      else p[k] = static_cast<T>(r.w[k / 2] >> (16 * (k % 2)));
    }
}

constexpr int kOrderThreads = 256;

template <typename T, int L>
__global__ __launch_bounds__(kOrderThreads) void gather_kernel(OrderArgs p) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (kOrderThreads / L) + threadIdx.x / L;
  if (r >= p.rows) return;
  const int at = threadIdx.x & (L - 1);
  const int dim = static_cast<int>(p.dim), runs = (dim + 7) / 8;
  const int64_t t = p.token[r];
  const bool in = t >= 0 && t < p.tokens;
  const T* from = static_cast<const T*>(p.x) + (in ? t : 0) * p.dim;
  T* to = static_cast<T*>(p.xs) + r * p.dim;
  constexpr int U = 8 * 2 / sizeof(T);  // runs in flight
  for (int c0 = at; c0 < runs; c0 += U * L) {
    Run8<T> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * L;
      if (in && c < runs) load8<T, false>(v[u], from + 8 * c, dim - 8 * c);
      else clear(v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * L;
      if (c < runs) put8(to + 8 * c, v[u], dim - 8 * c);
    }
  }
}

// K: topk, rounded up.  A run of all of a token's rows is read before the first is added.
template <typename T, typename R, int L, int K>
__global__ __launch_bounds__(kOrderThreads) void combine_kernel(OrderArgs p) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kOrderThreads / L) + threadIdx.x / L;
  if (t >= p.tokens) return;
  const int at = threadIdx.x & (L - 1);
  const int dim = static_cast<int>(p.dim), runs = (dim + 7) / 8;
  const T* from[K];
  float w[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int64_t r = j < p.topk ? p.slot[t * p.topk + j] : -1;
    const bool in = r >= 0 && r < p.rows;
    w[j] = in && p.weight ? p.weight[t * p.topk + j] : 1.0f;
    from[j] = in ? static_cast<const T*>(p.y) + r * p.dim : nullptr;
  }
  R* to = static_cast<R*>(p.out) + t * p.dim;
  const R* res = p.residual ? static_cast<const R*>(p.residual) + t * p.dim : nullptr;
  for (int c = at; c < runs; c += L) {
    const int left = dim - 8 * c;
    Run8<T> v[K];
    Run8<R> q;
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (from[j]) load8<T, false>(v[j], from[j] + 8 * c, left);
    if (res) load8<R, false>(q, res + 8 * c, left);
    float sum[8] = {};
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (from[j]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = fmaf(w[j], v[j].get(e), sum[e]);
      }
    if (res) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += q.get(e);
    }
    store8(to + 8 * c, sum, left < 8 ? left - 1 : 7);
  }
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L == 64) return wave_sum(v);
  return row16_sum(v);
}

// K: topk, rounded up.  A run of dout is read once for all of a token's rows; the
// dot products stay in registers until the row's end.
template <typename T, typename R, int L, int K>
__global__ __launch_bounds__(kOrderThreads) void combine_bwd_kernel(OrderArgs p) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kOrderThreads / L) + threadIdx.x / L;
  const bool live = t < p.tokens;
  const int at = threadIdx.x & (L - 1);
  const int dim = static_cast<int>(p.dim), runs = live ? (dim + 7) / 8 : 0;
  int64_t row[K];
  float w[K], dot[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    row[j] = live && j < p.topk ? p.slot[t * p.topk + j] : -1;
    if (row[j] >= p.rows) row[j] = -1;
    w[j] = row[j] >= 0 && p.weight ? p.weight[t * p.topk + j] : 1.0f;
    dot[j] = 0.0f;
  }
  const R* dout = static_cast<const R*>(p.dout) + t * p.dim;
  const T* y = static_cast<const T*>(p.y);
  T* dy = static_cast<T*>(p.dy);
  for (int c = at; c < runs; c += L) {
    const int left = dim - 8 * c, last = left < 8 ? left - 1 : 7;
    Run8<R> d;
    Run8<T> v[K];
    load8<R, false>(d, dout + 8 * c, left);
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (p.dweight && row[j] >= 0) load8<T, false>(v[j], y + row[j] * p.dim + 8 * c, left);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (row[j] < 0) continue;
      float g[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = w[j] * d.get(e);
      store8(dy + row[j] * p.dim + 8 * c, g, last);
      if (p.dweight) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dot[j] = fmaf(e <= last ? d.get(e) : 0.0f, e <= last ? v[j].get(e) : 0.0f, dot[j]);
      }
    }
  }
  if (!p.dweight) return;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const float v = lanes_sum<L>(dot[j]);
    if (live && at == 0 && j < p.topk) p.dweight[t * p.topk + j] = v;
  }
}

static unsigned order_grid(int64_t rows, int lanes) {
  return static_cast<unsigned>(div_up64(rows, kOrderThreads / lanes));
}
// Rows of up to 16 runs take 16 lanes.
static bool narrow(int64_t dim) { return dim <= 128; }

template <typename T>
static void launch_gather_typed(const OrderArgs& a, hipStream_t stream) {
  if (narrow(a.dim))
    gather_kernel<T, 16><<<order_grid(a.rows, 16), kOrderThreads, 0, stream>>>(a);
  else
    gather_kernel<T, 64><<<order_grid(a.rows, 64), kOrderThreads, 0, stream>>>(a);
}

template <typename T, typename R, int K>
static void launch_combine_k(const OrderArgs& a, hipStream_t stream) {
  if (narrow(a.dim))
    combine_kernel<T, R, 16, K><<<order_grid(a.tokens, 16), kOrderThreads, 0, stream>>>(a);
  else
    combine_kernel<T, R, 64, K><<<order_grid(a.tokens, 64), kOrderThreads, 0, stream>>>(a);
}

template <typename T, typename R>
static void launch_combine_typed(const OrderArgs& a, hipStream_t stream) {
  if (a.topk <= 1) launch_combine_k<T, R, 1>(a, stream);
  else if (a.topk <= 2) launch_combine_k<T, R, 2>(a, stream);
  else if (a.topk <= 4) launch_combine_k<T, R, 4>(a, stream);
  else if (a.topk <= 8) launch_combine_k<T, R, 8>(a, stream);
  else launch_combine_k<T, R, 16>(a, stream);
}

template <typename T, typename R, int K>
static void launch_combine_bwd_k(const OrderArgs& a, hipStream_t stream) {
  if (narrow(a.dim))
    combine_bwd_kernel<T, R, 16, K><<<order_grid(a.tokens, 16), kOrderThreads, 0, stream>>>(a);
  else
    combine_bwd_kernel<T, R, 64, K><<<order_grid(a.tokens, 64), kOrderThreads, 0, stream>>>(a);
}

template <typename T, typename R>
static void launch_combine_bwd_typed(const OrderArgs& a, hipStream_t stream) {
  if (a.topk <= 1) launch_combine_bwd_k<T, R, 1>(a, stream);
  else if (a.topk <= 2) launch_combine_bwd_k<T, R, 2>(a, stream);
  else if (a.topk <= 4) launch_combine_bwd_k<T, R, 4>(a, stream);
  else if (a.topk <= 8) launch_combine_bwd_k<T, R, 8>(a, stream);
  else launch_combine_bwd_k<T, R, 16>(a, stream);
}

hipError_t launch_gather(const OrderArgs& a, hipStream_t stream) {
  if (a.dtype == 0) launch_gather_typed<float>(a, stream);
  else launch_gather_typed<bf16_t>(a, stream);
  return hipGetLastError();
}

hipError_t launch_combine_fwd(const OrderArgs& a, hipStream_t stream) {
  if (a.dtype == 0) {
    if (a.residual_dtype == 0) launch_combine_typed<float, float>(a, stream);
    else launch_combine_typed<float, bf16_t>(a, stream);
  } else {
    if (a.residual_dtype == 0) launch_combine_typed<bf16_t, float>(a, stream);
    else launch_combine_typed<bf16_t, bf16_t>(a, stream);
  }
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const OrderArgs& a, hipStream_t stream) {
  if (a.dtype == 0) {
    if (a.residual_dtype == 0) launch_combine_bwd_typed<float, float>(a, stream);
    else launch_combine_bwd_typed<float, bf16_t>(a, stream);
  } else {
    if (a.residual_dtype == 0) launch_combine_bwd_typed<bf16_t, float>(a, stream);
    else launch_combine_bwd_typed<bf16_t, bf16_t>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace ssm
