// Gated linear recurrence for gfx950: forward over a sequence, backward, and
// the one-token step.  Per channel, with rho = sigmoid(r), iota = sigmoid(i):
//   a = exp(log_decay rho), beta = sqrt(1 - a^2),
//   h_t = a h_{t-1} + beta iota x_t.

#include "layer_internal.h"
#include "ssm_device.h"

namespace ssm {

// Carry waits that hit their bound.
__device__ unsigned g_gated_timeouts;

// rho, iota, a and beta of one step.  1 - a^2 cancels where a is close to 1
// (long memory), so with y = log_decay rho it is m (2 - m), m = -expm1(y): for
// |y| < 1/4 by the series to y^6 (truncation below 5e-8 relative) and
// a = 1 - m, elsewhere from a = exp(y), losing at most ~3e-7 relative.  lam2 =
// log_decay log2(e), so y2 = y log2(e) is the hardware exp's argument and the
// series' coefficients are -ln(2)^k / k!.
__device__ __forceinline__ void gate(float r, float lam2, float& rho, float& a, float& beta) {
  rho = sigmoid_f32(r);
  const float y2 = lam2 * rho;
  const float e = exp2_hw(y2);
  float p = -1.5403530e-4f;
  p = fmaf(p, y2, -1.3333558e-3f);
  p = fmaf(p, y2, -9.6181291e-3f);
  p = fmaf(p, y2, -5.5504109e-2f);
  p = fmaf(p, y2, -2.4022651e-1f);
  p = fmaf(p, y2, -6.9314718e-1f);
  const bool series = fabsf(y2) < 0.36067376f;
  const float m = series ? p * y2 : 1.0f - e;
  a = series ? 1.0f - m : e;
  beta = __builtin_amdgcn_sqrtf(fmaxf(m * (2.0f - m), 0.0f));
}

template <typename T>
__global__ __launch_bounds__(64) void gated_fwd_kernel(GatedArgs p) {
  const int64_t g = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  const int64_t D = p.dim, L = p.seqlen;
  if (g >= p.batch * D) return;
  const int64_t b = g / D, c = g - b * D;
  const T* x = static_cast<const T*>(p.x) + b * L * p.ld_x + c;
  const T* r = static_cast<const T*>(p.r) + b * L * p.ld_r + c;
  const T* in = static_cast<const T*>(p.i) + b * L * p.ld_i + c;
  T* out = p.out ? static_cast<T*>(p.out) + b * L * D + c : nullptr;
  const float lam2 = p.log_decay[c] * kLog2e;
  float h = p.h0 ? p.h0[g] : 0.0f;
  for (int64_t t = 0; t < L; ++t) {
    if (p.ckpt && t % kGatedRun == 0)
      p.ckpt[(b * div_up64(L, kGatedRun) + t / kGatedRun) * D + c] = h;
    float rho, a, beta;
    gate(to_f32(r[t * p.ld_r]), lam2, rho, a, beta);
    const float ix = sigmoid_f32(to_f32(in[t * p.ld_i])) * to_f32(x[t * p.ld_x]);
    h = (p.reset && p.reset[b * L + t]) ? ix : fmaf(a, h, beta * ix);
    if (out) store_act(out, t * D, h);
  }
  if (p.last_state) p.last_state[g] = h;
}

// part: [batch][dim] dlog_decay of each batch row
template <typename T>
__global__ __launch_bounds__(64) void gated_bwd_kernel(GatedArgs p, float* part) {
  const int64_t g = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  const int64_t D = p.dim, L = p.seqlen;
  if (g >= p.batch * D) return;
  const int64_t b = g / D, c = g - b * D;
  const T* x = static_cast<const T*>(p.x) + b * L * p.ld_x + c;
  const T* r = static_cast<const T*>(p.r) + b * L * p.ld_r + c;
  const T* in = static_cast<const T*>(p.i) + b * L * p.ld_i + c;
  const T* dout = static_cast<const T*>(p.dout) + b * L * D + c;
  T* dx = static_cast<T*>(p.dx) + b * L * D + c;
  T* dr = static_cast<T*>(p.dr) + b * L * D + c;
  T* di = static_cast<T*>(p.di) + b * L * D + c;
  const float lam = p.log_decay[c], lam2 = lam * kLog2e;
  float carry = p.dlast ? p.dlast[g] : 0.0f;
  float dlam = 0.0f;
  const int64_t runs = div_up64(L, kGatedRun);
  for (int64_t q = runs - 1; q >= 0; --q) {
    const int64_t t0 = q * kGatedRun;
    const int n = static_cast<int>(L - t0 < kGatedRun ? L - t0 : kGatedRun);
    float h = p.ckpt[(b * runs + q) * D + c];
    float before[kGatedRun];
    for (int j = 0; j < n; ++j) {
      const int64_t t = t0 + j;
      float rho, a, beta;
      gate(to_f32(r[t * p.ld_r]), lam2, rho, a, beta);
      const float ix = sigmoid_f32(to_f32(in[t * p.ld_i])) * to_f32(x[t * p.ld_x]);
      before[j] = h;
      h = (p.reset && p.reset[b * L + t]) ? ix : fmaf(a, h, beta * ix);
    }
    for (int j = n - 1; j >= 0; --j) {
      const int64_t t = t0 + j;
      float rho, a, beta;
      gate(to_f32(r[t * p.ld_r]), lam2, rho, a, beta);
      const float iota = sigmoid_f32(to_f32(in[t * p.ld_i])), xt = to_f32(x[t * p.ld_x]);
      const bool cut = p.reset && p.reset[b * L + t];
      const float gt = to_f32(dout[t * D]) + carry;
      carry = cut ? 0.0f : a * gt;
      const float bt = cut ? 1.0f : beta;
      const float dxt = gt * bt * iota;
      const float inv = beta > 0.0f ? rcp_hw(beta) : 0.0f;
      const float da = cut ? 0.0f : carry * before[j] - (a * a * inv) * (gt * iota * xt);
      const float dlr = da * rho;
      store_act(dx, t * D, dxt);
      store_act(di, t * D, dxt * xt * (1.0f - iota));
      store_act(dr, t * D, dlr * lam * (1.0f - rho));
      dlam += dlr;
    }
  }
  if (p.dh0) p.dh0[g] = carry;
  part[g] = dlam;
}

__global__ __launch_bounds__(64) void gated_sum_kernel(const float* part, int64_t rows, int64_t dim,
                                                       float* out) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (c >= dim) return;
  float s = 0.0f;
  for (int64_t q = 0; q < rows; ++q) s += part[q * dim + c];
  out[c] = s;
}

template <typename T>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedArgs p) {
  const int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (g >= p.batch * p.dim) return;
  const int64_t b = g / p.dim, c = g - b * p.dim;
  float rho, a, beta;
  gate(to_f32(static_cast<const T*>(p.r)[b * p.ld_r + c]), p.log_decay[c] * kLog2e, rho, a, beta);
  const float ix = sigmoid_f32(to_f32(static_cast<const T*>(p.i)[b * p.ld_i + c])) *
                   to_f32(static_cast<const T*>(p.x)[b * p.ld_x + c]);
  const float h = fmaf(a, p.state[g], beta * ix);
  p.state[g] = h;
  store_act(static_cast<T*>(p.out), g, h);
}

int64_t gated_fwd_work(int, int64_t, int64_t, int64_t) { return 0; }
int64_t gated_bwd_work(int, int64_t batch, int64_t, int64_t dim) { return batch * dim * 4; }

static unsigned blocks_of(int64_t n, int64_t per) {
  return static_cast<unsigned>(div_up64(n, per));
}

hipError_t launch_gated_fwd(const GatedArgs& a, hipStream_t stream) {
  const unsigned grid = blocks_of(a.batch * a.dim, 64);
  if (a.dtype == 0)
    gated_fwd_kernel<float><<<grid, 64, 0, stream>>>(a);
  else
    gated_fwd_kernel<bf16_t><<<grid, 64, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedArgs& a, hipStream_t stream) {
  const unsigned grid = blocks_of(a.batch * a.dim, 64);
  float* part = static_cast<float*>(a.work);
  if (a.dtype == 0)
    gated_bwd_kernel<float><<<grid, 64, 0, stream>>>(a, part);
  else
    gated_bwd_kernel<bf16_t><<<grid, 64, 0, stream>>>(a, part);
  gated_sum_kernel<<<blocks_of(a.dim, 64), 64, 0, stream>>>(part, a.batch, a.dim, a.dlog_decay);
  return hipGetLastError();
}

hipError_t launch_gated_step(const GatedArgs& a, hipStream_t stream) {
  const unsigned grid = blocks_of(a.batch * a.dim, 256);
  if (a.dtype == 0)
    gated_step_kernel<float><<<grid, 256, 0, stream>>>(a);
  else
    gated_step_kernel<bf16_t><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t read_and_clear_gated_errors(hipStream_t stream, unsigned* count) {
  hipError_t e = hipStreamSynchronize(stream);
  if (e != hipSuccess) return e;
  e = hipMemcpyFromSymbol(count, HIP_SYMBOL(g_gated_timeouts), sizeof(unsigned), 0,
                          hipMemcpyDeviceToHost);
  if (e != hipSuccess) return e;
  const unsigned zero = 0;
  return hipMemcpyToSymbol(HIP_SYMBOL(g_gated_timeouts), &zero, sizeof(unsigned), 0,
                           hipMemcpyHostToDevice);
}

}  // namespace ssm
