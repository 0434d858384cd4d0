// C ABI of the residual layer's operators: validation and dispatch.  The
// operations are documented in ssm_scan.h.

#include <stdint.h>
#include <stdlib.h>

#include <hip/hip_runtime.h>

#include "../../include/ssm_scan.h"
#include "layer_internal.h"

namespace {

constexpr int kDefaultSpinLimit = 1 << 24;
constexpr int64_t kMaxNormDim = 16384;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_dtype(int32_t t) { return t == SSM_F32 || t == SSM_BF16; }
uintptr_t elem(int32_t t) { return t == SSM_BF16 ? 2 : 4; }

// SSM_EINVAL if an output is an input or another output (nulls aside).

template <int NI, int NO>
int check_alias(const void* const (&ins)[NI], const void* const (&outs)[NO]) {
  for (int o = 0; o < NO; ++o) {
    if (!outs[o]) continue;
    for (int i = 0; i < NI; ++i)
      if (ins[i] == outs[o]) return SSM_EINVAL;
    for (int q = 0; q < o; ++q)
      if (outs[q] == outs[o]) return SSM_EINVAL;
  }
  return SSM_OK;
}

template <int N>
int check_aligned(const void* const (&ptrs)[N], uintptr_t a) {
  for (const void* p : ptrs)
    if (p && !aligned(p, a)) return SSM_EALIGN;
  return SSM_OK;
}

int check_gated(const gated_dims* d) {
  if (!d) return SSM_EINVAL;
  if (!valid_dtype(d->dtype)) return SSM_EDTYPE;
  if (d->batch <= 0 || d->seqlen <= 0 || d->dim <= 0) return SSM_EINVAL;
  // the limits of the launch arithmetic: 32-bit channel offsets within a row,
  // 31-bit work item counts (a piece is at least 16 steps of 64 channels)
  if (d->dim > (1LL << 24) || d->seqlen > (1LL << 31) - 1024 || d->batch > (1LL << 24))
    return SSM_EINVAL;
  if (d->batch * ssm::div_up64(d->dim, 64) > (1LL << 30)) return SSM_EINVAL;
  if (d->batch * ssm::div_up64(d->dim, 64) * ssm::div_up64(d->seqlen, ssm::kGatedRun) >
      (1LL << 31) - 1)
    return SSM_EINVAL;
  for (int64_t ld : {d->ld_x, d->ld_r, d->ld_i})
    if (ld < d->dim || ld > (1LL << 26)) return SSM_EINVAL;
  return SSM_OK;
}

int64_t up16(int64_t bytes) { return ssm::div_up64(bytes, 16) * 16; }

int spin_limit() {
  const char* v = getenv("SSM_TEST_SPIN_LIMIT");
  if (!v || !*v) return kDefaultSpinLimit;
  char* end = nullptr;
  const long x = strtol(v, &end, 10);
  return (end && *end == '\0') ? static_cast<int>(x) : kDefaultSpinLimit;
}

ssm::GatedArgs gated_args(const void* x, const void* r, const void* i, const float* log_decay,
                          const gated_dims* d) {
  ssm::GatedArgs a = {};
  a.dtype = d->dtype;
  a.batch = d->batch;
  a.seqlen = d->seqlen;
  a.dim = d->dim;
  a.ld_x = d->ld_x;
  a.ld_r = d->ld_r;
  a.ld_i = d->ld_i;
  a.x = x;
  a.r = r;
  a.i = i;
  a.log_decay = log_decay;
  a.spin_limit = spin_limit();
  return a;
}

int64_t ckpt_bytes(const gated_dims* d) {
  return d->batch * ssm::div_up64(d->seqlen, ssm::kGatedRun) * d->dim * 4;
}

int check_norm(const norm_dims* d) {
  if (!d) return SSM_EINVAL;
  if (!valid_dtype(d->dtype) || !valid_dtype(d->residual_dtype)) return SSM_EDTYPE;
  if (d->rows <= 0 || d->dim <= 0 || d->dim > kMaxNormDim || d->rows > (1LL << 31) - 1)
    return SSM_EINVAL;
  return SSM_OK;
}

int norm_fwd_impl(const void* x, const void* residual, const float* weight, float eps, void* y,
                  uint8_t* q, float* scale, void* residual_out, const norm_dims* dims,
                  bool norm, void* stream) {
  int rc = check_norm(dims);
  if (rc != SSM_OK) return rc;
  const bool fp8 = y == nullptr;
  if (!x || (norm && (!weight || !(eps > 0.0f)))) return SSM_EINVAL;
  if (fp8 ? (!q || !scale || dims->dim % 16) : q != nullptr) return SSM_EINVAL;
  if ((residual != nullptr) != (residual_out != nullptr)) return SSM_EINVAL;
  const void* acts[] = {x, y};
  const void* res[] = {residual, residual_out};
  const void* f32s[] = {weight, scale};
  if ((rc = check_aligned(acts, fp8 ? 16 : elem(dims->dtype))) != SSM_OK) return rc;
  if ((rc = check_aligned(res, fp8 ? 16 : elem(dims->residual_dtype))) != SSM_OK) return rc;
  if ((rc = check_aligned(f32s, 4)) != SSM_OK) return rc;
  if (fp8 && (!aligned(q, 16) || (weight && !aligned(weight, 16)))) return SSM_EALIGN;
  // residual_out may be residual itself: an element is read before it is written
  const void* ins[] = {x, residual == residual_out ? nullptr : residual, weight};
  const void* outs[] = {y, q, scale, residual_out};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::NormArgs a = {};
  a.dtype = dims->dtype;
  a.residual_dtype = residual ? dims->residual_dtype : dims->dtype;
  a.rows = dims->rows;
  a.dim = dims->dim;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.eps = eps;
  a.y = y;
  a.q = q;
  a.scale = scale;
  a.residual_out = residual_out;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t e = fp8 ? ssm::launch_norm_fp8(a, norm, st) : ssm::launch_norm_fwd(a, st);
  return e == hipSuccess ? SSM_OK : SSM_ELAUNCH;
}

int check_linear(const linear_dims* d) {
  if (!d) return SSM_EINVAL;
  if (!valid_dtype(d->dtype)) return SSM_EDTYPE;
  if (d->rows <= 0 || d->n <= 0 || d->k <= 0 || d->k % 16) return SSM_EINVAL;
  // 32-bit limits of the launch arithmetic
  if (d->rows > (1LL << 30) || d->n > (1LL << 24) || d->k > (1LL << 20)) return SSM_EINVAL;
  if (ssm::div_up64(d->rows, 16) * ssm::div_up64(d->n, 16) > (1LL << 31) - 1) return SSM_EINVAL;
  return SSM_OK;
}

}  // namespace

extern "C" {

int64_t gated_scan_work_bytes(const gated_dims* dims) {
  const int rc = check_gated(dims);
  if (rc != SSM_OK) return rc;
  return up16(ssm::gated_fwd_work(dims->dtype, dims->batch, dims->seqlen, dims->dim));
}

int64_t gated_ckpt_bytes(const gated_dims* dims) {
  const int rc = check_gated(dims);
  return rc != SSM_OK ? rc : up16(ckpt_bytes(dims));
}

int gated_scan_fwd(const void* x, const void* r, const void* i, const float* log_decay,
                   const uint8_t* reset, const float* h0, void* out, float* last_state,
                   float* ckpt, void* work, const gated_dims* dims, void* stream) {
  int rc = check_gated(dims);
  if (rc != SSM_OK) return rc;
  if (!x || !r || !i || !log_decay || (!out && !ckpt)) return SSM_EINVAL;
  if (!work && gated_scan_work_bytes(dims) > 0) return SSM_EINVAL;
  const void* acts[] = {x, r, i, out};
  const void* f32s[] = {log_decay, h0, last_state};
  const void* wide[] = {ckpt, work};
  if ((rc = check_aligned(acts, elem(dims->dtype))) != SSM_OK) return rc;
  if ((rc = check_aligned(f32s, 4)) != SSM_OK) return rc;
  if ((rc = check_aligned(wide, 16)) != SSM_OK) return rc;
  const void* ins[] = {x, r, i, log_decay, reset, h0};
  const void* outs[] = {out, last_state, ckpt, work};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::GatedArgs a = gated_args(x, r, i, log_decay, dims);
  a.reset = reset;
  a.h0 = h0;
  a.out = out;
  a.last_state = last_state;
  a.ckpt = ckpt;
  a.work = work;
  return ssm::launch_gated_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                 : SSM_ELAUNCH;
}

int64_t gated_scan_bwd_work_bytes(const gated_dims* dims, int has_ckpt) {
  const int rc = check_gated(dims);
  if (rc != SSM_OK) return rc;
  const int64_t own = up16(ssm::gated_bwd_work(dims->dtype, dims->batch, dims->seqlen, dims->dim));
  // without a checkpoint buffer the call runs the forward for one first
  const int64_t fwd = has_ckpt ? 0 : up16(ckpt_bytes(dims)) + gated_scan_work_bytes(dims);
  return own + fwd;
}

int gated_scan_bwd(const void* x, const void* r, const void* i, const float* log_decay,
                   const uint8_t* reset, const float* h0, const void* dout, const float* dlast,
                   const float* ckpt, void* dx, void* dr, void* di, float* dlog_decay,
                   float* dh0, void* work, const gated_dims* dims, void* stream) {
  int rc = check_gated(dims);
  if (rc != SSM_OK) return rc;
  if (!x || !r || !i || !log_decay || !dout || !dx || !dr || !di || !dlog_decay)
    return SSM_EINVAL;
  if (!work && gated_scan_bwd_work_bytes(dims, ckpt != nullptr) > 0) return SSM_EINVAL;
  const void* acts[] = {x, r, i, dout, dx, dr, di};
  const void* f32s[] = {log_decay, h0, dlast, dlog_decay, dh0};
  const void* wide[] = {ckpt, work};
  if ((rc = check_aligned(acts, elem(dims->dtype))) != SSM_OK) return rc;
  if ((rc = check_aligned(f32s, 4)) != SSM_OK) return rc;
  if ((rc = check_aligned(wide, 16)) != SSM_OK) return rc;
  const void* ins[] = {x, r, i, log_decay, reset, h0, dout, dlast, ckpt};
  const void* outs[] = {dx, dr, di, dlog_decay, dh0, work};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  ssm::GatedArgs a = gated_args(x, r, i, log_decay, dims);
  a.reset = reset;
  a.h0 = h0;
  a.work = work;
  if (!ckpt) {
    char* w = static_cast<char*>(work) +
              up16(ssm::gated_bwd_work(dims->dtype, dims->batch, dims->seqlen, dims->dim));
    ssm::GatedArgs f = a;
    f.ckpt = reinterpret_cast<float*>(w);
    f.work = w + up16(ckpt_bytes(dims));
    if (ssm::launch_gated_fwd(f, st) != hipSuccess) return SSM_ELAUNCH;
    ckpt = f.ckpt;
  }
  a.ckpt = const_cast<float*>(ckpt);  // read only
  a.dout = dout;
  a.dlast = dlast;
  a.dx = dx;
  a.dr = dr;
  a.di = di;
  a.dlog_decay = dlog_decay;
  a.dh0 = dh0;
  return ssm::launch_gated_bwd(a, st) == hipSuccess ? SSM_OK : SSM_ELAUNCH;
}

int gated_state_update(float* state, const void* x, const void* r, const void* i,
                       const float* log_decay, void* out, const gated_dims* dims,
                       void* stream) {
  int rc = check_gated(dims);
  if (rc != SSM_OK) return rc;
  if (dims->seqlen != 1 || !state || !x || !r || !i || !log_decay || !out) return SSM_EINVAL;
  const void* acts[] = {x, r, i, out};
  const void* f32s[] = {state, log_decay};
  if ((rc = check_aligned(acts, elem(dims->dtype))) != SSM_OK) return rc;
  if ((rc = check_aligned(f32s, 4)) != SSM_OK) return rc;
  const void* ins[] = {x, r, i, log_decay};
  const void* outs[] = {out, state};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::GatedArgs a = gated_args(x, r, i, log_decay, dims);
  a.state = state;
  a.out = out;
  return ssm::launch_gated_step(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                  : SSM_ELAUNCH;
}

int gated_check_device_errors(void* stream) {
  unsigned count = 0;
  if (ssm::read_and_clear_gated_errors(static_cast<hipStream_t>(stream), &count) != hipSuccess)
    return SSM_ELAUNCH;
  return count ? SSM_ETIMEOUT : SSM_OK;
}

int rms_norm_fwd(const void* x, const void* residual, const float* weight, float eps, void* y,
                 void* residual_out, const norm_dims* dims, void* stream) {
  if (!y) return SSM_EINVAL;
  return norm_fwd_impl(x, residual, weight, eps, y, nullptr, nullptr, residual_out, dims, true,
                       stream);
}

int rms_norm_fp8(const void* x, const void* residual, const float* weight, float eps, void* q,
                 float* scale, void* residual_out, const norm_dims* dims, void* stream) {
  return norm_fwd_impl(x, residual, weight, eps, nullptr, static_cast<uint8_t*>(q), scale,
                       residual_out, dims, true, stream);
}

int fp8_quantize(const void* x, void* q, float* scale, const norm_dims* dims, void* stream) {
  if (!dims) return SSM_EINVAL;
  norm_dims d = *dims;
  d.residual_dtype = d.dtype;  // no residual
  return norm_fwd_impl(x, nullptr, nullptr, 0.0f, nullptr, static_cast<uint8_t*>(q), scale,
                       nullptr, &d, false, stream);
}

int64_t rms_norm_bwd_work_bytes(const norm_dims* dims) {
  const int rc = check_norm(dims);
  if (rc != SSM_OK) return rc;
  return up16(ssm::norm_bwd_work(dims->rows, dims->dim));
}

int rms_norm_bwd(const void* dy, const void* s, const float* weight, float eps,
                 const void* dres, void* ds, float* dweight, void* work, const norm_dims* dims,
                 void* stream) {
  int rc = check_norm(dims);
  if (rc != SSM_OK) return rc;
  if (!dy || !s || !weight || !ds || !dweight || !(eps > 0.0f)) return SSM_EINVAL;
  if (!work && rms_norm_bwd_work_bytes(dims) > 0) return SSM_EINVAL;
  const void* acts[] = {dy};
  const void* res[] = {s, dres, ds};
  const void* f32s[] = {weight, dweight};
  const void* wide[] = {work};
  if ((rc = check_aligned(acts, elem(dims->dtype))) != SSM_OK) return rc;
  if ((rc = check_aligned(res, elem(dims->residual_dtype))) != SSM_OK) return rc;
  if ((rc = check_aligned(f32s, 4)) != SSM_OK) return rc;
  if ((rc = check_aligned(wide, 16)) != SSM_OK) return rc;
  const void* ins[] = {dy, s, weight, dres};
  const void* outs[] = {ds, dweight, work};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::NormArgs a = {};
  a.dtype = dims->dtype;
  a.residual_dtype = dims->residual_dtype;
  a.rows = dims->rows;
  a.dim = dims->dim;
  a.weight = weight;
  a.eps = eps;
  a.dy = dy;
  a.s = s;
  a.dres = dres;
  a.ds = ds;
  a.dweight = dweight;
  a.work = work;
  return ssm::launch_norm_bwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                : SSM_ELAUNCH;
}

int fp8_quantize_weight(const void* w, int dtype, int64_t n, int64_t k, void* q, float* scale,
                        void* stream) {
  if (!valid_dtype(dtype)) return SSM_EDTYPE;
  if (!w || !q || !scale || n <= 0 || k <= 0 || n > (1LL << 24) || k > (1LL << 20))
    return SSM_EINVAL;
  if (!aligned(w, elem(dtype)) || !aligned(scale, 4)) return SSM_EALIGN;
  const void* ins[] = {w};
  const void* outs[] = {q, scale};
  const int rc = check_alias(ins, outs);
  if (rc != SSM_OK) return rc;
  return ssm::launch_quantize_weight(w, dtype, n, k, static_cast<uint8_t*>(q), scale,
                                     static_cast<hipStream_t>(stream)) == hipSuccess
             ? SSM_OK
             : SSM_ELAUNCH;
}

int64_t fp8_linear_work_bytes(const linear_dims* dims) {
  const int rc = check_linear(dims);
  return rc != SSM_OK ? rc : up16(ssm::fp8_linear_work(dims->dtype, dims->rows, dims->n, dims->k));
}

int fp8_linear(const void* xq, const float* x_scale, const void* wq, const float* w_scale,
               const float* bias, void* out, void* work, const linear_dims* dims,
               void* stream) {
  int rc = check_linear(dims);
  if (rc != SSM_OK) return rc;
  if (!xq || !x_scale || !wq || !w_scale || !out) return SSM_EINVAL;
  if (!work && fp8_linear_work_bytes(dims) > 0) return SSM_EINVAL;
  const void* wide[] = {xq, wq, work};
  const void* f32s[] = {x_scale, w_scale, bias};
  if ((rc = check_aligned(wide, 16)) != SSM_OK) return rc;
  if ((rc = check_aligned(f32s, 4)) != SSM_OK) return rc;
  if (!aligned(out, elem(dims->dtype))) return SSM_EALIGN;
  const void* ins[] = {xq, x_scale, wq, w_scale, bias};
  const void* outs[] = {out, work};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::LinearArgs a = {};
  a.dtype = dims->dtype;
  a.rows = dims->rows;
  a.n = dims->n;
  a.k = dims->k;
  a.xq = static_cast<const uint8_t*>(xq);
  a.x_scale = x_scale;
  a.wq = static_cast<const uint8_t*>(wq);
  a.w_scale = w_scale;
  a.bias = bias;
  a.out = out;
  a.work = work;
  return ssm::launch_fp8_linear(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                  : SSM_ELAUNCH;
}

}  // extern "C"
