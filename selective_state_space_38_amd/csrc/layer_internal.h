// Launch interfaces between the residual layer's entry points (layer_api.hip)
// and their kernels.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

constexpr int64_t div_up64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Steps between two of the gated recurrence's checkpoints.
constexpr int kGatedRun = 16;
// Inputs that share an 8-bit scale.
constexpr int kFp8Group = 128;
constexpr float kFp8Max = 448.0f;                                // largest e4m3 value
constexpr float kFp8AmaxFloor = 7.888609052210118e-31f;          // 2^-100

struct GatedArgs {
  int dtype;
  int64_t batch, seqlen, dim, ld_x, ld_r, ld_i;
  const void *x, *r, *i;
  const float* log_decay;
  const uint8_t* reset;     // nullable
  const float* h0;          // nullable
  // forward
  void* out;                // nullable with ckpt
  float* last_state;        // nullable
  float* ckpt;              // forward: written (nullable); backward: read
  // backward
  const void* dout;
  const float* dlast;       // nullable
  void *dx, *dr, *di;
  float* dlog_decay;
  float* dh0;               // nullable
  // decode
  float* state;
  void* work;
  int spin_limit;           // bound on each carry wait
};

int64_t gated_fwd_work(int dtype, int64_t batch, int64_t seqlen, int64_t dim);
int64_t gated_bwd_work(int dtype, int64_t batch, int64_t seqlen, int64_t dim);
hipError_t launch_gated_fwd(const GatedArgs& a, hipStream_t stream);
hipError_t launch_gated_bwd(const GatedArgs& a, hipStream_t stream);
hipError_t launch_gated_step(const GatedArgs& a, hipStream_t stream);
// Reads and clears the count of carry waits that timed out (synchronises).
hipError_t read_and_clear_gated_errors(hipStream_t stream, unsigned* count);

// out[c] = sum over rows of part[row][c], in one fixed order.
void launch_column_sum(const float* part, int64_t rows, int64_t dim, float* out,
                       hipStream_t stream);

struct NormArgs {
  int dtype, residual_dtype;
  int64_t rows, dim;
  const void* x;            // backward: unused
  const void* residual;     // nullable
  const float* weight;
  float eps;
  void* y;
  uint8_t* q;
  float* scale;
  void* residual_out;
  const void* dy;
  const void* s;
  const void* dres;         // nullable
  void* ds;
  float* dweight;
  void* work;
};

int64_t norm_bwd_work(int64_t rows, int64_t dim);
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t stream);
// norm: y = rms norm of x + residual; otherwise y = x
hipError_t launch_norm_fp8(const NormArgs& a, bool norm, hipStream_t stream);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t stream);

struct LinearArgs {
  int dtype;
  int64_t rows, n, k;
  const uint8_t* xq;
  const float* x_scale;
  const uint8_t* wq;
  const float* w_scale;
  const float* bias;        // nullable
  void* out;
  void* work;
};

int64_t fp8_linear_work(int dtype, int64_t rows, int64_t n, int64_t k);
hipError_t launch_fp8_linear(const LinearArgs& a, hipStream_t stream);
hipError_t launch_quantize_weight(const void* w, int dtype, int64_t n, int64_t k, uint8_t* q,
                                  float* scale, hipStream_t stream);

}  // namespace ssm
