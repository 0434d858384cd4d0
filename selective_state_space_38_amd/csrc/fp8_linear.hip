// Linear product of 8-bit (e4m3) operands with block scales for gfx950:
//   out[m][n] = sum over blocks kb of 128 inputs of
//               xs[kb][m] ws[n/128][kb] sum_{k in kb} xq[m][k] wq[n][k]  (+ bias[n]),
// and the weights' conversion to that form.

#include "layer_internal.h"
#include "ssm_device.h"

namespace ssm {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// 16 x 16 outputs summed over 128 inputs: lane l holds 32 of row l % 16's 128
// bytes of either operand (the same 32 of both), and four results: rows
// 4 (l / 16) .. + 3 of a, column l % 16 of b.
//
// The 8-bit matrix instruction adds its products in a fixed-point window of
// about 13 bits below the largest of them: measured on normal data, a sum is
// off by 1.5e-5 of its magnitude (2e-4 of the terms' at worst).  That is far
// below a bfloat16 output's own rounding, 2e-3, but not a float32's, so with
// EXACT (float32 outputs) the operands are widened to bfloat16, which holds
// every e4m3 value, and summed by the bfloat16 instruction at half the rate.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ bf16x8 widen(int lo, int hi) {
  const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

template <bool EXACT>
__device__ __forceinline__ f32x4 mfma_fp8(i32x8 a, i32x8 b) {
  f32x4 c = {};
  if constexpr (EXACT) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(a[2 * j], a[2 * j + 1]),
                                                  widen(b[2 * j], b[2 * j + 1]), c, 0, 0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
  }
}

// The 32 bytes of a row that a lane holds, zero past the row's end and for
// rows past the operand's.
__device__ __forceinline__ i32x8 load_row(const uint8_t* base, int64_t row, int64_t rows, int64_t k,
                                          int64_t at) {
  i32x8 v = {};
  if (row < rows) {
    const uint8_t* p = base + row * k + at;
    if (at < k) {
      const int4 t = *reinterpret_cast<const int4*>(p);
      v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    }
    if (at + 16 < k) {
      const int4 t = *reinterpret_cast<const int4*>(p + 16);
      v[4] = t.x; v[5] = t.y; v[6] = t.z; v[7] = t.w;
    }
  }
  return v;
}

// One wave per 16 x 16 outputs; the weights are the first operand, so a lane
// holds four consecutive outputs of one token.
template <typename T>
__global__ __launch_bounds__(64) void fp8_linear_kernel(LinearArgs p) {
  const int lane = threadIdx.x, col = lane & 15, quad = lane >> 4;
  const int64_t tiles_n = div_up64(p.n, 16);
  const int64_t n0 = (blockIdx.x % tiles_n) * 16, m = (blockIdx.x / tiles_n) * 16 + col;
  const int64_t groups = div_up64(p.k, kFp8Group);
  f32x4 acc = {};
  for (int64_t g = 0; g < groups; ++g) {
    const int64_t at = g * kFp8Group + quad * 32;
    const f32x4 d = mfma_fp8<sizeof(T) == 4>(load_row(p.wq, n0 + col, p.n, p.k, at),
                                             load_row(p.xq, m, p.rows, p.k, at));
    const float scale = m < p.rows ? p.x_scale[g * p.rows + m] * p.w_scale[n0 / kFp8Group * groups + g]
                                   : 0.0f;
    for (int j = 0; j < 4; ++j) acc[j] = fmaf(d[j], scale, acc[j]);
  }
  if (m >= p.rows) return;
  for (int j = 0; j < 4; ++j) {
    const int64_t n = n0 + quad * 4 + j;
    if (n < p.n) store_act(static_cast<T*>(p.out), m * p.n + n, acc[j] + (p.bias ? p.bias[n] : 0.0f));
  }
}

// One workgroup per tile of 128 x 128 weights.
template <typename T>
__global__ __launch_bounds__(256) void quantize_weight_kernel(const T* w, int64_t n, int64_t k,
                                                              uint8_t* q, float* scale) {
  __shared__ float lds[4];
  const int64_t groups = div_up64(k, kFp8Group);
  const int64_t tn = blockIdx.x / groups, tk = blockIdx.x % groups;
  const int64_t r0 = tn * kFp8Group, c = tk * kFp8Group + (threadIdx.x & 127);
  const int rows = static_cast<int>(n - r0 < kFp8Group ? n - r0 : kFp8Group);
  const int first = threadIdx.x >> 7;
  float m = 0.0f;
  if (c < k)
    for (int r = first; r < rows; r += 2) m = fmaxf(m, fabsf(to_f32(w[(r0 + r) * k + c])));
  for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3])), kFp8AmaxFloor);
  if (c < k)
    for (int r = first; r < rows; r += 2)
      q[(r0 + r) * k + c] = static_cast<uint8_t>(
          __builtin_amdgcn_cvt_pk_fp8_f32(fp8_ratio(to_f32(w[(r0 + r) * k + c]), m), 0.0f, 0, false));
  if (threadIdx.x == 0) scale[blockIdx.x] = m / kFp8Max;
}

int64_t fp8_linear_work(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_fp8_linear(const LinearArgs& a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(div_up64(a.n, 16) * div_up64(a.rows, 16));
  if (a.dtype == 0)
    fp8_linear_kernel<float><<<grid, 64, 0, stream>>>(a);
  else
    fp8_linear_kernel<bf16_t><<<grid, 64, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_quantize_weight(const void* w, int dtype, int64_t n, int64_t k, uint8_t* q,
                                  float* scale, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(div_up64(n, kFp8Group) * div_up64(k, kFp8Group));
  if (dtype == 0)
    quantize_weight_kernel<<<grid, 256, 0, stream>>>(static_cast<const float*>(w), n, k, q, scale);
  else
    quantize_weight_kernel<<<grid, 256, 0, stream>>>(static_cast<const bf16_t*>(w), n, k, q, scale);
  return hipGetLastError();
}

}  // namespace ssm
