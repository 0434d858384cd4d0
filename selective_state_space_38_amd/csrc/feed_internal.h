// Launch interfaces between the feed-forward layer's entry points (feed_api.hip)
// and their kernels.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_internal.h"

namespace ssm {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 16;

enum Activation : int { kNoAct = 0, kSilu = 1, kGelu = 2, kSwiglu = 3, kGeglu = 4 };
constexpr bool is_gated(int act) { return act >= kSwiglu; }

struct RouteArgs {
  int dtype, experts, topk;
  bool sigmoid, renormalize;
  int64_t tokens;
  float scale;
  const void* logits;
  int32_t* index;           // forward: written; backward: read
  float* weight;
  float* score_sum;         // nullable
  const float* dweight;     // nullable with dscore_sum
  const float* dscore_sum;  // nullable
  void* dlogits;
  void* work;
};

int64_t route_work(int64_t tokens, int experts);
hipError_t launch_route_fwd(const RouteArgs& a, hipStream_t stream);
hipError_t launch_route_bwd(const RouteArgs& a, hipStream_t stream);

struct SortArgs {
  int experts, topk;
  int64_t tokens;
  const int32_t* index;
  int32_t *offsets, *token, *slot;
  void* work;
};

int64_t sort_work(int64_t entries, int experts);
hipError_t launch_sort(const SortArgs& a, hipStream_t stream);

struct OrderArgs {
  int dtype, residual_dtype, topk;
  int64_t tokens, rows, dim;
  const void* x;            // gather
  const int32_t* token;
  void* xs;
  const void* y;            // combine
  const int32_t* slot;
  const float* weight;      // nullable: 1
  const void* residual;     // nullable
  void* out;
  const void* dout;         // backward, of residual_dtype
  void* dy;
  float* dweight;           // nullable
};

hipError_t launch_gather(const OrderArgs& a, hipStream_t stream);
hipError_t launch_combine_fwd(const OrderArgs& a, hipStream_t stream);
hipError_t launch_combine_bwd(const OrderArgs& a, hipStream_t stream);

// Tiles of a product's launch at most: fewer than 2^32 lanes, an expert's padding and the other
// product of the gradient included.
constexpr int64_t kMostTiles = 1 << 21;

// A linear product's sizes and operands.  nw = n, or 2 n of a gated activation.
struct ProductArgs {
  int dtype, out_dtype, act, experts;  // experts 0: one matrix for all rows
  int64_t rows, n, k, x_rows, ld_x;
  const void* x;
  const int32_t* token;     // nullable: row r is x's row r
  const void* w;            // [experts][nw][k]
  const int32_t* offsets;   // [experts + 1], nullable with experts 0
  const float* bias;        // [experts][nw], nullable
  const void* residual;     // [rows][n] of out_dtype, nullable
  void* out;
  void* pre;                // [rows][nw] of dtype; forward: nullable
  // backward
  const void* dout;         // [rows][n] of out_dtype
  void* dx;                 // [rows][k], nullable
  void* dw;                 // nullable
  float* dbias;             // nullable
  void* work;
  int64_t nw() const { return is_gated(act) ? 2 * n : n; }
};

int64_t product_fwd_work(const ProductArgs& a);
int64_t product_bwd_work(const ProductArgs& a);
hipError_t launch_product_fwd(const ProductArgs& a, hipStream_t stream);
hipError_t launch_product_bwd(const ProductArgs& a, hipStream_t stream);

}  // namespace ssm
