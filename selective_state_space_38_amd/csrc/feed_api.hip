// C ABI of the feed-forward layer's operators, dense or of experts: validation and
// dispatch.  The operations are documented in ssm_scan.h.

#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/ssm_scan.h"
#include "feed_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool valid_dtype(int32_t t) { return t == SSM_F32 || t == SSM_BF16; }
uintptr_t elem(int32_t t) { return t == SSM_BF16 ? 2 : 4; }
int64_t up16(int64_t bytes) { return ssm::div_up64(bytes, 16) * 16; }

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

// topk pairs of every token, numbered in 32 bits
int check_pairs(int64_t tokens, int32_t experts, int32_t topk) {
  if (tokens <= 0 || topk <= 0 || topk > ssm::kMaxTopk) return SSM_EINVAL;
  if (experts <= 0 || experts > ssm::kMaxExperts) return SSM_EINVAL;
  return tokens > (1LL << 30) / topk ? SSM_EINVAL : SSM_OK;
}

// 16 or 64 lanes a token, or a row: a launch has fewer than 2^32.
constexpr int64_t kMostTokens = 1LL << 25;

int check_route(const route_dims* d) {
  if (!d) return SSM_EINVAL;
  if (!valid_dtype(d->dtype)) return SSM_EDTYPE;
  if (d->score != SSM_SOFTMAX && d->score != SSM_SIGMOID) return SSM_EINVAL;
  if (d->topk > d->experts || d->tokens > kMostTokens) return SSM_EINVAL;
  return check_pairs(d->tokens, d->experts, d->topk);
}

ssm::RouteArgs route_args(const route_dims* d, const void* logits, float scale) {
  ssm::RouteArgs a = {};
  a.dtype = d->dtype;
  a.experts = d->experts;
  a.topk = d->topk;
  a.sigmoid = d->score == SSM_SIGMOID;
  a.renormalize = d->renormalize != 0;
  a.tokens = d->tokens;
  a.scale = scale;
  a.logits = logits;
  return a;
}

int check_order(const order_dims* d) {
  if (!d) return SSM_EINVAL;
  if (!valid_dtype(d->dtype) || !valid_dtype(d->residual_dtype)) return SSM_EDTYPE;
  if (d->rows <= 0 || d->rows > kMostTokens || d->tokens > kMostTokens || d->dim <= 0 || d->dim > (1LL << 24)) return SSM_EINVAL;
  return check_pairs(d->tokens, 1, d->topk);
}

ssm::OrderArgs order_args(const order_dims* d) {
  ssm::OrderArgs a = {};
  a.dtype = d->dtype;
  a.residual_dtype = d->residual_dtype;
  a.topk = d->topk;
  a.tokens = d->tokens;
  a.rows = d->rows;
  a.dim = d->dim;
  return a;
}

int check_product(const product_dims* d) {
  if (!d) return SSM_EINVAL;
  if (!valid_dtype(d->dtype) || !valid_dtype(d->out_dtype)) return SSM_EDTYPE;
  if (d->activation < SSM_ACT_NONE || d->activation > SSM_ACT_GEGLU) return SSM_EINVAL;
  if (d->experts < 0 || d->experts > ssm::kMaxExperts) return SSM_EINVAL;
  if (d->rows <= 0 || d->n <= 0 || d->k <= 0 || d->k % 8 || d->x_rows <= 0)
    return SSM_EINVAL;
  if (d->ld_x < d->k || d->ld_x > (1LL << 26) || d->ld_x % 8) return SSM_EINVAL;
  // limits of the launch arithmetic: 32-bit row numbers and counts of tiles
  if (d->rows > (1LL << 30) || d->x_rows > (1LL << 30) || d->n > (1LL << 20) || d->k > (1LL << 20))
    return SSM_EINVAL;
  const int64_t nw = d->activation >= SSM_ACT_SWIGLU ? 2 * d->n : d->n;
  const int64_t row_tiles = ssm::div_up64(d->rows, 256) + d->experts;
  if (row_tiles * ssm::div_up64(nw > d->k ? nw : d->k, 256) > ssm::kMostTiles) return SSM_EINVAL;
  const int64_t matrices = d->experts ? d->experts : 1;
  if (matrices * ssm::div_up64(nw, 256) * ssm::div_up64(d->k, 256) > ssm::kMostTiles) return SSM_EINVAL;
  return SSM_OK;
}

ssm::ProductArgs product_args(const product_dims* d) {
  ssm::ProductArgs a = {};
  a.dtype = d->dtype;
  a.out_dtype = d->out_dtype;
  a.act = d->activation;
  a.experts = d->experts;
  a.rows = d->rows;
  a.n = d->n;
  a.k = d->k;
  a.x_rows = d->x_rows;
  a.ld_x = d->ld_x;
  return a;
}

// The gradients a backward call is asked for.
bool valid_wants(int32_t wants) { return wants > 0 && wants <= 7; }

}  // namespace

extern "C" {

int64_t expert_route_work_bytes(const route_dims* dims) {
  const int rc = check_route(dims);
  return rc != SSM_OK ? rc : up16(ssm::route_work(dims->tokens, dims->experts));
}

int expert_route_fwd(const void* logits, float scale, int32_t* index, float* weight,
                     float* score_sum, void* work, const route_dims* dims, void* stream) {
  int rc = check_route(dims);
  if (rc != SSM_OK) return rc;
  if (!logits || !index || !weight || (score_sum && !work)) return SSM_EINVAL;
  if (!aligned(logits, elem(dims->dtype))) return SSM_EALIGN;
  const void* words[] = {index, weight, score_sum};
  if ((rc = check_aligned(words, 4)) != SSM_OK) return rc;
  if (work && !aligned(work, 16)) return SSM_EALIGN;
  const void* ins[] = {logits};
  const void* outs[] = {index, weight, score_sum, work};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::RouteArgs a = route_args(dims, logits, scale);
  a.index = index;
  a.weight = weight;
  a.score_sum = score_sum;
  a.work = work;
  return ssm::launch_route_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                 : SSM_ELAUNCH;
}

int expert_route_bwd(const void* logits, float scale, const int32_t* index, const float* dweight,
                     const float* dscore_sum, void* dlogits, const route_dims* dims, void* stream) {
  int rc = check_route(dims);
  if (rc != SSM_OK) return rc;
  if (!logits || !dlogits || (!dweight && !dscore_sum) || (dweight && !index)) return SSM_EINVAL;
  const void* acts[] = {logits, dlogits};
  const void* words[] = {index, dweight, dscore_sum};
  if ((rc = check_aligned(acts, elem(dims->dtype))) != SSM_OK) return rc;
  if ((rc = check_aligned(words, 4)) != SSM_OK) return rc;
  const void* ins[] = {logits, index, dweight, dscore_sum};
  const void* outs[] = {dlogits};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::RouteArgs a = route_args(dims, logits, scale);
  a.index = const_cast<int32_t*>(index);  // read only
  a.dweight = dweight;
  a.dscore_sum = dscore_sum;
  a.dlogits = dlogits;
  return ssm::launch_route_bwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                 : SSM_ELAUNCH;
}

int64_t expert_sort_work_bytes(int64_t tokens, int32_t topk, int32_t experts) {
  const int rc = check_pairs(tokens, experts, topk);
  return rc != SSM_OK ? rc : up16(ssm::sort_work(tokens * topk, experts));
}

int expert_sort(const int32_t* index, int64_t tokens, int32_t topk, int32_t experts,
                int32_t* offsets, int32_t* token, int32_t* slot, void* work, void* stream) {
  int rc = check_pairs(tokens, experts, topk);
  if (rc != SSM_OK) return rc;
  if (!index || !offsets || !token || !slot) return SSM_EINVAL;
  if (!work && expert_sort_work_bytes(tokens, topk, experts) > 0) return SSM_EINVAL;
  const void* words[] = {index, offsets, token, slot};
  if ((rc = check_aligned(words, 4)) != SSM_OK) return rc;
  if (work && !aligned(work, 16)) return SSM_EALIGN;
  const void* ins[] = {index};
  const void* outs[] = {offsets, token, slot, work};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::SortArgs a = {experts, topk, tokens, index, offsets, token, slot, work};
  return ssm::launch_sort(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ELAUNCH;
}

int expert_gather(const void* x, const int32_t* token, void* xs, const order_dims* dims,
                  void* stream) {
  int rc = check_order(dims);
  if (rc != SSM_OK) return rc;
  if (!x || !token || !xs) return SSM_EINVAL;
  const void* acts[] = {x, xs};
  if ((rc = check_aligned(acts, elem(dims->dtype))) != SSM_OK) return rc;
  if (!aligned(token, 4)) return SSM_EALIGN;
  const void* ins[] = {x, token};
  const void* outs[] = {xs};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::OrderArgs a = order_args(dims);
  a.x = x;
  a.token = token;
  a.xs = xs;
  return ssm::launch_gather(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                              : SSM_ELAUNCH;
}

int expert_combine_fwd(const void* y, const int32_t* slot, const float* weight,
                       const void* residual, void* out, const order_dims* dims, void* stream) {
  int rc = check_order(dims);
  if (rc != SSM_OK) return rc;
  if (!y || !slot || !out) return SSM_EINVAL;
  const void* res[] = {residual, out};
  const void* words[] = {slot, weight};
  if (!aligned(y, elem(dims->dtype))) return SSM_EALIGN;
  if ((rc = check_aligned(res, elem(dims->residual_dtype))) != SSM_OK) return rc;
  if ((rc = check_aligned(words, 4)) != SSM_OK) return rc;
  // out may be residual itself: an element is read before it is written
  const void* ins[] = {y, slot, weight};
  const void* outs[] = {out};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::OrderArgs a = order_args(dims);
  a.y = y;
  a.slot = slot;
  a.weight = weight;
  a.residual = residual;
  a.out = out;
  return ssm::launch_combine_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                   : SSM_ELAUNCH;
}

int expert_combine_bwd(const void* dout, const void* y, const int32_t* slot, const float* weight,
                       void* dy, float* dweight, const order_dims* dims, void* stream) {
  int rc = check_order(dims);
  if (rc != SSM_OK) return rc;
  if (!dout || !slot || !dy || (dweight && (!y || !weight))) return SSM_EINVAL;
  const void* acts[] = {y, dy};
  const void* words[] = {slot, weight, dweight};
  if (!aligned(dout, elem(dims->residual_dtype))) return SSM_EALIGN;
  if ((rc = check_aligned(acts, elem(dims->dtype))) != SSM_OK) return rc;
  if ((rc = check_aligned(words, 4)) != SSM_OK) return rc;
  const void* ins[] = {dout, y, slot, weight};
  const void* outs[] = {dy, dweight};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::OrderArgs a = order_args(dims);
  a.dout = dout;
  a.y = y;
  a.slot = slot;
  a.weight = weight;
  a.dy = dy;
  a.dweight = dweight;
  return ssm::launch_combine_bwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                   : SSM_ELAUNCH;
}

int64_t linear_fwd_work_bytes(const product_dims* dims) {
  const int rc = check_product(dims);
  return rc != SSM_OK ? rc : up16(ssm::product_fwd_work(product_args(dims)));
}

int linear_fwd(const void* x, const int32_t* token, const void* w, const int32_t* offsets,
               const float* bias, const void* residual, void* out, void* pre, void* work,
               const product_dims* dims, void* stream) {
  int rc = check_product(dims);
  if (rc != SSM_OK) return rc;
  if (!x || !w || !out || (dims->experts > 0) != (offsets != nullptr)) return SSM_EINVAL;
  if (token ? dims->experts == 0 : dims->x_rows != dims->rows) return SSM_EINVAL;
  if (!work && linear_fwd_work_bytes(dims) > 0) return SSM_EINVAL;
  const void* wide[] = {x, w, bias, residual, out, pre, work};
  const void* words[] = {token, offsets};
  if ((rc = check_aligned(wide, 16)) != SSM_OK) return rc;
  if ((rc = check_aligned(words, 4)) != SSM_OK) return rc;
  // out may be residual itself: an element is read before it is written
  const void* ins[] = {x, token, w, offsets, bias, residual == out ? nullptr : residual};
  const void* outs[] = {out, pre, work};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::ProductArgs a = product_args(dims);
  a.x = x;
  a.token = token;
  a.w = w;
  a.offsets = offsets;
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.pre = pre;
  a.work = work;
  return ssm::launch_product_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                   : SSM_ELAUNCH;
}

int64_t linear_bwd_work_bytes(const product_dims* dims, int32_t wants) {
  const int rc = check_product(dims);
  if (rc != SSM_OK) return rc;
  if (!valid_wants(wants)) return SSM_EINVAL;
  ssm::ProductArgs a = product_args(dims);
  // the sizes alone count: any address stands for a gradient that is asked for
  char* any = reinterpret_cast<char*>(16);
  a.dx = wants & SSM_WANT_DX ? any : nullptr;
  a.dw = wants & SSM_WANT_DW ? any : nullptr;
  a.dbias = wants & SSM_WANT_DBIAS ? reinterpret_cast<float*>(any) : nullptr;
  return up16(ssm::product_bwd_work(a));
}

int linear_bwd(const void* dout, const void* x, const int32_t* token, const void* w,
               const int32_t* offsets, const void* pre, void* dx, void* dw, float* dbias,
               void* work, const product_dims* dims, void* stream) {
  int rc = check_product(dims);
  if (rc != SSM_OK) return rc;
  if (!dout || (!dx && !dw && !dbias) || (dx && !w) || (dw && !x)) return SSM_EINVAL;
  if ((dims->experts > 0) != (offsets != nullptr)) return SSM_EINVAL;
  if (token ? dims->experts == 0 : dims->x_rows != dims->rows) return SSM_EINVAL;
  if ((dims->activation != SSM_ACT_NONE) != (pre != nullptr)) return SSM_EINVAL;
  const int32_t wants = (dx ? SSM_WANT_DX : 0) | (dw ? SSM_WANT_DW : 0) | (dbias ? SSM_WANT_DBIAS : 0);
  if (!work && linear_bwd_work_bytes(dims, wants) > 0) return SSM_EINVAL;
  const void* wide[] = {dout, x, w, pre, dx, dw, work};
  const void* words[] = {token, offsets, dbias};
  if ((rc = check_aligned(wide, 16)) != SSM_OK) return rc;
  if ((rc = check_aligned(words, 4)) != SSM_OK) return rc;
  const void* ins[] = {dout, x, token, w, offsets, pre};
  const void* outs[] = {dx, dw, dbias, work};
  if ((rc = check_alias(ins, outs)) != SSM_OK) return rc;
  ssm::ProductArgs a = product_args(dims);
  a.dout = dout;
  a.x = x;
  a.token = token;
  a.w = w;
  a.offsets = offsets;
  a.pre = const_cast<void*>(pre);  // read only
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.work = work;
  return ssm::launch_product_bwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                   : SSM_ELAUNCH;
}

}  // extern "C"
