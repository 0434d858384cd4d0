// The router of a layer of experts and the order of its tokens, for gfx950:
// each expert's score, the choice of k experts, their weights, the gradient of
// both, and the stable sort of the chosen pairs by expert.

#include "feed_internal.h"
#include "layer_device.h"

namespace ssm {

// ---- router ----
//
// L lanes hold a token's E logits, V consecutive ones each.  With top the largest
// logit, s_e = exp(l_e - top) / sum (softmax), or s_e = 1 / (1 + exp(-l_e)).  The
// choice goes by the logits themselves (both scores grow with them), so no
// rounding decides it; equal ones go to the lowest index, which is the lowest
// lane's.  A NaN counts as the lowest finite logit there, and -inf is never
// chosen.
//
// The instructions of the choice bound it, k rounds of a maximum over V values and L
// lanes: of bfloat16 logits over one word of value and number, 8.8 us for 32768 tokens of 128
// experts, k 8 (12.2 by a maximum, a search for its lane and that lane's number, as float32
// logits need: theirs take 11.4; the logits' 8 MB and what is written 2.4).  16 lanes a token keep the
// maximum in one row of the wave, without LDS; from 257 experts on a lane would hold
// more than 16, and the whole wave takes a token.

template <typename T, int L, int V>
struct Scores {
  float x[V], s[V];  // logits (past the row's end: -inf), scores
  int first;         // the lane's first expert
  float base, scale; // softmax: s = exp(x - base) scale

  __device__ __forceinline__ static float all_max(float v) {
    v = row16_max(v);
    if constexpr (L == 64) {
      v = fmaxf(fmaxf(read_lane(v, 0), read_lane(v, 16)), fmaxf(read_lane(v, 32), read_lane(v, 48)));
    }
    return v;
  }
  __device__ __forceinline__ static uint32_t all_max(uint32_t v) {
    auto higher = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    auto turned = [&](auto by) { return __float_as_uint(row_ror<by.value>(__uint_as_float(v))); };
    v = higher(v, turned(std::integral_constant<int, 8>{}));
    v = higher(v, turned(std::integral_constant<int, 4>{}));
    v = higher(v, turned(std::integral_constant<int, 2>{}));
    v = higher(v, turned(std::integral_constant<int, 1>{}));
    if constexpr (L == 64) {
      auto row = [&](int at) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(v, at)); };
      v = higher(higher(row(0), row(16)), higher(row(32), row(48)));
    }
    return v;
  }
  __device__ __forceinline__ static float all_sum(float v) {
    if constexpr (L == 64) return wave_sum(v);
    return row16_sum(v);
  }

  __device__ __forceinline__ void load(const T* row, int experts, int lane) {
    first = lane * V;
    if (V % 8 == 0 && first + V <= experts) {
#pragma unroll
      for (int c = 0; c < V / 8; ++c) {
        Run8<T> run;
        run.load(row + first + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[8 * c + e] = run.get(e);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        x[v] = first + v < experts ? to_f32(row[first + v]) : -__builtin_inff();
    }
  }

  __device__ __forceinline__ void score(bool sigmoid) {
    if (sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = sigmoid_of(x[v]);
      return;
    }
    float top = x[0], sum = 0.0f;
#pragma unroll
    for (int v = 1; v < V; ++v) top = fmaxf(top, x[v]);
    top = all_max(top);
    base = top == -__builtin_inff() ? 0.0f : top;  // a row without an expert
#pragma unroll
    for (int v = 0; v < V; ++v) sum += s[v] = exp2_hw((x[v] - base) * kLog2e);
    sum = all_sum(sum);
    scale = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] *= scale;
  }

  // the score of logit x
  __device__ __forceinline__ float score_of(float x, bool sigmoid) const {
    return sigmoid ? sigmoid_of(x) : exp2_hw((x - base) * kLog2e) * scale;
  }
  __device__ __forceinline__ static float sigmoid_of(float x) {
    return 1.0f / (1.0f + exp2_hw(-x * kLog2e));
  }
  // exp(x - top) of a softmax, or sigmoid(x) over exp(min(top, 0)): what
  // renormalised weights are in proportion to.  Scaled so, they do not vanish
  // together.
  __device__ __forceinline__ static float share(float x, float top, bool sigmoid) {
    if (sigmoid)
      return exp2_hw((fminf(x, 0.0f) - fminf(top, 0.0f)) * kLog2e) /
             (1.0f + exp2_hw(-fabsf(x) * kLog2e));
    return exp2_hw((x - top) * kLog2e);
  }
};

constexpr int kRouteThreads = 256;
constexpr float kLowest = -3.402823466e38f;  // the lowest finite value

// A bfloat16's place among them as the upper half of a word: -inf the lowest, then a NaN
// with the lowest finite value, both zeros one.
constexpr uint32_t kLowestOrder = 0x00800000u;
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 + 0 = 0
  const uint32_t o = (b >> 31 ? ~b : b | 0x80000000u) & 0xffff0000u;
  return x != x ? kLowestOrder : o;
}

template <typename T, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void route_fwd_kernel(RouteArgs p) {
  using S = Scores<T, L, V>;
  constexpr int kPer = kRouteThreads / L;  // tokens a workgroup
  const int lane = threadIdx.x & 63, at = lane & (L - 1), group = lane / L;
  const int E = p.experts, K = p.topk;
  float total[V] = {};
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kPer; t0 < p.tokens;
       t0 += static_cast<int64_t>(gridDim.x) * kPer) {
    const int64_t t = t0 + threadIdx.x / L;
    const bool live = t < p.tokens;
    S r;
    r.load(static_cast<const T*>(p.logits) + (live ? t : p.tokens - 1) * E, E, at);
    r.score(p.sigmoid);
    if (p.score_sum && live) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (r.first + v < E) total[v] += r.s[v];
    }
    float mine = -__builtin_inff();  // choice `at`'s logit; lanes 0 .. K - 1
    int chosen = -1;
    if constexpr (sizeof(T) == 2) {
      // one word a logit: the value's order in the upper half, ahead of it the lower index
      uint32_t key[V], won = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = order_of(r.x[v]) | (0xffffu - (r.first + v));
      for (int j = 0; j < K; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = key[v] > m ? key[v] : m;
        m = S::all_max(m);
        if (m < kLowestOrder) break;
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = key[v] == m ? 0 : key[v];
        if (at == j) won = m;
      }
      if (won) {
        chosen = 0xffff - (won & 0xffff);
        mine = __uint_as_float((won >> 31 ? won ^ 0x80000000u : ~won) & 0xffff0000u);
        if ((won & 0xffff0000u) == kLowestOrder)  // or a NaN
          mine = to_f32(static_cast<const T*>(p.logits)[(live ? t : p.tokens - 1) * E + chosen]);
      }
    } else {
      float key[V];
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = r.x[v] != r.x[v] ? kLowest : r.x[v];
      for (int j = 0; j < K; ++j) {
        float m = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, key[v]);
        m = S::all_max(m);
        if (m == -__builtin_inff()) break;
        int v_of = -1;  // the lane's first of them
#pragma unroll
        for (int v = V - 1; v >= 0; --v) v_of = key[v] == m ? v : v_of;
        const uint64_t hit = __ballot(v_of >= 0) >> (group * L) & (L == 64 ? ~0ull : 0xffffull);
        const int who = __builtin_ctzll(hit);
        const int e = __shfl(r.first + v_of, group * L + who);
        if (at == who) {
#pragma unroll
          for (int v = 0; v < V; ++v) key[v] = v == v_of ? -__builtin_inff() : key[v];
        }
        if (at == j) mine = m, chosen = e;
      }
      if (chosen >= 0 && mine == kLowest)  // or a NaN
        mine = to_f32(static_cast<const T*>(p.logits)[(live ? t : p.tokens - 1) * E + chosen]);
    }
    const float top = __shfl(mine, group * L);
    float sum = 1.0f;
    if (p.renormalize) {
      mine = chosen >= 0 ? S::share(mine, top, p.sigmoid) : 0.0f;
      sum = S::all_sum(mine);
      // the shares know the chosen logits alone: another one that is not a number, or +inf,
      // leaves no score of a softmax
      if (!p.sigmoid && r.scale != r.scale) sum = r.scale;
    } else {
      mine = r.score_of(mine, p.sigmoid);
    }
    if (live && at < K) {
      p.index[t * K + at] = chosen;
      float w = 0.0f;
      if (chosen >= 0) w = p.scale * (p.renormalize ? mine / sum : mine);
      p.weight[t * K + at] = w;
    }
  }
  if (!p.score_sum) return;
  // the workgroup's sums over its tokens, joined in the order of its groups
  __shared__ float lds[kPer][L * V + 1];
#pragma unroll
  for (int v = 0; v < V; ++v) lds[threadIdx.x / L][at * V + v] = total[v];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kRouteThreads) {
    float s = 0.0f;
    for (int g = 0; g < kPer; ++g) s += lds[g][e];
    static_cast<float*>(p.work)[static_cast<int64_t>(blockIdx.x) * E + e] = s;
  }
}

// Gradient.  With g_e = scale dw_j at the chosen e and P'_e = dscore_sum:
//   softmax            dl_e = s_e (g_e + P'_e - sum_f s_f (g_f + P'_f))
//   sigmoid            dl_e = s_e (1 - s_e) (g_e + P'_e)
// and with renormalised weights, q the chosen ones' shares and c = sum_j q_j scale dw_j,
// the chosen e get q_e (scale dw_j - c) (sigmoid: times 1 - s_e) in place of g's terms.
// An entry of index outside 0 .. E - 1 takes no part.
template <typename T, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void route_bwd_kernel(RouteArgs p) {
  using S = Scores<T, L, V>;
  constexpr int kPer = kRouteThreads / L;
  const int lane = threadIdx.x & 63, at = lane & (L - 1), group = lane / L;
  const int E = p.experts, K = p.topk;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kPer + threadIdx.x / L;
  const bool live = t < p.tokens;
  const int64_t row = live ? t : p.tokens - 1;
  S r;
  r.load(static_cast<const T*>(p.logits) + row * E, E, at);
  r.score(p.sigmoid);
  float add[V], g[V] = {};
#pragma unroll
  for (int v = 0; v < V; ++v)
    add[v] = p.dscore_sum && r.first + v < E ? p.dscore_sum[r.first + v] : 0.0f;
  if (p.dweight) {
    const int my_e = at < K ? p.index[row * K + at] : -1;
    const float my_dw = at < K ? p.scale * p.dweight[row * K + at] : 0.0f;
    const bool in = my_e >= 0 && my_e < E;
    float mine_x = 0.0f, q = 0.0f, c = 0.0f;
    if (p.renormalize) {
      mine_x = in ? to_f32(static_cast<const T*>(p.logits)[row * E + my_e]) : -__builtin_inff();
      const float top = S::all_max(mine_x);
      q = in ? S::share(mine_x, top, p.sigmoid) : 0.0f;
      const float sum = S::all_sum(q);
      q = sum == 0.0f ? 0.0f : q / sum;
      c = S::all_sum(in ? q * my_dw : 0.0f);
    }
    float give = in ? my_dw : 0.0f;
    if (p.renormalize) {
      give = in ? q * (my_dw - c) : 0.0f;
      if (p.sigmoid && in) give *= S::sigmoid_of(-mine_x);
    }
    for (int j = 0; j < K; ++j) {
      const int e = __shfl(in ? my_e : -1, group * L + j) - r.first;
      const float d = __shfl(give, group * L + j);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v == e) g[v] += d;
    }
  }
  if (!p.renormalize) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      add[v] += g[v];
      g[v] = 0.0f;
    }
  }
  if (p.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] += r.s[v] * S::sigmoid_of(-r.x[v]) * add[v];
  } else {
    float mean = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) mean += r.s[v] * add[v];
    mean = S::all_sum(mean);
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] += r.s[v] * (add[v] - mean);
  }
  if (!live) return;
  T* to = static_cast<T*>(p.dlogits) + t * E + r.first;
  if (V % 8 == 0 && r.first + V <= E) {
#pragma unroll
    for (int c = 0; c < V / 8; ++c) {
      float part[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) part[e] = g[8 * c + e];
      store8(to + 8 * c, part);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (r.first + v < E) store_act(to, v, g[v]);
  }
}

static int64_t route_groups(int64_t tokens, int experts) {
  const int64_t per = kRouteThreads / (experts <= 256 ? 16 : 64);
  const int64_t all = div_up64(tokens, per);
  return all < 1024 ? all : 1024;
}

int64_t route_work(int64_t tokens, int experts) {
  return route_groups(tokens, experts) * experts * 4;
}

template <typename T, int L, int V>
static void launch_route(const RouteArgs& a, bool fwd, hipStream_t stream) {
  if (fwd) {
    const int64_t groups = a.score_sum ? route_groups(a.tokens, a.experts)
                                       : div_up64(a.tokens, kRouteThreads / L);
    route_fwd_kernel<T, L, V><<<static_cast<unsigned>(groups), kRouteThreads, 0, stream>>>(a);
    if (a.score_sum)
      launch_column_sum(static_cast<const float*>(a.work), groups, a.experts, a.score_sum, stream);
  } else {
    const unsigned groups = static_cast<unsigned>(div_up64(a.tokens, kRouteThreads / L));
    route_bwd_kernel<T, L, V><<<groups, kRouteThreads, 0, stream>>>(a);
  }
}

template <typename T>
static void launch_route_typed(const RouteArgs& a, bool fwd, hipStream_t stream) {
  const int e = a.experts;
  if (e <= 16) launch_route<T, 16, 1>(a, fwd, stream);
  else if (e <= 32) launch_route<T, 16, 2>(a, fwd, stream);
  else if (e <= 64) launch_route<T, 16, 4>(a, fwd, stream);
  else if (e <= 128) launch_route<T, 16, 8>(a, fwd, stream);
  else if (e <= 256) launch_route<T, 16, 16>(a, fwd, stream);
  else if (e <= 512) launch_route<T, 64, 8>(a, fwd, stream);
  else launch_route<T, 64, 16>(a, fwd, stream);
}

hipError_t launch_route_fwd(const RouteArgs& a, hipStream_t stream) {
  if (a.dtype == 0) launch_route_typed<float>(a, true, stream);
  else launch_route_typed<bf16_t>(a, true, stream);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteArgs& a, hipStream_t stream) {
  if (a.dtype == 0) launch_route_typed<float>(a, false, stream);
  else launch_route_typed<bf16_t>(a, false, stream);
  return hipGetLastError();
}

// ---- order ----
//
// A stable counting sort.  A workgroup takes kSortEntries pairs (token, choice) in
// their order, 64 a wave: the lanes that hold the same expert find each other by one
// ballot per bit of its number, so a pair's rank among its wave's is a population
// count, and the waves' counters stand in LDS.  The order is the pairs' own, whatever
// runs first.  With more than one workgroup a first launch counts; each workgroup of the
// last adds up the counts of those before it, or a launch between does.
//
// 262144 pairs of 128 experts: 2.9 + 8.5 us, a chain of short steps over 1 MB read and
// 2 MB written; with four runs a wave, a quarter of the workgroups, 3.6 + 10.8.  16384 of 64
// experts: 2.6 + 5.8 us, 3.2 + 8.3 with four.

constexpr int kSortWaves = 16;
constexpr int64_t kSortEntries = 64 * kSortWaves;

__device__ __forceinline__ uint64_t same_lanes(int e, int bits) {
  uint64_t same = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool one = e >> b & 1;
    const uint64_t with = __ballot(one);
    same &= one ? with : ~with;
  }
  return same;
}

// Bin of a pair: its expert, or E for none.
__device__ __forceinline__ int bin_of(int e, int experts) {
  return static_cast<unsigned>(e) < static_cast<unsigned>(experts) ? e : experts;
}

// Counts of a workgroup's pairs, 16 bits each, an even number of them.
__host__ __device__ __forceinline__ int count_words(int experts) { return (experts + 1) / 2; }

// counts[workgroup][2 count_words]
__global__ __launch_bounds__(64 * kSortWaves) void sort_count_kernel(SortArgs p, int64_t entries) {
  extern __shared__ int s_count[];  // [2 words]
  const int words = count_words(p.experts);
  for (int e = threadIdx.x; e < 2 * words; e += blockDim.x) s_count[e] = 0;
  __syncthreads();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kSortEntries + threadIdx.x;
  if (i < entries) {
    const int bin = bin_of(p.index[i], p.experts);
    if (bin < p.experts) atomicAdd(&s_count[bin], 1);  // whole numbers: any order
  }
  __syncthreads();
  uint32_t* to = static_cast<uint32_t*>(p.work) + static_cast<int64_t>(blockIdx.x) * words;
  for (int w = threadIdx.x; w < words; w += blockDim.x) to[w] = s_count[2 * w] | s_count[2 * w + 1] << 16;
}

// Exclusive sums over the workgroups of an expert's counts, their total behind: one workgroup
// an expert.
__global__ __launch_bounds__(256) void sort_scan_kernel(const uint16_t* counts, int stride, int groups,
                                                        int experts, int* sums) {
  __shared__ int s_sum[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int carry = 0;
  for (int g0 = 0; g0 < groups; g0 += 256) {
    const int g = g0 + threadIdx.x;
    const int c = g < groups ? counts[static_cast<int64_t>(g) * stride + blockIdx.x] : 0;
    int run = c;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int up = __shfl_up(run, d);
      if (lane >= d) run += up;
    }
    __syncthreads();
    if (lane == 63) s_sum[wave] = run;
    __syncthreads();
    int ahead = carry;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) ahead += s_sum[w];
      carry += s_sum[w];
    }
    if (g < groups) sums[static_cast<int64_t>(g) * experts + blockIdx.x] = ahead + run - c;
  }
  if (threadIdx.x == 0) sums[static_cast<int64_t>(groups) * experts + blockIdx.x] = carry;
}

// scanned: the exclusive sums, or null.
__global__ __launch_bounds__(64 * kSortWaves) void sort_place_kernel(SortArgs p, int64_t entries,
                                                                     int bits, const int* scanned) {
  extern __shared__ int lds[];  // first place, totals [E + 1], sums [2 waves], counters [waves][E + 1]
  const int bins = p.experts + 1;
  int* place = lds;
  int* s_total = place + bins;
  int* sums = s_total + bins;
  uint16_t* counters = reinterpret_cast<uint16_t*>(sums + 2 * kSortWaves);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < kSortWaves * bins; e += blockDim.x) counters[e] = 0;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kSortEntries + threadIdx.x;
  const int bin = i < entries ? bin_of(p.index[i], p.experts) : -1;
  __syncthreads();
  const uint64_t same = same_lanes(bin, bits) & __ballot(bin >= 0);
  const int rank = __popcll(same & ((1ull << lane) - 1));
  // the lowest of the lanes writes for all: one writer per counter
  if (bin >= 0 && rank == 0) counters[wave * bins + bin] = static_cast<uint16_t>(__popcll(same));
  __syncthreads();
  // the waves' counters become places within the workgroup's run of a bin
  const int e = threadIdx.x;
  int total = 0, earlier = 0;
  for (int b = e; b < bins; b += blockDim.x) {
    int sum = 0;
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = counters[w * bins + b];
      counters[w * bins + b] = static_cast<uint16_t>(sum);
      sum += c;
    }
    if (b == e) total = sum;
  }
  const int groups = static_cast<int>(gridDim.x), mine = static_cast<int>(blockIdx.x);
  if (groups > 1 && scanned) {
    if (e < p.experts) {
      earlier = scanned[static_cast<int64_t>(mine) * p.experts + e];
      total = scanned[static_cast<int64_t>(groups) * p.experts + e];
    }
  } else if (groups > 1) {
    // 1024 / span threads a word of two counts, each every so many-th workgroup's
    const uint32_t* counts = static_cast<const uint32_t*>(p.work);
    const int words = count_words(p.experts);
    int span = 64;
    while (span < words) span *= 2;
    const int stride = blockDim.x / span, word = e % span;
    int all[2] = {}, ahead[2] = {};
#pragma unroll 8
    for (int g = e / span; g < groups; g += stride) {
      const uint32_t c = word < words ? counts[g * words + word] : 0;
      const int c0 = c & 0xffff, c1 = c >> 16;
      all[0] += c0;
      all[1] += c1;
      ahead[0] += g < mine ? c0 : 0;
      ahead[1] += g < mine ? c1 : 0;
    }
    for (int b = e; b < bins; b += blockDim.x) place[b] = s_total[b] = 0;
    __syncthreads();
    if (word < words) {
      for (int h = 0; h < 2; ++h) {  // behind an odd number of experts: none, to the last bin
        atomicAdd(&s_total[2 * word + h], all[h]);  // whole numbers: any order
        atomicAdd(&place[2 * word + h], ahead[h]);
      }
    }
    __syncthreads();
    total = e < p.experts ? s_total[e] : 0;
    earlier = e < p.experts ? place[e] : 0;
    __syncthreads();
  }
  // exclusive sums over the experts (the bin of pairs without one starts where the
  // experts' end)
  const int own_total = e < p.experts ? total : 0;
  int run = own_total, before = earlier;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int up = __shfl_up(run, d);
    if (lane >= d) run += up;
    before += __shfl_xor(before, d);
  }
  if (lane == 63) {
    sums[wave] = run;
    sums[kSortWaves + wave] = before;
  }
  __syncthreads();
  int ahead = 0, all = 0, taken = 0;  // by the workgroups before
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) ahead += sums[w];
    all += sums[w];
    taken += sums[kSortWaves + w];
  }
  const int start = ahead + run - own_total;
  if (e < p.experts) {
    place[e] = start + earlier;
    if (mine == 0) p.offsets[e] = start;
  }
  if (e == 0) {
    place[p.experts] = all + mine * static_cast<int>(kSortEntries) - taken;
    if (mine == 0) p.offsets[p.experts] = all;
  }
  __syncthreads();
  if (bin < 0) return;
  const int at = place[bin] + counters[wave * bins + bin] + rank;
  const bool in = bin < p.experts;
  p.slot[i] = in ? at : -1;
  p.token[at] = in ? static_cast<int32_t>(i / p.topk) : -1;
}

// More words of counts than these are summed by a launch of its own: of 16384 (262144 pairs
// of 128 experts) the sums take every workgroup 2.1 us, the launch 3 and a gap.
constexpr int64_t kSortDirect = 20000;

static int64_t sort_sums_at(int64_t groups, int experts) {
  return (groups * count_words(experts) * 4 + 15) / 16 * 16;
}

static bool sort_scans(int64_t groups, int experts) {
  return groups > 1 && groups * count_words(experts) > kSortDirect;
}

int64_t sort_work(int64_t entries, int experts) {
  const int64_t groups = div_up64(entries, kSortEntries);
  if (groups <= 1) return 0;
  return sort_sums_at(groups, experts) +
         (sort_scans(groups, experts) ? (groups + 1) * experts * 4 : 0);
}

hipError_t launch_sort(const SortArgs& a, hipStream_t stream) {
  const int64_t entries = a.tokens * a.topk, groups = div_up64(entries, kSortEntries);
  const unsigned grid = static_cast<unsigned>(groups);
  const int words = count_words(a.experts), bins = a.experts + 1;
  int* sums = nullptr;
  int bits = 1;
  while (a.experts >> bits) ++bits;
  if (groups > 1) sort_count_kernel<<<grid, 64 * kSortWaves, words * 8, stream>>>(a, entries);
  if (sort_scans(groups, a.experts)) {
    sums = reinterpret_cast<int*>(static_cast<char*>(a.work) + sort_sums_at(groups, a.experts));
    sort_scan_kernel<<<a.experts, 256, 0, stream>>>(static_cast<const uint16_t*>(a.work), 2 * words,
                                                    static_cast<int>(groups), a.experts, sums);
  }
  sort_place_kernel<<<grid, 64 * kSortWaves, (2 * bins + 2 * kSortWaves) * 4 + kSortWaves * bins * 2,
                      stream>>>(a, entries, bits, sums);
  return hipGetLastError();
}

}  // namespace ssm
