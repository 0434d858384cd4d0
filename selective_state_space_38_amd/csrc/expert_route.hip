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
    float key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = r.x[v] != r.x[v] ? kLowest : r.x[v];
    float mine = 0.0f, sum = 0.0f, top = 0.0f;  // choice `at`'s weight; lanes 0 .. K - 1
    int chosen = -1;
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
      // its logit is m but for a NaN that counts as the lowest
      float x = m;
      if (m == kLowest) {
        float own = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) own = v == v_of ? r.x[v] : own;
        x = __shfl(own, group * L + who);
      }
      if (j == 0) top = x;
      const float s = p.renormalize ? S::share(x, top, p.sigmoid) : r.score_of(x, p.sigmoid);
      sum += s;
      if (at == j) mine = s, chosen = e;
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
// their order, each of its waves a run of them, 64 at a time: the lanes that hold
// the same expert find each other by one ballot per bit of its number, so a
// pair's rank among its wave's is a population count, and the wave's counters
// stand in LDS.  Nothing is added by atomics: the order is the pairs' own.  With
// more than one workgroup a first launch counts; each workgroup of the second
// adds up the counts of those before it.

constexpr int kSortWaves = 16;

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

// counts[workgroup][E + 1]
template <int ROUNDS>
__global__ __launch_bounds__(64 * kSortWaves) void sort_count_kernel(SortArgs p, int64_t entries) {
  extern __shared__ int s_count[];  // [E + 1]
  const int bins = p.experts + 1;
  for (int e = threadIdx.x; e < bins; e += blockDim.x) s_count[e] = 0;
  __syncthreads();
  const int64_t from = static_cast<int64_t>(blockIdx.x) * (64 * kSortWaves * ROUNDS);
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t i = from + r * (64 * kSortWaves) + threadIdx.x;
    if (i < entries) atomicAdd(&s_count[bin_of(p.index[i], p.experts)], 1);  // whole numbers: any order
  }
  __syncthreads();
  int* to = static_cast<int*>(p.work) + static_cast<int64_t>(blockIdx.x) * bins;
  for (int e = threadIdx.x; e < bins; e += blockDim.x) to[e] = s_count[e];
}

// Column e of counts[groups][E + 1] becomes its exclusive sums, their total in row
// `groups`: one workgroup a column.
__global__ __launch_bounds__(256) void sort_scan_kernel(int* counts, int groups, int bins) {
  __shared__ int s_sum[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int* column = counts + blockIdx.x;
  int carry = 0;
  for (int g0 = 0; g0 < groups; g0 += 256) {
    const int g = g0 + threadIdx.x;
    const int c = g < groups ? column[static_cast<int64_t>(g) * bins] : 0;
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
    if (g < groups) column[static_cast<int64_t>(g) * bins] = ahead + run - c;
  }
  if (threadIdx.x == 0) column[static_cast<int64_t>(groups) * bins] = carry;
}

// scanned: counts hold exclusive sums; otherwise, with several workgroups, counts.
template <int ROUNDS>
__global__ __launch_bounds__(64 * kSortWaves) void sort_place_kernel(SortArgs p, int64_t entries,
                                                                     int bits, bool scanned) {
  extern __shared__ int lds[];  // first place [E + 1], totals [E + 1], sums [waves], counters [waves][E + 1]
  const int bins = p.experts + 1;
  int* place = lds;
  int* s_total = place + bins;
  int* sums = s_total + bins;
  uint16_t* counters = reinterpret_cast<uint16_t*>(sums + kSortWaves);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < kSortWaves * bins; e += blockDim.x) counters[e] = 0;
  const int64_t from = static_cast<int64_t>(blockIdx.x) * (64 * kSortWaves * ROUNDS) +
                       wave * (64 * ROUNDS) + lane;
  int bin[ROUNDS], rank[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r)
    bin[r] = from + 64 * r < entries ? bin_of(p.index[from + 64 * r], p.experts) : -1;
  __syncthreads();
  volatile uint16_t* own = counters + wave * bins;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const uint64_t same = same_lanes(bin[r], bits) & __ballot(bin[r] >= 0);
    const int before = __popcll(same & ((1ull << lane) - 1));
    int base = 0;
    if (bin[r] >= 0) base = own[bin[r]];
    rank[r] = base + before;
    __builtin_amdgcn_wave_barrier();
    // the lowest of the lanes writes for all: one writer per counter
    if (bin[r] >= 0 && before == 0) own[bin[r]] = static_cast<uint16_t>(base + __popcll(same));
    __builtin_amdgcn_wave_barrier();
  }
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
  const int* counts = static_cast<const int*>(p.work);
  int missing = 0;  // pairs without an expert in the workgroups before (thread 0)
  if (groups > 1 && scanned) {
    if (e < bins) {
      earlier = counts[static_cast<int64_t>(mine) * bins + e];
      total = counts[static_cast<int64_t>(groups) * bins + e];
    }
    if (e == 0) missing = counts[static_cast<int64_t>(mine) * bins + p.experts];
  } else if (groups > 1) {
    // 1024 / span threads a bin, each every so many-th workgroup's count
    int span = 64;
    while (span < bins) span *= 2;
    if (span > blockDim.x) span = blockDim.x;  // the last bin (none) is thread 0's below
    const int stride = blockDim.x / span, bin0 = e % span;
    int all = 0, ahead = 0;
#pragma unroll 8
    for (int g = e / span; g < groups; g += stride) {
      const int c = bin0 < bins ? counts[g * bins + bin0] : 0;
      ahead += g < mine ? c : 0;
      all += c;
    }
    for (int b = e; b < bins; b += blockDim.x) place[b] = s_total[b] = 0;
    __syncthreads();
    if (bin0 < bins) {
      atomicAdd(&s_total[bin0], all);  // whole numbers: any order
      atomicAdd(&place[bin0], ahead);
    }
    __syncthreads();
    total = e < bins ? s_total[e] : 0;
    earlier = e < bins ? place[e] : 0;
    if (e == 0) {
      missing = p.experts < span ? place[p.experts] : 0;
      for (int g = 0; g < mine && p.experts >= span; ++g) missing += counts[g * bins + p.experts];
    }
    __syncthreads();
  }
  // exclusive sums over the experts (the bin of pairs without one starts where the
  // experts' end)
  const int own_total = e < p.experts ? total : 0;
  int run = own_total;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int up = __shfl_up(run, d);
    if (lane >= d) run += up;
  }
  if (lane == 63) sums[wave] = run;
  __syncthreads();
  int ahead = 0, all = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) ahead += sums[w];
    all += sums[w];
  }
  const int start = ahead + run - own_total;
  if (e < p.experts) {
    place[e] = start + earlier;
    if (mine == 0) p.offsets[e] = start;
  }
  if (e == 0) {
    place[p.experts] = all + missing;
    if (mine == 0) p.offsets[p.experts] = all;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    if (bin[r] < 0) continue;
    const int64_t i = from + 64 * r;
    const int at = place[bin[r]] + counters[wave * bins + bin[r]] + rank[r];
    const bool in = bin[r] < p.experts;
    p.slot[i] = in ? at : -1;
    p.token[at] = in ? static_cast<int32_t>(i / p.topk) : -1;
  }
}

// Pairs a workgroup takes: 64 per wave up to that many in all, then 256.
static int sort_rounds(int64_t entries) { return entries <= 64 * kSortWaves ? 1 : 4; }
// More workgroups than this have their counts summed by a launch of its own.
constexpr int64_t kSortDirect = 64;

int64_t sort_work(int64_t entries, int experts) {
  const int64_t groups = div_up64(entries, 64 * kSortWaves * sort_rounds(entries));
  return groups > 1 ? (groups + 1) * (experts + 1) * 4 : 0;
}

template <int ROUNDS>
static void launch_sort_rounds(const SortArgs& a, int64_t entries, hipStream_t stream) {
  const int64_t groups = div_up64(entries, 64 * kSortWaves * ROUNDS);
  const unsigned grid = static_cast<unsigned>(groups);
  const int bins = a.experts + 1;
  int bits = 1;
  while (a.experts >> bits) ++bits;
  if (groups > 1)
    sort_count_kernel<ROUNDS><<<grid, 64 * kSortWaves, bins * 4, stream>>>(a, entries);
  if (groups > kSortDirect)
    sort_scan_kernel<<<bins, 256, 0, stream>>>(static_cast<int*>(a.work), static_cast<int>(groups),
                                               bins);
  sort_place_kernel<ROUNDS>
      <<<grid, 64 * kSortWaves, (2 * bins + kSortWaves) * 4 + kSortWaves * bins * 2, stream>>>(
          a, entries, bits, groups > kSortDirect);
}

hipError_t launch_sort(const SortArgs& a, hipStream_t stream) {
  const int64_t entries = a.tokens * a.topk;
  if (sort_rounds(entries) == 1) launch_sort_rounds<1>(a, entries, stream);
  else launch_sort_rounds<4>(a, entries, stream);
  return hipGetLastError();
}

}  // namespace ssm
