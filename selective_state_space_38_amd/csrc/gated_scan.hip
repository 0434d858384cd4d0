// Gated linear recurrence for gfx950: forward over a sequence, backward, and
// the one-token step.  Per channel, with rho = sigmoid(r), iota = sigmoid(i):
//   a = exp(log_decay rho), beta = sqrt(1 - a^2),
//   h_t = a h_{t-1} + beta iota x_t.

#include <stdlib.h>

#include "layer_device.h"

namespace ssm {

// Carry waits that hit their bound.
__device__ unsigned g_gated_timeouts;

// rho, iota, a and beta of one step.  1 - a^2 cancels where a is close to 1
// (long memory), so with y = log_decay rho it is m (1 + a), m = -expm1(y): for
// |y| < 3/16 by a cubic for expm1(y) / y (least largest relative error, 8e-8) and
// a = 1 - m, elsewhere from a = exp(y), losing at most ~4e-7 relative.  lam2 =
// log_decay log2(e), so y2 = y log2(e) is the hardware exp's argument, and the
// cubic is in y2.  (The kernels' vector units are busy three quarters of the time:
// the series to y^6 that holds to |y| < 1/4 costs 3% of the forward's time.)  The
// clamp is for log_decay > 0; unlike fmaxf it keeps a beta that is not a number.
__device__ __forceinline__ void gate(float r, float lam2, float& rho, float& a, float& beta) {
  rho = sigmoid_f32(r);
  const float y2 = lam2 * rho;
  const float e = exp2_hw(y2);
  float p = -8.92426018e-3f;
  p = fmaf(p, y2, -5.53877385e-2f);
  p = fmaf(p, y2, -2.40220194e-1f);
  p = fmaf(p, y2, -6.93147127e-1f);
  const bool series = fabsf(y2) < 0.27050532f;
  const float m = series ? p * y2 : 1.0f - e;
  a = series ? 1.0f - m : e;
  beta = __builtin_amdgcn_sqrtf(__builtin_elementwise_maximum(fmaf(m, a, m), 0.0f));
}

// A wave owns V channels per lane (one dword of a row: 64 float32 or 128
// bfloat16 channels, 256 bytes) and a run of kGatedRun steps; a workgroup is
// several consecutive runs of the same channels, a chunk of the sequence.
// One pass over the run's gates and inputs leaves two numbers per step in
// registers, the product A_j of a since the run's start and the state H_j from
// zero; the runs' last ones meet in LDS, and once the state h before the run is
// known the outputs are A_j h + H_j.  Every input is read once and every output
// written once: 4 x 8192 steps of 5120 bfloat16 channels 273 us, 4.9 TB/s where a
// large copy reaches 5.2 and three reads to a write 6.0, the vector units 75%
// busy; with its backward 770 us, 4.8.
//
// Chunks of one channel block exchange carries through 8-byte records, one per
// channel, holding both numbers of an aggregate or the state itself, so a
// relaxed 8-byte load sees a whole record and nothing else is ordered.  A
// workgroup publishes its aggregate, walks back to the nearest state and folds
// the aggregates since then forward, h = A h + H, in sequence order.  Since a
// chunk's state is that same fold, where the walk stops does not change a bit
// of the result.  Work is taken in ticket order, chunk by chunk, so a wait is
// always for a workgroup that already runs.  (One counter hands out a ticket in
// 13 ns; several, the channel blocks dealt to them, measured faster for chunks of
// a few runs but slower for the larger ones, which are better than either.)
constexpr int kMaxWaves = 16;

// Record: state (code 1.0, sign clear) or aggregate (code -A, sign set); 0 is
// empty.
constexpr uint32_t kStateCode = 0x3f800000u;

__device__ __forceinline__ void put_record(uint64_t* p, uint32_t code, float h) {
  __hip_atomic_store(p, (static_cast<uint64_t>(code) << 32) | __float_as_uint(h), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}

template <int V>
__device__ __forceinline__ void put_records(uint64_t* p, bool state, const float (&A)[V],
                                            const float (&H)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v)
    put_record(p + v, state ? kStateCode : (__float_as_uint(A[v]) | 0x80000000u), H[v]);
}

// The state after chunk `newest` of a channel block, from its records (rec:
// this lane's record of chunk 0; consecutive chunks are 64 V apart).  Chunk 0
// always publishes its state, so the walk ends there at the latest.
template <int V>
__device__ __forceinline__ void look_back(const uint64_t* rec, int newest, int spin_limit,
                                          float (&h)[V]) {
  constexpr int K = 8 / V;  // records in flight per channel
  uint64_t win[K][V];
  auto load = [&](int base) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v)
        win[k][v] = __hip_atomic_load(
            rec + static_cast<int64_t>(base - k > 0 ? base - k : 0) * (64 * V) + v,
            __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  int base = newest;
  for (bool late = false;;) {
    bool found;
    for (int spins = 0;;) {
      load(base);
      bool ready = true;
      found = true;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        bool f = false;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          ready = ready && (f || win[k][v] != 0);
          f = f || (win[k][v] != 0 && (win[k][v] >> 63) == 0);
        }
        found = found && f;
      }
      if (__all(ready)) break;
      if (spins++ >= spin_limit) {
        late = true;
        if ((threadIdx.x & 63) == 0) atomicAdd(&g_gated_timeouts, 1u);
        break;
      }
      __builtin_amdgcn_s_sleep(1);
    }
    if (late || __all(found) || base < K) break;
    base -= K;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.0f;
  for (;;) {
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      if (base - k < 0) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t code = static_cast<uint32_t>(win[k][v] >> 32);
        const float H = __uint_as_float(static_cast<uint32_t>(win[k][v]));
        h[v] = (code >> 31) ? fmaf(__uint_as_float(code & 0x7fffffffu), h[v], H) : H;
      }
    }
    if (base == newest) return;
    base += K;
    load(base);
  }
}

// R rows of V channels per lane as loaded; rows past the last (n of them)
// repeat it.  base and ld are the wave's, off is the lane's byte offset.
template <typename T, int V, int R, bool STREAM>
struct Rows {
  uint32_t w[R];
  __device__ __forceinline__ void load(const void* base, int64_t elem0, int64_t ld, uint32_t off,
                                       int n) {
    const T* row = static_cast<const T*>(base) + elem0;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const T* p = add_bytes(row, off);
      row += j + 1 < n ? ld : 0;
      if constexpr (STREAM)
        w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32_any*>(p));
      else if constexpr (sizeof(T) * V == 4)
        w[j] = *reinterpret_cast<const u32_any*>(p);
      else
        w[j] = *p;
    }
  }
  __device__ __forceinline__ float get(int j, int v) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    return __uint_as_float(V == 2 && v == 1 ? (w[j] & 0xffff0000u) : (w[j] << 16));
  }
};

template <typename T, int V, bool STREAM>
__device__ __forceinline__ void store_row(void* base, int64_t elem, uint32_t off,
                                          const float (&v)[V]) {
  T* p = add_bytes(static_cast<T*>(base) + elem, off);
  if constexpr (sizeof(T) * V == 4) {
    uint32_t t;
    if constexpr (V == 2)
      t = pack_bf16x2(v[0], v[1]);
    else
      t = __float_as_uint(v[0]);
    if constexpr (STREAM)
      __builtin_nontemporal_store(t, reinterpret_cast<u32_any*>(p));
    else
      *reinterpret_cast<u32_any*>(p) = t;
  } else {
    store_act(p, 0, v[0]);
  }
}

// Where a wave works: one run of one channel block.
struct Place {
  int64_t b, t0;     // batch row, first step
  int64_t c0;        // first channel of the block
  int n;             // steps (<= 0: none)
  int chain, chunk;  // channel block over all batch rows; chunk in order of work
};

struct GatedGrid {
  int n_cblk, chains, chunks, waves;
  int* ticket;
  uint64_t* rec;
  float* part;       // backward: dlog_decay of every (batch row, chunk), [..][dim]
  bool stream;       // the arrays' rows are whole cache lines, each read or written once
};

template <int R, bool MULTI, bool REVERSE>
__device__ __forceinline__ Place find_place(const GatedArgs& p, const GatedGrid& g, int w,
                                            int* lds_ticket) {
  int task = blockIdx.x;
  if (MULTI) {
    if (threadIdx.x == 0) *lds_ticket = atomicAdd(g.ticket, 1);
    __syncthreads();
    task = __builtin_amdgcn_readfirstlane(*lds_ticket);
  }
  Place q;
  q.chunk = task / g.chains;
  q.chain = task - q.chunk * g.chains;
  q.b = q.chain / g.n_cblk;
  q.c0 = static_cast<int64_t>(q.chain - static_cast<int>(q.b) * g.n_cblk);
  const int64_t run = static_cast<int64_t>(REVERSE ? g.chunks - 1 - q.chunk : q.chunk) * g.waves + w;
  q.t0 = run * R;
  const int64_t left = p.seqlen - q.t0;
  q.n = left < R ? static_cast<int>(left) : R;
  return q;
}

// Bit j: step j of the run starts a document.
__device__ __forceinline__ uint32_t reset_bits(const GatedArgs& p, const Place& q, int lane) {
  const bool on = lane < q.n && p.reset[q.b * p.seqlen + q.t0 + (lane < q.n ? lane : 0)] != 0;
  return static_cast<uint32_t>(__ballot(on));
}

// What up to CAP waves of a workgroup share.
template <int V, int CAP>
struct Shared {
  float2 agg[CAP][64 * V];  // each run's product of a and state from zero
  float carry[64 * V];
  uint32_t cut[CAP];        // the run holds a reset
  int ticket;
};

// h after the runs k0, k0 + dk, ... (count of them), from h before them.
template <int V, bool RESET, typename S>
__device__ __forceinline__ void fold_runs(const S& sh, int lane, int k0, int dk, int count,
                                          float (&h)[V]) {
  for (int k = k0; count > 0; --count, k += dk) {
    const bool drop = RESET && sh.cut[k];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 ag = sh.agg[k][lane * V + v];
      h[v] = drop ? ag.y : fmaf(ag.x, h[v], ag.y);
    }
  }
}

// The state before a workgroup's chunk, into sh.carry: the chunk's aggregate
// (runs from k0 in steps of dk) is published, the state before it found, and
// the state after it published.  begin: the state before the sequence.  One
// wave's work.
template <int V, bool RESET, typename S>
__device__ __forceinline__ void exchange(const GatedGrid& g, const Place& q, int spin_limit,
                                         int lane, int k0, int dk, const float (&begin)[V], S& sh) {
  uint64_t* rec = g.rec + (static_cast<int64_t>(q.chain) * g.chunks) * (64 * V) + lane * V;
  uint64_t* own = rec + static_cast<int64_t>(q.chunk) * (64 * V);
  const bool last = q.chunk == g.chunks - 1;
  float A[V], H[V], h[V];
  bool drop_any = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    H[v] = 0.0f;
    h[v] = begin[v];
  }
  for (int c = 0, k = k0; c < g.waves; ++c, k += dk) {
    const bool drop = RESET && sh.cut[k];
    drop_any = drop_any || drop;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 ag = sh.agg[k][lane * V + v];
      H[v] = drop ? ag.y : fmaf(ag.x, H[v], ag.y);
      A[v] *= ag.x;
    }
  }
  // after a reset the chunk's end does not depend on what came before
  if (q.chunk && !last) put_records<V>(own, drop_any, A, H);
  if (q.chunk) look_back<V>(rec, q.chunk - 1, spin_limit, h);
  if (!last && !(drop_any && q.chunk)) {
    float end[V];
#pragma unroll
    for (int v = 0; v < V; ++v) end[v] = drop_any ? H[v] : fmaf(A[v], h[v], H[v]);
    put_records<V>(own, true, A, end);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) sh.carry[lane * V + v] = h[v];
}

template <typename T, int V, bool STREAM, bool RESET, bool MULTI>
__global__ __launch_bounds__(64 * kMaxWaves) void gated_fwd_kernel(GatedArgs p, GatedGrid g) {
  constexpr int R = kGatedRun;
  __shared__ Shared<V, kMaxWaves> sh;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t D = p.dim, L = p.seqlen;
  Place q = find_place<R, MULTI, false>(p, g, w, &sh.ticket);
  q.c0 *= 64 * V;
  const bool live = q.c0 + lane * V < D;
  // a dead lane repeats the last channels, and so does the half-filled last lane
  // of an odd dim: it computes and stores what its neighbour does
  const int64_t c = q.c0 + lane * V <= D - V ? q.c0 + lane * V : D - V;
  const int64_t cb = q.c0 <= D - V ? q.c0 : D - V;  // where the block's rows are addressed from
  const uint32_t off = static_cast<uint32_t>((c - cb) * static_cast<int64_t>(sizeof(T)));
  const int n = q.n;

  float lam2[V];
#pragma unroll
  for (int v = 0; v < V; ++v) lam2[v] = p.log_decay[c + v] * kLog2e;
  float first[V];  // the state before the sequence
#pragma unroll
  for (int v = 0; v < V; ++v) first[v] = p.h0 ? p.h0[q.b * D + c + v] : 0.0f;

  float A[R][V], H[R][V];
  uint32_t cut = 0;
  if (n > 0) {
    const int64_t row = q.b * L + q.t0;
    Rows<T, V, R, STREAM> x, r, in;
    r.load(p.r, row * p.ld_r + cb, p.ld_r, off, n);
    in.load(p.i, row * p.ld_i + cb, p.ld_i, off, n);
    x.load(p.x, row * p.ld_x + cb, p.ld_x, off, n);
    if (RESET) cut = reset_bits(p, q, lane);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool at_reset = RESET && (cut >> j & 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float rho, a, beta;
        gate(r.get(j, v), lam2[v], rho, a, beta);
        const float ix = sigmoid_f32(in.get(j, v)) * x.get(j, v);
        if (at_reset) {
          A[j][v] = 0.0f;
          H[j][v] = ix;
        } else if (j == 0) {
          A[j][v] = a;
          H[j][v] = beta * ix;
        } else {
          A[j][v] = A[j - 1][v] * a;
          H[j][v] = fmaf(a, H[j - 1][v], beta * ix);
        }
      }
    }
    if (n < R) {  // steps past the end leave the state alone
#pragma unroll
      for (int j = 1; j < R; ++j)
        if (j >= n) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            A[j][v] = A[j - 1][v];
            H[j][v] = H[j - 1][v];
          }
        }
    }
  } else {
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A[j][v] = 1.0f;
        H[j][v] = 0.0f;
      }
  }
  const int W = g.waves;
  if (MULTI || W > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) sh.agg[w][lane * V + v] = make_float2(A[R - 1][v], H[R - 1][v]);
    if (RESET && lane == 0) sh.cut[w] = cut;
    lds_barrier();
  }
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = first[v];
  if (MULTI) {
    if (w == 0) exchange<V, RESET>(g, q, p.spin_limit, lane, 0, 1, first, sh);
    lds_barrier();
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = sh.carry[lane * V + v];
  }
  fold_runs<V, RESET>(sh, lane, 0, 1, w, h);
  if (n <= 0 || !live) return;
  if (p.ckpt) {
    float* ck = p.ckpt + (q.b * div_up64(L, R) + q.t0 / R) * D + c;
#pragma unroll
    for (int v = 0; v < V; ++v) ck[v] = h[v];
  }
  const int64_t row = q.b * L + q.t0;
  float o[V];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    // after a reset the state before the run does not count, finite or not
    const bool since = RESET && (cut & ((2u << j) - 1)) != 0;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = since ? H[j][v] : fmaf(A[j][v], h[v], H[j][v]);
    if (p.out && j < n) store_row<T, V, STREAM>(p.out, (row + j) * D + cb, off, o);
  }
  if (p.last_state && q.t0 + n == L) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.last_state[q.b * D + c + v] = o[v];
  }
}

// Backward.  With g_t the gradient of h_t: g_t = dout_t + c_{t+1}, c_t = a_t
// g_t, c_L = dlast: the same recurrence from the end, on c.  A wave's run is
// half a checkpoint's (kBwdRun steps, so that what the second pass needs of each
// step, x, dout, a, beta and the state before, leaves two workgroups' registers on
// a CU): it computes the gates into registers, their sigmoids into LDS (computed
// again in the second pass they are a fifth of the kernel's vector instructions:
// 16000 steps of 1536 bfloat16 channels, batch 8, 586 us against 648), and the
// states from the checkpoint, the odd waves through their even neighbour's
// aggregate.  c runs through the chunk and over the chunks as h does forward
// (chunks are taken from the sequence's end).  CAP: 8 or 16 waves, so that the LDS
// of eight (76 KiB with two channels a lane) leaves room for a second workgroup.
constexpr int kBwdRun = kGatedRun / 2;

template <typename T, int V, bool STREAM, bool RESET, bool MULTI, int CAP>
__global__ __launch_bounds__(64 * CAP, 4) void gated_bwd_kernel(GatedArgs p, GatedGrid g) {
  constexpr int R = kBwdRun;
  typedef float Gates __attribute__((ext_vector_type(2 * V)));
  __shared__ Shared<V, CAP> sh;
  __shared__ float s_mid[CAP / 2][64 * V];  // state after an even wave's run
  __shared__ Gates s_gate[CAP][R][64];      // a step's rho and iota
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t D = p.dim, L = p.seqlen;
  Place q = find_place<R, MULTI, true>(p, g, w, &sh.ticket);
  q.c0 *= 64 * V;
  const bool live = q.c0 + lane * V < D;
  const int64_t c = q.c0 + lane * V <= D - V ? q.c0 + lane * V : D - V;
  const int64_t cb = q.c0 <= D - V ? q.c0 : D - V;  // where the block's rows are addressed from
  const uint32_t off = static_cast<uint32_t>((c - cb) * static_cast<int64_t>(sizeof(T)));
  const int n = q.n;
  const int64_t row = q.b * L + q.t0;

  float lam[V], last[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    lam[v] = p.log_decay[c + v];
    last[v] = p.dlast ? p.dlast[q.b * D + c + v] : 0.0f;
  }
  Rows<T, V, R, STREAM> x, dout;
  float a[R][V], beta[R][V], before[R][V], start[V];
  float A[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    H[v] = 0.0f;
  }
  uint32_t cut = 0;
  if (n > 0) {
    Rows<T, V, R, STREAM> r, in;
    r.load(p.r, row * p.ld_r + cb, p.ld_r, off, n);
    in.load(p.i, row * p.ld_i + cb, p.ld_i, off, n);
    x.load(p.x, row * p.ld_x + cb, p.ld_x, off, n);
    dout.load(p.dout, row * D + cb, D, off, n);
    if (RESET) cut = reset_bits(p, q, lane);
#pragma unroll
    for (int v = 0; v < V; ++v)
      start[v] = p.ckpt[(q.b * div_up64(L, kGatedRun) + q.t0 / kGatedRun) * D + c + v];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool at_reset = RESET && (cut >> j & 1);
      Gates gates;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float rho;
        gate(r.get(j, v), lam[v] * kLog2e, rho, a[j][v], beta[j][v]);
        const float io = sigmoid_f32(in.get(j, v));
        gates[v] = at_reset ? 0.0f : rho;  // r is not used there, whatever it holds
        gates[V + v] = io;
        before[j][v] = io * x.get(j, v);
      }
      s_gate[w][j][lane] = gates;
    }
  }
  // the states before each step, from the run's first, in place of iota x
  auto states = [&](float (&h)[V]) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool at_reset = RESET && (cut >> j & 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float ix = before[j][v];
        before[j][v] = h[v];
        h[v] = at_reset ? ix : fmaf(a[j][v], h[v], beta[j][v] * ix);
      }
    }
  };
  const int W = g.waves;
  if ((w & 1) == 0 && n > 0) {
    states(start);
#pragma unroll
    for (int v = 0; v < V; ++v) s_mid[w >> 1][lane * V + v] = start[v];
  }
  if (W > 1) lds_barrier();
  if ((w & 1) == 1 && n > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) start[v] = s_mid[w >> 1][lane * V + v];
    states(start);
  }
  if (n > 0) {
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
      const bool at_reset = RESET && (cut >> j & 1);
      if (j >= n) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        H[v] = at_reset ? 0.0f : a[j][v] * (dout.get(j, v) + H[v]);
        A[v] = at_reset ? 0.0f : A[v] * a[j][v];
      }
    }
  }
  if (MULTI || W > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) sh.agg[w][lane * V + v] = make_float2(A[v], H[v]);
    if (RESET && lane == 0) sh.cut[w] = cut;
    lds_barrier();
  }
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = last[v];
  if (MULTI) {
    if (w == 0) exchange<V, RESET>(g, q, p.spin_limit, lane, W - 1, -1, last, sh);
    lds_barrier();
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = sh.carry[lane * V + v];
  }
  fold_runs<V, RESET>(sh, lane, W - 1, -1, W - 1 - w, h);
  float dlam[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dlam[v] = 0.0f;
  if (n > 0) {
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
      if (j >= n) continue;
      const bool at_reset = RESET && (cut >> j & 1);
      float dx[V], dr[V], di[V];
      const Gates gates = s_gate[w][j][lane];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float xt = x.get(j, v), be = beta[j][v], al = a[j][v];
        const float rho = gates[v], io = gates[V + v];
        const float gt = dout.get(j, v) + h[v];
        const float gi = gt * io;
        h[v] = at_reset ? 0.0f : al * gt;
        dx[v] = at_reset ? gi : gi * be;
        di[v] = dx[v] * xt * (1.0f - io);
        const float inv = be > 0.0f ? rcp_hw(be) : 0.0f;
        const float da = at_reset ? 0.0f : fmaf(h[v], before[j][v], -(al * al * inv) * (gi * xt));
        const float dl = da * rho;
        dr[v] = dl * lam[v] * (1.0f - rho);
        dlam[v] += dl;
      }
      if (live) {
        store_row<T, V, STREAM>(p.dx, (row + j) * D + cb, off, dx);
        store_row<T, V, STREAM>(p.dr, (row + j) * D + cb, off, dr);
        store_row<T, V, STREAM>(p.di, (row + j) * D + cb, off, di);
      }
    }
    if (p.dh0 && q.t0 == 0 && live) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.dh0[q.b * D + c + v] = h[v];
    }
  }
  // the workgroup's dlog_decay, run by run
  lds_barrier();  // the aggregates were read by every wave's fold
#pragma unroll
  for (int v = 0; v < V; ++v) sh.agg[w][lane * V + v].x = dlam[v];
  lds_barrier();
  if (w == 0 && live) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float sum = 0.0f;
      for (int k = 0; k < W; ++k) sum += sh.agg[k][lane * V + v].x;
      g.part[(q.b * g.chunks + q.chunk) * D + c + v] = sum;
    }
  }
}

// out[c] = sum over rows of part[row][c]: 16 waves take every 16th row each,
// eight loads in flight, and their sums are added in order.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* part, int64_t rows,
                                                         int64_t dim, float* out) {
  __shared__ float lds[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const int64_t cc = c < dim ? c : dim - 1;
  float s = 0.0f;
  int64_t q = w;
  for (; q + 7 * 16 < rows; q += 8 * 16) {
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = part[(q + k * 16) * dim + cc];
#pragma unroll
    for (int k = 0; k < 8; ++k) s += t[k];
  }
  for (; q < rows; q += 16) s += part[q * dim + cc];
  lds[w][lane] = s;
  __syncthreads();
  if (w || c >= dim) return;
  s = 0.0f;
  for (int k = 0; k < 16; ++k) s += lds[k][lane];
  out[c] = s;
}

__global__ __launch_bounds__(256) void gated_clear_kernel(uint4* p, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = make_uint4(0, 0, 0, 0);
}

// One step, a thread per channel: 256 x 5120 bfloat16 6.1 us, launch included (21
// MB, 4.1 us of a copy's rate); 8.5 where no cache holds its inputs, float32 10.8
// (31 MB, 6.1 us).
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

static unsigned blocks_of(int64_t n, int64_t per) {
  return static_cast<unsigned>(div_up64(n, per));
}

void launch_column_sum(const float* part, int64_t rows, int64_t dim, float* out,
                       hipStream_t stream) {
  column_sum_kernel<<<blocks_of(dim, 64), 1024, 0, stream>>>(part, rows, dim, out);
}

// Shape of a pass in runs of `run` steps: channels per lane, waves per
// workgroup, channel blocks over all batch rows, chunks per sequence.
struct Cut {
  int v, waves;
  int64_t chains, chunks;
};
// A pass whose workgroups are at most one a CU takes the fewest waves, eight to
// sixteen, for which that holds (2 x 535 steps of 5056 bfloat16 channels: 18.7 us
// so, 21.7 with eight), first with one channel per lane, then, of bfloat16, with
// two where more than 64 channels fill them (64 channels, batch 8, 16000 steps: 44
// us against 30).  Larger ones have two workgroups of eight waves on a CU
// (2.8B-shaped layer 270 us against 324 with sixteen, 301 with four), backward
// sixteen waves up to some 1500 workgroups (2 x 2048 x 2560: 47.5 us against 50.3,
// but 2 x 4096 x 5120 147 against 143).  Where a long sequence has few channel
// blocks, what bounds it is the hop from chunk to chunk (70 ns each), so the
// chunks are large (a million steps of 64 bfloat16 channels: 261 us, 448 with two
// channels per lane, 478 with eight waves, 856 with both; of 256 float32 channels
// 764 us against 912).
// SSM_FORCE_GATED_WAVES overrides (tests, tuning).
static Cut cut_of(int dtype, int64_t batch, int64_t seqlen, int64_t dim, int run) {
  const int64_t runs = div_up64(seqlen, run);
  auto one_a_cu = [&](int64_t chains) {
    for (int w = 8; w <= kMaxWaves; w += 2)
      if (chains * div_up64(runs, w) <= 256) return w;
    return 0;
  };
  Cut c;
  c.v = 1;
  c.chains = batch * div_up64(dim, 64);
  c.waves = one_a_cu(c.chains);
  if (!c.waves && dtype != 0 && dim > 64 && c.chains > 8) {
    c.v = 2;
    c.chains = batch * div_up64(dim, 128);
    c.waves = one_a_cu(c.chains);
  }
  if (!c.waves) {
    const bool few = run == kBwdRun && c.chains * div_up64(runs, kMaxWaves) <= 1500;
    c.waves = c.chains <= 8 || few ? kMaxWaves : 8;
  }
  const char* force = getenv("SSM_FORCE_GATED_WAVES");
  if (force && *force) {
    const int w = atoi(force) & ~1;  // the backward's waves work in pairs
    c.waves = w < 2 ? 2 : (w > kMaxWaves ? kMaxWaves : w);
  }
  c.chunks = div_up64(seqlen, c.waves * run);
  // what sixteen waves hold is one chunk: no records, one launch less
  if (seqlen <= (force && *force ? c.waves : kMaxWaves) * run) {
    c.chunks = 1;
    c.waves = static_cast<int>(div_up64(seqlen, run));
  }
  return c;
}

// Scratch of a pass over chunks: a ticket (16 bytes) and the records.
static int64_t record_bytes(const Cut& c) {
  return c.chunks <= 1 ? 0 : 16 + c.chains * c.chunks * c.v * 64 * 8;
}

int64_t gated_fwd_work(int dtype, int64_t batch, int64_t seqlen, int64_t dim) {
  return record_bytes(cut_of(dtype, batch, seqlen, dim, kGatedRun));
}
int64_t gated_bwd_work(int dtype, int64_t batch, int64_t seqlen, int64_t dim) {
  const Cut c = cut_of(dtype, batch, seqlen, dim, kBwdRun);
  return record_bytes(c) + batch * c.chunks * dim * 4;
}

// Rows that are whole cache lines stream past the caches (16384 steps of 5120
// bfloat16 channels 155 us against 161, backward 299 against 312); parts of lines
// meet in them (9000 steps of 1001 float32 channels, batch 4: 144 us against 166,
// backward 278 against 335).
static bool whole_lines(const GatedArgs& a) {
  const int64_t size = a.dtype == 0 ? 4 : 2;
  uint64_t bits = (a.dim | a.ld_x | a.ld_r | a.ld_i) * size;
  for (const void* t : {a.x, a.r, a.i, a.dout, static_cast<const void*>(a.out),
                        static_cast<const void*>(a.dx), static_cast<const void*>(a.dr),
                        static_cast<const void*>(a.di)})
    bits |= reinterpret_cast<uintptr_t>(t);
  return bits % 128 == 0;
}

static GatedGrid grid_of(const GatedArgs& a, int run, int* v, hipStream_t stream) {
  const Cut c = cut_of(a.dtype, a.batch, a.seqlen, a.dim, run);
  GatedGrid g = {};
  g.n_cblk = static_cast<int>(div_up64(a.dim, 64 * c.v));
  g.chains = static_cast<int>(c.chains);
  g.chunks = static_cast<int>(c.chunks);
  g.waves = c.waves;
  g.stream = whole_lines(a);
  *v = c.v;
  const int64_t bytes = record_bytes(c);
  if (bytes) {
    g.ticket = static_cast<int*>(a.work);
    g.rec = reinterpret_cast<uint64_t*>(static_cast<char*>(a.work) + 16);
    gated_clear_kernel<<<blocks_of(bytes / 16, 256), 256, 0, stream>>>(
        static_cast<uint4*>(a.work), bytes / 16);
  }
  g.part = reinterpret_cast<float*>(static_cast<char*>(a.work) + bytes);
  return g;
}

// LAUNCH(T, V, STREAM, RESET, MULTI)
#define SSM_GATED_BY_TYPE(LAUNCH)                  \
  do {                                             \
    if (a.dtype == 0 && g.stream) {                \
      SSM_GATED_BY_FORM(LAUNCH, float, 1, true);   \
    } else if (a.dtype == 0) {                     \
      SSM_GATED_BY_FORM(LAUNCH, float, 1, false);  \
    } else if (v == 2 && g.stream) {               \
      SSM_GATED_BY_FORM(LAUNCH, bf16_t, 2, true);  \
    } else if (v == 2) {                           \
      SSM_GATED_BY_FORM(LAUNCH, bf16_t, 2, false); \
    } else {                                       \
      SSM_GATED_BY_FORM(LAUNCH, bf16_t, 1, false); \
    }                                              \
  } while (0)
#define SSM_GATED_BY_FORM(LAUNCH, T, V, STREAM)    \
  if (a.reset) {                                   \
    if (g.chunks > 1)                              \
      LAUNCH(T, V, STREAM, true, true);            \
    else                                           \
      LAUNCH(T, V, STREAM, true, false);           \
  } else if (g.chunks > 1) {                       \
    LAUNCH(T, V, STREAM, false, true);             \
  } else {                                         \
    LAUNCH(T, V, STREAM, false, false);            \
  }

hipError_t launch_gated_fwd(const GatedArgs& a, hipStream_t stream) {
  int v;
  const GatedGrid g = grid_of(a, kGatedRun, &v, stream);
  const unsigned grid = static_cast<unsigned>(g.chains) * static_cast<unsigned>(g.chunks);
#define SSM_LAUNCH(...) gated_fwd_kernel<__VA_ARGS__><<<grid, 64 * g.waves, 0, stream>>>(a, g)
  SSM_GATED_BY_TYPE(SSM_LAUNCH);
#undef SSM_LAUNCH
  return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedArgs& a, hipStream_t stream) {
  int v;
  GatedGrid g = grid_of(a, kBwdRun, &v, stream);
  if (a.batch * g.chunks == 1) g.part = a.dlog_decay;  // one row: the sum itself
  const unsigned grid = static_cast<unsigned>(g.chains) * static_cast<unsigned>(g.chunks);
#define SSM_LAUNCH(...)                                                                 \
  if (g.waves <= kMaxWaves / 2)                                                         \
    gated_bwd_kernel<__VA_ARGS__, kMaxWaves / 2><<<grid, 64 * g.waves, 0, stream>>>(a, g); \
  else                                                                                  \
    gated_bwd_kernel<__VA_ARGS__, kMaxWaves><<<grid, 64 * g.waves, 0, stream>>>(a, g)
  SSM_GATED_BY_TYPE(SSM_LAUNCH);
#undef SSM_LAUNCH
  if (a.batch * g.chunks > 1)
    launch_column_sum(g.part, a.batch * g.chunks, a.dim, a.dlog_decay, stream);
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
