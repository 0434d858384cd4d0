// Linear product of 8-bit (e4m3) operands with block scales for gfx950:
//   out[m][n] = sum over blocks kb of 128 inputs of
//               xs[kb][m] ws[n/128][kb] sum_{k in kb} xq[m][k] wq[n][k]  (+ bias[n]),
// and the weights' conversion to that form.

#include <stdlib.h>

#include "layer_device.h"

namespace ssm {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// 16 x 16 outputs summed over 128 inputs: lane l holds 32 of row l % 16's 128
// bytes of either operand (the same 32 of both), and four results: rows
// 4 (l / 16) .. + 3 of a, column l % 16 of b.
//
// The 8-bit matrix instruction does not sum in float32: of 8 consecutive inputs
// it cuts every product, towards zero, to a multiple of 2^(E - 13), where E is the
// largest sum of a pair's exponents among the 8, a subnormal's counting as -6
// (measured with one product beside a larger one; sums of 8 are then added in
// float32).  So up to seven products
// beside a large one lose less than 2^-13 of it each, at worst 7 2^-13 = 2^-10.2
// of the largest product of every 8.  A sum of 2560 normal values is off by 1.5e-5
// of its magnitude; with one input in 128 a thousand times the others the product
// differs from one summed in float32 by less than the bfloat16 output's rounding
// (both 1.6e-3 of the exact one on the norm), but a sum whose terms cancel keeps
// the cut.  EXACT widens the operands to bfloat16, which holds every e4m3 value
// and sums in float32, at half the rate.  It is taken for float32 outputs, and
// where the weights' bytes bound the product in any case (up to 32 tokens).  Tiles
// of bfloat16 outputs keep the 8-bit instruction: 512 x 5120 x 2560 15.6 us
// against 22.9 by the same tiles with EXACT, 2048 x 5120 x 2560 41 against 60.
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

// ---- few tokens: the weights' stream ----
//
// With at most 32 tokens the weights' bytes bound the product, so each is read
// once, straight into the matrix instruction's registers: a workgroup takes 16
// rows of weights, its waves the blocks of 128 inputs in turn (a wave's lanes
// read 4 x 32 bytes of each row's block, whole cache lines); the activations come
// from the L2.  The waves' sums meet in LDS and are added in wave order.  Products
// are summed in float32 for either output type, which costs nothing here.  8
// tokens, 5120 x 2560 weights: 6.6 us, launch included, 3 us of it a call of any
// size; 32 rows a workgroup measured 6.0 there, but 9.0 against 6.7 at 2560 x 5120,
// where they leave most CUs idle, and more blocks in flight a wave nothing.

__device__ __forceinline__ i32x8 load_row(const uint8_t* row, int at, int k) {
  i32x8 v = {};
  if (at < k) {
    const int4 t = *reinterpret_cast<const int4*>(row + at);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  }
  if (at + 16 < k) {
    const int4 t = *reinterpret_cast<const int4*>(row + at + 16);
    v[4] = t.x; v[5] = t.y; v[6] = t.z; v[7] = t.w;
  }
  return v;
}

template <typename T, int MT>
__global__ __launch_bounds__(1024) void fp8_stream_kernel(LinearArgs p) {
  __shared__ f32x4 s_sum[16][MT][64];
  const int lane = threadIdx.x & 63, i = lane & 15, quad = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int W = blockDim.x >> 6;
  const int k = static_cast<int>(p.k), groups = (k + kFp8Group - 1) / kFp8Group;
  const int rows = static_cast<int>(p.rows);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const uint8_t* wrow = p.wq + (n0 + i < p.n ? n0 + i : p.n - 1) * p.k;
  const uint8_t* xrow[MT];
  int tok[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    tok[m] = m * 16 + i < rows ? m * 16 + i : rows - 1;
    xrow[m] = p.xq + tok[m] * p.k;
  }
  const float* sw = p.w_scale + (n0 / kFp8Group) * groups;  // 16 rows lie in one tile
  f32x4 acc[MT] = {};
  for (int g = w; g < groups; g += W) {
    const int at = g * kFp8Group + quad * 32;
    const i32x8 a = load_row(wrow, at, k);
    i32x8 b[MT];
    float mult[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      b[m] = load_row(xrow[m], at, k);
      mult[m] = p.x_scale[static_cast<int64_t>(g) * rows + tok[m]] * sw[g];
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const f32x4 d = mfma_fp8<true>(a, b[m]);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][j] = fmaf(d[j], mult[m], acc[m][j]);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) s_sum[w][m][lane] = acc[m];
  __syncthreads();
  const bool whole = p.n % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % (4 * sizeof(T)) == 0;
  for (int t = w; t < MT; t += W) {
    f32x4 v = s_sum[0][t][lane];
    for (int q = 1; q < W; ++q) v += s_sum[q][t][lane];
    const int m = t * 16 + i;
    const int64_t n = n0 + quad * 4;
    if (m >= rows || n >= p.n) continue;
    const int last = static_cast<int>(p.n - n < 4 ? p.n - n - 1 : 3);
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = v[j] + (p.bias ? p.bias[n + (j < last ? j : last)] : 0.0f);
    store_run<T, 4>(static_cast<T*>(p.out) + m * p.n + n, o, whole, last);
  }
}

// ---- tiles: large M ----
//
// A workgroup computes BN outputs of BM tokens, a block of 128 inputs at a time.
// Both operands' blocks go from global memory straight to LDS (16 bytes a lane),
// two blocks' buffers in turn.  LDS rows are the 128 bytes of a row's block as 8
// chunks of 16, chunk c at place c ^ key(row), so that the lanes that read at a
// time hit different banks.
//
// The weights are the matrix instruction's first operand, so a lane holds four
// consecutive outputs of one token, and one multiplier (the token's scale times
// the weight tile's) serves every result of a token column: four FMAs per matrix
// instruction, issued two instructions later.  Weight row i of tile t is output
// (t / 2) 32 + (i / 4) 8 + (t % 2) 4 + i % 4 of the wave's: two tiles give a lane
// 8 consecutive outputs to store.
//
// The barrier of a block stands before its last row of tiles, when every operand
// of the block has been read from LDS: behind it the buffer takes the block after
// next, and the next block's first operands are read while the last row is
// multiplied.
//
// Tiles of 128 outputs by 256 tokens (ONE) keep a single buffer for the tokens,
// whose block is in registers once its first row of tiles is multiplied: a second
// barrier there, and it takes the next block.  So two workgroups fit a CU, each
// multiplying while the other waits, starts or stores.
//
// 32768 x 5120 x 2560: bfloat16 outputs 384 to 429 us by box, 2.1 PFLOP/s, where a library
// product without block scales takes 301; the matrix pipes are busy half the time
// (343 us without loads in the loop, 353 without stores, 22 fewer without the
// scales' FMAs).  float32 outputs, at half the matrix rate, 786 to 847.

typedef const __attribute__((address_space(1))) void* global_ptr;
typedef __attribute__((address_space(3))) void* lds_ptr;

// A 16-byte read is served 16 lanes at a time from 64 banks, two rows' worth, so
// the 8 even rows of a tile and the 8 odd ones each have keys of their own; and
// the lanes served together can belong to two neighbouring quads (whose chunks
// differ by 2), the middle 8 rows to one and the outer 8 to the other, so the
// middle rows' keys are 0 .. 3 and the outer ones' 4 .. 7, sets that stay apart
// under an exclusive or of either.  pair: half the row's number in the tile.
__device__ __forceinline__ int key_of(int pair) { return ((pair + 2) & 7) ^ 4; }
__device__ __forceinline__ int key_w(int row) { return key_of(((row >> 2) & 6) | ((row >> 1) & 1)); }
__device__ __forceinline__ int key_x(int row) { return key_of((row >> 1) & 7); }

// What a lane loads for a place past a row's end.
__device__ const uint4 g_zeros = {0, 0, 0, 0};

// One operand's block of ROWS rows to LDS, 8 rows per wave at a time.
template <int ROWS, int WAVES, bool WEIGHTS>
struct Loader {
  static constexpr int kRounds = ROWS / (8 * WAVES);
  uint32_t off[kRounds];  // the lane's bytes, from the operand's rows and block
  // place of the lane's chunk in a row's block, round j
  __device__ __forceinline__ static int place(int j, int wave, int lane) {
    const int r = (j * WAVES + wave) * 8 + (lane >> 3);
    return ((lane & 7) ^ (WEIGHTS ? key_w(r) : key_x(r))) * 16;
  }
  __device__ __forceinline__ void init(int wave, int lane, int64_t row0, int64_t rows, int64_t k) {
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      const int r = (j * WAVES + wave) * 8 + (lane >> 3);
      const int64_t row = row0 + r < rows ? r : rows - 1 - row0;  // past the end: the last row
      off[j] = static_cast<uint32_t>(row * k + place(j, wave, lane));
    }
  }
  // left: bytes of a row from the block's start; what lies past them is zero in LDS
  __device__ __forceinline__ void load(const uint8_t* block, uint8_t* lds, int wave, int lane,
                                       int left) const {
    if (left >= kFp8Group) {
#pragma unroll
      for (int j = 0; j < kRounds; ++j)
        __builtin_amdgcn_global_load_lds((global_ptr)(block + off[j]),
                                         (lds_ptr)(lds + (j * WAVES + wave) * 1024), 16, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < kRounds; ++j) {
        const uint8_t* from = block + off[j];
        if (place(j, wave, lane) >= left) from = reinterpret_cast<const uint8_t*>(&g_zeros);
        __builtin_amdgcn_global_load_lds((global_ptr)from,
                                         (lds_ptr)(lds + (j * WAVES + wave) * 1024), 16, 0, 0);
      }
    }
  }
};

// A lane's 32 bytes of a row's block, as two chunks.  One sum of integers per
// access: the compiler then still sees which LDS object it is in.
__device__ __forceinline__ i32x8 read_lds(const uint8_t* obj, uint32_t lo, uint32_t hi) {
  const int4 u = *reinterpret_cast<const int4*>(obj + lo);
  const int4 v = *reinterpret_cast<const int4*>(obj + hi);
  return i32x8{u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
}

// Place of the workgroup's tile: consecutive workgroups go to the 8 XCDs in
// turn, so each XCD gets a range of tiles of its own, walked in strips of four
// token tiles by all output tiles, so that the tiles an XCD has in flight share
// their rows in its L2.
__device__ __forceinline__ void tile_of(int64_t tiles_m, int64_t tiles_n, int64_t* tm, int64_t* tn) {
  const int64_t tiles = tiles_m * tiles_n, bid = blockIdx.x;
  const int64_t xcd = bid % 8, each = tiles / 8, more = tiles % 8;
  const int64_t t = xcd * each + (xcd < more ? xcd : more) + bid / 8;
  const int64_t strip = t / (4 * tiles_n), m0 = strip * 4;
  const int64_t high = tiles_m - m0 < 4 ? tiles_m - m0 : 4, in = t - strip * 4 * tiles_n;
  *tm = m0 + in % high;
  *tn = in / high;
}

template <typename T, int BN, int BM, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM, 2) void fp8_tile_kernel(LinearArgs p) {
  constexpr int WAVES = WN * WM, NT = BN / WN / 16, MT = BM / WM / 16;
  constexpr bool EXACT = sizeof(T) == 4, ONE = BM > BN;
  // separate objects, so that reads of one are known not to wait for loads into another
  __shared__ __align__(1024) uint8_t s_w0[BN * kFp8Group];
  __shared__ __align__(1024) uint8_t s_w1[BN * kFp8Group];
  __shared__ __align__(1024) uint8_t s_x0[BM * kFp8Group];
  __shared__ __align__(1024) uint8_t s_x1[ONE ? 16 : BM * kFp8Group];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % WN, wm = wave / WN;
  int64_t tm, tn;
  tile_of(div_up64(p.rows, BM), div_up64(p.n, BN), &tm, &tn);
  const int64_t n0 = tn * BN, m0 = tm * BM;
  // with the inputs split over gridDim.y workgroups: blocks first .. first + groups - 1
  const int all = static_cast<int>(div_up64(p.k, kFp8Group)), part = blockIdx.y;
  const int each = (all + gridDim.y - 1) / gridDim.y, first = part * each;
  const int groups = all - first < each ? all - first : each;
  const int k = static_cast<int>(p.k) - first * kFp8Group;  // inputs from the first block on

  Loader<BN, WAVES, true> lw;
  Loader<BM, WAVES, false> lx;
  lw.init(wave, lane, n0, p.n, p.k);
  lx.init(wave, lane, m0, p.rows, p.k);
  const uint8_t* gw = p.wq + n0 * p.k + first * kFp8Group;
  const uint8_t* gx = p.xq + m0 * p.k + first * kFp8Group;
  const float* x_scale = p.x_scale + first * p.rows;
  const int64_t nw = n0 + wn * (BN / WN);  // the wave's first output, in one tile of weights
  const float* sw = p.w_scale + (nw < p.n ? nw / kFp8Group : 0) * all + first;
  uint32_t sx_off[MT];  // bytes of the lane's tokens' scales in a block's row of them
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t tok = m0 + (wm * MT + m) * 16 + (lane & 15);
    sx_off[m] = static_cast<uint32_t>((tok < p.rows ? tok : p.rows - 1) * 4);
  }

  f32x4 acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = f32x4{};

  lw.load(gw, s_w0, wave, lane, k);
  lx.load(gx, s_x0, wave, lane, k);
  // the multipliers of block 0, and the scales of block 1
  float mult[MT], raw[MT];
  const int second = groups > 1 ? 1 : 0;
  float wscale = sw[second];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mult[m] = *add_bytes(x_scale, sx_off[m]) * sw[0];
    raw[m] = *add_bytes(x_scale + second * p.rows, sx_off[m]);
  }
  __syncthreads();
  if (groups > 1) {
    lw.load(gw + kFp8Group, s_w1, wave, lane, k - kFp8Group);
    if constexpr (!ONE) lx.load(gx + kFp8Group, s_x1, wave, lane, k - kFp8Group);
  }

  const int i = lane & 15, quad = lane >> 4;
  const int w_row = wn * (BN / WN) + (i >> 2) * 8 + (i & 3), x_row = wm * (BM / WM) + i;
  const uint32_t w_lo = w_row * kFp8Group + ((quad * 2) ^ key_w(w_row)) * 16;
  const uint32_t w_hi = w_row * kFp8Group + ((quad * 2 + 1) ^ key_w(w_row)) * 16;
  const uint32_t x_lo = x_row * kFp8Group + ((quad * 2) ^ key_x(x_row)) * 16;
  const uint32_t x_hi = x_row * kFp8Group + ((quad * 2 + 1) ^ key_x(x_row)) * 16;
  // row tile n of the wave's weights, token tile m of its activations
  auto read_w = [&](const uint8_t* obj, int n) {
    const uint32_t at = ((n >> 1) * 32 + (n & 1) * 4) * kFp8Group;
    return read_lds(obj, w_lo + at, w_hi + at);
  };
  auto read_x = [&](const uint8_t* obj, int m) {
    const uint32_t at = m * 16 * kFp8Group;
    return read_lds(obj, x_lo + at, x_hi + at);
  };
  i32x8 a[2], b[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) b[m] = read_x(s_x0, m);
  a[0] = read_w(s_w0, 0);

  // Block g from (cw, cx), its first operands already read; the next is in (ow,
  // ox).  Product t's sums follow product t + 2, when its result is there, and
  // the order is fixed as written (left to itself the compiler reads a row's
  // operands just before they are needed).
  auto step = [&](int g, uint8_t* cw, uint8_t* cx, const uint8_t* ow, const uint8_t* ox) {
    f32x4 d[3];
    auto add = [&](int t) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[t / MT][t % MT][j] = fmaf(d[t % 3][j], mult[t % MT], acc[t / MT][t % MT][j]);
      // the sum is taken here: moved past later products, it would keep their
      // results in registers of their own
      asm volatile("" : "+v"(acc[t / MT][t % MT]));
    };
#pragma unroll
    for (int t = 0; t < NT * MT; ++t) {
      const int n = t / MT, m = t % MT;
      if (m == 0) {
        if (ONE && n == 1 && g + 1 < groups) {
          // every wave's tokens are in registers: LDS reads only are waited for
          lds_barrier();
          const int at = (g + 1) * kFp8Group;
          lx.load(gx + at, cx, wave, lane, k - at);
        }
        if (n + 1 < NT) {
          a[(n + 1) & 1] = read_w(cw, n + 1);
        } else {
          __syncthreads();
          a[NT & 1] = read_w(ow, 0);
        }
      }
      d[t % 3] = mfma_fp8<EXACT>(a[n & 1], b[m]);
      if (n + 1 == NT) b[m] = read_x(ox, m);
      if (t >= 2) add(t - 2);
      __builtin_amdgcn_sched_barrier(0);
    }
    add(NT * MT - 2);
    add(NT * MT - 1);
#pragma unroll
    for (int m = 0; m < MT; ++m) mult[m] = raw[m] * wscale;
    const int late = g + 2 < groups ? g + 2 : groups - 1;
    wscale = sw[late];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      asm volatile("" : "+v"(sx_off[m]));  // stays an offset: no 64-bit sum per token
      raw[m] = *add_bytes(x_scale + static_cast<int64_t>(late) * p.rows, sx_off[m]);
    }
    if (g + 2 < groups) {
      const int at = (g + 2) * kFp8Group;
      lw.load(gw + at, cw, wave, lane, k - at);
      if constexpr (!ONE) lx.load(gx + at, cx, wave, lane, k - at);
    }
  };
  uint8_t* const x1 = ONE ? s_x0 : s_x1;
  int g = 0;
  for (; g + 1 < groups; g += 2) {
    step(g, s_w0, s_x0, s_w1, x1);
    step(g + 1, s_w1, x1, s_w0, s_x0);
  }
  if (g < groups) step(g, s_w0, s_x0, s_w1, x1);

  // Of bfloat16 outputs the wave's tile goes through LDS, where the operands were,
  // so that whole rows of it leave at a time: a lane's own 8 outputs of a token
  // leave in pieces of 64 bytes (12911 x 1153 x 1152: 29 us against 47, 32768 x
  // 5120 x 2560: 404 against 418; float32's pieces of 128 bytes are as fast).  Rows
  // are chunks of 16 bytes, chunk c at c ^ key(token): the 16 lanes that write or
  // read at a time hit different banks.
  auto store = [&](auto* out, const float* bias_of) __attribute__((always_inline)) {
    using O = typename std::remove_reference<decltype(*out)>::type;
    constexpr int N = NT * 16, M = MT * 16;           // the wave's tile
    constexpr int C = N / 8;                          // chunks of a row
    if (bias_of) {
#pragma unroll
      for (int t = 0; t < NT / 2; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t n = nw + t * 32 + quad * 8 + e;
          const float bias = bias_of[n < p.n ? n : p.n - 1];
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[t * 2 + e / 4][m][e % 4] += bias;
        }
    }
    if constexpr (sizeof(O) == 2) {
      constexpr int kBytes = N * M * 2;
      constexpr int kPer = BN * kFp8Group / kBytes;  // waves' tiles in an operand's buffer
      static_assert(ONE ? BM == 2 * BN && kPer * 4 == WAVES : BN == BM && kPer * 4 >= WAVES,
                    "room for every wave's tile");
      const int at = wave / kPer;
      uint8_t* lds = at == 0 ? s_w0 : at == 1 ? s_w1 : at == 2 ? s_x0 : ONE ? s_x0 + kPer * kBytes : s_x1;
      lds += wave % kPer * kBytes;
      auto key = [](int tok) { return tok / (16 / C) & (C - 1); };
      __syncthreads();  // no wave reads operands any more
#pragma unroll
      for (int t = 0; t < NT / 2; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int tok = m * 16 + i;
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = acc[t * 2 + e / 4][m][e % 4];
          *reinterpret_cast<u32x4*>(lds + tok * (C * 16) + ((t * 4 + quad) ^ key(tok)) * 16) =
              u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7])};
        }
#pragma unroll
      for (int f0 = 0; f0 < M * C; f0 += 64) {
        const int f = f0 + lane, tok = f / C, c = f % C;
        const u32x4 v = *reinterpret_cast<const u32x4*>(lds + tok * (C * 16) + (c ^ key(tok)) * 16);
        const int64_t row = m0 + wm * M + tok, n = nw + c * 8;
        if (row >= p.rows || n >= p.n) continue;
        O* to = out + row * p.n + n;
        if (n + 8 <= p.n) {
          // the largest tiles' outputs exceed the caches: they stream past them
          if constexpr (BM == 256)
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(to));
          else
            *reinterpret_cast<u32x4_any*>(to) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (n + e < p.n) to[e] = static_cast<O>(v[e / 2] >> (16 * (e % 2)));
        }
      }
    } else {
#pragma unroll
      for (int t = 0; t < NT / 2; ++t) {
        const int64_t n = nw + t * 32 + quad * 8;
        if (n >= p.n) continue;
        const int last = static_cast<int>(p.n - n < 8 ? p.n - n - 1 : 7);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int64_t tok = m0 + (wm * MT + m) * 16 + i;
          if (tok >= p.rows) continue;
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = acc[t * 2 + e / 4][m][e % 4];
          store8(out + tok * p.n + n, v, last);
        }
      }
    }
  };
  if (gridDim.y == 1)
    store(static_cast<T*>(p.out), p.bias);
  else
    store(static_cast<float*>(p.work) + part * p.rows * p.n, static_cast<const float*>(nullptr));
}

// Joins the parts of a product whose inputs were split, in order.
template <typename T>
__global__ __launch_bounds__(256) void fp8_join_kernel(LinearArgs p, int parts) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4, all = p.rows * p.n;
  if (at >= all) return;
  const float* part = static_cast<const float*>(p.work);
  const int last = static_cast<int>(all - at < 4 ? all - at - 1 : 3);
  float v[4] = {};
  if (all % 4 == 0) {
    for (int q = 0; q < parts; ++q) {
      const float4 t = *reinterpret_cast<const float4*>(part + q * all + at);
      v[0] += t.x; v[1] += t.y; v[2] += t.z; v[3] += t.w;
    }
  } else {
    for (int q = 0; q < parts; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += part[q * all + at + (e < last ? e : last)];
  }
  if (p.bias) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += p.bias[(at + (e < last ? e : last)) % p.n];
  }
  const bool whole = all % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % (4 * sizeof(T)) == 0;
  store_run<T, 4>(static_cast<T*>(p.out) + at, v, whole, last);
}

// One workgroup per tile of 128 x 128 weights, which stays in registers (runs of 8
// of a row, 16 rows at a time) between its maximum and the conversion: read once,
// written once: 10240 x 10240 float32 98 us, 5.3 TB/s.
// TAIL: k is no multiple of 8.
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

template <typename T, bool TAIL>
__global__ __launch_bounds__(256) void quantize_weight_kernel(const T* w, int64_t n, int64_t k,
                                                              uint8_t* q, float* scale) {
  __shared__ float lds[4];
  const int64_t groups = div_up64(k, kFp8Group);
  const int64_t tn = blockIdx.x / groups, tk = blockIdx.x % groups;
  const int64_t r0 = tn * kFp8Group, c = tk * kFp8Group + (threadIdx.x & 15) * 8;
  const int rows = static_cast<int>(n - r0 < kFp8Group ? n - r0 : kFp8Group);
  const int first = threadIdx.x >> 4, last = static_cast<int>(k - c < 8 ? k - c - 1 : 7);
  Run8<T> v[8];
  float m = 0.0f;
  if (c < k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // past the end: the last row, and its last value, again
      const int row = first + 16 * j < rows ? first + 16 * j : rows - 1;
      const T* from = w + (r0 + row) * k + c;
      if (TAIL && last < 7)
        v[j].load_elems(from, last);
      else
        v[j].load(from);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[j].get(e)));
  }
  m = row16_max(m);
  m = fmaxf(fmaxf(read_lane(m, 0), read_lane(m, 16)), fmaxf(read_lane(m, 32), read_lane(m, 48)));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3])), kFp8AmaxFloor);
  if (threadIdx.x == 0) scale[blockIdx.x] = m / kFp8Max;
  if (c >= k) return;
  const Fp8Scaler to(m);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (first + 16 * j >= rows) return;
    uint8_t* at = q + (r0 + first + 16 * j) * k + c;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = to(v[j].get(e));
    const uint32_t lo = pack_fp8x4(y[0], y[1], y[2], y[3]), hi = pack_fp8x4(y[4], y[5], y[6], y[7]);
    if (TAIL && last < 7) {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e <= last) at[e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e % 4)));
    } else {
      *reinterpret_cast<u32x2_any*>(at) = u32x2_any{lo, hi};
    }
  }
}

enum Shape : int { kStream = 0, kTile64 = 1, kTile128 = 2, kTile256 = 3, kTile128x256 = 4 };
constexpr int64_t kStreamRows = 32;  // most tokens of the streaming kernel

struct Plan {
  int shape, parts;
};

static int forced(const char* name) {
  const char* v = getenv(name);
  return v && *v ? atoi(v) : -1;
}

// Few tokens stream the weights.  More take the largest tile of which there are
// enough: with fewer tiles than CUs, the smaller tile's larger share of loads
// costs less than the idle CUs (bfloat16 outputs: 160 tiles of 256 x 256 36 us
// where 640 of 128 x 128 take 42, but 80 take 60 against 40; 320 of 128 x 128 23.5
// us against 31 for 64 x 64, 160 36 against 30; float32 outputs: 480 of 128 x 128
// 43 us against 53, 320 44 against 41).  Tiles of 256 x 256 come one a CU at a
// time, so where their last round leaves more than a tenth of the CUs idle, tiles
// of 128 x 256, two a CU, are taken: 4096 x 5120 x 2560 (1.25 rounds) 61 us against
// 72, 8192 x 2560 x 5120 (1.25) 112 against 128, 8192 x 5120 x 2560 (2.5) 97
// against 108; but 32768 x 5120 x 2560 (10) 388 against 384.
//
// 64 x 64 tiles may split the inputs into parts.  Measured: about 0.42 us a
// block; for the join 2 us, its traffic, written and read at 2.5 TB/s, and its
// launch on the host, which takes another 2 from a caller that launches one call
// after the other; the least sum of the two is taken.  SSM_FORCE_LINEAR_SHAPE and _PARTS override
// (tests, tuning).
static Plan plan_of(int dtype, int64_t rows, int64_t n, int64_t k) {
  Plan q = {kStream, 1};
  const int shape = forced("SSM_FORCE_LINEAR_SHAPE"), parts = forced("SSM_FORCE_LINEAR_PARTS");
  const int64_t groups = div_up64(k, kFp8Group);
  auto tiles = [&](int64_t side) { return div_up64(n, side) * div_up64(rows, side); };
  if (rows > kStreamRows) {
    if (dtype != 0 && tiles(256) >= 150) {
      const int64_t t = tiles(256), rounds = div_up64(t, 256);
      q.shape = rounds > 1 && 10 * t < 9 * 256 * rounds ? kTile128x256 : kTile256;
    } else if (tiles(128) >= (dtype == 0 ? 384 : 256)) {
      q.shape = kTile128;
    } else {
      q.shape = kTile64;
      double best = 0.0;
      for (int t = 1; t <= 8 && t <= groups; ++t) {
        const double blocks = static_cast<double>(div_up64(groups, t)) * div_up64(tiles(64) * t, 512);
        const double us = 0.42 * blocks + (t > 1 ? 4.0 + 8e-6 / 2.5 * rows * n * t : 0.0);
        if (t == 1 || us < best) {
          best = us;
          q.parts = t;
        }
      }
    }
  }
  if (shape >= 0 && shape <= kTile128x256 && (shape != kStream || rows <= kStreamRows) &&
      (shape < kTile256 || dtype != 0)) {
    q.shape = shape;
    q.parts = 1;
  }
  if (q.shape != kStream && parts > 0) q.parts = parts;
  if (q.parts > groups) q.parts = static_cast<int>(groups);
  // every part has a block: with each = ceil(groups / parts), drop the empty ones
  q.parts = static_cast<int>(div_up64(groups, div_up64(groups, q.parts)));
  return q;
}

int64_t fp8_linear_work(int dtype, int64_t rows, int64_t n, int64_t k) {
  const Plan q = plan_of(dtype, rows, n, k);
  return q.parts > 1 ? q.parts * rows * n * 4 : 0;
}

template <typename T, int MT>
static void launch_stream(const LinearArgs& a, hipStream_t stream) {
  const int64_t groups = div_up64(a.k, kFp8Group);
  // up to 16 waves, as many as give each the same number of blocks
  const int waves = static_cast<int>(div_up64(groups, div_up64(groups, 16)));
  fp8_stream_kernel<T, MT>
      <<<static_cast<unsigned>(div_up64(a.n, 16)), 64 * waves, 0, stream>>>(a);
}

template <typename T, int BN, int BM, int WN, int WM>
static void launch_tiles(const LinearArgs& a, int parts, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(div_up64(a.n, BN) * div_up64(a.rows, BM)), parts);
  fp8_tile_kernel<T, BN, BM, WN, WM><<<grid, 64 * WN * WM, 0, stream>>>(a);
  if (parts > 1)
    fp8_join_kernel<T>
        <<<static_cast<unsigned>(div_up64(a.rows * a.n, 1024)), 256, 0, stream>>>(a, parts);
}

template <typename T>
static void launch_linear_typed(const LinearArgs& a, hipStream_t stream) {
  const Plan q = plan_of(a.dtype, a.rows, a.n, a.k);
  switch (q.shape) {
    case kStream:
      if (a.rows <= 16) launch_stream<T, 1>(a, stream);
      else launch_stream<T, 2>(a, stream);
      break;
    case kTile64: launch_tiles<T, 64, 64, 2, 2>(a, q.parts, stream); break;
    case kTile128: launch_tiles<T, 128, 128, 2, 2>(a, q.parts, stream); break;
    // bfloat16 outputs only (float32 ones' widened operands do not fit the registers)
    case kTile256:
      if constexpr (sizeof(T) == 2) launch_tiles<T, 256, 256, 2, 4>(a, q.parts, stream);
      break;
    default:
      if constexpr (sizeof(T) == 2) launch_tiles<T, 128, 256, 1, 4>(a, q.parts, stream);
  }
}

hipError_t launch_fp8_linear(const LinearArgs& a, hipStream_t stream) {
  if (a.dtype == 0)
    launch_linear_typed<float>(a, stream);
  else
    launch_linear_typed<bf16_t>(a, stream);
  return hipGetLastError();
}

template <typename T>
static void launch_quantize_typed(const void* w, int64_t n, int64_t k, uint8_t* q, float* scale,
                                  hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(div_up64(n, kFp8Group) * div_up64(k, kFp8Group));
  const T* from = static_cast<const T*>(w);
  if (k % 8)
    quantize_weight_kernel<T, true><<<grid, 256, 0, stream>>>(from, n, k, q, scale);
  else
    quantize_weight_kernel<T, false><<<grid, 256, 0, stream>>>(from, n, k, q, scale);
}

hipError_t launch_quantize_weight(const void* w, int dtype, int64_t n, int64_t k, uint8_t* q,
                                  float* scale, hipStream_t stream) {
  if (dtype == 0)
    launch_quantize_typed<float>(w, n, k, q, scale, stream);
  else
    launch_quantize_typed<bf16_t>(w, n, k, q, scale, stream);
  return hipGetLastError();
}

}  // namespace ssm
