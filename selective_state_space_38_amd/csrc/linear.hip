// Linear product with bias, activation and residual for gfx950, of one matrix or of
// one matrix per expert over the rows of each, and its gradient:
//   pre[r][m] = sum_k x[r][k] w[m][k] + bias[m],   out = act(pre) (+ residual),
//   dpre = act'(pre) dout,   dx = dpre w,   dw = dpre^T x,   dbias = sum_r dpre.
// Built once for float32 and once for bfloat16 activations (SSM_LINEAR_DTYPE); all
// sums are float32.

#include "feed_internal.h"
#include "layer_device.h"

#ifndef SSM_LINEAR_DTYPE
#error "SSM_LINEAR_DTYPE is 0 (float32) or 1 (bfloat16)"
#endif

namespace ssm {
namespace {

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

#if SSM_LINEAR_DTYPE == 0
using Act = float;
#else
using Act = bf16_t;
#endif
constexpr int kSize = sizeof(Act);
constexpr int kBlockBytes = 128;               // of a row, in a block of the summed axis
constexpr int kBlock = kBlockBytes / kSize;    // values of it: 64 bfloat16, 32 float32

// ---- activations ----

// Phi(v), the normal distribution function: its tail beyond |v| is
// exp(-v^2 / 2) t P(t), t = 1 / (1 + 0.21 |v|), P fitted to erfcx by weighted least
// squares over t in (0, 1] (relative error 2e-8 before rounding).
__device__ __forceinline__ float normal_cdf(float v) {
  const float z = fabsf(v), t = rcp_hw(fmaf(0.21f, z, 1.0f));
  float p = -7.166303470e-02f;
  p = fmaf(p, t, 2.836218028e-01f);
  p = fmaf(p, t, -3.303235851e-01f);
  p = fmaf(p, t, 3.494836718e-01f);
  p = fmaf(p, t, -9.398447824e-02f);
  p = fmaf(p, t, 1.248991949e-01f);
  p = fmaf(p, t, 6.918498976e-02f);
  p = fmaf(p, t, 8.506993906e-02f);
  p = fmaf(p, t, 8.371150652e-02f);
  const float tail = p * t * exp2_hw(-0.5f * kLog2e * z * z);
  return v < 0.0f ? tail : 1.0f - tail;
}

// f(v), f silu (silu, swiglu) or gelu (gelu, geglu).
constexpr bool is_silu(int act) { return act == kSilu || act == kSwiglu; }
template <bool SILU>
__device__ __forceinline__ float bend_as(float v) {
  return v * (SILU ? sigmoid_f32(v) : normal_cdf(v));
}
__device__ __forceinline__ float bend(int act, float v) {
  return is_silu(act) ? bend_as<true>(v) : bend_as<false>(v);
}
// f(v), and its derivative in *slope.
__device__ __forceinline__ float bend_grad(int act, float v, float* slope) {
  if (is_silu(act)) {
    const float g = sigmoid_f32(v), f = v * g;
    *slope = fmaf(f, 1.0f - g, g);
    return f;
  }
  const float g = normal_cdf(v);
  *slope = fmaf(v * 0.3989422804f, exp2_hw(-0.5f * kLog2e * v * v), g);
  return v * g;
}

// ---- which rows are whose ----

// Rows [from, to) of expert e.  What offsets hold is the caller's: kept within the
// rows, so that wrong ones read and write nothing outside.
struct Range {
  int64_t from, to;
};
__device__ __forceinline__ Range rows_of(const int32_t* offsets, int e, int64_t rows) {
  if (!offsets) return {0, rows};
  const int64_t a = offsets[e], b = offsets[e + 1];
  const int64_t from = a < 0 ? 0 : a > rows ? rows : a;
  return {from, b < from ? from : b > rows ? rows : b};
}

// Tiles of BM rows, expert by expert: their number, and (find) the expert and the
// place in it of tile `tile`.  The whole wave works on it, 64 experts at a time.
struct Tiles {
  const int32_t* offsets;
  int experts;
  int64_t rows;
  int bm;
  __device__ __forceinline__ int count(int e) const {
    if (e >= experts) return 0;
    const Range r = rows_of(offsets, e, rows);
    return static_cast<int>((r.to - r.from + bm - 1) / bm);
  }
  __device__ __forceinline__ static int running(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int up = __shfl_up(v, d);
      if (lane >= d) v += up;
    }
    return v;
  }
  __device__ __forceinline__ int total() const {
    if (!offsets) return static_cast<int>((rows + bm - 1) / bm);
    int sum = 0;
    for (int e0 = 0; e0 < experts; e0 += 64)
      sum += __builtin_amdgcn_readlane(running(count(e0 + (threadIdx.x & 63))), 63);
    return sum;
  }
  // *at: the tile's number among its expert's; false if there is no such tile
  __device__ __forceinline__ bool find(int tile, int* expert, int* at) const {
    *expert = 0;
    *at = tile;
    if (!offsets) return tile < (rows + bm - 1) / bm;
    int before = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
      const int own = count(e0 + (threadIdx.x & 63)), upto = before + running(own);
      const uint64_t past = __ballot(upto > tile);
      if (past) {
        const int who = __builtin_ctzll(past);
        *expert = e0 + who;
        *at = tile - __builtin_amdgcn_readlane(upto - own, who);
        return true;
      }
      before = __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
  }
};

// ---- tiles of the product ----
//
// D[row][column] = sum over an axis of b's row with a's column, by 16 x 16 tiles of
// the matrix instruction.  The operands' blocks of 128 bytes of a row go from
// global memory straight to LDS (16 bytes a lane), two blocks' buffers in turn.
//
//            columns (a)                rows (b)               summed axis
//   kFwd     w's rows                   x's rows               k
//   kGlu     w's rows, gate and up      x's rows               k
//   kDx      w's columns                dpre's rows            w's rows
//   kDw      x's columns                dpre's columns         the expert's rows
//
// An operand whose rows run along the summed axis stands in LDS as rows of 128
// bytes, chunk c of 16 at place c ^ key(row); a lane reads 32 bytes of a row, its
// quad's share of the block.  One whose columns do stands as it is in memory, a
// block's rows of the summed axis after another, and is transposed on the way to
// the registers, 4 rows by 16 columns at a time (bfloat16), or read value by value
// (float32).
//
// The matrix instruction bounds a large product.  256 x 256 tiles, eight waves of 128 x
// 64, read an operand's value from LDS 2 or 4 times and move 64 KB a block for 0.6 us of
// products: bfloat16 32768 x 5120 x 2560 with silu 720 to 780 us by card (1.1 to 1.2 PFLOP/s;
// the library's product alone 558 to 746), the pipes busy in 55% of the cycles at 1.73
// GHz, which is what the card's power allows.  Four waves of 128 x 128 read half as much from LDS:
// 3 to 5% faster forward, 4 to 12% slower for dw, with the accumulators pinned by hand.  float32
// keeps 2.1 GHz; 64 x 64 tiles, four workgroups a CU, fill 76% of the cycles, 128 x 128
// 82% (11686 x 1344 x 2960 767 us, the library 773).  Two buffers: four or five slots of
// a ring gained nothing, since a CU's other waves work through a wait.
enum Mode { kFwd, kGlu, kDx, kDw };

struct TileArgs {
  const void *a, *b;
  int64_t lda, ldb;         // elements between their rows
  int64_t stride_a;         // elements between two experts' matrices of a
  int64_t cols;             // columns of D (kGlu: of either half)
  int64_t high;             // kDw: rows of D
  int64_t depth;            // length of the summed axis (kDw: the expert's rows)
  int64_t rows, x_rows;
  const int32_t *token, *offsets;
  int experts, act, parts;
  bool out_f32;
  const float* bias;
  const void* residual;
  void *out, *pre;
  float* part;              // parts > 1: [parts][...] sums
  int64_t part_stride;
};

typedef const __attribute__((address_space(1))) void* global_ptr;
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(3))) s16x4* lds_tr_ptr;

// What a lane loads for a place past a row's or the axis' end.
__device__ const uint4 g_zeros = {0, 0, 0, 0};

// A 16-byte read is served 16 lanes at a time from 64 banks, two rows' worth of an
// operand of 128-byte rows: the keys of the 8 even rows and of the 8 odd rows of a
// tile differ, and those of neighbouring quads, whose chunks differ by 2, stay apart.
__device__ __forceinline__ int row_key(int row) { return ((((row >> 1) & 7) + 2) & 7) ^ 4; }

// Columns in LDS, bfloat16: units of 32 bytes (16 columns), unit u of row k at
// u ^ col_key(k): the 4 rows that a transposing read takes and the two quads served
// with it (16 rows apart) hit different banks.  float32: units of 64 bytes, the
// quads' rows 8 apart.
template <int SIDE>
__device__ __forceinline__ int col_key(int row) {
  if constexpr (kSize == 4) return (row >> 3) & 3;
  if constexpr (SIDE >= 128) return (row & 3) | ((row >> 4) & 1) << 2;
  return ((row >> 1) & 1) | ((row >> 4) & 1) << 1;
}

// Rows along the summed axis, SIDE of them.  GATHER: rows of x by token.
template <int SIDE, int WAVES, bool GATHER>
struct RowLoader {
  static constexpr int kRounds = SIDE / (8 * WAVES);
  static_assert(WAVES % 2 == 0, "a lane's place is the same in every round");
  const char* from[kRounds];
  int place;
  uint32_t lds_at;

  // row_of(r): element offset of LDS row r, or -1 for zeros
  template <typename F>
  __device__ __forceinline__ void init(const void* base, int wave, int lane, F row_of) {
    place = ((lane & 7) ^ row_key(wave * 8 + (lane >> 3))) * 16;
    lds_at = wave * 1024;
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      const int64_t at = row_of((j * WAVES + wave) * 8 + (lane >> 3));
      from[j] = GATHER && at < 0 ? nullptr : static_cast<const char*>(base) + at * kSize + place;
    }
  }
  // block g; left: values of the axis from the block's start
  __device__ __forceinline__ void load(uint8_t* lds, int64_t g, int64_t left) {
    const int64_t at = g * kBlockBytes;
    const bool whole = left >= kBlock;
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      const char* p = from[j] + at;
      if (GATHER && !from[j]) p = reinterpret_cast<const char*>(&g_zeros);
      if (!whole && place >= left * kSize) p = reinterpret_cast<const char*>(&g_zeros);
      __builtin_amdgcn_global_load_lds((global_ptr)p, (lds_ptr)(lds + lds_at + j * WAVES * 1024),
                                       16, 0, 0);
    }
  }
};

// Columns, SIDE of them, kBlock rows of the summed axis a block.
template <int SIDE, int WAVES, bool GATHER>
struct ColLoader {
  static constexpr int kRounds = SIDE / (8 * WAVES);
  static constexpr int kChunks = SIDE * kSize / 16;          // of a row
  static constexpr int kStep = WAVES * 64 / kChunks;         // rows a round
  static_assert(kStep * kRounds == kBlock, "");
  const char* base;
  int64_t ld;           // bytes
  int row, shift[kRounds];  // bytes of the lane's chunk within a row, < 0 past the last column
  uint32_t lds_at;
  const int32_t* token;
  int64_t x_rows;
  int next[kRounds];    // GATHER: the next block's rows of x

  __device__ __forceinline__ void init(const void* b, int64_t ld_elems, int64_t col0, int64_t cols,
                                       int wave, int lane) {
    const int f = wave * 64 + lane, c = f % kChunks;
    base = static_cast<const char*>(b) + col0 * kSize;
    ld = ld_elems * kSize;
    row = f / kChunks;
    lds_at = wave * 1024;
    constexpr int kUnit = kSize == 4 ? 4 : 2;                // chunks of a swizzled unit
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      const int from = ((c / kUnit) ^ col_key<SIDE>(row + j * kStep)) * kUnit + c % kUnit;
      shift[j] = col0 + from * (16 / kSize) < cols ? from * 16 : -1;
    }
  }
  __device__ __forceinline__ void tokens(int64_t row0, int64_t left) {
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      const int r = row + j * kStep;
      next[j] = r < left ? token[row0 + r] : -1;
    }
  }
  // block of rows from row0 on, of which `left` are there
  __device__ __forceinline__ void load(uint8_t* lds, int64_t row0, int64_t left) {
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      const int r = row + j * kStep;
      int64_t at = row0 + r;
      bool in = r < left && shift[j] >= 0;
      if constexpr (GATHER) {
        if (token) {
          at = next[j];
          in = in && at >= 0 && at < x_rows;
        }
      }
      const char* p = in ? base + at * ld + shift[j] : reinterpret_cast<const char*>(&g_zeros);
      __builtin_amdgcn_global_load_lds((global_ptr)p, (lds_ptr)(lds + lds_at + j * WAVES * 1024),
                                       16, 0, 0);
    }
  }
};

// A lane's 32 bytes of a row's block, as two chunks.  One sum of integers per
// access: the compiler then still sees which LDS object it is in.
__device__ __forceinline__ i32x8 read_row(const uint8_t* obj, uint32_t lo, uint32_t hi) {
  const int4 u = *reinterpret_cast<const int4*>(obj + lo);
  const int4 v = *reinterpret_cast<const int4*>(obj + hi);
  return i32x8{u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
}

// The same values of a column tile: bfloat16, rows quad 16 + 8 s + 4 h + 0 .. 3 by the
// transposing read (lane 4 j + c of 16 names row j, columns 4 c .. 4 c + 3, and gets
// column 4 j + c of the four rows); float32, rows quad 8 + 0 .. 7.  at: the lane's
// address within the object, of row quad 16 (8).
template <int SIDE>
__device__ __forceinline__ i32x8 read_col(const uint8_t* obj, uint32_t at) {
  constexpr int RB = SIDE * kSize;
  i32x8 v;
  if constexpr (kSize == 2) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_ptr)(obj + at + h * 4 * RB));
      const i32x2 u = __builtin_bit_cast(i32x2, t);
      v[2 * h] = u[0];
      v[2 * h + 1] = u[1];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = *reinterpret_cast<const int*>(obj + at + e * RB);
  }
  return v;
}

// Where a lane finds its values of row (column) tile 0 of a wave, and of tile t.
template <int SIDE, bool COL>
struct Reader {
  uint32_t lo, hi;
  __device__ __forceinline__ Reader(int first, int lane) {
    const int i = lane & 15, quad = lane >> 4;
    if constexpr (COL) {
      constexpr int RB = SIDE * kSize;
      if constexpr (kSize == 2) {
        const int k = quad * 16 + (i >> 2);
        lo = k * RB + (col_key<SIDE>(k) * 32) + (i & 3) * 8;
      } else {
        lo = quad * 8 * RB + (col_key<SIDE>(quad * 8) * 64) + i * 4;
      }
      hi = first / 16;
    } else {
      const int row = first + i;
      lo = row * kBlockBytes + ((quad * 2) ^ row_key(row)) * 16;
      hi = row * kBlockBytes + ((quad * 2 + 1) ^ row_key(row)) * 16;
    }
  }
  __device__ __forceinline__ i32x8 read(const uint8_t* obj, int t) const {
    if constexpr (COL) return read_col<SIDE>(obj, lo ^ ((hi + t) * (16 * kSize)));
    return read_row(obj, lo + t * 16 * kBlockBytes, hi + t * 16 * kBlockBytes);
  }
};

// Step s of a block: 32 (bfloat16; 2 steps) or 4 (float32; 8 steps) values of the
// summed axis, the lane's quad's share of them.
constexpr int kSteps = kSize == 2 ? 2 : 8;
__device__ __forceinline__ f32x4 mfma(const i32x8& a, const i32x8& b, int s, f32x4 c) {
#if SSM_LINEAR_DTYPE == 0
  return __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(a[s]), __int_as_float(b[s]), c, 0, 0, 0);
#else
  const i32x4 u = s == 0 ? i32x4{a[0], a[1], a[2], a[3]} : i32x4{a[4], a[5], a[6], a[7]};
  const i32x4 v = s == 0 ? i32x4{b[0], b[1], b[2], b[3]} : i32x4{b[4], b[5], b[6], b[7]};
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, u),
                                                 __builtin_bit_cast(bf16x8, v), c, 0, 0, 0);
#endif
}

// Place of tile number t of tm x tn, walked in strips of four row tiles.
__device__ __forceinline__ void place_of(int64_t t, int64_t tiles_m, int64_t tiles_n, int64_t* tm,
                                         int64_t* tn) {
  const int64_t strip = t / (4 * tiles_n), m0 = strip * 4;
  const int64_t high = tiles_m - m0 < 4 ? tiles_m - m0 : 4, in = t - strip * 4 * tiles_n;
  *tm = m0 + in % high;
  *tn = in / high;
}

// Consecutive workgroups go to the 8 XCDs in turn: each XCD gets a range of the
// `tiles` tiles of its own, so that the tiles it has in flight share their operands in
// its L2.  -1: none left.
__device__ __forceinline__ int64_t tile_number(int64_t tiles, int64_t bid) {
  const int64_t xcd = bid % 8, each = tiles / 8, more = tiles % 8;
  if (bid / 8 >= each + (xcd < more ? 1 : 0)) return -1;
  return xcd * each + (xcd < more ? xcd : more) + bid / 8;
}

// kDw: `each` tiles for every expert, whose rows differ in number: the XCDs share each
// expert's (one expert an XCD at a time left some idle: 950 us against 480 for 16 experts'
// 16384 rows, 5120 x 2560).  Fewer than 16 tiles an expert go round as they come.
__host__ __device__ __forceinline__ int64_t expert_grid(int64_t each, int64_t experts) {
  return each < 16 ? each * experts : (each + 7) / 8 * 8 * experts;
}
__device__ __forceinline__ bool expert_tile(int64_t each, int64_t experts, int64_t bid, int* expert,
                                            int64_t* t) {
  if (each < 16) {
    *expert = static_cast<int>(bid / each);
    *t = bid - *expert * each;
    return *expert < experts;
  }
  const int64_t share = (each + 7) / 8, in = bid / 8;
  *expert = static_cast<int>(in / share);
  *t = bid % 8 * share + (in - *expert * share);
  return *expert < experts && *t < each;
}

typedef u32x2 u32x2_any __attribute__((aligned(2)));

// 4 values, of which those past `last` are not there: loaded as the last one, not stored.
__device__ __forceinline__ f32x4 load4(const float* p, int last) {
  if (last >= 3) {
    const u32x4 t = *reinterpret_cast<const u32x4_any*>(p);
    return f32x4{__uint_as_float(t[0]), __uint_as_float(t[1]), __uint_as_float(t[2]), __uint_as_float(t[3])};
  }
  return f32x4{p[0], p[last < 1 ? last : 1], p[last < 2 ? last : 2], p[last]};
}
__device__ __forceinline__ f32x4 load4(const bf16_t* p, int last) {
  if (last >= 3) {
    const u32x2 t = *reinterpret_cast<const u32x2_any*>(p);
    return f32x4{__uint_as_float(t[0] << 16), __uint_as_float(t[0] & 0xffff0000u),
                 __uint_as_float(t[1] << 16), __uint_as_float(t[1] & 0xffff0000u)};
  }
  return f32x4{to_f32(p[0]), to_f32(p[last < 1 ? last : 1]), to_f32(p[last < 2 ? last : 2]), to_f32(p[last])};
}
__device__ __forceinline__ void store4(float* p, f32x4 v, int last) {
  if (last >= 3) {
    *reinterpret_cast<u32x4_any*>(p) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                             __float_as_uint(v[2]), __float_as_uint(v[3])};
    return;
  }
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j <= last) p[j] = v[j];
}
__device__ __forceinline__ void store4(bf16_t* p, f32x4 v, int last) {
  if (last >= 3) {
    *reinterpret_cast<u32x2_any*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j <= last) store_act(p, j, v[j]);
}

// Values 0 .. last of 8 to p; STREAM: past the caches, which the operands need.
template <bool STREAM, typename T>
__device__ __forceinline__ void put8(T* p, const float (&v)[8], int last = 7) {
  if (!STREAM || last < 7) {
    store8(p, v, last);
  } else if constexpr (sizeof(T) == 2) {
    __builtin_nontemporal_store(u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])},
                                reinterpret_cast<u32x4_any*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      __builtin_nontemporal_store(u32x4{__float_as_uint(v[i]), __float_as_uint(v[i + 1]),
                                        __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3])},
                                  reinterpret_cast<u32x4_any*>(p + i));
  }
}

// Tile number `bid`, part `part` of it.  The LDS objects are separate, so that reads of one
// are known not to wait for loads into another.
template <int MODE, int BN, int BM, int WN, int WM>
__device__ __forceinline__ void product_tile(const TileArgs& p, int64_t bid, int part, uint8_t* s_a0,
                                             uint8_t* s_a1, uint8_t* s_b0, uint8_t* s_b1) {
  constexpr int WAVES = WN * WM, NT = BN / WN / 16, MT = BM / WM / 16;
  constexpr bool GLU = MODE == kGlu, A_COL = MODE == kDx || MODE == kDw, B_COL = MODE == kDw;
  constexpr bool STREAM = BM == 256;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % WN, wm = wave / WN;

  // the tile: rows from m0 to m_end of D, columns from c0 on; the expert
  constexpr int kCols = GLU ? BN / 2 : BN;
  const int64_t tiles_n = (p.cols + kCols - 1) / kCols;
  int64_t tm, tn, m0, m_end;
  int expert = 0;
  Range range = {0, p.rows};
  if constexpr (MODE == kDw) {
    const int64_t tiles_m = (p.high + BM - 1) / BM, each = tiles_m * tiles_n;
    int64_t t;
    if (!expert_tile(each, p.offsets ? p.experts : 1, bid, &expert, &t)) return;
    place_of(t, tiles_m, tiles_n, &tm, &tn);
    range = rows_of(p.offsets, expert, p.rows);
    m0 = tm * BM;
    m_end = p.high;
  } else {
    const Tiles tiles = {p.offsets, p.experts, p.rows, BM};
    const int64_t total = tiles.total(), t = tile_number(total * tiles_n, bid);
    if (t < 0) return;
    place_of(t, total, tiles_n, &tm, &tn);
    int at;
    if (!tiles.find(static_cast<int>(tm), &expert, &at)) return;
    range = rows_of(p.offsets, expert, p.rows);
    m0 = range.from + static_cast<int64_t>(at) * BM;
    m_end = range.to;
  }
  const int64_t c0 = tn * kCols;

  // with the summed axis split over p.parts workgroups: blocks first .. first + groups - 1
  const int64_t depth = MODE == kDw ? range.to - range.from : p.depth;
  const int all = static_cast<int>((depth + kBlock - 1) / kBlock);
  const int each = (all + p.parts - 1) / p.parts, first = part * each;
  const int groups = all - first < each ? (all - first > 0 ? all - first : 0) : each;

  const Act* a = static_cast<const Act*>(p.a) + (MODE == kDw ? 0 : expert * p.stride_a);
  const Act* b = static_cast<const Act*>(p.b);
  typename std::conditional<A_COL, ColLoader<BN, WAVES, MODE == kDw>, RowLoader<BN, WAVES, false>>::type la;
  typename std::conditional<B_COL, ColLoader<BM, WAVES, false>,
                            RowLoader<BM, WAVES, MODE != kDx>>::type lb;
  if constexpr (A_COL) {
    la.init(a, p.lda, c0, p.cols, wave, lane);
    la.token = p.token;
    la.x_rows = p.x_rows;
  } else {
    la.init(a, wave, lane, [&](int r) {
      int64_t c = c0 + (GLU ? (r >> 5) * 16 + (r & 15) : r);
      c = c < p.cols ? c : p.cols - 1;  // past the end: the last one
      if (GLU && (r & 16)) c += p.cols;
      return c * p.lda;
    });
  }
  if constexpr (B_COL) {
    lb.init(b, p.ldb, m0, p.high, wave, lane);
  } else {
    lb.init(b, wave, lane, [&](int r) {
      const int64_t row = m0 + r < m_end ? m0 + r : m_end - 1;
      if (MODE == kDx || !p.token) return row * p.ldb;
      const int64_t t = p.token[row];
      return t >= 0 && t < p.x_rows ? t * p.ldb : static_cast<int64_t>(-1);
    });
  }
  // block g of this workgroup's
  auto load_a = [&](uint8_t* lds, int g) {
    const int64_t at = static_cast<int64_t>(first + g) * kBlock;
    if constexpr (A_COL) {
      la.load(lds, (MODE == kDw ? range.from : 0) + at, depth - at);
      if (MODE == kDw && p.token && g + 1 < groups) la.tokens(range.from + at + kBlock, depth - at - kBlock);
    } else {
      la.load(lds, first + g, depth - at);
    }
  };
  auto load_b = [&](uint8_t* lds, int g) {
    const int64_t at = static_cast<int64_t>(first + g) * kBlock;
    if constexpr (B_COL) lb.load(lds, range.from + at, depth - at);
    else lb.load(lds, first + g, depth - at);
  };

  f32x4 acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = f32x4{};

  // A wave without rows only loads its share of the operands: the other wave of its SIMD
  // has the matrix instruction to itself (an expert's last tile).
  if (MODE != kDw && m0 + wm * (BM / WM) >= m_end) {
    if (groups > 0) {
      load_a(s_a0, 0);
      load_b(s_b0, 0);
      __syncthreads();
    }
    if (groups > 1) {
      load_a(s_a1, 1);
      load_b(s_b1, 1);
    }
    for (int g = 0; g < groups; ++g) {
      __syncthreads();
      if (g + 2 < groups) {
        load_a(g % 2 ? s_a1 : s_a0, g + 2);
        load_b(g % 2 ? s_b1 : s_b0, g + 2);
      }
    }
    __syncthreads();  // as the others do in front of their stores
    return;
  }

  if (groups > 0) {
    if constexpr (MODE == kDw) {
      const int64_t at = static_cast<int64_t>(first) * kBlock;
      if (p.token) la.tokens(range.from + at, depth - at);
    }
    load_a(s_a0, 0);
    load_b(s_b0, 0);
    __syncthreads();
    if (groups > 1) {
      load_a(s_a1, 1);
      load_b(s_b1, 1);
    }
    const Reader<BN, A_COL> ra(wn * (BN / WN), lane);
    const Reader<BM, B_COL> rb(wm * (BM / WM), lane);
    i32x8 fa[2], fb[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) fb[m] = rb.read(s_b0, m);
    fa[0] = ra.read(s_a0, 0);

    // Block g from (ca, cb), its first operands already read; the next is in (oa, ob).
    // The barrier of a block stands before its last row of tiles, when every operand
    // of the block has been read: behind it the buffer takes the block after next, and
    // the next block's first operands are read while the last row is multiplied.
    auto step = [&](int g, uint8_t* ca, uint8_t* cb, const uint8_t* oa, const uint8_t* ob) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n + 1 < NT) {
          fa[(n + 1) & 1] = ra.read(ca, n + 1);
        } else {
          __syncthreads();
          fa[NT & 1] = ra.read(oa, 0);
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            acc[n][m] = mfma(fa[n & 1], fb[m], s, acc[n][m]);
            if (n + 1 == NT && s + 1 == kSteps) fb[m] = rb.read(ob, m);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (g + 2 < groups) {
        load_a(ca, g + 2);
        load_b(cb, g + 2);
      }
    };
    int g = 0;
    for (; g + 1 < groups; g += 2) {
      step(g, s_a0, s_b0, s_a1, s_b1);
      step(g + 1, s_a1, s_b1, s_a0, s_b0);
    }
    if (g < groups) step(g, s_a0, s_b0, s_a1, s_b1);
  }

  // A lane holds four consecutive columns of a row: of tile (n, m) columns 16 n + 4 quad
  // .. + 3 of row 16 m + lane % 16.  The wave's tile goes through LDS, where the operands
  // were, so that what follows takes 8 consecutive columns a lane, whole rows at a time,
  // in a short loop.  Rows of C chunks of 4 columns, chunk c at c ^ key(row).
  constexpr int N = NT * 16, C = N / 4, OUT = GLU ? N / 2 : N, C8 = OUT / 8;
  constexpr int kRegion = 2 * (BN + BM) * kBlockBytes / WAVES;           // bytes a wave
  constexpr int PM = kRegion / (16 * N * 4) < MT ? kRegion / (16 * N * 4) : MT;  // row tiles a pass
  static_assert(PM > 0 && MT % PM == 0 && BN == BM && WAVES % 4 == 0 && 64 % C8 == 0, "");
  constexpr int kObject = WAVES / 4;  // waves an object
  uint8_t* lds = wave / kObject == 0 ? s_a0 : wave / kObject == 1 ? s_a1 : wave / kObject == 2 ? s_b0 : s_b1;
  lds += wave % kObject * kRegion;
  auto place = [](int row, int c) { return (row * C + (c ^ ((C >= 16 ? row : row >> 1) & (C >= 16 ? 15 : 7)))) * 16; };
  const int i = lane & 15, quad = lane >> 4;
  const int64_t width = GLU ? 2 * p.cols : p.cols;
  const int c8 = lane % C8;
  const int64_t col = c0 + static_cast<int64_t>(wn) * OUT + c8 * 8;  // the lane's, every time
  const bool live = col < p.cols;
  const int last = p.cols - col < 8 ? static_cast<int>(p.cols - col) - 1 : 7;
  const int chunk = GLU ? (c8 >> 1) * 8 + (c8 & 1) * 2 : c8 * 2;
  const bool odd = C >= 32 && !GLU && (lane & 8);  // these read the second chunk first: no bank twice
  float bias[2][8] = {};
  if ((MODE == kFwd || MODE == kGlu) && p.bias && p.parts == 1 && live) {
    const float* from = p.bias + static_cast<int64_t>(expert) * width + col;
#pragma unroll
    for (int h = 0; h < (GLU ? 2 : 1); ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) bias[h][e] = from[h * p.cols + (e < last ? e : last)];
  }
#pragma unroll
  for (int m1 = 0; m1 < MT; m1 += PM) {
    if (m1 == 0) __syncthreads();  // nobody reads operands any more
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int m = 0; m < PM; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<f32x4*>(lds + place(m * 16 + i, n * 4 + quad)) = acc[n][m1 + m];
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int r0 = 0; r0 < PM * 16; r0 += 64 / C8) {
      const int row = r0 + lane / C8;
      const int64_t r = m0 + (wm * MT + m1) * 16 + row;
      if (r >= m_end || !live) continue;
      auto get = [&](int c, float (&v)[8]) {
        const f32x4 s0 = *reinterpret_cast<const f32x4*>(lds + place(row, c + odd));
        const f32x4 s1 = *reinterpret_cast<const f32x4*>(lds + place(row, c + !odd));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = odd ? s1[e] : s0[e];
          v[4 + e] = odd ? s0[e] : s1[e];
        }
      };
      float v[8], u[8];
      get(chunk, v);
      if constexpr (GLU) get(chunk + 4, u);
      if (p.parts > 1) {
        float* to = p.part + part * p.part_stride + (MODE == kDw ? expert * p.high + r : r) * width + col;
        put8<STREAM>(to, v, last);
        if constexpr (GLU) put8<STREAM>(to + p.cols, u, last);
        continue;
      }
      if constexpr (MODE == kDx) {
        put8<STREAM>(static_cast<Act*>(p.out) + r * p.cols + col, v, last);
      } else if constexpr (MODE == kDw) {
        put8<STREAM>(static_cast<Act*>(p.out) + (expert * p.high + r) * p.cols + col, v, last);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] += bias[0][e];
          if constexpr (GLU) u[e] += bias[1][e];
        }
        if (p.pre) {
          put8<STREAM>(static_cast<Act*>(p.pre) + r * width + col, v, last);
          if constexpr (GLU) put8<STREAM>(static_cast<Act*>(p.pre) + r * width + p.cols + col, u, last);
        }
        if (is_silu(p.act)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = bend_as<true>(v[e]);
        } else if (p.act != kNoAct) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = bend_as<false>(v[e]);
        }
        if constexpr (GLU) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= u[e];
        }
        if (p.residual) {
          if (p.out_f32) {
            Run8<float> t;
            const float* res = static_cast<const float*>(p.residual) + r * p.cols + col;
            if (last < 7) t.load_elems(res, last);
            else t.load(res);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += t.get(e);
          } else {
            Run8<bf16_t> t;
            const bf16_t* res = static_cast<const bf16_t*>(p.residual) + r * p.cols + col;
            if (last < 7) t.load_elems(res, last);
            else t.load(res);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += t.get(e);
          }
        }
        if (p.out_f32) put8<STREAM>(static_cast<float*>(p.out) + r * p.cols + col, v, last);
        else put8<STREAM>(static_cast<bf16_t*>(p.out) + r * p.cols + col, v, last);
      }
    }
  }
}

#define SSM_PRODUCT_LDS(SIDE)                                \
  __shared__ __align__(1024) uint8_t s_a0[SIDE * kBlockBytes]; \
  __shared__ __align__(1024) uint8_t s_a1[SIDE * kBlockBytes]; \
  __shared__ __align__(1024) uint8_t s_b0[SIDE * kBlockBytes]; \
  __shared__ __align__(1024) uint8_t s_b1[SIDE * kBlockBytes]

template <int MODE, int SIDE, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM, 2) void product_kernel(TileArgs p) {
  SSM_PRODUCT_LDS(SIDE);
  product_tile<MODE, SIDE, SIDE, WN, WM>(p, blockIdx.x, blockIdx.y, s_a0, s_a1, s_b0, s_b1);
}

// Joins the parts of a product whose summed axis was split, in order, four columns a
// thread.  Rows ahead of the first expert's and past the last one's stay as they are.
struct JoinArgs {
  const float* part;
  int parts, act;
  bool out_f32;
  int64_t part_stride, rows, cols;  // cols: of out
  const int32_t* offsets;           // of the experts that have the rows, nullable
  int experts;
  const float* bias;
  const void* residual;
  void *out, *pre;
};

__global__ __launch_bounds__(256) void join_kernel(JoinArgs p) {
  const int64_t quads = (p.cols + 3) / 4, at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = at / quads, c = (at - row * quads) * 4;
  if (row >= p.rows || (p.offsets && (row < p.offsets[0] || row >= p.offsets[p.experts]))) return;
  const bool glu = is_gated(p.act);
  const int64_t width = glu ? 2 * p.cols : p.cols;
  const int last = p.cols - c < 4 ? static_cast<int>(p.cols - c) - 1 : 3;
  f32x4 v = {}, u = {};
  for (int q = 0; q < p.parts; ++q) {
    const float* from = p.part + q * p.part_stride + row * width + c;
    v += load4(from, last);
    if (glu) u += load4(from + p.cols, last);
  }
  if (p.bias) {
    int e = 0;
    if (p.offsets) {
      for (int hi = p.experts - 1; e < hi;) {  // the first expert that ends past the row
        const int mid = (e + hi) / 2;
        if (p.offsets[mid + 1] <= row) e = mid + 1;
        else hi = mid;
      }
    }
    const float* bias = p.bias + e * width + c;
    v += load4(bias, last);
    if (glu) u += load4(bias + p.cols, last);
  }
  if (p.pre) {
    Act* pre = static_cast<Act*>(p.pre) + row * width + c;
    store4(pre, v, last);
    if (glu) store4(pre + p.cols, u, last);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (glu) v[j] = bend(p.act, v[j]) * u[j];
    else if (p.act != kNoAct) v[j] = bend(p.act, v[j]);
  }
  const int64_t to = row * p.cols + c;
  if (p.residual)
    v += p.out_f32 ? load4(static_cast<const float*>(p.residual) + to, last)
                   : load4(static_cast<const bf16_t*>(p.residual) + to, last);
  if (p.out_f32) store4(static_cast<float*>(p.out) + to, v, last);
  else store4(static_cast<bf16_t*>(p.out) + to, v, last);
}

// ---- few rows: the weights' stream ----
//
// With few rows a matrix the weights' bytes bound the product, so each is read once,
// straight into the matrix instruction's registers: a workgroup takes 16 rows of one
// matrix (of a gated one 16 of either half), its waves the blocks of 128 bytes in
// turn; the activations come from the L2.  The waves' sums meet in LDS and are added
// in wave order.  A matrix with more than 16 rows is read again for the next ones.
//
// Two workgroups a CU, 16 waves, keep the reads in flight: with three registers more
// than 128 a lane it is one, and 8 tokens' rows of 4 of 64 experts (2560 -> 2 x 1280 gated,
// bfloat16, 340 MB of weights) take 70 us, not 52 (6.5 TB/s); with fewer blocks in flight
// for three workgroups 71.  One dense matrix of 26 MB and 8 rows is over before the reads
// reach their rate: 10.8 us.
constexpr int kStreamWaves = 8;

template <bool GLU>
__global__ __launch_bounds__(64 * kStreamWaves, 4) void stream_kernel(TileArgs p) {
  constexpr int H = GLU ? 2 : 1;
  __shared__ f32x4 s_sum[kStreamWaves][H][64];
  const int lane = threadIdx.x & 63, i = lane & 15, quad = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int W = blockDim.x >> 6;
  int expert = blockIdx.y;
  if (p.offsets && gridDim.y < static_cast<unsigned>(p.experts)) {
    // fewer rows than experts: the expert whose first row is row blockIdx.y
    const int64_t row = blockIdx.y;
    bool found = false;
    for (int e0 = 0; e0 < p.experts && !found; e0 += 64) {
      const Range r = e0 + lane < p.experts ? rows_of(p.offsets, e0 + lane, p.rows) : Range{0, 0};
      const uint64_t hit = __ballot(r.from == row && r.to > row);
      if (hit) {
        expert = e0 + __builtin_ctzll(hit);
        found = true;
      }
    }
    if (!found) return;
  }
  const Range range = rows_of(p.offsets, expert, p.rows);
  if (range.from >= range.to) return;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int64_t c_lane = c0 + i < p.cols ? c0 + i : p.cols - 1;
  const char* wrow[H];
#pragma unroll
  for (int h = 0; h < H; ++h)
    wrow[h] = static_cast<const char*>(p.a) +
              (expert * p.stride_a + (c_lane + h * p.cols) * p.lda) * kSize;
  const int bytes = static_cast<int>(p.depth) * kSize;
  const int groups = (bytes + kBlockBytes - 1) / kBlockBytes;
  // the quad's 16 bytes of either half of a row's 128: 64 bytes a row by one access
  auto load32 = [&](const char* row, int at) {
    i32x8 v = {};
    if (at < bytes) {
      const int4 t = *reinterpret_cast<const int4*>(row + at);
      v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    }
    if (at + 64 < bytes) {
      const int4 t = *reinterpret_cast<const int4*>(row + at + 64);
      v[4] = t.x; v[5] = t.y; v[6] = t.z; v[7] = t.w;
    }
    return v;
  };
  for (int64_t m0 = range.from; m0 < range.to; m0 += 16) {
    const int64_t r = m0 + i;
    int64_t t = r < range.to ? r : range.to - 1;
    bool in = true;
    if (p.token) {
      t = p.token[t];
      in = t >= 0 && t < p.x_rows;
    }
    const char* xrow = static_cast<const char*>(p.b) + (in ? t : 0) * p.ldb * kSize;
    f32x4 acc[H] = {};
    constexpr int U = GLU ? 2 : 4;  // blocks in flight
    for (int g0 = w; g0 < groups; g0 += U * W) {
      i32x8 a[U][H], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = (g0 + u * W) * kBlockBytes + quad * 16;
#pragma unroll
        for (int h = 0; h < H; ++h) a[u][h] = load32(wrow[h], at);
        b[u] = load32(xrow, in ? at : bytes);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int h = 0; h < H; ++h) acc[h] = mfma(a[u][h], b[u], s, acc[h]);
    }
#pragma unroll
    for (int h = 0; h < H; ++h) s_sum[w][h][lane] = acc[h];
    __syncthreads();
    const int64_t c = c0 + quad * 4;
    if (w == 0 && r < range.to && c < p.cols) {
      f32x4 v[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        v[h] = s_sum[0][h][lane];
        for (int q = 1; q < W; ++q) v[h] += s_sum[q][h][lane];
      }
      const int last = p.cols - c < 4 ? static_cast<int>(p.cols - c) - 1 : 3;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (p.bias) v[h] += load4(p.bias + (static_cast<int64_t>(expert) * H + h) * p.cols + c, last);
        if (p.pre) store4(static_cast<Act*>(p.pre) + (r * H + h) * p.cols + c, v[h], last);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (GLU) v[0][j] = bend(p.act, v[0][j]) * v[H - 1][j];
        else if (p.act != kNoAct) v[0][j] = bend(p.act, v[0][j]);
      }
      const int64_t to = r * p.cols + c;
      if (p.residual)
        v[0] += p.out_f32 ? load4(static_cast<const float*>(p.residual) + to, last)
                          : load4(static_cast<const bf16_t*>(p.residual) + to, last);
      if (p.out_f32) store4(static_cast<float*>(p.out) + to, v[0], last);
      else store4(static_cast<bf16_t*>(p.out) + to, v[0], last);
    }
    __syncthreads();
  }
}

// ---- backward: the activation's gradient and the bias' ----
//
// dpre in the activations' type for the two products, and its sums over the rows of
// each tile of p.tile rows of an expert from the values before that rounding.  A wave
// takes 512 columns, 8 a lane, of every fourth row.  Memory bounds it: 16384 x 5120 bfloat16
// of a gelu or silu 91 us (503 MB, 5.5 TB/s), 16384 rows of 16 experts, 2 x 2560 gated, 84.  In the
// products themselves it would be done once for every tile of the other axis.
//
// bfloat16: the matrix instruction takes bfloat16 operands, so dpre is rounded once, also a
// float32 dout without activation.  Carried as two bfloat16 parts it would double both products.
// The rounding adds as much as the outputs' own: 2048 x 5120 x 2560, dx and dw are off float64 by
// 0.0023 of their norm, 0.0017 with dpre in float32.  The bias' sums take it before.
// Without dx and dw only the sums are written: 16384 x 5120 76 us as a call.

struct BendArgs {
  const void *dout, *pre;
  void* dpre;               // nullable: dout serves as it is, or there is no product
  float* part;              // [tiles][nw], nullable
  const int32_t* offsets;
  int experts, act, tile;
  int64_t rows, n, max_tiles;
  int64_t ld;               // of dpre's rows: nw, up to the next multiple of 8; zeros past nw
};

// Rows of a tile: few where 128 would leave the CUs without work (bias alone: 2047 x 768 float32
// 4.3 us by 32 rows, 8.0 by 128, 2047 x 5120 bfloat16 5.8 and 10.5, 16384 x 5120 28 and 25).
int bend_rows(int64_t rows, int64_t n) { return rows * n < (1 << 25) ? 32 : 128; }

template <typename D>
__global__ __launch_bounds__(256) void bend_kernel(BendArgs p) {
  __shared__ float s_part[4][64][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Tiles tiles = {p.offsets, p.experts, p.rows, p.tile};
  int expert, at;
  if (!tiles.find(static_cast<int>(blockIdx.x), &expert, &at)) return;
  const Range range = rows_of(p.offsets, expert, p.rows);
  const int64_t m0 = range.from + static_cast<int64_t>(at) * p.tile;
  const int64_t m_end = m0 + p.tile < range.to ? m0 + p.tile : range.to;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * 512 + lane * 8;
  const bool live = c < p.n, glu = is_gated(p.act);
  const int64_t width = glu ? 2 * p.n : p.n;
  const int last = p.n - c < 8 ? static_cast<int>(p.n - c) - 1 : 7;
  const int pad = static_cast<int>(p.ld - width);
  float sum[16] = {};
  if (live) {
    for (int64_t r = m0 + wave; r < m_end; r += 4) {
      auto load = [&](auto& run, const auto* from) __attribute__((always_inline)) {
        if (last < 7) run.load_elems(from, last);
        else run.load(from);
      };
      Run8<D> d;
      load(d, static_cast<const D*>(p.dout) + r * p.n + c);
      float g[8], h[8] = {};
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = d.get(e);
      if (p.act != kNoAct) {
        Run8<Act> v, u;
        load(v, static_cast<const Act*>(p.pre) + r * width + c);
        if (glu) load(u, static_cast<const Act*>(p.pre) + r * width + p.n + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float slope;
          const float f = bend_grad(p.act, v.get(e), &slope);
          if (glu) {
            h[e] = g[e] * f;
            g[e] *= u.get(e);
          }
          g[e] *= slope;
        }
      }
      if (p.dpre) {
        Act* to = static_cast<Act*>(p.dpre) + r * p.ld + c;
        store8(to, g, last);
        if (glu) store8(to + p.n, h, last);
        if (c + 8 >= p.n)  // the row's end, which the products read
          for (int e = 0; e < pad; ++e) store_act(static_cast<Act*>(p.dpre), r * p.ld + width + e, 0.0f);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[e] += g[e];
        sum[8 + e] += h[e];
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int e = 0; e < 16; ++e) s_part[wave][lane][e] = sum[e];
  __syncthreads();
  if (static_cast<int64_t>(blockIdx.x) >= p.max_tiles) return;
  float* to = p.part + static_cast<int64_t>(blockIdx.x) * width + static_cast<int64_t>(blockIdx.y) * 512;
  for (int f = threadIdx.x; f < (glu ? 1024 : 512); f += 256) {
    const int h = f / 512, col = f % 512;
    if (static_cast<int64_t>(blockIdx.y) * 512 + col >= p.n) continue;
    const int l = col / 8, e = col % 8 + 8 * h;
    to[h * p.n + col] = (s_part[0][l][e] + s_part[1][l][e]) + (s_part[2][l][e] + s_part[3][l][e]);
  }
}

// dbias[e] = the sum of the expert's tiles: columns 64 block .. + 63, by `waves` waves.  The tiles
// are added in 16 strands and these in turn, however many waves there are.
__device__ __forceinline__ void bias_columns(const BendArgs& p, float* dbias, int64_t block, int expert,
                                             int waves, float (*s_part)[64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t width = is_gated(p.act) ? 2 * p.n : p.n, c = block * 64 + lane;
  const Tiles tiles = {p.offsets, p.experts, p.rows, p.tile};
  int64_t from = 0, count = (p.rows + p.tile - 1) / p.tile;
  if (p.offsets) {
    count = tiles.count(expert);
    for (int e0 = 0; e0 < expert; e0 += 64) {
      const int own = e0 + lane < expert ? tiles.count(e0 + lane) : 0;
      from += __builtin_amdgcn_readlane(Tiles::running(own), 63);
    }
    if (from + count > p.max_tiles) count = p.max_tiles > from ? p.max_tiles - from : 0;
  }
  for (int strand = wave; strand < 16; strand += waves) {
    float sum = 0.0f;
    if (c < width)
#pragma unroll 4
      for (int64_t t = from + strand; t < from + count; t += 16) sum += p.part[t * width + c];
    s_part[strand][lane] = sum;
  }
  __syncthreads();
  if (wave == 0 && c < width) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) sum += s_part[w][lane];
    dbias[expert * width + c] = sum;
  }
}

__global__ __launch_bounds__(1024) void bias_kernel(BendArgs p, float* dbias) {
  __shared__ float s_part[16][64];
  bias_columns(p, dbias, blockIdx.x, blockIdx.y, 16, s_part);
}

// Both products of the gradient by one launch, and the last sums of the bias': first the tiles of
// dw, `each` workgroups (a multiple of the XCDs) for every part, then those of dx up to workgroup
// `end`, which fill the CUs that the last of the others leave free, then `groups` workgroups an expert
// for dbias (5 us as a launch of its own).
struct PairArgs {
  TileArgs w, x;
  BendArgs bend;
  float* dbias;
  int64_t each, end, groups;
};

template <int SIDE, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM, 2) void pair_kernel(PairArgs p) {
  SSM_PRODUCT_LDS(SIDE);
  const int64_t bid = blockIdx.x, behind = bid - p.each * p.w.parts;
  if (behind < 0) {
    const int part = static_cast<int>(bid / p.each);
    product_tile<kDw, SIDE, SIDE, WN, WM>(p.w, bid - part * p.each, part, s_a0, s_a1, s_b0, s_b1);
  } else if (bid < p.end) {
    product_tile<kDx, SIDE, SIDE, WN, WM>(p.x, behind, 0, s_a0, s_a1, s_b0, s_b1);
  } else {
    const int expert = static_cast<int>((bid - p.end) / p.groups);
    bias_columns(p.bend, p.dbias, bid - p.end - expert * p.groups, expert, WN * WM,
                 reinterpret_cast<float (*)[64]>(s_a0));
  }
}
#undef SSM_PRODUCT_LDS

// ---- plans ----

int forced(const char* name) {
  const char* v = getenv(name);
  return v && *v ? atoi(v) : -1;
}

enum Shape : int { kStream = 0, kTile64 = 1, kTile128 = 2, kTile256 = 3 };

struct Plan {
  int shape, parts;
  double us;  // the estimate that they were chosen by
};

// Parts of `blocks` blocks, each ceil(blocks / parts) of them, without those that get none.
int whole_parts(int64_t blocks, int parts) {
  if (parts > blocks) parts = static_cast<int>(blocks);
  return parts <= 1 ? 1 : static_cast<int>(div_up64(blocks, div_up64(blocks, parts)));
}

constexpr int64_t kCus = 256;

// Most tiles of `side` rows that `rows` rows of the experts make: each expert's last
// may be filled in part.
int64_t most_tiles(int64_t rows, int experts, int64_t side) {
  if (experts == 0) return div_up64(rows, side);
  const int64_t some = experts < rows ? experts : rows;
  return rows / side + some;
}

constexpr int kMostParts = 32;

// What one block of the summed axis takes on a CU that has `n` tiles of this shape to
// do, in us, for all of them: the figures of products that fill 1 to 40 tiles a CU, within
// a tenth of the measured times with 2 blocks (float32) or 5 (bfloat16) added a tile for
// its start and its epilogue.  A float32 tile all but fills the matrix units by itself, so
// that tiles of one CU add up (a second of 128 x 128 gains an eighth); a bfloat16 tile waits
// for its loads, and a second of 128 x 128 or three more of 64 x 64 run meanwhile.
double block_us(int shape, int64_t n) {
  const double d = static_cast<double>(n);
  if (kSize == 4 && shape == kTile128) return 3.95 * (n / 2) + 2.25 * (n % 2);
  if (kSize == 4) return d * (shape == kTile256 ? 7.9 : 0.56);
  if (shape == kTile256) return 1.4 * d;
  if (shape == kTile128) return 0.9 * (n / 2) + 0.75 * (n % 2);
  return 0.72 * (n / 4) + (n % 4 ? 0.45 + 0.05 * (n % 4) : 0.0);
}

struct Sizes {  // of a product in tiles
  int64_t high, cols, blocks, matrices;
  int64_t tiles(int64_t side) const { return matrices * div_up64(high, side) * div_up64(cols, side); }
  double join_us(int parts) const {
    return parts > 1 ? 6.0 + 8e-6 / 10.0 * static_cast<double>(matrices) * high * cols * parts : 0.0;
  }
};
Sizes sizes_of(const ProductArgs& a, int mode) {
  const int64_t nw = a.nw(), matrices = a.experts ? a.experts : 1, mean = div_up64(a.rows, matrices);
  if (mode == kDw) return {nw, a.k, div_up64(mean, kBlock), matrices};
  return {mean, mode == kDx ? a.k : nw, div_up64(mode == kDx ? nw : a.k, kBlock), matrices};
}
constexpr int kSides[] = {0, 64, 128, 256};
constexpr int kExtra = kSize == 4 ? 2 : 5;  // blocks a tile, its start and its epilogue

// The tile and the parts of the summed axis of the least cost: what the fullest CU has
// to do, and for parts the join, 6 us and its traffic at 10 TB/s (the parts are still in a cache).  The largest tile moves
// the least memory, but 276 of them keep 256 CUs for two rounds, the second nearly
// empty: float32, 11686 rows x 1344 x 2960 takes 1469 us by 256 x 256 tiles and 768 by
// 128 x 128 ones, bfloat16 4096 x 5120 x 2560 126 and 116; bfloat16 2048 x 5120 x 2560 60
// (160 tiles, one round) and 79.  Few tiles with a long sum are split: bfloat16, the rows'
// gradient of 1024 x 5120 x 2560 takes 64 us by 160 tiles of 128 x 128, 48 by two parts of each.
// Few rows of a matrix take the stream kernel: 16 bfloat16 rows x 5120 x 2560 12.9 us, 14.6 by 64 x 64
// tiles in parts, 24 rows, for which it reads the weights twice, 20.9 and 15.0.  Experts' rows
// differ in number: 64 experts of 2 x 1280 x 2560 with 8 rows at the mean 157 us, 160 by tiles,
// with 16 237 and 163; float32 345 and 373, 540 and 382.  The host knows the mean alone: 512 rows of
// those 64 experts 157 us, 181 with half of them one expert's, 250 with all (float32 356, 421, 509).
// SSM_FORCE_PRODUCT_SHAPE and _PARTS override (tests, tuning), for the gradient
// SSM_FORCE_PRODUCT_PAIR.
Plan plan_tiles(const ProductArgs& a, int mode) {
  const Sizes z = sizes_of(a, mode);
  Plan q = {kTile64, 1, 0.0};
  if ((mode == kFwd || mode == kGlu) && z.high <= (a.experts ? 8 : 16)) q.shape = kStream;
  for (int s = kTile64; s <= kTile256 && q.shape != kStream; ++s) {
    const int64_t all = z.tiles(kSides[s]);
    if (all > kMostTiles && s != kTile256) continue;
    for (int t = 1; t <= (s == kTile256 ? 1 : kMostParts) && t <= z.blocks; ++t) {
      const double us =
          (div_up64(z.blocks, t) + kExtra) * block_us(s, div_up64(all * t, kCus)) + z.join_us(t);
      if (q.us == 0.0 || us < q.us) q = {s, t, us};
    }
  }
  const int shape = forced("SSM_FORCE_PRODUCT_SHAPE"), parts = forced("SSM_FORCE_PRODUCT_PARTS");
  if (shape >= kTile64 && shape <= kTile256) q = {shape, 1, 0.0};
  if (shape == kStream && (mode == kFwd || mode == kGlu)) q = {kStream, 1, 0.0};
  if (q.shape == kStream) return q;
  if (parts > 0) q.parts = parts;
  q.parts = whole_parts(z.blocks, q.parts);
  return q;
}

// Both products of the gradient by one launch, dw in parts: of shape kStream if two are better.
// What the CUs have to do is shared evenly but for half a tile at the end: bfloat16, 16384 x
// 5120 x 2560 in 200 tiles of 256 blocks and 640 of 80, 753 us against 808 by two launches,
// 2048 x 1536 x 768 27 against 42, 32768 x 5120 x 2560, whole rounds by themselves, 1520 either
// way.  A tile of dw that is much longer than those of dx would end last (float32, 2047 x 768 x
// 1536: 118 us, in two parts 102, two launches 117).
Plan plan_pair(const ProductArgs& a, const Plan& dx, const Plan& dw) {
  const Sizes x = sizes_of(a, kDx), w = sizes_of(a, kDw);
  Plan q = {kStream, 1, dx.us + dw.us + 5.0};  // (a launch's start)
  const int pair = forced("SSM_FORCE_PRODUCT_PAIR"), shape = forced("SSM_FORCE_PRODUCT_SHAPE"),
            parts = forced("SSM_FORCE_PRODUCT_PARTS");
  if (pair == 0 || (pair < 0 && (shape >= 0 || dx.parts > 1))) return q;
  for (int s = kTile64; s <= kTile256; ++s) {
    if (shape >= 0 && s != shape) continue;
    if (x.tiles(kSides[s]) > kMostTiles) continue;
    const int full = s == kTile64 ? 4 : s == kTile128 ? 2 : 1;  // tiles that a CU works on at once
    for (int t = 1; t <= kMostParts && t <= w.blocks && w.tiles(kSides[s]) * t <= kMostTiles; ++t) {
      const int64_t tiles_w = w.tiles(kSides[s]) * t, tiles_x = x.tiles(kSides[s]);
      const double own = div_up64(w.blocks, t) + kExtra, other = x.blocks + kExtra;
      const double shared = (tiles_w * own + tiles_x * other) / kCus * block_us(s, full) / full +
                            0.5 * other * block_us(s, 1) / (full * full);
      // the longest takes so long: one of dw among the others of its CU, one of dx with nobody else
      const int64_t most = div_up64(tiles_w + tiles_x, kCus);
      const double last = other * block_us(s, 1), first = own * block_us(s, most < full ? most : full);
      const double alone = first > last ? first : last;
      const double us = (shared > alone ? shared : alone) + w.join_us(t);
      if (us < q.us || (pair > 0 && q.shape == kStream)) q = {s, t, us};
    }
  }
  if (q.shape != kStream) q.parts = whole_parts(w.blocks, parts > 0 ? parts : q.parts);
  return q;
}

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

// Bytes of the parts of a product.
int64_t parts_bytes(const ProductArgs& a, int mode, const Plan& q) {
  if (q.parts <= 1) return 0;
  const int64_t matrices = a.experts ? a.experts : 1;
  const int64_t values = mode == kDw ? matrices * a.nw() * a.k
                                     : a.rows * (mode == kDx ? a.k : a.nw());
  return up16(q.parts * values * 4);
}

// Workgroups for the tiles of one part.
template <int MODE, int SIDE>
int64_t grid_of(const TileArgs& t) {
  const int experts = t.offsets ? t.experts : 0;
  const int64_t tiles_n = div_up64(t.cols, MODE == kGlu ? SIDE / 2 : SIDE);
  if (MODE == kDw) return expert_grid(div_up64(t.high, SIDE) * tiles_n, experts ? experts : 1);
  return most_tiles(t.rows, experts, SIDE) * tiles_n;
}

template <int MODE, int SIDE, int WN, int WM>
void launch_side(const TileArgs& t, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(grid_of<MODE, SIDE>(t)), t.parts);
  product_kernel<MODE, SIDE, WN, WM><<<grid, 64 * WN * WM, 0, stream>>>(t);
}

template <int MODE>
void launch_tiles(const TileArgs& t, int shape, hipStream_t stream) {
  if (shape == kTile256) launch_side<MODE, 256, 2, 4>(t, stream);
  else if (shape == kTile128) launch_side<MODE, 128, 2, 2>(t, stream);
  else launch_side<MODE, 64, 2, 2>(t, stream);
}

template <int SIDE, int WN, int WM>
void launch_pair_side(PairArgs& p, hipStream_t stream) {
  p.each = div_up64(grid_of<kDw, SIDE>(p.w), 8) * 8;
  p.end = p.each * p.w.parts + grid_of<kDx, SIDE>(p.x);
  const int64_t sums = p.dbias ? p.groups * (p.w.offsets ? p.w.experts : 1) : 0;
  pair_kernel<SIDE, WN, WM><<<static_cast<unsigned>(p.end + sums), 64 * WN * WM, 0, stream>>>(p);
}

void launch_pair(PairArgs& p, int shape, hipStream_t stream) {
  if (shape == kTile256) launch_pair_side<256, 2, 4>(p, stream);
  else if (shape == kTile128) launch_pair_side<128, 2, 2>(p, stream);
  else launch_pair_side<64, 2, 2>(p, stream);
}

void launch_stream(const TileArgs& t, bool glu, hipStream_t stream) {
  const int64_t groups = div_up64(t.depth * kSize, kBlockBytes);
  const int waves = static_cast<int>(div_up64(groups, div_up64(groups, kStreamWaves)));
  const int64_t y = !t.offsets ? 1 : t.rows < t.experts ? t.rows : t.experts;
  const dim3 grid(static_cast<unsigned>(div_up64(t.cols, 16)), static_cast<unsigned>(y));
  if (glu) stream_kernel<true><<<grid, 64 * waves, 0, stream>>>(t);
  else stream_kernel<false><<<grid, 64 * waves, 0, stream>>>(t);
}

void launch_join(const TileArgs& t, int64_t rows, bool of_rows, int act, hipStream_t stream) {
  JoinArgs j = {};
  j.part = t.part;
  j.parts = t.parts;
  j.act = act;
  j.out_f32 = t.out_f32;
  j.part_stride = t.part_stride;
  j.rows = rows;
  j.cols = t.cols;
  j.offsets = of_rows ? t.offsets : nullptr;
  j.experts = t.offsets ? t.experts : 0;
  j.bias = t.bias;
  j.residual = t.residual;
  j.out = t.out;
  j.pre = t.pre;
  join_kernel<<<static_cast<unsigned>(div_up64(rows * div_up64(t.cols, 4), 256)), 256, 0, stream>>>(j);
}

int64_t ld_dpre(const ProductArgs& a) { return div_up64(a.nw(), 8) * 8; }

struct BwdLayout {
  Plan dx, dw;
  bool pair;                // both products by one launch
  bool bend;                // a pass over dout is needed
  int64_t dpre, bias, parts, total;  // bytes
  int64_t tiles;
};

BwdLayout bwd_layout(const ProductArgs& a) {
  BwdLayout l = {};
  // the products' dpre; dout serves as it unless its rows are not whole runs of 16 bytes
  const bool copy = (a.dx || a.dw) && (a.act != kNoAct || a.out_dtype != a.dtype || a.n % 8);
  l.bend = copy || a.dbias;
  l.dpre = copy ? up16(a.rows * ld_dpre(a) * kSize) : 0;
  l.tiles = most_tiles(a.rows, a.experts, bend_rows(a.rows, a.n));
  l.bias = a.dbias ? up16(l.tiles * a.nw() * 4) : 0;
  if (a.dx) {
    l.dx = plan_tiles(a, kDx);
    l.parts = parts_bytes(a, kDx, l.dx);
  }
  if (a.dw) {
    l.dw = plan_tiles(a, kDw);
    if (a.dx) {
      const Plan both = plan_pair(a, l.dx, l.dw);
      l.pair = both.shape != kStream;
      if (l.pair) {
        l.dx = {both.shape, 1, 0.0};
        l.dw = both;
        l.parts = 0;
      }
    }
    const int64_t b = parts_bytes(a, kDw, l.dw);
    l.parts = b > l.parts ? b : l.parts;  // one after the other: the same place
  }
  l.total = l.dpre + l.bias + l.parts;
  return l;
}

}  // namespace

#if SSM_LINEAR_DTYPE == 0
#define SSM_TYPED(name) name##_f32
#else
#define SSM_TYPED(name) name##_bf16
#endif

int64_t SSM_TYPED(product_fwd_work)(const ProductArgs& a) {
  const int mode = is_gated(a.act) ? kGlu : kFwd;
  return parts_bytes(a, mode, plan_tiles(a, mode));
}

int64_t SSM_TYPED(product_bwd_work)(const ProductArgs& a) { return bwd_layout(a).total; }

hipError_t SSM_TYPED(launch_product_fwd)(const ProductArgs& a, hipStream_t stream) {
  const bool glu = is_gated(a.act);
  const Plan q = plan_tiles(a, glu ? kGlu : kFwd);
  TileArgs t = {};
  t.a = a.w;
  t.b = a.x;
  t.lda = a.k;
  t.ldb = a.ld_x;
  t.stride_a = a.nw() * a.k;
  t.cols = a.n;
  t.depth = a.k;
  t.rows = a.rows;
  t.x_rows = a.x_rows;
  t.token = a.token;
  t.offsets = a.experts ? a.offsets : nullptr;
  t.experts = a.experts;
  t.act = a.act;
  t.parts = q.parts;
  t.out_f32 = a.out_dtype == 0;
  t.bias = a.bias;
  t.residual = a.residual;
  t.out = a.out;
  t.pre = a.pre;
  t.part = static_cast<float*>(a.work);
  t.part_stride = a.rows * a.nw();
  if (q.shape == kStream) {
    launch_stream(t, glu, stream);
  } else {
    if (glu) launch_tiles<kGlu>(t, q.shape, stream);
    else launch_tiles<kFwd>(t, q.shape, stream);
    if (q.parts > 1) launch_join(t, a.rows, true, a.act, stream);
  }
  return hipGetLastError();
}

hipError_t SSM_TYPED(launch_product_bwd)(const ProductArgs& a, hipStream_t stream) {
  const BwdLayout l = bwd_layout(a);
  char* work = static_cast<char*>(a.work);
  const int64_t nw = a.nw();
  const int32_t* offsets = a.experts ? a.offsets : nullptr;
  const void* dpre = a.dout;
  BendArgs b = {};
  const int64_t sums = div_up64(nw, 64);  // workgroups an expert for dbias
  if (l.bend) {
    b.dout = a.dout;
    b.pre = a.pre;
    b.dpre = l.dpre ? work : nullptr;
    b.part = l.bias ? reinterpret_cast<float*>(work + l.dpre) : nullptr;
    b.offsets = offsets;
    b.experts = a.experts;
    b.act = a.act;
    b.tile = bend_rows(a.rows, a.n);
    b.rows = a.rows;
    b.n = a.n;
    b.ld = ld_dpre(a);
    b.max_tiles = l.tiles;
    const dim3 grid(static_cast<unsigned>(l.tiles), static_cast<unsigned>(div_up64(a.n, 512)));
    if (a.out_dtype == 0) bend_kernel<float><<<grid, 256, 0, stream>>>(b);
    else bend_kernel<bf16_t><<<grid, 256, 0, stream>>>(b);
    if (l.bias && !l.pair) {
      const dim3 grid(static_cast<unsigned>(sums), a.experts ? a.experts : 1);
      bias_kernel<<<grid, 1024, 0, stream>>>(b, a.dbias);
    }
    if (l.dpre) dpre = work;
  }
  const int64_t matrices = a.experts ? a.experts : 1;
  TileArgs x = {};
  x.rows = a.rows;
  x.x_rows = a.x_rows;
  x.offsets = offsets;
  x.experts = a.experts;
  x.out_f32 = a.dtype == 0;
  x.part = reinterpret_cast<float*>(work + l.dpre + l.bias);
  x.b = dpre;
  x.ldb = ld_dpre(a);
  x.cols = a.k;
  TileArgs w = x;
  x.a = a.w;
  x.lda = a.k;
  x.stride_a = nw * a.k;
  x.depth = nw;
  x.out = a.dx;
  x.parts = l.dx.parts;
  x.part_stride = a.rows * a.k;
  w.a = a.x;
  w.lda = a.ld_x;
  w.high = nw;
  w.token = a.token;
  w.out = a.dw;
  w.parts = l.dw.parts;
  w.part_stride = matrices * nw * a.k;
  if (l.pair) {
    PairArgs p = {w, x, b, a.dbias, 0, 0, sums};
    launch_pair(p, l.dw.shape, stream);
  }
  if (a.dx && !l.pair) {
    launch_tiles<kDx>(x, l.dx.shape, stream);
    if (x.parts > 1) launch_join(x, a.rows, true, kNoAct, stream);
  }
  if (a.dw) {
    if (!l.pair) launch_tiles<kDw>(w, l.dw.shape, stream);
    if (w.parts > 1) launch_join(w, matrices * nw, false, kNoAct, stream);
  }
  return hipGetLastError();
}

#if SSM_LINEAR_DTYPE == 0
// The entry points' calls, by type.
int64_t product_fwd_work_bf16(const ProductArgs& a);
int64_t product_bwd_work_bf16(const ProductArgs& a);
hipError_t launch_product_fwd_bf16(const ProductArgs& a, hipStream_t stream);
hipError_t launch_product_bwd_bf16(const ProductArgs& a, hipStream_t stream);

int64_t product_fwd_work(const ProductArgs& a) {
  return a.dtype == 0 ? product_fwd_work_f32(a) : product_fwd_work_bf16(a);
}
int64_t product_bwd_work(const ProductArgs& a) {
  return a.dtype == 0 ? product_bwd_work_f32(a) : product_bwd_work_bf16(a);
}
hipError_t launch_product_fwd(const ProductArgs& a, hipStream_t stream) {
  return a.dtype == 0 ? launch_product_fwd_f32(a, stream) : launch_product_fwd_bf16(a, stream);
}
hipError_t launch_product_bwd(const ProductArgs& a, hipStream_t stream) {
  return a.dtype == 0 ? launch_product_bwd_f32(a, stream) : launch_product_bwd_bf16(a, stream);
}
#endif

}  // namespace ssm
