// attend.hip -- attention of one new token over a paged key / value cache.
//
// For each query head of each sequence, over its positions j in [lo, n): s_j = q . k_j, and with m = max s and
// p_j = exp(scale (s_j - m)):  out = sum p_j v_j / sum p_j,  lse = scale m + log sum p_j,  weight_j = p_j / sum p_j.
//
// One pass over the cache: the running maximum m, the sum and the accumulated output of what a wave has seen are rescaled when
// the maximum grows. Both products go through the matrix cores with up to 16 query heads that share a key / value head as the
// 16 columns: S^T = K Q^T, then O^T = V^T P^T. Few of their rates are needed (a wave's tile of 32 positions x 128 dims takes 8 + 16
// products, about 5% of the time its 16 KB take at the chip's read rate), so columns without a head and P in two parts cost
// nothing, and the cache's bytes bound the kernel. In the layouts of these products (lane l: g = l / 16, i = l % 16)
//   A and B operands   row or column i, contraction indexes g * 8 .. + 8 (fp32: g),
//   results            column i, rows g * 4 .. + 4,
// a lane's results S^T[positions g * 4 .. + 4][head i] are exactly its part of the second product's B operand, with the
// contraction running over positions in the order (g, half tile, r): P never leaves its lanes. Its A operand has to
// bring dim i of those positions: lane (g, i) loads 8 consecutive dims i * 8 of each of its positions, 16 bytes, so that 16 lanes
// read a position's whole row, and the 8 x 8 block is turned in registers (fp32 needs no turning). No LDS and no
// barrier between the loads and the products.
//
// P is rounded to 16 bits twice, hi = P and lo = P - hi, and both are multiplied: what is lost is 2^-17 of a weight
// (bf16) or less, where a single rounding would lose 2^-9, more than the output's own rounding when many weights
// cancel. fp16's P carries a factor of 2^15, so that weights down to 2^-39 of the largest stay above fp16's smallest number.
// m, sums and outputs are fp32.
//
// The work is the list of all rows' tiles (a row: 16 query heads of a sequence), cut into equal stretches, one for each wave that
// the chip holds at once: ragged batches and few long rows fill it alike, and waves wait for each other once, at the
// end. A row that lies in one stretch is finished by its wave, one that lies in a workgroup's stretches by the workgroup;
// the workgroups' parts of others (at most two a workgroup) are joined by a second kernel.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "topselect.h"
#include "ts_device.hpp"
#include "ts_host.hpp"
#include "ts_logits.hpp"
#include "ts_pages.hpp"

using namespace tsd;
using tsh::check_device;
using tsh::fail;
using tsl::u32x4;
using tsp::Divisor;

namespace {

constexpr int kAT = 256;       // threads
constexpr int kAW = kAT / 64;  // waves; each takes every kAW-th tile of a segment
constexpr int kCols = 16;      // query heads a row
constexpr int kMaxDim = 256;
enum { kFull, kPart, kTiny };  // a head's dims: the padded ones, fewer, fewer than 16 bytes
#ifdef EXP_NT
#define LOADK tsl::load16_once
#else
#define LOADK tsl::load16
#endif

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Layout of a type and of a head's dims padded to DP.
template <int DT, int DP>
struct Shape {
  static constexpr bool kF32 = DT == TS_DTYPE_F32;
  static constexpr int kSize = kF32 ? 4 : 2;
  static constexpr int kTok = kF32 ? 16 : 32;                // positions a tile
  static constexpr int kHalves = kTok / 16;
  static constexpr int kKC = DP * kSize / 64;                // 16-byte pieces of a key a lane
  static constexpr int kCW = kF32 ? 4 : (DP >= 128 ? 8 : 4); // consecutive dims of a value a lane
  static constexpr int kNP = DP / (16 * kCW);                // times
  static constexpr int kVR = kF32 ? 4 : 8;                   // positions whose values a lane loads
  static constexpr int kAcc = kNP * kCW;                     // result vectors
  static constexpr float kBias = DT == TS_DTYPE_F16 ? 15.0f : 0.0f;
};

struct AParams {
  const char *q, *k, *v;
  int64_t q_b, q_h, k_page, k_head, k_slot, v_page, v_head, v_slot;   // bytes
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lengths;
  int32_t batch, q_heads, kv_heads, group, head_tiles, dim, pages, page_slots, max_len, window;
  Divisor by_page;
  float scale, c;                 // c = scale log2(e)
  char* out;
  int64_t out_b, out_h;
  float* lse;
  int32_t* status;
  char* weights;
  int64_t w_b, w_h;               // bytes
  int32_t w_slots;
  float* score;                   // [batch * q_heads, score_stride]: s_j, where weights are asked for
  int64_t score_stride;
  float2* norm;                   // [batch * q_heads]: the row's m and 1 / sum (with fp16's factor), for the weights
  int64_t* start;                 // [batch + 1]: tiles of the sequences before; then the share's size
  float* part;                    // [workgroups, 2, part_floats]
  int32_t whole;                  // a workgroup a row, no parts
  int32_t tiny;                   // a row shorter than 16 bytes
  int32_t end_block;              // the block of 64 bytes in which a row ends, -1: with its 16 bytes
};

__device__ __forceinline__ int rows_of(const AParams& P) { return P.kv_heads * P.head_tiles; }

// A sequence's positions [lo, n) and status.
struct Span {
  int32_t lo, n, status;
};
__device__ __forceinline__ Span span_of(const AParams& P, int b) {
  const int32_t n = P.lengths[b];
  if (n < 0 || n > P.max_len) return Span{0, 0, TS_ROW_BAD_LENGTH};
  return Span{P.window > 0 ? max(0, n - P.window) : 0, n, TS_ROW_OK};
}
template <int TOK>
__device__ __forceinline__ int32_t tiles_of(const Span& s) {
  return (s.n + TOK - 1) / TOK - s.lo / TOK;
}

// ------------------------------------------------------------------ loads
// BYTES of a row's dims. The loads take no branch for a dim below the padded one: a piece that would reach past the row's end is
// moved back to end with it (Piece below says where it starts), so every address is in the row. A row shorter than a piece
// (`tiny`) is loaded by elements.
template <int BYTES>
__device__ __forceinline__ void load_piece(uint32_t* to, const char* at) {
  if constexpr (BYTES == 16) {
    const u32x4 x = LOADK(at);
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = x[i];
  } else {
    const u32x2 x = *reinterpret_cast<const u32x2_any*>(at);
    to[0] = x[0];
    to[1] = x[1];
  }
}
template <int SIZE, int BYTES>
__device__ __forceinline__ void load_tiny(uint32_t* to, const char* row, int byte, int row_bytes) {
#pragma unroll
  for (int i = 0; i < BYTES / SIZE; ++i) {
    const int at = byte + i * SIZE;
    if (SIZE == 4) {
      to[i] = at < row_bytes ? *reinterpret_cast<const uint32_t*>(row + at) : 0;
    } else {
      const uint32_t x = at < row_bytes ? *reinterpret_cast<const uint16_t*>(row + at) : 0;
      to[i / 2] = (i & 1) ? to[i / 2] | x << 16 : x;
    }
  }
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The largest of the four lanes (16 apart) that hold a column.
__device__ __forceinline__ float column_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float column_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

template <int DT>
__device__ __forceinline__ f32x4 mma(const uint32_t* a, const uint32_t* b, f32x4 c) {
  if constexpr (DT == TS_DTYPE_BF16) {
    bf16x8 x, y;
    __builtin_memcpy(&x, a, 16);
    __builtin_memcpy(&y, b, 16);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
  } else {
    f16x8 x, y;
    __builtin_memcpy(&x, a, 16);
    __builtin_memcpy(&y, b, 16);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
  }
}

// Two fp32 values rounded to 16 bits, and what the rounding left over, rounded too.
template <int DT>
__device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& lo) {
  if constexpr (DT == TS_DTYPE_BF16) {
    // hi is cut off, not rounded: the rest is then never negative, and 2^-16 of the value at the rounding of lo
    const uint32_t ua = __float_as_uint(a) & 0xFFFF0000u, ub = __float_as_uint(b) & 0xFFFF0000u;
    hi = (ua >> 16) | ub;
    const __bf16 la = (__bf16)(a - __uint_as_float(ua)), lb = (__bf16)(b - __uint_as_float(ub));
    lo = (uint32_t)__builtin_bit_cast(unsigned short, la) | ((uint32_t)__builtin_bit_cast(unsigned short, lb) << 16);
  } else {
    const _Float16 ha = (_Float16)a, hb = (_Float16)b;
    const _Float16 la = (_Float16)(a - (float)ha), lb = (_Float16)(b - (float)hb);
    hi = (uint32_t)__builtin_bit_cast(unsigned short, ha) | ((uint32_t)__builtin_bit_cast(unsigned short, hb) << 16);
    lo = (uint32_t)__builtin_bit_cast(unsigned short, la) | ((uint32_t)__builtin_bit_cast(unsigned short, lb) << 16);
  }
}

// ------------------------------------------------------------------ where a tile's positions lie
// UNI: pages of a multiple of 16 slots, so that each half tile lies in one page. Positions outside [lo, n) are replaced by the
// nearest inside (a half tile as a whole first, so that it stays in one page): their loads are in bounds, of attended
// positions' pages only, and what they bring is masked.
template <int HALVES, bool UNI>
struct Place {
  int64_t page[HALVES];          // UNI: of the half tile; else of position i of it, in lane i
  int32_t slot[HALVES];          // of position 0 of the half tile (UNI) or of position i
  int32_t base[HALVES];          // UNI: the half tile's first position
  __device__ __forceinline__ void find(const AParams& P, const int32_t* table, int first, int lo, int n, bool& bad) {
    const int i = lane() & 15;
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      int j = first + 16 * h;
      if constexpr (UNI) {
        j = max(min(j, (n - 1) & ~15), lo & ~15);
        base[h] = j;
      } else {
        j = max(min(j + i, n - 1), lo);
      }
      const int at = (int)P.by_page.of((uint32_t)j);
      slot[h] = j - at * P.page_slots;
      int32_t id = table[at];
      const bool out = (uint32_t)id >= (uint32_t)P.pages;
      bad = bad || out;
      page[h] = out ? 0 : id;
    }
  }
};

// ------------------------------------------------------------------ a wave's running state
__device__ const uint32_t zeros[4] = {0, 0, 0, 0};

template <int DT, int DP, int MODE, bool UNI>
struct Wave {
  using S = Shape<DT, DP>;
  static constexpr bool FULL = MODE == kFull;
  uint32_t q[S::kKC][4];
  uint32_t k[S::kHalves][S::kKC][4];
  uint32_t v[S::kVR][S::kNP][S::kCW * S::kSize / 4];
  f32x4 o[S::kAcc];
  uint32_t keep[4];
  float m, l;

  // A piece that would reach past the row's end is moved back to end with it, and its first bytes, another piece's, are cleared
  // before use: they lie in the one block of 64 bytes in which the row ends. Pieces past the end come from zeros.
  __device__ __forceinline__ void prepare(const AParams& P) {
    if constexpr (MODE == kPart) {
      const int end = P.dim * S::kSize, over = end / 64 * 64 + (lane() >> 4) * 16 + 16 - end;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int skip = over >= 16 ? 0 : min(4, max(0, over - 4 * w));
        keep[w] = skip == 4 ? 0u : 0xFFFFFFFFu << (8 * skip);
      }
    }
  }
  __device__ __forceinline__ void clear(const AParams& P, int c, uint32_t* x) const {
    if constexpr (MODE == kPart) {
      if (c != P.end_block) return;   // the same for all lanes
#pragma unroll
      for (int w = 0; w < 4; ++w) x[w] &= keep[w];
    }
  }
  __device__ __forceinline__ void load_row(const AParams& P, uint32_t (*to)[4], const char* row) const {
    const int g = lane() >> 4, end = P.dim * S::kSize;
    if constexpr (MODE == kTiny) {
#pragma unroll
      for (int c = 0; c < S::kKC; ++c) load_tiny<S::kSize, 16>(to[c], row, c * 64 + g * 16, end);
      return;
    }
#pragma unroll
    for (int c = 0; c < S::kKC; ++c) {
      const int byte = c * 64 + g * 16;
      const char* at = row + byte;
      if constexpr (!FULL) at = byte < end ? row + min(byte, end - 16) : reinterpret_cast<const char*>(zeros);
      load_piece<16>(to[c], at);
    }
  }
  __device__ __forceinline__ void clear_state() {
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int a = 0; a < S::kAcc; ++a) o[a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  __device__ __forceinline__ void load_q(const AParams& P, int b, int head0, int heads) {
    const int i = lane() & 15;
    load_row(P, q, P.q + b * P.q_b + (int64_t)(head0 + min(i, heads - 1)) * P.q_h);
#pragma unroll
    for (int c = 0; c < S::kKC; ++c) {
      clear(P, c, q[c]);
      if (i >= heads) q[c][0] = q[c][1] = q[c][2] = q[c][3] = 0;
    }
  }
  __device__ __forceinline__ void load_k(const AParams& P, const char* kh, const Place<S::kHalves, UNI>& at, int first, int lo, int n) {
    const int i = lane() & 15;
#pragma unroll
    for (int h = 0; h < S::kHalves; ++h) {
      int32_t slot = at.slot[h];
      if constexpr (UNI) slot += max(min(first + 16 * h + i, n - 1), lo) - at.base[h];
      load_row(P, k[h], kh + at.page[h] * P.k_page + (int64_t)slot * P.k_slot);
    }
  }
  __device__ __forceinline__ void load_v(const AParams& P, const char* vh, const Place<S::kHalves, UNI>& at, int first, int lo, int n) {
    const int g = lane() >> 4, i = lane() & 15, end = P.dim * S::kSize;
    constexpr int bytes = S::kCW * S::kSize;
#pragma unroll
    for (int x = 0; x < S::kVR; ++x) {
      const int h = x >> 2, in = g * 4 + (x & 3);
      int64_t page = at.page[h];
      int32_t slot = at.slot[h];
      if constexpr (UNI) {
        slot += max(min(first + 16 * h + in, n - 1), lo) - at.base[h];
      } else {
        page = __shfl((int32_t)page, in);
        slot = __shfl(slot, in);
      }
      const char* row = vh + page * P.v_page + (int64_t)slot * P.v_slot;
#pragma unroll
      for (int p = 0; p < S::kNP; ++p) {
        const int byte = (p * 16 + i) * bytes;
        if constexpr (MODE == kTiny) load_tiny<S::kSize, bytes>(v[x][p], row, byte, end);
        else load_piece<bytes>(v[x][p], row + (FULL ? byte : min(byte, end - bytes)));   // what lies past the dims is not stored
      }
    }
  }
  // Scores of the loaded keys: s[h][r] is position first + 16 h + 4 g + r under head i.
  __device__ __forceinline__ void scores(const AParams& P, f32x4* s) {
#pragma unroll
    for (int h = 0; h < S::kHalves; ++h) {
      s[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < S::kKC; ++c) {
        clear(P, c, k[h][c]);
        if constexpr (S::kF32) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[h] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[h][c][j]), __uint_as_float(q[c][j]), s[h], 0, 0, 0);
        } else {
          s[h] = mma<DT>(k[h][c], q[c], s[h]);
        }
      }
    }
  }
  // Positions outside [lo, n): no score, and values that cannot disturb.
  __device__ __forceinline__ void mask(f32x4* s, int first, int lo, int n) {
    const int g = lane() >> 4;
#pragma unroll
    for (int x = 0; x < S::kVR; ++x) {
      const int j = first + 16 * (x >> 2) + g * 4 + (x & 3);
      if (j < lo || j >= n) {
        s[x >> 2][x & 3] = -INFINITY;
#pragma unroll
        for (int p = 0; p < S::kNP; ++p)
#pragma unroll
          for (int w = 0; w < S::kCW * S::kSize / 4; ++w) v[x][p][w] = 0;
      }
    }
  }
  __device__ __forceinline__ void weigh(f32x4* s, float c) {
    float top = -INFINITY;
#pragma unroll
    for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
      for (int r = 0; r < 4; ++r) top = fmaxf(top, s[h][r]);
    if (__builtin_amdgcn_ballot_w64(top > m) != 0) {
      const float grown = fmaxf(m, column_max(top));
      const float f = m == grown ? 1.0f : exp2_fast((m - grown) * c);
      m = grown;
      l *= f;
#pragma unroll
      for (int a = 0; a < S::kAcc; ++a) o[a] *= f;
    }
    const float base = m == -INFINITY ? 0.0f : m;   // no score yet: exp2(-inf) below, not of a NaN
#pragma unroll
    for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[h][r] = exp2_fast((s[h][r] - base) * c + S::kBias);
        l += s[h][r];
      }
  }
  __device__ __forceinline__ void accumulate(const f32x4* s) {
    if constexpr (S::kF32) {
#pragma unroll
      for (int p = 0; p < S::kNP; ++p)
#pragma unroll
        for (int n = 0; n < S::kCW; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            o[p * S::kCW + n] =
                __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(v[r][p][n]), s[0][r], o[p * S::kCW + n], 0, 0, 0);
    } else {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) split<DT>(s[x >> 1][2 * (x & 1)], s[x >> 1][2 * (x & 1) + 1], hi[x], lo[x]);
#pragma unroll
      for (int p = 0; p < S::kNP; ++p)
#pragma unroll
        for (int n = 0; n < S::kCW; ++n) {
          uint32_t a[4];   // dim n of the lane's eight positions
#pragma unroll
          for (int x = 0; x < 4; ++x)
            a[x] = __builtin_amdgcn_perm(v[2 * x + 1][p][n >> 1], v[2 * x][p][n >> 1], (n & 1) ? 0x07060302u : 0x05040100u);
          o[p * S::kCW + n] = mma<DT>(a, hi, o[p * S::kCW + n]);
          o[p * S::kCW + n] = mma<DT>(a, lo, o[p * S::kCW + n]);
        }
    }
  }
};

// CW results of a head, the dims from d0 on, rounded once. (The values' piece there was moved back to end with the row.)
template <int DT, int CW>
__device__ __forceinline__ void store_dims(char* row, int d0, int dim, bool tiny, const float* x) {
  const int at = tiny ? d0 : min(d0, dim - CW);
#pragma unroll
  for (int n = 0; n < CW; ++n) {
    if (at + n < d0 || at + n >= dim) continue;
    if constexpr (DT == TS_DTYPE_F32) reinterpret_cast<float*>(row)[at + n] = x[n];
    else if constexpr (DT == TS_DTYPE_BF16) reinterpret_cast<__bf16*>(row)[at + n] = (__bf16)x[n];
    else reinterpret_cast<_Float16*>(row)[at + n] = (_Float16)x[n];
  }
}

// What a workgroup leaves of a row that it has a part of: the results of every lane, then m and the sum of every column, and
// whether a page number was outside the cache.
template <int DT, int DP>
constexpr int kPartFloats = Shape<DT, DP>::kAcc * 4 * 64 + 2 * kCols + 64;

struct RowOut {
  int b, head0, heads;
};
__device__ __forceinline__ RowOut row_out(const AParams& P, int b, int r) {
  const int hk = r / P.head_tiles, ht = r - hk * P.head_tiles;
  return RowOut{b, hk * P.group + ht * kCols, min(kCols, P.group - ht * kCols)};
}

// A column's lse and norm, by lanes i < heads of one wave. `sum` carries fp16's factor 2^bias.
__device__ __forceinline__ void store_norm(const AParams& P, const RowOut& R, float m, float sum, float bias, int status) {
  const int i = lane();
  if (i >= R.heads) return;
  const int64_t at = (int64_t)R.b * P.q_heads + R.head0 + i;
  if (P.lse) P.lse[at] = status != TS_ROW_OK ? NAN : sum == 0.0f ? -INFINITY : m * P.scale + logf(ldexpf(sum, -(int)bias));
  if (P.norm) P.norm[at] = status != TS_ROW_OK ? float2{0.0f, NAN} : float2{m, sum == 0.0f ? 0.0f : 1.0f / sum};
}

// ------------------------------------------------------------------ the pass over the cache
// A tile of a row, and how many are left of a wave's stretch, this one included.
struct Cursor {
  int32_t b, r;                  // sequence and its row
  int32_t lo, n, tiles;          // of the sequence
  int32_t tile;                  // of the row
  int64_t left;
};
template <int TOK>
__device__ __forceinline__ void enter(const AParams& P, Cursor& c, int b) {
  const Span span = span_of(P, b);
  c.b = b;
  c.lo = span.lo;
  c.n = span.n;
  c.tiles = tiles_of<TOK>(span);
}
template <int TOK>
__device__ __forceinline__ bool advance(const AParams& P, Cursor& c) {
  if (--c.left <= 0) return false;
  if (++c.tile < c.tiles) return true;
  c.tile = 0;
  if (++c.r < rows_of(P)) return true;
  c.r = 0;
  do {
    enter<TOK>(P, c, c.b + 1);
  } while (c.tiles == 0);   // there are tiles left, so a sequence with some follows
  return true;
}
// The wave's stretch of the list of all tiles. Every wave adds up the tiles of all sequences by itself (lane x takes some
// sequences in a row), so that no barrier stands before the first loads.
template <int TOK>
__device__ __forceinline__ bool begin(const AParams& P, int wv, Cursor& c) {
  const int rows = rows_of(P), own = (P.batch + 63) / 64, first = min(P.batch, lane() * own), last = min(P.batch, first + own);
  uint64_t sum = 0;
  for (int x = first; x < last; ++x) sum += (uint64_t)tiles_of<TOK>(span_of(P, x)) * rows;
  const uint64_t incl = wave_incl_scan64(sum), total = readlane64(incl, 63);
  const int64_t groups = gridDim.x * (int64_t)kAW;
  const int64_t stretch = max(((int64_t)total + groups - 1) / groups, (int64_t)1);
  const int64_t pos = (blockIdx.x * (int64_t)kAW + wv) * stretch;
  if (blockIdx.x == 0 && wv == 0) {
    int64_t at = (int64_t)(incl - sum);
    for (int x = first; x < last; ++x) {
      P.start[x] = at;
      at += (int64_t)tiles_of<TOK>(span_of(P, x)) * rows;
    }
    if (lane() == 0) {
      P.start[P.batch] = (int64_t)total;
      P.start[P.batch + 1] = stretch * kAW;
    }
  }
  if (pos >= (int64_t)total) return false;
  const uint64_t past = __builtin_amdgcn_ballot_w64((int64_t)incl > pos);   // not 0: the last lane's is the total
  const int l = __builtin_ctzll(past);
  int64_t in = pos - (int64_t)readlane64(incl - sum, l);
  int b = l * own;
  for (;; ++b) {
    const int64_t n = (int64_t)tiles_of<TOK>(span_of(P, b)) * rows;
    if (in < n) break;
    in -= n;
  }
  enter<TOK>(P, c, b);
  c.left = min(stretch, (int64_t)total - pos);
  c.r = (int)(in / c.tiles);
  c.tile = (int32_t)(in - (int64_t)c.r * c.tiles);
  return true;
}

// What a wave leaves for its workgroup of a row that it has a part of.
struct Part {
  int32_t b, r;                  // b < 0: none
  int32_t begins, ends, bad;
};

template <int DT, int DP, int MODE, bool UNI>
__global__ __launch_bounds__(kAT, DP > 128 ? 1 : 2) void ts_attend_kernel(const AParams P) {
  using S = Shape<DT, DP>;
  constexpr int TOK = S::kTok;
  // A wave has at most two rows in part: the one that its stretch starts in and the one that it ends in.
  __shared__ float sm_o[kAW * 2][S::kAcc * 4][64];
  __shared__ float sm_m[kAW * 2][kCols], sm_l[kAW * 2][kCols];
  __shared__ Part sm_part[kAW * 2];
  const int wv = __builtin_amdgcn_readfirstlane(wave()), g = lane() >> 4, i = lane() & 15;
  Cursor c;
  bool have;
  if (P.whole) {
    const int rows = rows_of(P), b = blockIdx.x / (unsigned)rows;
    enter<TOK>(P, c, b);
    c.r = blockIdx.x - b * rows;
    const int own = (c.tiles + kAW - 1) / kAW;
    c.tile = wv * own;
    c.left = min(own, c.tiles - c.tile);
    have = c.left > 0;
    if (c.tiles == 0) {   // no positions, or none that the table could hold
      const int status = span_of(P, b).status;
      const RowOut R = row_out(P, b, c.r);
      float x[S::kCW];
#pragma unroll
      for (int e = 0; e < S::kCW; ++e) x[e] = status == TS_ROW_OK ? 0.0f : NAN;
      for (int y = wv; y < S::kNP * 4; y += kAW)
        if (i < R.heads)
          store_dims<DT, S::kCW>(P.out + b * P.out_b + (int64_t)(R.head0 + i) * P.out_h,
                                 (y >> 2) * 16 * S::kCW + (g * 4 + (y & 3)) * S::kCW, P.dim, P.tiny, x);
      if (wv == 0) {
        store_norm(P, R, -INFINITY, 0.0f, S::kBias, status);
        if (P.status && lane() == 0) P.status[b] = status;
      }
      return;
    }
  } else {
    have = begin<TOK>(P, wv, c);
  }
  if (lane() < 2) sm_part[wv * 2 + lane()].b = -1;
  Wave<DT, DP, MODE, UNI> W;
  W.prepare(P);
  Place<S::kHalves, UNI> at;
  auto position = [&](const Cursor& c) { return (c.lo / TOK + c.tile) * TOK; };
  auto find = [&](const Cursor& c, bool& bad) {
    at.find(P, P.table + (int64_t)c.b * P.table_stride, position(c), c.lo, c.n, bad);
  };
  auto load_q = [&](const Cursor& c) {
    const RowOut R = row_out(P, c.b, c.r);
    W.load_q(P, c.b, R.head0, R.heads);
  };
  auto load_k = [&](const Cursor& c) { W.load_k(P, P.k + (c.r / P.head_tiles) * P.k_head, at, position(c), c.lo, c.n); };
  auto load_v = [&](const Cursor& c) { W.load_v(P, P.v + (c.r / P.head_tiles) * P.v_head, at, position(c), c.lo, c.n); };
  bool bad = false;              // a page of the row so far was outside the cache
  int32_t begins = 1;            // the row's first tile was this wave's
  if (have) {
    find(c, bad);
    load_q(c);
    load_k(c);
    load_v(c);
    begins = c.tile == 0;
    W.clear_state();
  }
  while (have) {
    const int first = position(c);
    Cursor next = c;
    have = advance<TOK>(P, next);
    const bool ends = c.tile + 1 == c.tiles, other = ends || !have;   // the row, or this wave's part of it, ends here
    bool next_bad = false;
    f32x4 s[S::kHalves];
    if (have) find(next, next_bad);
    W.scores(P, s);
    if (have) {   // into the registers that the products have read
      if (ends) load_q(next);
      load_k(next);
    }
    if (first < c.lo || first + TOK > c.n) W.mask(s, first, c.lo, c.n);
    if (P.score) {
      const RowOut R = row_out(P, c.b, c.r);
      float* to = P.score + ((int64_t)c.b * P.q_heads + R.head0 + i) * P.score_stride + first + g * 4;
      if (i < R.heads) {
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h) *reinterpret_cast<f32x4*>(to + 16 * h) = s[h];
      }
    }
    W.weigh(s, P.c);
    W.accumulate(s);
    if (have) load_v(next);
    if (other) {
      const float l = column_sum(W.l);
      const bool spoilt = __builtin_amdgcn_ballot_w64(bad) != 0;
      if (begins && ends) {      // the row is this wave's alone
        const RowOut R = row_out(P, c.b, c.r);
        const float inv = spoilt ? NAN : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int x = 0; x < S::kNP * 4; ++x) {
          float y[S::kCW];
#pragma unroll
          for (int e = 0; e < S::kCW; ++e) y[e] = !spoilt && l == 0.0f ? 0.0f : W.o[(x >> 2) * S::kCW + e][x & 3] * inv;
          if (i < R.heads)
            store_dims<DT, S::kCW>(P.out + c.b * P.out_b + (int64_t)(R.head0 + i) * P.out_h,
                                   (x >> 2) * 16 * S::kCW + (g * 4 + (x & 3)) * S::kCW, P.dim, P.tiny, y);
        }
        store_norm(P, R, W.m, l, S::kBias, spoilt ? TS_ROW_BAD_PAGE : TS_ROW_OK);
        if (P.status && lane() == 0) P.status[c.b] = spoilt ? TS_ROW_BAD_PAGE : TS_ROW_OK;   // every row of a sequence finds the same
      } else {
        const int slot = wv * 2 + begins;
        if (lane() < kCols) {
          sm_m[slot][i] = W.m;
          sm_l[slot][i] = l;
        }
        if (lane() == 0) sm_part[slot] = Part{c.b, c.r, begins, ends, spoilt};
#pragma unroll
        for (int x = 0; x < S::kNP * 4; ++x)
#pragma unroll
          for (int e = 0; e < S::kCW; ++e) sm_o[slot][x * S::kCW + e][lane()] = W.o[(x >> 2) * S::kCW + e][x & 3];
      }
      W.clear_state();
      begins = 1;
      bad = false;
    }
    bad = bad || next_bad;
    c = next;
  }
  bar();
  // Parts of one row follow each other.
  for (int k = 0; k < kAW * 2;) {
    const Part head = sm_part[k];
    if (head.b < 0) {
      ++k;
      continue;
    }
    int end = k + 1, ends = head.ends, spoilt = head.bad;
    float m = sm_m[k][i];
    for (int j = k + 1; j < kAW * 2; ++j) {
      const Part p = sm_part[j];
      if (p.b < 0) continue;
      if (p.b != head.b || p.r != head.r) break;
      m = fmaxf(m, sm_m[j][i]);
      ends = p.ends;
      spoilt |= p.bad;
      end = j + 1;
    }
    const bool complete = head.begins && ends;
    float l = 0.0f, sum[S::kNP][S::kCW];
#pragma unroll
    for (int p = 0; p < S::kNP; ++p)
#pragma unroll
      for (int e = 0; e < S::kCW; ++e) sum[p][e] = 0.0f;
    for (int j = k; j < end; ++j) {
      if (sm_part[j].b < 0) continue;
      const float mj = sm_m[j][i], f = mj == m ? 1.0f : exp2_fast((mj - m) * P.c);   // also where both are -inf: no sum there but 0 or NaN
      l += f * sm_l[j][i];
#pragma unroll
      for (int p = 0; p < S::kNP; ++p)
#pragma unroll
        for (int e = 0; e < S::kCW; ++e) sum[p][e] += f * sm_o[j][(p * 4 + wv) * S::kCW + e][lane()];
    }
    const int status = spoilt ? TS_ROW_BAD_PAGE : TS_ROW_OK;
    const RowOut R = row_out(P, head.b, head.r);
    float* part = P.part + ((int64_t)blockIdx.x * 2 + head.begins) * kPartFloats<DT, DP>;
    const float inv = spoilt ? NAN : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int p = 0; p < S::kNP; ++p) {   // wave x: row x of the results
      if (complete) {
#pragma unroll
        for (int e = 0; e < S::kCW; ++e) sum[p][e] = !spoilt && l == 0.0f ? 0.0f : sum[p][e] * inv;
        if (i < R.heads)
          store_dims<DT, S::kCW>(P.out + head.b * P.out_b + (int64_t)(R.head0 + i) * P.out_h, p * 16 * S::kCW + (g * 4 + wv) * S::kCW,
                                 P.dim, P.tiny, sum[p]);
      } else {
#pragma unroll
        for (int e = 0; e < S::kCW; ++e) part[((p * 4 + wv) * S::kCW + e) * 64 + lane()] = sum[p][e];
      }
    }
    if (wv == 0) {
      if (complete) {
        store_norm(P, R, m, l, S::kBias, status);
        if (P.status && lane() == 0) P.status[head.b] = status;
      } else {
        float* tail = part + S::kAcc * 4 * 64;
        if (lane() < kCols) {
          tail[i] = m;
          tail[kCols + i] = l;
        }
        if (lane() == 0) tail[2 * kCols] = spoilt ? 1.0f : 0.0f;
      }
    }
    k = end;
  }
}

// ------------------------------------------------------------------ rows that several workgroups share
// A workgroup a row and one of its 4 passes of results; its waves take the parts in turn, each with a running maximum.
template <int DT, int DP, int NW>
__global__ __launch_bounds__(NW * 64) void ts_attend_join_kernel(const AParams P) {
  using S = Shape<DT, DP>;
  __shared__ float sm_o[NW][S::kCW][64];
  __shared__ float sm_m[NW][64], sm_l[NW][64];
  __shared__ int any_bad;
  const int wv = __builtin_amdgcn_readfirstlane(wave()), g = lane() >> 4, i = lane() & 15;
  const int rows = rows_of(P), groups = S::kNP * 4;
  const int x = blockIdx.x % groups, row = blockIdx.x / groups, b = row / rows, r = row - b * rows;
  const int64_t share = P.start[P.batch + 1], before = P.start[b];
  const Span span = span_of(P, b);
  const int32_t tiles = tiles_of<S::kTok>(span);
  const RowOut R = row_out(P, b, r);
  const int64_t from = before + (int64_t)r * tiles;
  const int64_t w0 = from / share, w1 = tiles ? (from + tiles - 1) / share : w0;
  if (tiles && w0 == w1) return;   // finished by its workgroup
  constexpr int64_t size = kPartFloats<DT, DP>;
  const int count = tiles ? (int)(w1 - w0 + 1) : 0;
  // the first part is its workgroup's second one, as the row starts inside the share or with it
  const float* first = P.part + (w0 * 2 + 1) * size;
  if (threadIdx.x == 0) any_bad = 0;
  bool bad = false;
  float m = -INFINITY, l = 0.0f, sum[S::kCW];
#pragma unroll
  for (int c = 0; c < S::kCW; ++c) sum[c] = 0.0f;
#pragma unroll 4
  for (int p = wv; p < count; p += NW) {
    const float* part = p == 0 ? first : first + (2 * p - 1) * size;   // workgroup w0 + p, its first one
    const float* tail = part + S::kAcc * 4 * 64;
    const float mp = tail[i], lp = tail[kCols + i];
    bad = bad || tail[2 * kCols] != 0.0f;
    const float grown = fmaxf(m, mp);
    const float f = m == grown ? 1.0f : exp2_fast((m - grown) * P.c), fp = mp == grown ? 1.0f : exp2_fast((mp - grown) * P.c);
    m = grown;
    l = l * f + lp * fp;
#pragma unroll
    for (int c = 0; c < S::kCW; ++c) sum[c] = sum[c] * f + part[(x * S::kCW + c) * 64 + lane()] * fp;
  }
  bar();
  if (__builtin_amdgcn_ballot_w64(bad)) any_bad = 1;
  sm_m[wv][lane()] = m;
  sm_l[wv][lane()] = l;
#pragma unroll
  for (int c = 0; c < S::kCW; ++c) sm_o[wv][c][lane()] = sum[c];
  bar();
  if (wv != 0) return;
#pragma unroll 4
  for (int w = 1; w < NW; ++w) m = fmaxf(m, sm_m[w][lane()]);
  l = 0.0f;
#pragma unroll
  for (int c = 0; c < S::kCW; ++c) sum[c] = 0.0f;
#pragma unroll 4
  for (int w = 0; w < NW; ++w) {
    const float mw = sm_m[w][lane()], f = mw == m ? 1.0f : exp2_fast((mw - m) * P.c);
    l += f * sm_l[w][lane()];
#pragma unroll
    for (int c = 0; c < S::kCW; ++c) sum[c] += f * sm_o[w][c][lane()];
  }
  const int status = span.status != TS_ROW_OK ? span.status : any_bad ? TS_ROW_BAD_PAGE : TS_ROW_OK;
#pragma unroll
  for (int c = 0; c < S::kCW; ++c) sum[c] = status != TS_ROW_OK ? NAN : l == 0.0f ? 0.0f : sum[c] * (1.0f / l);
  if (i < R.heads)
    store_dims<DT, S::kCW>(P.out + b * P.out_b + (int64_t)(R.head0 + i) * P.out_h,
                           (x >> 2) * 16 * S::kCW + (g * 4 + (x & 3)) * S::kCW, P.dim, P.tiny, sum);
  if (x == 0) {
    store_norm(P, R, m, l, S::kBias, status);
    if (P.status && lane() == 0) P.status[b] = status;
  }
}

// ------------------------------------------------------------------ weights
// exp(scale (s - m)) / sum of every position, 0 outside [lo, n), from the stored scores.
constexpr int kWT = 256, kWE = 4;   // threads, positions a thread
template <int WT>
__global__ __launch_bounds__(kWT) void ts_attend_weights_kernel(const AParams P, float bias, int blocks) {
  const int64_t row = blockIdx.x / (unsigned)blocks;
  const int j0 = (int)((blockIdx.x - row * blocks) * kWT + threadIdx.x) * kWE;
  const int b = (int)(row / P.q_heads), head = (int)(row - (int64_t)b * P.q_heads);
  const Span span = span_of(P, b);
  const float2 norm = P.norm[row];
  const float base = norm.x == -INFINITY ? 0.0f : norm.x;
  const float* s = P.score + row * P.score_stride;
  char* to = P.weights + (int64_t)b * P.w_b + (int64_t)head * P.w_h;
  if (j0 >= P.w_slots) return;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (j0 < span.n && j0 + kWE > span.lo) x = *reinterpret_cast<const f32x4*>(s + j0);
#pragma unroll
  for (int e = 0; e < kWE; ++e) {
    const int j = j0 + e;
    if (j >= P.w_slots) return;
    float w = 0.0f;
    if (j >= span.lo && j < span.n) w = exp2_fast((x[e] - base) * P.c + bias) * norm.y;
    if (span.status != TS_ROW_OK || norm.y != norm.y) w = NAN;
    if constexpr (WT == TS_DTYPE_F32) reinterpret_cast<float*>(to)[j] = w;
    else if constexpr (WT == TS_DTYPE_BF16) reinterpret_cast<__bf16*>(to)[j] = (__bf16)w;
    else reinterpret_cast<_Float16*>(to)[j] = (_Float16)w;
  }
}

// ------------------------------------------------------------------ host side
constexpr unsigned kWideJoin = 512;   // workgroups of the join that have 16 waves: few rows have many parts each
// Workgroups of the pass: as many as the chip holds at once, by their registers and LDS.
constexpr int groups_of(int dp) { return dp == 64 ? 1024 : dp == 128 ? 512 : 256; }

int dtype_size(int dtype) {
  return dtype == TS_DTYPE_F32 ? 4 : (dtype == TS_DTYPE_BF16 || dtype == TS_DTYPE_F16) ? 2 : 0;
}
int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

struct APlan {
  int64_t rows = 0, score_stride = 0;
  size_t off_norm = 0, off_start = 0, off_part = 0, total = 0;
  bool whole = false;
};
// Rows of so few positions are left to one workgroup each: what would be joined is less than the join.
constexpr int64_t kWholeSlots = 256;

bool attend_plan(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim, int64_t max_len, int64_t w_slots, APlan& pl) {
  if (batch < 0 || batch > (1 << 24) || kv_heads < 1 || q_heads < kv_heads || q_heads > (1 << 16) || q_heads % kv_heads || dim < 1 ||
      dim > kMaxDim || max_len < 0 || max_len > 0x7FFFFF00 || w_slots < 0 || w_slots > 0x7FFFFF00)
    return false;
  const int64_t tiles = (q_heads / kv_heads + kCols - 1) / kCols;
  pl.rows = batch * kv_heads * tiles;
  if (pl.rows * 16 > (int64_t)0xFFFFFFFF / kAT) return false;
  pl.whole = max_len <= kWholeSlots;
  pl.score_stride = w_slots ? (w_slots + 31) / 32 * 32 : 0;
  if (w_slots && batch * q_heads * ((w_slots + kWT * kWE - 1) / (kWT * kWE)) > (int64_t)0xFFFFFFFF / kWT) return false;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
  };
  if (w_slots) {
    take((size_t)(batch * q_heads) * (size_t)pl.score_stride * 4);
    pl.off_norm = take((size_t)(batch * q_heads) * sizeof(float2));
  }
  if (!pl.whole) {
    pl.off_start = take((size_t)(batch + 2) * 8);
    const int dp = padded_dim((int)dim);
    pl.off_part = take((size_t)groups_of(dp) * 2 * (dp * 16 + 2 * kCols + 64) * 4);
  }
  pl.total = at;
  return true;
}

template <int DT, int DP, int MODE, bool UNI>
void launch_attend(const AParams& P, int64_t rows, hipStream_t s) {
  const unsigned grid = P.whole ? (unsigned)rows : (unsigned)groups_of(DP);
  hipLaunchKernelGGL((ts_attend_kernel<DT, DP, MODE, UNI>), dim3(grid), dim3(kAT), 0, s, P);
}

template <int DT, int DP>
hipError_t launch_type(AParams& P, int64_t rows, hipStream_t s) {
  static_assert(kPartFloats<DT, DP> == DP * 16 + 2 * kCols + 64, "a part's size");
  const bool uni = P.page_slots % 16 == 0;
  if (P.dim == DP) {
    if (uni) launch_attend<DT, DP, kFull, true>(P, rows, s);
    else launch_attend<DT, DP, kFull, false>(P, rows, s);
  } else if (!P.tiny) {
    if (uni) launch_attend<DT, DP, kPart, true>(P, rows, s);
    else launch_attend<DT, DP, kPart, false>(P, rows, s);
  } else if constexpr (DP == 64) {
    launch_attend<DT, DP, kTiny, false>(P, rows, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || P.whole) return e;
  const dim3 grid((unsigned)(rows * Shape<DT, DP>::kNP * 4));
  if (grid.x <= kWideJoin) hipLaunchKernelGGL((ts_attend_join_kernel<DT, DP, 16>), grid, dim3(1024), 0, s, P);
  else hipLaunchKernelGGL((ts_attend_join_kernel<DT, DP, 4>), grid, dim3(256), 0, s, P);
  return hipGetLastError();
}
template <int DT>
hipError_t launch_dim(AParams& P, int64_t rows, hipStream_t s) {
  switch (padded_dim(P.dim)) {
    case 64: return launch_type<DT, 64>(P, rows, s);
    case 128: return launch_type<DT, 128>(P, rows, s);
    default: return launch_type<DT, 256>(P, rows, s);
  }
}

}  // namespace

extern "C" size_t ts_cache_attend_workspace(int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len,
                                            int64_t weights_slots) {
  APlan pl;
  return attend_plan(batch, q_heads, kv_heads, dim, max_len, weights_slots, pl) ? pl.total : 0;
}

extern "C" int ts_cache_attend(const void* q, int dtype, int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t dim,
                               int64_t q_batch_stride, int64_t q_head_stride, const ts_paged* k_pages, const ts_paged* v_pages,
                               int64_t pages, int32_t page_slots, const int32_t* table, int64_t table_width, int64_t table_stride,
                               const int32_t* lengths, float scale, int32_t window, void* out, int64_t out_batch_stride,
                               int64_t out_head_stride, float* out_lse, void* out_weights, int weights_dtype,
                               int64_t weights_slots, int64_t weights_batch_stride, int64_t weights_head_stride,
                               int32_t* row_status, void* workspace, size_t workspace_bytes, void* stream) {
  const int size = dtype_size(dtype);
  if (!size) return fail(TS_ERR_INVALID_ARG, "dtype = %d is none of TS_DTYPE_*", dtype);
  if (batch < 0) return fail(TS_ERR_INVALID_ARG, "batch = %lld < 0", (long long)batch);
  if (kv_heads < 1 || q_heads < 1 || q_heads % kv_heads)
    return fail(TS_ERR_INVALID_ARG, "q_heads = %d is no multiple of kv_heads = %d", (int)q_heads, (int)kv_heads);
  if (q_heads > 1 << 16) return fail(TS_ERR_INVALID_ARG, "q_heads = %d is too large", (int)q_heads);
  if (dim < 1 || dim > kMaxDim) return fail(TS_ERR_INVALID_ARG, "dim = %d outside [1, %d]", (int)dim, kMaxDim);
  if (!(scale >= 0x1p-64f && scale <= 0x1p64f)) return fail(TS_ERR_INVALID_ARG, "scale = %g outside [2^-64, 2^64]", (double)scale);
  if (window < 0) return fail(TS_ERR_INVALID_ARG, "window = %d < 0", (int)window);
  int rc = tsp::check_table(pages, page_slots, table_width, table_stride);
  if (rc != TS_OK) return rc;
  const int w_size = dtype_size(weights_dtype);
  if (out_weights) {
    if (!w_size) return fail(TS_ERR_INVALID_ARG, "weights_dtype = %d is none of TS_DTYPE_*", weights_dtype);
    if (weights_slots < 1) return fail(TS_ERR_INVALID_ARG, "weights_slots = %lld < 1", (long long)weights_slots);
  } else if (weights_slots != 0 && batch > 0) {
    return fail(TS_ERR_INVALID_ARG, "weights_slots = %lld without out_weights", (long long)weights_slots);
  }
  if (batch == 0) return TS_OK;
  if (!q || (!table && table_width > 0) || !lengths || !out) return fail(TS_ERR_INVALID_ARG, "q, table, lengths and out are required (NULL given)");
  if (pages < 1) return fail(TS_ERR_INVALID_ARG, "pages = %lld < 1", (long long)pages);
  if ((uintptr_t)q % size || (uintptr_t)out % size || (out_weights && (uintptr_t)out_weights % w_size))
    return fail(TS_ERR_INVALID_ARG, "q, out or out_weights is not aligned to its type");
  if (!tsp::reaches(dim, {{q_batch_stride, batch}, {q_head_stride, q_heads}}, size))
    return fail(TS_ERR_INVALID_ARG, "q: negative or too large strides");
  if (!tsp::apart(dim, {{out_batch_stride, batch}, {out_head_stride, q_heads}}, size))
    return fail(TS_ERR_INVALID_ARG, "out: rows overlap, or negative or too large strides");
  if (out_weights && !tsp::apart(weights_slots, {{weights_batch_stride, batch}, {weights_head_stride, q_heads}}, w_size))
    return fail(TS_ERR_INVALID_ARG, "out_weights: rows overlap, or negative or too large strides");
  for (auto [c, name] : {std::pair{k_pages, "k_pages"}, std::pair{v_pages, "v_pages"}}) {
    if (!c || !c->data) return fail(TS_ERR_INVALID_ARG, "%s: data is NULL", name);
    if ((uintptr_t)c->data % size || c->page_stride % size || c->head_stride % size || c->slot_stride % size)
      return fail(TS_ERR_INVALID_ARG, "%s: address or strides are not aligned to the type", name);
    if (!tsp::reaches((int64_t)dim * size, {{c->page_stride, pages}, {c->head_stride, kv_heads}, {c->slot_stride, page_slots}}, 1))
      return fail(TS_ERR_INVALID_ARG, "%s: negative or too large strides", name);
  }
  APlan pl;
  const int64_t max_len = std::min<int64_t>(std::min<int64_t>(table_width * page_slots, tsp::kMaxLen),
                                            out_weights ? weights_slots : tsp::kMaxLen);
  if (!attend_plan(batch, q_heads, kv_heads, dim, max_len, weights_slots, pl))
    return fail(TS_ERR_INVALID_ARG, "batch x heads x slots too large");
  if (pl.total) {
    if (!workspace) return fail(TS_ERR_WORKSPACE, "workspace is NULL");
    if (((uintptr_t)workspace & 255u) != 0) return fail(TS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    if (workspace_bytes < pl.total) return fail(TS_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, pl.total);
  }
  int dev;
  rc = check_device(&dev);
  if (rc != TS_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  AParams P{};
  P.q = static_cast<const char*>(q);
  P.q_b = q_batch_stride * size;
  P.q_h = q_head_stride * size;
  P.k = static_cast<const char*>(k_pages->data);
  P.k_page = k_pages->page_stride;
  P.k_head = k_pages->head_stride;
  P.k_slot = k_pages->slot_stride;
  P.v = static_cast<const char*>(v_pages->data);
  P.v_page = v_pages->page_stride;
  P.v_head = v_pages->head_stride;
  P.v_slot = v_pages->slot_stride;
  P.table = table;
  P.table_stride = table_stride;
  P.lengths = lengths;
  P.batch = (int32_t)batch;
  P.q_heads = q_heads;
  P.kv_heads = kv_heads;
  P.group = q_heads / kv_heads;
  P.head_tiles = (P.group + kCols - 1) / kCols;
  P.dim = dim;
  P.pages = (int32_t)pages;
  P.page_slots = page_slots;
  P.max_len = (int32_t)max_len;
  P.window = window;
  P.by_page = Divisor(page_slots);
  P.scale = scale;
  P.c = (float)((double)scale * kLog2e);
  P.out = static_cast<char*>(out);
  P.out_b = out_batch_stride * size;
  P.out_h = out_head_stride * size;
  P.lse = out_lse;
  P.status = row_status;
  if (out_weights) {
    P.weights = static_cast<char*>(out_weights);
    P.w_b = weights_batch_stride * w_size;
    P.w_h = weights_head_stride * w_size;
    P.w_slots = (int32_t)weights_slots;
    P.score = reinterpret_cast<float*>(ws);
    P.score_stride = pl.score_stride;
    P.norm = reinterpret_cast<float2*>(ws + pl.off_norm);
  }
  P.start = reinterpret_cast<int64_t*>(ws + pl.off_start);
  P.part = reinterpret_cast<float*>(ws + pl.off_part);
  P.whole = pl.whole ? 1 : 0;
  P.tiny = dim * size < 16;
  P.end_block = dim * size % 16 ? dim * size / 64 : -1;
  const hipStream_t s = (hipStream_t)stream;
  hipError_t e = dtype == TS_DTYPE_F32    ? launch_dim<TS_DTYPE_F32>(P, pl.rows, s)
                 : dtype == TS_DTYPE_BF16 ? launch_dim<TS_DTYPE_BF16>(P, pl.rows, s)
                                          : launch_dim<TS_DTYPE_F16>(P, pl.rows, s);
  if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "attention launch failed: %s", hipGetErrorString(e));
  if (out_weights) {
    const int blocks = (int)((weights_slots + kWT * kWE - 1) / (kWT * kWE));
    const dim3 grid((unsigned)(batch * q_heads * blocks)), block(kWT);
    const float bias = dtype == TS_DTYPE_F16 ? Shape<TS_DTYPE_F16, 64>::kBias : 0.0f;
    if (weights_dtype == TS_DTYPE_F32) hipLaunchKernelGGL(ts_attend_weights_kernel<TS_DTYPE_F32>, grid, block, 0, s, P, bias, blocks);
    else if (weights_dtype == TS_DTYPE_BF16)
      hipLaunchKernelGGL(ts_attend_weights_kernel<TS_DTYPE_BF16>, grid, block, 0, s, P, bias, blocks);
    else hipLaunchKernelGGL(ts_attend_weights_kernel<TS_DTYPE_F16>, grid, block, 0, s, P, bias, blocks);
    e = hipGetLastError();
    if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "attention weights launch failed: %s", hipGetErrorString(e));
  }
  return TS_OK;
}
