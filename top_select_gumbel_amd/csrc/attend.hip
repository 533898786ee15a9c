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
// P is taken in two 16-bit parts, hi of P (bf16's cut off, fp16's rounded) and lo = P - hi rounded, and both are multiplied: what
// is lost is 2^-16 of a weight (fp16: 2^-22) or less, where a single rounding would lose 2^-8 (2^-11), more than the output's
// own rounding when many weights cancel. fp16's P carries a factor of 2^15, so that weights down to 2^-39 of the largest stay
// above fp16's smallest number; below 2^-18 of the largest, where lo has no normal numbers left, 2^-40 of the largest is lost.
// m, sums and outputs are fp32.
//
// The work is the list of all rows' tiles (a row: 16 query heads of a sequence), cut into equal stretches, one for each wave that
// the chip holds at once: ragged batches and few long rows fill it alike, and waves wait for each other once, at the
// end. A row that lies in one stretch is finished by its wave, one that lies in a workgroup's stretches by the workgroup;
// the workgroups' parts of others (at most two a workgroup) are joined by a second kernel.
//
// Measured, 32 query heads on 8 of 128 dims in bf16: 64 sequences of up to 4096 positions, 583 MB, 98 us for the pass (6.0 TB/s; a
// plain read 6.8) and 7 for the join; one of n positions 9.5 us at 2000, 17.9 at 16000, 88 at 128000 (524 MB), and 13.6 at 500,
// which takes no join. The first 7 us are a chain of misses (lengths, page numbers, keys); from there on the memory bounds it.
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
constexpr int kAW = kAT / 64;  // waves
constexpr int kCols = 16;      // query heads a row
constexpr int kMaxDim = 256;
enum { kFull, kPart, kTiny };  // a head's dims: the padded ones, fewer, fewer than 16 bytes

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
  static constexpr int kVR = kTok / 4;                       // positions whose values a lane holds
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
  int32_t w_dtype, join_blocks;
  int64_t w_b, w_h;               // bytes
  int32_t w_slots;
  float* score;                   // [batch * q_heads, score_stride]: s_j, where weights are asked for
  int64_t score_stride;
  float2* norm;                   // [batch * q_heads]: the row's m (NaN: it is refused) and 1 / sum (with fp16's factor), for the weights
  int64_t* start;                 // [batch + 1]: places of the sequences before; then how many workgroups share them
  float* part;                    // [workgroups, 2, part_floats]
  int32_t whole;                  // a workgroup a row, no parts
  int32_t once;                   // the cache does not fit the last-level cache, and is read once
  int32_t tiny;                   // a row shorter than 16 bytes
  int32_t end_block;              // the block of 64 bytes in which a row ends, -1: with its 16 bytes
};

__device__ __forceinline__ int rows_of(const AParams& P) { return P.kv_heads * P.head_tiles; }

// a / b of what hardly ever needs 64 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// A sequence's positions [lo, n) and status.
struct Span {
  int32_t lo, n, status;
};
__device__ __forceinline__ Span span_from(const AParams& P, int32_t n) {
  if (n < 0 || n > P.max_len) return Span{0, 0, TS_ROW_BAD_LENGTH};
  return Span{P.window > 0 ? max(0, n - P.window) : 0, n, TS_ROW_OK};
}
__device__ __forceinline__ Span span_of(const AParams& P, int b) { return span_from(P, P.lengths[b]); }
template <int TOK>
__device__ __forceinline__ int32_t tiles_of(const Span& s) {
  return (s.n + TOK - 1) / TOK - s.lo / TOK;
}

// ------------------------------------------------------------------ loads
// BYTES of a row. The loads take no branch for a dim below the padded one: a piece that would reach past the row's end is moved back
// to end with it, so every address is in the row. (With a branch a piece, heads of 80 fp32 dims took 24 us where these take 9.)
// A row shorter than a piece (kTiny) is loaded by elements. ONCE: past the caches.
template <int BYTES, bool ONCE>
__device__ __forceinline__ void load_piece(uint32_t* to, const char* at) {
  if constexpr (BYTES == 16) {
    const u32x4 x = ONCE ? tsl::load16_once(at) : tsl::load16(at);
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = x[i];
  } else {
    const u32x2 x = ONCE ? __builtin_nontemporal_load(reinterpret_cast<const u32x2_any*>(at)) : *reinterpret_cast<const u32x2_any*>(at);
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

// Two fp32 values in 16 bits, and what that left over, rounded to 16 bits too.
template <int DT>
__device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& lo) {
  if constexpr (DT == TS_DTYPE_BF16) {
    // hi is cut off (one operation less than rounded): the rest is below 2^-7 of the value, and lo loses half a step of that, 2^-16
    // of the value at most
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

template <int DT, int DP, int MODE, bool UNI, bool ONCE>
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
      load_piece<16, ONCE>(to[c], at);
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
        else load_piece<bytes, ONCE>(v[x][p], row + (FULL ? byte : min(byte, end - bytes)));   // what lies past the dims is not stored
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

template <int DT>
__device__ __forceinline__ uint32_t round16(float x) {
  if constexpr (DT == TS_DTYPE_BF16) return __builtin_bit_cast(unsigned short, (__bf16)x);
  else return __builtin_bit_cast(unsigned short, (_Float16)x);
}
// Results e0 .. + CE of the CW of a head's dims from d0 on, rounded once. (The values' piece there was moved back to end with the row.)
template <int DT, int CW, int CE = CW>
__device__ __forceinline__ void store_dims(char* row, int d0, int dim, bool tiny, const float* x, int e0 = 0) {
  if constexpr (CE == CW) {
    if (d0 + CW <= dim) {
      if constexpr (DT == TS_DTYPE_F32) {
        tsl::store16(row + d0 * 4, u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])});
      } else {
        uint32_t w[CW / 2];
#pragma unroll
        for (int n = 0; n < CW / 2; ++n) w[n] = round16<DT>(x[2 * n]) | round16<DT>(x[2 * n + 1]) << 16;
        if constexpr (CW == 8) tsl::store16(row + d0 * 2, u32x4{w[0], w[1], w[2], w[3]});
        else *reinterpret_cast<u32x2_any*>(row + d0 * 2) = u32x2{w[0], w[1]};
      }
      return;
    }
  }
  const int at = (tiny ? d0 : min(d0, dim - CW)) + e0;
#pragma unroll
  for (int n = 0; n < CE; ++n) {
    if (at + n < d0 || at + n >= dim) continue;
    if constexpr (DT == TS_DTYPE_F32) reinterpret_cast<float*>(row)[at + n] = x[n];
    else reinterpret_cast<uint16_t*>(row)[at + n] = (uint16_t)round16<DT>(x[n]);
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
  if (P.norm) P.norm[at] = status != TS_ROW_OK ? float2{NAN, NAN} : float2{m, sum == 0.0f ? 0.0f : 1.0f / sum};
}

// ------------------------------------------------------------------ the pass over the cache
// The list of all rows' tiles has one more place after each row's: what it costs to finish a row (a wave of 16 rows of one
// tile would else be the last to end).
template <int TOK>
__device__ __forceinline__ int64_t places_of(const AParams& P, const Span& s) {
  const int32_t tiles = tiles_of<TOK>(s);
  return tiles ? (int64_t)(tiles + 1) * rows_of(P) : 0;
}
// A tile of a row, and how many places are left of a wave's stretch, this one included.
struct Cursor {
  int32_t b, r;                  // sequence and its row
  int32_t lo, n, tiles;          // of the sequence
  int32_t tile;                  // of the row
  int64_t left;
};
template <int TOK>
__device__ __forceinline__ void enter(const AParams& P, Cursor& c, int b, int32_t n) {
  const Span span = span_from(P, n);
  c.b = b;
  c.lo = span.lo;
  c.n = span.n;
  c.tiles = tiles_of<TOK>(span);
}
template <int TOK>
__device__ __forceinline__ bool advance(const AParams& P, Cursor& c) {
  if (--c.left <= 0) return false;
  if (++c.tile < c.tiles) return true;
  if (--c.left <= 0) return false;
  c.tile = 0;
  if (++c.r < rows_of(P)) return true;
  c.r = 0;
  do {                           // there are tiles left, so a sequence with some follows
    if (c.b + 1 >= P.batch) return false;
    enter<TOK>(P, c, c.b + 1, P.lengths[c.b + 1]);
  } while (c.tiles == 0);
  return true;
}
// The wave's stretch of the list. Every wave adds up the places of all sequences by itself (lane x takes some
// sequences in a row), so that no barrier stands before the first loads.
template <int TOK>
__device__ __forceinline__ bool begin(const AParams& P, int wv, Cursor& c) {
  const int own = (P.batch + 63) / 64, first = min(P.batch, lane() * own), last = min(P.batch, first + own);
  uint64_t sum = 0;
  int32_t n = 0;                 // of the lane's last sequence
  for (int x = first; x < last; ++x) {
    n = P.lengths[x];
    sum += (uint64_t)places_of<TOK>(P, span_from(P, n));
  }
  const uint64_t incl = wave_incl_scan64(sum), total = readlane64(incl, 63);
  // Workgroup w of G has places w total / G .. (w + 1) total / G (rounded down), and its waves likewise: within one of each other.
  // Every wave has one, unless there are fewer than a workgroup's waves.
  const int64_t groups = max(min((int64_t)gridDim.x, (int64_t)total / kAW), (int64_t)1);
  if (blockIdx.x == 0 && wv == 0) {
    int64_t at = (int64_t)(incl - sum);
    for (int x = first; x < last; ++x) {
      P.start[x] = at;
      at += places_of<TOK>(P, span_of(P, x));
    }
    if (lane() == 0) {
      P.start[P.batch] = (int64_t)total;
      P.start[P.batch + 1] = groups;
    }
  }
  if (blockIdx.x >= groups) return false;
  const int64_t v = blockIdx.x * (int64_t)kAW + wv, pos = quotient(v * (int64_t)total, groups * kAW);
  c.left = quotient((v + 1) * (int64_t)total, groups * kAW) - pos;
  if (c.left == 0) return false;
  const uint64_t past = __builtin_amdgcn_ballot_w64((int64_t)incl > pos);   // not 0: the last lane's is the total
  const int l = __builtin_ctzll(past);
  int64_t in = pos - (int64_t)readlane64(incl - sum, l);
  int b = l * own;
  n = __builtin_amdgcn_readlane(n, l);
  if (own > 1) {
    for (; b + 1 < P.batch; ++b) {
      const int64_t places = places_of<TOK>(P, span_of(P, b));
      if (in < places) break;
      in -= places;
    }
    n = P.lengths[b];
  }
  enter<TOK>(P, c, b, n);
  c.r = (int)quotient(in, c.tiles + 1);
  c.tile = (int32_t)(in - (int64_t)c.r * (c.tiles + 1));
  if (c.tile < c.tiles) return true;
  --c.tile;                      // past a row's end: to the next row
  ++c.left;
  return advance<TOK>(P, c);
}

// What a wave leaves for its workgroup of a row that began before it.
struct Part {
  int32_t b, r;                  // b = -1: none, -2: it has no tiles
  int32_t ends, bad;
};

template <int DT, int DP, int MODE, bool UNI, bool ONCE>
__global__ __launch_bounds__(kAT, DP > 128 ? 1 : 2) void ts_attend_kernel(const AParams P) {
  using S = Shape<DT, DP>;
  constexpr int TOK = S::kTok;
  __shared__ float sm_o[kAW][S::kAcc * 4][64];
  __shared__ float sm_m[kAW][kCols], sm_l[kAW][kCols];
  __shared__ Part sm_part[kAW];
  const int wv = __builtin_amdgcn_readfirstlane(wave()), g = lane() >> 4, i = lane() & 15;
  Cursor c;
  bool have;
  if (P.whole) {
    const int rows = rows_of(P), b = blockIdx.x / (unsigned)rows;
    enter<TOK>(P, c, b, P.lengths[b]);
    c.r = blockIdx.x - b * rows;
    const int own = (c.tiles + kAW - 1) / kAW;
    c.tile = wv * own;
    c.left = min(own, c.tiles - c.tile);   // one row: its end's place is not reached
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
  if (lane() == 0) sm_part[wv].b = have ? -1 : -2;
  Wave<DT, DP, MODE, UNI, ONCE> W;
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
  // The row's results, as far as they are in W: finished, or left to the join.
  auto finish = [&](int b, int r, bool begins, bool complete, float l, bool spoilt) {
    const RowOut R = row_out(P, b, r);
    const int status = spoilt ? TS_ROW_BAD_PAGE : TS_ROW_OK;
    if (complete) {
      const float inv = spoilt ? NAN : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int x = 0; x < S::kNP * 4; ++x) {
        float y[S::kCW];
#pragma unroll
        for (int e = 0; e < S::kCW; ++e) y[e] = !spoilt && l == 0.0f ? 0.0f : W.o[(x >> 2) * S::kCW + e][x & 3] * inv;
        if (i < R.heads)
          store_dims<DT, S::kCW>(P.out + b * P.out_b + (int64_t)(R.head0 + i) * P.out_h,
                                 (x >> 2) * 16 * S::kCW + (g * 4 + (x & 3)) * S::kCW, P.dim, P.tiny, y);
      }
      store_norm(P, R, W.m, l, S::kBias, status);
      if (P.status && lane() == 0) P.status[b] = status;   // every row of a sequence finds the same
    } else {
      float* part = P.part + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * kPartFloats<DT, DP>;
#pragma unroll
      for (int x = 0; x < S::kNP * 4; ++x)
#pragma unroll
        for (int e = 0; e < S::kCW; ++e) part[(x * S::kCW + e) * 64 + lane()] = W.o[(x >> 2) * S::kCW + e][x & 3];
      float* tail = part + S::kAcc * 4 * 64;
      if (lane() < kCols) {
        tail[i] = W.m;
        tail[kCols + i] = l;
      }
      if (lane() == 0) tail[2 * kCols] = spoilt ? 1.0f : 0.0f;
    }
  };
  bool bad = false;              // a page of the row so far was outside the cache
  bool begins = true;            // the row's first tile was this wave's
  bool open = false;             // W holds a part of a row that goes on in the next wave
  float l = 0.0f;
  bool spoilt = false;
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
    const bool ends = c.tile + 1 == c.tiles;
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
    if (ends || !have) {
      l = column_sum(W.l);
      spoilt = __builtin_amdgcn_ballot_w64(bad) != 0;
      if (begins && ends) {
        finish(c.b, c.r, true, true, l, spoilt);
      } else if (begins) {
        open = true;
        break;                   // the stretch ends here
      } else {
        if (lane() < kCols) {
          sm_m[wv][i] = W.m;
          sm_l[wv][i] = l;
        }
        if (lane() == 0) sm_part[wv] = Part{c.b, c.r, ends, spoilt};
#pragma unroll
        for (int x = 0; x < S::kNP * 4; ++x)
#pragma unroll
          for (int e = 0; e < S::kCW; ++e) sm_o[wv][x * S::kCW + e][lane()] = W.o[(x >> 2) * S::kCW + e][x & 3];
      }
      W.clear_state();
      begins = true;
      bad = false;
    }
    bad = bad || next_bad;
    c = next;
  }
  bar();
  // A row's parts follow each other, wave after wave. The wave that it begins in joins them; what began before the workgroup
  // is joined by the first.
  auto add_following = [&](int b, int r, int w, bool& ended) {
    for (; w < kAW; ++w) {
      const Part p = sm_part[w];
      if (p.b == -2) continue;
      if (p.b != b || p.r != r) break;
      const float mw = sm_m[w][i], m = fmaxf(W.m, mw);
      const float f = W.m == m ? 1.0f : exp2_fast((W.m - m) * P.c), fw = mw == m ? 1.0f : exp2_fast((mw - m) * P.c);
      W.m = m;
      l = l * f + sm_l[w][i] * fw;
#pragma unroll
      for (int x = 0; x < S::kNP * 4; ++x)
#pragma unroll
        for (int e = 0; e < S::kCW; ++e) {
          float& o = reinterpret_cast<float*>(&W.o[(x >> 2) * S::kCW + e])[x & 3];
          o = o * f + sm_o[w][x * S::kCW + e][lane()] * fw;
        }
      spoilt = spoilt || p.bad;
      ended = p.ends;
    }
  };
  if (open) {
    bool ended = false;
    add_following(c.b, c.r, wv + 1, ended);
    finish(c.b, c.r, true, ended, l, spoilt);
  }
  if (wv == 0) {
    int w = 0;
    while (w < kAW - 1 && sm_part[w].b == -2) ++w;
    const Part p = sm_part[w];
    if (p.b >= 0) {
      bool ended = false;
      W.clear_state();
      l = 0.0f;
      spoilt = false;
      add_following(p.b, p.r, w, ended);
      finish(p.b, p.r, false, false, l, spoilt);
    }
  }
}

// ------------------------------------------------------------------ rows that several workgroups share
// The parts of a row: workgroup w0's second one (the row starts inside its share or with it), then the next workgroups' first.
template <int DT, int DP>
struct Parts {
  const float* first;
  int32_t count;                 // 0: no tiles; 1: finished by its workgroup
  static constexpr int64_t kSize = kPartFloats<DT, DP>;
  static constexpr int kTail = Shape<DT, DP>::kAcc * 4 * 64;
  __device__ __forceinline__ Parts(const AParams& P, int b, int r, int32_t tiles) {
    const int64_t total = P.start[P.batch], shares = P.start[P.batch + 1];
    const int64_t from = P.start[b] + (int64_t)r * (tiles + 1);
    // place x is workgroup w's if w total / shares < x + 1
    const int64_t w0 = tiles ? quotient((from + 1) * shares - 1, total) : 0;
    count = tiles ? (int)(quotient((from + tiles) * shares - 1, total) - w0 + 1) : 0;
    first = P.part + (w0 * 2 + 1) * kSize;
  }
  __device__ __forceinline__ const float* at(int p) const { return first + max(2 * p - 1, 0) * kSize; }
};

// exp(scale (s - m)) / sum of positions j0 .. + 4 of a query head, 0 outside [lo, n), from the stored scores; all NaN in a refused
// row. An m of NaN is what tells that: a running maximum passes over NaN scores, while the sum of a sound row may well be NaN.
__device__ __forceinline__ void store_weights(const AParams& P, int b, int head, const Span& span, float m, float inv, float bias, int j0) {
  if (j0 >= P.w_slots) return;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (j0 < span.n && j0 + 4 > span.lo) x = *reinterpret_cast<const f32x4*>(P.score + ((int64_t)b * P.q_heads + head) * P.score_stride + j0);
  const float base = m == -INFINITY ? 0.0f : m;
  char* to = P.weights + (int64_t)b * P.w_b + (int64_t)head * P.w_h;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = j0 + e;
    float w = m != m ? NAN : 0.0f;
    if (j >= span.lo && j < span.n) w = exp2_fast((x[e] - base) * P.c + bias) * inv;
    x[e] = w;
  }
  if (P.w_dtype == TS_DTYPE_F32) {
    float* row = reinterpret_cast<float*>(to);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j0 + e < P.w_slots) row[j0 + e] = x[e];
  } else {
    uint16_t* row = reinterpret_cast<uint16_t*>(to);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j0 + e < P.w_slots) row[j0 + e] = (uint16_t)(P.w_dtype == TS_DTYPE_BF16 ? round16<TS_DTYPE_BF16>(x[e]) : round16<TS_DTYPE_F16>(x[e]));
  }
}

// A workgroup a row and CE of every lane's results; its waves take the parts in turn, each with a running maximum. The
// workgroups from P.join_blocks on: the weights of 4 positions a thread of one query head.
template <int DT, int DP, int NW, int CE>
__global__ __launch_bounds__(NW * 64) void ts_attend_join_kernel(const AParams P) {
  using S = Shape<DT, DP>;
  __shared__ float sm_o[NW][CE][64];
  __shared__ float sm_m[NW][64], sm_l[NW][64];
  __shared__ int any_bad;
  const int wv = __builtin_amdgcn_readfirstlane(wave()), g = lane() >> 4, i = lane() & 15;
  const int rows = rows_of(P), groups = S::kAcc * 4 / CE;
  if ((int)blockIdx.x >= P.join_blocks) {
    const int of_head = (P.w_slots + NW * 256 - 1) / (NW * 256), x = (int)blockIdx.x - P.join_blocks, row = x / of_head;
    const int b = row / P.q_heads, head = row - b * P.q_heads, hk = head / P.group, in = head - hk * P.group;
    const int j0 = ((x - row * of_head) * NW * 64 + (int)threadIdx.x) * 4;
    const Span span = span_of(P, b);
    const int32_t tiles = tiles_of<S::kTok>(span);
    float2 norm;
    if (P.whole) {
      norm = P.norm[row];
    } else if (tiles == 0) {
      norm = float2{span.status != TS_ROW_OK ? NAN : -INFINITY, 0.0f};
    } else if (const Parts<DT, DP> parts(P, b, hk * P.head_tiles + in / kCols, tiles); parts.count == 1) {
      norm = P.norm[row];
    } else {
      const int col = in % kCols;
      float m = -INFINITY, l = 0.0f;
      bool bad = false;
      for (int p = lane(); p < parts.count; p += 64) {
        const float* tail = parts.at(p) + parts.kTail;
        const float mp = tail[col], grown = fmaxf(m, mp);
        l = l * (m == grown ? 1.0f : exp2_fast((m - grown) * P.c)) + tail[kCols + col] * (mp == grown ? 1.0f : exp2_fast((mp - grown) * P.c));
        m = grown;
        bad = bad || tail[2 * kCols] != 0.0f;
      }
#pragma unroll
      for (int step = 1; step < 64; step *= 2) {
        const float mo = __shfl_xor(m, step), lo = __shfl_xor(l, step), grown = fmaxf(m, mo);
        l = l * (m == grown ? 1.0f : exp2_fast((m - grown) * P.c)) + lo * (mo == grown ? 1.0f : exp2_fast((mo - grown) * P.c));
        m = grown;
      }
      norm = __builtin_amdgcn_ballot_w64(bad) ? float2{NAN, NAN} : float2{m, l == 0.0f ? 0.0f : 1.0f / l};
    }
    store_weights(P, b, head, span, norm.x, norm.y, S::kBias, j0);
    return;
  }
  const int y = blockIdx.x % groups, row = blockIdx.x / groups, b = row / rows, r = row - b * rows;
  const Span span = span_of(P, b);
  const int32_t tiles = tiles_of<S::kTok>(span);
  const RowOut R = row_out(P, b, r);
  const Parts<DT, DP> parts(P, b, r, tiles);
  const int count = parts.count;
  if (count == 1) return;
  if (threadIdx.x == 0) any_bad = 0;
  bool bad = false;
  float m = -INFINITY, l = 0.0f, sum[CE];
#pragma unroll
  for (int c = 0; c < CE; ++c) sum[c] = 0.0f;
  constexpr int kBatch = CE == 1 ? 8 : 4;   // parts whose loads are in flight together
  for (int p0 = wv; p0 < count; p0 += NW * kBatch) {
    float mp[kBatch], lp[kBatch], x[kBatch][CE], wrong[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int p = min(p0 + u * NW, count - 1);
      const float* part = parts.at(p);
      mp[u] = part[parts.kTail + i];
      lp[u] = part[parts.kTail + kCols + i];
      wrong[u] = part[parts.kTail + 2 * kCols];
#pragma unroll
      for (int c = 0; c < CE; ++c) x[u][c] = part[(y * CE + c) * 64 + lane()];
    }
    float grown = m;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (p0 + u * NW >= count) mp[u] = -INFINITY;
      grown = fmaxf(grown, mp[u]);
    }
    const float f = m == grown ? 1.0f : exp2_fast((m - grown) * P.c);
    m = grown;
    l *= f;
#pragma unroll
    for (int c = 0; c < CE; ++c) sum[c] *= f;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (p0 + u * NW >= count) break;
      const float fp = mp[u] == grown ? 1.0f : exp2_fast((mp[u] - grown) * P.c);
      bad = bad || wrong[u] != 0.0f;
      l += lp[u] * fp;
#pragma unroll
      for (int c = 0; c < CE; ++c) sum[c] += x[u][c] * fp;
    }
  }
  bar();
  if (__builtin_amdgcn_ballot_w64(bad)) any_bad = 1;
  sm_m[wv][lane()] = m;
  sm_l[wv][lane()] = l;
#pragma unroll
  for (int c = 0; c < CE; ++c) sm_o[wv][c][lane()] = sum[c];
  bar();
  if (wv != 0) return;
#pragma unroll 4
  for (int w = 1; w < NW; ++w) m = fmaxf(m, sm_m[w][lane()]);
  l = 0.0f;
#pragma unroll
  for (int c = 0; c < CE; ++c) sum[c] = 0.0f;
#pragma unroll 4
  for (int w = 0; w < NW; ++w) {
    const float mw = sm_m[w][lane()], f = mw == m ? 1.0f : exp2_fast((mw - m) * P.c);
    l += f * sm_l[w][lane()];
#pragma unroll
    for (int c = 0; c < CE; ++c) sum[c] += f * sm_o[w][c][lane()];
  }
  const int status = span.status != TS_ROW_OK ? span.status : any_bad ? TS_ROW_BAD_PAGE : TS_ROW_OK;
#pragma unroll
  for (int c = 0; c < CE; ++c) sum[c] = status != TS_ROW_OK ? NAN : l == 0.0f ? 0.0f : sum[c] * (1.0f / l);
  const int x = y * CE / S::kCW, e0 = y * CE % S::kCW;   // results e0 .. + CE of row x % 4 of pass x / 4
  if (i < R.heads)
    store_dims<DT, S::kCW, CE>(P.out + b * P.out_b + (int64_t)(R.head0 + i) * P.out_h,
                               (x >> 2) * 16 * S::kCW + (g * 4 + (x & 3)) * S::kCW, P.dim, P.tiny, sum, e0);
  if (y == 0) {
    store_norm(P, R, m, l, S::kBias, status);
    if (P.status && lane() == 0) P.status[b] = status;
  }
}

// ------------------------------------------------------------------ host side
// How the join's work is cut: by rows' results of 8 a lane, unless rows are so few that single ones fill the chip better (at most
// kFineJoin workgroups); rows of very many parts each have 16 waves. (us a call: 64 rows of 33 tiles 20.7, by single results 23.9;
// 16 rows of 4096 tiles 174.7 with 4 waves, 177.6 with 16; 8 rows of 63 tiles 14.0 and 15.1; one row of 4096 tiles 34.7 with 16.)
constexpr int64_t kFineJoin = 512, kWideJoin = 2;
constexpr double kCacheBytes = 256e6;   // the last-level cache
// Workgroups of the pass: as many as the chip holds at once, by their registers and LDS.
constexpr int groups_of(int dp) { return dp <= 128 ? 512 : 256; }

int dtype_size(int dtype) {
  return dtype == TS_DTYPE_F32 ? 4 : (dtype == TS_DTYPE_BF16 || dtype == TS_DTYPE_F16) ? 2 : 0;
}
int tile_of(int dtype) { return dtype == TS_DTYPE_F32 ? Shape<TS_DTYPE_F32, 64>::kTok : Shape<TS_DTYPE_BF16, 64>::kTok; }
int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

struct APlan {
  int64_t rows = 0, score_stride = 0;
  size_t off_norm = 0, off_start = 0, off_part = 0, total = 0;
  bool whole = false;
};
// Rows of few tiles are left to one workgroup each, which saves the join's launch; of more where there are rows enough to fill
// the chip that way, but not so many that equal shares do, whatever their lengths. (us a call, a workgroup a row against
// shares, tiles of 32; sequences of 8 rows: 64 x 250 positions 14.4 against 20.6, 8 x 500 14.4 against 18, 256 x 500 93 against 96,
// 8 x 1000 22 against 18, 64 x 1000 46 against 51, 64 of up to 1000 36 against 38, 256 of up to 1000 108 against 105.)
constexpr int64_t kWholeTiles = 16, kWholeMore = 32, kWholeRows = 256, kWholeMost = 1024;

// Weights of a head: a workgroup's positions (16 waves' 4096 at most) past the last one stay in 31 bits.
constexpr int64_t kMaxWeights = 0x7FFFF000;

bool attend_plan(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim, int64_t max_len, int64_t w_slots, int tile, APlan& pl) {
  if (batch < 0 || batch > (1 << 24) || kv_heads < 1 || q_heads < kv_heads || q_heads > (1 << 16) || q_heads % kv_heads || dim < 1 ||
      dim > kMaxDim || max_len < 0 || max_len > tsp::kMaxLen || w_slots < 0 || w_slots > kMaxWeights)
    return false;
  const int64_t tiles = (q_heads / kv_heads + kCols - 1) / kCols;
  pl.rows = batch * kv_heads * tiles;
  if (pl.rows * 16 > (int64_t)0xFFFFFFFF / 512) return false;   // a launch has fewer than 2^32 threads, a join's 16 x 256 a row at most
  pl.whole = max_len <= kWholeTiles * tile || (max_len <= kWholeMore * tile && pl.rows >= kWholeRows && pl.rows <= kWholeMost);
  pl.score_stride = w_slots ? (w_slots + 31) / 32 * 32 : 0;
  if (w_slots && batch * q_heads * ((w_slots + 1023) / 1024) > (int64_t)0xFFFFFFFF / 512) return false;
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
  const dim3 grid(P.whole ? (unsigned)rows : (unsigned)groups_of(DP));
  if (P.once && MODE != kTiny) hipLaunchKernelGGL((ts_attend_kernel<DT, DP, MODE, UNI, MODE != kTiny>), grid, dim3(kAT), 0, s, P);
  else hipLaunchKernelGGL((ts_attend_kernel<DT, DP, MODE, UNI, false>), grid, dim3(kAT), 0, s, P);
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
  if (e != hipSuccess || (P.whole && !P.weights)) return e;
  using S = Shape<DT, DP>;
  const int64_t coarse = P.whole ? 0 : rows * S::kNP * 4;
  auto join = [&](auto kernel, int64_t blocks, int threads) {
    P.join_blocks = (int32_t)blocks;
    if (P.weights) blocks += (int64_t)P.batch * P.q_heads * ((P.w_slots + threads * 4 - 1) / (threads * 4));
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), 0, s, P);
  };
  if (P.whole || coarse * S::kCW > kFineJoin) join(ts_attend_join_kernel<DT, DP, 4, S::kCW>, coarse, 256);
  else if (rows > kWideJoin) join(ts_attend_join_kernel<DT, DP, 4, 1>, coarse * S::kCW, 256);
  else join(ts_attend_join_kernel<DT, DP, 16, 1>, coarse * S::kCW, 1024);
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

extern "C" size_t ts_cache_attend_workspace(int dtype, int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len,
                                            int64_t weights_slots) {
  APlan pl;
  if (!dtype_size(dtype)) return 0;
  if (weights_slots > 0) max_len = std::min(max_len, weights_slots);
  return attend_plan(batch, q_heads, kv_heads, dim, std::min(max_len, tsp::kMaxLen), weights_slots, tile_of(dtype), pl) ? pl.total : 0;
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
  if (out == q) return fail(TS_ERR_INVALID_ARG, "out may not be q: other waves still read it");
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
  if (!attend_plan(batch, q_heads, kv_heads, dim, window > 0 ? std::min<int64_t>(max_len, window) : max_len, weights_slots,
                   tile_of(dtype), pl))
    return fail(TS_ERR_INVALID_ARG, "batch x heads x slots too large");
  if (tsp::meet({(uintptr_t)q, (int64_t)dim * size, {q_batch_stride * size, q_head_stride * size}, {batch, q_heads}},
                {(uintptr_t)out, (int64_t)dim * size, {out_batch_stride * size, out_head_stride * size}, {batch, q_heads}}))
    return fail(TS_ERR_INVALID_ARG, "out overlaps q, which other waves still read");
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
    P.w_dtype = weights_dtype;
    P.score = reinterpret_cast<float*>(ws);
    P.score_stride = pl.score_stride;
    P.norm = reinterpret_cast<float2*>(ws + pl.off_norm);
  }
  P.start = reinterpret_cast<int64_t*>(ws + pl.off_start);
  P.part = reinterpret_cast<float*>(ws + pl.off_part);
  P.whole = pl.whole ? 1 : 0;
  // Past the caches, where the sequences hold more than the last-level cache does (64 of up to 4096 positions, 0.5 GB: 106 us
  // against 117; 67 MB: 45 against 43) and nothing is read twice.
  const int64_t most = std::min<int64_t>(pages, batch * ((max_len + page_slots - 1) / page_slots));
  P.once = P.head_tiles == 1 && (double)most * page_slots * kv_heads * dim * size * 2 > kCacheBytes;
  P.tiny = dim * size < 16;
  P.end_block = dim * size % 16 ? dim * size / 64 : -1;
  const hipStream_t s = (hipStream_t)stream;
  hipError_t e = dtype == TS_DTYPE_F32    ? launch_dim<TS_DTYPE_F32>(P, pl.rows, s)
                 : dtype == TS_DTYPE_BF16 ? launch_dim<TS_DTYPE_BF16>(P, pl.rows, s)
                                          : launch_dim<TS_DTYPE_F16>(P, pl.rows, s);
  if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "attention launch failed: %s", hipGetErrorString(e));
  return TS_OK;
}
