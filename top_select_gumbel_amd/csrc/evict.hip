// evict.hip -- eviction from key / value caches by accumulated attention weight.
//
// A cache row (one head of one sequence) holds n positions in slots 0 .. n-1. With s_j = score_j + sum_w weight[w, j]
// (binary64, rounded once to the fp32 that is kept), the row keeps its first k = min(keep, n) slots in the order
// (protected first, s descending, slot ascending); protected are the positions below `sinks` and the newest
// `recent` ones. The i-th slot below k that is not kept takes over the i-th kept slot at or past k, so
// that a row of which few positions go moves few, and nothing that is read is written.
//
// Short rows (ts_evict_row_kernel, one workgroup a row, its sums in registers) are summed, cut and listed, and their few
// moves made, in one launch where one compute unit alone reads and copies that fast enough (64 rows of 1025 slots, 4
// weights each: 8.8 us, all of it the latency of a dozen dependent steps); else the sums come from ts_evict_sum_kernel
// and the moves go to ts_evict_move_kernel, both spread over the chip.
//
// Long rows are spread in every step but the cut (a tile of 1024 slots a workgroup), a launch each (in brackets: us for 8 rows
// of 131072 slots, 4 fp32 weights each, cut to 8192 positions of 2 x 256 bytes):
//   sum    s, and each tile's largest position and extreme keys [9.0, 25 MB]
//   bin    both classes (protected, others) counted by the first 11 bits of u = key - smallest key of the row [7.0]
//   list   the bin that holds the cut, its slots listed [5.5]
//   cut    one workgroup a row: the cut's (u, slot) [6.3]
//   emit   what stays in place; each tile's freed slots and fillers [5.8]
//   move   the i-th freed slot of a row receives the i-th filler (found by the tiles' counts), caches and small outputs
//          [17, 63 MB]
// The four in the middle read 4 MB from the caches each and are bound by the latency of their few dependent loads.
//
// The cut is found by radix select on u = key - smallest key of the row (ordered keys, so that the first 2048 bins
// span the row's own range and not the whole of fp32), then, once few slots share its bin, by ranking those.
//
// The limit of this: a long row's cut whose first bin holds more than 4096 slots. They are not listed then, and the row's one
// workgroup goes through all of the row in memory, two to five times; the time is that of its dependent loads, 1.3 us for 1000
// slots of the row. Such are rows that keep some of thousands of equal weights, and long ones: evenly spread weights from 524288
// slots on, heavy-tailed ones from 2^20 on, both sooner where one sum is 0 and stretches the range. (One row, us a call, listed
// against not: 131072 slots, 8 rows, 46 against 110-166; 524288 slots 42 against 490-530; 2^20 slots 52 against 1200-1360; 2^22
// slots 5200-5400. A sort of the row in elementary operations takes 470-760, 600-1200 and 1300-2900 for the last three.)
#include <algorithm>
#include <type_traits>

#include "topselect.h"
#include "ts_device.hpp"
#include "ts_host.hpp"
#include "ts_logits.hpp"

using namespace tsd;
using tsh::check_device;
using tsh::fail;

namespace {

constexpr int kST = 256;                 // threads of the sum kernel
constexpr int kSumSlots = 4;             // slots a thread
template <int DT>
constexpr int kSumBatch = DT == TS_DTYPE_F32 ? 8 : 16;   // weight rows a thread has in flight: 128 bytes
constexpr int kRowBatch = 4;             // the same where a row kernel sums: few weight rows
constexpr int kSumTile = kST * kSumSlots;
constexpr int kET = 1024;                // threads of the row kernels, of rows of up to kSmallSlots slots 256
constexpr int kEW = kET / 64;
constexpr int kSmallT = 256;
constexpr int kSmallSlots = 2 * 4 * kSmallT;
constexpr int kEBits = 11;
constexpr int kEBins = 1 << kEBits;
constexpr int kMaxTiles = TS_EVICT_MAX_SLOTS / kSumTile;
// Rows held in registers by one workgroup: two 16-byte vectors a thread, or four where there are rows enough to fill the
// chip that way. Longer ones are spread. (Rows x slots, one position dropped, one workgroup a row against spread: 8 x 8192
// 19 us against 25, 512 x 8192 50 against 94; 8 x 16384 31 against 26, 64 x 16384 38 against 42, 512 x 16384 106
// against 151.)
constexpr int kRowSlots = 2 * 4 * kET;
constexpr int kWideSlots = 4 * 4 * kET, kWideRows = 64;
constexpr int kListRow = 256;            // slots of the cut's bin that are ranked rather than binned again, ...
constexpr int kListLong = 4096;          // ... and that are listed for a long row's cut
constexpr int kMT = 256;                 // threads of the move kernel

// What a tile of the sum kernel leaves for long rows: largest position, smallest and largest key.
struct TileInfo {
  int32_t newest;
  uint32_t kmin, kmax, pad;
};

// What the steps of a long row leave for the next ones.
struct RowInfo {
  uint32_t protected_;         // bin: protected slots
  uint32_t among_first;        // list: whether the cut falls among the protected slots
  uint32_t prefix, lo;         // the cut's bin: u >> lo == prefix
  uint32_t need, in_bin;       // the cut is the need-th of the in_bin slots in it
  uint32_t whole;              // 0: a cut is to be found; 1: the class stays as a whole
  uint32_t cut_u, cut_slot;    // cut
  int32_t st, k, tiles;        // cut: the row's status, new length, tiles in use
};
// What a tile of a long row leaves: slots of the cut's bin and their extreme u; freed slots and fillers.
struct TileBin {
  uint32_t count, umin, umax, holes, fills, pad[3];
};

struct Cache {
  char* p;
  int64_t batch, head, slot;   // bytes
  int32_t units, last;         // units of the copy a slot (0: no cache) and where its last one starts
};

struct EParams {
  const float* score;
  int64_t score_stride;
  const char* weights;
  int64_t w_row, w_stride;               // bytes
  int32_t n_w;
  const int32_t* position;
  int64_t position_stride;
  const int32_t* lengths;
  const int32_t* keep;
  int32_t rows, slots, keep_max, sinks, recent;
  float* out_score;
  int64_t out_score_stride;
  int32_t* out_position;
  int64_t out_position_stride;
  int32_t* out_lengths;
  int32_t* out_source;
  int32_t* status;
  float* sum;                            // [rows, sum_stride]
  int64_t sum_stride;                    // slots, rounded up to whole vectors
  TileInfo* info;                        // [rows, tiles]
  RowInfo* row;                          // [rows] long rows, like the next ones
  TileBin* bin;                          // [rows, tiles]
  uint32_t* hist;                        // [rows, 2, kEBins]
  int32_t* fill_position;                // [rows, sum_stride]; hole and fill are [rows, sum_stride] there, by tiles
  int32_t tiles;
  int32_t spread;                        // long rows
  int32_t* moves;                        // [rows]
  int32_t* hole;                         // [rows, cap]: the freed slots, ascending
  int32_t* fill;                         // [rows, cap]: what each takes over, ascending
  int32_t cap;
  Cache k, v;
  int32_t heads;
  int32_t lane_bits;                     // of the threads that copy one move
};

__device__ __forceinline__ int row_length(const EParams& P, int r) { return max(0, min(P.lengths[r], P.slots)); }

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef i32x4 i32x4_any __attribute__((aligned(4)));

// Slots j .. j + 3 of an array of n; what lies past the end is `rest`.
template <class V, class VA, class T>
__device__ __forceinline__ V load4(const T* p, int j, int n, T rest) {
  if (j + 4 <= n) return *reinterpret_cast<const VA*>(p + j);
  V v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = j + i < n ? p[j + i] : rest;
  return v;
}

// Four weights at w: 16 bytes, or 8 in the first half of the vector.
template <int DT>
__device__ __forceinline__ tsl::u32x4 load_weights(const char* w) {
  if constexpr (DT == TS_DTYPE_F32) {
    return tsl::load16(w);
  } else {
    typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    const u32x2 h = *reinterpret_cast<const u32x2_any*>(w);
    return tsl::u32x4{h[0], h[1], 0u, 0u};
  }
}

// The sums of slots j .. j + 3 in binary64, in the order of the weight rows. All loads of a batch of weight rows are
// in flight before the first is added.
template <int DT, int BATCH>
__device__ __forceinline__ void sum_slots(const EParams& P, int r, int j, int n, double* s) {
  const char* w = P.weights + (int64_t)r * P.w_row + (int64_t)j * tsl::Logits<DT>::kSize;
  const float* score = P.score + (int64_t)r * P.score_stride;
  if (j + 4 <= n) {
    const f32x4 v = *reinterpret_cast<const f32x4_any*>(score + j);
    // Weight rows q .. q + BATCH - 1; past the last one it is loaded again and -0, which changes no sum, added.
    auto batch = [&](int q, bool start) {
      tsl::u32x4 x[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) x[b] = load_weights<DT>(w + (int64_t)min(q + b, P.n_w - 1) * P.w_stride);
      if (start) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = (double)v[i];
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += (double)(q + b < P.n_w ? tsl::unpack<DT>(x[b], i) : -0.0f);
    };
    if (P.n_w > 0) {
      batch(0, true);
      for (int q = BATCH; q < P.n_w; q += BATCH) batch(q, false);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = (double)v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = j + i < n ? (double)score[j + i] : 0.0;
    for (int q = 0; q < P.n_w; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + i < n) s[i] += (double)tsl::load_logit<DT>(w + (int64_t)q * P.w_stride, i);
  }
}

template <int DT>
__global__ __launch_bounds__(kST) void ts_evict_sum_kernel(EParams P) {
  __shared__ uint32_t red[3 * kST / 64];
  int r, tile;
  tsl::place_block(P.tiles, r, tile);
  const int n = row_length(P, r);
  const int j = tile * kSumTile + (int)threadIdx.x * kSumSlots;
  uint32_t newest = 0, kmin = 0xFFFFFFFFu, kmax = 0;
  if (j < n) {
    double s[kSumSlots];
    sum_slots<DT, kSumBatch<DT>>(P, r, j, n, s);
    f32x4* out = reinterpret_cast<f32x4*>(P.sum + (int64_t)r * P.sum_stride + j);
    *out = f32x4{(float)s[0], (float)s[1], (float)s[2], (float)s[3]};
    if (P.spread) {
      const int32_t* pos = P.position + (int64_t)r * P.position_stride;
#pragma unroll
      for (int i = 0; i < kSumSlots; ++i) {
        if (j + i >= n) continue;
        newest = max(newest, (uint32_t)pos[j + i] ^ 0x80000000u);
        const uint32_t k = f2key((float)s[i]);
        kmin = min(kmin, k);
        kmax = max(kmax, k);
      }
    }
  }
  if (!P.spread) return;
  if (tile == 0) {
    uint32_t* h = P.hist + (int64_t)r * 2 * kEBins;
    for (int i = threadIdx.x; i < 2 * kEBins; i += kST) h[i] = 0u;
    if (threadIdx.x == 0) P.row[r] = RowInfo{};
  }
  newest = wave_max(newest);
  kmin = wave_min(kmin);
  kmax = wave_max(kmax);
  if (lane() == 0) {
    red[3 * wave()] = newest;
    red[3 * wave() + 1] = kmin;
    red[3 * wave() + 2] = kmax;
  }
  bar();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kST / 64; ++w) {
      newest = max(newest, red[3 * w]);
      kmin = min(kmin, red[3 * w + 1]);
      kmax = max(kmax, red[3 * w + 2]);
    }
    P.info[(int64_t)r * P.tiles + tile] = TileInfo{(int32_t)(newest ^ 0x80000000u), kmin, kmax, 0u};
  }
}

// ------------------------------------------------------------------ selection within a row
struct ESmem {
  uint32_t hist[kEBins];
  uint2 list[kListRow];        // (u, slot) of the cut's bin
  uint32_t red[kEW], red2[kEW], red3[kEW];
  uint32_t res[3];
  uint32_t count;
  uint32_t cut_u, cut_slot;
};

// Exclusive prefix over the waves of two counts that every wave holds uniformly, and their totals.
template <int NW>
__device__ __forceinline__ void wave_offsets(ESmem& sm, uint32_t a, uint32_t b, uint32_t& ea, uint32_t& eb, uint32_t& ta,
                                             uint32_t& tb) {
  if (lane() == 0) {
    sm.red[wave()] = a;
    sm.red2[wave()] = b;
  }
  bar();
  ea = eb = ta = tb = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const uint32_t x = sm.red[w], y = sm.red2[w];
    ea += w < wave() ? x : 0u;
    eb += w < wave() ? y : 0u;
    ta += x;
    tb += y;
  }
  bar();
}
template <int NW>
__device__ __forceinline__ uint32_t block_total(ESmem& sm, uint32_t per_wave) {
  uint32_t a, b, t, u;
  wave_offsets<NW>(sm, per_wave, 0u, a, b, t, u);
  return t;
}

// A row's parameters and status.
struct Row {
  int n, k, st;
  int64_t from;       // positions above this are protected
  int32_t sinks;
  uint32_t kmin;
  __device__ __forceinline__ bool first(int32_t p) const { return p < sinks || (int64_t)p > from; }
  __device__ __forceinline__ uint32_t u(float s) const { return f2key(s) - kmin; }
};

// Kept of the cut's class: u above `u`, or equal to it and the slot not past `slot`.
struct Cut {
  uint32_t u, slot;
  __device__ __forceinline__ bool keeps(uint32_t x, int j) const { return x > u || (x == u && (uint32_t)j <= slot); }
};

// Finds the bin of the need-th largest of the binned values: sm.res = {bin, count above it, count in it}.
template <int NT>
__device__ __forceinline__ void find_bin(ESmem& sm, uint32_t need) {
  constexpr int kOwn = kEBins / NT;
  const int t = threadIdx.x;
  uint32_t c[kOwn], sum = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    c[i] = sm.hist[kOwn * t + i];
    sum += c[i];
  }
  const uint32_t incl = wave_incl_scan(sum);
  uint32_t before, eb, all, tb;
  wave_offsets<NT / 64>(sm, wave_total(incl), 0u, before, eb, all, tb);
  uint32_t above = all - (before + incl);
  if (above < need && above + sum >= need) {
    uint32_t bin = 0, in_bin = 0;
    bool found = false;
#pragma unroll
    for (int i = kOwn - 1; i >= 0; --i) {
      if (found) continue;
      bin = kOwn * t + i;
      in_bin = c[i];
      found = above + c[i] >= need;
      above += found ? 0u : c[i];
    }
    sm.res[0] = bin;
    sm.res[1] = above;
    sm.res[2] = in_bin;
  }
  bar();
}

// The cut among the `count` (u, slot) pairs of sm.list: its need-th in the order (u descending, slot ascending).
__device__ __forceinline__ Cut rank_list(ESmem& sm, uint32_t count, uint32_t need) {
  if (threadIdx.x < count) {
    const uint2 me = sm.list[threadIdx.x];
    uint32_t above = 0;
    for (uint32_t i = 0; i < count; ++i) {
      const uint2 o = sm.list[i];
      above += (o.x > me.x || (o.x == me.x && o.y < me.y)) ? 1u : 0u;
    }
    if (above + 1 == need) {
      sm.cut_u = me.x;
      sm.cut_slot = me.y;
    }
  }
  bar();
  return Cut{sm.cut_u, sm.cut_slot};
}

// The cut of a class: the need-th of its slots (1 <= need < their number). each(f) calls f(u, slot) for the calling
// thread's slots of the class; ordered(bin_lo, need) finds the need-th slot, in slot order, whose u is bin_lo.
// It lies among those with u >> lo == prefix.
template <int NT, class E, class O>
__device__ __forceinline__ Cut find_cut(ESmem& sm, int lo, uint32_t prefix, uint32_t need, E each, O ordered) {
  if (lo == 0) return Cut{prefix, ordered(prefix, need)};
  while (true) {
    const int d = min(kEBits, lo), sh = lo - d;
#pragma unroll
    for (int i = 0; i < kEBins; i += NT) sm.hist[i + threadIdx.x] = 0u;
    bar();
    const uint32_t mask = (1u << d) - 1u;
    each([&](uint32_t u, int) {
      if (shr(u, lo) == prefix) atomicAdd(&sm.hist[(u >> sh) & mask], 1u);
    });
    bar();
    find_bin<NT>(sm, need);
    prefix = shl(prefix, d) | sm.res[0];
    need -= sm.res[1];
    const uint32_t in_bin = sm.res[2];
    lo = sh;
    bar();
    if (in_bin == need) return Cut{shl(prefix, lo), 0xFFFFFFFFu};   // the whole bin stays
    if (in_bin <= (uint32_t)kListRow) {
      if (threadIdx.x == 0) sm.count = 0;
      bar();
      each([&](uint32_t u, int j) {
        if (shr(u, lo) == prefix) sm.list[atomicAdd(&sm.count, 1u)] = make_uint2(u, (uint32_t)j);
      });
      bar();
      return rank_list(sm, in_bin, need);
    }
    if (lo == 0) return Cut{prefix, ordered(prefix, need)};   // many equal: the lowest slots stay
  }
}

// Status, k and the class of the cut, once the row's extremes are known.
__device__ __forceinline__ Row row_of(const EParams& P, int r, uint32_t newest, uint32_t kmin, uint32_t kmax) {
  Row R;
  R.n = row_length(P, r);
  const int32_t keep = P.keep[r];
  R.k = min(keep, R.n);
  R.from = (int64_t)(int32_t)(newest ^ 0x80000000u) - P.recent;
  R.sinks = P.sinks;
  R.kmin = kmin;
  const bool bad = R.n > 0 && (kmax >= kKeyPosInf || kmin <= kKeyNegInf);
  R.st = bad ? TS_ROW_NONFINITE : (keep < 1 || R.k > P.keep_max) ? TS_ROW_BAD_K : TS_ROW_OK;
  return R;
}

// A rejected row: nothing of it changes, and outputs that are not its inputs are poisoned.
template <int NT>
__device__ __forceinline__ void reject_row(const EParams& P, int r, const Row& R) {
  int32_t* source = P.out_source + (int64_t)r * P.keep_max;
  float* score = P.out_score + (int64_t)r * P.out_score_stride;
  int32_t* place = P.out_position + (int64_t)r * P.out_position_stride;
  for (int j = threadIdx.x; j < P.keep_max; j += NT) {
    source[j] = -1;
    if (P.out_score != P.score) score[j] = __uint_as_float(0x7FC00000u);
    if (P.out_position != P.position) place[j] = -1;
  }
  if (threadIdx.x == 0) {
    P.out_lengths[r] = R.n;
    P.moves[r] = 0;
    if (P.status) P.status[r] = R.st;
  }
}

// Copies moves lo .. hi - 1 of a row by a workgroup of T threads: 2^lane_bits threads (about the units of U bytes that a slot
// has) take a move, kCopyBatch moves of a cache, or of both, in flight at a time. A share's last batch repeats its last
// move's loads and stores them once. (The last unit of a slot that is no whole number of them overlaps the one before; both
// write the same bytes there.)
constexpr int kCopyBatch = 4;
typedef unsigned int u32x4_byte __attribute__((ext_vector_type(4), aligned(1)));   // 16 bytes at any address
template <class U>
__device__ __forceinline__ U load_unit(const char* p) {
  if constexpr (sizeof(U) == 16) return *reinterpret_cast<const u32x4_byte*>(p);
  else return *reinterpret_cast<const U*>(p);
}
template <class U>
__device__ __forceinline__ void store_unit(char* p, U v) {
  if constexpr (sizeof(U) == 16) *reinterpret_cast<u32x4_byte*>(p) = v;
  else *reinterpret_cast<U*>(p) = v;
}
template <class U, int T, bool TWO>
__device__ __forceinline__ void copy_slots(const Cache& A, const Cache& B, int b, int h, int lane_bits, const int32_t* hole,
                                           const int32_t* fill, int lo, int hi) {
  char* ap = A.p + (int64_t)b * A.batch + (int64_t)h * A.head;
  char* bp = B.p + (int64_t)b * B.batch + (int64_t)h * B.head;
  const int lanes = 1 << lane_bits, sub = (int)threadIdx.x & (lanes - 1), per = T >> lane_bits;
  for (int m0 = lo + ((int)threadIdx.x >> lane_bits); m0 < hi; m0 += per * kCopyBatch) {
    int f[kCopyBatch], t[kCopyBatch];
#pragma unroll
    for (int i = 0; i < kCopyBatch; ++i) {
      const int m = min(m0 + i * per, hi - 1);
      f[i] = fill[m];
      t[i] = hole[m];
    }
    for (int u = sub; u < A.units; u += lanes) {
      U a[kCopyBatch], c[kCopyBatch];
      const int at = u * (int)sizeof(U), aa = min(at, A.last), ba = min(at, B.last);
#pragma unroll
      for (int i = 0; i < kCopyBatch; ++i) {
        a[i] = load_unit<U>(ap + (int64_t)f[i] * A.slot + aa);
        if (TWO) c[i] = load_unit<U>(bp + (int64_t)f[i] * B.slot + ba);
      }
#pragma unroll
      for (int i = 0; i < kCopyBatch; ++i) {
        if (m0 + i * per >= hi) continue;
        store_unit<U>(ap + (int64_t)t[i] * A.slot + aa, a[i]);
        if (TWO) store_unit<U>(bp + (int64_t)t[i] * B.slot + ba, c[i]);
      }
    }
  }
}
template <class U, int T>
__device__ __forceinline__ void copy_moves(const EParams& P, int r, const int32_t* hole, const int32_t* fill, int lo, int hi) {
  if (lo >= hi) return;
  const int b = r / P.heads, h = r - b * P.heads;
  if (P.k.units == P.v.units) {
    copy_slots<U, T, true>(P.k, P.v, b, h, P.lane_bits, hole, fill, lo, hi);
  } else {
    copy_slots<U, T, false>(P.k, P.k, b, h, P.lane_bits, hole, fill, lo, hi);
    copy_slots<U, T, false>(P.v, P.v, b, h, P.lane_bits, hole, fill, lo, hi);
  }
}

// The row's lists are whole: the freed slots' small outputs, the unused places, the length.
template <int NT>
__device__ __forceinline__ void finish_row(const EParams& P, int r, const Row& R, uint32_t moves) {
  const int32_t* pos = P.position + (int64_t)r * P.position_stride;
  const float* sum = P.sum + (int64_t)r * P.sum_stride;
  int32_t* source = P.out_source + (int64_t)r * P.keep_max;
  float* score = P.out_score + (int64_t)r * P.out_score_stride;
  int32_t* place = P.out_position + (int64_t)r * P.out_position_stride;
  const int32_t* hole = P.hole + (int64_t)r * P.cap;
  const int32_t* fill = P.fill + (int64_t)r * P.cap;
  for (uint32_t i = threadIdx.x; i < moves; i += NT) {
    const int h = hole[i], f = fill[i];
    source[h] = f;
    score[h] = sum[f];
    place[h] = pos[f];
  }
  bar_all();   // in place, the unused places below may be fillers' own
  for (int j = R.k + (int)threadIdx.x; j < P.keep_max; j += NT) {
    source[j] = -1;
    score[j] = 0.0f;
    place[j] = -1;
  }
  if (threadIdx.x == 0) {
    P.out_lengths[r] = R.k;
    P.moves[r] = (int32_t)moves;
    if (P.status) P.status[r] = TS_ROW_OK;
  }
}

// Ranks of a vector's four flags among all flags of the wave's vector (lanes, then elements, in order).
__device__ __forceinline__ uint32_t rank4(const uint64_t* m, int i) {
  uint32_t before = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) before += mbcnt(m[e]);
#pragma unroll
  for (int e = 0; e < 4; ++e) before += e < i ? (uint32_t)((m[e] >> lane()) & 1u) : 0u;
  return before;
}
__device__ __forceinline__ uint32_t count4(const uint64_t* m) {
  return (uint32_t)(__popcll(m[0]) + __popcll(m[1]) + __popcll(m[2]) + __popcll(m[3]));
}

// A vector of four slots from j on whose kept ones are the bits of `kept`: writes what stays in place and lists
// freed slots and fillers from ih and jf on (both advanced).
__device__ __forceinline__ void emit4(const EParams& P, int r, const Row& R, int j, uint32_t kept, const f32x4& s, const i32x4& p,
                                      uint32_t& ih, uint32_t& jf, bool keep_sums) {
  int32_t* source = P.out_source + (int64_t)r * P.keep_max;
  float* score = P.out_score + (int64_t)r * P.out_score_stride;
  int32_t* place = P.out_position + (int64_t)r * P.out_position_stride;
  int32_t* hole = P.hole + (int64_t)r * P.cap;
  int32_t* fill = P.fill + (int64_t)r * P.cap;
  const bool same_place = P.out_position == P.position;
  uint64_t mh[4], mf[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool in = (kept >> i) & 1u;
    mh[i] = __ballot(j + i < R.k && !in);
    mf[i] = __ballot(j + i >= R.k && in);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool in = (kept >> i) & 1u;
    if (j + i < R.k) {
      if (in) {
        source[j + i] = j + i;
        score[j + i] = s[i];
        if (!same_place) place[j + i] = p[i];
      } else {
        hole[ih + rank4(mh, i)] = j + i;
      }
    } else if (in) {
      fill[jf + rank4(mf, i)] = j + i;
      if (keep_sums) P.sum[(int64_t)r * P.sum_stride + j + i] = s[i];
    }
  }
  ih += count4(mh);
  jf += count4(mf);
}

// NT threads. SRC: the weights' type where the row is summed here, -1 where the sum kernel has run. NV: vectors a thread.
template <int NT, int NV, int SRC, class U>
__global__ __launch_bounds__(NT) void ts_evict_row_kernel(EParams P) {
  __shared__ ESmem sm;
  const int r = (int)blockIdx.x, l = lane();
  const int n = row_length(P, r);
  const int32_t* pos = P.position + (int64_t)r * P.position_stride;
  const float* sum = P.sum + (int64_t)r * P.sum_stride;
  const int base = wave() * NV * 256 + 4 * l;   // a wave's slots are consecutive
  f32x4 s[NV];
  i32x4 p[NV];
  uint32_t newest = 0, kmin = 0xFFFFFFFFu, kmax = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int j = base + 256 * v;
    if constexpr (SRC < 0) {
      s[v] = j < n ? *reinterpret_cast<const f32x4*>(sum + j) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    } else {
      double d[4] = {0.0, 0.0, 0.0, 0.0};
      if (j < n) sum_slots<SRC, kRowBatch>(P, r, j, n, d);
      s[v] = f32x4{(float)d[0], (float)d[1], (float)d[2], (float)d[3]};
    }
    p[v] = load4<i32x4, i32x4_any>(pos, j, n, (int32_t)0x80000000);
  }
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (base + 256 * v + i >= n) continue;
      newest = max(newest, (uint32_t)p[v][i] ^ 0x80000000u);
      const uint32_t k = f2key(s[v][i]);
      kmin = min(kmin, k);
      kmax = max(kmax, k);
    }
  newest = wave_max(newest);
  kmin = wave_min(kmin);
  kmax = wave_max(kmax);
  if (l == 0) {
    sm.red[wave()] = newest;
    sm.red2[wave()] = kmin;
    sm.red3[wave()] = kmax;
  }
  bar();
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    newest = max(newest, sm.red[w]);
    kmin = min(kmin, sm.red2[w]);
    kmax = max(kmax, sm.red3[w]);
  }
  bar();
  const Row R = row_of(P, r, newest, kmin, kmax);
  if (R.st != TS_ROW_OK) {
    reject_row<NT>(P, r, R);
    return;
  }
  // bit 4v + i: slot i of vector v is in use, is protected
  uint32_t live = 0, first = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = base + 256 * v + i < n;
      live |= (in ? 1u : 0u) << (4 * v + i);
      first |= (in && R.first(p[v][i]) ? 1u : 0u) << (4 * v + i);
    }
  const uint32_t total = block_total<NT / 64>(sm, wave_total(wave_incl_scan((uint32_t)__popc(first))));
  const bool among_first = total >= (uint32_t)R.k;
  const uint32_t need = among_first ? (uint32_t)R.k : (uint32_t)R.k - total;
  const uint32_t pool = among_first ? total : (uint32_t)n - total;
  const uint32_t cls = among_first ? first : live & ~first;   // the cut's class
  Cut cut{0u, 0xFFFFFFFFu};                                    // all of it
  if (need < pool) {
    cut = find_cut<NT>(
        sm, bitlen(kmax - kmin), 0u, need,
        [&](auto f) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((cls >> (4 * v + i)) & 1u) f(R.u(s[v][i]), base + 256 * v + i);
        },
        [&](uint32_t u, uint32_t nth) {
          uint32_t c = 0;
          uint64_t m[NV][4];
#pragma unroll
          for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) m[v][i] = __ballot(((cls >> (4 * v + i)) & 1u) && R.u(s[v][i]) == u);
            c += count4(m[v]);
          }
          uint32_t run, e, t0, t1;
          wave_offsets<NT / 64>(sm, c, 0u, run, e, t0, t1);
#pragma unroll
          for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (((m[v][i] >> l) & 1u) && run + rank4(m[v], i) + 1 == nth) sm.cut_slot = (uint32_t)(base + 256 * v + i);
            run += count4(m[v]);
          }
          bar();
          return sm.cut_slot;
        });
  }
  uint32_t kept = among_first ? 0u : first;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (((cls >> (4 * v + i)) & 1u) && cut.keeps(R.u(s[v][i]), base + 256 * v + i)) kept |= 1u << (4 * v + i);
  uint32_t ch = 0, cf = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = base + 256 * v + i;
      const bool in = (kept >> (4 * v + i)) & 1u;
      ch += (uint32_t)__popcll(__ballot(j < R.k && !in));
      cf += (uint32_t)__popcll(__ballot(j >= R.k && in));
    }
  uint32_t ih, jf, moves, tf;
  wave_offsets<NT / 64>(sm, ch, cf, ih, jf, moves, tf);
#pragma unroll
  for (int v = 0; v < NV; ++v)
    emit4(P, r, R, base + 256 * v, (kept >> (4 * v)) & 15u, s[v], p[v], ih, jf, SRC >= 0);
  bar_all();
  finish_row<NT>(P, r, R, moves);
  if constexpr (!std::is_void_v<U>) {
    const int32_t* hole = P.hole + (int64_t)r * P.cap;
    const int32_t* fill = P.fill + (int64_t)r * P.cap;
    if (P.k.units | P.v.units) copy_moves<U, NT>(P, r, hole, fill, 0, (int)moves);
  }
}

// ------------------------------------------------------------------ long rows
constexpr int kSW = kST / 64;
constexpr int kBinTiles = 4;

// The row's extremes from its tiles; every thread of the workgroup of NW waves gets them. red: 3 words a wave.
template <int NW>
__device__ __forceinline__ Row long_row(const EParams& P, int r, uint32_t* red, uint32_t& range) {
  const int n = row_length(P, r);
  uint32_t newest = 0, kmin = 0xFFFFFFFFu, kmax = 0;
  for (int i = threadIdx.x; (int64_t)i * kSumTile < n; i += 64 * NW) {
    const TileInfo ti = P.info[(int64_t)r * P.tiles + i];
    newest = max(newest, (uint32_t)ti.newest ^ 0x80000000u);
    kmin = min(kmin, ti.kmin);
    kmax = max(kmax, ti.kmax);
  }
  newest = wave_max(newest);
  kmin = wave_min(kmin);
  kmax = wave_max(kmax);
  if (lane() == 0) {
    red[3 * wave()] = newest;
    red[3 * wave() + 1] = kmin;
    red[3 * wave() + 2] = kmax;
  }
  bar();
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    newest = max(newest, red[3 * w]);
    kmin = min(kmin, red[3 * w + 1]);
    kmax = max(kmax, red[3 * w + 2]);
  }
  bar();
  range = kmax - kmin;
  return row_of(P, r, newest, kmin, kmax);
}

// A thread's four slots of a tile of a long row.
struct Quad {
  int j;
  f32x4 s;
  i32x4 p;
};
__device__ __forceinline__ Quad load_quad(const EParams& P, int r, int j, int n) {
  Quad q;
  q.j = j + (int)threadIdx.x * 4;
  q.s = q.j < n ? *reinterpret_cast<const f32x4*>(P.sum + (int64_t)r * P.sum_stride + q.j) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  q.p = load4<i32x4, i32x4_any>(P.position + (int64_t)r * P.position_stride, q.j, n, (int32_t)0x80000000);
  return q;
}

// A workgroup bins kBinTiles tiles: what it counts goes to the row's bins by an atomic for each bin that it met.
__global__ __launch_bounds__(kET) void ts_evict_bin_kernel(EParams P, int groups) {
  __shared__ uint32_t hist[2][kEBins];
  __shared__ uint32_t red[3 * kEW];
  __shared__ uint32_t np;
  const int r = (int)(blockIdx.x / (unsigned)groups), tile = (int)(blockIdx.x - (unsigned)r * (unsigned)groups) * kBinTiles * (kET / kST);
  const int n = row_length(P, r);
  if (tile * kSumTile >= n) return;
  Quad q[kBinTiles];
#pragma unroll
  for (int b = 0; b < kBinTiles; ++b) q[b] = load_quad(P, r, (tile + b * (kET / kST)) * kSumTile, n);
  for (int i = threadIdx.x; i < 2 * kEBins; i += kET) (&hist[0][0])[i] = 0u;
  if (threadIdx.x == 0) np = 0;
  uint32_t range;
  const Row R = long_row<kEW>(P, r, red, range);
  if (R.st != TS_ROW_OK) return;
  const int sh = max(bitlen(range) - kEBits, 0);
#pragma unroll
  for (int b = 0; b < kBinTiles; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (q[b].j + i >= n) continue;
      const bool f = R.first(q[b].p[i]);
      atomicAdd(&hist[f ? 1 : 0][R.u(q[b].s[i]) >> sh], 1u);
      if (f) atomicAdd(&np, 1u);
    }
  bar();
  uint32_t* h = P.hist + (int64_t)r * 2 * kEBins;
  for (int i = threadIdx.x; i < 2 * kEBins; i += kET) {
    const uint32_t c = (&hist[0][0])[i];
    if (c) atomicAdd(&h[i], c);
  }
  if (threadIdx.x == 0 && np) atomicAdd(&P.row[r].protected_, np);
}

__global__ __launch_bounds__(kST) void ts_evict_list_kernel(EParams P) {
  __shared__ uint32_t red[3 * kSW];
  __shared__ uint32_t res[3];
  int r, tile;
  tsl::place_block(P.tiles, r, tile);
  const int n = row_length(P, r), t = threadIdx.x;
  if (tile * kSumTile >= n) return;
  const Quad q = load_quad(P, r, tile * kSumTile, n);
  const uint32_t total = P.row[r].protected_;
  uint32_t range;
  const Row R = long_row<kSW>(P, r, red, range);
  if (R.st != TS_ROW_OK) return;
  const bool among_first = total >= (uint32_t)R.k;
  const uint32_t need = among_first ? (uint32_t)R.k : (uint32_t)R.k - total;
  const uint32_t pool = among_first ? total : (uint32_t)n - total;
  uint32_t out_count = 0, out_umin = 0xFFFFFFFFu, out_umax = 0;
  if (need < pool) {
    // thread t owns eight bins
    constexpr int kOwn = kEBins / kST;
    const uint32_t* h = P.hist + ((int64_t)r * 2 + (among_first ? 1 : 0)) * kEBins + t * kOwn;
    uint32_t c[kOwn], sum = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      c[i] = h[i];
      sum += c[i];
    }
    uint32_t all;
    const uint32_t before = block_excl_scan<kSW>(sum, red, all);
    uint32_t above = all - before - sum;
    if (above < need && above + sum >= need) {
      uint32_t bin = 0, in_bin = 0;
      bool found = false;
#pragma unroll
      for (int i = kOwn - 1; i >= 0; --i) {
        if (found) continue;
        bin = t * kOwn + i;
        in_bin = c[i];
        found = above + c[i] >= need;
        above += found ? 0u : c[i];
      }
      res[0] = bin;
      res[1] = above;
      res[2] = in_bin;
    }
    bar();
    const int lo = max(bitlen(range) - kEBits, 0);
    const uint32_t bin = res[0], left = need - res[1], in_bin = res[2];
    const bool listed = in_bin > left && in_bin <= (uint32_t)kListLong;
    uint32_t umin = 0xFFFFFFFFu, umax = 0;
    uint64_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = R.u(q.s[i]);
      const bool in = q.j + i < n && R.first(q.p[i]) == among_first && (u >> lo) == bin;
      if (in) {
        umin = min(umin, u);
        umax = max(umax, u);
      }
      m[i] = __ballot(in);
    }
    const uint32_t count = count4(m);
    umin = wave_min(umin);
    umax = wave_max(umax);
    if (lane() == 0) {
      red[3 * wave()] = count;
      red[3 * wave() + 1] = umin;
      red[3 * wave() + 2] = umax;
    }
    bar();
#pragma unroll
    for (int w = 0; w < kSW; ++w) {
      out_count += red[3 * w];
      out_umin = min(out_umin, red[3 * w + 1]);
      out_umax = max(out_umax, red[3 * w + 2]);
    }
    if (listed) {   // in the tile's own place, which its freed slots and fillers take later
      int64_t at = (int64_t)r * P.sum_stride + (int64_t)tile * kSumTile;
      for (int w = 0; w < wave(); ++w) at += red[3 * w];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((m[i] >> lane()) & 1u) {
          const uint32_t o = rank4(m, i);
          P.hole[at + o] = (int32_t)R.u(q.s[i]);
          P.fill[at + o] = q.j + i;
        }
    }
    if (tile == 0 && t == 0) {
      RowInfo& I = P.row[r];
      I.among_first = among_first ? 1u : 0u;
      I.prefix = bin;
      I.lo = (uint32_t)lo;
      I.need = left;
      I.in_bin = in_bin;
      I.whole = 0u;
    }
  } else if (tile == 0 && t == 0) {
    P.row[r].among_first = among_first ? 1u : 0u;
    P.row[r].whole = 1u;
  }
  if (t == 0) {   // (member by member: a struct of its own would be put into LDS, whose place the compiler finds by the
                  // dispatch packet, in host memory: 12 us)
    TileBin& out = P.bin[(int64_t)r * P.tiles + tile];
    out.count = out_count;
    out.umin = out_umin;
    out.umax = out_umax;
  }
}

// The tile whose share holds item `rank`: the last whose start is at most rank and below the next one's.
__device__ __forceinline__ int tile_of(const uint32_t* start, int tiles, uint32_t rank) {
  int x = 0, y = tiles;
  while (y - x > 1) {
    const int m = (x + y) >> 1;
    if (start[m] <= rank) x = m;
    else y = m;
  }
  return x;
}

// One workgroup a row: the cut's u and slot, and the row's status and length.
__global__ __launch_bounds__(kET) void ts_evict_cut_kernel(EParams P) {
  __shared__ ESmem sm;
  __shared__ uint32_t red[3 * kEW];
  __shared__ uint2 list[kListLong];
  __shared__ uint32_t start[kMaxTiles + 1];
  const int r = (int)blockIdx.x, t = threadIdx.x, l = lane();
  uint32_t range;
  const Row R = long_row<kEW>(P, r, red, range);
  if (t == 0) {
    P.row[r].st = R.st;
    P.row[r].k = R.k;
    P.row[r].tiles = (R.n + kSumTile - 1) / kSumTile;
  }
  if (R.st != TS_ROW_OK) {
    reject_row<kET>(P, r, R);
    return;
  }
  const RowInfo I = P.row[r];
  Cut cut{0u, 0xFFFFFFFFu};
  if (!I.whole && I.in_bin == I.need) {
    cut.u = I.prefix << I.lo;
  } else if (!I.whole && I.in_bin <= (uint32_t)kListLong) {
    // the tiles' shares, one after the other
    const int tiles = (R.n + kSumTile - 1) / kSumTile, own = (tiles + kET - 1) / kET;
    uint32_t c = 0, all;
    for (int i = t * own; i < min(tiles, (t + 1) * own); ++i) c += P.bin[(int64_t)r * P.tiles + i].count;
    uint32_t at = block_excl_scan<kEW>(c, sm.red, all);
    for (int i = t * own; i < min(tiles, (t + 1) * own); ++i) {
      start[i] = at;
      at += P.bin[(int64_t)r * P.tiles + i].count;
    }
    if (t == 0) start[tiles] = all;
    bar();
    for (uint32_t i = t; i < I.in_bin; i += kET) {
      const int x = tile_of(start, tiles, i);
      const int64_t o = (int64_t)r * P.sum_stride + (int64_t)x * kSumTile + (i - start[x]);
      list[i] = make_uint2((uint32_t)P.hole[o], (uint32_t)P.fill[o]);
    }
    bar();
    cut = find_cut<kET>(
        sm, (int)I.lo, I.prefix, I.need,
        [&](auto f) {
          for (uint32_t i = t; i < I.in_bin; i += kET) f(list[i].x, (int)list[i].y);
        },
        [&](uint32_t u, uint32_t nth) {   // equal u: the nth smallest slot of the list, by counting
          for (uint32_t i = t; i < I.in_bin; i += kET) {
            const uint2 me = list[i];
            if (me.x != u) continue;
            uint32_t below = 0;
            for (uint32_t o = 0; o < I.in_bin; ++o) below += list[o].x == u && list[o].y < me.y ? 1u : 0u;
            if (below + 1 == nth) sm.cut_slot = me.y;
          }
          bar();
          return sm.cut_slot;
        });
  } else if (!I.whole) {
    // Too many to list. The extreme u of the tiles' shares say whether all are equal.
    const bool af = I.among_first != 0;
    uint32_t umin = 0xFFFFFFFFu, umax = 0;
    for (int i = t; (int64_t)i * kSumTile < R.n; i += kET) {
      const TileBin b = P.bin[(int64_t)r * P.tiles + i];
      if (!b.count) continue;
      umin = min(umin, b.umin);
      umax = max(umax, b.umax);
    }
    umin = block_min_u32<kEW>(umin, sm.red);
    umax = block_max_u32<kEW>(umax, sm.red);
    const int32_t* pos = P.position + (int64_t)r * P.position_stride;
    const float* sum = P.sum + (int64_t)r * P.sum_stride;
    const int span = (((R.n + kEW - 1) / kEW) + 63) & ~63;
    const int w0 = min(R.n, wave() * span), w1 = min(R.n, w0 + span);
    auto of_class = [&](int j) { return j < w1 && R.first(pos[j]) == af; };
    auto ordered = [&](uint32_t u, uint32_t nth) {
      uint32_t c = 0;
      for (int b = w0; b < w1; b += 64) c += (uint32_t)__popcll(__ballot(of_class(b + l) && R.u(sum[b + l]) == u));
      uint32_t run, e0, t0, t1;
      wave_offsets<kEW>(sm, c, 0u, run, e0, t0, t1);
      if (run < nth && run + c >= nth) {
        for (int b = w0; b < w1; b += 64) {
          const uint64_t m = __ballot(of_class(b + l) && R.u(sum[b + l]) == u);
          if (((m >> l) & 1u) && run + mbcnt(m) + 1 == nth) sm.cut_slot = (uint32_t)(b + l);
          run += (uint32_t)__popcll(m);
        }
      }
      bar();
      return sm.cut_slot;
    };
    if (umin == umax) cut = Cut{umin, ordered(umin, I.need)};
    else
      cut = find_cut<kET>(
          sm, (int)I.lo, I.prefix, I.need,
          [&](auto f) {
            for (int j = w0 + l; j < w1; j += 64)
              if (of_class(j)) f(R.u(sum[j]), j);
          },
          ordered);
  }
  if (t == 0) {
    P.row[r].cut_u = cut.u;
    P.row[r].cut_slot = cut.slot;
  }
}

__global__ __launch_bounds__(kST) void ts_evict_emit_kernel(EParams P) {
  __shared__ uint32_t red[3 * kSW];
  int r, tile;
  tsl::place_block(P.tiles, r, tile);
  const int n = row_length(P, r);
  if (tile * kSumTile >= n) return;
  const Quad q = load_quad(P, r, tile * kSumTile, n);
  const RowInfo I = P.row[r];
  uint32_t range;
  const Row R = long_row<kSW>(P, r, red, range);
  if (R.st != TS_ROW_OK) return;
  const Cut cut{I.cut_u, I.cut_slot};
  const bool af = I.among_first != 0;
  uint32_t kept = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool f = R.first(q.p[i]);
    const bool in = q.j + i < n && (f != af ? f : cut.keeps(R.u(q.s[i]), q.j + i));
    kept |= (in ? 1u : 0u) << i;
  }
  uint64_t mh[4], mf[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mh[i] = __ballot(q.j + i < R.k && !((kept >> i) & 1u));
    mf[i] = __ballot(q.j + i >= R.k && ((kept >> i) & 1u));
  }
  if (lane() == 0) {
    red[2 * wave()] = count4(mh);
    red[2 * wave() + 1] = count4(mf);
  }
  bar();
  uint32_t ih = 0, jf = 0, holes = 0, fills = 0;
#pragma unroll
  for (int w = 0; w < kSW; ++w) {
    ih += w < wave() ? red[2 * w] : 0u;
    jf += w < wave() ? red[2 * w + 1] : 0u;
    holes += red[2 * w];
    fills += red[2 * w + 1];
  }
  const int64_t at = (int64_t)r * P.sum_stride + (int64_t)tile * kSumTile;
  int32_t* source = P.out_source + (int64_t)r * P.keep_max;
  float* score = P.out_score + (int64_t)r * P.out_score_stride;
  int32_t* place = P.out_position + (int64_t)r * P.out_position_stride;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = q.j + i;
    const bool in = (kept >> i) & 1u;
    if (j < R.k) {
      if (in) {
        source[j] = j;
        score[j] = q.s[i];
        if (P.out_position != P.position) place[j] = q.p[i];
      } else {
        P.hole[at + ih + rank4(mh, i)] = j;
      }
    } else if (in) {
      const uint32_t o = jf + rank4(mf, i);
      P.fill[at + o] = j;
      P.fill_position[at + o] = q.p[i];
    }
  }
  if (threadIdx.x == 0) {
    P.bin[(int64_t)r * P.tiles + tile].holes = holes;
    P.bin[(int64_t)r * P.tiles + tile].fills = fills;
  }
}

// A workgroup takes a share (one of `parts`) of a row's moves.
template <class U>
__global__ __launch_bounds__(kMT) void ts_evict_move_kernel(EParams P, int parts) {
  const int r = (int)(blockIdx.x / (unsigned)parts), part = (int)(blockIdx.x - (unsigned)r * (unsigned)parts);
  const int64_t n = P.moves[r];
  copy_moves<U, kMT>(P, r, P.hole + (int64_t)r * P.cap, P.fill + (int64_t)r * P.cap, (int)(n * part / parts),
                     (int)(n * (part + 1) / parts));
}

// Long rows: a workgroup takes a share (one of `parts`) of a tile's freed slots. Their ranks among the row's freed slots
// are those of their fillers among the row's fillers, which are found by the running count of the tiles' fillers.
template <class U>
__global__ __launch_bounds__(kMT) void ts_evict_long_move_kernel(EParams P, int hole_tiles, int parts) {
  __shared__ uint32_t red[kMT / 64];
  __shared__ uint32_t start[kMaxTiles + 1];     // fillers before each tile
  __shared__ uint32_t before;                   // freed slots before this workgroup's tile
  __shared__ int32_t to[kSumTile], from[kSumTile], place_of[kSumTile];
  const unsigned per = (unsigned)hole_tiles * (unsigned)parts;
  const int r = (int)(blockIdx.x / per), t = (int)threadIdx.x;
  const unsigned rest = blockIdx.x - (unsigned)r * per;
  const int tile = (int)(rest / (unsigned)parts), part = (int)(rest - (unsigned)tile * (unsigned)parts);
  const RowInfo I = P.row[r];
  if (I.st != TS_ROW_OK) return;
  int32_t* source = P.out_source + (int64_t)r * P.keep_max;
  float* score = P.out_score + (int64_t)r * P.out_score_stride;
  int32_t* place = P.out_position + (int64_t)r * P.out_position_stride;
  for (int j = max(I.k, tile * kSumTile) + part * kMT + t; j < min(P.keep_max, (tile + 1) * kSumTile); j += parts * kMT) {
    source[j] = -1;
    score[j] = 0.0f;
    place[j] = -1;
  }
  if (tile == 0 && part == 0 && t == 0) {
    P.out_lengths[r] = I.k;
    if (P.status) P.status[r] = TS_ROW_OK;
  }
  if (tile * kSumTile >= I.k) return;
  const TileBin* bin = P.bin + (int64_t)r * P.tiles;
  const uint32_t mine = bin[tile].holes;
  const uint32_t lo = (uint32_t)((uint64_t)mine * part / parts), hi = (uint32_t)((uint64_t)mine * (part + 1) / parts);
  if (lo == hi) return;
  const int own = (I.tiles + kMT - 1) / kMT;     // consecutive tiles a thread
  uint32_t fills = 0, holes = 0;
  for (int i = t * own; i < min(I.tiles, (t + 1) * own); ++i) {
    fills += bin[i].fills;
    holes += i < tile ? bin[i].holes : 0u;
  }
  uint32_t total;
  const uint32_t h = block_excl_scan<kMT / 64>(holes, red, total);
  (void)h;
  if (t == 0) before = total;
  uint32_t f = block_excl_scan<kMT / 64>(fills, red, total);
  for (int i = t * own; i < min(I.tiles, (t + 1) * own); ++i) {
    start[i] = f;
    f += bin[i].fills;
  }
  if (t == 0) start[I.tiles] = total;
  bar();
  const int64_t base = (int64_t)r * P.sum_stride;
  for (uint32_t i = lo + t; i < hi; i += kMT) {
    const uint32_t rank = before + i;
    const int x = tile_of(start, I.tiles, rank);
    const int64_t at = base + (int64_t)x * kSumTile + (rank - start[x]);
    to[i - lo] = P.hole[base + (int64_t)tile * kSumTile + i];
    from[i - lo] = P.fill[at];
    place_of[i - lo] = P.fill_position[at];
  }
  bar();
  if (P.k.units | P.v.units) copy_moves<U, kMT>(P, r, to, from, 0, (int)(hi - lo));
  for (int i = t; i < (int)(hi - lo); i += kMT) {
    const int dst = to[i], src = from[i];
    source[dst] = src;
    score[dst] = P.sum[base + src];
    place[dst] = place_of[i];
  }
}

// ------------------------------------------------------------------ host side
struct EPlan {
  int64_t cap = 0, sum_stride = 0, tiles = 0;
  bool spread = false;
  size_t off_info = 0, off_row = 0, off_bin = 0, off_hist = 0, off_moves = 0, off_hole = 0, off_fill = 0,
         off_fill_position = 0, total = 0;
};
bool evict_plan(int64_t rows, int64_t slots, int64_t keep_max, EPlan& pl) {
  if (rows < 0 || slots < 1 || slots > TS_EVICT_MAX_SLOTS || keep_max < 1 || keep_max > TS_EVICT_MAX_SLOTS) return false;
  pl.tiles = (slots + kSumTile - 1) / kSumTile;
  // a launch holds at most 2^32 - 1 threads
  if (rows > (int64_t)0xFFFFFFFF / kET || rows * pl.tiles > (int64_t)0xFFFFFFFF / kST ||
      rows * ((keep_max + kSumTile - 1) / kSumTile) > (int64_t)0xFFFFFFFF / kMT)
    return false;
  // a row moves at most min(k, n - k) positions
  pl.cap = std::min(keep_max, std::max<int64_t>(slots / 2, 1));
  pl.sum_stride = pl.tiles * kSumTile;
  pl.spread = slots > kWideSlots || (slots > kRowSlots && rows < kWideRows);
  const size_t rr = (size_t)std::max<int64_t>(rows, 1), listed = rr * (size_t)(pl.spread ? pl.sum_stride : pl.cap) * 4;
  size_t b = 0;
  auto take = [&](size_t bytes) {
    const size_t at = b;
    b += (bytes + 255) & ~(size_t)255;
    return at;
  };
  take(rr * (size_t)pl.sum_stride * 4);
  pl.off_moves = take(rr * 4);
  pl.off_hole = take(listed);
  pl.off_fill = take(listed);
  if (pl.spread) {
    pl.off_fill_position = take(listed);
    pl.off_info = take(rr * (size_t)pl.tiles * sizeof(TileInfo));
    pl.off_bin = take(rr * (size_t)pl.tiles * sizeof(TileBin));
    pl.off_row = take(rr * sizeof(RowInfo));
    pl.off_hist = take(rr * 2 * kEBins * 4);
  }
  pl.total = b;
  return true;
}

int dtype_size(int dtype) {
  return dtype == TS_DTYPE_F32 ? 4 : (dtype == TS_DTYPE_BF16 || dtype == TS_DTYPE_F16) ? 2 : 0;
}

// The copies' unit: 16 bytes at any address, where every slot has so many, else 4 where every address is a multiple, else 1.
int copy_unit(const ts_cache* k, const ts_cache* v) {
  uint64_t all = 0;
  bool wide = true;
  for (const ts_cache* c : {k, v})
    if (c) {
      wide = wide && c->slot_bytes >= 16;
      all |= (uint64_t)(uintptr_t)c->data | (uint64_t)c->batch_stride | (uint64_t)c->head_stride | (uint64_t)c->slot_stride |
             (uint64_t)c->slot_bytes;
    }
  return wide ? 16 : all % 4 == 0 ? 4 : 1;
}
Cache cache_of(const ts_cache* c, int unit) {
  if (!c) return Cache{nullptr, 0, 0, 0, 0, 0};
  return Cache{static_cast<char*>(c->data), c->batch_stride, c->head_stride, c->slot_stride,
               (int32_t)((c->slot_bytes + unit - 1) / unit), (int32_t)(c->slot_bytes - unit)};
}
// f(U) with the unit's type
template <class F>
void with_unit(int unit, F f) {
  switch (unit) {
    case 1: f(uint8_t{}); break;
    case 4: f(uint32_t{}); break;
    default: f(tsl::u32x4{}); break;
  }
}

// Where a row is also summed, and its moves also made, by its one workgroup: what a launch costs against what one
// compute unit reads and copies alone. (64 rows, one position dropped, summed here against a launch of its own: 1025
// slots, 4 weights of 2 bytes 9 us against 14; 4096 slots, 16 weights 16.6 against 16.9, 64 weights 26.9 against 25.8.
// Moves of 512 bytes made here: 2048 slots, one 9.8 us against 11.6, 1024 moves 24 against 18; the row's bound counts, as the
// number is known on the device only.)
constexpr int64_t kFusedBytes = 128 << 10;   // weights of a row
constexpr int64_t kFusedCopies = 8192;       // the threads' copies that a row's moves can take: 512 moves of 2 x 256 bytes
constexpr int64_t kMoveGroups = 1024;        // workgroups that moves are spread over, about (61,000 moves of 512 bytes: 17 us, with 2048 19.5),
constexpr int64_t kMoveParts = 32;           // and at most so many to a tile's

// The row kernel with the threads and vectors that hold the row: a fourth of the threads for short rows, of which then
// several share a compute unit (1025 slots: 64 rows 8.8 us against 8.6 with 1024 threads, 512 rows 11 against 17, 2048
// rows 26 against 65). U: the moves' unit, void: they are made elsewhere.
template <int SRC, class U>
void launch_rows(const EParams& P, hipStream_t s) {
  const dim3 grid((unsigned)P.rows);
  if (P.slots <= kSmallSlots) hipLaunchKernelGGL((ts_evict_row_kernel<kSmallT, 2, SRC, U>), grid, dim3(kSmallT), 0, s, P);
  else if (P.slots <= 4 * kET) hipLaunchKernelGGL((ts_evict_row_kernel<kET, 1, SRC, U>), grid, dim3(kET), 0, s, P);
  else if (P.slots <= kRowSlots) hipLaunchKernelGGL((ts_evict_row_kernel<kET, 2, SRC, U>), grid, dim3(kET), 0, s, P);
  else if constexpr (SRC < 0) hipLaunchKernelGGL((ts_evict_row_kernel<kET, 4, SRC, U>), grid, dim3(kET), 0, s, P);
}

int check_cache(const ts_cache* c, const char* name) {
  if (!c) return TS_OK;
  if (!c->data) return fail(TS_ERR_INVALID_ARG, "%s: data is NULL", name);
  if (c->slot_bytes < 1 || c->slot_bytes > (int64_t)1 << 24)
    return fail(TS_ERR_INVALID_ARG, "%s: slot_bytes = %lld outside [1, 2^24]", name, (long long)c->slot_bytes);
  if (c->slot_stride < c->slot_bytes)
    return fail(TS_ERR_INVALID_ARG, "%s: slot_stride %lld < slot_bytes %lld", name, (long long)c->slot_stride,
                (long long)c->slot_bytes);
  if (c->batch_stride < 0 || c->head_stride < 0) return fail(TS_ERR_INVALID_ARG, "%s: negative stride", name);
  return TS_OK;
}

}  // namespace

namespace tsh {
size_t cache_evict_workspace(int64_t rows, int64_t slots, int64_t keep_max) {
  EPlan pl;
  return evict_plan(rows, slots, keep_max, pl) ? pl.total : 0;
}
}  // namespace tsh

extern "C" int ts_cache_evict(const float* score, int64_t rows, int64_t slots, int64_t score_stride, const int32_t* position,
                              int64_t position_stride, const int32_t* lengths, const int32_t* keep, int32_t keep_max,
                              const void* weights, int weights_dtype, int64_t n_weights, int64_t weights_row_stride,
                              int64_t weights_stride, int32_t sinks, int32_t recent, float* out_score,
                              int64_t out_score_stride, int32_t* out_position, int64_t out_position_stride,
                              int32_t* out_lengths, int32_t* out_source, int32_t* row_status, const ts_cache* k_cache,
                              const ts_cache* v_cache, int64_t heads, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (rows < 0) return fail(TS_ERR_INVALID_ARG, "rows = %lld < 0", (long long)rows);
  if (slots < 1 || slots > TS_EVICT_MAX_SLOTS) return fail(TS_ERR_INVALID_ARG, "slots = %lld outside [1, 2^22]", (long long)slots);
  if (score_stride < slots || position_stride < slots)
    return fail(TS_ERR_INVALID_ARG, "score_stride %lld or position_stride %lld < slots %lld", (long long)score_stride,
                (long long)position_stride, (long long)slots);
  if (keep_max < 1 || keep_max > TS_EVICT_MAX_SLOTS)
    return fail(TS_ERR_INVALID_ARG, "keep_max = %d outside [1, 2^22]", (int)keep_max);
  if (out_score_stride < keep_max || out_position_stride < keep_max)
    return fail(TS_ERR_INVALID_ARG, "out_score_stride %lld or out_position_stride %lld < keep_max %d",
                (long long)out_score_stride, (long long)out_position_stride, (int)keep_max);
  if (sinks < 0 || recent < 0) return fail(TS_ERR_INVALID_ARG, "sinks = %d or recent = %d < 0", (int)sinks, (int)recent);
  if (n_weights < 0 || n_weights > 0x7FFFFFFF) return fail(TS_ERR_INVALID_ARG, "n_weights = %lld", (long long)n_weights);
  if (n_weights > 0) {
    if (!dtype_size(weights_dtype)) return fail(TS_ERR_INVALID_ARG, "weights_dtype = %d is none of TS_DTYPE_*", weights_dtype);
    if (weights_stride < 0 || weights_row_stride < 0) return fail(TS_ERR_INVALID_ARG, "negative weights stride");
  }
  if (heads < 1 || rows % heads) return fail(TS_ERR_INVALID_ARG, "heads = %lld does not divide rows", (long long)heads);
  if (rows == 0) return TS_OK;
  if (!score || !position || !lengths || !keep) return fail(TS_ERR_INVALID_ARG, "score, position, lengths and keep are required");
  if (!out_score || !out_position || !out_lengths || !out_source)
    return fail(TS_ERR_INVALID_ARG, "out_score, out_position, out_lengths and out_source are required");
  if ((out_score == score && out_score_stride != score_stride) ||
      (out_position == position && out_position_stride != position_stride))
    return fail(TS_ERR_INVALID_ARG, "an output in its input's place needs the input's stride");
  if (n_weights > 0 && !weights) return fail(TS_ERR_INVALID_ARG, "weights is NULL");
  if (n_weights > 0 && (uintptr_t)weights % dtype_size(weights_dtype))
    return fail(TS_ERR_INVALID_ARG, "weights are not aligned to their type");
  int rc = check_cache(k_cache, "k_cache");
  if (rc == TS_OK) rc = check_cache(v_cache, "v_cache");
  if (rc != TS_OK) return rc;
  EPlan pl;
  if (!evict_plan(rows, slots, keep_max, pl)) return fail(TS_ERR_INVALID_ARG, "rows x slots too large");
  if (!workspace) return fail(TS_ERR_WORKSPACE, "workspace is NULL");
  if (((uintptr_t)workspace & 255u) != 0) return fail(TS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (workspace_bytes < pl.total)
    return fail(TS_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, pl.total);
  int dev;
  rc = check_device(&dev);
  if (rc != TS_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  const int size = n_weights ? dtype_size(weights_dtype) : 4;
  EParams P;
  P.score = score;
  P.score_stride = score_stride;
  P.weights = static_cast<const char*>(weights);
  P.w_row = weights_row_stride * size;
  P.w_stride = weights_stride * size;
  P.n_w = (int32_t)n_weights;
  P.position = position;
  P.position_stride = position_stride;
  P.lengths = lengths;
  P.keep = keep;
  P.rows = (int32_t)rows;
  P.slots = (int32_t)slots;
  P.keep_max = keep_max;
  P.sinks = sinks;
  P.recent = recent;
  P.out_score = out_score;
  P.out_score_stride = out_score_stride;
  P.out_position = out_position;
  P.out_position_stride = out_position_stride;
  P.out_lengths = out_lengths;
  P.out_source = out_source;
  P.status = row_status;
  P.sum = reinterpret_cast<float*>(ws);
  P.sum_stride = pl.sum_stride;
  P.info = reinterpret_cast<TileInfo*>(ws + pl.off_info);
  P.row = reinterpret_cast<RowInfo*>(ws + pl.off_row);
  P.bin = reinterpret_cast<TileBin*>(ws + pl.off_bin);
  P.hist = reinterpret_cast<uint32_t*>(ws + pl.off_hist);
  P.fill_position = reinterpret_cast<int32_t*>(ws + pl.off_fill_position);
  P.tiles = (int32_t)pl.tiles;
  P.spread = pl.spread ? 1 : 0;
  P.moves = reinterpret_cast<int32_t*>(ws + pl.off_moves);
  P.hole = reinterpret_cast<int32_t*>(ws + pl.off_hole);
  P.fill = reinterpret_cast<int32_t*>(ws + pl.off_fill);
  P.cap = (int32_t)pl.cap;
  const int unit = copy_unit(k_cache, v_cache);
  P.k = cache_of(k_cache, unit);
  P.v = cache_of(v_cache, unit);
  P.heads = (int32_t)heads;
  const int64_t units = std::max(P.k.units, P.v.units);
  P.lane_bits = 0;
  while ((1 << P.lane_bits) < units && (1 << P.lane_bits) < kMT) ++P.lane_bits;
  const hipStream_t s = (hipStream_t)stream;
  const int type = n_weights ? weights_dtype : TS_DTYPE_F32;
  const bool sum_here = slots <= kRowSlots && slots * n_weights * size <= kFusedBytes;
  const bool move_here = sum_here && pl.cap * std::max<int64_t>(units, 1 << P.lane_bits) <= kFusedCopies;
  auto with_type = [&](auto f) {
    if (type == TS_DTYPE_F32) f(std::integral_constant<int, TS_DTYPE_F32>{});
    else if (type == TS_DTYPE_BF16) f(std::integral_constant<int, TS_DTYPE_BF16>{});
    else f(std::integral_constant<int, TS_DTYPE_F16>{});
  };
  hipError_t e;
  if (move_here) {
    with_type([&](auto dt) { with_unit(unit, [&](auto u) { launch_rows<dt(), decltype(u)>(P, s); }); });
    e = hipGetLastError();
    return e == hipSuccess ? TS_OK : fail(TS_ERR_LAUNCH, "eviction launch failed: %s", hipGetErrorString(e));
  }
  if (sum_here) {
    with_type([&](auto dt) { launch_rows<dt(), void>(P, s); });
  } else {
    const dim3 grid((unsigned)(rows * pl.tiles)), block(kST);
    with_type([&](auto dt) { hipLaunchKernelGGL(ts_evict_sum_kernel<dt()>, grid, block, 0, s, P); });
    e = hipGetLastError();
    if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "eviction sum launch failed: %s", hipGetErrorString(e));
    if (pl.spread) {
      const int64_t groups = (slots + kBinTiles * 4 * kET - 1) / (kBinTiles * 4 * kET);
      hipLaunchKernelGGL(ts_evict_bin_kernel, dim3((unsigned)(rows * groups)), dim3(kET), 0, s, P, (int)groups);
      hipLaunchKernelGGL(ts_evict_list_kernel, grid, block, 0, s, P);
      hipLaunchKernelGGL(ts_evict_cut_kernel, dim3((unsigned)rows), dim3(kET), 0, s, P);
      hipLaunchKernelGGL(ts_evict_emit_kernel, grid, block, 0, s, P);
      const int64_t hole_tiles = (keep_max + kSumTile - 1) / kSumTile;
      const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(kMoveParts, kMoveGroups / (rows * hole_tiles)));
      with_unit(unit, [&](auto u) {
        hipLaunchKernelGGL(ts_evict_long_move_kernel<decltype(u)>, dim3((unsigned)(rows * hole_tiles * parts)), dim3(kMT), 0, s, P,
                           (int)hole_tiles, (int)parts);
      });
      e = hipGetLastError();
      return e == hipSuccess ? TS_OK : fail(TS_ERR_LAUNCH, "eviction launch failed: %s", hipGetErrorString(e));
    }
    launch_rows<-1, void>(P, s);
  }
  e = hipGetLastError();
  if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "eviction row launch failed: %s", hipGetErrorString(e));
  if (units) {
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((pl.cap << P.lane_bits) / (kMT * kCopyBatch), kMoveGroups / rows));
    with_unit(unit, [&](auto u) {
      hipLaunchKernelGGL(ts_evict_move_kernel<decltype(u)>, dim3((unsigned)(rows * blocks)), dim3(kMT), 0, s, P, (int)blocks);
    });
    e = hipGetLastError();
    if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "eviction move launch failed: %s", hipGetErrorString(e));
  }
  return TS_OK;
}
