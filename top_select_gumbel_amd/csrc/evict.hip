// evict.hip -- eviction from key / value caches by accumulated attention weight.
//
// A cache row (one head of one sequence) holds n positions in slots 0 .. n-1. With s_j = score_j + sum_w weight[w, j]
// (binary64, rounded once to the fp32 that is kept), the row keeps its first k = min(keep, n) slots in the order
// (protected first, s descending, slot ascending); protected are the positions below `sinks` and the newest
// `recent` ones. The i-th slot below k that is not kept takes over the i-th kept slot at or past k, so
// that a row of which few positions go moves few, and nothing that is read is written.
//
// ts_evict_sum_kernel     s of every slot (grid over rows and slots): reads the weights once.
// ts_evict_select_kernel  one workgroup a row: the k-th slot of the order by radix select on ordered keys, then the
//                         freed slots and their fillers in slot order, and the row's small outputs.
// ts_evict_move_kernel    copies the fillers' keys and values (grid over rows and moves).
#include <algorithm>

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
constexpr int kET = 1024;                // threads of the select kernel
constexpr int kEW = kET / 64;
constexpr int kEBits = 11;
constexpr int kEBins = 1 << kEBits;
constexpr int kMT = 256;                 // threads of the move kernel

struct EParams {
  const float* score;
  int64_t score_stride;
  const char* weights;
  int64_t w_row, w_stride;               // bytes
  int32_t w_type, n_w;
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
  float* sum;                            // [rows, slots]
  int32_t* moves;                        // [rows]
  int32_t* hole;                         // [rows, cap]: the freed slots, ascending
  int32_t* fill;                         // [rows, cap]: what each takes over, ascending
  int32_t cap;
};

__device__ __forceinline__ int row_length(const EParams& P, int r) { return max(0, min(P.lengths[r], P.slots)); }

template <int DT>
__device__ __forceinline__ double weight_at(const char* w, int j) {
  return (double)tsl::load_logit<DT>(w, j);
}

template <int DT>
__global__ __launch_bounds__(kST) void ts_evict_sum_kernel(EParams P, int blocks) {
  const int r = (int)(blockIdx.x / (unsigned)blocks);
  const int j0 = (int)(blockIdx.x - (unsigned)r * (unsigned)blocks) * kST * kSumSlots + (int)threadIdx.x;
  const int n = row_length(P, r);
  const float* score = P.score + (int64_t)r * P.score_stride;
  const char* wr = P.weights + (int64_t)r * P.w_row;
#pragma unroll
  for (int i = 0; i < kSumSlots; ++i) {
    const int j = j0 + i * kST;
    if (j >= n) continue;
    double s = (double)score[j];
    for (int w = 0; w < P.n_w; ++w) s += weight_at<DT>(wr + (int64_t)w * P.w_stride, j);
    P.sum[(int64_t)r * P.slots + j] = (float)s;
  }
}

struct ESmem {
  uint32_t hist[kEBins];
  uint32_t red[kEW];
  uint32_t red2[kEW];
  uint32_t res[4];
};

// Exclusive prefix over the waves of two counts that every wave holds uniformly, and their totals.
__device__ __forceinline__ void wave_offsets(ESmem& sm, uint32_t a, uint32_t b, uint32_t& ea, uint32_t& eb, uint32_t& ta,
                                             uint32_t& tb) {
  if (lane() == 0) {
    sm.red[wave()] = a;
    sm.red2[wave()] = b;
  }
  bar();
  ea = eb = ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kEW; ++w) {
    const uint32_t x = sm.red[w], y = sm.red2[w];
    ea += w < wave() ? x : 0u;
    eb += w < wave() ? y : 0u;
    ta += x;
    tb += y;
  }
  bar();
}

__global__ __launch_bounds__(kET) void ts_evict_select_kernel(EParams P) {
  __shared__ ESmem sm;
  const int r = (int)blockIdx.x, t = (int)threadIdx.x, l = lane();
  const int n = row_length(P, r);
  const int32_t kr = P.keep[r];
  const int k = min(kr, n);
  const float* sum = P.sum + (int64_t)r * P.slots;
  const int32_t* pos = P.position + (int64_t)r * P.position_stride;
  int32_t* source = P.out_source + (int64_t)r * P.keep_max;
  float* score = P.out_score + (int64_t)r * P.out_score_stride;
  int32_t* place = P.out_position + (int64_t)r * P.out_position_stride;
  const bool same_score = P.out_score == P.score, same_place = P.out_position == P.position;

  // newest position, finiteness
  uint32_t newest = 0, bad = 0;
  for (int j = t; j < n; j += kET) {
    newest = max(newest, (uint32_t)pos[j] ^ 0x80000000u);
    const uint32_t b = __float_as_uint(sum[j]);
    bad |= (b & 0x7F800000u) == 0x7F800000u ? 1u : 0u;
  }
  newest = block_max_u32<kEW>(newest, sm.red);
  bad = block_max_u32<kEW>(bad, sm.red);
  const int st = bad ? TS_ROW_NONFINITE : (kr < 1 || k > P.keep_max) ? TS_ROW_BAD_K : TS_ROW_OK;
  if (st != TS_ROW_OK) {   // the row stays as it is
    for (int j = t; j < P.keep_max; j += kET) {
      source[j] = -1;
      if (!same_score) score[j] = __uint_as_float(0x7FC00000u);
      if (!same_place) place[j] = -1;
    }
    if (t == 0) {
      P.out_lengths[r] = n;
      P.moves[r] = 0;
      if (P.status) P.status[r] = st;
    }
    return;
  }
  const int64_t from = (int64_t)(int32_t)(newest ^ 0x80000000u) - P.recent;
  auto first = [&](int32_t p) { return p < P.sinks || (int64_t)p > from; };

  // Which class the cut falls into: among the protected slots where they alone fill the row, else among the others.
  uint32_t np = 0;
  for (int j = t; j < n; j += kET) np += first(pos[j]) ? 1u : 0u;
  np = wave_incl_scan(np);
  uint32_t ea, eb, total, unused;
  wave_offsets(sm, wave_total(np), 0u, ea, eb, total, unused);
  const bool among_first = total >= (uint32_t)k;
  uint32_t need = among_first ? (uint32_t)k : (uint32_t)k - total;
  const uint32_t pool = among_first ? total : (uint32_t)n - total;

  // Radix select of the need-th largest key of that class; the kept ones are those whose top (32 - lo) bits are above
  // `prefix`, or equal it with a slot not past `last`.
  uint32_t prefix = 0, last = 0xFFFFFFFFu;
  int lo = 32;
  if (need < pool) {
    while (lo > 0) {
      const int d = min(kEBits, lo), sh = lo - d;
      for (int i = t; i < kEBins; i += kET) sm.hist[i] = 0u;
      bar();
      for (int j = t; j < n; j += kET) {
        const uint32_t key = f2key(sum[j]);
        if (first(pos[j]) == among_first && shr(key, lo) == prefix) atomicAdd(&sm.hist[(key >> sh) & ((1u << d) - 1u)], 1u);
      }
      bar();
      // thread t owns bins 2t, 2t + 1
      const uint32_t c0 = sm.hist[2 * t], c1 = sm.hist[2 * t + 1];
      const uint32_t incl = wave_incl_scan(c0 + c1);
      uint32_t before, all;
      wave_offsets(sm, wave_total(incl), 0u, before, eb, all, unused);
      const uint32_t above = all - (before + incl);         // in the bins above this thread's
      if (above < need && above + c1 >= need) {
        sm.res[0] = 2 * t + 1;
        sm.res[1] = above;
        sm.res[2] = c1;
      } else if (above + c1 < need && above + c1 + c0 >= need) {
        sm.res[0] = 2 * t;
        sm.res[1] = above + c1;
        sm.res[2] = c0;
      }
      bar();
      prefix = shl(prefix, d) | sm.res[0];
      need -= sm.res[1];
      const uint32_t in_bin = sm.res[2];
      lo = sh;
      bar();
      if (in_bin == need) {
        need = 0;
        break;
      }
    }
  } else {
    need = 0;   // the whole class
  }
  auto inside = [&](int j) {
    const bool f = first(pos[j]);
    if (f != among_first) return f;              // protected slots beside a cut among the others
    const uint32_t h = shr(f2key(sum[j]), lo);
    return h > prefix || (h == prefix && (uint32_t)j <= last);
  };
  // A wave looks at consecutive slots, 64 at a time.
  const int span = ((n + kEW - 1) / kEW + 63) & ~63;
  const int w0 = wave() * span, w1 = min(n, w0 + span);
  if (need > 0) {   // equal keys on both sides of the cut: the lowest slots stay
    uint32_t c = 0;
    for (int j = w0 + l; j - l < w1; j += 64)
      c += (uint32_t)__popcll(__ballot(j < w1 && first(pos[j]) == among_first && f2key(sum[j]) == prefix));
    wave_offsets(sm, c, 0u, ea, eb, total, unused);
    if (ea < need && ea + c >= need) {
      uint32_t run = ea;
      for (int j = w0 + l; j - l < w1; j += 64) {
        const bool eq = j < w1 && first(pos[j]) == among_first && f2key(sum[j]) == prefix;
        const uint64_t m = __ballot(eq);
        if (eq && run + mbcnt(m) + 1 == need) sm.res[3] = (uint32_t)j;
        run += (uint32_t)__popcll(m);
      }
    }
    bar();
    last = sm.res[3];
  }

  // Freed slots and fillers, in slot order.
  uint32_t ch = 0, cf = 0;
  for (int j = w0 + l; j - l < w1; j += 64) {
    const bool in = j < w1 && inside(j);
    ch += (uint32_t)__popcll(__ballot(j < w1 && j < k && !in));
    cf += (uint32_t)__popcll(__ballot(j >= k && in));
  }
  uint32_t ih, jf, th, tf;
  wave_offsets(sm, ch, cf, ih, jf, th, tf);
  int32_t* hole = P.hole + (int64_t)r * P.cap;
  int32_t* fill = P.fill + (int64_t)r * P.cap;
  for (int j = w0 + l; j - l < w1; j += 64) {
    const bool in = j < w1 && inside(j);
    const bool h = j < w1 && j < k && !in, f = j >= k && in;
    const uint64_t mh = __ballot(h), mf = __ballot(f);
    if (h) hole[ih + mbcnt(mh)] = j;
    if (f) fill[jf + mbcnt(mf)] = j;
    if (in && j < k) {
      source[j] = j;
      score[j] = sum[j];
      if (!same_place) place[j] = pos[j];
    }
    ih += (uint32_t)__popcll(mh);
    jf += (uint32_t)__popcll(mf);
  }
  bar_all();
  for (uint32_t i = t; i < th; i += kET) {
    const int h = hole[i], f = fill[i];
    source[h] = f;
    score[h] = sum[f];
    place[h] = pos[f];
  }
  bar_all();
  for (int j = k + t; j < P.keep_max; j += kET) {
    source[j] = -1;
    score[j] = 0.0f;
    place[j] = -1;
  }
  if (t == 0) {
    P.out_lengths[r] = k;
    P.moves[r] = (int32_t)th;
    if (P.status) P.status[r] = TS_ROW_OK;
  }
}

struct Cache {
  char* p;
  int64_t batch, head, slot;   // bytes
  int32_t units;               // units of U bytes a slot
};

// Copies units of U bytes: thread i of a row's moves takes unit i % units of move i / units.
template <class U>
__global__ __launch_bounds__(kMT) void ts_evict_move_kernel(EParams P, Cache C, int heads, int blocks) {
  const int r = (int)(blockIdx.x / (unsigned)blocks);
  const int64_t i0 = (int64_t)(blockIdx.x - (unsigned)r * (unsigned)blocks) * kMT + threadIdx.x;
  const int64_t n = (int64_t)P.moves[r] * C.units;
  char* base = C.p + (int64_t)(r / heads) * C.batch + (int64_t)(r % heads) * C.head;
  const int32_t* hole = P.hole + (int64_t)r * P.cap;
  const int32_t* fill = P.fill + (int64_t)r * P.cap;
  for (int64_t i = i0; i < n; i += (int64_t)blocks * kMT) {
    const int64_t m = i / C.units, u = i - m * C.units;
    const U v = *reinterpret_cast<const U*>(base + (int64_t)fill[m] * C.slot + u * (int64_t)sizeof(U));
    *reinterpret_cast<U*>(base + (int64_t)hole[m] * C.slot + u * (int64_t)sizeof(U)) = v;
  }
}

// ------------------------------------------------------------------ host side
struct EPlan {
  int64_t cap = 0;
  size_t off_moves = 0, off_hole = 0, off_fill = 0, total = 0;
};
bool evict_plan(int64_t rows, int64_t slots, int64_t keep_max, EPlan& pl) {
  if (rows < 0 || slots < 1 || slots > TS_MAX_VOCAB || keep_max < 1 || keep_max > TS_MAX_VOCAB) return false;
  if (rows > 0x7FFFFF) return false;
  // a row moves at most min(k, n - k) positions
  pl.cap = std::min(keep_max, std::max<int64_t>(slots / 2, 1));
  const size_t rr = (size_t)std::max<int64_t>(rows, 1);
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  size_t b = up(rr * (size_t)slots * 4);
  pl.off_moves = b;
  b += up(rr * 4);
  pl.off_hole = b;
  b += up(rr * (size_t)pl.cap * 4);
  pl.off_fill = b;
  b += up(rr * (size_t)pl.cap * 4);
  pl.total = b;
  return true;
}

int dtype_size(int dtype) {
  return dtype == TS_DTYPE_F32 ? 4 : (dtype == TS_DTYPE_BF16 || dtype == TS_DTYPE_F16) ? 2 : 0;
}

template <class U>
void launch_move(const EParams& P, const Cache& C, int heads, int64_t blocks, hipStream_t s) {
  hipLaunchKernelGGL(ts_evict_move_kernel<U>, dim3((unsigned)(P.rows * blocks)), dim3(kMT), 0, s, P, C, heads, (int)blocks);
}

hipError_t move_cache(const EParams& P, const ts_cache& c, int heads, hipStream_t s) {
  // the widest unit that divides every address
  const uint64_t all = (uint64_t)(uintptr_t)c.data | (uint64_t)c.batch_stride | (uint64_t)c.head_stride |
                       (uint64_t)c.slot_stride | (uint64_t)c.slot_bytes;
  const int unit = (all & 1) ? 1 : (all & 2) ? 2 : (all & 4) ? 4 : (all & 8) ? 8 : 16;
  Cache C{static_cast<char*>(c.data), c.batch_stride, c.head_stride, c.slot_stride, (int32_t)(c.slot_bytes / unit)};
  const int64_t most = (int64_t)P.cap * C.units;
  int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((most + kMT - 1) / kMT, std::max<int64_t>(1, 4096 / P.rows)));
  switch (unit) {
    case 1: launch_move<uint8_t>(P, C, heads, blocks, s); break;
    case 2: launch_move<uint16_t>(P, C, heads, blocks, s); break;
    case 4: launch_move<uint32_t>(P, C, heads, blocks, s); break;
    case 8: launch_move<uint2>(P, C, heads, blocks, s); break;
    default: launch_move<uint4>(P, C, heads, blocks, s); break;
  }
  return hipGetLastError();
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
  if (slots < 1 || slots > TS_MAX_VOCAB) return fail(TS_ERR_INVALID_ARG, "slots = %lld outside [1, 2^30]", (long long)slots);
  if (score_stride < slots || position_stride < slots)
    return fail(TS_ERR_INVALID_ARG, "score_stride %lld or position_stride %lld < slots %lld", (long long)score_stride,
                (long long)position_stride, (long long)slots);
  if (keep_max < 1 || keep_max > TS_MAX_VOCAB) return fail(TS_ERR_INVALID_ARG, "keep_max = %d outside [1, 2^30]", (int)keep_max);
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
  if (!evict_plan(rows, slots, keep_max, pl)) return fail(TS_ERR_INVALID_ARG, "rows too large");
  const int64_t per = (slots + kST * kSumSlots - 1) / (kST * kSumSlots);
  if (rows * per > (int64_t)0xFFFFFFFF / kST) return fail(TS_ERR_INVALID_ARG, "rows x slots too large");
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
  P.w_type = weights_dtype;
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
  P.moves = reinterpret_cast<int32_t*>(ws + pl.off_moves);
  P.hole = reinterpret_cast<int32_t*>(ws + pl.off_hole);
  P.fill = reinterpret_cast<int32_t*>(ws + pl.off_fill);
  P.cap = (int32_t)pl.cap;
  const hipStream_t s = (hipStream_t)stream;
  const dim3 grid((unsigned)(rows * per)), block(kST);
  if (n_weights == 0 || weights_dtype == TS_DTYPE_F32) hipLaunchKernelGGL(ts_evict_sum_kernel<TS_DTYPE_F32>, grid, block, 0, s, P, (int)per);
  else if (weights_dtype == TS_DTYPE_BF16) hipLaunchKernelGGL(ts_evict_sum_kernel<TS_DTYPE_BF16>, grid, block, 0, s, P, (int)per);
  else hipLaunchKernelGGL(ts_evict_sum_kernel<TS_DTYPE_F16>, grid, block, 0, s, P, (int)per);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "eviction sum launch failed: %s", hipGetErrorString(e));
  hipLaunchKernelGGL(ts_evict_select_kernel, dim3((unsigned)rows), dim3(kET), 0, s, P);
  e = hipGetLastError();
  if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "eviction select launch failed: %s", hipGetErrorString(e));
  for (const ts_cache* c : {k_cache, v_cache}) {
    if (!c) continue;
    e = move_cache(P, *c, (int)heads, s);
    if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "eviction move launch failed: %s", hipGetErrorString(e));
  }
  return TS_OK;
}
