// logprobs.hip -- log probabilities of given tokens with rank, entropy and the best alternatives, and their gradient.
//
// For a row x of V logits at temperature T, with m = max x, d_i = (x_i - m) / T and S = sum exp(d_i):
//   logp_t  = d_t - log S                      lse = m / T + log S
//   entropy = log S - (1/S) sum exp(d_i) d_i   rank_t = 1 + #{x_i > x_t} + #{i < t : x_i = x_t}
// and with a, h, l the gradients of logp, entropy and lse, p_i = exp(d_i) / S and D = (1/S) sum exp(d_i) d_i
//   dL/dx_i = (a [i = t] + p_i (l - a - h (d_i - D))) / T
// since log p_i + entropy = d_i - D.
//
// ts_logp_tile_kernel  reads a tile of a row (8192 logits, 32 a thread, in registers) once: its maximum, the two sums
//                      relative to it, how many logits rank above the given token, and, where alternatives are asked
//                      for, every logit that can be among the row's best n. The sums are fp32 over a thread's
//                      32 terms and binary64 beyond. A row of one tile is finished by the same workgroup.
// ts_logp_row_kernel   joins a row's tiles in tile order (binary64), a row a wave.
// ts_logp_top_kernel   the same, while other waves find the row's best n among the tiles' candidates.
// ts_logp_grad_kernel  one pass: reads a tile, writes its gradient.
//
// Measured (MI355X; a plain read of the same bytes takes 92 us for 2048 x 151936 in bf16, 68 us for 1777 x 128256):
//   2048 x 151936 bf16  tile 93-116 us (6.7-5.4 TB/s), row 6 us, gradient 187 us (6.7 TB/s read and written)
//   1777 x 128256 bf16  tile 80 us without ranks and alternatives (5.7 TB/s), 95-98 us with both (n = 5), top 8 us
//   64 x 151936 fp32    tile 12-15 us with ranks and 20 alternatives, top 5.6 us (a plain read: 8 us)
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "topselect.h"
#include "ts_device.hpp"
#include "ts_host.hpp"
#include "ts_logits.hpp"

using namespace tsd;
using namespace tsl;
using tsh::check_device;
using tsh::fail;

namespace {

constexpr int kLW = kLT / 64;        // waves a tile
constexpr double kLn2 = 0.6931471805599453;

// What a tile leaves for its row: its maximum (NaN seen: +inf; nothing but -inf: -inf), the sums of 2^z and
// 2^z z over it (z = (x - m) log2(e) / T) and how many of its logits rank above the given token.
struct Part {
  double s, d;
  float m;
  uint32_t above;
  uint32_t pad[2];
};
static_assert(sizeof(Part) == 32, "Part layout");

struct LParams {
  const char* x;
  int64_t stride;              // bytes
  int32_t V, rows, tiles, n_top, cap;
  const int32_t* tokens;
  const float* t;
  float* logp;
  int32_t* rank;
  float* entropy;
  float* lse;
  int32_t* top_idx;
  float* top_logp;
  float4* stats;
  int32_t* status;
  Part* part;
  uint2* cand;                 // per (row, tile): cap (key, id) slots, unused ones 0
};

// Candidates kept a tile: at least n, and room for the threads that hold several.
__host__ __device__ constexpr int cand_cap(int n) { return n ? (2 * n + 32 + 15) / 16 * 16 : 0; }
constexpr int kCapMax = cand_cap(TS_LOGP_TOP_MAX);
static_assert((kCapMax + 63) / 64 <= 4, "what is left of the candidates joins the four groups of a lane");

struct LSmem {
  uint32_t tk[kLT];            // each thread's largest key
  float2 sums[kLT];            // each thread's sums of 2^z and 2^z z
  uint2 list[kCapMax];         // (key, id), in no order
  uint8_t who[kLT];            // threads with candidates
  uint32_t count;
  uint32_t redn[kLW];
  Part part;
  float m;
  double log_s, c2;
  int32_t ok;
};

// Sum over the wave, in a fixed order: the lane moves of wave_incl_scan on both halves. Every lane gets it.
template <int CTRL, int RMASK>
__device__ __forceinline__ double moved(double v) {
  return __longlong_as_double((long long)dpp64<CTRL, RMASK>((uint64_t)__double_as_longlong(v)));
}
__device__ __forceinline__ double wave_sum_f64(double v) {
  v += moved<0x111, 0xf>(v);
  v += moved<0x112, 0xf>(v);
  v += moved<0x114, 0xf>(v);
  v += moved<0x118, 0xf>(v);
  v += moved<0x142, 0xa>(v);
  v += moved<0x143, 0xc>(v);
  return __longlong_as_double((long long)readlane64((uint64_t)__double_as_longlong(v), 63));
}

// ------------------------------------------------------------------ the best n
// The key whose leading bits are u's: the fraction bits that the type lacks are 0 in its logits, 1 in the keys of negative ones.
template <int DT>
__device__ __forceinline__ uint32_t whole_key(uint32_t u) {
  return u >> 31 ? u : u | ((1u << tsl::Logits<DT>::kLowBits) - 1u);
}

// A bound that at least n of some items reach and, where large items are spread over their 256 groups, few more: about the
// n-th largest of the groups' largest keys (keys up to that of -inf are absent items). Called by one
// wave, which has four of those keys a lane in k4; kmax is the largest. The bits above the highest one in which they differ
// are common to all; the others are found one by one, until at most n + 8 groups reach the bound: each further bit would
// cost more than the items it saves. Not so where that is more than half of the groups that have items (a short row, a mask
// that leaves a few neighbours): each then has several above it (1325 x 100 in fp16, n = 5: 80 us for that reason).
template <int DT>
__device__ __forceinline__ uint32_t find_low(const uint32_t* k4, uint32_t kmax, int n) {
  uint32_t kmin = k4[0];
#pragma unroll
  for (int w = 1; w < kLW; ++w) kmin = min(kmin, k4[w]);
  const uint32_t differ = kmax ^ wave_min(kmin);
  const int bits = bitlen(differ);
  uint32_t low = bits == 32 ? 0u : kmax >> bits << bits;
  int live = 0;
#pragma unroll
  for (int w = 0; w < kLW; ++w) live += __popcll(__ballot(k4[w] > kKeyNegInf));
  const int enough = min(n + 8, live / 2);
  for (int b = bits - 1; b >= tsl::Logits<DT>::kLowBits; --b) {
    const uint32_t t = low | (1u << b);
    int c = 0;
#pragma unroll
    for (int w = 0; w < kLW; ++w) c += __popcll(__ballot(k4[w] >= t));
    if (c >= n) {
      low = t;
      if (c <= enough) break;
    }
  }
  return whole_key<DT>(max(low, kKeyNegInf + 1));
}

// A tile's exact best n, where more candidates reach the bound `low` than the list holds: many equal logits around it (a mask
// of the type's lowest value, a constant row), or the large ones in few threads (a sorted row, a mask that leaves a
// few neighbours). One wave reads the vectors of the `threads` threads with candidates again, in id order, once for each
// count where they are more than it holds in registers; so this path holds no registers of the usual one. The row has more than
// n logits, so at least a vector's.
template <int DT>
__device__ void exact_tile(LSmem& sm, const char* row, int V, int tile, int n, uint32_t low, uint32_t kmax, int threads) {
  using L = Logits<DT>;
  constexpr int kBatch = 4;
  const int total = threads * L::kNV;
  const uint32_t inverse = ((1u << 20) + (uint32_t)threads - 1) / (uint32_t)threads;   // exact for quotients of numbers up to 2^11
  u32x4 raw[kBatch];
  int at[kBatch];
  bool held = false;
  // f(first id, keys) for a vector a lane, until it returns true; what does not count is -inf, below every candidate.
  auto each = [&](auto f) {
#pragma nounroll
    for (int q0 = 0; q0 < total; q0 += 64 * kBatch) {
      if (!held || total > 64 * kBatch) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int q = q0 + 64 * i + lane(), in = min(q, total - 1), v = (int)((uint32_t)in * inverse >> 20);
          const Place<DT> pl(tile, sm.who[in - v * threads], v, V);
          at[i] = pl.at;
          raw[i] = load16(row + (int64_t)pl.at * L::kSize);
#pragma unroll
          for (int j = 0; j < L::kW; ++j) {
            const uint32_t half = L::kSize == 4 ? 0xFFFFFFFFu : (j & 1) ? 0xFFFF0000u : 0x0000FFFFu;
            const int w = j * L::kSize / 4;
            if (q >= total || !pl.counts(j, V)) raw[i][w] = (raw[i][w] & ~half) | (L::kNegInf & half);
          }
        }
        held = true;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (q0 + 64 * i >= total) continue;
        uint32_t key[L::kW];
#pragma unroll
        for (int j = 0; j < L::kW; ++j) key[j] = f2key(unpack<DT>(raw[i], j));
        if (f(at[i], key)) return;
      }
    }
  };
  auto count = [&](uint32_t least) {   // of keys from `least` on, up to n
    uint32_t c = 0;
    each([&](int, const uint32_t* key) {
#pragma unroll
      for (int j = 0; j < L::kW; ++j) c += (uint32_t)__popcll(__ballot(key[j] >= least));
      return c >= (uint32_t)n;
    });
    return c;
  };
  // t becomes the n-th largest key: the bound itself where fewer are above it, else, between it and the tile's largest, bit by bit.
  uint32_t t = low, above = low < kmax ? count(low + 1) : 0u;
  if (above >= (uint32_t)n) {
    const int bits = bitlen(low ^ kmax);
    t = bits == 32 ? 0u : low >> bits << bits;
#pragma nounroll
    for (int b = bits - 1; b >= L::kLowBits; --b) {
      const uint32_t u = t | (1u << b);
      if (count(u) >= (uint32_t)n) t = u;
    }
    t = whole_key<DT>(t);
    above = count(t + 1);
  }
  const uint32_t need = n - above;   // of the logits equal to it, in id order
  uint32_t seen = 0, put = 0;
  each([&](int at, const uint32_t* key) {
    uint32_t eq = 0;
#pragma unroll
    for (int j = 0; j < L::kW; ++j) eq += key[j] == t ? 1u : 0u;
    const uint32_t incl = wave_incl_scan(eq);
    uint32_t rank = seen + incl - eq;
    seen += wave_total(incl);
#pragma unroll
    for (int j = 0; j < L::kW; ++j) {
      const bool in = key[j] > t || (key[j] == t && rank < need);
      rank += key[j] == t ? 1u : 0u;
      const uint64_t m = __ballot(in);
      const uint32_t o = put + mbcnt(m);
      if (in && o < (uint32_t)kCapMax) sm.list[o] = make_uint2(key[j], (uint32_t)(at + j));
      put += (uint32_t)__popcll(m);
    }
    return put == (uint32_t)n;
  });
}

// The tile's candidates, into sm.list, by one wave: those of the threads' logits that reach `low`, of the threads whose
// largest does (their keys in k4). Returns their number. The few threads' logits are read again, from the caches, by
// as many lanes as they have vectors: looking through all threads' registers takes every wave longer.
template <int DT>
__device__ __forceinline__ int tile_candidates(LSmem& sm, const char* row, int V, int tile, int n, int cap, uint32_t low,
                                               uint32_t kmax, const uint32_t* k4) {
  using L = Logits<DT>;
  uint32_t threads = 0;
#pragma unroll
  for (int w = 0; w < kLW; ++w) {
    const uint64_t m = __ballot(k4[w] >= low);
    if (k4[w] >= low) sm.who[threads + mbcnt(m)] = (uint8_t)(64 * w + lane());
    threads += (uint32_t)__popcll(m);
  }
  wave_lds_sync();
  const float low_f = key2f(low);
  const bool whole = (tile + 1) * kTile <= V;
  uint32_t put = 0;
  for (uint32_t q0 = 0; q0 < threads * L::kNV && put <= (uint32_t)cap; q0 += 64) {
    const uint32_t q = q0 + lane();
    const bool mine = q < threads * L::kNV;
    const Place<DT> pl(tile, mine ? sm.who[q / L::kNV] : 0, (int)(q % L::kNV), V);
    u32x4 raw = {L::kNegInf, L::kNegInf, L::kNegInf, L::kNegInf};
    if (V >= L::kW && mine) raw = load16(row + (int64_t)pl.at * L::kSize);
#pragma unroll
    for (int j = 0; j < L::kW; ++j) {
      float x = unpack<DT>(raw, j);
      if (!whole) {
        if (V < L::kW && mine && j < V) x = load_logit<DT>(row, j);
        if (!pl.counts(j, V)) x = -INFINITY;
      }
      const uint64_t m = __ballot(x >= low_f);
      if (!m) continue;
      const uint32_t o = put + mbcnt(m);
      if (x >= low_f && o < (uint32_t)kCapMax) sm.list[o] = make_uint2(f2key(x), (uint32_t)(pl.at + j));
      put += (uint32_t)__popcll(m);
    }
  }
  if (put > (uint32_t)cap) {
    exact_tile<DT>(sm, row, V, tile, n, low, kmax, (int)threads);
    put = n;
  }
  wave_lds_sync();
  return (int)put;
}

// The exact best n of items that a wave's lanes hold N each, more than n of which reach `low` and none is above kmax, found bit
// by bit: the n-th largest key, then, among those equal to it, the id of the last that stays (ids are below V and differ).
template <int N>
__device__ __forceinline__ void exact_items(uint2* list, const uint2* c, int n, uint32_t low, uint32_t kmax, int V) {
  auto count = [&](auto pred) {
    uint32_t k = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) k += (uint32_t)__popcll(__ballot(pred(c[i])));
    return k;
  };
  const int bits = bitlen(low ^ kmax);
  uint32_t t = bits == 32 ? 0u : low >> bits << bits, last = 0;
#pragma nounroll
  for (int b = bits - 1; b >= 0; --b) {
    const uint32_t u = t | (1u << b);
    if (count([&](const uint2& q) { return q.x >= u; }) >= (uint32_t)n) t = u;
  }
  const uint32_t need = n - count([&](const uint2& q) { return q.x > t; });
#pragma nounroll
  for (int b = bitlen((uint32_t)V - 1u) - 1; b >= 0; --b) {
    const uint32_t u = last | (1u << b);
    if (count([&](const uint2& q) { return q.x == t && q.y < u; }) < need) last = u;
  }
  uint32_t put = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool in = c[i].x > t || (c[i].x == t && c[i].y <= last);
    const uint64_t m = __ballot(in);
    const uint32_t o = put + mbcnt(m);
    if (in && o < (uint32_t)kCapMax) list[o] = c[i];
    put += (uint32_t)__popcll(m);
  }
}

// ------------------------------------------------------------------ a row's parameters
struct RowIn {
  float t;
  int32_t token;    // -1: none
  bool bad_t, bad_token;
};
__device__ __forceinline__ RowIn row_in(const LParams& P, int r) {
  RowIn in;
  in.t = P.t ? P.t[r] : 1.0f;
  in.bad_t = !(in.t >= 0.0f && in.t <= 3.402823466e38f);
  in.token = P.tokens ? P.tokens[r] : -1;
  in.bad_token = in.token < -1 || in.token >= P.V;
  if (in.bad_token) in.token = -1;
  return in;
}

// ------------------------------------------------------------------ a tile
// log2(e) / T rounded once, or nearly (r + r e is 1/T to twice fp32's bits, and kHi + kLo log2(e)).
__device__ __forceinline__ float scale32(const LParams& P, float t) {
  constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
  if (!P.t) return kHi;
  t = fmaxf(t, 0x1p-100f);
  const float r = 1.0f / t, e = fmaf(-r, t, 1.0f);
  return fmaf(kHi, r, fmaf(kLo, r, kHi * (e * r)));
}

// How many of the wave's logits of the tile, whose largest key is k, rank above the given token.
template <int DT>
__device__ __forceinline__ uint32_t wave_above(const LParams& P, const RowIn& in, int tile, const float* xs,
                                               uint32_t k, float xt) {
  if (f2key(xt) > k) return 0;   // most tiles of a likely token
  const int at = in.token / kTile;
  uint32_t above = 0;
  if (tile < at) {
#pragma unroll
    for (int i = 0; i < kLE; ++i) above += (uint32_t)__popcll(__ballot(xs[i] >= xt));
  } else if (tile > at) {
#pragma unroll
    for (int i = 0; i < kLE; ++i) above += (uint32_t)__popcll(__ballot(xs[i] > xt));
  } else {
#pragma unroll
    for (int v = 0; v < Logits<DT>::kNV; ++v) {
      const Place<DT> pl(tile, threadIdx.x, v, P.V);
#pragma unroll
      for (int j = 0; j < Logits<DT>::kW; ++j) {
        const float x = xs[v * Logits<DT>::kW + j];
        above += (uint32_t)__popcll(__ballot(x > xt || (x == xt && pl.at + j < in.token && pl.counts(j, P.V))));
      }
    }
  }
  return above;
}

// The largest of N logits, NaN if one is.
template <int N>
__device__ __forceinline__ float max_of(const float* xs) {
  float m = xs[0];
#pragma unroll
  for (int i = 1; i + 1 < N; i += 2)
    m = __builtin_elementwise_maximum(m, __builtin_elementwise_maximum(xs[i], xs[i + 1]));
  if (N % 2 == 0) m = __builtin_elementwise_maximum(m, xs[N - 1]);
  return m;
}

// ------------------------------------------------------------------ a row
// Joins a row's tiles and writes its scalars; called by one whole wave. Leaves in sm (thread 0's copy) what the
// alternatives need.
template <int DT>
__device__ __forceinline__ void finish_row(const LParams& P, const RowIn& in, int r, const Part* part, LSmem* sm) {
  const int l = lane();
  const float nan = __uint_as_float(0x7FC00000u);
  const float xt = (P.tokens && in.token >= 0) ? load_logit<DT>(P.x + (int64_t)r * P.stride, in.token) : 0.0f;
  uint32_t km = 0;
  for (int i = l; i < P.tiles; i += 64) km = max(km, f2key(part[i].m));
  km = wave_max(km);
  const float m = key2f(km);
  const double c2 = exponent_scale(in.t);
  double s = 0.0, d = 0.0;
  uint32_t above = 0;
  const bool finite = km < kKeyPosInf && km > kKeyNegInf;
  if (finite) {
    for (int i = l; i < P.tiles; i += 64) {
      const Part p = part[i];
      above += p.above;
      if (p.m == -INFINITY) continue;
      const double dz = ((double)p.m - (double)m) * c2;
      const double w = exp2(dz);
      if (w > 0.0) {
        s += w * p.s;
        d += w * (p.d + dz * p.s);
      }
    }
    s = wave_sum_f64(s);
    d = wave_sum_f64(d);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) above += (uint32_t)__shfl_xor((int)above, o);
  }
  if (l != 0) return;
  int st = TS_ROW_OK;
  if (!finite) st = TS_ROW_NONFINITE;
  else if (in.bad_t) st = TS_ROW_BAD_T;
  else if (in.bad_token) st = TS_ROW_BAD_TOKEN;
  const bool ok = st == TS_ROW_OK, greedy = in.t == 0.0f, given = in.token >= 0;
  const double log_s = ok && !greedy ? log(s) : 0.0, mean = ok && !greedy ? d / s * kLn2 : 0.0;
  float logp = 0.0f;
  if (given && greedy) logp = above == 0 ? 0.0f : -INFINITY;
  else if (given) logp = fminf((float)(((double)xt - (double)m) * c2 * kLn2 - log_s), 0.0f);
  if (P.logp) P.logp[r] = ok ? logp : nan;
  if (P.rank) P.rank[r] = ok ? (given ? (int32_t)above + 1 : 0) : -1;
  if (P.entropy) P.entropy[r] = ok ? fmaxf((float)(log_s - mean), 0.0f) : nan;
  if (P.lse) P.lse[r] = ok ? (greedy ? INFINITY : (float)((double)m * c2 * kLn2 + log_s)) : nan;
  if (P.stats) {   // maximum, S, D, 1 - 1/S
    const double ss = greedy ? 1.0 : s;
    P.stats[r] = ok ? make_float4(m, (float)ss, (float)mean, (float)((ss - 1.0) / ss)) : make_float4(nan, nan, nan, nan);
  }
  if (P.status) P.status[r] = st;
  if (sm) {
    sm->m = m;
    sm->log_s = log_s;
    sm->c2 = c2;
    sm->ok = ok ? (greedy ? 2 : 1) : 0;
  }
}

// Ranks the `count` candidates of sm.list and writes the row's n_top alternatives; called by a workgroup of T threads, after
// finish_row.
template <int T>
__device__ __forceinline__ void write_top(const LParams& P, int r, int count, const LSmem& sm) {
  const int t = (int)threadIdx.x, ok = sm.ok;
  int32_t* idx = P.top_idx + (int64_t)r * P.n_top;
  float* lp = P.top_logp + (int64_t)r * P.n_top;
  const float unused = ok ? -INFINITY : __uint_as_float(0x7FC00000u);
  if (!ok) count = 0;
  for (int i = count + t; i < P.n_top; i += T) {
    idx[i] = -1;
    lp[i] = unused;
  }
  // Key and id as one number, larger for an earlier one; each is held by a lane and compared with all (key and id by themselves, two
  // conditions and a branch each, for one of a lane's at a time: 64 x 151936, n = 64, row step 17.2 us against 9.7).
  constexpr int kOwn = (kCapMax + T - 1) / T, kStep = 8;
  auto order = [](uint2 c) { return (uint64_t)c.x << 32 | (uint32_t)~c.y; };
  uint64_t mine[kOwn];
  int above[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int at = T * i + t;
    mine[i] = at < count ? order(sm.list[at]) : 0u;
    above[i] = 0;
  }
  for (int j = 0; j < count; j += kStep) {
    uint64_t o[kStep];
#pragma unroll
    for (int e = 0; e < kStep; ++e) o[e] = order(sm.list[min(j + e, count - 1)]);
#pragma unroll
    for (int e = 0; e < kStep; ++e) {
      if (j + e >= count) o[e] = 0u;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) above[i] += o[e] > mine[i] ? 1 : 0;
    }
  }
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    if (T * i + t >= count || above[i] >= P.n_top) continue;
    idx[above[i]] = (int32_t)~(uint32_t)mine[i];
    const float v = (float)(((double)key2f((uint32_t)(mine[i] >> 32)) - (double)sm.m) * sm.c2 * kLn2 - sm.log_s);
    lp[above[i]] = ok == 2 ? (above[i] == 0 ? 0.0f : -INFINITY) : fminf(v, 0.0f);
  }
}

// A tile's sum of 2^z without its one largest logit, by one wave: where that term, 1, is nearly all of S, log S lives in
// what the others add, which the fp32 sum of the thread that holds it has rounded away. That thread's other logits are
// read again. (Sums below 1.5 have one largest logit.)
template <int DT, class E>
__device__ __forceinline__ double sum_beside_top(const LSmem& sm, const char* row, int V, int tile, const uint32_t* k4, uint32_t k,
                                                 float m, E exponent) {
  using L = Logits<DT>;
  int top = 0;
#pragma unroll
  for (int i = kLW - 1; i >= 0; --i) {
    const uint64_t at = __ballot(k4[i] == k);
    if (at) top = 64 * i + __ffsll((unsigned long long)at) - 1;
  }
  const int e = lane() & (kLE - 1), j = e % L::kW;
  const Place<DT> pl(tile, top, e / L::kW, V);
  const bool counts = lane() < kLE && pl.counts(j, V);
  const float x = counts ? load_logit<DT>(row, pl.at + j) : m;
  double s = x == m ? 0.0 : (double)__builtin_amdgcn_exp2f(exponent(x));
#pragma unroll
  for (int i = 0; i < kLW; ++i) s += 64 * i + lane() == top ? 0.0 : (double)sm.sums[64 * i + lane()].x;
  return wave_sum_f64(s);
}

// The exponent of a term is z = fma(x, c, -fl(m c)), c = log2(e) / T: one operation and one rounding, and off by the
// same eta = m c - fl(m c) in every term, which is known exactly (an fma) and taken out of the sums at the end. Where
// |m c| is so large that 2^-eta needs more than the terms taken below, z is (x - m) c.
//
// What bounds it: the vector unit, for 16-bit logits (an unpacking, half a maximum, fma, exp2 at a quarter of the rate,
// add and fma a logit: 183 instructions for a lane's 32, and about 110 beside them; 64 logits a lane took no
// less time, as fewer waves then hide the loads); HBM for fp32 ones (1024 x 151936: 108 us, a read 92 us). So what can be done
// once a workgroup is done by one wave, a different one in neighbouring workgroups: the last steps of the sums and the
// search of the candidates' bound.
template <int DT, bool TOP, bool WHOLE>
__global__ __launch_bounds__(kLT) __attribute__((amdgpu_waves_per_eu(7))) void ts_logp_tile_kernel(LParams P) {
  __shared__ LSmem sm;
  int r, tile;
  if (WHOLE) r = (int)blockIdx.x, tile = 0;
  else place_block(P.tiles, r, tile);
  const int t = (int)threadIdx.x, w = __builtin_amdgcn_readfirstlane(wave());
  const bool lead = w == (int)(blockIdx.x % kLW);
  const char* row = P.x + (int64_t)r * P.stride;
  // The given token's logit is asked for right behind the tile's, so that its wait is hidden behind theirs (1777 x 128256
  // in bf16: about 95 us with ranks, 99 us where it was loaded after the tile had come, 83 us without ranks).
  const RowIn in = row_in(P, r);
  Tile<DT> raw;
  raw.load(row, P.V, tile, t);
  const bool ranks = P.tokens && in.token >= 0 && (P.rank || in.t == 0.0f);
  const float xt = ranks ? load_logit<DT>(row, in.token) : 0.0f;
  float xs[kLE];
  raw.values(row, P.V, tile, t, xs);
  float tm = max_of<kLE>(xs);
  if (tm != tm) tm = INFINITY;
  sm.tk[t] = f2key(tm);
  bar();

  uint32_t k4[kLW], k = 0;
#pragma unroll
  for (int i = 0; i < kLW; ++i) {
    k4[i] = sm.tk[64 * i + lane()];
    k = max(k, k4[i]);
  }
  k = wave_max(k);
  const uint32_t low = TOP && lead ? find_low<DT>(k4, k, P.n_top) : 0u;
  const float m = k == kKeyNegInf ? 0.0f : key2f(k);
  const float c = scale32(P, in.t), mc = m * c;
  const bool fused = fabsf(mc) <= 4096.0f;                       // eta below 2^-12
  {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    // The exponent's lower bound is left out at first, where nothing is known to need it: a masked logit's 0 * -inf shows
    // in the products (as a NaN does, which S tells). The unused places of the row's last tile are -inf.
    bool careful = (tile + 1) * kTile > P.V || !fused;
    if (!careful) {
#pragma unroll
      for (int i = 0; i < kLE; ++i) {
        const float z = fmaf(xs[i], c, -mc);
        const float e = __builtin_amdgcn_exp2f(z);
        s[i & 3] += e;
        d[i & 3] = fmaf(e, z, d[i & 3]);
      }
      const float dd = (d[0] + d[1]) + (d[2] + d[3]);
      careful = __ballot(dd != dd) != 0;
    }
    if (careful) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = d[i] = 0.0f;
      auto sums = [&](auto exponent) {
#pragma unroll
        for (int i = 0; i < kLE; ++i) {
          float x = xs[i];
          asm volatile("" : "+v"(x));   // computed anew: the first sums' values are not kept for these
          const float z = fmaxf(exponent(x), kZMin);
          const float e = __builtin_amdgcn_exp2f(z);
          s[i & 3] += e;
          d[i & 3] = fmaf(e, z, d[i & 3]);
        }
      };
      if (fused) sums([&](float x) { return fmaf(x, c, -mc); });
      else sums([&](float x) { return (x - m) * c; });
    }
    sm.sums[t] = make_float2((s[0] + s[1]) + (s[2] + s[3]), (d[0] + d[1]) + (d[2] + d[3]));
  }
  const uint32_t ahead = ranks ? wave_above<DT>(P, in, tile, xs, k, xt) : 0u;
  if (lane() == 0) sm.redn[w] = ahead;
  bar();

  if (w == (int)((blockIdx.x + 1) % kLW)) {
    double s = 0.0, d = 0.0;
    uint32_t above = 0;
#pragma unroll
    for (int i = 0; i < kLW; ++i) {
      const float2 q = sm.sums[64 * i + lane()];
      s += (double)q.x;
      d += (double)q.y;
      above += sm.redn[i];
    }
    s = wave_sum_f64(s);
    d = wave_sum_f64(d);
    double scale = 1.0;
    if (fused) {
      const double eta = (double)fmaf(m, c, -mc), y = eta * kLn2;
      scale = 1.0 + y * (-1.0 + y * (0.5 - y * (1.0 / 6.0)));   // 2^-eta, within 1e-15 of it
      s *= scale;
      d = d * scale - eta * s;
    }
    if (s < 1.5 && k != kKeyNegInf)
      s = 1.0 + scale * sum_beside_top<DT>(sm, row, P.V, tile, k4, k, m, [&](float x) { return fused ? fmaf(x, c, -mc) : (x - m) * c; });
    Part* out = WHOLE ? &sm.part : P.part + ((int64_t)r * P.tiles + tile);
    if (lane() == 0) {
      out->s = s;
      out->d = d;
      out->m = key2f(k);
      out->above = above;
    }
    if (WHOLE) {
      wave_lds_sync();
      finish_row<DT>(P, in, r, &sm.part, &sm);
    }
  }
  if (!TOP) return;
  if (lead) {
    const int count = tile_candidates<DT>(sm, row, P.V, tile, P.n_top, P.cap, low, k, k4);
    if (WHOLE) {
      sm.count = (uint32_t)count;
    } else {
      uint2* out = P.cand + ((int64_t)r * P.tiles + tile) * P.cap;
      for (int i = lane(); i < P.cap; i += 64) out[i] = i < count ? sm.list[i] : make_uint2(0u, 0u);
    }
  }
  if (WHOLE) {
    bar();
    write_top<kLT>(P, r, (int)sm.count, sm);
  }
}

// One row a wave.
template <int DT>
__global__ __launch_bounds__(kLT) void ts_logp_row_kernel(LParams P) {
  const int r = (int)(blockIdx.x * kLW + wave());
  if (r < P.rows) finish_row<DT>(P, row_in(P, r), r, P.part + (int64_t)r * P.tiles, nullptr);
}

// The best n of slots begin, begin + 1, ... of n_slots (key and id; 0: none) by one wave, into `list`, in no order: kBatch slots at
// a time, every `step`, 24 a lane (four groups of six: find_low's 256 groups), and what is left of the ones before.
constexpr int kGroup = 6, kItems = 4 * kGroup, kBatch = 64 * kItems;
template <int DT, class I>
__device__ __forceinline__ int best_of(const LParams& P, uint2* list, I item, int64_t begin, int64_t n_slots, int64_t step) {
  constexpr int kLeft = (kCapMax + 63) / 64;
  const int l = lane();
  int count = 0;
  for (int64_t base = begin; base < n_slots; base += step) {
    uint2 c[kItems + kLeft];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int64_t at = base + 64 * i + l;
      c[i] = at < n_slots ? item(at) : make_uint2(0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kLeft; ++i) c[kItems + i] = 64 * i + l < count ? list[64 * i + l] : make_uint2(0u, 0u);
    wave_lds_sync();
    uint32_t k4[4], k = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      k4[g] = g < kLeft ? c[kItems + g].x : 0u;
#pragma unroll
      for (int i = 0; i < kGroup; ++i) k4[g] = max(k4[g], c[4 * i + g].x);   // a few slots fall into as many groups
      k = max(k, k4[g]);
    }
    k = wave_max(k);
    const uint32_t low = find_low<DT>(k4, k, P.n_top);
    count = 0;
#pragma unroll
    for (int i = 0; i < kItems + kLeft; ++i) {
      const uint64_t m = __ballot(c[i].x >= low);
      if (!m) continue;
      const int o = count + (int)mbcnt(m);
      if (c[i].x >= low && o < kCapMax) list[o] = c[i];
      count += __popcll(m);
    }
    if (count > P.cap) {
      exact_items<kItems + kLeft>(list, c, P.n_top, low, k, P.V);
      count = P.n_top;
    }
    wave_lds_sync();
  }
  return count;
}

// One row a workgroup of F + 1 waves: one joins the tiles, the others find the best n of the candidates meanwhile, F shares of
// their batches, whose best one of them joins.
constexpr int kFinders = 7;   // kFinders x kCapMax slots are one batch
static_assert(kFinders * kCapMax <= kBatch, "the shares' best are one batch");
template <int DT, int F>
__global__ __launch_bounds__(64 * (F + 1)) void ts_logp_top_kernel(LParams P) {
  __shared__ LSmem sm;
  __shared__ uint2 shares[F > 1 ? F : 1][kCapMax];
  __shared__ int counts[F];
  const int r = (int)blockIdx.x, w = __builtin_amdgcn_readfirstlane(wave());
  const uint2* cand = P.cand + (int64_t)r * P.tiles * P.cap;
  const int64_t n = (int64_t)P.tiles * P.cap;
  if (w == 0) {
    finish_row<DT>(P, row_in(P, r), r, P.part + (int64_t)r * P.tiles, &sm);
  } else {
    const int count = best_of<DT>(P, F > 1 ? shares[w - 1] : sm.list, [&](int64_t at) { return cand[at]; }, (int64_t)(w - 1) * kBatch, n,
                                  (int64_t)F * kBatch);
    if (lane() == 0) {
      if (F > 1) counts[w - 1] = count;
      else sm.count = (uint32_t)count;
    }
  }
  bar();
  if (F > 1) {
    if (w == 1) {
      const int count = best_of<DT>(
          P, sm.list,
          [&](int64_t at) {
            const int f = (int)at / kCapMax, i = (int)at - f * kCapMax;
            return i < counts[f] ? shares[f][i] : make_uint2(0u, 0u);
          },
          0, F * kCapMax, kBatch);
      if (lane() == 0) sm.count = (uint32_t)count;
    }
    bar();
  }
  write_top<64 * (F + 1)>(P, r, (int)sm.count, sm);
}

// ------------------------------------------------------------------ gradient
struct GParams {
  const char* x;
  char* g;
  int64_t x_stride, g_stride;   // bytes
  int32_t V, rows, tiles;
  const int32_t* tokens;
  const float* t;
  const float4* stats;
  const float* g_logp;
  const float* g_entropy;
  const float* g_lse;
};

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == TS_DTYPE_BF16) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, bf2));   // round to nearest even
  } else {
    // whole fp32 numbers first: some of the products would else be rounded to fp16 with their last operation, others after it
    asm("" : "+v"(a), "+v"(b));
    return (uint32_t)__half_as_ushort(__float2half_rn(a)) | ((uint32_t)__half_as_ushort(__float2half_rn(b)) << 16);
  }
}
template <int DT>
__device__ __forceinline__ void store_logit(char* row, int64_t i, float v) {
  if constexpr (DT == TS_DTYPE_F32) reinterpret_cast<float*>(row)[i] = v;
  else reinterpret_cast<unsigned short*>(row)[i] = (unsigned short)pack2<DT>(v, 0.0f);
}

// Bound by HBM: bytes read and written. ONCE, for logits and gradient that do not fit the last-level cache together: loads
// and stores past the caches (2048 x 151936 bf16: 187 us against 209; 301 x 65537 fp32, which fits: 26 us against 25).
// Each element is read and then written by one thread and read by no other, so the gradient may take the
// logits' own place. (A row's last vector, where it is not whole, is taken element by element for that.)
template <int DT, bool ONCE>
__global__ __launch_bounds__(kLT) __attribute__((amdgpu_waves_per_eu(8))) void ts_logp_grad_kernel(GParams P) {
  using L = Logits<DT>;
  int r, tile;
  place_block(P.tiles, r, tile);
  const char* row = P.x + (int64_t)r * P.x_stride;
  char* out = P.g + (int64_t)r * P.g_stride;
  const int t0 = tile * kTile + (int)threadIdx.x * L::kW;
  u32x4 raw[L::kNV];
#pragma unroll
  for (int v = 0; v < L::kNV; ++v) {
    const int at = t0 + v * kLT * L::kW;
    if (at + L::kW <= P.V) raw[v] = ONCE ? load16_once(row + (int64_t)at * L::kSize) : load16(row + (int64_t)at * L::kSize);
  }
  const float4 st = P.stats[r];
  const float temp = P.t ? P.t[r] : 1.0f;
  const int32_t token = P.tokens ? P.tokens[r] : -1;
  float a = P.g_logp ? P.g_logp[r] : 0.0f;
  float h = P.g_entropy ? P.g_entropy[r] : 0.0f;
  float l = P.g_lse ? P.g_lse[r] : 0.0f;
  const bool ok = st.x == st.x && temp >= 0.0f && temp <= 3.402823466e38f && token >= -1 && token < P.V;
  if (token < 0) a = 0.0f;
  // A large T and the gradients are both taken by 2^-64, where 1 / (T S) could lie below the normal numbers and lose its bits.
  const float by = temp > 0x1p64f ? 0x1p-64f : 1.0f;
  a *= by;
  h *= by;
  l *= by;
  const float inv_t = temp > 0.0f ? 1.0f / fmaxf(temp * by, 0x1p-100f) : 0.0f;   // greedy rows do not depend on the logits
  const float c2 = (float)(2.0 * exponent_scale(temp));
  // p (l - a - h (d - D)) / T = 2^z (k0 + k1 z)
  const float q = inv_t / st.y;
  float k0 = q * (l - a + h * st.z), k1 = -q * h * (float)kLn2;
  const float add = a * inv_t, m = st.x, half_m = 0.5f * m;
  if (!ok) k0 = k1 = __uint_as_float(0x7FC00000u);
  const bool here = token >= 0 && token / kTile == tile;   // the tile holds the token
  // Where the given token is the maximum and nearly all of S, fp32 loses a / T - p a / T: its part of a is a (1 - p) / T then, by
  // the forward call's 1 - 1/S. (Not where l makes up for a: then the sum is not small, and the usual one the closer.)
  const bool sharp = here && ok && st.w < 0.25f && fabsf(l - a + h * st.z) >= 0.5f * fabsf(a);
  const float top = fmaf(q, fmaf(h, st.z, l), a * (st.w * inv_t));
  auto grad = [&](float x) -> float {
    // half the distance: at a large T one beyond the largest number counts. Rounded once, as x - m elsewhere
    const float z = fmaxf(fmaf(x, 0.5f, -half_m) * c2, kZMin);
    return __builtin_amdgcn_exp2f(z) * fmaf(k1, z, k0);
  };
  auto token_grad = [&](float x, float g) -> float { return sharp && x == m ? top : g + add; };
  // A tile without the token, as most are, has no choice to make at its logits (64 of 525 instructions a wave). Past the caches,
  // where it is whole, its vectors have none either: each one's wait would be for the stores of those before it too (2048 x 151936
  // bf16, the call: 294 us against 299; in the caches the stores then come too close: 300 x 65536 fp32 51.7 us against 49.8).
  auto vectors = [&](auto plain) {
#pragma unroll
    for (int v = 0; v < L::kNV; ++v) {
      const int at = t0 + v * kLT * L::kW;
      if ((ONCE && plain()) || at + L::kW <= P.V) {
        float g[L::kW];
#pragma unroll
        for (int j = 0; j < L::kW; ++j) {
          const float x = unpack<DT>(raw[v], j);
          g[j] = grad(x);
          if (!plain() && here && at + j == token) g[j] = token_grad(x, g[j]);
        }
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (DT == TS_DTYPE_F32) o[j] = __float_as_uint(g[j]);
          else o[j] = pack2<DT>(g[2 * j], g[2 * j + 1]);
        }
        if (ONCE) store16_once(out + (int64_t)at * L::kSize, o);
        else store16(out + (int64_t)at * L::kSize, o);
      }
    }
  };
  if (!here && (!ONCE || (tile + 1) * kTile <= P.V)) vectors(std::true_type{});
  else vectors(std::false_type{});
  // the row's last, partial vector
  const int tail = P.V / L::kW * L::kW, off = tail - t0;
  if (tail < P.V && off >= 0 && off < kTile && off % (kLT * L::kW) == 0) {
#pragma nounroll
    for (int j = tail; j < P.V; ++j) {
      const float x = load_logit<DT>(row, j), g = grad(x);
      store_logit<DT>(out, j, j == token ? token_grad(x, g) : g);
    }
  }
}

// ------------------------------------------------------------------ host side
struct LPlan {
  int64_t tiles = 0;
  int cap = 0;
  size_t off_cand = 0, total = 0;
};
// Whether one launch, of at most 2^32 - 1 threads, holds the rows' tiles. (Divided: any number of rows is asked for, and a
// product could wrap to a small one.)
bool rows_fit(int64_t rows, int64_t V) { return rows <= (int64_t)0xFFFFFFFF / kLT / ((V + kTile - 1) / kTile); }
bool logp_plan(int64_t rows, int64_t V, int n_top, LPlan& pl) {
  if (rows < 0 || V < 1 || V > TS_MAX_VOCAB || n_top < 0 || n_top > TS_LOGP_TOP_MAX || !rows_fit(rows, V)) return false;
  pl.tiles = (V + kTile - 1) / kTile;
  pl.cap = cand_cap(n_top);
  if (pl.tiles == 1) {
    pl.total = 256;
    return true;
  }
  const size_t parts = (size_t)(std::max<int64_t>(rows, 1) * pl.tiles);
  pl.off_cand = (parts * sizeof(Part) + 255) & ~(size_t)255;
  pl.total = pl.off_cand + ((parts * pl.cap * sizeof(uint2) + 255) & ~(size_t)255);
  return true;
}

template <int DT>
hipError_t launch_logp(const LParams& P, hipStream_t s) {
  const dim3 tiles((unsigned)((int64_t)P.rows * P.tiles)), block(kLT);
  const bool top = P.n_top > 0;
  if (P.tiles == 1) {
    if (top) hipLaunchKernelGGL((ts_logp_tile_kernel<DT, true, true>), tiles, block, 0, s, P);
    else hipLaunchKernelGGL((ts_logp_tile_kernel<DT, false, true>), tiles, block, 0, s, P);
    return hipGetLastError();
  }
  if (top) hipLaunchKernelGGL((ts_logp_tile_kernel<DT, true, false>), tiles, block, 0, s, P);
  else hipLaunchKernelGGL((ts_logp_tile_kernel<DT, false, false>), tiles, block, 0, s, P);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Several finders from the third batch of candidates on (64 x 151936, n = 64, two batches: row step 11.0 us against 9.8; 64 x
  // 262144, n = 64, four: the call 30 us against 34; 1 x 4000000, n = 20: 26 against 63).
  if (top && (int64_t)P.tiles * P.cap > 2 * kBatch)
    hipLaunchKernelGGL((ts_logp_top_kernel<DT, kFinders>), dim3((unsigned)P.rows), dim3(64 * (kFinders + 1)), 0, s, P);
  else if (top)
    hipLaunchKernelGGL((ts_logp_top_kernel<DT, 1>), dim3((unsigned)P.rows), dim3(128), 0, s, P);
  else hipLaunchKernelGGL((ts_logp_row_kernel<DT>), dim3((unsigned)((P.rows + kLW - 1) / kLW)), block, 0, s, P);
  return hipGetLastError();
}

constexpr int64_t kCacheBytes = 256 << 20;   // the last-level cache

int dtype_size(int dtype) {
  return dtype == TS_DTYPE_F32 ? 4 : (dtype == TS_DTYPE_BF16 || dtype == TS_DTYPE_F16) ? 2 : 0;
}

// Rows a stride apart end within 2^60 elements, so that their addresses' arithmetic does not wrap.
bool stride_fits(int64_t rows, int64_t stride) { return stride <= ((int64_t)1 << 60) / std::max<int64_t>(rows, 1); }

// The checks that both entry points share; TS_OK also for an empty batch.
int check_logits(const void* x, int dtype, int64_t rows, int64_t vocab, int64_t stride) {
  if (rows < 0) return fail(TS_ERR_INVALID_ARG, "rows = %lld < 0", (long long)rows);
  if (vocab < 1 || vocab > TS_MAX_VOCAB) return fail(TS_ERR_INVALID_ARG, "vocab = %lld outside [1, 2^30]", (long long)vocab);
  if (stride < vocab) return fail(TS_ERR_INVALID_ARG, "row_stride %lld < vocab %lld", (long long)stride, (long long)vocab);
  if (!dtype_size(dtype)) return fail(TS_ERR_INVALID_ARG, "dtype = %d is none of TS_DTYPE_*", dtype);
  if (rows == 0) return TS_OK;
  if (!x) return fail(TS_ERR_INVALID_ARG, "logits pointer is NULL");
  if ((uintptr_t)x % dtype_size(dtype)) return fail(TS_ERR_INVALID_ARG, "logits are not aligned to their type");
  if (!rows_fit(rows, vocab)) return fail(TS_ERR_INVALID_ARG, "rows x tiles too large");
  if (!stride_fits(rows, stride)) return fail(TS_ERR_INVALID_ARG, "rows x row_stride too large");
  return TS_OK;
}

}  // namespace

namespace tsh {
size_t token_logp_workspace(int64_t rows, int64_t vocab, int n_top) {
  LPlan pl;
  return logp_plan(rows, vocab, n_top, pl) ? pl.total : 0;
}
}  // namespace tsh

extern "C" {

int ts_token_logp(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride, const int32_t* tokens,
                  const float* temperature, int32_t n_top, float* out_logp, int32_t* out_rank, float* out_entropy,
                  float* out_lse, int32_t* out_top_idx, float* out_top_logp, float* out_stats, int32_t* row_status,
                  void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_logits(logits, dtype, rows, vocab, row_stride);
  if (rc != TS_OK) return rc;
  if (n_top < 0 || n_top > TS_LOGP_TOP_MAX)
    return fail(TS_ERR_INVALID_ARG, "n_top = %d outside [0, %d]", (int)n_top, TS_LOGP_TOP_MAX);
  if (rows == 0) return TS_OK;
  if (!tokens && (out_logp || out_rank)) return fail(TS_ERR_INVALID_ARG, "out_logp and out_rank need tokens");
  if (n_top > 0 && (!out_top_idx || !out_top_logp))
    return fail(TS_ERR_INVALID_ARG, "n_top > 0 needs out_top_idx and out_top_logp");
  if (((uintptr_t)out_stats & 15u) != 0) return fail(TS_ERR_INVALID_ARG, "out_stats is not 16-byte aligned");
  LPlan pl;
  logp_plan(rows, vocab, n_top, pl);   // (of sizes that the checks above have let through)
  if (pl.tiles > 1) {
    if (!workspace) return fail(TS_ERR_WORKSPACE, "workspace is NULL");
    if (((uintptr_t)workspace & 255u) != 0) return fail(TS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    if (workspace_bytes < pl.total)
      return fail(TS_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, pl.total);
  }
  int dev;
  rc = check_device(&dev);
  if (rc != TS_OK) return rc;
  LParams P;
  P.x = static_cast<const char*>(logits);
  P.stride = row_stride * dtype_size(dtype);
  P.V = (int32_t)vocab;
  P.rows = (int32_t)rows;
  P.tiles = (int32_t)pl.tiles;
  P.n_top = n_top;
  P.cap = pl.cap;
  P.tokens = tokens;
  P.t = temperature;
  P.logp = out_logp;
  P.rank = out_rank;
  P.entropy = out_entropy;
  P.lse = out_lse;
  P.top_idx = out_top_idx;
  P.top_logp = out_top_logp;
  P.stats = reinterpret_cast<float4*>(out_stats);
  P.status = row_status;
  P.part = static_cast<Part*>(workspace);
  P.cand = reinterpret_cast<uint2*>(static_cast<char*>(workspace) + pl.off_cand);
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == TS_DTYPE_F32    ? launch_logp<TS_DTYPE_F32>(P, s)
                       : dtype == TS_DTYPE_BF16 ? launch_logp<TS_DTYPE_BF16>(P, s)
                                                : launch_logp<TS_DTYPE_F16>(P, s);
  if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "token logprob launch failed: %s", hipGetErrorString(e));
  return TS_OK;
}

int ts_token_logp_backward(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                           const int32_t* tokens, const float* temperature, const float* stats, const float* grad_logp,
                           const float* grad_entropy, const float* grad_lse, void* grad_logits, int64_t grad_stride,
                           void* stream) {
  int rc = check_logits(logits, dtype, rows, vocab, row_stride);
  if (rc != TS_OK) return rc;
  if (grad_stride < vocab)
    return fail(TS_ERR_INVALID_ARG, "grad_stride %lld < vocab %lld", (long long)grad_stride, (long long)vocab);
  if (rows == 0) return TS_OK;
  if (!stats || !grad_logits) return fail(TS_ERR_INVALID_ARG, "stats and grad_logits are required");
  if (grad_logp && !tokens) return fail(TS_ERR_INVALID_ARG, "grad_logp needs tokens");
  if (((uintptr_t)stats & 15u) != 0) return fail(TS_ERR_INVALID_ARG, "stats is not 16-byte aligned");
  const int size = dtype_size(dtype);
  if ((uintptr_t)grad_logits % size) return fail(TS_ERR_INVALID_ARG, "grad_logits are not aligned to their type");
  if (!stride_fits(rows, grad_stride)) return fail(TS_ERR_INVALID_ARG, "rows x grad_stride too large");
  // The gradient may take the logits' place exactly; otherwise no element may be shared. Rows equally far apart may lie between
  // each other: `by` bytes behind the start of one's row, the other's has to fit between its end and the next one's start.
  const uint64_t width = (uint64_t)vocab * size, step = (uint64_t)row_stride * size;
  const uintptr_t x0 = (uintptr_t)logits, x1 = x0 + (uint64_t)(rows - 1) * step + width;
  const uintptr_t g0 = (uintptr_t)grad_logits, g1 = g0 + (uint64_t)(rows - 1) * grad_stride * size + width;
  if (g0 < x1 && x0 < g1 && !(g0 == x0 && grad_stride == row_stride)) {
    const uint64_t by = g0 >= x0 ? (g0 - x0) % step : step - 1 - (x0 - g0 - 1) % step;
    if (grad_stride != row_stride || by < width || by > step - width)
      return fail(TS_ERR_INVALID_ARG, "grad_logits overlap the logits without taking their place");
  }
  const int64_t tiles = (vocab + kTile - 1) / kTile;
  int dev;
  rc = check_device(&dev);
  if (rc != TS_OK) return rc;
  GParams P;
  P.x = static_cast<const char*>(logits);
  P.g = static_cast<char*>(grad_logits);
  P.x_stride = row_stride * size;
  P.g_stride = grad_stride * size;
  P.V = (int32_t)vocab;
  P.rows = (int32_t)rows;
  P.tiles = (int32_t)tiles;
  P.tokens = tokens;
  P.t = temperature;
  P.stats = reinterpret_cast<const float4*>(stats);
  P.g_logp = grad_logp;
  P.g_entropy = grad_entropy;
  P.g_lse = grad_lse;
  const bool once = 2 * rows * vocab * size > kCacheBytes;
  const dim3 grid((unsigned)(rows * tiles)), block(kLT);
  const hipStream_t s = (hipStream_t)stream;
  auto launch = [&](auto dt) {
    if (once) hipLaunchKernelGGL((ts_logp_grad_kernel<dt(), true>), grid, block, 0, s, P);
    else hipLaunchKernelGGL((ts_logp_grad_kernel<dt(), false>), grid, block, 0, s, P);
  };
  if (dtype == TS_DTYPE_F32) launch(std::integral_constant<int, TS_DTYPE_F32>{});
  else if (dtype == TS_DTYPE_BF16) launch(std::integral_constant<int, TS_DTYPE_BF16>{});
  else launch(std::integral_constant<int, TS_DTYPE_F16>{});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TS_ERR_LAUNCH, "token logprob gradient launch failed: %s", hipGetErrorString(e));
  return TS_OK;
}

}  // extern "C"
