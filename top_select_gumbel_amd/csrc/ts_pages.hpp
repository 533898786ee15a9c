// ts_pages.hpp -- what the kernels of paged caches share: division by the page size and the host's checks of layouts.
#pragma once
#include <algorithm>
#include <initializer_list>
#include <utility>

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "topselect.h"
#include "ts_host.hpp"

namespace tsp {

constexpr int64_t kMaxLen = 0x7FFFFF00;      // positions of a sequence: tiles past the last one stay in 31 bits
constexpr int64_t kMaxPages = 0x7FFFFFFF;

// j / d for j < 2^31 by a product: with 2^(l-1) < d <= 2^l and mul = ceil(2^(31+l) / d) < 2^32 the product exceeds the
// quotient's by less than j 2^l / 2^(31+l) < 1 of the next multiple.
struct Divisor {
  uint32_t mul;
  int32_t shift;
  Divisor() = default;
  explicit Divisor(int32_t d) {
    int l = 0;
    while (((int64_t)1 << l) < d) ++l;
    mul = (uint32_t)((((uint64_t)1 << (31 + l)) + (uint64_t)d - 1) / (uint64_t)d);
    shift = 31 + l;
  }
  __host__ __device__ uint32_t of(uint32_t j) const { return (uint32_t)(((uint64_t)j * mul) >> shift); }
};

typedef std::initializer_list<std::pair<int64_t, int64_t>> Strides;   // (stride, count)

// Whether every element of `inner` consecutive ones at these strides (none negative) lies within 2^62 bytes.
inline bool reaches(int64_t inner, Strides strides, int64_t size) {
  __int128 end = inner;
  for (auto [stride, n] : strides) {
    if (stride < 0 && n > 1) return false;
    if (n > 1) end += (__int128)stride * (n - 1);
  }
  return end * size <= (__int128)1 << 62;
}
// ... and whether no two of them share memory: along the ascending strides each clears what lies below it.
inline bool apart(int64_t inner, Strides strides, int64_t size) {
  if (!reaches(inner, strides, size)) return false;
  int64_t end = inner, last = 0;
  int given = 0;   // the strides up to `last`, in the order that they are given, have been taken
  for (size_t taken = 0; taken < strides.size(); ++taken) {
    // the smallest of those that are left
    const std::pair<int64_t, int64_t>* next = nullptr;
    int at = 0, of = 0;
    for (const auto& s : strides) {
      const bool done = taken > 0 && (s.first < last || (s.first == last && at < given));
      if (!done && (!next || s.first < next->first)) {
        next = &s;
        of = at;
      }
      ++at;
    }
    last = next->first;
    given = of + 1;
    if (next->second <= 1) continue;
    if (next->first < end) return false;
    end += next->first * (next->second - 1);
  }
  return true;
}

// Rows of `bytes` bytes at `at` + i * stride[0] + j * stride[1], i < count[0], j < count[1] (bytes; within 2^62, as `reaches` has it).
struct Rows {
  uintptr_t at;
  int64_t bytes, stride[2], count[2];
  int64_t step(int d) const { return count[d] > 1 ? stride[d] : 0; }
  // Rows that follow each other without a gap are one.
  Rows joined() const {
    Rows r = *this;
    for (int d : {1, 0})
      if (r.step(d) == r.bytes) {
        r.bytes *= r.count[d];
        r.count[d] = 1;
      }
    return r;
  }
  uintptr_t end() const { return at + (uintptr_t)(step(0) * (count[0] - 1) + step(1) * (count[1] - 1) + bytes); }
};
// Whether a row of a shares memory with a row of b, whose rows are `apart`. Of two arrays that lie between each other's rows each row of
// a is looked up among b's (64 x 32 rows 17 us of the host, 64 of 32 joined heads below 1): those begin at places that grow with the
// wider stride's index, then with the other's.
inline bool meet(const Rows& rows_a, const Rows& rows_b) {
  const Rows a = rows_a.joined(), b = rows_b.joined();
  if (a.at >= b.end() || b.at >= a.end()) return false;
  const int wide = b.step(0) >= b.step(1) ? 0 : 1;
  auto last_below = [](int64_t x, int64_t step, int64_t count) {   // the last index whose place lies below x > 0
    return step ? std::min((x - 1) / step, count - 1) : 0;
  };
  const int64_t n0 = a.step(0) ? a.count[0] : 1, n1 = a.step(1) ? a.count[1] : 1;
  for (int64_t i = 0; i < n0; ++i)
    for (int64_t j = 0; j < n1; ++j) {
      const int64_t from = (int64_t)(a.at - b.at) + i * a.stride[0] + j * a.stride[1];   // the row's place, counted from b's first
      if (from + a.bytes <= 0) continue;
      // b's last row that begins below this one's end; under the wide index before it, too, a row may reach into this one
      const int64_t w = last_below(from + a.bytes, b.step(wide), b.count[wide]);
      for (int64_t x = std::max<int64_t>(0, w - 1); x <= w; ++x) {
        const int64_t left = from + a.bytes - x * b.step(wide);
        if (x * b.step(wide) + last_below(left, b.step(1 - wide), b.count[1 - wide]) * b.step(1 - wide) + b.bytes > from) return true;
      }
    }
  return false;
}

inline int check_table(int64_t pages, int64_t page_slots, int64_t table_width, int64_t table_stride) {
  if (pages < 0 || pages > kMaxPages) return tsh::fail(TS_ERR_INVALID_ARG, "pages = %lld outside [0, 2^31)", (long long)pages);
  if (page_slots < 1 || page_slots > 1 << 30)
    return tsh::fail(TS_ERR_INVALID_ARG, "page_slots = %lld outside [1, 2^30]", (long long)page_slots);
  if (table_width < 0 || table_width > kMaxLen)
    return tsh::fail(TS_ERR_INVALID_ARG, "table_width = %lld is negative or too large", (long long)table_width);
  if (table_stride < table_width || table_stride > (int64_t)1 << 40)
    return tsh::fail(TS_ERR_INVALID_ARG, "table_stride %lld < table_width %lld, or too large", (long long)table_stride,
                     (long long)table_width);
  return TS_OK;
}

}  // namespace tsp
