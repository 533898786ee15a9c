// ts_logits.hpp -- 16-byte loads of logits in fp32, bf16 or fp16 as fp32 values, by tiles of a row.
//
// A row is cut into tiles of kTile logits, whatever its type and wherever the batch puts it, so that
// every sum over a tile has the same terms in the same order in every call. A tile belongs to kLT
// threads; thread t holds the 16-byte vectors t, t + kLT, ... of it, kLE logits in all. Rows
// start at any multiple of their element's size: gfx950 loads and stores 16 bytes from any address, so
// the vectors are counted from the row's first logit and not from an aligned address.
#pragma once
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "topselect.h"
#include "ts_device.hpp"

namespace tsl {

constexpr int kLT = 256;          // threads a tile
constexpr int kLE = 32;           // logits a thread
constexpr int kTile = kLT * kLE;  // 8192

// A workgroup's row and tile in a grid of rows x tiles. Workgroups go to the eight XCDs, and to their compute units, in
// turn; each row starts at another tile, so that tiles of one place in their rows, which cost another time than others
// (a row's last logits, the unused slots of a cache), do not all fall to the same ones. (Logits, 1777 rows of 16 tiles in
// bf16: 112 us without it, the last tiles all on one XCD, where rows of 16 whole tiles took 85 us.)
__device__ __forceinline__ void place_block(int32_t tiles, int& r, int& tile) {
  const unsigned b = blockIdx.x, n = (unsigned)tiles;
  r = (int)(b / n);
  const unsigned i = b - (unsigned)r * n + (unsigned)r % n;
  tile = (int)(i >= n ? i - n : i);
}

template <int DT>
struct Logits {
  static constexpr uint32_t kNegInf = DT == TS_DTYPE_F32 ? 0xFF800000u : DT == TS_DTYPE_BF16 ? 0xFF80FF80u : 0xFC00FC00u;   // a word of -inf
  static constexpr int kSize = DT == TS_DTYPE_F32 ? 4 : 2;
  static constexpr int kW = 16 / kSize;     // logits a vector
  static constexpr int kLowBits = DT == TS_DTYPE_F32 ? 0 : DT == TS_DTYPE_BF16 ? 16 : 13;   // fraction bits that fp32 has more
  static constexpr int kNV = kLE / kW;      // vectors a thread
};

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));   // 16 bytes at any logit's address

__device__ __forceinline__ u32x4 load16(const char* p) { return *reinterpret_cast<const u32x4_any*>(p); }
__device__ __forceinline__ void store16(char* p, u32x4 v) { *reinterpret_cast<u32x4_any*>(p) = v; }
// Past the caches, for more than they hold.
__device__ __forceinline__ u32x4 load16_once(const char* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
}
__device__ __forceinline__ void store16_once(char* p, u32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
}

// Element j of a vector as fp32 (exact for every type).
template <int DT>
__device__ __forceinline__ float unpack(const u32x4& v, int j) {
  if constexpr (DT == TS_DTYPE_F32) {
    return __uint_as_float(v[j]);
  } else if constexpr (DT == TS_DTYPE_BF16) {
    return __uint_as_float((j & 1) ? (v[j >> 1] & 0xFFFF0000u) : (v[j >> 1] << 16));
  } else {
    return __half2float(__ushort_as_half((unsigned short)((j & 1) ? (v[j >> 1] >> 16) : v[j >> 1])));
  }
}
template <int DT>
__device__ __forceinline__ float load_logit(const char* row, int64_t i) {
  if constexpr (DT == TS_DTYPE_F32) return reinterpret_cast<const float*>(row)[i];
  const unsigned short b = reinterpret_cast<const unsigned short*>(row)[i];
  if constexpr (DT == TS_DTYPE_BF16) return __uint_as_float((uint32_t)b << 16);
  return __half2float(__ushort_as_half(b));
}

// Where thread t's vector v of a tile starts: its first logit's id. `own` is where it starts by the
// layout; a vector that would reach past the row's end is moved back to end with the row (or
// starts at 0 where the row is shorter than a vector), and only its logits at or past `own` count.
template <int DT>
struct Place {
  int own, at;
  __device__ __forceinline__ Place(int tile, int t, int v, int V) {
    own = tile * kTile + (v * kLT + t) * Logits<DT>::kW;
    at = min(own, max(V - Logits<DT>::kW, 0));
  }
  __device__ __forceinline__ bool counts(int j, int V) const { return at + j >= own && at + j < V; }
};

// The thread's kLE logits of a tile: the loads, every address in the row, and later the values; what does not count is
// -inf. (A row shorter than a vector is loaded with the values.)
template <int DT>
struct Tile {
  using L = Logits<DT>;
  u32x4 raw[L::kNV];
  __device__ __forceinline__ void load(const char* row, int V, int tile, int t) {
    if ((tile + 1) * kTile <= V) {
      const char* p = row + ((int64_t)tile * kTile + (int64_t)t * L::kW) * L::kSize;
#pragma unroll
      for (int v = 0; v < L::kNV; ++v) raw[v] = load16(p + v * (kLT * 16));
    } else if (V >= L::kW) {
#pragma unroll
      for (int v = 0; v < L::kNV; ++v) raw[v] = load16(row + (int64_t)Place<DT>(tile, t, v, V).at * L::kSize);
    }
  }
  __device__ __forceinline__ void values(const char* row, int V, int tile, int t, float* xs) const {
    if ((tile + 1) * kTile <= V) {
#pragma unroll
      for (int v = 0; v < L::kNV; ++v)
#pragma unroll
        for (int j = 0; j < L::kW; ++j) xs[v * L::kW + j] = unpack<DT>(raw[v], j);
    } else if (V >= L::kW) {
#pragma unroll
      for (int v = 0; v < L::kNV; ++v) {
        const Place<DT> pl(tile, t, v, V);
#pragma unroll
        for (int j = 0; j < L::kW; ++j) xs[v * L::kW + j] = pl.at + j >= pl.own ? unpack<DT>(raw[v], j) : -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLE; ++i) xs[i] = -INFINITY;
      if (t == 0) {
#pragma unroll
        for (int j = 0; j < L::kW; ++j)
          if (j < V) xs[j] = load_logit<DT>(row, j);
      }
    }
  }
};

// 1/T in the base-2 exponent. A temperature below 2^-100 acts as 2^-100: beside the maximum every
// logit more than 2^-93 below it has weight 0 there, as it would at the smaller one.
__device__ __forceinline__ double exponent_scale(float t) { return tsd::kLog2e / (double)fmaxf(t, 0x1p-100f); }

// 2^z is 0 here, so that max(z, kZMin) in a product 2^z z gives 0 for -inf too.
constexpr float kZMin = -151.0f;

}  // namespace tsl
