// pages.hip -- the pages of a cache: writing new tokens into them, forking, growing and freeing sequences, compacting the pages in
// use, and copying pages.
//
// Position j of sequence s lies in page table[s, j / page_slots], slot j % page_slots. refs[p] counts the table entries that name
// page p; a page is free when it is not above 0. No other state: what is free is found by counting, tiles of pages first, so that
// the i-th free page is the same whatever the launch. Everything stays on the device; nothing waits for the host.
//
// All of it is bound by memory: a page's copy by the rate of a large copy (1024 pages of 8 x 32 KB 107 us, 5.0 TB/s read and written;
// 51119 tokens of 4 KB appended 83 us, 5.0 TB/s), the bookkeeping by what one compute unit reads or by the latency of a few
// dependent launches (64 sequences and 20000 pages 17.2 + 4.0 us).
#include <algorithm>
#include <type_traits>

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

constexpr int kPT = 256;                    // threads
constexpr int kPW = kPT / 64;
constexpr int kPE = 16;                     // pages a thread of a tile of pages
constexpr int kPTile = kPT * kPE;
constexpr int kPoolsMax = 64;               // pools a launch of the copy
constexpr int kCopyU = 4;                   // units a thread has in flight
constexpr int64_t kMoveGroups = 4096;       // workgroups that copies are spread over, about

__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* red) {
  const uint32_t incl = wave_incl_scan(v);
  if (lane() == 63) red[wave()] = incl;
  bar();
  uint32_t s = 0;
#pragma unroll
  for (int w = 0; w < kPW; ++w) s += red[w];
  bar();
  return s;
}

// ------------------------------------------------------------------ copies of pages
struct Pool {
  char* data;
  int64_t page_stride;
};
struct MoveArgs {
  Pool pool[kPoolsMax];
  const int32_t *source, *target;   // pairs of pages; a source of -1 is no copy
  const int32_t* count;             // how many (NULL: `most`)
  int32_t most, pools, parts;       // parts: workgroups a pair
  int64_t page_bytes;
};

// ONCE: past the caches.
template <class U, bool ONCE>
__device__ __forceinline__ U load_unit(const char* p) {
  if constexpr (sizeof(U) == 16) return ONCE ? tsl::load16_once(p) : tsl::load16(p);
  else return *reinterpret_cast<const U*>(p);
}
template <class U, bool ONCE>
__device__ __forceinline__ void store_unit(char* p, U v) {
  if constexpr (sizeof(U) != 16) *reinterpret_cast<U*>(p) = v;
  else if constexpr (ONCE) tsl::store16_once(p, v);
  else tsl::store16(p, v);
}

// `part` of `parts` of page `from` of every pool to page `to`. The last unit of a page ends with it, over the ones before. Past the
// caches: 1024 pages of 8 x 32 KB 108 us against 113 through them (4.9 TB/s read and written; a copy of 600 MB 5.2), 1800 such
// pages compacted 181 against 200, 25 MB 18.4 either way. (Eight units in flight instead of four: 112 and 192 us.)
template <class U>
__device__ __forceinline__ void copy_page(const MoveArgs& M, int from, int to, int part) {
  constexpr int span = kPT * kCopyU;
  const int64_t units = (M.page_bytes + (int64_t)sizeof(U) - 1) / (int64_t)sizeof(U), last = M.page_bytes - (int64_t)sizeof(U);
  const int64_t chunks = (units + span - 1) / span;
  for (int64_t w = part; w < chunks * M.pools; w += M.parts) {
    const int p = (int)(w / chunks);
    const int64_t c = w - p * chunks;
    const char* src = M.pool[p].data + (int64_t)from * M.pool[p].page_stride;
    char* dst = M.pool[p].data + (int64_t)to * M.pool[p].page_stride;
    U x[kCopyU];
#pragma unroll
    for (int u = 0; u < kCopyU; ++u) {
      const int64_t at = c * span + u * kPT + threadIdx.x;
      if (at < units) x[u] = load_unit<U, true>(src + min(at * (int64_t)sizeof(U), last));
    }
#pragma unroll
    for (int u = 0; u < kCopyU; ++u) {
      const int64_t at = c * span + u * kPT + threadIdx.x;
      if (at < units) store_unit<U, true>(dst + min(at * (int64_t)sizeof(U), last), x[u]);
    }
  }
}

// Workgroup `block` of those that copy a list's pages.
template <class U>
__device__ __forceinline__ void move_pages(const MoveArgs& M, unsigned block) {
  const int pair = block / (unsigned)M.parts, part = block - pair * M.parts;
  if (M.count && pair >= *M.count) return;
  const int from = M.source[pair];
  if (from >= 0) copy_page<U>(M, from, M.target[pair], part);
}

// ------------------------------------------------------------------ copy
// The source of the last sound pair before `pair` with its target, -1: there is none. The pairs before it a workgroup's width at a time
// from the last one on, a thread a pair: has it this target and a source that is a page and no pair's target? (A source that is
// the target itself is `pair`'s target.) The targets go through LDS, once for each such width that has a candidate: no cost where no
// pair is refused, 11 us where the last of 1024 with one target is, 0.9 and 226 ms where all but the first of 4096 and 65536 are.
__device__ __forceinline__ int last_sound_source(const MoveArgs& M, int pages, int pair, int to) {
  __shared__ __attribute__((aligned(16))) int targets[kPT];
  __shared__ uint32_t red[kPW];
  const int t = threadIdx.x;
  auto first_of = [&](bool x) {   // the lowest thread for which x holds, kPT: none
    const uint32_t low = wave_min(x ? (uint32_t)t : (uint32_t)kPT);
    if (lane() == 0) red[wave()] = low;
    bar();
    uint32_t first = kPT;
#pragma unroll
    for (int w = 0; w < kPW; ++w) first = min(first, red[w]);
    bar();
    return (int)first;
  };
  for (int end = pair; end > 0; end -= kPT) {
    const int i = end - 1 - t;
    const int s = i >= 0 && M.target[i] == to ? M.source[i] : -1;
    bool sound = (uint32_t)s < (uint32_t)pages && s != to;
    if (first_of(sound) == kPT) continue;
    for (int x = 0; x < M.most; x += kPT) {
      targets[t] = x + t < M.most ? M.target[x + t] : -1;
      bar();
      bool found = false;   // no branch, so that the reads of LDS go out one behind the other (with one: four times as long)
#pragma unroll 16
      for (int u = 0; u < kPT; ++u) found |= targets[u] == s;
      sound &= !found;
      bar();
    }
    const int first = first_of(sound);
    if (first < kPT) return M.source[end - 1 - first];
  }
  return -1;
}

// Pair i is refused where its pages are no pages, or its source is some other pair's target (whether it would be read before or
// after that copy is not determined). Of the sound pairs with one target the last one's copy stands alone; the workgroups of the
// last pair of all with that target make it, be that pair sound or not.
template <class U>
__global__ __launch_bounds__(kPT) void ts_pages_copy_kernel(const MoveArgs M, int pages, int32_t* status) {
  __shared__ int hit[2];
  const int pair = blockIdx.x / (unsigned)M.parts, part = blockIdx.x - pair * M.parts;
  int from = M.source[pair];
  const int to = M.target[pair];
  if (threadIdx.x < 2) hit[threadIdx.x] = 0;
  bar();
  bool read = false, later = false;
  for (int i = threadIdx.x; i < M.most; i += kPT) {
    const int t = M.target[i];
    read = read || (t == from && i != pair);
    later = later || (t == to && i > pair);
  }
  if (read) hit[0] = 1;
  if (later) hit[1] = 1;
  bar();
  const bool bad = (uint32_t)from >= (uint32_t)pages || (uint32_t)to >= (uint32_t)pages || hit[0];
  if (part == 0 && threadIdx.x == 0 && status) status[pair] = bad ? TS_ROW_BAD_PAGE : TS_ROW_OK;
  if (hit[1] || (uint32_t)to >= (uint32_t)pages) return;
  if (bad) {
    from = last_sound_source(M, pages, pair, to);
    if (from < 0) return;
  }
  if (from == to) return;
  copy_page<U>(M, from, to, part);
}

// ------------------------------------------------------------------ append
struct AppendArgs {
  const char *k_new, *v_new;
  int64_t kn_token, kn_head, vn_token, vn_head;                  // bytes
  char *k, *v;
  int64_t k_page, k_head, k_slot, v_page, v_head, v_slot;
  const int32_t *offsets, *lengths, *table;
  int64_t table_stride;
  int32_t* status;
  int32_t tokens, batch, heads, pages, page_slots, max_len, token_blocks, slot_bytes;
  Divisor by_page;
};
constexpr int kTokens = 4;   // tokens a workgroup

template <class U, bool ONCE>
__global__ __launch_bounds__(kPT) void ts_cache_append_kernel(const AppendArgs A) {
  const int t = threadIdx.x;
  if ((int)blockIdx.x >= A.token_blocks) {   // a wave a sequence: its verdict
    const int s = ((int)blockIdx.x - A.token_blocks) * kPW + wave();
    if (s >= A.batch || !A.status) return;
    const int n = A.lengths[s], from = A.offsets[s], to = A.offsets[s + 1], fresh = to - from;
    int st = TS_ROW_OK;
    if (from < 0 || to < from || to > A.tokens || n < fresh || n > A.max_len) st = TS_ROW_BAD_LENGTH;
    else if (fresh > 0) {
      bool bad = false;
      const int last = (int)A.by_page.of(n - 1);
      for (int p = (int)A.by_page.of(n - fresh) + lane(); p <= last; p += 64)
        bad = bad || (uint32_t)A.table[s * A.table_stride + p] >= (uint32_t)A.pages;
      if (__builtin_amdgcn_ballot_w64(bad)) st = TS_ROW_BAD_PAGE;
    }
    if (lane() == 0) A.status[s] = st;
    return;
  }
  __shared__ int64_t where[kTokens][2];
  if (t < kTokens) {
    const int token = blockIdx.x * kTokens + t;
    int64_t ko = -1, vo = -1;
    if (token < A.tokens && A.batch > 0 && A.offsets[0] <= token && token < A.offsets[A.batch]) {
      int s = 0, e = A.batch;   // offsets[s] <= token < offsets[e]
      while (e - s > 1) {
        const int mid = (s + e) >> 1;
        if (A.offsets[mid] <= token) s = mid;
        else e = mid;
      }
      const int n = A.lengths[s], from = A.offsets[s], to = A.offsets[s + 1];
      if (from >= 0 && to <= A.tokens && n >= to - from && n <= A.max_len) {
        const int j = n - (to - token);
        const int at = (int)A.by_page.of(j), slot = j - at * A.page_slots;
        const int page = A.table[s * A.table_stride + at];
        if ((uint32_t)page < (uint32_t)A.pages) {
          ko = page * A.k_page + slot * A.k_slot;
          vo = page * A.v_page + slot * A.v_slot;
        }
      }
    }
    where[t][0] = ko;
    where[t][1] = vo;
  }
  bar();
  const int units = (A.slot_bytes + (int)sizeof(U) - 1) / (int)sizeof(U), last = A.slot_bytes - (int)sizeof(U);
  const int of_token = units * A.heads;
  for (int w = t; w < kTokens * 2 * of_token; w += kPT) {
    const int which = w / of_token, x = w - which * of_token, token = which >> 1;
    const int64_t to = where[token][which & 1];
    if (to < 0) continue;
    const int head = x / units;
    const int64_t at = min((x - head * units) * (int)sizeof(U), last), row = (int64_t)blockIdx.x * kTokens + token;
    if (which & 1) store_unit<U, ONCE>(A.v + to + head * A.v_head + at, load_unit<U, ONCE>(A.v_new + row * A.vn_token + head * A.vn_head + at));
    else store_unit<U, ONCE>(A.k + to + head * A.k_head + at, load_unit<U, ONCE>(A.k_new + row * A.kn_token + head * A.kn_head + at));
  }
}

// ------------------------------------------------------------------ fork
struct SeqInfo {
  int32_t children, first;      // sequences that continue it, and the first of those
  int32_t length, status;       // -1 unless status is TS_ROW_OK
};
struct ChildInfo {
  int32_t old, grown;           // positions inherited, and with the new ones
  uint32_t need;                // fresh pages: a copy's, then the growth's
  int32_t copies, status;
};
// What a child's row ends up with.
struct EndInfo {
  int32_t inherited, filled;    // pages of its parent's row as they are; pages in all, the fresh ones between
  int32_t back;                 // whole pages of its parent that it would have shared, had it found a page for its copy
};
struct ForkArgs {
  const int32_t *table, *lengths, *refs, *parent, *n_new;
  int32_t *out_table, *out_lengths, *out_refs, *status;
  int64_t table_stride, out_stride;
  int32_t seqs, children, table_width, out_width, pages, page_slots, max_len, out_max, tiles;
  Divisor by_page, by_width;    // by_width: for the one workgroup
  SeqInfo* seq;                 // [seqs]
  ChildInfo* child;             // [children]
  EndInfo* end;                 // [children]
  uint32_t* start;              // [children + 1]: fresh pages of the children before
  uint32_t* tile_free;          // [tiles]
  int32_t *source, *target;     // [children]: pages to copy
};
__device__ __forceinline__ int pages_of(const Divisor& by_page, int n) { return n > 0 ? (int)by_page.of(n - 1) + 1 : 0; }

// A workgroup a sequence: is its row sound, and who continues it? Also the counts' copy where they are not updated in place.
__global__ __launch_bounds__(kPT) void ts_pages_plan_kernel(const ForkArgs F) {
  __shared__ uint32_t red[kPW];
  if (F.out_refs != F.refs)
    for (int64_t p = (int64_t)blockIdx.x * kPT + threadIdx.x; p < F.pages; p += (int64_t)gridDim.x * kPT) F.out_refs[p] = F.refs[p];
  const int s = blockIdx.x;
  if (s >= F.seqs) return;
  const int n = F.lengths[s];
  int st = n < 0 || n > F.max_len ? TS_ROW_BAD_LENGTH : TS_ROW_OK;
  uint32_t bad = 0;
  if (st == TS_ROW_OK) {
    const int held = pages_of(F.by_page, n);
    for (int p = threadIdx.x; p < held; p += kPT) bad |= (uint32_t)F.table[s * F.table_stride + p] >= (uint32_t)F.pages;
  }
  uint32_t mine = 0, first = 0xFFFFFFFFu;
  for (int c = threadIdx.x; c < F.children; c += kPT)
    if (F.parent[c] == s) {
      ++mine;
      first = min(first, (uint32_t)c);
    }
  bad = block_sum(bad, red);
  const uint32_t all = block_sum(mine, red);
  const uint32_t low = wave_min(first);
  if (lane() == 0) red[wave()] = low;
  bar();
  first = 0xFFFFFFFFu;
#pragma unroll
  for (int w = 0; w < kPW; ++w) first = min(first, red[w]);
  if (threadIdx.x == 0) {
    if (st == TS_ROW_OK && bad) st = TS_ROW_BAD_PAGE;
    // a length that the new table has no room for: nobody can take it over
    F.seq[s] = SeqInfo{n > F.out_max ? 0 : (int)all, (int)first, st == TS_ROW_OK ? n : -1, st};
  }
}

// A workgroup a sequence: its pages' counts go by what became of it. A thread a child: what it inherits and needs.
__global__ __launch_bounds__(kPT) void ts_pages_share_kernel(const ForkArgs F) {
  if ((int)blockIdx.x < F.seqs) {
    const int s = blockIdx.x;
    const SeqInfo I = F.seq[s];
    if (I.status != TS_ROW_OK) return;
    const int whole = (int)F.by_page.of(I.length), held = pages_of(F.by_page, I.length);
    if (I.children != 1)
      for (int p = threadIdx.x; p < whole; p += kPT) atomicAdd(&F.out_refs[F.table[s * F.table_stride + p]], I.children - 1);
    if (held > whole && I.children == 0 && threadIdx.x == 0) atomicAdd(&F.out_refs[F.table[s * F.table_stride + whole]], -1);
    return;
  }
  const int c = ((int)blockIdx.x - F.seqs) * kPT + threadIdx.x;
  if (c >= F.children) return;
  const int p = F.parent[c], grow = F.n_new ? F.n_new[c] : 0;
  ChildInfo C{0, 0, 0, 0, TS_ROW_OK};
  if (p < -1 || p >= F.seqs) {
    C.status = TS_ROW_BAD_PARENT;
  } else if (p >= 0) {
    const SeqInfo I = F.seq[p];
    if (I.status != TS_ROW_OK) C.status = I.status;
    else if (I.length > F.out_max) C.status = TS_ROW_BAD_LENGTH;
    else {
      C.old = I.length;
      C.copies = I.first != c && (int)F.by_page.of(I.length) != pages_of(F.by_page, I.length);
    }
  }
  C.grown = C.old;
  if (C.status == TS_ROW_OK) {
    if (grow < 0 || grow > F.out_max - C.old) C.status = TS_ROW_BAD_LENGTH;
    else C.grown = C.old + grow;
  }
  C.need = (uint32_t)(C.copies + pages_of(F.by_page, C.grown) - pages_of(F.by_page, C.old));
  F.child[c] = C;
}

// Whether a child's fresh pages are among the free ones, given the needs of those before it. One that needs none always fits,
// also behind a child that asked for too many.
__device__ __forceinline__ bool fits(const ChildInfo& C, uint32_t before, uint32_t free) { return C.need == 0 || before + C.need <= free; }

// A child's outputs, once it is known whether its fresh pages are there.
__device__ __forceinline__ void end_child(const ForkArgs& F, int c, const ChildInfo& C, bool found) {
  const bool empty = !found && C.copies;
  const int length = found ? C.grown : empty ? 0 : C.old;
  F.out_lengths[c] = length;
  if (F.status) F.status[c] = C.status != TS_ROW_OK ? C.status : found ? TS_ROW_OK : TS_ROW_NO_PAGE;
  if (!(found && C.copies)) F.source[c] = -1;   // else the copy's pages are filled in with the page that it gets
  F.end[c] = EndInfo{empty ? 0 : pages_of(F.by_page, C.old) - C.copies, pages_of(F.by_page, length),
                     empty ? (int)F.by_page.of(C.old) : 0};
}

// A workgroup a tile of pages: its free ones. The last workgroup: the children's needs, summed.
__global__ __launch_bounds__(kPT) void ts_pages_count_kernel(const ForkArgs F) {
  __shared__ uint32_t red[kPW];
  if ((int)blockIdx.x == F.tiles) {
    const int own = (F.children + kPT - 1) / kPT, a = min(F.children, (int)threadIdx.x * own), z = min(F.children, a + own);
    uint32_t sum = 0;
    for (int c = a; c < z; ++c) sum += F.child[c].need;
    const uint32_t incl = wave_incl_scan(sum);
    if (lane() == 63) red[wave()] = incl;
    bar();
    uint32_t at = incl - sum;
    for (int w = 0; w < wave(); ++w) at += red[w];
    for (int c = a; c < z; ++c) {
      F.start[c] = at;
      at += F.child[c].need;
    }
    if (threadIdx.x == kPT - 1) F.start[F.children] = at;   // the last thread's stretch ends the list, be it empty
    return;
  }
  uint32_t free = 0;
#pragma unroll
  for (int e = 0; e < kPE; ++e) {
    const int64_t p = (int64_t)blockIdx.x * kPTile + e * kPT + threadIdx.x;
    free += p < F.pages && F.out_refs[p] <= 0;
  }
  free = block_sum(free, red);
  if (threadIdx.x == 0) F.tile_free[blockIdx.x] = free;
}

// A workgroup a tile of pages: its free pages go to the children whose turn it is. Then a thread a child: its length and status.
__global__ __launch_bounds__(kPT) void ts_pages_assign_kernel(const ForkArgs F) {
  __shared__ uint32_t red[kPW];
  const bool tile_block = (int)blockIdx.x < F.tiles;
  uint32_t before = 0, all = 0;
  for (int i = threadIdx.x; i < F.tiles; i += kPT) {
    const uint32_t x = F.tile_free[i];
    all += x;
    before += i < (int)blockIdx.x ? x : 0;
  }
  all = block_sum(all, red);
  before = block_sum(before, red);
  if (!tile_block) {
    const int c = ((int)blockIdx.x - F.tiles) * kPT + threadIdx.x;
    if (c >= F.children) return;
    const ChildInfo C = F.child[c];
    end_child(F, c, C, fits(C, F.start[c], all));
    return;
  }
  const uint32_t wanted = F.start[F.children];
  if (before >= wanted) return;
  // the tile's pages in order: thread t holds kPE in a row
  const int64_t first = (int64_t)blockIdx.x * kPTile + threadIdx.x * kPE;
  uint32_t mine = 0;
#pragma unroll
  for (int e = 0; e < kPE; ++e) mine += first + e < F.pages && F.out_refs[first + e] <= 0 ? 1u << e : 0;
  const uint32_t n = __popc(mine);
  const uint32_t incl = wave_incl_scan(n);
  if (lane() == 63) red[wave()] = incl;
  bar();
  uint32_t rank = before + incl - n;
  for (int w = 0; w < wave(); ++w) rank += red[w];
  for (uint32_t left = mine; left && rank < wanted; left &= left - 1, ++rank) {
    const int page = (int)first + __builtin_ctz(left);
    int lo = 0, hi = F.children;   // start[lo] <= rank < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (F.start[mid] <= rank) lo = mid;
      else hi = mid;
    }
    const ChildInfo C = F.child[lo];
    if (F.start[lo] + C.need > all) continue;
    const int k = (int)(rank - F.start[lo]) - C.copies, at = k < 0 ? (int)F.by_page.of(C.old) : pages_of(F.by_page, C.old) + k;
    if (k < 0) {
      F.source[lo] = F.table[F.parent[lo] * F.table_stride + at];
      F.target[lo] = page;
    }
    F.out_table[lo * F.out_stride + at] = page;
    F.out_refs[page] = 1;
  }
}

// A workgroup a child: its row, but for the fresh pages, and what it gives back. Then the copies of pages.
template <class U>
__global__ __launch_bounds__(kPT) void ts_pages_hand_over_kernel(const ForkArgs F, const MoveArgs M, int rows) {
  if ((int)blockIdx.x >= rows) {
    move_pages<U>(M, blockIdx.x - rows);
    return;
  }
  const int c = blockIdx.x;
  const EndInfo E = F.end[c];
  const int of = F.parent[c];
  int32_t* row = F.out_table + c * F.out_stride;
  for (int x = threadIdx.x; x < F.out_width; x += kPT) {
    if (x < E.inherited) row[x] = F.table[of * F.table_stride + x];
    else if (x >= E.filled) row[x] = -1;
  }
  for (int x = threadIdx.x; x < E.back; x += kPT) atomicAdd(&F.out_refs[F.table[of * F.table_stride + x]], -1);
}

// All but that last step by one workgroup, where it goes through the counts and tables in less time than four launches take.
constexpr int kOT = 1024, kOW = kOT / 64;    // its threads
constexpr int kOneSeqs = kOT;                // most sequences, and children: one a thread
// Most pages and entries of the old table together, and most pages of a compaction. (us a call, one workgroup against all of them;
// fork, pages + entries: 8000 + 3000 18.6 and 26.0, 30000 + 16000 21.4 and 25.9, 40000 + 20000 25.3 and 26.1, 50000 + 24000
// 28.9 and 26.2; compaction, pages: 8000 18.4 and 21.0, 30000 20.5 and 21.4, 40000 25.3 and 24.2.)
constexpr int64_t kOneFork = 1 << 16, kOneCompact = 1 << 15;
static_assert(kOneFork <= 64 * kOT && kOneCompact <= 64 * kOT, "a count a thread for each chunk of 64 pages");

// Sum over the workgroup of the values of the threads before this one, and of all.
__device__ __forceinline__ uint32_t one_scan(uint32_t v, uint32_t* red, uint32_t& all) {
  const uint32_t incl = wave_incl_scan(v);
  if (lane() == 63) red[wave()] = incl;
  bar();
  uint32_t before = incl - v;
  all = 0;
#pragma unroll
  for (int w = 0; w < kOW; ++w) {
    before += w < wave() ? red[w] : 0;
    all += red[w];
  }
  bar();
  return before;
}
// masks[c]: for which of the counts 64 c .. + 64 `test` holds; before[c]: for how many before those. Returns how many in all.
template <class F>
__device__ __forceinline__ uint32_t count_chunks(const int32_t* refs, int pages, uint64_t* masks, uint32_t* before, uint32_t* red, F test) {
  const int chunks = (pages + 63) / 64;
  for (int c0 = wave(); c0 < chunks; c0 += 8 * kOW) {
    int32_t r[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) r[u] = refs[min((c0 + u * kOW) * 64 + lane(), pages - 1)];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = c0 + u * kOW;
      const uint64_t m = __builtin_amdgcn_ballot_w64(c * 64 + lane() < pages && test(r[u]));
      if (c < chunks && lane() == 0) masks[c] = m;
    }
  }
  bar();
  uint32_t all;
  const int t = threadIdx.x;
  before[t] = one_scan(t < chunks ? (uint32_t)__popcll(masks[t]) : 0u, red, all);
  bar();
  return all;
}

__global__ __launch_bounds__(kOT) void ts_pages_fork_one_kernel(const ForkArgs F) {
  __shared__ int32_t children[kOneSeqs], length[kOneSeqs], parents[kOneSeqs];
  __shared__ uint32_t first[kOneSeqs], bad[kOneSeqs], start[kOneSeqs + 1];
  __shared__ ChildInfo info[kOneSeqs];
  __shared__ uint64_t masks[kOT];
  __shared__ uint32_t before_chunk[kOT], red[kOW];
  const int t = threadIdx.x;
  if (F.out_refs != F.refs) {
#pragma unroll 8
    for (int p = t; p < F.pages; p += kOT) F.out_refs[p] = F.refs[p];
  }
  children[t] = 0;
  first[t] = 0xFFFFFFFFu;
  bad[t] = 0;
  length[t] = t < F.seqs ? F.lengths[t] : 0;
  const int parent = t < F.children ? F.parent[t] : -1, grow = t < F.children && F.n_new ? F.n_new[t] : 0;
  parents[t] = parent;
  bar();
  if (length[t] < 0 || length[t] > F.max_len) bad[t] = TS_ROW_BAD_LENGTH;
  if (parent >= 0 && parent < F.seqs) {
    atomicAdd(&children[parent], 1);
    atomicMin(&first[parent], (uint32_t)t);
  }
  bar();
#pragma unroll 8
  for (int i = t; i < F.seqs * F.table_width; i += kOT) {
    const int s = (int)F.by_width.of((uint32_t)i), x = i - s * F.table_width;
    const int page = F.table[s * F.table_stride + x];
    if (bad[s] != TS_ROW_BAD_LENGTH && x < pages_of(F.by_page, length[s]) && (uint32_t)page >= (uint32_t)F.pages) bad[s] = TS_ROW_BAD_PAGE;
  }
  bar_all();
  ChildInfo C{0, 0, 0, 0, TS_ROW_OK};
  if (t < F.children) {
    if (parent < -1 || parent >= F.seqs) {
      C.status = TS_ROW_BAD_PARENT;
    } else if (parent >= 0) {
      const int n = length[parent];
      if (bad[parent]) C.status = (int32_t)bad[parent];
      else if (n > F.out_max) C.status = TS_ROW_BAD_LENGTH;
      else {
        C.old = n;
        C.copies = first[parent] != (uint32_t)t && (int)F.by_page.of(n) != pages_of(F.by_page, n);
      }
    }
    C.grown = C.old;
    if (C.status == TS_ROW_OK) {
      if (grow < 0 || grow > F.out_max - C.old) C.status = TS_ROW_BAD_LENGTH;
      else C.grown = C.old + grow;
    }
    C.need = (uint32_t)(C.copies + pages_of(F.by_page, C.grown) - pages_of(F.by_page, C.old));
    info[t] = C;
  }
  uint32_t wanted, all;
  const uint32_t mine = one_scan(C.need, red, wanted);
  start[t] = mine;
  if (t == 0) start[F.children] = wanted;   // of the threads past the children, too
#pragma unroll 8
  for (int i = t; i < F.seqs * F.table_width; i += kOT) {
    const int s = (int)F.by_width.of((uint32_t)i), x = i - s * F.table_width, n = length[s];
    const int heirs = n > F.out_max ? 0 : children[s], whole = bad[s] ? 0 : (int)F.by_page.of(n);
    if (heirs == 1 || bad[s]) continue;
    if (x < whole) atomicAdd(&F.out_refs[F.table[s * F.table_stride + x]], heirs - 1);
    else if (heirs == 0 && x < pages_of(F.by_page, n)) atomicAdd(&F.out_refs[F.table[s * F.table_stride + x]], -1);
  }
  bar_all();
  // the free pages, in order: as many as are wanted
  all = count_chunks(F.out_refs, F.pages, masks, before_chunk, red, [](int32_t r) { return r <= 0; });
  for (int c = wave(); c < (F.pages + 63) / 64; c += kOW) {
    if (before_chunk[c] >= wanted) break;
    const uint32_t rank = before_chunk[c] + mbcnt(masks[c]);
    const int page = c * 64 + lane();
    if (!(masks[c] >> lane() & 1) || rank >= wanted) continue;
    int lo = 0, hi = F.children;   // start[lo] <= rank < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= rank) lo = mid;
      else hi = mid;
    }
    const ChildInfo& I = info[lo];
    if (start[lo] + I.need > all) continue;
    const int k = (int)(rank - start[lo]) - I.copies, at = k < 0 ? (int)F.by_page.of(I.old) : pages_of(F.by_page, I.old) + k;
    if (k < 0) {
      F.source[lo] = F.table[parents[lo] * F.table_stride + at];
      F.target[lo] = page;
    }
    F.out_table[lo * F.out_stride + at] = page;
    F.out_refs[page] = 1;
  }
  if (t < F.children) end_child(F, t, C, fits(C, mine, all));
}

// ------------------------------------------------------------------ compact
struct CompactArgs {
  const int32_t *table, *lengths, *refs;
  int32_t *out_table, *out_refs, *map, *count, *status;
  int64_t table_stride, out_stride;
  int32_t seqs, table_width, pages, page_slots, max_len, tiles;
  Divisor by_page;
  uint32_t* tile_live;              // [tiles]
  int32_t *source, *target;         // [pages / 2]: what moves where
  int32_t* moves;                   // how many; pages in use
};

__global__ __launch_bounds__(kPT) void ts_pages_live_kernel(const CompactArgs C) {
  __shared__ uint32_t red[kPW];
  uint32_t live = 0;
#pragma unroll
  for (int e = 0; e < kPE; ++e) {
    const int64_t p = (int64_t)blockIdx.x * kPTile + e * kPT + threadIdx.x;
    live += p < C.pages && C.refs[p] > 0;
  }
  live = block_sum(live, red);
  if (threadIdx.x == 0) C.tile_live[blockIdx.x] = live;
}

// A workgroup a tile: the free pages below the count and the pages in use past it, each at its rank among its kind. A page that
// moves has -2 - rank in the map for now.
__global__ __launch_bounds__(kPT) void ts_pages_list_kernel(const CompactArgs C) {
  __shared__ uint32_t red[kPW];
  uint32_t before = 0, all = 0;
  for (int i = threadIdx.x; i < C.tiles; i += kPT) {
    const uint32_t x = C.tile_live[i];
    all += x;
    before += i < (int)blockIdx.x ? x : 0;
  }
  all = block_sum(all, red);
  before = block_sum(before, red);
  // pages in use below the count: the whole tiles' and a part of one
  const int cut = (int)(all / kPTile);
  uint32_t below = 0;
  for (int i = threadIdx.x; i < cut; i += kPT) below += C.tile_live[i];
  for (int64_t p = (int64_t)cut * kPTile + threadIdx.x; p < (int64_t)all; p += kPT) below += C.refs[p] > 0;
  below = block_sum(below, red);
  const int64_t first = (int64_t)blockIdx.x * kPTile + threadIdx.x * kPE;
  uint32_t mine = 0;
#pragma unroll
  for (int e = 0; e < kPE; ++e) mine += first + e < C.pages && C.refs[first + e] > 0 ? 1u << e : 0;
  const uint32_t n = __popc(mine);
  const uint32_t incl = wave_incl_scan(n);
  if (lane() == 63) red[wave()] = incl;
  bar();
  uint32_t rank = before + incl - n;   // pages in use before this one
  for (int w = 0; w < wave(); ++w) rank += red[w];
#pragma unroll
  for (int e = 0; e < kPE; ++e) {
    const int64_t p = first + e;
    if (p >= C.pages) break;
    const bool live = mine >> e & 1;
    if (p < (int64_t)all) {
      if (!live) C.target[p - rank] = (int)p;
      C.map[p] = live ? (int)p : -1;
    } else {
      if (live) C.source[rank - below] = (int)p;
      C.map[p] = live ? -2 - (int)(rank - below) : -1;
    }
    rank += live;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    C.moves[0] = (int)(all - below);
    C.moves[1] = (int)all;
    if (C.count) *C.count = (int)all;
  }
}

// A workgroup a sequence: its row renumbered. Then tiles of pages: the counts and the map of what moves. Then the copies.
template <class U>
__global__ __launch_bounds__(kPT) void ts_pages_settle_kernel(const CompactArgs C, const MoveArgs M, int groups) {
  __shared__ uint32_t red[kPW];
  if ((int)blockIdx.x >= C.seqs + groups) {
    move_pages<U>(M, blockIdx.x - C.seqs - groups);
    return;
  }
  if ((int)blockIdx.x < C.seqs) {
    const int s = blockIdx.x, n = C.lengths[s];
    const bool sound = n >= 0 && n <= C.max_len;
    const int held = sound ? pages_of(C.by_page, n) : 0;
    uint32_t bad = 0;
    for (int x = threadIdx.x; x < C.table_width; x += kPT) {
      int to = sound ? -1 : C.table[s * C.table_stride + x];
      if (x < held) {
        const int page = C.table[s * C.table_stride + x];
        to = page;
        if ((uint32_t)page < (uint32_t)C.pages) {
          // the other workgroups replace these by what they stand for: either answers
          const int m = __hip_atomic_load(&C.map[page], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          if (m == -1) bad = 1;
          else to = m <= -2 ? C.target[-2 - m] : m;
        } else {
          bad = 1;
        }
      }
      C.out_table[s * C.out_stride + x] = to;
    }
    bad = block_sum(bad, red);
    if (threadIdx.x == 0 && C.status) C.status[s] = !sound ? TS_ROW_BAD_LENGTH : bad ? TS_ROW_BAD_PAGE : TS_ROW_OK;
    return;
  }
  const int moves = *C.moves;
  const int64_t from = ((int64_t)blockIdx.x - C.seqs) * kPT + threadIdx.x, step = (int64_t)groups * kPT;
  const int all = C.moves[1];
  for (int64_t p = from; p < C.pages; p += step) {
    const int m = __hip_atomic_load(&C.map[p], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (m == p) {
      if (C.out_refs != C.refs) C.out_refs[p] = C.refs[p];
    } else if (m == -1 && p >= all) {   // a free page below the count receives one
      C.out_refs[p] = 0;
    }
  }
  for (int64_t i = from; i < moves; i += step) {
    const int src = C.source[i], dst = C.target[i];
    C.out_refs[dst] = C.refs[src];
    C.out_refs[src] = 0;
    __hip_atomic_store(&C.map[src], dst, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// The count and the list by one workgroup, as for the fork.
__global__ __launch_bounds__(kOT) void ts_pages_compact_one_kernel(const CompactArgs C) {
  __shared__ uint64_t masks[kOT];
  __shared__ uint32_t before_chunk[kOT], red[kOW];
  const int chunks = (C.pages + 63) / 64;
  const uint32_t all = count_chunks(C.refs, C.pages, masks, before_chunk, red, [](int32_t r) { return r > 0; });
  // pages in use below the count
  const int cut = (int)(all / 64);
  const uint32_t below = cut < chunks ? before_chunk[cut] + (uint32_t)__popcll(masks[cut] & (((uint64_t)1 << (all % 64)) - 1)) : all;
#pragma unroll 4
  for (int c = wave(); c < chunks; c += kOW) {
    const int p = c * 64 + lane();
    if (p >= C.pages) continue;
    const bool is = masks[c] >> lane() & 1;
    const uint32_t rank = before_chunk[c] + mbcnt(masks[c]);   // pages in use before this one
    if (p < (int)all) {
      if (!is) C.target[p - rank] = p;
      C.map[p] = is ? p : -1;
    } else {
      if (is) C.source[rank - below] = p;
      C.map[p] = is ? -2 - (int)(rank - below) : -1;
    }
  }
  if (threadIdx.x == 0) {
    C.moves[0] = (int)(all - below);
    C.moves[1] = (int)all;
    if (C.count) *C.count = (int)all;
  }
}

// ------------------------------------------------------------------ host side
int check_pools(const ts_pool* pools, int32_t n, int64_t pages) {
  if (n < 0 || n > 4096) return fail(TS_ERR_INVALID_ARG, "n_pools = %d outside [0, 4096]", (int)n);
  if (n > 0 && !pools) return fail(TS_ERR_INVALID_ARG, "pools is NULL");
  for (int32_t i = 0; i < n; ++i) {
    const ts_pool& p = pools[i];
    if (p.page_bytes < 1 || p.page_bytes > (int64_t)1 << 40)
      return fail(TS_ERR_INVALID_ARG, "pool %d: page_bytes = %lld outside [1, 2^40]", (int)i, (long long)p.page_bytes);
    if (!p.data && pages > 0) return fail(TS_ERR_INVALID_ARG, "pool %d: data is NULL", (int)i);
    if (!tsp::apart(p.page_bytes, {{p.page_stride, pages}}, 1))
      return fail(TS_ERR_INVALID_ARG, "pool %d: page_stride %lld < page_bytes %lld, or too large", (int)i,
                  (long long)p.page_stride, (long long)p.page_bytes);
  }
  return TS_OK;
}

// The first pool with pool i's page size.
int32_t first_of(const ts_pool* pools, int32_t i) {
  int32_t j = 0;
  while (pools && pools[j].page_bytes != pools[i].page_bytes) ++j;
  return j;
}
// f(args, U, workgroups): a launch for up to kPoolsMax pools of one page size, with the copies' unit: 16 bytes at any address where
// a page has so many, else single bytes. One launch at least, where there are no pools.
template <class F>
hipError_t each_pools(const ts_pool* pools, int32_t n, MoveArgs M, F f) {
  int32_t next = 0;
  for (int32_t i = 0; i < std::max(n, 1); i = next) {
    // from pool i on, those of its page size; after the last of them, the next size's first
    M.page_bytes = n ? pools[i].page_bytes : 1;
    M.pools = 0;
    int32_t j = i;
    for (; j < n && M.pools < kPoolsMax; ++j)
      if (pools[j].page_bytes == M.page_bytes) M.pool[M.pools++] = Pool{static_cast<char*>(pools[j].data), pools[j].page_stride};
    while (j < n && pools[j].page_bytes != M.page_bytes) ++j;
    if (j < n) {
      next = j;
    } else {
      const int32_t head = first_of(pools, i);
      for (next = head + 1; next < n && first_of(pools, next) != next; ++next) {}
    }
    const int64_t unit = M.page_bytes >= 16 ? 16 : 1, span = (int64_t)kPT * kCopyU * unit;
    const int64_t chunks = (M.page_bytes + span - 1) / span * M.pools;
    const int64_t pairs = std::max<int64_t>(M.most, 1);
    M.parts = (int32_t)std::max<int64_t>(1, std::min<int64_t>({chunks, (kMoveGroups + pairs - 1) / pairs, 0x7FFFFFFF}));
    const int64_t groups = M.pools ? (int64_t)M.most * M.parts : 0;
    if (unit == 16) f(M, u32x4{}, groups);
    else f(M, uint8_t{}, groups);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
MoveArgs moves_of(const int32_t* source, const int32_t* target, const int32_t* count, int64_t most) {
  MoveArgs M{};
  M.source = source;
  M.target = target;
  M.count = count;
  M.most = (int32_t)most;
  return M;
}

struct ForkPlan {
  size_t off_child = 0, off_end = 0, off_start = 0, off_free = 0, off_source = 0, off_target = 0, total = 0;
  int64_t tiles = 0;
};
constexpr int64_t kMaxSeqs = 1 << 22;   // rows of a table, so that a launch of a workgroup each has fewer than 2^32 threads
// Each sequence looks through all children for its own, each pair of a copy through all targets: of so many at most (a fork of 65536
// sequences 1.3 ms, of 8192 59 us; 65536 pairs 1.5 ms).
constexpr int64_t kMaxFork = 1 << 16, kMaxPairs = 1 << 16;
bool fork_plan(int64_t seqs, int64_t children, int64_t pages, ForkPlan& pl) {
  if (seqs < 0 || seqs > kMaxFork || children < 0 || children > kMaxFork || pages < 0 || pages > tsp::kMaxPages) return false;
  pl.tiles = (pages + kPTile - 1) / kPTile;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
  };
  take((size_t)seqs * sizeof(SeqInfo));
  pl.off_child = take((size_t)children * sizeof(ChildInfo));
  pl.off_end = take((size_t)children * sizeof(EndInfo));
  pl.off_start = take((size_t)(children + 1) * 4);
  pl.off_free = take((size_t)pl.tiles * 4);
  pl.off_source = take((size_t)children * 4);
  pl.off_target = take((size_t)children * 4);
  pl.total = at;
  return true;
}
struct CompactPlan {
  size_t off_source = 0, off_target = 0, off_moves = 0, total = 0;
  int64_t tiles = 0;
};
bool compact_plan(int64_t pages, CompactPlan& pl) {
  if (pages < 0 || pages > 1 << 24) return false;   // a launch has a workgroup for each page that may move
  pl.tiles = (pages + kPTile - 1) / kPTile;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
  };
  take((size_t)pl.tiles * 4);
  pl.off_source = take((size_t)(pages / 2) * 4);
  pl.off_target = take((size_t)(pages / 2) * 4);
  pl.off_moves = take(8);
  pl.total = at;
  return true;
}
int check_workspace(const void* workspace, size_t bytes, size_t needed) {
  if (!workspace) return fail(TS_ERR_WORKSPACE, "workspace is NULL");
  if (((uintptr_t)workspace & 255u) != 0) return fail(TS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (bytes < needed) return fail(TS_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, needed);
  return TS_OK;
}
int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? TS_OK : fail(TS_ERR_LAUNCH, "%s launch failed: %s", what, hipGetErrorString(e));
}

}  // namespace

extern "C" {

int ts_cache_append(const void* k_new, const void* v_new, int64_t tokens, int64_t batch, int32_t kv_heads, int64_t slot_bytes,
                    int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                    const int32_t* offsets, const ts_paged* k_pages, const ts_paged* v_pages, int64_t pages, int32_t page_slots,
                    const int32_t* table, int64_t table_width, int64_t table_stride, const int32_t* lengths, int32_t* row_status,
                    void* stream) {
  if (tokens < 0 || tokens > 0x7FFFFFFF) return fail(TS_ERR_INVALID_ARG, "tokens = %lld outside [0, 2^31)", (long long)tokens);
  if (batch < 0 || batch > kMaxSeqs) return fail(TS_ERR_INVALID_ARG, "batch = %lld outside [0, 2^22]", (long long)batch);
  if (kv_heads < 1 || kv_heads > 1 << 16) return fail(TS_ERR_INVALID_ARG, "kv_heads = %d outside [1, 2^16]", (int)kv_heads);
  if (slot_bytes < 1 || slot_bytes > 1 << 12) return fail(TS_ERR_INVALID_ARG, "slot_bytes = %lld outside [1, 4096]", (long long)slot_bytes);
  int rc = tsp::check_table(pages, page_slots, table_width, table_stride);
  if (rc != TS_OK) return rc;
  if (batch == 0) return TS_OK;
  if (!offsets || (!table && table_width > 0) || !lengths) return fail(TS_ERR_INVALID_ARG, "offsets, table and lengths are required (NULL given)");
  if (tokens > 0 && (!k_new || !v_new)) return fail(TS_ERR_INVALID_ARG, "k_new or v_new is NULL");
  if (!tsp::reaches(slot_bytes, {{k_token_stride, tokens}, {k_head_stride, kv_heads}}, 1) ||
      !tsp::reaches(slot_bytes, {{v_token_stride, tokens}, {v_head_stride, kv_heads}}, 1))
    return fail(TS_ERR_INVALID_ARG, "k_new or v_new: negative or too large strides");
  for (auto [c, name] : {std::pair{k_pages, "k_pages"}, std::pair{v_pages, "v_pages"}}) {
    if (!c || (!c->data && pages > 0)) return fail(TS_ERR_INVALID_ARG, "%s: data is NULL", name);
    if (!tsp::apart(slot_bytes, {{c->page_stride, pages}, {c->head_stride, kv_heads}, {c->slot_stride, page_slots}}, 1))
      return fail(TS_ERR_INVALID_ARG, "%s: slots share memory, or negative or too large strides", name);
  }
  int dev;
  rc = check_device(&dev);
  if (rc != TS_OK) return rc;
  AppendArgs A{};
  A.k_new = static_cast<const char*>(k_new);
  A.v_new = static_cast<const char*>(v_new);
  A.kn_token = k_token_stride;
  A.kn_head = k_head_stride;
  A.vn_token = v_token_stride;
  A.vn_head = v_head_stride;
  A.k = static_cast<char*>(k_pages->data);
  A.k_page = k_pages->page_stride;
  A.k_head = k_pages->head_stride;
  A.k_slot = k_pages->slot_stride;
  A.v = static_cast<char*>(v_pages->data);
  A.v_page = v_pages->page_stride;
  A.v_head = v_pages->head_stride;
  A.v_slot = v_pages->slot_stride;
  A.offsets = offsets;
  A.lengths = lengths;
  A.table = table;
  A.table_stride = table_stride;
  A.status = row_status;
  A.tokens = (int32_t)tokens;
  A.batch = (int32_t)batch;
  A.heads = kv_heads;
  A.pages = (int32_t)pages;
  A.page_slots = page_slots;
  A.max_len = (int32_t)std::min<int64_t>(table_width * page_slots, tsp::kMaxLen);
  A.token_blocks = (int32_t)((tokens + kTokens - 1) / kTokens);
  A.slot_bytes = (int32_t)slot_bytes;
  A.by_page = Divisor(page_slots);
  const int64_t grid = A.token_blocks + (batch + kPW - 1) / kPW;
  if (grid > (int64_t)0xFFFFFFFF / kPT) return fail(TS_ERR_INVALID_ARG, "tokens too large");
  const hipStream_t s = (hipStream_t)stream;
  // What is read and written past the caches: more than they hold (51119 tokens of 4 KB, 418 MB: 82.5 us against 85.3). A step's
  // tokens are left in them for the attention that follows.
  if (slot_bytes < 16) hipLaunchKernelGGL((ts_cache_append_kernel<uint8_t, false>), dim3((unsigned)grid), dim3(kPT), 0, s, A);
  else if (4.0 * tokens * kv_heads * slot_bytes > 256e6)
    hipLaunchKernelGGL((ts_cache_append_kernel<u32x4, true>), dim3((unsigned)grid), dim3(kPT), 0, s, A);
  else hipLaunchKernelGGL((ts_cache_append_kernel<u32x4, false>), dim3((unsigned)grid), dim3(kPT), 0, s, A);
  return launched("append");
}

size_t ts_pages_fork_workspace(int64_t seqs, int64_t children, int64_t pages) {
  ForkPlan pl;
  return fork_plan(seqs, children, pages, pl) ? pl.total : 0;
}

int ts_pages_fork(const int32_t* table, int64_t seqs, int64_t table_width, int64_t table_stride, const int32_t* lengths,
                  const int32_t* refs, int64_t pages, int32_t page_slots, const int32_t* parent, const int32_t* n_new,
                  int64_t children, int32_t* out_table, int64_t out_width, int64_t out_stride, int32_t* out_lengths,
                  int32_t* out_refs, const ts_pool* pools, int32_t n_pools, int32_t* row_status, void* workspace,
                  size_t workspace_bytes, void* stream) {
  int rc = tsp::check_table(pages, page_slots, table_width, table_stride);
  if (rc == TS_OK) rc = tsp::check_table(pages, page_slots, out_width, out_stride);
  if (rc == TS_OK) rc = check_pools(pools, n_pools, pages);
  if (rc != TS_OK) return rc;
  ForkPlan pl;
  if (!fork_plan(seqs, children, pages, pl))
    return fail(TS_ERR_INVALID_ARG, "seqs = %lld or children = %lld outside [0, 65536]", (long long)seqs, (long long)children);
  if (children > 0 && out_width > 0x7FFFFFFF / children - 1) return fail(TS_ERR_INVALID_ARG, "children x out_width too large");
  if (seqs == 0 && children == 0 && pages == 0) return TS_OK;
  if (seqs > 0 && ((!table && table_width > 0) || !lengths)) return fail(TS_ERR_INVALID_ARG, "table and lengths are required (NULL given)");
  if (children > 0 && (!parent || (!out_table && out_width > 0) || !out_lengths))
    return fail(TS_ERR_INVALID_ARG, "parent, out_table and out_lengths are required (NULL given)");
  if (pages > 0 && (!refs || !out_refs)) return fail(TS_ERR_INVALID_ARG, "refs and out_refs are required (NULL given)");
  if (out_table && out_table == table) return fail(TS_ERR_INVALID_ARG, "out_table may not be the table");
  rc = check_workspace(workspace, workspace_bytes, pl.total);
  int dev;
  if (rc == TS_OK) rc = check_device(&dev);
  if (rc != TS_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  ForkArgs F{};
  F.table = table;
  F.lengths = lengths;
  F.refs = refs;
  F.parent = parent;
  F.n_new = n_new;
  F.out_table = out_table;
  F.out_lengths = out_lengths;
  F.out_refs = out_refs;
  F.status = row_status;
  F.table_stride = table_stride;
  F.out_stride = out_stride;
  F.seqs = (int32_t)seqs;
  F.children = (int32_t)children;
  F.table_width = (int32_t)table_width;
  F.out_width = (int32_t)out_width;
  F.pages = (int32_t)pages;
  F.page_slots = page_slots;
  F.max_len = (int32_t)std::min<int64_t>(table_width * page_slots, tsp::kMaxLen);
  F.out_max = (int32_t)std::min<int64_t>(out_width * page_slots, tsp::kMaxLen);
  F.tiles = (int32_t)pl.tiles;
  F.by_page = Divisor(page_slots);
  F.by_width = Divisor((int32_t)std::min<int64_t>(std::max<int64_t>(table_width, 1), kOneFork));
  F.seq = reinterpret_cast<SeqInfo*>(ws);
  F.child = reinterpret_cast<ChildInfo*>(ws + pl.off_child);
  F.end = reinterpret_cast<EndInfo*>(ws + pl.off_end);
  F.start = reinterpret_cast<uint32_t*>(ws + pl.off_start);
  F.tile_free = reinterpret_cast<uint32_t*>(ws + pl.off_free);
  F.source = reinterpret_cast<int32_t*>(ws + pl.off_source);
  F.target = reinterpret_cast<int32_t*>(ws + pl.off_target);
  const hipStream_t s = (hipStream_t)stream;
  if (children > 0 && seqs <= kOneSeqs && children <= kOneSeqs && pages + seqs * table_width <= kOneFork) {
    hipLaunchKernelGGL(ts_pages_fork_one_kernel, dim3(1), dim3(kOT), 0, s, F);
    rc = launched("fork");
  } else {
    const int64_t plan_grid = std::max<int64_t>({seqs, std::min<int64_t>(1024, pl.tiles), 1}), child_blocks = (children + kPT - 1) / kPT;
    hipLaunchKernelGGL(ts_pages_plan_kernel, dim3((unsigned)plan_grid), dim3(kPT), 0, s, F);
    rc = launched("fork plan");
    if (rc != TS_OK || seqs + children == 0) return rc;
    hipLaunchKernelGGL(ts_pages_share_kernel, dim3((unsigned)(seqs + child_blocks)), dim3(kPT), 0, s, F);
    rc = launched("fork share");
    if (rc != TS_OK || children == 0) return rc;
    hipLaunchKernelGGL(ts_pages_count_kernel, dim3((unsigned)(pl.tiles + 1)), dim3(kPT), 0, s, F);
    rc = launched("fork count");
    if (rc != TS_OK) return rc;
    hipLaunchKernelGGL(ts_pages_assign_kernel, dim3((unsigned)(pl.tiles + child_blocks)), dim3(kPT), 0, s, F);
    rc = launched("fork assign");
  }
  if (rc != TS_OK) return rc;
  int rows = (int)children;   // by the first launch
  const hipError_t e = each_pools(pools, n_pools, moves_of(F.source, F.target, nullptr, children), [&](const MoveArgs& m, auto u, int64_t n) {
    hipLaunchKernelGGL(ts_pages_hand_over_kernel<decltype(u)>, dim3((unsigned)(rows + n)), dim3(kPT), 0, s, F, m, rows);
    rows = 0;
  });
  return e == hipSuccess ? TS_OK : fail(TS_ERR_LAUNCH, "fork copy launch failed: %s", hipGetErrorString(e));
}

size_t ts_pages_compact_workspace(int64_t pages) {
  CompactPlan pl;
  return compact_plan(pages, pl) ? pl.total : 0;
}

int ts_pages_compact(const int32_t* table, int64_t seqs, int64_t table_width, int64_t table_stride, const int32_t* lengths,
                     const int32_t* refs, int64_t pages, int32_t page_slots, int32_t* out_table, int64_t out_stride,
                     int32_t* out_refs, int32_t* out_map, int32_t* out_count, const ts_pool* pools, int32_t n_pools,
                     int32_t* row_status, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = tsp::check_table(pages, page_slots, table_width, table_stride);
  if (rc == TS_OK) rc = check_pools(pools, n_pools, pages);
  if (rc != TS_OK) return rc;
  CompactPlan pl;
  if (!compact_plan(pages, pl)) return fail(TS_ERR_INVALID_ARG, "pages = %lld outside [1, 2^24]", (long long)pages);
  if (seqs < 0 || seqs > kMaxSeqs) return fail(TS_ERR_INVALID_ARG, "seqs = %lld outside [0, 2^22]", (long long)seqs);
  if (out_stride < table_width) return fail(TS_ERR_INVALID_ARG, "out_stride %lld < table_width %lld", (long long)out_stride, (long long)table_width);
  if (seqs > 0 && (((!table || !out_table) && table_width > 0) || !lengths))
    return fail(TS_ERR_INVALID_ARG, "table, out_table and lengths are required (NULL given)");
  if (out_table && out_table == table && out_stride != table_stride)
    return fail(TS_ERR_INVALID_ARG, "an output in its input's place needs the input's stride");
  if (pages < 1) return fail(TS_ERR_INVALID_ARG, "pages = %lld < 1", (long long)pages);
  if (!refs || !out_refs || !out_map) return fail(TS_ERR_INVALID_ARG, "refs, out_refs and out_map are required (NULL given)");
  rc = check_workspace(workspace, workspace_bytes, pl.total);
  int dev;
  if (rc == TS_OK) rc = check_device(&dev);
  if (rc != TS_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  CompactArgs C{};
  C.table = table;
  C.lengths = lengths;
  C.refs = refs;
  C.out_table = out_table;
  C.out_refs = out_refs;
  C.map = out_map;
  C.count = out_count;
  C.status = row_status;
  C.table_stride = table_stride;
  C.out_stride = out_stride;
  C.seqs = (int32_t)seqs;
  C.table_width = (int32_t)table_width;
  C.pages = (int32_t)pages;
  C.page_slots = page_slots;
  C.max_len = (int32_t)std::min<int64_t>(table_width * page_slots, tsp::kMaxLen);
  C.tiles = (int32_t)pl.tiles;
  C.by_page = Divisor(page_slots);
  C.tile_live = reinterpret_cast<uint32_t*>(ws);
  C.source = reinterpret_cast<int32_t*>(ws + pl.off_source);
  C.target = reinterpret_cast<int32_t*>(ws + pl.off_target);
  C.moves = reinterpret_cast<int32_t*>(ws + pl.off_moves);
  const hipStream_t s = (hipStream_t)stream;
  if (pages <= kOneCompact) {
    hipLaunchKernelGGL(ts_pages_compact_one_kernel, dim3(1), dim3(kOT), 0, s, C);
    rc = launched("compact");
  } else {
    hipLaunchKernelGGL(ts_pages_live_kernel, dim3((unsigned)pl.tiles), dim3(kPT), 0, s, C);
    rc = launched("compact count");
    if (rc != TS_OK) return rc;
    hipLaunchKernelGGL(ts_pages_list_kernel, dim3((unsigned)pl.tiles), dim3(kPT), 0, s, C);
    rc = launched("compact list");
  }
  if (rc != TS_OK) return rc;
  const int groups = (int)std::min<int64_t>(1024, pl.tiles * 4);
  bool first = true;
  const hipError_t e = each_pools(pools, n_pools, moves_of(C.source, C.target, C.moves, pages / 2), [&](const MoveArgs& m, auto u, int64_t n) {
    CompactArgs c = C;
    if (!first) c.seqs = 0;
    const int g = first ? groups : 0;
    first = false;
    if (c.seqs + g + n > 0)
      hipLaunchKernelGGL(ts_pages_settle_kernel<decltype(u)>, dim3((unsigned)(c.seqs + g + n)), dim3(kPT), 0, s, c, m, g);
  });
  return e == hipSuccess ? TS_OK : fail(TS_ERR_LAUNCH, "compact copy launch failed: %s", hipGetErrorString(e));
}

int ts_pages_copy(const int32_t* source, const int32_t* target, int64_t n, int64_t pages, const ts_pool* pools, int32_t n_pools,
                  int32_t* pair_status, void* stream) {
  if (n < 0 || n > kMaxPairs) return fail(TS_ERR_INVALID_ARG, "n = %lld outside [0, 65536]", (long long)n);
  if (pages < 0 || pages > tsp::kMaxPages) return fail(TS_ERR_INVALID_ARG, "pages = %lld outside [0, 2^31)", (long long)pages);
  int rc = check_pools(pools, n_pools, pages);
  if (rc != TS_OK) return rc;
  if (n == 0) return TS_OK;
  if (!source || !target) return fail(TS_ERR_INVALID_ARG, "source and target are required (NULL given)");
  int dev;
  rc = check_device(&dev);
  if (rc != TS_OK) return rc;
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e = each_pools(pools, n_pools, moves_of(source, target, nullptr, n), [&](const MoveArgs& m, auto u, int64_t) {
    hipLaunchKernelGGL(ts_pages_copy_kernel<decltype(u)>, dim3((unsigned)(n * m.parts)), dim3(kPT), 0, s, m, (int)pages, pair_status);
  });
  return e == hipSuccess ? TS_OK : fail(TS_ERR_LAUNCH, "page copy launch failed: %s", hipGetErrorString(e));
}

}  // extern "C"
