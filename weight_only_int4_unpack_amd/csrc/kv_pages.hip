// Pages of the cache: who holds them (fork, resize), their copies, and the tokens of an
// accepted path moved together.
//
// Copies and moves are bound by HBM (or, for a few pages, by the launch): 16 bytes a lane,
// read once and written once. Forks and resizes are a few dependent looks at the table and
// the counts, one workgroup: their time is latency.
#include "batch_internal.h"
#include "serve_device.h"

namespace w4a16 {
namespace {

using namespace serve;

// ---- forks and resizes
// Every listed change needs `need` new pages, which go into consecutive entries of its row
// from `entry` on. Pages are handed out in the order of the list, lowest first, from those
// that nobody held at the start: what this call takes back is for later calls, so that no
// page that is to be read (src) is one that is to be written (dst).
struct PagesLds {
  int32_t row[kPagesMaxList];
  int32_t entry[kPagesMaxList];
  int32_t upto[kPagesMaxList + 1];       // pages that the changes before i need
  int32_t wave[kPagesThreads / 64];
  int32_t sum;
};

// Sum of `x` over the threads before this one; the whole in l.sum.
__device__ __forceinline__ int block_prefix(PagesLds& l, int x, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  int upto = x;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int y = __shfl_up(upto, s);
    if (lane >= s) upto += y;
  }
  if (lane == 63) l.wave[wave] = upto;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPagesThreads / 64; ++i) {
    const int v = l.wave[i];
    before += i < wave ? v : 0;
    all += v;
  }
  if (tid == 0) l.sum = all;
  __syncthreads();
  return before + upto - x;
}

// Calls take(k, page) with the k-th free page, k < want, in ascending order; returns how
// many there are (stops looking when there are enough).
template <typename Take>
__device__ __forceinline__ int free_pages(PagesLds& l, const int32_t* refs, int pages, int want, int tid, Take take) {
  constexpr int kEach = 8;
  int found = 0;
  for (int base = 0; base < pages && found < want; base += kPagesThreads * kEach) {
    const int first = base + tid * kEach;
    int held[kEach], mine = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) held[e] = first + e < pages ? refs[first + e] : 1;
#pragma unroll
    for (int e = 0; e < kEach; ++e) mine += held[e] == 0;
    int k = found + block_prefix(l, mine, tid);
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (held[e] == 0) {
        if (k < want) take(k, first + e);
        ++k;
      }
    found += l.sum;
    __syncthreads();
  }
  return found;
}

template <bool FORK>
__global__ __launch_bounds__(kPagesThreads) void pages_kernel(PagesParams p) {
  __shared__ PagesLds l;
  const int tid = threadIdx.x;
  const int size = 1 << p.page_shift;
  const int64_t room = (int64_t)p.table_pages << p.page_shift;
  constexpr int kEach = kPagesMaxList / kPagesThreads;
  auto pages_of = [&](int tokens) { return (tokens >> p.page_shift) + ((tokens & (size - 1)) != 0); };
  auto length_of = [&](int row) { return (int)min((int64_t)max(p.lens[row], 0), room); };
  auto entry_of = [&](int row, int k) -> int32_t& { return p.table[row * p.table_stride + k]; };
  auto known = [&](int page) { return page >= 0 && page < p.pages; };
  auto release = [&](int page) {
    if (known(page) && atomicSub(p.refs + page, 1) <= 0) atomicAdd(p.refs + page, 1);
  };

  // the rows that change: each once
  for (int i = tid; i < p.count; i += kPagesThreads) l.row[i] = FORK ? p.to[i] : p.from[i];
  __syncthreads();
  int need[kEach], old_len[kEach], new_len[kEach];
  bool good[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = tid * kEach + e;
    need[e] = 0;
    good[e] = false;
    old_len[e] = new_len[e] = 0;
    if (i >= p.count) continue;
    const int row = l.row[i];
    bool ok = row >= 0 && row < p.rows;
    for (int j = 0; j < i && ok; ++j) ok = l.row[j] != row;
    int src = -1, entry = 0;
    if constexpr (FORK) {
      const int parent = p.from[i];
      ok = ok && parent >= 0 && parent < p.rows && parent != row && p.lens[row] <= 0;
      if (ok) {
        new_len[e] = length_of(parent);
        entry = new_len[e] >> p.page_shift;
        if (new_len[e] & (size - 1)) {
          need[e] = 1;
          src = entry_of(parent, entry);
        }
      }
    } else {
      const int want = p.to[i];
      ok = ok && want >= 0 && want <= room;
      if (ok) {
        old_len[e] = length_of(row);
        new_len[e] = want;
        const int kept = min(old_len[e], want);
        entry = pages_of(old_len[e]);
        need[e] = max(pages_of(want) - entry, 0);
        if (kept & (size - 1)) {
          const int last = kept >> p.page_shift;
          const int page = entry_of(row, last);
          if (known(page) && p.refs[page] > 1) {
            src = page;
            entry = last;
            ++need[e];
          }
        }
      }
    }
    good[e] = ok;
    l.entry[i] = entry;
    p.src[i] = known(src) ? src : -1;
    p.dst[i] = -1;
  }
  // what the changes before each need: saturated, as nothing past the pages is served
  {
    int64_t mine = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) mine += need[e];
    const int lane = tid & 63, wave = tid >> 6;
    int64_t upto = mine;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int64_t y = __shfl_up(upto, s);
      if (lane >= s) upto += y;
    }
    if (lane == 63) l.wave[wave] = (int)min(upto, (int64_t)p.pages + 1);
    __syncthreads();
    int64_t before = upto - mine;
    for (int i = 0; i < wave; ++i) before += l.wave[i];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = tid * kEach + e;
      if (i <= p.count) l.upto[i] = (int)min(before, (int64_t)p.pages + 1);
      before += need[e];
      if (i == kPagesMaxList - 1) l.upto[i + 1] = (int)min(before, (int64_t)p.pages + 1);
    }
    __syncthreads();
  }
  const int want = l.upto[p.count];
  const int free = want == 0 ? 0 : free_pages(l, p.refs, p.pages, want, tid, [](int, int) {});
  if (want > 0) {
    free_pages(l, p.refs, p.pages, min(want, free), tid, [&](int k, int page) {
      int lo = 0, hi = p.count;          // the last change with upto <= k
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (l.upto[mid] <= k) lo = mid; else hi = mid;
      }
      if (l.upto[lo + 1] > free) return;  // not served
      entry_of(l.row[lo], l.entry[lo] + k - l.upto[lo]) = page;
      p.refs[page] = 1;
      if (k == l.upto[lo] && (FORK || p.src[lo] >= 0)) p.dst[lo] = page;
    });
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = tid * kEach + e;
    if (i < p.count) good[e] = good[e] && (need[e] == 0 || l.upto[i + 1] <= free);
  }
  __syncthreads();
  // Lengths; and what is left to do for each change, which whole waves take below.
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = tid * kEach + e;
    if (i >= p.count) continue;
    const bool ok = good[e];
    p.served[i] = ok;
    if (!ok) p.src[i] = -1;
    if (!FORK && ok && p.src[i] >= 0) release(p.src[i]);
    if (ok) p.lens[l.row[i]] = new_len[e];
    // pages: [first, last) of this row are taken back, or of the parent's row shared
    if (FORK) {
      l.entry[i] = ok ? new_len[e] >> p.page_shift : 0;
    } else {
      l.entry[i] = pages_of(new_len[e]);
      l.upto[i] = ok ? pages_of(old_len[e]) : 0;
    }
    if (!ok) l.row[i] = -1;
  }
  __syncthreads();
  const int lane = tid & 63;
  for (int i = tid >> 6; i < p.count; i += kPagesThreads / 64) {
    const int row = l.row[i];
    if (row < 0) continue;
    if constexpr (FORK) {
      const int parent = p.from[i];
      for (int k = lane; k < l.entry[i]; k += 64) {
        const int page = entry_of(parent, k);
        entry_of(row, k) = page;
        if (known(page)) atomicAdd(p.refs + page, 1);
      }
    } else {
      for (int k = l.entry[i] + lane; k < l.upto[i]; k += 64) {
        release(entry_of(row, k));
        entry_of(row, k) = -1;
      }
    }
  }
}

// ---- copies of pages
// A workgroup copies kCopyEach * 256 units of 16 bytes of one pair in one cache; k, v and
// their scales count as one run of units.
__global__ __launch_bounds__(kCopyThreads) void copy_pages_kernel(CopyPagesParams p) {
  uint32_t at = blockIdx.x;
  const uint32_t chunk = at % p.chunks;
  at /= p.chunks;
  const uint32_t cache = at % (uint32_t)p.count, pair = at / (uint32_t)p.count;
  const int64_t src = p.src[pair], dst = p.dst[pair];
  if (src < 0 || src >= p.pages || dst < 0 || dst >= p.pages || src == dst) return;
  const CacheAddresses& c = p.caches[cache];
  char* base[kCopyEach];
  u32x4 held[kCopyEach];
  const uint32_t first = chunk * (kCopyThreads * kCopyEach) + threadIdx.x;
  const uint32_t all = 2 * (p.page_units + p.scale_units);
#pragma unroll
  for (int e = 0; e < kCopyEach; ++e) {
    uint32_t u = first + e * kCopyThreads;
    base[e] = nullptr;
    if (u >= all) continue;
    char* x = c.k;
    uint32_t units = p.page_units;
    if (u >= 2 * p.page_units) {
      u -= 2 * p.page_units;
      units = p.scale_units;
      x = u >= units ? c.v_scale : c.k_scale;
    } else if (u >= units) {
      x = c.v;
    }
    if (u >= units) u -= units;
    const char* from = x + (src * units + u) * 16;
    base[e] = x + (dst * units + u) * 16;
    held[e] = load16(from);
  }
#pragma unroll
  for (int e = 0; e < kCopyEach; ++e)
    if (base[e]) *(u32x4*)base[e] = held[e];
}

// ---- compaction
// A thread moves one unit (16 bytes of a head's row, or a scale) of every kept token, in
// order. Place j is read, if at all, as the source of a token before the j-th (a path
// ascends): by the same thread, before it writes there. Loads of a few tokens are ahead of
// their stores: they only get earlier.
constexpr int kCompactList = 64;
__global__ __launch_bounds__(kCompactThreads) void compact_kernel(CompactParams p) {
  __shared__ int64_t from[kCompactList], to[kCompactList];   // token rows of head 0
  __shared__ int kept_total, moves;
  uint32_t at = blockIdx.x;
  const uint32_t block = at % (uint32_t)p.blocks;
  at /= (uint32_t)p.blocks;
  const uint32_t cache = at % (uint32_t)p.count;
  const int b = at / (uint32_t)p.count;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t start = p.q_starts[b], end = p.q_starts[b + 1];
  const int64_t len = p.kv_lens[b], n = end - start;
  const int64_t first = len - n;
  const bool any = n > 0 && first >= 0;
  const int listed = any ? min(max(p.counts[b], 0), p.width) : 0;
  const int32_t* path = p.path + (int64_t)b * p.width;

  // unit of this thread
  const int work = block * kCompactThreads + tid;
  const int units = 2 * p.heads * p.row_units, scales = p.scaled ? 2 * p.heads : 0;
  const bool moves_unit = work < units, moves_scale = !moves_unit && work < units + scales;
  char* base = nullptr;
  int64_t head_rows = 0;                 // rows of the heads before this one in a page
  int part = 0;
  if (moves_unit) {
    const int head = work / p.row_units;
    part = work - head * p.row_units;
    base = head >= p.heads ? p.caches[cache].v : p.caches[cache].k;
    head_rows = (int64_t)(head >= p.heads ? head - p.heads : head) << p.page_shift;
  } else if (moves_scale) {
    const int head = work - units;
    base = head >= p.heads ? p.caches[cache].v_scale : p.caches[cache].k_scale;
    head_rows = (int64_t)(head >= p.heads ? head - p.heads : head) << p.page_shift;
  }

  int64_t above = -1;                    // the path's entry before
  int kept = 0;
  for (int base_j = 0; base_j < listed; base_j += kCompactList) {
    __syncthreads();                     // the list is read no more
    if (tid < 64) {
      const int j = base_j + lane;
      const int64_t node = j < listed ? path[j] : -1;
      const int64_t before = lane == 0 ? above : j < listed ? path[j - 1] : -1;
      const bool good = j < listed && node > before && node < n && node >= 0;
      const int run = __builtin_ctzll(~__ballot(good) | (1ull << 63)) +
                      (int)(__ballot(good) == ~0ull);
      // row of token t of the sequence, head 0; -1: nowhere
      auto place = [&](int64_t t) -> int64_t {
        const int64_t k = t >> p.page_shift;
        if (k >= p.table_pages) return -1;
        const int64_t page = p.block_table[b * p.table_stride + k];
        if (page < 0 || page >= p.pages) return -1;
        return ((page * p.heads) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
      };
      const bool moved = lane < run && node != j;
      const int64_t src = moved ? place(first + node) : -1, dst = moved ? place(first + j) : -1;
      const uint64_t lanes = __ballot(src >= 0 && dst >= 0);
      if (src >= 0 && dst >= 0) {
        const int k = __popcll(lanes & ((1ull << lane) - 1));
        from[k] = src;
        to[k] = dst;
      }
      if (lane == 0) {
        moves = __popcll(lanes);
        kept_total = kept + run;
      }
    }
    __syncthreads();
    const int count = moves;
    const bool whole = kept_total - kept == min(kCompactList, listed - base_j);
    kept = kept_total;
    above = path[min(base_j + kCompactList, listed) - 1];
    constexpr int kAhead = 8;
    for (int i = 0; i < count; i += kAhead) {
      if (moves_unit) {
        u32x4 held[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (i + e < count) held[e] = load16(base + ((from[i + e] + head_rows) * p.row_units + part) * 16);
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (i + e < count) *(u32x4*)(base + ((to[i + e] + head_rows) * p.row_units + part) * 16) = held[e];
      } else if (moves_scale) {
        float held[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (i + e < count) held[e] = ((const float*)base)[from[i + e] + head_rows];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (i + e < count) ((float*)base)[to[i + e] + head_rows] = held[e];
      }
    }
    if (!whole) break;
  }
  if (p.new_lens && block == 0 && cache == 0 && tid == 0) p.new_lens[b] = (int32_t)(any ? first + kept : len);
}

}  // namespace

hipError_t launch_pages(const PagesParams& p, bool fork, hipStream_t stream) {
  if (fork)
    pages_kernel<true><<<1, kPagesThreads, 0, stream>>>(p);
  else
    pages_kernel<false><<<1, kPagesThreads, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_copy_pages(const CopyPagesParams& p, hipStream_t stream) {
  copy_pages_kernel<<<(unsigned)(p.pairs * p.count * p.chunks), kCopyThreads, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_compact(const CompactParams& p, hipStream_t stream) {
  compact_kernel<<<(unsigned)((int64_t)p.sequences * p.count * p.blocks), kCompactThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace w4a16
