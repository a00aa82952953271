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
// One sequence forked in 3 ways 6.1 us, 10 in 4 each 7.5; resized 4.0 and 5.7: waits are 75 %.
// (The first look at the counts only when their number is known, and a wave for each row in
// turn: 9.1 and 7.2 us for the 40.)
// Every listed change needs `need` new pages, which go into consecutive entries of its row
// from `entry` on. Pages are handed out in the order of the list, lowest first, from those
// that nobody held at the start: what this call takes back is for later calls, so that no
// page that is to be read (src) is one that is to be written (dst).
constexpr int kPagesWaves = kPagesThreads / 64;
constexpr int kPagesFound = 2048;        // free pages that are kept from the first look
struct PagesLds {
  int32_t row[kPagesMaxList];
  int32_t entry[kPagesMaxList];
  uint32_t upto[kPagesMaxList + 1];      // pages that the changes before i need
  int32_t found[kPagesFound];
  uint32_t wave[kPagesWaves];
};

// Sums stop at one more than any pool has pages: nothing behind that is served.
constexpr uint32_t kPagesLimit = (1u << 30) + 1;
__device__ __forceinline__ uint32_t add_pages(uint32_t x, uint32_t y) { return min(x + y, kPagesLimit); }

// Sum of `x` over the threads before this one; *all: over all of them.
__device__ __forceinline__ uint32_t block_prefix(PagesLds& l, uint32_t x, int tid, uint32_t* all) {
  const int lane = tid & 63, wave = tid >> 6;
  uint32_t upto = x;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const uint32_t y = __shfl_up(upto, s);
    if (lane >= s) upto = add_pages(upto, y);
  }
  const uint32_t here = __shfl_up(upto, 1);
  __syncthreads();                       // the sums of the call before are read
  if (lane == 63) l.wave[wave] = upto;
  __syncthreads();
  uint32_t before = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < kPagesWaves; ++i) {
    const uint32_t v = l.wave[i];
    before = i < wave ? add_pages(before, v) : before;
    sum = add_pages(sum, v);
  }
  *all = sum;
  return lane == 0 ? before : add_pages(before, here);
}

// Counts of the pages that a thread looks at, at a time; 1 behind the last page.
constexpr int kPagesLook = 8;
struct Look {
  int held[kPagesLook];
};
__device__ __forceinline__ Look look(const int32_t* refs, int pages, int64_t base, int tid) {
  Look x;
  const int64_t first = base + tid * kPagesLook;
#pragma unroll
  for (int e = 0; e < kPagesLook; ++e) x.held[e] = first + e < pages ? refs[first + e] : 1;
  return x;
}
// Calls take(k, page) with the k-th free page, k < want, in ascending order; returns how
// many there are (stops looking when there are enough). `x`: the first look.
template <typename Take>
__device__ __forceinline__ uint32_t free_pages(PagesLds& l, const int32_t* refs, int pages, uint32_t want, int tid,
                                               Look x, Take take) {
  uint32_t found = 0;
  for (int64_t base = 0; base < pages && found < want;) {
    const int64_t first = base + tid * kPagesLook;
    uint32_t mine = 0;
#pragma unroll
    for (int e = 0; e < kPagesLook; ++e) mine += x.held[e] == 0;
    uint32_t all, k = found + block_prefix(l, mine, tid, &all);
#pragma unroll
    for (int e = 0; e < kPagesLook; ++e)
      if (x.held[e] == 0) {
        if (k < want) take(k, (int)(first + e));
        ++k;
      }
    found += all;
    base += kPagesThreads * kPagesLook;
    x = look(refs, pages, base, tid);
  }
  return found;
}

template <bool FORK>
__global__ __launch_bounds__(kPagesThreads) void pages_kernel(PagesParams p) {
  __shared__ PagesLds l;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int size = 1 << p.page_shift;
  const int64_t room = (int64_t)p.table_pages << p.page_shift;
  constexpr int kEach = kPagesMaxList / kPagesThreads;   // changes of a thread: tid, tid + kPagesThreads, ...
  auto pages_of = [&](int tokens) { return (tokens >> p.page_shift) + ((tokens & (size - 1)) != 0); };
  auto length_of = [&](int row) { return (int)min((int64_t)max(p.lens[row], 0), room); };
  auto entry_of = [&](int row, int k) -> int32_t& { return p.table[row * p.table_stride + k]; };
  auto known = [&](int page) { return page >= 0 && page < p.pages; };
  auto release = [&](int page) {
    if (known(page) && atomicSub(p.refs + page, 1) <= 0) atomicAdd(p.refs + page, 1);
  };

  // the rows that change, each once: a wave looks for one among those before it
  for (int i = tid; i < p.count; i += kPagesThreads) l.row[i] = FORK ? p.to[i] : p.from[i];
  __syncthreads();
  for (int i = wave; i < p.count; i += kPagesWaves) {
    const int row = l.row[i];
    bool before = false;
    for (int j = lane; j < i; j += 64) before |= l.row[j] == row;
    const bool twice = __ballot(before) != 0;
    if (lane == 0) l.entry[i] = twice;
  }
  __syncthreads();
  const Look first_look = look(p.refs, p.pages, 0, tid);   // on its way while the changes are read
  uint32_t need[kEach], carry = 0;
  int old_len[kEach], new_len[kEach], src[kEach], entry[kEach], from[kEach];
  bool good[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    if (e * kPagesThreads >= p.count) break;
    const int i = tid + e * kPagesThreads;
    need[e] = 0;
    old_len[e] = new_len[e] = entry[e] = from[e] = 0;
    src[e] = -1;
    good[e] = false;
    if (i < p.count) {
      const int row = l.row[i];
      bool ok = row >= 0 && row < p.rows && l.entry[i] == 0;
      if constexpr (FORK) {
        const int parent = from[e] = p.from[i];
        ok = ok && parent >= 0 && parent < p.rows && parent != row;
        if (ok) {
          const int held = p.lens[row];
          new_len[e] = length_of(parent);
          entry[e] = new_len[e] >> p.page_shift;
          ok = held <= 0;
          if (ok && (new_len[e] & (size - 1))) {
            need[e] = 1;
            src[e] = entry_of(parent, entry[e]);
          }
        }
      } else {
        const int want = p.to[i];
        ok = ok && want >= 0 && want <= room;
        if (ok) {
          old_len[e] = length_of(row);
          new_len[e] = want;
          const int kept = min(old_len[e], want);
          entry[e] = pages_of(old_len[e]);
          need[e] = max(pages_of(want) - entry[e], 0);
          if (kept & (size - 1)) {
            const int last = kept >> p.page_shift;
            const int page = entry_of(row, last);
            if (known(page) && p.refs[page] > 1) {
              src[e] = page;
              entry[e] = last;
              ++need[e];
            }
          }
        }
      }
      good[e] = ok;
      src[e] = known(src[e]) ? src[e] : -1;
      p.dst[i] = -1;
    }
    uint32_t all;
    const uint32_t before = add_pages(carry, block_prefix(l, need[e], tid, &all));
    carry = add_pages(carry, all);
    if (i < p.count) {
      l.upto[i] = before;
      l.entry[i] = FORK || src[e] >= 0 ? entry[e] : -1 - entry[e];   // negative: its first page is no copy
    }
  }
  if (tid == 0) l.upto[p.count] = carry;
  __syncthreads();
  const uint32_t want = carry;
  if (want > 0) {
    const uint32_t free = free_pages(l, p.refs, p.pages, want, tid, first_look, [&](uint32_t k, int page) {
      if (k < kPagesFound) l.found[k] = page;
    });
    __syncthreads();
    auto give = [&](uint32_t k, int page) {
      int lo = 0, hi = p.count;          // the last change with upto <= k
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (l.upto[mid] <= k) lo = mid; else hi = mid;
      }
      if (l.upto[lo + 1] > free) return;  // not served
      const int at = l.entry[lo], in = k - l.upto[lo];
      entry_of(l.row[lo], (at < 0 ? -1 - at : at) + in) = page;
      p.refs[page] = 1;
      if (in == 0 && at >= 0) p.dst[lo] = page;
    };
    const uint32_t given = min(want, free);
    if (given <= kPagesFound) {
      for (uint32_t k = tid; k < given; k += kPagesThreads) give(k, l.found[k]);
    } else {
      free_pages(l, p.refs, p.pages, given, tid, look(p.refs, p.pages, 0, tid), give);
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (e * kPagesThreads >= p.count) break;
      const int i = tid + e * kPagesThreads;
      if (i < p.count && need[e] > 0 && l.upto[i + 1] > free) good[e] = false;
    }
    __syncthreads();
  }
  // Lengths; and what is left to do for each change, which many threads take below.
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    if (e * kPagesThreads >= p.count) break;
    const int i = tid + e * kPagesThreads;
    if (i >= p.count) continue;
    const bool ok = good[e];
    p.served[i] = ok;
    p.src[i] = ok ? src[e] : -1;
    if (!FORK && ok && src[e] >= 0) release(src[e]);
    if (ok) p.lens[l.row[i]] = new_len[e];
    // pages: [first, last) of this row are taken back, or of the parent's row shared. The lists are
    // read no more: they may be views of the lengths, which change here.
    if (FORK) {
      l.entry[i] = ok ? new_len[e] >> p.page_shift : 0;
      l.upto[i] = from[e];
    } else {
      l.entry[i] = pages_of(new_len[e]);
      l.upto[i] = ok ? pages_of(old_len[e]) : 0;
    }
    if (!ok) l.row[i] = -1;
  }
  __syncthreads();
  // as many threads a change as there are for all of them, 16 at least
  const int shift = min(p.count > 1 ? 32 - __builtin_clz(p.count - 1) : 0, 6), lanes = kPagesThreads >> shift;
  for (int i = tid / lanes; i < p.count; i += 1 << shift) {
    const int row = l.row[i];
    if (row < 0) continue;
    if constexpr (FORK) {
      const int parent = (int)l.upto[i];
      for (int k = tid % lanes; k < l.entry[i]; k += lanes) {
        const int page = entry_of(parent, k);
        entry_of(row, k) = page;
        if (known(page)) atomicAdd(p.refs + page, 1);
      }
    } else {
      for (int k = l.entry[i] + tid % lanes; k < (int)l.upto[i]; k += lanes) {
        const int page = entry_of(row, k);
        release(page);
        entry_of(row, k) = -1;
      }
    }
  }
}

// ---- copies of pages
// A workgroup copies kCopyEach * 256 units of 16 bytes of one pair in one cache; k, v and
// their scales count as one run of units. 40 pages of 64 tokens in 16 caches of 8 bf16 heads
// of 128: 57 us, 5.9 TB/s read and written.
template <int N>
__global__ __launch_bounds__(kCopyThreads) void copy_pages_kernel(CopyPagesParams p, CacheList<N> caches) {
  uint32_t at = blockIdx.x;
  const uint32_t chunk = at % p.chunks;
  at /= p.chunks;
  const uint32_t cache = at % (uint32_t)p.count, pair = at / (uint32_t)p.count;
  const int64_t src = p.src[pair], dst = p.dst[pair];
  if (src < 0 || src >= p.pages || dst < 0 || dst >= p.pages || src == dst) return;
  const CacheAddresses& c = caches.at[cache];
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
// their stores: they only get earlier. 64 sequences, up to 5 tokens each, 32 caches of 8 e4m3
// heads of 128: 8.5 us, 2.2 TB/s; one sequence 4: path, table and tokens follow one another
// (waits: 72 %).
constexpr int kCompactList = 64;
template <int N>
__global__ __launch_bounds__(kCompactThreads) void compact_kernel(CompactParams p, CacheList<N> caches) {
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
    base = head >= p.heads ? caches.at[cache].v : caches.at[cache].k;
    head_rows = (int64_t)(head >= p.heads ? head - p.heads : head) << p.page_shift;
  } else if (moves_scale) {
    const int head = work - units;
    base = head >= p.heads ? caches.at[cache].v_scale : caches.at[cache].k_scale;
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

CacheList<kFewCaches> few(const CacheList<kGroupCaches>& caches) {
  CacheList<kFewCaches> l;
  for (int i = 0; i < kFewCaches; ++i) l.at[i] = caches.at[i];
  return l;
}

}  // namespace

hipError_t launch_pages(const PagesParams& p, bool fork, hipStream_t stream) {
  if (fork)
    pages_kernel<true><<<1, kPagesThreads, 0, stream>>>(p);
  else
    pages_kernel<false><<<1, kPagesThreads, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_copy_pages(const CopyPagesParams& p, const CacheList<kGroupCaches>& caches, hipStream_t stream) {
  const unsigned grid = (unsigned)(p.pairs * p.count * p.chunks);
  if (p.count <= kFewCaches)
    copy_pages_kernel<<<grid, kCopyThreads, 0, stream>>>(p, few(caches));
  else
    copy_pages_kernel<<<grid, kCopyThreads, 0, stream>>>(p, caches);
  return hipGetLastError();
}

hipError_t launch_compact(const CompactParams& p, const CacheList<kGroupCaches>& caches, hipStream_t stream) {
  const unsigned grid = (unsigned)((int64_t)p.sequences * p.count * p.blocks);
  if (p.count <= kFewCaches)
    compact_kernel<<<grid, kCompactThreads, 0, stream>>>(p, few(caches));
  else
    compact_kernel<<<grid, kCompactThreads, 0, stream>>>(p, caches);
  return hipGetLastError();
}

}  // namespace w4a16
