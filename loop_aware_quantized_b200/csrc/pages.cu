// Block tables and slot maps from request lengths, and pages given back, for
// sm_100a: the bookkeeping of the paged cells on the device.
//
// Both calls are a prefix sum over the requests followed by a flat expansion:
//   page_map      rows  r of the slot map: request b with start_b <= r,
//                 position len_b + r - start_b, its page from the table (the
//                 partly filled one) or from the free list (a new one; every
//                 new page holds one of the new tokens at offset 0, and the
//                 thread of that row enters it in the table);
//   page_release  pages i of the free list's new end: request b with
//                 start_b <= i, its table entry.
// Every CTA reads the lengths and does the (short) prefix sum for itself, so
// CTAs need not wait for one another, and the first one stores the new lengths
// and free count.  Where these take the old ones' place, nothing may read the
// old ones any more: a short call is one CTA and a block barrier; a long one is a
// grid that expands, and one more CTA, launched while the grid runs, that
// repeats the prefix sum, waits for the grid's end and stores (a million rows
// brought and cut again: 13.9 us a pair, 12.1 where the outputs lie elsewhere and
// the grid does it all).  So lengths are updated in place, and a call can be
// captured and replayed.  What bounds it: a short call, the launch and two
// dependent memory round trips (lengths, then free list or table), 3.4 us for 32
// requests' step and 3.1 for the release of a small batch; a long one, instructions
// (67 and 54 % of the issue slots: a search, a division and an address per row or
// page), 8.2 us for a million rows and 6.6 for half a million pages given back.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "loopkv_internal.cuh"

namespace loopkv {
namespace {

constexpr int kPageThreads = 1024;
constexpr int kPerThread = LOOPKV_MAX_PAGED_BATCH / kPageThreads;  // requests per thread at most
constexpr int kUnroll = 4;      // rows a lane looks up at a time
constexpr int kSms = 148;
constexpr int kShortWork = 256;    // rows or pages of a one-CTA call
constexpr int kShortRelease = 4096; // pages that requests may hold, of a release in place
constexpr int kLongWork = 1 << 18;  // rows or pages that take 512 threads
constexpr long long kSatRows = 0x7fffffffLL;

// Exclusive prefix sum over the block's threads; *total gets the sum.  any: the
// warp has requests (the others only need the barriers; a million rows of 256
// requests: 8.5 -> 8.2 us).
// one: the first warp has all of them, and only it gets a meaningful answer.
__device__ __forceinline__ long long block_scan(long long x, bool any, bool one, long long* warp_sums,
                                                long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long inc = x;
  if (any) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
  }
  if (one) {
    *total = __shfl_sync(0xffffffffu, inc, 31);
    return inc - x;
  }
  __syncthreads();  // the last scan's readers are done
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    long long s = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (lane < warps) warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[warps - 1];
  return (warp == 0 ? 0 : warp_sums[warp - 1]) + inc - x;
}

// Largest b in [lo, hi] with start[b] <= r (start ascends, start[lo] <= r):
// among requests without rows, which share a start, the one that has row r.
__device__ __forceinline__ int find_request(const int* start, int lo, int hi, int r) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= r) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The rows (or pages) of this warp: equal runs of whole warp widths.
struct Run {
  int begin, end;
};
__device__ __forceinline__ Run warp_run(int n) {
  const int warps = (int)(gridDim.x * (blockDim.x >> 5)), warp = (int)(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5));
  const long long share = (((long long)n + warps - 1) / warps + 31) / 32 * 32;
  const long long begin = warp * share, end = begin + share;
  return {(int)(begin < n ? begin : n), (int)(end < n ? end : n)};
}

constexpr int kFirst = 1 << 30;  // a row at offset 0 of a new page: its table index instead of the offset

struct PageParams {
  const int32_t* len;
  const int32_t* count;        // new tokens (map), new lengths (release)
  int32_t* table;
  int32_t* free;
  const int32_t* free_count;
  int32_t* slots;
  int32_t* starts;
  int32_t* newest;
  int32_t* len_out;
  int32_t* free_count_out;
  uint32_t* status;
  int32_t batch, max_pages, n_pages, n_rows;
  bool expand, finish;         // what this launch does: both, or one of them
  PageDiv div;
};

// Per request, in shared memory: start[batch + 1], then two values the
// expansion needs (map: length or -1, index into the free list of its first
// new page; release: first page given back, unused).
struct Shared {
  int* start;
  int* a;
  int* b;
};

__device__ __forceinline__ Shared shared_arrays(int* mem, int batch) {
  return {mem, mem + batch + 1, mem + 2 * batch + 1};
}

__global__ void __launch_bounds__(kPageThreads) page_map_kernel(const __grid_constant__ PageParams p) {
  extern __shared__ int mem[];
  __shared__ long long warp_sums[32];
  const Shared sh = shared_arrays(mem, p.batch);
  // The finishing launch reads the lengths before it waits, so the expanding one
  // lets it start only when what came before is done.
  if (p.expand) wait_for_previous();
  if (!p.finish) let_next_launch();
  const int tid = threadIdx.x, threads = blockDim.x, per = (p.batch + threads - 1) / threads;
  const bool any = (tid & ~31) * per < p.batch, one = p.batch <= 32;
  uint32_t status = 0;

  int len[kPerThread], add[kPerThread];
  long long rows = 0;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = tid * per + k;
    const bool in = k < per && b < p.batch;
    len[k] = in ? p.len[b] : 0;
    add[k] = in ? p.count[b] : 0;
    rows += add[k] > 0 ? add[k] : 0;
  }
  int free_count = *p.free_count;
  if (free_count < 0 || free_count > p.n_pages) {
    status |= LOOPKV_PAGE_BAD_LENGTH;
    free_count = 0;
  }
  long long all_rows, all_need;
  long long start = block_scan(rows, any, one, warp_sums, &all_rows);
  const long long capacity = (long long)p.max_pages * p.div.size;
  int need[kPerThread];
  long long sum = 0;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = tid * per + k;
    need[k] = 0;
    if (k >= per || b >= p.batch) continue;
    const long long n = add[k] > 0 ? add[k] : 0;
    uint32_t bad = 0;
    if (len[k] < 0 || add[k] < 0) bad = LOOPKV_PAGE_BAD_LENGTH;
    else if ((long long)len[k] + n > capacity) bad = LOOPKV_PAGE_NO_TABLE;
    else if (start + n > p.n_rows) bad = LOOPKV_PAGE_NO_ROWS;
    sh.start[b] = (int)(start < kSatRows ? start : kSatRows);
    start += n;
    if (bad) {
      status |= bad;
      add[k] = -1;  // refused
    } else {
      need[k] = p.div.pages(len[k] + (int)n) - p.div.pages(len[k]);
      sum += need[k];
    }
  }
  long long before = block_scan(sum, any, one, warp_sums, &all_need);
  long long taken = 0;  // pages of the admitted requests so far
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = tid * per + k;
    if (k >= per || b >= p.batch) continue;
    if (need[k] > 0 && before + need[k] > free_count) {
      status |= LOOPKV_PAGE_NO_PAGES;
      add[k] = -1;
    } else if (need[k] > 0) {
      taken = before + need[k];  // admitted requests that need pages are a prefix
    }
    sh.a[b] = add[k] < 0 ? -1 : len[k];
    sh.b[b] = (int)(free_count - 1 - before);
    before += need[k];
  }
  if (tid == 0) sh.start[p.batch] = (int)(all_rows < kSatRows ? all_rows : kSatRows);
  __syncthreads();
  const int total = sh.start[p.batch];

  const int lane = tid & 31;
  if (p.expand) {
    // Rows, a contiguous run to every warp.
    const Run run = warp_run(p.n_rows);
    const int r0 = run.begin, r1 = run.end;
    if (r0 < r1) {
      const int lo = find_request(sh.start, 0, p.batch - 1, r0);
      const int hi = find_request(sh.start, lo, p.batch - 1, r1 - 1);
      for (int r = r0 + lane; r < r1; r += 32 * kUnroll) {
        int b[kUnroll], page[kUnroll], off[kUnroll];
        bool is_new[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          const int row = r + 32 * k;
          b[k] = -1;
          if (row >= r1 || row >= total) continue;
          const int req = find_request(sh.start, lo, hi, row);
          const int n = sh.a[req];
          if (n < 0) continue;
          const int pos = n + (row - sh.start[req]);
          const int held = p.div.pages(n), j = p.div.page(pos);
          b[k] = req;
          off[k] = pos - j * p.div.size;
          is_new[k] = j >= held;
          page[k] = is_new[k] ? p.free[sh.b[req] - (j - held)] : p.table[(size_t)req * p.max_pages + j];
          if (is_new[k] && off[k] == 0) off[k] = j | kFirst;
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          const int row = r + 32 * k;
          if (row >= r1) continue;
          int slot = -1;
          if (b[k] >= 0) {
            const bool good = page[k] >= 0 && page[k] < p.n_pages, enter = (off[k] & kFirst) != 0;
            if (enter) p.table[(size_t)b[k] * p.max_pages + (off[k] & ~kFirst)] = good ? page[k] : -1;
            if (good) slot = page[k] * p.div.size + (enter ? 0 : off[k]);
            else status |= LOOPKV_PAGE_BAD_PAGE;
            if (p.newest && row + 1 == sh.start[b[k] + 1]) p.newest[b[k]] = slot;
          }
          if (p.slots) p.slots[row] = slot;
        }
      }
    }
    if (blockIdx.x == 0) {
      for (int b = tid; b <= p.batch; b += threads) {
        p.starts[b] = sh.start[b];
        // the other requests' newest slots come from the threads of their last rows
        if (p.newest && b < p.batch && (sh.a[b] < 0 || sh.start[b] == sh.start[b + 1])) p.newest[b] = -1;
      }
    }
  }
  if (status && p.status) atomicOr(p.status, status);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const long long y = __shfl_xor_sync(0xffffffffu, taken, o);
    taken = y > taken ? y : taken;
  }
  if (!p.finish || blockIdx.x != 0) return;
  if (lane == 0) warp_sums[tid >> 5] = taken;
  if (!p.expand) wait_for_previous();
  __syncthreads();  // every thread has read the lengths and the free count
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = tid * per + k;
    if (k < per && b < p.batch) p.len_out[b] = add[k] > 0 ? len[k] + add[k] : len[k];
  }
  if (tid == 0) {
    long long most = 0;
    for (int w = 0; w < threads / 32; ++w) most = warp_sums[w] > most ? warp_sums[w] : most;
    *p.free_count_out = free_count - (int)most;
  }
}

__global__ void __launch_bounds__(kPageThreads)
page_release_kernel(const __grid_constant__ PageParams p) {
  extern __shared__ int mem[];
  __shared__ long long warp_sums[32];
  const Shared sh = shared_arrays(mem, p.batch);
  // The finishing launch reads the lengths before it waits, so the expanding one
  // lets it start only when what came before is done.
  if (p.expand) wait_for_previous();
  if (!p.finish) let_next_launch();
  const int tid = threadIdx.x, threads = blockDim.x, per = (p.batch + threads - 1) / threads;
  const bool any = (tid & ~31) * per < p.batch, one = p.batch <= 32;
  uint32_t status = 0;

  int len[kPerThread], cut[kPerThread], gone[kPerThread];
  int free_count = *p.free_count, room = 0;
  if (free_count >= 0 && free_count <= p.n_pages) {
    room = p.n_pages - free_count;
  } else {
    // Nothing is pushed, and the count that is stored offers no page: where the
    // free pages are is not known, and requests may hold any of the list's.
    status |= LOOPKV_PAGE_BAD_LENGTH;
    free_count = 0;
  }
  const long long capacity = (long long)p.max_pages * p.div.size;
  long long sum = 0;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = tid * per + k;
    gone[k] = 0;
    if (k >= per || b >= p.batch) continue;
    len[k] = p.len[b];
    cut[k] = p.count[b];
    if (cut[k] < 0 || cut[k] > len[k] || len[k] > capacity) {
      status |= LOOPKV_PAGE_BAD_LENGTH;
      cut[k] = len[k];
    } else {
      gone[k] = p.div.pages(len[k]) - p.div.pages(cut[k]);
      sum += gone[k];
    }
  }
  long long all;
  long long before = block_scan(sum, any, one, warp_sums, &all);
  long long pushed = 0;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = tid * per + k;
    if (k >= per || b >= p.batch) continue;
    // refused requests start at or behind the pages pushed, where no push is made
    sh.start[b] = (int)(before < room ? before : room);
    sh.a[b] = gone[k] > 0 ? p.div.pages(cut[k]) : 0;
    before += gone[k];
    if (gone[k] > 0 && before > room) {
      status |= LOOPKV_PAGE_NO_PAGES;
      cut[k] = len[k];
    } else if (gone[k] > 0) {
      pushed = before;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const long long y = __shfl_xor_sync(0xffffffffu, pushed, o);
    pushed = y > pushed ? y : pushed;
  }
  __syncthreads();  // the scan's readers of warp_sums are done
  const int lane = tid & 31;
  if (lane == 0) warp_sums[tid >> 5] = pushed;
  __syncthreads();
  long long most = 0;
  for (int w = 0; w < threads / 32; ++w) most = warp_sums[w] > most ? warp_sums[w] : most;

  const int total = (int)most;  // pages pushed: those of the admitted requests, a prefix
  if (p.expand) {
    const Run run = warp_run(total);
    const int i0 = run.begin, i1 = run.end;
    if (i0 < i1) {
      const int lo = find_request(sh.start, 0, p.batch - 1, i0);
      const int hi = find_request(sh.start, lo, p.batch - 1, i1 - 1);
      for (int i = i0 + lane; i < i1; i += 32 * kUnroll) {
        int page[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          const int at = i + 32 * k;
          if (at >= i1) continue;
          const int b = find_request(sh.start, lo, hi, at);
          page[k] = p.table[(size_t)b * p.max_pages + sh.a[b] + (at - sh.start[b])];
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          const int at = i + 32 * k;
          if (at >= i1) continue;
          const bool good = page[k] >= 0 && page[k] < p.n_pages;
          if (!good) status |= LOOPKV_PAGE_BAD_PAGE;
          p.free[free_count + at] = good ? page[k] : -1;
        }
      }
    }
  }
  if (status && p.status) atomicOr(p.status, status);
  if (!p.finish || blockIdx.x != 0) return;
  if (!p.expand) wait_for_previous();
  __syncthreads();  // every thread has read the lengths and the free count
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = tid * per + k;
    if (k < per && b < p.batch) p.len_out[b] = cut[k];
  }
  if (tid == 0) *p.free_count_out = free_count + total;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool page_args_ok(int32_t batch, int32_t page_size, int32_t max_pages, int32_t n_pages) {
  return batch >= 1 && batch <= LOOPKV_MAX_PAGED_BATCH && page_size >= 1 &&
         page_size <= kMaxPageSize && max_pages >= 1 &&
         (long long)max_pages * page_size <= LOOPKV_MAX_PAGED_TOKENS && n_pages >= 1 &&
         (long long)n_pages * page_size < (1LL << 31);
}

// work: rows (map) or pages (release) the call may have to expand, at most; one:
// by one CTA; in_place: an output takes an input's place.  One CTA takes 256
// rows (700 rows of 30 requests: 4.3 us by one, 4.0 by a grid and a finishing
// launch, 3.4 by a grid alone; 4000 rows of 200: 6.4, 4.5 and 4.0), a release in
// place more pages, because few of those that requests may hold are given back
// by one call (60 requests of 64 pages: 2.5 us by one, 3.0 by two launches).  A
// CTA has as few threads as do (the start of one, its barriers and its idle
// warps count): 200 requests of which a few end 5.3 us with 1024 and 3.4 with 256,
// 1024 rows of 1024 requests by one CTA 6.5 with 1024, 7.0 with 256 and 5.8 with
// 512, a million rows 8.3, 8.7 and 8.2.
loopkv_status launch_pages(void (*kernel)(PageParams), PageParams p, long long work, bool one, bool in_place,
                           void* stream) {
  const int threads = p.batch > kPerThread * 512 ? kPageThreads : p.batch > 512 || work > kLongWork ? 512 : 256;
  auto shared = [](int batch) { return sizeof(int) * (3 * (size_t)batch + 1); };
  const size_t smem = shared(p.batch);
  // 48 KB less the static part need no asking
  if (smem > 40 * 1024 && !allow_shared(kernel, shared(LOOPKV_MAX_PAGED_BATCH))) return LOOPKV_ERR_CUDA;
  p.expand = true;
  p.finish = one || !in_place;
  const long long most = (long long)kSms * kPageThreads / threads;
  const long long ctas = one ? 1 : std::min<long long>((work + threads - 1) / threads, most);
  const loopkv_status rc = launch_early(kernel, dim3((unsigned)ctas), threads, smem, stream, p);
  if (rc != LOOPKV_OK || p.finish) return rc;
  p.expand = false;
  p.finish = true;
  return launch_early(kernel, dim3(1), threads, smem, stream, p);
}

}  // namespace
}  // namespace loopkv

using namespace loopkv;

extern "C" loopkv_status loopkv_page_map(int32_t batch, int32_t page_size, int32_t max_pages,
                                         int32_t n_pages, int32_t n_rows, const int32_t* d_len,
                                         const int32_t* d_new, int32_t* d_table,
                                         const int32_t* d_free, const int32_t* d_free_count,
                                         int32_t* d_slots, int32_t* d_starts, int32_t* d_newest,
                                         int32_t* d_len_out, int32_t* d_free_count_out,
                                         uint32_t* d_status, void* stream) {
  if (!page_args_ok(batch, page_size, max_pages, n_pages) || n_rows < 0 || n_rows > (1 << 30))
    return LOOPKV_ERR_INVALID_ARG;
  const void* ptrs[8] = {d_len, d_new, d_table, d_free, d_free_count, d_starts, d_len_out,
                         d_free_count_out};
  for (const void* ptr : ptrs)
    if (ptr == nullptr || !aligned4(ptr)) return LOOPKV_ERR_INVALID_ARG;
  if (!aligned4(d_slots) || !aligned4(d_newest) || !aligned4(d_status)) return LOOPKV_ERR_INVALID_ARG;
  if (d_len_out == d_new) return LOOPKV_ERR_INVALID_ARG;  // (every block reads the counts)
  PageParams p{};
  p.len = d_len;
  p.count = d_new;
  p.table = d_table;
  p.free = const_cast<int32_t*>(d_free);
  p.free_count = d_free_count;
  p.slots = d_slots;
  p.starts = d_starts;
  p.newest = d_newest;
  p.len_out = d_len_out;
  p.free_count_out = d_free_count_out;
  p.status = d_status;
  p.batch = batch;
  p.max_pages = max_pages;
  p.n_pages = n_pages;
  p.n_rows = n_rows;
  p.div = PageDiv(page_size);
  return launch_pages(page_map_kernel, p, n_rows, n_rows <= kShortWork, d_len_out == d_len || d_free_count_out == d_free_count, stream);
}

extern "C" loopkv_status loopkv_page_release(int32_t batch, int32_t page_size, int32_t max_pages,
                                             int32_t n_pages, const int32_t* d_len,
                                             const int32_t* d_new_len, const int32_t* d_table,
                                             int32_t* d_free, const int32_t* d_free_count,
                                             int32_t* d_len_out, int32_t* d_free_count_out,
                                             uint32_t* d_status, void* stream) {
  if (!page_args_ok(batch, page_size, max_pages, n_pages)) return LOOPKV_ERR_INVALID_ARG;
  const void* ptrs[7] = {d_len, d_new_len, d_table, d_free, d_free_count, d_len_out,
                         d_free_count_out};
  for (const void* ptr : ptrs)
    if (ptr == nullptr || !aligned4(ptr)) return LOOPKV_ERR_INVALID_ARG;
  if (!aligned4(d_status)) return LOOPKV_ERR_INVALID_ARG;
  PageParams p{};
  p.len = d_len;
  p.count = d_new_len;
  p.table = const_cast<int32_t*>(d_table);
  p.free = d_free;
  p.free_count = d_free_count;
  p.len_out = d_len_out;
  p.free_count_out = d_free_count_out;
  p.status = d_status;
  p.batch = batch;
  p.max_pages = max_pages;
  p.n_pages = n_pages;
  p.div = PageDiv(page_size);
  const long long most = std::min<long long>((long long)batch * max_pages, n_pages);
  const bool in_place = d_len_out == d_len || d_len_out == d_new_len || d_free_count_out == d_free_count;
  return launch_pages(page_release_kernel, p, most, most <= (in_place ? kShortRelease : kShortWork), in_place, stream);
}
