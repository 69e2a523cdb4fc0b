// page_plan.cu — block table, slot map and positions of a step, from request
// lengths on the device; and the return of finished requests' pages.
//
// With page size P, request r of old length l and n new tokens needs
//     need_r = ceil((l + n) / P) - ceil(l / P)
// further pages.  Let c_r be the inclusive sum of the needs.  The free pages
// are a stack; request r takes its pages at depth c_r - need_r, so the result
// depends on the request order alone.  r is served iff it fits its table row
// and (n > 0) the slot rows, and need_r = 0 or c_r <= free: the sums never fall, so the
// served takers are a prefix and their stack ranges do not overlap.
//
// Bound by latency: a step of 64 requests moves 2 KB.  One CTA does the sums
// and all state, a row of requests per pass, and with few slot rows also writes
// those and the new table entries, since a thread holds what its request
// needs.  With many (prompts), all SMs write rows and entries: each CTA adds up
// the requests itself, or, with more than it keeps or with outputs in place, a
// second kernel takes them from the first's outputs and the workspace.
// Measured: 64 requests 2.6 us; 517 requests with 268k slot rows 6.8 us (29 us
// by one CTA, 8.5 by two kernels).
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "diffattn.h"
#include "kernels.h"
#include "kv4.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kMaxRequests = 1 << 16;

struct PlanArgs {
  const int* new_lens;
  const int* lens;
  int* table;
  const int* stack;
  const int* count;
  int requests, max_pages, page_shift, n_pages, n_slots;
  int* slots;
  int* positions;
  int* offsets;
  int* served;
  int* lens_out;
  int* count_out;
  int* depth;  // [requests], for the second kernel
  int* dev_status;
};

// Inclusive sum over the block of one value per thread; `total` gets the sum.
// `sh` holds 33 values; every thread of the block calls it.
__device__ long long block_scan(long long x, long long* sh, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();  // the previous use of sh is over
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int n = (int)(blockDim.x >> 5);
    long long y = lane < n ? sh[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long z = __shfl_up_sync(0xffffffffu, y, off);
      if (lane >= off) y += z;
    }
    sh[lane] = y;
  }
  __syncthreads();
  total = sh[(blockDim.x >> 5) - 1];
  return x + (warp ? sh[warp - 1] : 0);
}

// Slot of a position on a page; -1, and `bad` set, if it is no page.
__device__ __forceinline__ int slot_of(const PlanArgs& a, int page, int pos, bool& bad) {
  if ((unsigned)page >= (unsigned)a.n_pages) {
    bad = true;
    return -1;
  }
  return (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

__device__ __forceinline__ int free_pages_of(const PlanArgs& a) {
  const int n = *a.count;
  return n < 0 ? 0 : (n > a.n_pages ? a.n_pages : n);
}
__device__ __forceinline__ int clamped(long long x) { return (int)(x < INT_MAX ? x : INT_MAX); }

// What request r gets; the block's threads take a row of requests together.
struct Share {
  bool live, ok;
  int n, len, old, need;
  long long at, end;  // slot rows [at, end)
  long long upto;     // pages asked for by it and those before
};
__device__ __forceinline__ Share share_of(const PlanArgs& a, int r, int free0, long long* sh,
                                          long long& tok_base, long long& need_base) {
  const int ps = 1 << a.page_shift;
  Share s;
  s.live = r < a.requests;
  s.n = s.live ? max(a.new_lens[r], 0) : 0;
  s.len = s.live ? max(a.lens[r], 0) : 0;
  long long total;
  s.end = tok_base + block_scan(s.n, sh, total);
  tok_base += total;
  s.at = s.end - s.n;
  const long long after = (long long)s.len + s.n;
  const bool fits = s.live && after <= (long long)a.max_pages << a.page_shift &&
                    (s.n == 0 || s.end <= a.n_slots);
  s.old = fits ? (int)(((long long)s.len + ps - 1) >> a.page_shift) : 0;
  s.need = fits ? (int)((after + ps - 1) >> a.page_shift) - s.old : 0;
  s.upto = need_base + block_scan(s.need, sh, total);
  need_base += total;
  s.ok = fits && (s.need == 0 || s.upto <= free0);
  return s;
}
// The request's outputs; `taken`: the most pages a served request reaches down to.
__device__ __forceinline__ void put_share(const PlanArgs& a, int r, const Share& s, int& taken,
                                          bool& refused) {
  if (s.ok && s.need) taken = max(taken, (int)s.upto);
  refused |= s.live && !s.ok;
  if (!s.live) return;
  a.offsets[r] = clamped(s.at);
  if (r == a.requests - 1) a.offsets[r + 1] = clamped(s.end);
  a.served[r] = s.ok ? 1 : 0;
  a.lens_out[r] = s.ok ? s.len + s.n : s.len;
}
// The pages left, and what went wrong; the whole block calls it.
__device__ __forceinline__ void put_count(const PlanArgs& a, int free0, int taken, bool refused,
                                          long long* sh) {
  taken = __reduce_max_sync(0xffffffffu, taken);
  __syncthreads();
  int* top = reinterpret_cast<int*>(sh);
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = taken;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) taken = max(taken, top[w]);
    *a.count_out = free0 - taken;
  }
  if (refused) report(a.dev_status, DA_ERR_CACHE_FULL);
}

// `with_slots`: this launch writes the slot rows and table entries too.
__global__ void __launch_bounds__(1024, 1) page_plan_kernel(const PlanArgs a, int with_slots) {
  __shared__ long long sh[33];
  let_next_start();
  after_previous();
  const int tid = threadIdx.x, lane = tid & 31;
  const int free0 = free_pages_of(a);
  long long tok_base = 0, need_base = 0;
  int taken = 0;
  bool refused = false, bad = false;
  for (int base = 0; base < a.requests; base += (int)blockDim.x) {
    const int r = base + tid;
    const Share s = share_of(a, r, free0, sh, tok_base, need_base);
    put_share(a, r, s, taken, refused);
    if (s.live && !with_slots) a.depth[r] = s.ok && s.need ? (int)(free0 - s.upto + s.need) : 0;
    const int len = s.len, old = s.old;
    const long long tok_at = s.at;
    const bool ok = s.ok;
    // New table entries and slot rows: a thread writes its own request's when
    // they are few, else its whole warp does, one request at a time.
    const int depth = (int)(s.upto - s.need);
    const int rows = with_slots && s.live && tok_at < a.n_slots
                         ? (int)(s.end < a.n_slots ? s.n : a.n_slots - tok_at) : 0;
    const int pages = with_slots && ok ? s.need : 0;
    const bool many = pages > 2 || rows > 2;
    int* row = a.table + (size_t)(s.live ? r : 0) * a.max_pages;
    if (!many) {
      for (int j = 0; j < pages; ++j) row[old + j] = a.stack[free0 - 1 - (depth + j)];
      for (int j = 0; j < rows; ++j) {
        const int pos = (int)((unsigned)len + (unsigned)j), blk = pos >> a.page_shift;
        int slot = -1;
        if (ok)
          slot = slot_of(a, blk < old ? row[blk] : a.stack[free0 - 1 - (depth + blk - old)], pos,
                         bad);
        a.slots[tok_at + j] = slot;
        a.positions[tok_at + j] = pos;
      }
    }
    unsigned todo = __ballot_sync(0xffffffffu, many);
    while (todo) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const int w_pages = __shfl_sync(0xffffffffu, pages, src);
      const int w_rows = __shfl_sync(0xffffffffu, rows, src);
      const int w_old = __shfl_sync(0xffffffffu, old, src);
      const int w_depth = __shfl_sync(0xffffffffu, depth, src);
      const int w_len = __shfl_sync(0xffffffffu, len, src);
      const int w_ok = __shfl_sync(0xffffffffu, (int)ok, src);
      const long long w_at = __shfl_sync(0xffffffffu, tok_at, src);
      int* w_row = a.table + (size_t)(base + tid - lane + src) * a.max_pages;
      for (int j = lane; j < w_pages; j += 32)
        w_row[w_old + j] = a.stack[free0 - 1 - (w_depth + j)];
      for (int j = lane; j < w_rows; j += 32) {
        const int pos = (int)((unsigned)w_len + (unsigned)j), blk = pos >> a.page_shift;
        int slot = -1;
        if (w_ok)
          slot = slot_of(
              a, blk < w_old ? w_row[blk] : a.stack[free0 - 1 - (w_depth + blk - w_old)], pos,
              bad);
        a.slots[w_at + j] = slot;
        a.positions[w_at + j] = pos;
      }
    }
  }
  if (with_slots) {  // rows behind the last token
    for (long long i = tok_base + tid; i < a.n_slots; i += blockDim.x) {
      a.slots[i] = -1;
      a.positions[i] = 0;
    }
  }
  put_count(a, free0, taken, refused, sh);
  if (bad) report(a.dev_status, DA_ERR_PAGE);
}

// Slot rows of a large step: each is bisected for its request.  The row that
// begins a new page writes its table entry: a new page's first position is a
// new token's.
constexpr int kFillRows = 1024;  // of a CTA

struct Request {
  int offset, len, depth;  // the first new page lies below stack[depth]; < 0: not served
};

// Last r in [lo, hi] whose offset is at most i.
template <typename F>
__device__ __forceinline__ int upper_request(F offset, int lo, int hi, int i) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offset(mid) <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int fill_row(const PlanArgs& a, int i, int r, const Request& q,
                                        int& pos, bool& bad) {
  const int mask = (1 << a.page_shift) - 1;
  pos = (int)((unsigned)q.len + (unsigned)(i - q.offset));
  if (q.depth < 0) return -1;
  const int blk = pos >> a.page_shift;
  const int old = (int)(((unsigned)q.len + (unsigned)mask) >> a.page_shift);
  int* entry = a.table + (size_t)r * a.max_pages + blk;
  int page;
  if (blk < old) {
    page = *entry;
  } else {
    page = a.stack[q.depth - 1 - (blk - old)];
    if ((pos & mask) == 0) *entry = page;
  }
  return slot_of(a, page, pos, bad);
}

// One launch for large steps of up to kWideRequests requests: every CTA adds up
// the requests itself (1 us) and keeps them in shared memory for its rows; the
// first writes the requests' outputs.  Those must not be the inputs, which the
// other CTAs may still read.
constexpr int kWideRequests = 2048;

__global__ void __launch_bounds__(1024) page_plan_wide_kernel(const PlanArgs a) {
  __shared__ long long sh[33];
  __shared__ Request keep[kWideRequests];
  let_next_start();
  after_previous();
  const int free0 = free_pages_of(a);
  long long tok_base = 0, need_base = 0;
  int taken = 0;
  bool refused = false, bad = false;
  for (int base = 0; base < a.requests; base += (int)blockDim.x) {
    const int r = base + (int)threadIdx.x;
    const Share s = share_of(a, r, free0, sh, tok_base, need_base);
    if (s.live)
      keep[r] = {clamped(s.at), s.len,
                 !s.ok ? -1 : s.need ? (int)(free0 - s.upto + s.need) : 0};
    if (blockIdx.x == 0) put_share(a, r, s, taken, refused);
  }
  if (blockIdx.x == 0) put_count(a, free0, taken, refused, sh);
  __syncthreads();
  const int first = (int)blockIdx.x * kFillRows;
  const int last = min(first + kFillRows, a.n_slots) - 1;
  auto offset = [&](int r) { return keep[r].offset; };
  const int lo = upper_request(offset, 0, a.requests - 1, first);
  const int hi = upper_request(offset, lo, a.requests - 1, last);
  for (int i = first + (int)threadIdx.x; i <= last; i += (int)blockDim.x) {
    int slot = -1, pos = 0;
    if (i < tok_base) {
      const int r = upper_request(offset, lo, hi, i);
      slot = fill_row(a, i, r, keep[r], pos, bad);
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
  if (bad) report(a.dev_status, DA_ERR_PAGE);
}

// The same rows after page_plan_kernel, for more requests or outputs in place: a
// CTA finds its requests in the written offsets and, if they are few, keeps
// what it needs of them in shared memory.
constexpr int kFillThreads = 256;
constexpr int kFillKeep = 1536;

__device__ __forceinline__ Request request_of(const PlanArgs& a, int r) {
  const int n = a.new_lens[r], ok = a.served[r];
  return {a.offsets[r], (int)((unsigned)a.lens_out[r] - (unsigned)(ok && n > 0 ? n : 0)),
          ok ? a.depth[r] : -1};
}

__global__ void __launch_bounds__(kFillThreads) page_slots_kernel(const PlanArgs a) {
  __shared__ int ends[2];
  __shared__ Request keep[kFillKeep];
  let_next_start();
  after_previous();
  const int first = blockIdx.x * kFillRows;
  const int last = min(first + kFillRows, a.n_slots) - 1;
  auto global = [&](int r) { return a.offsets[r]; };
  if (threadIdx.x < 2)
    ends[threadIdx.x] = upper_request(global, 0, a.requests - 1, threadIdx.x ? last : first);
  __syncthreads();
  const int lo = ends[0], hi = ends[1];
  const bool kept = hi - lo < kFillKeep;
  if (kept)
    for (int r = lo + threadIdx.x; r <= hi; r += kFillThreads) keep[r - lo] = request_of(a, r);
  __syncthreads();
  const int total = a.offsets[a.requests];
  bool bad = false;
  for (int i = first + threadIdx.x; i <= last; i += kFillThreads) {
    int slot = -1, pos = 0;
    if (i < total) {
      const int r = kept ? lo + upper_request([&](int k) { return keep[k].offset; }, 0, hi - lo, i)
                         : upper_request(global, lo, hi, i);
      slot = fill_row(a, i, r, kept ? keep[r - lo] : request_of(a, r), pos, bad);
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
  if (bad) report(a.dev_status, DA_ERR_PAGE);
}

// Pages of the released requests go back on the stack in request order.
struct ReleaseArgs {
  const int* release;
  int* lens;
  int* table;
  int* stack;
  int* count;
  int requests, max_pages, page_shift, n_pages;
  int* dev_status;
};

__global__ void __launch_bounds__(1024) page_release_kernel(const ReleaseArgs a) {
  __shared__ long long sh[33];
  let_next_start();
  after_previous();
  const int tid = threadIdx.x, lane = tid & 31;
  const int ps = 1 << a.page_shift;
  int free0 = *a.count;
  free0 = free0 < 0 ? 0 : (free0 > a.n_pages ? a.n_pages : free0);
  long long at_base = free0;
  bool bad = false;
  for (int base = 0; base < a.requests; base += (int)blockDim.x) {
    const int r = base + tid;
    const bool out = r < a.requests && a.release[r] != 0;
    int pages = 0;
    if (out) {
      const int len = a.lens[r];
      const long long p = len > 0 ? ((long long)len + ps - 1) >> a.page_shift : 0;
      pages = (int)(p < a.max_pages ? p : a.max_pages);
      a.lens[r] = 0;
    }
    // A warp takes its requests one at a time: first it counts the entries
    // that are pages (others are left out), then it moves them.
    int good = 0;
    for (unsigned todo = __ballot_sync(0xffffffffu, pages > 0); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int n = __shfl_sync(0xffffffffu, pages, src);
      const int* mine = a.table + (size_t)(base + tid - lane + src) * a.max_pages;
      int c = 0;
      for (int j = lane; j < n; j += 32) c += (unsigned)mine[j] < (unsigned)a.n_pages;
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == src) good = c;
    }
    bad |= good < pages;
    long long total;
    const long long at = at_base + block_scan(good, sh, total) - good;
    for (unsigned todo = __ballot_sync(0xffffffffu, pages > 0); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int n = __shfl_sync(0xffffffffu, pages, src);
      long long to = __shfl_sync(0xffffffffu, at, src);
      int* row = a.table + (size_t)(base + tid - lane + src) * a.max_pages;
      for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        const int page = j < n ? row[j] : -1;
        if (j < n) row[j] = -1;
        const bool ok = (unsigned)page < (unsigned)a.n_pages;
        const unsigned put = __ballot_sync(0xffffffffu, ok);
        const long long where = to + __popc(put & ((1u << lane) - 1u));
        if (ok && where < a.n_pages) a.stack[where] = page;
        bad |= ok && where >= a.n_pages;
        to += __popc(put);
      }
    }
    at_base += total;
  }
  if (tid == 0) *a.count = (int)(at_base < a.n_pages ? at_base : a.n_pages);
  if (bad) report(a.dev_status, DA_ERR_PAGE);
}

int threads_for(int requests) {
  int t = 32;
  while (t < requests && t < 1024) t <<= 1;
  return t;
}

int check(int requests, int max_pages, int n_pages, int page_size) {
  if (requests < 1 || max_pages < 1 || n_pages < 1 || page_size < 1) return DA_ERR_INVALID_ARG;
  if (!kv4_page_size_ok(page_size) || requests > kMaxRequests) return DA_ERR_UNSUPPORTED;
  if ((long long)n_pages * page_size >= (1LL << 31) ||
      (long long)max_pages * page_size >= (1LL << 31))
    return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

// Whether the one CTA of the plan writes the slot rows itself: few of them for
// each request (a decode step, with spare rows).  Measured (one CTA, all SMs):
// 64 requests and 64 rows 2.6 and 3.6 us, 256 rows 2.9 and 3.8, 1024 rows 5.7
// and 4.3, 12864 rows 27 and 4.1; 512 requests and 1024 rows 3.4 and 4.4; 1500
// requests and 6500 rows 6.9 and 7.7.
bool one_cta(int requests, int n_slots) {
  return n_slots <= 16384 && n_slots <= 256 + 4LL * requests;
}

}  // namespace
}  // namespace da

extern "C" size_t diffattn_page_plan_workspace_size(int requests, int n_slots) {
  if (requests < 1 || da::one_cta(requests, n_slots)) return 0;
  return (size_t)requests * sizeof(int);
}

extern "C" int diffattn_page_plan(const int* new_lens, const int* cache_lens, int* block_table,
                                  const int* free_pages, const int* free_count, int requests,
                                  int max_pages, int n_pages, int page_size, int n_slots,
                                  int* slots, int* positions, int* offsets, int* served,
                                  int* cache_lens_out, int* free_count_out, void* workspace,
                                  size_t workspace_bytes, int* dev_status, void* stream) {
  if (!new_lens || !cache_lens || !block_table || !free_pages || !free_count || !offsets ||
      !served || !cache_lens_out || !free_count_out)
    return DA_ERR_INVALID_ARG;
  if (n_slots < 0 || (n_slots > 0 && (!slots || !positions))) return DA_ERR_INVALID_ARG;
  const int st = da::check(requests, max_pages, n_pages, page_size);
  if (st != DA_OK) return st;
  if (n_slots > (1 << 30)) return DA_ERR_UNSUPPORTED;
  const size_t need = diffattn_page_plan_workspace_size(requests, n_slots);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DA_ERR_WORKSPACE;
  if (need > 0 && reinterpret_cast<uintptr_t>(workspace) % sizeof(int)) return DA_ERR_ALIGNMENT;
  da::PlanArgs a{};
  a.new_lens = new_lens;
  a.lens = cache_lens;
  a.table = block_table;
  a.stack = free_pages;
  a.count = free_count;
  a.requests = requests;
  a.max_pages = max_pages;
  a.page_shift = da::kv4_shift(page_size);
  a.n_pages = n_pages;
  a.n_slots = n_slots;
  a.slots = slots;
  a.positions = positions;
  a.offsets = offsets;
  a.served = served;
  a.lens_out = cache_lens_out;
  a.count_out = free_count_out;
  a.depth = static_cast<int*>(workspace);
  a.dev_status = dev_status;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const dim3 fill((unsigned)((n_slots + da::kFillRows - 1) / da::kFillRows));
  if (need > 0 && requests <= da::kWideRequests && cache_lens_out != cache_lens &&
      free_count_out != free_count)
    return da::launch_after(da::page_plan_wide_kernel, fill, requests <= 512 ? 512 : 1024, 0, cs, a) ==
                   cudaSuccess
               ? DA_OK
               : DA_ERR_CUDA;
  if (da::launch_after(da::page_plan_kernel, dim3(1), da::threads_for(requests), 0, cs, a,
                       (int)(need == 0)) != cudaSuccess)
    return DA_ERR_CUDA;
  if (need > 0 && da::launch_after(da::page_slots_kernel, fill, da::kFillThreads, 0, cs, a) !=
                      cudaSuccess)
    return DA_ERR_CUDA;
  return DA_OK;
}

extern "C" int diffattn_page_release(const int* release, int* cache_lens, int* block_table,
                                     int* free_pages, int* free_count, int requests,
                                     int max_pages, int n_pages, int page_size, int* dev_status,
                                     void* stream) {
  if (!release || !cache_lens || !block_table || !free_pages || !free_count)
    return DA_ERR_INVALID_ARG;
  const int st = da::check(requests, max_pages, n_pages, page_size);
  if (st != DA_OK) return st;
  da::ReleaseArgs a{};
  a.release = release;
  a.lens = cache_lens;
  a.table = block_table;
  a.stack = free_pages;
  a.count = free_count;
  a.requests = requests;
  a.max_pages = max_pages;
  a.page_shift = da::kv4_shift(page_size);
  a.n_pages = n_pages;
  a.dev_status = dev_status;
  return da::launch_after(da::page_release_kernel, dim3(1), da::threads_for(requests), 0,
                          static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? DA_OK
             : DA_ERR_CUDA;
}
