// page_plan.cu -- the bookkeeping of a paged K/V cache on the device: pages
// given to new tokens, with the tables, lengths and slot map that the cache's
// writes and its attention take, and pages given back.
//
// A plan is two prefix sums over the sequences, of new tokens (cu_seqlens) and of
// pages needed (which entries of the stack are whose), and an expansion to rows: a
// row finds its sequence among the sums by bisection, its page from the table where the
// sequence had it already and from the stack where it is new, and the row at a
// new page's first position writes the table's entry.  Every entry is thus known without
// reading one that this call writes.
//
// Giving back is one prefix sum, of the entries of each sequence that name a page, and a
// copy of those entries.
//
// Small calls are one block, whose time is its dependent loads (lengths, then entries, then stores:
// 3 us): a second launch would cost as much again.  Large ones are memory's: the sums in one block (or, for what
// goes back, the counts in all), and a second launch that expands with every SM.
#include "internal.h"

namespace chain {
namespace {

constexpr int THREADS = 1024;     // of a block that sums
constexpr int ONE_BATCH = 1024;   // most sequences of a one-block plan: their sums lie in shared memory
constexpr int WIDE = 256;         // threads of a block that expands
constexpr int64_t ONE_ROWS = 8192;
constexpr int64_t ONE_ENTRIES = 1 << 17;

__device__ __forceinline__ void report(DevStatus *s) { atomicExch(&s->reserved[0], 1); }

// Exclusive sum of `v` over the block's threads, and the sum of all.
__device__ __forceinline__ long long block_sum(long long v, long long &all, long long *warps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  __syncthreads();  // the last call's sums are read
  if (lane == 31) warps[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < (int)(blockDim.x >> 5) ? warps[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += x;
    }
    warps[lane] = w;
  }
  __syncthreads();
  all = warps[31];
  return (warp ? warps[warp - 1] : 0) + upto - v;
}

// What rows need of a sequence beside cu_seqlens.
struct Grown {
  int len;   // cached positions before the call
  int off;   // pages given to the sequences before it
};

// Last b with cu[b] <= r, for cu[lo] <= r < cu[hi].
template <typename F>
__device__ __forceinline__ int owner(int lo, int hi, int r, const F &cu) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu(mid) <= r)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// One row: token r - first of sequence b.
__device__ __forceinline__ void put_row(const PagePlanArgs &a, int r, int b, int first, Grown g, int count) {
  const int pos = g.len + (r - first), k = pos >> a.page_shift, have = (int)(((long long)g.len + (1 << a.page_shift) - 1) >> a.page_shift);
  int page = -1;
  if (k < a.max_pages) {
    int *entry = a.table + (int64_t)b * a.table_stride + k;
    if (k < have) {
      page = *entry;
    } else {
      const int at = count - 1 - g.off - (k - have);
      if (at >= 0) page = __ldg(a.free_pages + at);
      if ((pos & ((1 << a.page_shift) - 1)) == 0) *entry = page;
    }
  }
  if (page < 0) report(a.status);
  a.positions[r] = pos;
  a.slots[r] = page < 0 ? -1 : ((long long)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// Lengths as they may be: a negative one counts as 0, one past the table as the table's end.
__device__ __forceinline__ int length_of(const PagePlanArgs &a, int b, bool &bad) {
  const int x = a.kv_lens[b], most = a.max_pages << a.page_shift;
  bad |= x < 0 || x > most;
  return x < 0 ? 0 : (x > most ? most : x);
}
__device__ __forceinline__ int new_of(const PagePlanArgs &a, int b, bool &bad) {
  const int x = a.new_lens[b];
  bad |= x < 0;
  return x < 0 ? 0 : x;
}
__device__ __forceinline__ int count_of(const int *count, int64_t capacity, bool &bad) {
  const int x = *count;
  bad |= x < 0 || x > capacity;
  return x < 0 ? 0 : (x > capacity ? (int)capacity : x);
}

// The sums; and, where WHOLE, the rows.
template <bool WHOLE>
__global__ void __launch_bounds__(THREADS, 1) plan_kernel(const PagePlanArgs a) {
  __shared__ long long warps[32];
  __shared__ int cu[WHOLE ? ONE_BATCH + 1 : 1];
  __shared__ Grown grown[WHOLE ? ONE_BATCH : 1];
  const int per = (a.batch + THREADS - 1) / THREADS;
  const int b0 = min((int64_t)threadIdx.x * per, (int64_t)a.batch), b1 = min(b0 + per, a.batch);
  bool bad = false;
  const int count = count_of(a.free_count, a.capacity, bad);
  long long n = 0, all;
  for (int b = b0; b < b1; ++b) n += new_of(a, b, bad);
  const long long before = block_sum(n, all, warps);
  const int rows = (int)min(all, (long long)a.rows);
  bad |= all > a.rows;
  // tokens behind the rows are not planned
  auto clipped = [&](long long at) { return (int)min(at, (long long)a.rows); };
  auto pages = [&](long long len) { return min((len + (1 << a.page_shift) - 1) >> a.page_shift, (long long)a.max_pages); };
  long long need = 0, at = before;
  for (int b = b0; b < b1; ++b) {
    const int x = new_of(a, b, bad), len = length_of(a, b, bad), m = clipped(at + x) - clipped(at);
    need += pages((long long)len + m) - pages(len);
    at += x;
  }
  long long given;
  long long off = block_sum(need, given, warps);
  bad |= given > count;
  at = before;
  for (int b = b0; b < b1; ++b) {
    const int x = new_of(a, b, bad), len = length_of(a, b, bad), m = clipped(at + x) - clipped(at);
    const Grown g = {len, (int)off};
    a.cu[b] = clipped(at);
    if (WHOLE) {
      cu[b] = clipped(at);
      grown[b] = g;
    } else {
      static_cast<Grown *>(a.workspace)[1 + b] = g;
    }
    off += pages((long long)len + m) - pages(len);
    a.kv_out[b] = len + m;
    at += x;
  }
  // every thread has read the count: block_sum's barriers lie between
  if (threadIdx.x == 0) {
    a.cu[a.batch] = rows;
    if (WHOLE) cu[a.batch] = rows;
    *a.count_out = (int)max((long long)count - given, 0ll);
    if (!WHOLE) static_cast<Grown *>(a.workspace)[0] = Grown{rows, count};
  }
  if (bad) report(a.status);
  if (WHOLE) {
    __syncthreads();
    for (int r = threadIdx.x; r < a.rows; r += THREADS) {
      if (r >= rows) {
        a.positions[r] = -1;
        a.slots[r] = -1;
      } else {
        const int b = owner(0, a.batch, r, [&](int i) { return cu[i]; });
        put_row(a, r, b, cu[b], grown[b], count);
      }
    }
  } else {
    pdl_launch_dependents();
  }
}

__global__ void __launch_bounds__(WIDE) rows_kernel(const PagePlanArgs a) {
  constexpr int SPAN = 4 * WIDE;  // rows of a block
  __shared__ int range[2];
  pdl_wait();
  const Grown *ws = static_cast<const Grown *>(a.workspace);
  const int rows = ws[0].len, count = ws[0].off;
  auto cu = [&](int i) { return a.cu[i]; };
  const int64_t r0 = (int64_t)blockIdx.x * SPAN;
  if (threadIdx.x < 2 && r0 < rows)  // the first row's sequence and the last one's
    range[threadIdx.x] = owner(0, a.batch, (int)min(r0 + threadIdx.x * (SPAN - 1), (int64_t)rows - 1), cu);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + i * WIDE + threadIdx.x;
    if (r >= a.rows) break;
    if (r >= rows) {
      a.positions[r] = -1;
      a.slots[r] = -1;
    } else {
      const int b = owner(range[0], range[1] + 1, (int)r, cu);
      put_row(a, (int)r, b, a.cu[b], ws[1 + b], count);
    }
  }
}

// ------------------------------------------------------------------ pages back
// A sequence's entries [first, last) go back; of those, the ones that name a page.
struct Cut {
  int first, last;
};

__device__ __forceinline__ Cut cut_of(const PageTrimArgs &a, int b, int &left, bool &bad) {
  const int most = a.max_pages << a.page_shift, up = (1 << a.page_shift) - 1;
  int len = a.kv_lens[b];
  bad |= len < 0 || len > most;
  len = len < 0 ? 0 : (len > most ? most : len);
  const int keep = a.keep[b];
  left = keep < 0 ? 0 : (keep < len ? keep : len);
  return Cut{(left + up) >> a.page_shift, (len + up) >> a.page_shift};
}

// The warp counts the entries that name a page, or puts them on the stack from `to` on.
template <bool PUT>
__device__ __forceinline__ int entries(const PageTrimArgs &a, int b, Cut c, long long to, bool &bad) {
  const int lane = threadIdx.x & 31;
  const int *table = a.table + (int64_t)b * a.table_stride;
  int n = 0;
  for (int k = c.first; k < c.last; k += 32) {
    const int x = k + lane < c.last ? table[k + lane] : -1;
    const bool is = x >= 0 && x < a.num_pages;
    const uint32_t in = __ballot_sync(0xffffffffu, is);
    if (PUT && is) {
      const long long at = to + n + __popc(in & ((1u << lane) - 1));
      if (at < a.capacity) a.free_pages[at] = x;
    }
    bad |= k + lane < c.last && !is;
    n += __popc(in);
  }
  return n;
}

// All in one block.
__global__ void __launch_bounds__(THREADS, 1) trim_kernel(const PageTrimArgs a) {
  __shared__ long long warps[32];
  __shared__ Cut cuts[ONE_BATCH];
  __shared__ int sums[ONE_BATCH];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = threadIdx.x;
  bool bad = false;
  const int count = count_of(a.free_count, a.capacity, bad);
  if (b < a.batch) {
    int left;
    cuts[b] = cut_of(a, b, left, bad);
    a.kv_out[b] = left;
  }
  __syncthreads();
  for (int i = warp; i < a.batch; i += THREADS / 32) {
    const int n = entries<false>(a, i, cuts[i], 0, bad);
    if (lane == 0) sums[i] = n;
  }
  __syncthreads();
  long long all;
  const long long before = block_sum(b < a.batch ? sums[b] : 0, all, warps);
  if (b < a.batch) sums[b] = (int)before;
  __syncthreads();
  for (int i = warp; i < a.batch; i += THREADS / 32) entries<true>(a, i, cuts[i], (long long)count + sums[i], bad);
  bad |= count + all > a.capacity;
  if (threadIdx.x == 0) *a.count_out = (int)min(count + all, (long long)a.capacity);
  if (bad) report(a.status);
}

// In two launches: a warp counts a sequence's entries, then puts them.
struct Back {
  Cut cut;
  int n;
};

__global__ void __launch_bounds__(WIDE) trim_count_kernel(const PageTrimArgs a) {
  const int b = blockIdx.x * (WIDE / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  Back *ws = static_cast<Back *>(a.workspace);
  bool bad = false;
  if (b == 0 && lane == 0) ws[0].n = count_of(a.free_count, a.capacity, bad);
  if (b < a.batch) {
    int left;
    Back x;
    x.cut = cut_of(a, b, left, bad);
    x.n = entries<false>(a, b, x.cut, 0, bad);
    if (lane == 0) {
      ws[1 + b] = x;
      a.kv_out[b] = left;
    }
  }
  if (bad) report(a.status);
  pdl_launch_dependents();
}

__global__ void __launch_bounds__(WIDE) trim_put_kernel(const PageTrimArgs a) {
  __shared__ long long warps[32];
  pdl_wait();
  const Back *ws = static_cast<const Back *>(a.workspace);
  const int b0 = blockIdx.x * (WIDE / 32), b = b0 + (threadIdx.x >> 5);
  const int count = ws[0].n;
  // entries of the sequences before the block's; block 0 takes all, for the new count
  long long n = 0, all;
  for (int i = threadIdx.x; i < (blockIdx.x ? b0 : a.batch); i += WIDE) n += ws[1 + i].n;
  block_sum(n, all, warps);
  bool bad = false;
  if (blockIdx.x == 0) {
    bad = count + all > a.capacity;
    if (threadIdx.x == 0) *a.count_out = (int)min(count + all, (long long)a.capacity);
    all = 0;
  }
  if (b < a.batch) {
    long long to = count + all;
    for (int i = b0; i < b; ++i) to += ws[1 + i].n;
    bool seen = false;  // reported by the count
    entries<true>(a, b, ws[1 + b].cut, to, seen);
  }
  if (bad) report(a.status);
}

template <typename A>
cudaError_t after(void (*kernel)(A), unsigned grid, int threads, const A &a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

size_t page_plan_workspace(int batch) { return (size_t)(batch + 1) * sizeof(Grown); }
size_t page_trim_workspace(int batch) { return (size_t)(batch + 1) * sizeof(Back); }

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t st) {
  if (a.batch <= ONE_BATCH && a.rows <= ONE_ROWS) {
    plan_kernel<true><<<1, THREADS, 0, st>>>(a);
    return cudaGetLastError();
  }
  plan_kernel<false><<<1, THREADS, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.rows == 0) return e;
  return after(rows_kernel, (unsigned)((a.rows + 4 * WIDE - 1) / (4 * WIDE)), WIDE, a, st);
}

cudaError_t launch_page_trim(const PageTrimArgs &a, cudaStream_t st) {
  if (a.batch <= ONE_BATCH && (int64_t)a.batch * a.max_pages <= ONE_ENTRIES) {
    trim_kernel<<<1, THREADS, 0, st>>>(a);
    return cudaGetLastError();
  }
  const unsigned grid = (a.batch + WIDE / 32 - 1) / (WIDE / 32);
  trim_count_kernel<<<grid, WIDE, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : after(trim_put_kernel, grid, WIDE, a, st);
}

}  // namespace chain
