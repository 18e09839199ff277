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
// Small calls are one block, whose time is its dependent loads (lengths, sums, entries, stores): one step of
// 512 requests 3.9 us, of one 2.7 (again and again in a graph; 9.4 and 7.3 with the second-level cache cold and a
// graph's start).  Large ones take two launches, the sums in one block (or, for what goes back, the counts in all) and
// the expansion by every SM: 64 prompts of 951,000 rows 10 us, 12 MB; 366,000 pages of 512 sequences given back 10 us
// (28 with one warp to a sequence).
#include "internal.h"

namespace chain {
namespace {

constexpr int THREADS = 1024;     // of a block that sums
constexpr int ONE_BATCH = 1024;   // most sequences of a one-block plan: their sums lie in shared memory
constexpr int WIDE = 256;         // threads of a block that expands
// Most rows, and most entries of a table, that one block takes.  Rows, one block and two launches: 1,024 3.5 us and
// 6.8, 4,096 6.2 and 7.1, 8,192 9.4 and 6.8.  Entries: where a few tokens go back 2.9 us and 4.3 at any size of the table;
// where whole sequences do, 15,600 entries 9.9 and 4.6, 64,000 20.7 and 4.1.
constexpr int64_t ONE_ROWS = 4096;
constexpr int64_t ONE_ENTRIES = 1 << 15;

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

// A stack's count as it may be.
__device__ __forceinline__ int count_of(const int *count, int64_t capacity, bool &bad) {
  const int x = *count;
  bad |= x < 0 || x > capacity;
  return x < 0 ? 0 : (x > capacity ? (int)capacity : x);
}

// The sums; and, where WHOLE, the rows.  A thread takes PER sequences and reads their lengths once, all at a time.
template <bool WHOLE, int PER>
__global__ void __launch_bounds__(THREADS, 1) plan_kernel(const PagePlanArgs a) {
  __shared__ long long warps[32];
  __shared__ int cu[WHOLE ? ONE_BATCH + 1 : 1];
  __shared__ Grown grown[WHOLE ? ONE_BATCH : 1];
  const int b0 = threadIdx.x * PER;
  bool bad = false;
  int fresh[PER], len[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    fresh[i] = b0 + i < a.batch ? a.new_lens[b0 + i] : 0;
    len[i] = b0 + i < a.batch ? a.kv_lens[b0 + i] : 0;
  }
  const int count = count_of(a.free_count, a.capacity, bad);
  const int most = a.max_pages << a.page_shift;
  long long n = 0, all, given;
#pragma unroll
  for (int i = 0; i < PER; ++i) {  // lengths as they may be
    bad |= fresh[i] < 0 || len[i] < 0 || len[i] > most;
    fresh[i] = max(fresh[i], 0);
    len[i] = min(max(len[i], 0), most);
    n += fresh[i];
  }
  long long at = block_sum(n, all, warps);
  const int rows = (int)min(all, (long long)a.rows);
  bad |= all > a.rows;
  auto pages = [&](long long x) { return min((x + (1 << a.page_shift) - 1) >> a.page_shift, (long long)a.max_pages); };
  int first[PER], pages_of[PER];
  long long need = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {  // tokens behind the rows are not planned
    first[i] = (int)min(at, (long long)a.rows);
    at += fresh[i];
    fresh[i] = (int)min(at, (long long)a.rows) - first[i];
    pages_of[i] = (int)(pages((long long)len[i] + fresh[i]) - pages(len[i]));
    need += pages_of[i];
  }
  long long off = block_sum(need, given, warps);  // its barriers lie between the reads above and the writes below
  bad |= given > count;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (b0 + i >= a.batch) break;
    const Grown g = {len[i], (int)off};
    a.cu[b0 + i] = first[i];
    a.kv_out[b0 + i] = len[i] + fresh[i];
    if (WHOLE) {
      cu[b0 + i] = first[i];
      grown[b0 + i] = g;
    } else {
      static_cast<Grown *>(a.workspace)[1 + b0 + i] = g;
    }
    off += pages_of[i];
  }
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
  // The first row's sequence and the last one's, a warp for each, 32 places at a time.
  if (threadIdx.x < 64 && r0 < rows) {
    const int end = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = (int)min(r0 + end * (SPAN - 1), (int64_t)rows - 1);
    int lo = 0, hi = a.batch;  // cu[lo] <= r < cu[hi]
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, mid = min(lo + lane * step, hi);
      const uint32_t in = __ballot_sync(0xffffffffu, mid < hi && cu(mid) <= r);
      const int k = 31 - __clz(in);  // lane 0 is always in
      hi = min(hi, lo + (k + 1) * step);
      lo += k * step;
    }
    if (lane == 0) range[end] = lo;
  }
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

// A warp counts the entries of [c.first, c.last) that name a page, or puts them on the stack from `to` on.
template <bool PUT>
__device__ __forceinline__ int entries(const PageTrimArgs &a, int b, Cut c, long long to, bool &bad) {
  constexpr int BATCH = 4;  // loads under way
  const int lane = threadIdx.x & 31;
  const int *table = a.table + (int64_t)b * a.table_stride;
  int n = 0;
  for (int k = c.first; k < c.last; k += 32 * BATCH) {
    int x[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) x[i] = k + 32 * i + lane < c.last ? table[k + 32 * i + lane] : -1;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const bool is = x[i] >= 0 && x[i] < a.num_pages;
      const uint32_t in = __ballot_sync(0xffffffffu, is);
      if (PUT && is) {
        const long long at = to + n + __popc(in & ((1u << lane) - 1));
        if (at < a.capacity) a.free_pages[at] = x[i];
      }
      bad |= k + 32 * i + lane < c.last && !is;
      n += __popc(in);
    }
  }
  return n;
}

// All in one block: a thread takes a sequence that gives back few pages, a warp one that gives back many.
__global__ void __launch_bounds__(THREADS, 1) trim_kernel(const PageTrimArgs a) {
  constexpr int FEW = 4;
  __shared__ long long warps[32];
  __shared__ Cut cuts[ONE_BATCH];
  __shared__ int sums[ONE_BATCH];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = threadIdx.x;
  bool bad = false;
  const int count = count_of(a.free_count, a.capacity, bad);
  Cut c = {0, 0};
  int x[FEW], n = 0;
  if (b < a.batch) {
    int left;
    c = cut_of(a, b, left, bad);
    a.kv_out[b] = left;
  }
  const bool few = c.last - c.first <= FEW;
#pragma unroll
  for (int i = 0; i < FEW; ++i) {
    x[i] = few && c.first + i < c.last ? a.table[(int64_t)b * a.table_stride + c.first + i] : -1;
    const bool is = x[i] >= 0 && x[i] < a.num_pages;
    bad |= few && c.first + i < c.last && !is;
    if (!is) x[i] = -1;
    n += is;
  }
  cuts[b] = c;
  const bool many = __syncthreads_or(!few);
  auto each = [&](auto &&f) {  // the sequences that a warp takes
    for (int i = warp; many && i < a.batch; i += THREADS / 32)
      if (cuts[i].last - cuts[i].first > FEW) f(i);
  };
  each([&](int i) {
    const int got = entries<false>(a, i, cuts[i], 0, bad);
    if (lane == 0) sums[i] = got;
  });
  __syncthreads();
  if (!few) n = sums[b];
  long long all;
  long long to = count + block_sum(n, all, warps);
  sums[b] = (int)(to - count);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FEW; ++i)
    if (x[i] >= 0) {
      if (to < a.capacity) a.free_pages[to] = x[i];
      ++to;
    }
  bool seen = false;  // reported by the count
  each([&](int i) { entries<true>(a, i, cuts[i], (long long)count + sums[i], seen); });
  bad |= count + all > a.capacity;
  if (threadIdx.x == 0) *a.count_out = (int)min(count + all, (long long)a.capacity);
  if (bad) report(a.status);
}

// In two launches, a block a sequence: a warp counts a piece of its entries, then puts them.
constexpr int PIECES = WIDE / 32;
struct Back {
  int n[PIECES];
};
__device__ __forceinline__ Cut piece_of(Cut c, int warp) {
  const int step = ((c.last - c.first + PIECES - 1) / PIECES + 31) & ~31;
  const int first = min(c.first + warp * step, c.last);
  return Cut{first, min(first + step, c.last)};
}
// The workspace: the count, the cut and the entries of each sequence, and those of its pieces.
struct TrimSpace {
  int *count, *sums;
  Cut *cuts;
  Back *pieces;
};
__host__ __device__ inline TrimSpace trim_space(void *p, int batch) {
  TrimSpace s;
  s.pieces = static_cast<Back *>(p);
  s.cuts = reinterpret_cast<Cut *>(s.pieces + batch);
  s.sums = reinterpret_cast<int *>(s.cuts + batch);
  s.count = s.sums + batch;
  return s;
}

__global__ void __launch_bounds__(WIDE) trim_count_kernel(const PageTrimArgs a) {
  __shared__ int sum;
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const TrimSpace ws = trim_space(a.workspace, a.batch);
  bool bad = false;
  if (threadIdx.x == 0) sum = 0;
  if (threadIdx.x == 0 && b == 0) *ws.count = count_of(a.free_count, a.capacity, bad);
  int left;
  const Cut c = cut_of(a, b, left, bad);
  __syncthreads();
  const int n = entries<false>(a, b, piece_of(c, warp), 0, bad);
  if (lane == 0) {
    ws.pieces[b].n[warp] = n;
    atomicAdd(&sum, n);
  }
  __syncthreads();  // kv_out may be kv_lens, which every warp has read
  if (threadIdx.x == 0) {
    ws.cuts[b] = c;
    ws.sums[b] = sum;
    a.kv_out[b] = left;
  }
  if (bad) report(a.status);
  pdl_launch_dependents();
}

__global__ void __launch_bounds__(WIDE) trim_put_kernel(const PageTrimArgs a) {
  __shared__ long long warps[32];
  pdl_wait();
  const TrimSpace ws = trim_space(a.workspace, a.batch);
  const int b = blockIdx.x, warp = threadIdx.x >> 5;
  const int count = *ws.count;
  // entries of the sequences before; block 0 takes all, for the new count
  long long n = 0, all;
  for (int i = threadIdx.x; i < (b ? b : a.batch); i += WIDE) n += ws.sums[i];
  const Cut c = ws.cuts[b];
  const Back back = ws.pieces[b];
  block_sum(n, all, warps);
  if (b == 0) {
    if (count + all > a.capacity) report(a.status);
    if (threadIdx.x == 0) *a.count_out = (int)min(count + all, (long long)a.capacity);
    all = 0;
  }
  long long to = count + all;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) to += i < warp ? back.n[i] : 0;
  bool seen = false;  // reported by the count
  entries<true>(a, b, piece_of(c, warp), to, seen);
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
size_t page_trim_workspace(int batch) { return (size_t)batch * (sizeof(Back) + sizeof(Cut) + sizeof(int)) + 16; }

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t st) {
  timing_mark(st, 0);
  if (a.batch <= ONE_BATCH && a.rows <= ONE_ROWS) {
    plan_kernel<true, 1><<<1, THREADS, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    timing_mark(st, 1);
    return e;
  }
  if (a.batch <= THREADS)
    plan_kernel<false, 1><<<1, THREADS, 0, st>>>(a);
  else
    plan_kernel<false, kMaxPagedBatch / THREADS><<<1, THREADS, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  timing_mark(st, 1);
  if (e != cudaSuccess || a.rows == 0) return e;
  e = after(rows_kernel, (unsigned)((a.rows + 4 * WIDE - 1) / (4 * WIDE)), WIDE, a, st);
  timing_mark(st, 2);
  return e;
}

cudaError_t launch_page_trim(const PageTrimArgs &a, cudaStream_t st) {
  timing_mark(st, 0);
  if (a.batch <= ONE_BATCH && (int64_t)a.batch * a.max_pages <= ONE_ENTRIES) {
    trim_kernel<<<1, THREADS, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    timing_mark(st, 1);
    return e;
  }
  trim_count_kernel<<<a.batch, WIDE, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  timing_mark(st, 1);
  if (e != cudaSuccess) return e;
  e = after(trim_put_kernel, a.batch, WIDE, a, st);
  timing_mark(st, 2);
  return e;
}

}  // namespace chain
