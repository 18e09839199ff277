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
// graph's start).  Large plans take two launches, the sums in one block and the expansion by every SM: 64 prompts of
// 951,000 rows 10 us, 12 MB.  Trims of larger tables are a cluster's, and of the largest two launches, the counts by a
// block a sequence and then the copies: 300 sequences that give back a page or none 4.9 us, 512 that give back 366,000
// pages 5.5.
#include "internal.h"

namespace chain {
namespace {

constexpr int THREADS = 1024;     // of a block that sums
constexpr int ONE_BATCH = 1024;   // most sequences of a one-block plan: their sums lie in shared memory
constexpr int WIDE = 256;         // threads of a block that expands
// Most rows that one block takes: one block and two launches, 1,024 rows 3.5 us and 6.8, 4,096 6.2 and 7.1, 8,192 9.4 and 6.8.
constexpr int64_t ONE_ROWS = 4096;
// Entries of a table whose trim one block, a cluster, or two launches take, by what goes back in a graph, a few pages
// and all of them: 4,096 entries 3.5 and 6.1, 4.8 and 6.3, 3.6 and 3.7 us; 8,192 3.5 and 6.0, 4.8 and 6.2; 31,500 3.5 and 18.8,
// 4.8 and 6.8, 4.2 and 4.3; 128,000 3.6 and 58.8, 4.9 and 13.3, 4.8 and 5.4; 366,000 the last 3.7 and 152, 5.0 and
// 26.4, 4.8 and 5.5.  Called one by one a second launch takes 2.5 us of the host's time (5.7 and 8.2 us a call), so that
// one is preferred as long as a call that gives everything back, which is rare, stays near that.
constexpr int64_t ONE_ENTRIES = 1 << 13;
constexpr int CLUSTER = 8;  // blocks
constexpr int64_t CLUSTER_ENTRIES = 1 << 17;

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

// All in one launch, of one block or a cluster of C.  A thread takes a sequence, and their entries, laid end to end, are cut
// into one piece for each warp: whatever the mix of sequences, the warps have as much to do.  A lane finds its entry's
// sequence among the sums by bisection, and keeps it for its next entry.  Every block finds the cuts and sums by itself; what
// its piece puts on the stack it tells the others through their shared memory.
template <int C>
__global__ void __launch_bounds__(THREADS, 1) trim_kernel(const PageTrimArgs a) {
  constexpr int BATCH = 8;  // loads under way
  static_assert(C > 1 || ONE_ENTRIES <= 32 * 32 * BATCH, "a warp's piece of one block's table is one batch");
  __shared__ long long warps[32];
  __shared__ int off[ONE_BATCH + 1], shift[ONE_BATCH];  // entries before a sequence's; an entry's place less its number
  __shared__ int puts[32], totals[C];                   // entries that name a page: of the warps, of the blocks
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = threadIdx.x;
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  bool bad = false;
  const int count = count_of(a.free_count, a.capacity, bad);
  Cut c = {0, 0};
  int left = 0;
  if (b < a.batch) c = cut_of(a, b, left, bad);
  if (C > 1) cluster_sync_all();  // every block is there to be written to
  long long all;
  const int at = (int)block_sum(c.last - c.first, all, warps), end = (int)all;
  if (b < a.batch) {
    off[b] = at;
    shift[b] = c.first - at;
  }
  if (b == 0) off[a.batch] = end;
  __syncthreads();
  const int step = ((end + 32 * C - 1) / (32 * C) + 31) & ~31;
  const int lo = (int)min((long long)(rank * 32 + warp) * step, all), hi = (int)min((long long)lo + step, all);
  int x[BATCH], seq = -1;
  const int pool = (int)a.num_pages;
  auto load = [&](int e0) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int e = e0 + 32 * i + lane;
      x[i] = -1;
      if (e < hi) {
        if (seq < 0 || e >= off[seq + 1]) {  // most often the next one
          if (seq < 0 || e >= off[++seq + 1]) seq = owner(max(seq, 0), a.batch, e, [&](int s) { return off[s]; });
        }
        x[i] = a.table[(int64_t)seq * a.table_stride + shift[seq] + e];
      }
    }
  };
  auto is = [&](int i) { return x[i] >= 0 && x[i] < pool; };
  int n = 0;
  for (int e0 = lo; e0 < hi; e0 += 32 * BATCH) {
    load(e0);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      n += __popc(__ballot_sync(0xffffffffu, is(i)));
      bad |= e0 + 32 * i + lane < hi && !is(i);
    }
  }
  if (lane == 0) puts[warp] = n;
  __syncthreads();
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? puts[lane] : 0);
  int total = __reduce_add_sync(0xffffffffu, puts[lane]), base = 0;
  if (C > 1) {
    if (b < C)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&totals[rank]), b)), "r"(total) : "memory");
    cluster_sync_all();  // and every block has read the lengths and the count, which may be written in place
    const int of = lane < C ? totals[lane] : 0;
    base = __reduce_add_sync(0xffffffffu, lane < rank ? of : 0);
    total = __reduce_add_sync(0xffffffffu, of);
  }
  long long to = (long long)count + base + before;
  for (int e0 = lo; e0 < hi; e0 += 32 * BATCH) {
    if constexpr (C > 1) {
      if (step > 32 * BATCH) {  // else they are still there
        if (e0 == lo) seq = -1;
        load(e0);
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const uint32_t in = __ballot_sync(0xffffffffu, is(i));
      const long long place = to + __popc(in & ((1u << lane) - 1));
      if (is(i) && place < a.capacity) a.free_pages[place] = x[i];
      to += __popc(in);
    }
  }
  bad |= (long long)count + total > a.capacity;
  if (rank == 0) {
    if (b < a.batch) a.kv_out[b] = left;
    if (b == 0) *a.count_out = (int)min((long long)count + total, (long long)a.capacity);
  }
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
  const int64_t entries = (int64_t)a.batch * a.max_pages;
  if (a.batch <= ONE_BATCH && entries <= CLUSTER_ENTRIES) {
    cudaError_t e;
    if (entries <= ONE_ENTRIES) {
      trim_kernel<1><<<1, THREADS, 0, st>>>(a);
      e = cudaGetLastError();
    } else {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(CLUSTER);
      cfg.blockDim = dim3(THREADS);
      cfg.stream = st;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = CLUSTER;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaLaunchKernelEx(&cfg, trim_kernel<CLUSTER>, a);
    }
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
