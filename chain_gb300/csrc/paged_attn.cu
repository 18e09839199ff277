// paged_attn.cu -- softmax attention of a chunk of new tokens over a paged
// K/V cache (the unit O = f(A B) C with f = row softmax, K and V read from
// the pages that a sequence's table names).
//
// New token i of sequence b, with n_b new tokens and lens[b] cached
// positions (the new ones included), sees the keys j < lens[b], and of those
// only j <= lens[b] - n_b + i under the causal mask.  A row that sees none
// gets O = 0 and LSE = -inf.
//
// Rows.  The G = H / Hkv query heads of a K/V head share its keys, so a
// 128-row query tile holds TPT = floor(128 / G) tokens times G heads (row
// = token * G + head): one token of grouped heads reads each cached key
// once.  A unit of work is one sequence, one K/V head and up to two tiles
// (2 TPT tokens), over the 128-key tiles its last token sees.
//
// Split.  The lengths are on the device, so the work is dealt there: the
// units' costs (key tiles), laid end to end, are cut into one equal run for
// each of the CTAS persistent blocks, whatever the mix of lengths.  A block works
// through the units of its run; a unit cut by a run's end leaves partial
// (O, m, l) in the workspace, which paged_combine_kernel joins.  A block has
// at most two partial units, the first and the last of its run.
//
// Inside a block (384 threads, one block an SM):
//   warps 0-3, 4-7  softmax of streams 0 and 1, one row a thread, as in the
//              forward kernels: S from tensor memory, running maximum and sum in
//              fp32, P back into S's columns as a pair of bf16, P_hi = bf16(P) and P_lo =
//              bf16(P - P_hi), O rescaled only when the maximum grew by 2^8.  One bf16
//              of P would add as much error to O as O's own rounding does, at any number of
//              keys (sum|O - ref| / sum|ref| 2.1e-3 to 2.2e-3, above the library's bound of 2e-3;
//              1.4e-3 with the pair).  l sums the unrounded P.
//   warp 8     TMA producer: Q tiles, then K and V tiles through one ring of
//              NS tile slots in the order K0 V0 K1 V1 ...; a tile of 128 keys is
//              128 / page boxes, their pages looked up one tile ahead, one lane a box.
//   warp 9     MMA issuer.
//   warp 10    scheduler: finds the run's units and hands them to the other
//              warps through a small ring.
// Two streams share the tensor core, so that one multiplies while the other
// exponentiates.  With more than TPT tokens the streams are the unit's two
// query tiles over the same keys; with fewer (single tokens, short chunks) they are
// its even and odd key tiles for one query tile, joined before the store.
//
// Calls of single tokens go to paged_token_kernel, further down, which shares the split.
//
// Bounds, and what was measured (32 heads on 8, pages of 64 to 128):
//   chunks: the chain of softmax and products.  d = 128, 2,048 tokens over 32,768: 1,090 us,
//   980 TFLOP/s (P_lo's product not counted; 775 us with one bf16 of P), the tensor pipe 61% busy: a
//   stream's softmax and its three products follow each other, since P shares S's columns; two
//   streams overlap them.  d = 64: 765 us, 700 TFLOP/s, the tensor pipe 39% busy.
//   single tokens: memory.  d = 128, 64 sequences of 8,192: 363 us, 2.15 GB at 5.9 TB/s;
//   d = 64: 196 us, 1.07 GB at 5.5 TB/s.  One sequence of 131,072: 99 us, 5.4 TB/s, with
//   the start, the join and the ends of the runs; of 100: 6.4 us, all latency.
#include <atomic>

#include "internal.h"

namespace chain {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int CTAS = 152;     // one block on each SM
constexpr int THREADS = 384;
constexpr int NU = 4;         // units in flight between the scheduler and the other warps
constexpr int MAX_BATCH = 8192;
constexpr uint32_t REGS_SOFTMAX = 184, REGS_CONTROL = 136;  // 256 x 184 + 128 x 136 = 384 x 168
constexpr float RESCALE_THRESHOLD = 8.0f;                   // log2 units

enum : int {
  SITE_PAGED_PROD = 0x601,
  SITE_PAGED_MMA = 0x602,
  SITE_PAGED_SOFTMAX = 0x603,
  SITE_PAGED_EPI = 0x604,
  SITE_PAGED_SCHED = 0x605,
  SITE_PAGED_DRAIN = 0x606
};

// One unit's part of a block's run, as the scheduler hands it over.
struct Unit {
  int tok0, ntok;  // packed rows
  int head, b;     // K/V head (-1: no more units), sequence
  int j0, j1;      // key tiles
  int ja;          // end of the key tiles that tile 0 sees
  int lim0;        // keys that the first token sees (any value up to len)
  int len;         // keys of the sequence
  int slot;        // -1: all of the unit's key tiles, else the workspace slot
};
static_assert(sizeof(Unit) <= 48, "unit ring");

// Where a run begins, for the join: written by every block, cut or not.
struct Boundary {
  long long u0;     // cost at which the unit that it falls into begins
  long long total;  // cost of all units
  int nt, w;        // the unit's key tiles, cost of each
  int cut;          // it falls behind the unit's first key tile
  int tok0, ntok, head;
};

template <int D>
struct Layout {
  static constexpr uint32_t TILE = BM * D * 2;  // a Q, K or V tile
  static constexpr int NS = D == 128 ? 5 : 12;  // 160 or 192 KB of K and V in flight
  // Costs, in quarters of a key tile against one query tile, chosen by time over mixed batches (24
  // chunks and tokens of up to 300 over up to 5,000 keys, 32 heads of 128 on 8 / 15 of 64 on 5: 278 us /
  // 123 us; with 5, 14 / 6, 20 for the last two 296 / 125, with 6, 9 / 7, 12 284 / 130).  The last is a
  // unit's start and end, raised, as dearer units leave fewer of them cut and joined.
  static constexpr int COST1 = 4, COST2 = D == 128 ? 6 : 7, OVERHEAD = D == 128 ? 20 : 28;
  // Tensor memory: S0 [0,128), S1 [128,256), O0 [256,384), O1 [384,512).  P overwrites S: keys
  // [16g, 16g + 16) take columns [16g, 16g + 8) (P_hi) and [16g + 8, 16g + 16) (P_lo).
  static __host__ __device__ constexpr uint32_t o_col(int t) { return 256 + 128 * t; }
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_RING = 2 * TILE;
  static constexpr uint32_t OFF_BAR = OFF_RING + NS * TILE;
  // q_full[2], q_empty[2], full[NS], empty[NS], s_full[2], p_ready[2],
  // pv_done[2], u_full[NU], u_empty[NU], joined[2], drain
  static constexpr uint32_t NBAR = 4 + 2 * NS + 6 + 2 * NU + 2 + 1;
  static constexpr uint32_t OFF_UNITS = (OFF_BAR + NBAR * 8 + 15) & ~15u;
  static constexpr uint32_t OFF_ML = OFF_UNITS + NU * 48;
  static constexpr uint32_t OFF_MISC = OFF_ML + BM * 8;
  static constexpr uint32_t BYTES = OFF_MISC + 16;
  static constexpr uint32_t ALLOC = BYTES + 1024;
  static_assert(ALLOC <= 232448, "shared memory");
  static_assert(MAX_BATCH * 8 <= NS * TILE, "the schedule's sums use the ring");
};

struct Params {
  PagedSeqs s;
  int total, G, Hkv, causal;
  int above, upto;             // new tokens of the sequences that this launch serves: above < n <= upto
  int tpt, utok;               // tokens of a query tile, of a unit
  int cost1, cost2, overhead;  // of a key tile against one and two query tiles, of a unit
  float scale_log2;
  __nv_bfloat16 *O;
  int64_t o_stok, o_shead;
  float *LSE;
  int64_t lse_shead;
  float *part_o;   // [CTAS][2][D / 4][2 BM][4]
  float2 *part_ml; // [CTAS][2][2 BM]
  Boundary *bounds;
  // for the kernel of few rows, which makes its own copies
  const __nv_bfloat16 *Q;
  int64_t q_stok, q_shead;
  PagedSide kc, vc;
  WaitCfg wc;
};

__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity, const WaitCfg &wc) {
  volatile int never = 0;
  mbar_wait(bar, parity, wc, &never, SITE_PAGED_DRAIN);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// Each lane holds 64 bytes of its own row and `at`, their place in memory.
// Four lanes exchange 16-byte chunks, so that one store writes 64 bytes of each of
// eight rows: a lane storing its own row would touch 32 lines an instruction,
// and the stores of a tile took 4,000 cycles.
__device__ __forceinline__ void store_rows(uint4 (&v)[4], __nv_bfloat16 *at, bool valid, int lane) {
  auto trade = [&](uint4 &a, uint4 &b, int bit) {
    // of a pair of lanes, the lower one keeps a and the upper one b
    const bool up = lane & bit;
    uint4 give = up ? a : b;
    give.x = __shfl_xor_sync(0xffffffffu, give.x, bit);
    give.y = __shfl_xor_sync(0xffffffffu, give.y, bit);
    give.z = __shfl_xor_sync(0xffffffffu, give.z, bit);
    give.w = __shfl_xor_sync(0xffffffffu, give.w, bit);
    (up ? a : b) = give;
  };
  trade(v[0], v[1], 1);
  trade(v[2], v[3], 1);
  trade(v[0], v[2], 2);
  trade(v[1], v[3], 2);
  // v[i] is now chunk lane % 4 of the row of lane lane - lane % 4 + i
  const unsigned long long own = valid ? reinterpret_cast<unsigned long long>(at) : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long a = __shfl_sync(0xffffffffu, own, (lane & ~3) + i);
    if (a) reinterpret_cast<uint4 *>(a)[lane & 3] = v[i];
  }
}

// ------------------------------------------------------------------ schedule
struct Seq {
  int lo, n, len;  // first packed row, new tokens, cached positions
};

__device__ __forceinline__ Seq seq_of(const Params &p, int b, bool report) {
  int lo = __ldg(p.s.cu + b), hi = __ldg(p.s.cu + b + 1), len = __ldg(p.s.lens + b);
  lo = lo < 0 ? 0 : (lo > p.total ? p.total : lo);
  hi = hi < lo ? lo : (hi > p.total ? p.total : hi);
  const int most = p.s.max_pages << p.s.page_shift;
  if (len < 0 || len > most) {
    if (report) atomicExch(&p.wc.status->reserved[0], 1);
    len = len < 0 ? 0 : most;
  }
  const int n = hi - lo;
  return Seq{lo, n > p.above && n <= p.upto ? n : 0, len};
}

// Key tiles that tokens below `end` of the sequence see; at least one, so
// that rows which see nothing are still written.
__device__ __forceinline__ int tiles_to(const Params &p, const Seq &s, int end) {
  const int seen = p.causal ? s.len - s.n + (end < s.n ? end : s.n) : s.len;
  return seen <= BN ? 1 : (seen + BN - 1) / BN;
}

__device__ __forceinline__ int units_of(const Params &p, const Seq &s) {
  return (s.n + p.utok - 1) / p.utok;
}

// Cost of a unit: its key tiles, and `overhead` for its start and end.
__device__ __forceinline__ int tile_cost(const Params &p, int ntok) { return ntok > p.tpt ? p.cost2 : p.cost1; }
__device__ __forceinline__ long long unit_cost(const Params &p, const Seq &s, int q) {
  const int i0 = q * p.utok;
  return p.overhead + (long long)tile_cost(p, s.n - i0) * tiles_to(p, s, i0 + p.utok);
}
// 64-bit division takes hundreds of cycles and is hardly ever needed
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Key tile at a cost offset into a unit.
__device__ __forceinline__ int tile_at(const Params &p, long long off, int w) {
  return off <= p.overhead ? 0 : (int)quotient(off - p.overhead, w);
}

// Cost of one K/V head of the sequence
__device__ __forceinline__ long long head_cost(const Params &p, const Seq &s) {
  const int nu = units_of(p, s);
  long long t = 0;
  for (int q = 0; q < nu; ++q) t += unit_cost(p, s, q);
  return t;
}

struct Place {
  int b, head, q;  // sequence, K/V head, unit of the head
  long long off;   // cost offset into the unit
};

// Of 32 lanes' costs `own`, the lane that `t` falls into, or -1; t becomes the
// offset into it, or past all of them.
__device__ __forceinline__ int find(long long own, long long &t, int lane) {
  long long upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  const uint32_t hit = __ballot_sync(0xffffffffu, t < upto);
  const int l = hit ? __ffs(hit) - 1 : -1;
  t -= __shfl_sync(0xffffffffu, hit ? upto - own : upto, hit ? l : 31);
  return l;
}

// The warp finds cost `t` (below the total) in the whole work; sums[b] = cost of
// one head of sequence b.
__device__ __forceinline__ Place locate(const Params &p, const long long *sums, long long t, int lane) {
  Place at = {0, 0, 0, 0};
  for (int c = 0; c < p.s.batch && p.s.batch > 1; c += 32) {
    const int l = find(c + lane < p.s.batch ? sums[c + lane] * p.Hkv : 0, t, lane);
    if (l >= 0) {
      at.b = c + l;
      break;
    }
  }
  const Seq s = seq_of(p, at.b, false);
  const int nu = units_of(p, s);
  const long long per = sums[at.b];
  at.head = (int)quotient(t, per);
  t -= at.head * per;
  for (int c = 0; c < nu && nu > 1; c += 32) {
    const int l = find(c + lane < nu ? unit_cost(p, s, c + lane) : 0, t, lane);
    if (l >= 0) {
      at.q = c + l;
      break;
    }
  }
  at.off = t;
  return at;
}

template <int RUNS>
__device__ __forceinline__ long long run_start(long long total, int cta) {
  return total * cta / RUNS;
}

// A block's run: what is left of it, and where it goes on.
struct Run {
  long long t, t1;  // cost offsets into all of the work
  Place at;
  Seq s;
};

// A warp finds where the block's run begins, writes its boundary, and says whether
// there is anything in it.
template <int RUNS>
__device__ __forceinline__ bool begin_run(const Params &p, const long long *sums, Run &r, int lane) {
  long long total = 0;
  for (int b = lane; b < p.s.batch; b += 32) total += sums[b];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total *= p.Hkv;
  r.t = run_start<RUNS>(total, blockIdx.x);
  r.t1 = run_start<RUNS>(total, blockIdx.x + 1);
  r.at = Place{0, 0, 0, 0};
  r.s = Seq{0, 0, 0};
  Boundary bd = {0, total, 0, 1, 0, 0, 0, 0};
  bool work = false;
  if (r.t < total) {
    r.at = locate(p, sums, r.t, lane);
    r.s = seq_of(p, r.at.b, false);
    const int i0 = r.at.q * p.utok;
    bd.u0 = r.t - r.at.off;
    bd.nt = tiles_to(p, r.s, i0 + p.utok);
    bd.w = tile_cost(p, r.s.n - i0);
    bd.cut = tile_at(p, r.at.off, bd.w) > 0;
    bd.tok0 = r.s.lo + i0;
    bd.ntok = min(r.s.n - i0, p.utok);
    bd.head = r.at.head;
    // a run that ends before the first key tile that it reaches has nothing to do
    const long long end = r.at.off + (r.t1 - r.t), cost = p.overhead + (long long)bd.w * bd.nt;
    work = r.t < r.t1 && (end >= cost || tile_at(p, end, bd.w) > tile_at(p, r.at.off, bd.w));
  }
  if (lane == 0) p.bounds[blockIdx.x] = bd;
  return work;
}

// The run's next unit; head = -1 at its end.
__device__ __forceinline__ Unit next_of(const Params &p, Run &r) {
  Unit u = {};
  u.head = -1;
  if (r.t < r.t1) {
    const int i0 = r.at.q * p.utok, nt = tiles_to(p, r.s, i0 + p.utok);
    const int w = tile_cost(p, r.s.n - i0);
    const long long cost = p.overhead + (long long)w * nt, end = r.at.off + (r.t1 - r.t);
    u.j0 = tile_at(p, r.at.off, w);
    u.j1 = end >= cost ? nt : tile_at(p, end, w);
    if (u.j1 > u.j0) {  // else the run ends before the unit's first key tile
      u.tok0 = r.s.lo + i0;
      u.ntok = min(r.s.n - i0, p.utok);
      u.head = r.at.head;
      u.b = r.at.b;
      u.ja = tiles_to(p, r.s, i0 + p.tpt);
      u.lim0 = p.causal ? r.s.len - r.s.n + i0 + 1 : r.s.len;
      u.len = r.s.len;
      u.slot = u.j0 > 0 ? 0 : (u.j1 < nt ? 1 : -1);
    }
    r.t += cost - r.at.off;
    // on to the next unit: of the head, the next head, the next sequence with new tokens
    r.at.off = 0;
    if (r.t < r.t1 && ++r.at.q == units_of(p, r.s)) {
      r.at.q = 0;
      if (++r.at.head == p.Hkv) {
        r.at.head = 0;
        do {
          r.s = seq_of(p, ++r.at.b, false);
        } while (r.s.n == 0 && r.at.b + 1 < p.s.batch);
      }
    }
  }
  return u;
}

// --------------------------------------------------------------- main kernel
template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const Params p) {
  using L = Layout<D>;
  constexpr int NS = L::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);  // [2]
  uint64_t *q_empty = q_full + 2;                                      // [2]
  uint64_t *full = q_empty + 2;                                        // [NS]
  uint64_t *empty = full + NS;                                         // [NS]
  uint64_t *s_full = empty + NS;                                       // [2]
  uint64_t *p_ready = s_full + 2;                                      // [2]
  uint64_t *pv_done = p_ready + 2;                                     // [2]
  uint64_t *u_full = pv_done + 2;                                      // [NU]
  uint64_t *u_empty = u_full + NU;                                     // [NU]
  uint64_t *joined = u_empty + NU;                                     // [2]: stream 1's (m, l); O1 read
  uint64_t *mma_drain = joined + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 4);
  volatile int *has_work = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 8);
  float2 *ml = reinterpret_cast<float2 *>(smem + L::OFF_ML);
  long long *sums = reinterpret_cast<long long *>(smem + L::OFF_RING);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_ready[t], 128);
      mbar_init(&pv_done[t], 1);
      mbar_init(&joined[t], 128);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < NU; ++s) {
      mbar_init(&u_full[s], 1);
      mbar_init(&u_empty[s], 10);  // producer, MMA warp, eight softmax warps
    }
    mbar_init(mma_drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  for (int b = threadIdx.x; b < p.s.batch; b += THREADS)
    sums[b] = head_cost(p, seq_of(p, b, blockIdx.x == 0));
  fence_proxy_async_smem();  // the ring's first copies come after these writes and their reads
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();  // the join may be launched; it waits for this grid

  // The scheduler warp finds where the block's run begins.
  Run run;
  if (warp == 10) {
    const bool work = begin_run<CTAS>(p, sums, run, lane);
    if (lane == 0) *has_work = work;
  }
  __syncthreads();
  if (!*has_work) {
    if (warp == 9) tmem_dealloc(tmem, 512);
    return;
  }

  // The softmax warps' wait: every lane polls, since every lane reads tensor memory next, the warp goes
  // on or gives up as one, and its lanes are together again before that access, which needs them so.
  auto warp_wait = [&](uint64_t *bar, uint32_t parity, int site) -> bool {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, p.wc, abort_flag, site));
    __syncwarp();
    return ok;
  };
  // Reads the next unit; false when the run is done or a wait expired.  Lane 0 polls: no vote
  // in the producer and the issuer, whose lanes leave a poll at different times.
  auto next_unit = [&](int &k, Unit &u, int site) -> bool {
    const int s = k % NU;
    if (!mbar_wait_warp(&u_full[s], (k / NU) & 1, p.wc, abort_flag, site)) return false;
    __syncwarp();  // what lane 0 saw, every lane may read
    u = *reinterpret_cast<const Unit *>(smem + L::OFF_UNITS + s * 48);
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_empty[s]);
    __syncwarp();  // what follows elects a lane or reads tensor memory
    ++k;
    return u.head >= 0;
  };

  auto role_scheduler = [&]() {
    int k = 0;
    bool ok = true;
    while (true) {
      const Unit u = next_of(p, run);
      const int sl = k % NU;
      if (k >= NU) ok = mbar_wait_warp(&u_empty[sl], ((k / NU) - 1) & 1, p.wc, abort_flag, SITE_PAGED_SCHED);
      if (!ok) break;
      if (lane == 0) {
        *reinterpret_cast<Unit *>(smem + L::OFF_UNITS + sl * 48) = u;
        mbar_arrive(&u_full[sl]);
      }
      ++k;
      if (u.head < 0) break;
    }
    __syncwarp();
  };

  auto role_producer = [&]() {
    Unit u;
    int k = 0;
    uint32_t q_uses[2] = {0, 0}, qsel = 0;
    uint32_t seq = 0;  // tiles put into the ring
    bool ok = true;
    constexpr int HALVES = D / 64;
    const int page = 1 << p.s.page_shift;
    const int rows = page < BN ? page : BN;        // of a box
    const int boxes = BN / rows * HALVES;          // of a tile, at most 16
    const int part = lane / HALVES, half = lane % HALVES;
    const uint32_t q_bytes = (uint32_t)(p.G * p.tpt) * D * 2;
    while (ok && next_unit(k, u, SITE_PAGED_PROD)) {
      const bool two = u.ntok > p.tpt;
      // 32 entries of the table at a time, one a lane, the next 32 on their way and
      // checked only when their turn comes; the pool's end, which reads as zeros, where the
      // sequence has no keys or the table names no page
      const int *table = p.s.table + u.b * p.s.table_stride;
      const int pool = (int)p.s.num_pages;
      auto keys_at = [&](int at) { return ((long long)at << p.s.page_shift) < u.len; };
      auto entry = [&](int at) { return keys_at(at) ? __ldg(table + at) : pool; };
      auto checked = [&](int pg, int at) {
        if (pg >= 0 && pg < pool) return pg;
        if (keys_at(at)) atomicExch(&p.wc.status->reserved[0], 1);
        return pool;
      };
      int first = u.j0 * BN >> p.s.page_shift;
      int pages = entry(first + lane), ahead = entry(first + 32 + lane);
      for (int t = 0; t < (two ? 2 : 1); ++t) {
        const int buf = two ? t : (int)qsel;
        if (q_uses[buf] > 0)
          ok = ok && mbar_wait_warp(&q_empty[buf], (q_uses[buf] - 1) & 1, p.wc, abort_flag, SITE_PAGED_PROD);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[buf], q_bytes);
#pragma unroll
          for (int c = 0; c < HALVES; ++c)
            tma_load_3d(smem + L::OFF_Q + buf * L::TILE + c * (BM * 128), &tmQ, &q_full[buf], c * 64,
                        u.head * p.G, u.tok0 + t * p.tpt);
        }
        ++q_uses[buf];
      }
      if (!two) qsel ^= 1;
      pages = checked(pages, first + lane);
      for (int j = u.j0; ok && j < u.j1; ++j) {
        int e = (j * BN >> p.s.page_shift) - first;  // the tile's first entry
        if (e >= 32) {
          first += 32;
          e -= 32;
          pages = checked(ahead, first + lane);
          ahead = entry(first + 32 + lane);
        }
        const int pg = __shfl_sync(0xffffffffu, pages, (e + part) & 31);
        const int at = page > BN ? (j * BN) & (page - 1) : 0;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int st = seq % NS;
          if (seq >= NS)
            ok = mbar_wait_warp(&empty[st], ((seq / NS) - 1) & 1, p.wc, abort_flag, SITE_PAGED_PROD);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[st], L::TILE);
          __syncwarp();
          if (lane < boxes)
            tma_load_4d(smem + L::OFF_RING + st * L::TILE + half * (BN * 128) + part * (rows * 128),
                        kv ? &tmV : &tmK, &full[st], half * 64, at, u.head, pg);
          ++seq;
        }
      }
    }
    if (*abort_flag && lane == 0) {
      // let every copy still in flight land before shared memory is freed
      for (int t = 0; t < 2; ++t)
        if (q_uses[t]) drain_wait(&q_full[t], (q_uses[t] - 1) & 1, p.wc);
      for (uint32_t s = seq > NS ? seq - NS : 0; s < seq; ++s)
        drain_wait(&full[s % NS], (s / NS) & 1, p.wc);
    }
    __syncwarp();
  };

  // Issues the products of both streams, whose order keeps them half a step apart: one
  // multiplies while the other exponentiates.  (An issuer for each let them fall into step: at
  // d = 128 single tokens took 389 us that take 336, at d = 64 a chunk over 32,768 positions 1,131
  // and 770.)  Measured at d = 64 and dropped: columns of P_hi's own and P_lo in shared memory, so
  // that a stream's next S is computed while its softmax still runs, with two issuers: the chunk 750 us, 24
  // mixed sequences no faster, and every buffer freed by two warps that run apart.
  auto role_mma = [&]() {
    const uint32_t idS = idesc_bf16_f32(BM, BN, 0, 0), idO = idesc_bf16_f32(BM, D, 0, 1);
    const SDesc dQ = sdesc_make(smem_u32(smem + L::OFF_Q), 16, 1024);
    const SDesc dK = sdesc_make(smem_u32(smem + L::OFF_RING), 16, 1024);
    const SDesc dV = sdesc_make(smem_u32(smem + L::OFF_RING), BN * 128, 1024);
    Unit u;
    int k = 0;
    uint32_t q_uses[2] = {0, 0}, qsel = 0;
    uint32_t base = 0;             // ring number of the unit's first K tile
    uint32_t steps[2] = {0, 0};    // P V products of each stream so far
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return mbar_wait_warp(bar, parity, p.wc, abort_flag, SITE_PAGED_MMA);
    };
    // Two barriers in one go, and whether a third is there already: lane 0 polls, as in
    // mbar_wait_warp, and one exchange tells the others.  Returns bit 0: both over, bit 1: the third.
    auto wait_pair = [&](uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1, uint64_t *b2, uint32_t p2) -> int {
      int r = 0;
      if (lane == 0) {
        const uint32_t a0 = smem_u32(b0), a1 = smem_u32(b1);
        const bool r0 = mbar_try_wait(a0, p0), r1 = mbar_try_wait(a1, p1);
        r = (r0 || mbar_wait(b0, p0, p.wc, abort_flag, SITE_PAGED_MMA)) &&
            (r1 || mbar_wait(b1, p1, p.wc, abort_flag, SITE_PAGED_MMA));
        if (r && b2 && mbar_try_wait(smem_u32(b2), p2)) r |= 2;
      }
      return __shfl_sync(0xffffffffu, r, 0);
    };
    while (ok && next_unit(k, u, SITE_PAGED_MMA)) {
      const bool two = u.ntok > p.tpt;
      const int n = u.j1 - u.j0;
      int ns[2];
      ns[0] = two ? max(0, min(u.ja, u.j1) - u.j0) : (n + 1) / 2;
      ns[1] = two ? n : n / 2;
      const int single = (int)qsel;  // the Q tile of a unit that has one
      for (int b = 0; b < 2; ++b)
        if (two || b == single) {
          ok = ok && wait(&q_full[b], q_uses[b] & 1);
          ++q_uses[b];
        }
      if (!two) qsel ^= 1;
      // whether stream t's product is the last that reads its K or V tile
      auto last_reader = [&](int t) { return !two || t == 1; };
      // no key tile of this part is seen by tile 0
      if (ok && two && ns[0] == 0 && elect_one()) umma_commit(&q_empty[0]);
      __syncwarp();
      auto k_seq = [&](int t, int i) { return base + 2 * (two ? i : 2 * i + t); };
      // S of step i into columns [128 t, 128 t + 128), by the elected lane
      auto put_s = [&](int t, int i) {
        const uint32_t st = k_seq(t, i) % NS, qo = (uint32_t)(two ? t : single) * L::TILE, ko = st * L::TILE;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * (BM * 128) + (kk & 3) * 32;
          umma_f16_ss(tmem + t * BN, sdesc_at(dQ, qo + off), sdesc_at(dK, ko + off), idS, kk > 0);
        }
        umma_commit(&s_full[t]);
        if (last_reader(t)) umma_commit(&empty[st]);
        if (two ? i == ns[t] - 1 : 2 * i + t == n - 1) umma_commit(&q_empty[two ? t : single]);
      };
      auto issue_s = [&](int t, int i) -> bool {
        const uint32_t seq = k_seq(t, i);
        if (!wait(&full[seq % NS], (seq / NS) & 1)) return false;
        tc_fence_after();
        if (elect_one()) put_s(t, i);
        __syncwarp();
        return true;
      };
      // O_t += P_hi V + P_lo V of step i, with S of the stream's next step right behind it if its K
      // tile is there
      auto issue_pv = [&](int t, int i) -> bool {
        const uint32_t seq = k_seq(t, i) + 1, st = seq % NS;
        const bool next_s = i + 1 < ns[t];
        const uint32_t nseq = k_seq(t, i + 1);
        const int got = wait_pair(&full[st], (seq / NS) & 1, &p_ready[t], steps[t] & 1,
                                  next_s ? &full[nseq % NS] : nullptr, (nseq / NS) & 1);
        if (!(got & 1)) return false;
        // The last page may hold anything behind the sequence's end, and 0 times a NaN
        // is not 0: those rows of V become zeros (twice, where both streams read them).
        const int valid = u.len - (u.j0 + (two ? i : 2 * i + t)) * BN;
        if (valid > 0 && valid < BN) {
          const int page = 1 << p.s.page_shift;
          const int upto = min(BN, (valid + page - 1) & ~(page - 1));
          for (int c = lane; c < (upto - valid) * (D / 8); c += 32) {
            const int r = valid + c / (D / 8), q = c % (D / 8);
            st_shared_v4(smem_u32(smem + L::OFF_RING + st * L::TILE + (q >> 3) * (BN * 128) + r * 128 + (q & 7) * 16),
                         0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        ++steps[t];
        tc_fence_after();
        if (elect_one()) {
          const uint32_t vo = st * L::TILE;
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              umma_f16_ts(tmem + L::o_col(t), tmem + t * BN + kk * 16 + part * 8, sdesc_at(dV, vo + kk * 2048), idO,
                          i > 0 || part > 0 || kk > 0);
          umma_commit(&pv_done[t]);
          if (last_reader(t)) umma_commit(&empty[st]);
          if (got & 2) put_s(t, i + 1);
        }
        __syncwarp();
        return !next_s || (got & 2) || issue_s(t, i + 1);
      };
      for (int t = 0; ok && t < 2; ++t)
        if (ns[t] > 0) ok = issue_s(t, 0);
      for (int i = 0; ok && i < max(ns[0], ns[1]); ++i)
        for (int t = 0; ok && t < 2; ++t)
          if (i < ns[t]) ok = issue_pv(t, i);
      base += 2 * n;
    }
    // no MMA may still be running when tensor memory is released
    __syncwarp();
    if (elect_one()) umma_commit(mma_drain);
    __syncwarp();
    if (lane == 0) drain_wait(mma_drain, 0, p.wc);
    __syncwarp();
  };

  auto role_softmax = [&]() {
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + t * BN;
    const int rtok = row / p.G, rhead = row - rtok * p.G;  // token of the tile, head of the group
    Unit u;
    int k = 0;
    uint32_t steps[2] = {0, 0}, joins = 0;  // S tiles of each stream, units joined
    bool ok = true;
    while (ok && next_unit(k, u, SITE_PAGED_SOFTMAX)) {
      const bool two = u.ntok > p.tpt;
      const int n = u.j1 - u.j0;
      const int n0 = two ? max(0, min(u.ja, u.j1) - u.j0) : (n + 1) / 2;
      const int n1 = two ? n : n / 2;
      const int mine = t ? n1 : n0;
      const int tok = (two ? t * p.tpt : 0) + rtok;  // of the unit
      const bool valid = rtok < p.tpt && tok < u.ntok;
      const bool active = __any_sync(0xffffffffu, valid);
      const int lim = valid ? (p.causal ? u.lim0 + tok : u.len) : u.len;  // keys below it are seen
      float m = -INFINITY, l = 0.0f;
      for (int i = 0; i < mine; ++i) {
        ok = warp_wait(&s_full[t], (steps[t] + i) & 1, SITE_PAGED_SOFTMAX);
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const int kv0 = (u.j0 + (two ? i : 2 * i + t)) * BN;
          uint32_t s[BN];
#pragma unroll
          for (int c = 0; c < BN / 32; ++c)
            tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[c * 32]));
          tmem_wait_ld();
          if (kv0 + BN > lim) {
#pragma unroll
            for (int e = 0; e < BN; ++e)
              if (kv0 + e >= lim) s[e] = __float_as_uint(-INFINITY);
          }
          __syncwarp();
          float mx4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx4[e] = fmaxf(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
#pragma unroll
          for (int c = 8; c < BN; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx4[e] = fmax3(mx4[e], __uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1]));
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.scale_log2;
          float alpha = 1.0f;
          bool rescale = false;
          if (i == 0) {
            m = mx;
          } else if (mx > m + RESCALE_THRESHOLD) {
            alpha = ex2(m - mx);
            m = mx;
            rescale = true;
          }
          __syncwarp();  // the stores of P are the whole warp's
          const float mref = m == -INFINITY ? 0.0f : m;
          // P = 2^(s scale log2e - m) = P_hi + P_lo, sixteen keys at a time
          const uint64_t sc2 = f32x2(p.scale_log2, p.scale_log2), nm2 = f32x2(-mref, -mref);
          uint64_t rs2[4] = {0, 0, 0, 0};
#pragma unroll
          for (int g = 0; g < BN / 16; ++g) {
            uint32_t pk[16];  // P_hi, P_lo
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float x0, x1;
              f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[g * 16 + e]), __uint_as_float(s[g * 16 + e + 1])),
                                    sc2, nm2),
                          x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              rs2[(e >> 1) & 3] = add_f32x2(rs2[(e >> 1) & 3], f32x2(p0, p1));
              const uint32_t h = pack_bf16(p0, p1);
              pk[e >> 1] = h;
              pk[8 + (e >> 1)] = pack_bf16(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u));
            }
            tmem_st16(tS + g * 16, pk);
          }
          float rs = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a0, a1;
            f32x2_split(rs2[e], a0, a1);
            rs += a0 + a1;
          }
          // the previous step's P V is done: O holds every earlier key
          if (__any_sync(0xffffffffu, rescale)) {
            const uint32_t tO = tmem + lane_off + L::o_col(t);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + c * 32, o);
            }
          }
          l = l * alpha + rs;
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&p_ready[t]);
      }
      if (!ok) break;
      steps[0] += n0;
      steps[1] += n1;
      // ----------------------------------------------------------- epilogue
      if (!two && t == 1) {
        // stream 1's row statistics to stream 0, which reads its O too
        ml[row] = make_float2(m, l);
        mbar_arrive(&joined[0]);
        ok = warp_wait(&joined[1], joins & 1, SITE_PAGED_EPI);
        tc_fence_after();
        ++joins;
        continue;
      }
      float w[2] = {t == 0 ? 1.0f : 0.0f, t == 1 ? 1.0f : 0.0f};  // weights of the two streams' O
      bool has[2] = {t == 0 && n0 > 0, t == 1};
      if (!two) {
        ok = warp_wait(&joined[0], joins & 1, SITE_PAGED_EPI);
        if (!ok) break;
        has[1] = n1 > 0;
        const float2 o = ml[row];
        const float top = fmaxf(m, o.x);
        if (top != -INFINITY) {
          w[0] = ex2(m - top);
          w[1] = ex2(o.x - top);
          l = l * w[0] + o.y * w[1];
        }
        m = top;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (has[e] && ok) ok = warp_wait(&pv_done[e], (steps[e] - 1) & 1, SITE_PAGED_EPI);
      if (!ok) break;
      tc_fence_after();
      if (active) {
        const bool whole = u.slot < 0;
        if (whole) {
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
          w[0] *= inv;
          w[1] *= inv;
        }
        const int64_t qhead = (int64_t)u.head * p.G + rhead;
        __nv_bfloat16 *orow = p.O + ((int64_t)u.tok0 + tok) * p.o_stok + qhead * p.o_shead;
        // a slot's O is [D / 4][2 BM][4], so that lanes, which hold rows, write side by side
        const int64_t slot = (int64_t)blockIdx.x * 2 + u.slot;
        float4 *prow = reinterpret_cast<float4 *>(p.part_o) + slot * (2 * BM * D / 4) + t * BM + row;
#pragma unroll 1
        for (int c = 0; c < D / 32 && (has[0] || has[1]); ++c) {
          uint32_t x[32];
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.0f;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (!has[y]) continue;
            tmem_ld32(tmem + lane_off + L::o_col(y) + c * 32, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(x[e]), w[y], o[e]);
          }
          if (whole) {
            uint4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
            store_rows(v, orow + c * 32, valid, lane);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (valid) prow[(c * 8 + e) * (2 * BM)] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          __syncwarp();
        }
        if (valid) {
          if (whole)
            p.LSE[qhead * p.lse_shead + u.tok0 + tok] = l > 0.0f ? (m + lg2(l)) * 0.69314718055994531f : -INFINITY;
          else
            p.part_ml[slot * (2 * BM) + t * BM + row] = make_float2(m, l);
        }
      }
      if (!two) {
        tc_fence_before();
        mbar_arrive(&joined[1]);
        ++joins;
      }
    }
  };

  if (warp >= 8) {  // warp 11 only hands its registers over
    setmaxnreg_dec<REGS_CONTROL>();
    if (warp == 8)
      role_producer();
    else if (warp == 10)
      role_scheduler();
    else if (warp == 9)
      role_mma();
  } else {
    setmaxnreg_inc<REGS_SOFTMAX>();
    role_softmax();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------- few rows
// Single tokens, whose G query heads fill a few of a query tile's 128 rows.  There the
// kernel above waits: one warp of four has rows, each lane exponentiates a row's 128 keys
// one after another, and a key tile's chain of copies, products and softmax, some 4,000
// cycles, shows wherever a unit has few tiles.  Here a tile has 16 rows, the least that a
// warp's own products take (mma.sync: with this few rows the work is memory's, and the
// tensor cores' rate does not matter), and eight warps an SM work for themselves: a warp
// takes its share of a tile's 128 keys, copies them, keeps its own running (m, l, O), and the
// block joins its warps' at the end of a unit.  Units, runs and partial results are those of
// the kernel above.  Two stages of 8 KB a warp; a third, or more blocks, made the memory
// slower (64 sequences of 16,384: 356 us with two stages, 374 with three).
constexpr int TOK_ROWS = 16;
template <int D, int WARPS>
struct TokenLayout {
  static constexpr int BLOCKS = 8 / WARPS, RUNS = CTAS * BLOCKS;
  static constexpr int KEYS = BN / WARPS;                       // of a key tile, a warp's
  static constexpr int KS = KEYS < 2048 / D ? KEYS : 2048 / D;  // of a stage: 8 KB of K and V at most
  static constexpr int STAGES = 2;
  static constexpr uint32_t HALF = KS * D * 2, STAGE = 2 * HALF;
  static constexpr uint32_t WARP = STAGES * STAGE;  // a warp's ring; then its share of O
  static constexpr uint32_t ALLOC = WARPS * WARP;
  static constexpr int OPITCH = D + 4;
  static constexpr int COST = 4, OVERHEAD = D == 128 ? 4 : 8;
  static_assert(MAX_BATCH * 8 <= ALLOC, "the schedule's sums use the rings");
  static_assert(TOK_ROWS * OPITCH * 4 <= WARP, "O in the ring");
  static_assert(KEYS % KS == 0 && KS % 16 == 0, "keys");
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// c [16][8] += a [16][16] b [16][8]
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void copy_or_zero(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

template <int D, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, TokenLayout<D, WARPS>::BLOCKS) paged_token_kernel(const Params p) {
  using L = TokenLayout<D, WARPS>;
  constexpr int CH = D / 8;             // 16-byte chunks of a row
  constexpr int RPC = 32 / CH;          // rows that a copy of the warp covers
  constexpr int PER = L::KEYS / L::KS;  // stages of a key tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ Unit next;
  __shared__ float2 ml[WARPS][TOK_ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long *sums = reinterpret_cast<long long *>(smem_raw);
  for (int b = threadIdx.x; b < p.s.batch; b += 32 * WARPS) sums[b] = head_cost(p, seq_of(p, b, blockIdx.x == 0));
  __syncthreads();
  pdl_launch_dependents();  // the join may be launched; it waits for this grid
  Run run;
  if (warp == 0) begin_run<L::RUNS>(p, sums, run, lane);
  const uint32_t ring = smem_u32(smem_raw) + warp * L::WARP;
  const int page = 1 << p.s.page_shift, pool = (int)p.s.num_pages;
  while (true) {
    if (warp == 0) {
      const Unit u = next_of(p, run);
      if (lane == 0) next = u;
    }
    __syncthreads();
    const Unit u = next;
    if (u.head < 0) break;
    const int steps = (u.j1 - u.j0) * PER;
    const int *table = p.s.table + u.b * p.s.table_stride;
    const __nv_bfloat16 *kc = static_cast<const __nv_bfloat16 *>(p.kc.ptr) + u.head * p.kc.s_head;
    const __nv_bfloat16 *vc = static_cast<const __nv_bfloat16 *>(p.vc.ptr) + u.head * p.vc.s_head;
    auto first_key = [&](int i) { return (u.j0 + i / PER) * BN + warp * L::KEYS + i % PER * L::KS; };
    // page numbers of a stage's keys (KS <= 32 and pages of 16 at least: two at most), looked up one stage ahead
    int ids[2];
    auto look_up = [&](int i) {
#pragma unroll
      for (int h = 0; h < L::KS / 16; ++h) {
        const int pos = first_key(i) + 16 * h;
        ids[h] = i < steps && pos < u.len ? __ldg(table + (pos >> p.s.page_shift)) : pool;
      }
    };
    auto fetch = [&](int i) {
      if (i < steps) {
        const int base = first_key(i);
        const uint32_t at = ring + i % L::STAGES * L::STAGE;
#pragma unroll
        for (int h = 0; h < L::KS / 16; ++h) {  // 16 positions lie in one page
          const int pos = base + 16 * h, id = ids[h];
          const bool known = id >= 0 && id < pool;
          if (pos < u.len && !known && lane == 0) atomicExch(&p.wc.status->reserved[0], 1);
          const int left = known ? u.len - pos : 0, r0 = lane / CH, c = lane % CH;
          const int64_t slot = left > 0 ? pos & (page - 1) : 0, pg = left > 0 ? id : 0;
          const __nv_bfloat16 *k = kc + pg * p.kc.s_page + (slot + r0) * p.kc.s_slot + c * 8;
          const __nv_bfloat16 *v = vc + pg * p.vc.s_page + (slot + r0) * p.vc.s_slot + c * 8;
#pragma unroll
          for (int it = 0; it < 16 / RPC; ++it) {
            const int r = it * RPC + r0;
            const uint32_t dst = at + (16 * h + r) * (D * 2) + ((c ^ (r & 7)) << 4);
            copy_or_zero(dst, k, r < left);
            copy_or_zero(dst + L::HALF, v, r < left);
            k += RPC * p.kc.s_slot;
            v += RPC * p.vc.s_slot;
          }
        }
        look_up(i + 1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up(0);
#pragma unroll
    for (int i = 0; i < L::STAGES - 1; ++i) fetch(i);

    // The lane's rows lane / 4 and lane / 4 + 8; Q in the products' layout
    uint32_t q[D / 16][4];
    int lim[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = lane / 4 + 8 * h, tok = row / p.G;
      const bool valid = tok < u.ntok && tok < p.tpt;
      lim[h] = valid ? (p.causal ? u.lim0 + tok : u.len) : 0;  // keys below it are seen
      const __nv_bfloat16 *src =
          p.Q + ((int64_t)u.tok0 + tok) * p.q_stok + ((int64_t)u.head * p.G + row - tok * p.G) * p.q_shead + lane % 4 * 2;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        q[kk][h] = valid ? *reinterpret_cast<const uint32_t *>(src + kk * 16) : 0u;
        q[kk][2 + h] = valid ? *reinterpret_cast<const uint32_t *>(src + kk * 16 + 8) : 0u;
      }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;

    for (int i = 0; i < steps; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(L::STAGES - 2) : "memory");
      __syncwarp();  // every lane's copies are there, and every lane has read the stage before
      fetch(i + L::STAGES - 1);
      const uint32_t at = ring + i % L::STAGES * L::STAGE;
#pragma unroll
      for (int g = 0; g < L::KS / 16; ++g) {
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
        const int krow = g * 16 + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t b[4];
          ldmatrix4(b, at + krow * (D * 2) + (((kk * 2 + ((lane >> 3) & 1)) ^ (krow & 7)) << 4));
          mma_16x8x16(s[0], q[kk], b[0], b[1]);
          mma_16x8x16(s[1], q[kk], b[2], b[3]);
        }
        const int key = first_key(i) + g * 16 + lane % 4 * 2;
        float alpha[2], ref[2];
        bool moved = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = -INFINITY;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (key + n * 8 + e >= lim[h]) s[n][2 * h + e] = -INFINITY;
              mx = fmaxf(mx, s[n][2 * h + e]);
            }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * p.scale_log2;
          alpha[h] = 1.0f;
          if (mx > m[h]) {
            alpha[h] = ex2(m[h] - mx);
            m[h] = mx;
            moved = true;
          }
          ref[h] = m[h] == -INFINITY ? 0.0f : m[h];
          l[h] *= alpha[h];
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= alpha[e >> 1];
        }
        // P = 2^(s scale log2e - m) as a pair of bf16, P_hi = bf16(P) and P_lo = bf16(P - P_hi): one bf16
        // would add as much error to O as O's own rounding does.  l sums P unrounded.
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[n][e] = ex2(fmaf(s[n][e], p.scale_log2, -ref[e >> 1]));
            l[e >> 1] += s[n][e];
          }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p0 = s[e >> 1][2 * (e & 1)], p1 = s[e >> 1][2 * (e & 1) + 1];
          hi[e] = pack_bf16(p0, p1);
          lo[e] = pack_bf16(p0 - __uint_as_float(hi[e] << 16), p1 - __uint_as_float(hi[e] & 0xffff0000u));
        }
        const int vrow = g * 16 + (lane & 15);
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t b[4];
          ldmatrix4_trans(b, at + L::HALF + vrow * (D * 2) + (((n * 2 + (lane >> 4)) ^ (vrow & 7)) << 4));
          mma_16x8x16(o[2 * n], hi, b[0], b[1]);
          mma_16x8x16(o[2 * n + 1], hi, b[2], b[3]);
          mma_16x8x16(o[2 * n], lo, b[0], b[1]);
          mma_16x8x16(o[2 * n + 1], lo, b[2], b[3]);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    // the warps' shares: O over the warp's own ring
    float *mine = reinterpret_cast<float *>(smem_raw + warp * L::WARP);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = lane / 4 + 8 * h;
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (lane % 4 == 0) ml[warp][row] = make_float2(m[h], l[h]);
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2 *>(mine + row * L::OPITCH + n * 8 + lane % 4 * 2) =
            make_float2(o[n][2 * h], o[n][2 * h + 1]);
    }
    __syncthreads();
    {
      constexpr int COLS = D / 8;  // a thread's, of row threadIdx.x / 8
      const int row = threadIdx.x >> 3, c0 = (threadIdx.x & 7) * COLS, tok = row / p.G;
      if (row < TOK_ROWS && tok < u.ntok && tok < p.tpt) {
        float top = -INFINITY, sum = 0.0f, x[COLS];
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[w][row].x);
#pragma unroll
        for (int c = 0; c < COLS; ++c) x[c] = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float2 v = ml[w][row];
          const float f = v.x == -INFINITY ? 0.0f : ex2(v.x - top);
          sum = fmaf(v.y, f, sum);
          const float4 *src =
              reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem_raw + w * L::WARP) + row * L::OPITCH + c0);
#pragma unroll
          for (int c = 0; c < COLS / 4; ++c) {
            const float4 y = src[c];
            x[4 * c] = fmaf(y.x, f, x[4 * c]);
            x[4 * c + 1] = fmaf(y.y, f, x[4 * c + 1]);
            x[4 * c + 2] = fmaf(y.z, f, x[4 * c + 2]);
            x[4 * c + 3] = fmaf(y.w, f, x[4 * c + 3]);
          }
        }
        if (u.slot < 0) {
          const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
          const int64_t qhead = (int64_t)u.head * p.G + row - tok * p.G;
          uint4 *dst = reinterpret_cast<uint4 *>(p.O + ((int64_t)u.tok0 + tok) * p.o_stok + qhead * p.o_shead + c0);
#pragma unroll
          for (int c = 0; c < COLS / 8; ++c)
            dst[c] = make_uint4(pack_bf16(x[8 * c] * inv, x[8 * c + 1] * inv), pack_bf16(x[8 * c + 2] * inv, x[8 * c + 3] * inv),
                                pack_bf16(x[8 * c + 4] * inv, x[8 * c + 5] * inv),
                                pack_bf16(x[8 * c + 6] * inv, x[8 * c + 7] * inv));
          if ((threadIdx.x & 7) == 0)
            p.LSE[qhead * p.lse_shead + u.tok0 + tok] =
                sum > 0.0f ? (top + lg2(sum)) * 0.69314718055994531f : -INFINITY;
        } else {
          const int64_t slot = (int64_t)blockIdx.x * 2 + u.slot;
          float4 *dst = reinterpret_cast<float4 *>(p.part_o) + slot * (TOK_ROWS * D / 4) + row;
#pragma unroll
          for (int c = 0; c < COLS / 4; ++c)
            dst[(c0 / 4 + c) * TOK_ROWS] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
          if ((threadIdx.x & 7) == 0) p.part_ml[slot * TOK_ROWS + row] = make_float2(top, sum);
        }
      }
    }
    __syncthreads();  // the rings, ml and `next` are free
  }
}

// Whether a call's rows may be few: with a query head's group that fits 16 rows, no more new
// tokens than sequences, or so few that they fit one tile.  Single tokens, 32 heads on 8, this kernel
// and the one above: 64 sequences of 300 at d = 64 19.5 us and 44.1, at d = 128 27.2 and 53.3; of
// 1,000 57 and 90, of 4,000 190 and 212, of 8,192 366 and 369 (d = 64 206 and 252); 200 of 300 62 and 140.
// One sequence of 100: 6.4 and 11.9, of 4,096: 14.6 and 19.7, of 131,072: 101 and 107.
bool few_rows(const PagedAttnArgs &a, int G) {
  return G <= TOK_ROWS && (a.total <= a.seqs.batch || (int64_t)a.total * G <= TOK_ROWS);
}
// The counts themselves are on the device.  As many tokens as sequences are single tokens but for a
// coincidence; fewer may be a chunk in a batch that is padded with empty sequences, whose keys 16-row
// tiles would read once for every 16 rows.  Then sequences of more than two tiles are left to a launch
// of the kernel above, which finds nothing to do where there are none (32 heads on 8, d = 128, a batch
// of 256 padded with empty sequences: 200 tokens over 8,192 keys 61 us, 217 without that launch; 64 single
// tokens over 300 keys 33 and 28).
bool may_have_chunks(const PagedAttnArgs &a, int G) {
  return a.total < a.seqs.batch && (int64_t)a.total * G > 2 * TOK_ROWS;
}

// Joins a unit that runs' ends cut into parts: block (c, y) the unit that
// boundary c + 1 falls into, if that is the unit's first boundary.  A block takes
// `ROWS` rows and a warp D / 8 columns of them; a lane takes a row, as in the
// parts, and every GROUPS-th part of it, PB loaded at once: the kernel is a
// few dependent loads long.  Rows go out through shared memory.
template <int D, int RUNS, int SLOT, int ROWS>
__device__ __forceinline__ void combine_rows(const Params &p, const Boundary &bd, int c, int first_row,
                                             uint2 (*rows)[D / 4 + 1]) {
  constexpr int Q = D / 32, PB = 2, GROUPS = 32 / ROWS;  // Q: float4 a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane / ROWS;
  const int r = first_row + lane % ROWS;
  const int rt = (r % BM) / p.G, tok = (r / BM) * p.tpt + rt;
  const bool valid = rt < p.tpt && tok < bd.ntok;
  float m = -INFINITY, l = 0.0f;
  float4 o[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) o[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // block c - 1 holds the first part, as its last unit; the next blocks the others, as
  // their first, down to the one that holds the unit's last key tile
  const long long end = bd.u0 + p.overhead + (long long)bd.w * bd.nt;
  auto begins = [&](int k) { return k < RUNS && run_start<RUNS>(bd.total, k) < end; };
  // Where a lane takes many parts, one after another, their end is found first (8 tokens over
  // 4,096 keys: 26.3 us -> 22.6); a single token's lanes take one or two (17.3 us, 16.6 without).
  int k1 = c - 1;
  for (uint32_t in = ~0u; ROWS == 32 && in == ~0u;) {
    in = __ballot_sync(0xffffffffu, begins(k1 + lane));
    k1 += __popc(in);
  }
  auto in_unit = [&](int k) { return ROWS == 32 ? k < k1 : begins(k); };
  // a run shorter than a key tile may hold none of it, and then no part
  const bool tiny = bd.total < (long long)RUNS * (bd.w + 1);
  auto has_part = [&](int k) {
    if (!in_unit(k)) return false;
    if (!tiny) return true;
    const int j0 = tile_at(p, run_start<RUNS>(bd.total, k) - bd.u0, bd.w);
    return run_start<RUNS>(bd.total, k + 1) >= end || tile_at(p, run_start<RUNS>(bd.total, k + 1) - bd.u0, bd.w) > j0;
  };
  for (int k0 = c - 1; in_unit(k0); k0 += PB * GROUPS) {
    float2 x[PB];
    float4 v[PB][Q];
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const int k = k0 + i * GROUPS + group;
      x[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int q = 0; q < Q; ++q) v[i][q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (valid && has_part(k)) {
        const int64_t slot = (int64_t)k * 2 + (k < c ? 1 : 0);
        const float4 *po = reinterpret_cast<const float4 *>(p.part_o) + slot * (SLOT * D / 4) + r;
        x[i] = p.part_ml[slot * SLOT + r];
#pragma unroll
        for (int q = 0; q < Q; ++q) v[i][q] = po[(warp * Q + q) * SLOT];
      }
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < PB; ++i) top = fmaxf(top, x[i].x);
    if (top == -INFINITY) continue;
    const float w0 = ex2(m - top);
    m = top;
    l *= w0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      o[q].x *= w0;
      o[q].y *= w0;
      o[q].z *= w0;
      o[q].w *= w0;
    }
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const float w = ex2(x[i].x - top);
      l = fmaf(w, x[i].y, l);
      if (x[i].x == -INFINITY) continue;  // no visible key in this part: it may have no O
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        o[q].x = fmaf(w, v[i][q].x, o[q].x);
        o[q].y = fmaf(w, v[i][q].y, o[q].y);
        o[q].z = fmaf(w, v[i][q].z, o[q].z);
        o[q].w = fmaf(w, v[i][q].w, o[q].w);
      }
    }
  }
  __syncwarp();
  // the groups' shares of the row
#pragma unroll
  for (int step = ROWS; step < 32; step <<= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, step), top = fmaxf(m, om);
    const float w0 = top == -INFINITY ? 0.0f : ex2(m - top), w1 = top == -INFINITY ? 0.0f : ex2(om - top);
    m = top;
    l = l * w0 + __shfl_xor_sync(0xffffffffu, l, step) * w1;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      o[q].x = o[q].x * w0 + __shfl_xor_sync(0xffffffffu, o[q].x, step) * w1;
      o[q].y = o[q].y * w0 + __shfl_xor_sync(0xffffffffu, o[q].y, step) * w1;
      o[q].z = o[q].z * w0 + __shfl_xor_sync(0xffffffffu, o[q].z, step) * w1;
      o[q].w = o[q].w * w0 + __shfl_xor_sync(0xffffffffu, o[q].w, step) * w1;
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  if (group == 0) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      rows[lane % ROWS][warp * Q + q] =
          make_uint2(pack_bf16(o[q].x * inv, o[q].y * inv), pack_bf16(o[q].z * inv, o[q].w * inv));
    if (warp == 0 && valid)
      p.LSE[((int64_t)bd.head * p.G + r % BM - rt * p.G) * p.lse_shead + bd.tok0 + tok] =
          l > 0.0f ? (m + lg2(l)) * 0.69314718055994531f : -INFINITY;
  }
  __syncthreads();
  for (int i = warp; i < ROWS; i += 8) {
    const int ri = first_row + i, ti = (ri % BM) / p.G, tk = (ri / BM) * p.tpt + ti;
    if (ti >= p.tpt || tk >= bd.ntok) continue;
    uint2 *dst = reinterpret_cast<uint2 *>(
        p.O + ((int64_t)bd.tok0 + tk) * p.o_stok +
        ((int64_t)bd.head * p.G + ri % BM - ti * p.G) * p.o_shead);
    if (lane < D / 4) dst[lane] = rows[i][lane];
  }
}

template <int D, int RUNS, int SLOT>
__global__ void __launch_bounds__(256, 4) paged_combine_kernel(const Params p) {
  __shared__ uint2 rows[32][D / 4 + 1];
  pdl_wait();  // the parts and boundaries
  const int c = blockIdx.x + 1, y = blockIdx.y;
  const Boundary bd = p.bounds[c];
  const int tiles = bd.ntok > p.tpt ? 2 : 1;  // rows are numbered as in the unit's query tiles
  if (!bd.cut || y >= tiles * BM / 32) return;
  // no row of this block: those of a tile's tokens lie together from its first row on
  const int tok = bd.ntok - (y * 32 / BM) * p.tpt;
  if ((y * 32) % BM >= min(tok, p.tpt) * p.G) return;
  if (tile_at(p, run_start<RUNS>(bd.total, c - 1) - bd.u0, bd.w) > 0) return;
  // a single token's few rows, over many blocks' parts: the parts are shared out among lanes
  if (bd.ntok * p.G <= 8)
    combine_rows<D, RUNS, SLOT, 8>(p, bd, c, 0, rows);
  else
    combine_rows<D, RUNS, SLOT, 32>(p, bd, c, y * 32, rows);
}

size_t part_bytes(int d) { return (size_t)CTAS * 2 * 2 * BM * d * sizeof(float); }
size_t ml_bytes() { return (size_t)CTAS * 2 * 2 * BM * sizeof(float2); }

// Behind the kernel that made the parts: a boundary is a block's, 32 rows of it at a time.
template <int D, int RUNS, int SLOT>
cudaError_t launch_join(const PagedAttnArgs &a, const Params &p, cudaStream_t st) {
  // no sequence is longer than a key tile: no unit is cut
  if (((int64_t)a.seqs.max_pages << a.seqs.page_shift) <= BN) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(RUNS - 1, SLOT < 32 ? 1 : SLOT / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<D, RUNS, SLOT>, p);
}

template <int D, int WARPS>
cudaError_t launch_tokens(const PagedAttnArgs &a, Params p, cudaStream_t st) {
  using L = TokenLayout<D, WARPS>;
  p.tpt = p.utok = TOK_ROWS / p.G;
  if (may_have_chunks(a, p.G)) p.upto = 2 * p.utok;
  p.cost1 = p.cost2 = L::COST;
  p.overhead = L::OVERHEAD;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  constexpr size_t SLOTS = (size_t)L::RUNS * 2 * TOK_ROWS;
  static_assert(SLOTS * (D * 4 + 8) + L::RUNS * sizeof(Boundary) <= (size_t)CTAS * 4 * BM * D * 4, "workspace");
  p.part_o = reinterpret_cast<float *>(ws);
  p.part_ml = reinterpret_cast<float2 *>(ws + SLOTS * D * 4);
  p.bounds = reinterpret_cast<Boundary *>(ws + SLOTS * (D * 4 + 8));
  auto kernel = paged_token_kernel<D, WARPS>;
  static std::atomic<uint64_t> allowed{0};  // devices on which the kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  timing_mark(st, 0);
  kernel<<<L::RUNS, 32 * WARPS, L::ALLOC, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  timing_mark(st, 1);
  return launch_join<D, L::RUNS, TOK_ROWS>(a, p, st);
}

template <int D>
cudaError_t launch(const PagedAttnArgs &a, const WaitCfg &wc, cudaStream_t st) {
  using L = Layout<D>;
  Params p = {};
  p.s = a.seqs;
  p.total = a.total;
  p.G = a.H / a.Hkv;
  p.Hkv = a.Hkv;
  p.tpt = BM / p.G;
  p.utok = 2 * p.tpt;
  p.causal = a.causal;
  p.above = 0;
  p.upto = a.total;
  p.cost1 = L::COST1;
  p.cost2 = L::COST2;
  p.overhead = L::OVERHEAD;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.O = static_cast<__nv_bfloat16 *>(a.O);
  p.o_stok = a.o_stok;
  p.o_shead = a.o_shead;
  p.LSE = a.LSE;
  p.lse_shead = a.lse_shead;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  p.part_o = reinterpret_cast<float *>(ws);
  p.part_ml = reinterpret_cast<float2 *>(ws + part_bytes(D));
  p.bounds = reinterpret_cast<Boundary *>(ws + part_bytes(D) + ml_bytes());
  p.wc = wc;
  p.Q = static_cast<const __nv_bfloat16 *>(a.Q);
  p.q_stok = a.q_stok;
  p.q_shead = a.q_shead;
  p.kc = a.kc;
  p.vc = a.vc;
  // Few units are spread over the warps of one block an SM, more over two blocks, whose starts and
  // ends overlap (1,000 keys a sequence, 8 K/V heads: 2 sequences 10.8 us, 13.5 with two blocks;
  // 4 sequences 11.8 and 12.3; 8 15.6 and 14.2; 16 21.5 and 19.2)
  cudaError_t e;
  int mark = 0;  // kernel boundaries so far
  if (few_rows(a, p.G)) {
    e = (int64_t)a.seqs.batch * p.Hkv <= CTAS / 3 ? launch_tokens<D, 8>(a, p, st) : launch_tokens<D, 4>(a, p, st);
    if (e != cudaSuccess || !may_have_chunks(a, p.G)) return e;
    p.above = 2 * (TOK_ROWS / p.G);
    mark = 1;
  }
  // Q: {d, head, token}, a tile's box G heads of TPT tokens.  Strides of
  // extents of one are not given: any valid value does.
  CUtensorMap mq, mk, mv;
  const uint64_t row_bytes = (uint64_t)D * 2;
  const uint64_t dq[3] = {(uint64_t)D, (uint64_t)a.H, (uint64_t)a.total};
  const uint64_t sq[2] = {a.q_shead ? (uint64_t)a.q_shead * 2 : row_bytes,
                          a.q_stok ? (uint64_t)a.q_stok * 2 : row_bytes};
  const uint32_t bq[3] = {64, (uint32_t)p.G, (uint32_t)p.tpt};
  // K, V: {d, slot, head, page}
  const int page = 1 << a.seqs.page_shift;
  const uint64_t dk[4] = {(uint64_t)D, (uint64_t)page, (uint64_t)a.Hkv, (uint64_t)a.seqs.num_pages};
  const uint64_t sk[3] = {(uint64_t)a.kc.s_slot * 2, (uint64_t)a.kc.s_head * 2, (uint64_t)a.kc.s_page * 2};
  const uint64_t sv[3] = {(uint64_t)a.vc.s_slot * 2, (uint64_t)a.vc.s_head * 2, (uint64_t)a.vc.s_page * 2};
  const uint32_t bk[4] = {64, (uint32_t)(page < BN ? page : BN), 1, 1};
  // A token's row of one K/V head is 128 bytes at d = 64, and the bytes after it belong to
  // another head, which another unit reads much later: fetched 256 at a time, they are read for
  // nothing (single tokens of 64 sequences of 8,192 keys, 64 heads on 2: 75 us, 79 with 256).  At
  // d = 128 the row is the 256 bytes.
  const CUtensorMapL2promotion promote =
      D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  if ((e = make_tmap(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.Q, dq, sq, bq)) != cudaSuccess ||
      (e = make_tmap(&mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.kc.ptr, dk, sk, bk, promote)) != cudaSuccess ||
      (e = make_tmap(&mv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.vc.ptr, dk, sv, bk, promote)) != cudaSuccess)
    return e;
  e = cudaFuncSetAttribute(paged_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
  if (e != cudaSuccess) return e;
  if (mark == 0) timing_mark(st, 0);
  paged_attn_kernel<D><<<CTAS, THREADS, L::ALLOC, st>>>(mq, mk, mv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  timing_mark(st, mark + 1);
  return launch_join<D, CTAS, 2 * BM>(a, p, st);
}

}  // namespace

size_t paged_attn_workspace(int d) { return part_bytes(d) + ml_bytes() + CTAS * sizeof(Boundary) + 256; }

cudaError_t launch_paged_attn(const PagedAttnArgs &a, const WaitCfg &wc, cudaStream_t st) {
  return a.d == 128 ? launch<128>(a, wc, st) : launch<64>(a, wc, st);
}

}  // namespace chain
