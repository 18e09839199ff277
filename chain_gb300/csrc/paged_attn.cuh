// paged_attn.cuh -- softmax attention of a chunk of new tokens over a paged
// K/V cache (the unit O = f(A B) C with f = row softmax, K and V read from
// the pages that a sequence's table names): the kernels of paged_attn.cu, and in two more
// forms, MODE, of prefix_attn.cu, which says what those are for.
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
//   warp 9     MMA issuer, one lane of it through a unit's steps.
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
//   chunks: the tensor pipe, 77% busy at d = 128, and the chain that leaves the rest of it.  2,048 tokens over
//   32,768: 877 us, 1,215 TFLOP/s (P_lo's product not counted): a stream's softmax and its three products
//   follow each other, since P shares S's columns; two streams overlap them.  In copies made to be timed only, without any
//   softmax it takes 733 us, without P_lo and its product 691, without the exponentials no less.  d = 64: 703 us,
//   757 TFLOP/s.
//   single tokens: memory.  d = 128, 64 sequences of 8,192: 324 us, 2.15 GB at 6.6 TB/s;
//   d = 64: 184 us, 1.07 GB at 5.9 TB/s.  One sequence of 131,072: 89 us, 6.0 TB/s, with
//   the start, the join and the ends of the runs; of 100: 6.7 us, all latency.
#pragma once
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

// ALONE: each sequence's keys, into O.  SHARED: the sequences of a group as one, whose keys are the
// group's prefix, into unnormalised sums of 32 bits.  OWN: each sequence's keys behind its group's prefix,
// joined with those sums.
enum : int { ALONE, SHARED, OWN };

// One unit's part of a block's run, as the scheduler hands it over.
struct Unit {
  int tok0, ntok;  // packed rows
  int head, b;     // K/V head (-1: no more units), sequence
  int j0, j1;      // key tiles
  int ja;          // end of the key tiles that tile 0 sees
  int lim0;        // keys that the first token sees (any value up to len)
  int len;         // keys of the sequence
  int slot;        // -1: all of the unit's key tiles, else the workspace slot
  int pre;         // OWN: the rows have sums of their group's prefix
};
static_assert(sizeof(Unit) <= 48, "unit ring");

// Where a run begins, for the join: written by every block, cut or not.
struct Boundary {
  long long u0;     // cost at which the unit that it falls into begins
  long long total;  // cost of all units
  int nt, w;        // the unit's key tiles, cost of each
  short cut;        // it falls behind the unit's first key tile
  short pre;        // as a unit's
  int tok0, ntok, head;
};

template <int D>
struct Layout {
  static constexpr uint32_t TILE = BM * D * 2;  // a Q, K or V tile
  static constexpr int NS = D == 128 ? 5 : 12;  // 160 or 192 KB of K and V in flight
  // Costs, in quarters of a key tile against one query tile, chosen by time over mixed batches (24
  // chunks and tokens of up to 300 over up to 5,000 keys, 32 heads of 128 on 8 / 15 of 64 on 5: 278 us /
  // 123 us then, 251 / 109 now; with 5, 14 / 6, 20 for the last two 296 / 125 then, with 6, 9 / 7, 12 284 / 130).  The last is a
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
  // SHARED, OWN: group g is the sequences [group_cu[g], group_cu[g + 1]), whose first
  // group_lens[g] positions lie in the same pages
  const int *group_cu, *group_lens;
  int groups;
  float *pre_o;    // [Hkv][D / 4][total G][4]; null: no prefix is taken together
  float2 *pre_ml;  // [Hkv][total G]
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

// tmem_ld32, and the largest of the lane's 32 columns as fp32.
__device__ __forceinline__ float tmem_ld32_max(uint32_t taddr, uint32_t (&r)[32]) {
  float top;
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]),
        "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=f"(top)
      : "r"(taddr)
      : "memory");
  return top;
}

// What a row's sums give: 1 / l and the LSE.  l is 0 where the row sees no key (a sum has at least 2^0 from its largest
// score), and NaN where a score is NaN or +infinity: a maximum does not show that, the sum does, so every
// join keeps it, and the row's O and LSE become NaN with it.
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + lg2(l)) * 0.69314718055994531f;
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
  int j;           // first key tile (0 but with OWN)
};

// Sequences of the work; with SHARED a group is one.
template <int MODE>
__device__ __forceinline__ int seqs_of(const Params &p) {
  return MODE == SHARED ? p.groups : p.s.batch;
}

// The positions of a group's prefix that are taken together: whole key tiles.
__device__ __forceinline__ int shared_len(const Params &p, int len) {
  const int most = p.s.max_pages << p.s.page_shift;
  return (len < 0 ? 0 : (len > most ? most : len)) & ~(BN - 1);
}

// The group of sequence b, or -1.
__device__ __forceinline__ int group_of(const Params &p, int b) {
  int lo = 0, hi = p.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.group_cu + mid) <= b)
      lo = mid;
    else
      hi = mid;
  }
  return __ldg(p.group_cu + lo) <= b && b < __ldg(p.group_cu + lo + 1) ? lo : -1;
}

// The packed rows of sequences [b0, b1).
__device__ __forceinline__ Seq rows_of(const Params &p, int b0, int b1) {
  int lo = __ldg(p.s.cu + b0), hi = __ldg(p.s.cu + b1);
  lo = lo < 0 ? 0 : (lo > p.total ? p.total : lo);
  hi = hi < lo ? lo : (hi > p.total ? p.total : hi);
  return Seq{lo, hi - lo, 0, 0};
}

// The sequences of group g.
__device__ __forceinline__ int2 members(const Params &p, int g) {
  int b0 = __ldg(p.group_cu + g), b1 = __ldg(p.group_cu + g + 1);
  b0 = b0 < 0 ? 0 : (b0 > p.s.batch ? p.s.batch : b0);
  b1 = b1 < b0 ? b0 : (b1 > p.s.batch ? p.s.batch : b1);
  return make_int2(b0, b1);
}

template <int MODE>
__device__ __forceinline__ Seq seq_of(const Params &p, int b, bool report) {
  Seq s;
  if (MODE == SHARED) {
    const int2 m = members(p, b);
    s = rows_of(p, m.x, m.y);
    s.len = shared_len(p, __ldg(p.group_lens + b));
    if (s.len == 0) s.n = 0;
  } else {
    s = rows_of(p, b, b + 1);
    s.len = __ldg(p.s.lens + b);
    const int most = p.s.max_pages << p.s.page_shift;
    if (s.len < 0 || s.len > most) {
      if (report) atomicExch(&p.wc.status->reserved[0], 1);
      s.len = s.len < 0 ? 0 : most;
    }
    if (MODE == OWN) {
      const int g = group_of(p, b);
      if (g >= 0) {
        const int len = __ldg(p.group_lens + g);
        if (p.pre_o) s.j = shared_len(p, len) / BN;
        // every new token must see the whole prefix
        if (report && s.n > 0 && (len < 0 || len > (p.causal ? s.len - s.n : s.len)))
          atomicExch(&p.wc.status->reserved[0], 1);
      }
    }
  }
  if (!(s.n > p.above && s.n <= p.upto)) s.n = 0;
  return s;
}

// A sequence whose table names the pages of sequence b: with SHARED the group's first that
// has new tokens (the others may be padding), found by the warp.
template <int MODE>
__device__ __forceinline__ int table_of(const Params &p, int b, int lane) {
  if (MODE != SHARED) return b;
  const int2 m = members(p, b);
  for (int c = m.x; c < m.y; c += 32) {
    const bool has = c + lane < m.y && rows_of(p, c + lane, c + lane + 1).n > 0;
    const uint32_t hit = __ballot_sync(0xffffffffu, has);
    if (hit) return c + __ffs(hit) - 1;
  }
  return m.x;
}

// Key tiles, from the sequence's first on, that tokens below `end` of it see; at least one, so
// that rows which see nothing are still written.
__device__ __forceinline__ int tiles_to(const Params &p, const Seq &s, int end) {
  const int seen = p.causal ? s.len - s.n + (end < s.n ? end : s.n) : s.len;
  return seen <= BN * (s.j + 1) ? 1 : (seen + BN - 1) / BN - s.j;
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
template <int MODE>
__device__ __forceinline__ Place locate(const Params &p, const long long *sums, long long t, int lane) {
  Place at = {0, 0, 0, 0};
  const int count = seqs_of<MODE>(p);
  for (int c = 0; c < count && count > 1; c += 32) {
    const int l = find(c + lane < count ? sums[c + lane] * p.Hkv : 0, t, lane);
    if (l >= 0) {
      at.b = c + l;
      break;
    }
  }
  const Seq s = seq_of<MODE>(p, at.b, false);
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

// The first run that begins at cost x or behind it.
template <int RUNS>
__device__ __forceinline__ int run_from(long long total, long long x) {
  return (int)min(quotient(x * RUNS + total - 1, total), (long long)RUNS);
}

// A block's run: what is left of it, and where it goes on.
struct Run {
  long long t, t1;  // cost offsets into all of the work
  Place at;
  Seq s;
};

// A warp finds where the block's run begins, writes its boundary, and says whether
// there is anything in it.
template <int RUNS, int MODE>
__device__ __forceinline__ bool begin_run(const Params &p, const long long *sums, Run &r, int lane) {
  long long total = 0;
  for (int b = lane; b < seqs_of<MODE>(p); b += 32) total += sums[b];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total *= p.Hkv;
  r.t = run_start<RUNS>(total, blockIdx.x);
  r.t1 = run_start<RUNS>(total, blockIdx.x + 1);
  r.at = Place{0, 0, 0, 0};
  r.s = Seq{0, 0, 0, 0};
  Boundary bd = {0, total, 0, 1, 0, 0, 0, 0, 0};
  bool work = false;
  if (r.t < total) {
    r.at = locate<MODE>(p, sums, r.t, lane);
    r.s = seq_of<MODE>(p, r.at.b, false);
    const int i0 = r.at.q * p.utok;
    bd.u0 = r.t - r.at.off;
    bd.nt = tiles_to(p, r.s, i0 + p.utok);
    bd.w = tile_cost(p, r.s.n - i0);
    bd.cut = tile_at(p, r.at.off, bd.w) > 0;
    bd.pre = r.s.j > 0;
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

// The run's next unit, found by a warp; head = -1 at its end.
template <int MODE>
__device__ __forceinline__ Unit next_of(const Params &p, Run &r, int lane) {
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
      u.b = table_of<MODE>(p, r.at.b, lane);
      u.ja = r.s.j + tiles_to(p, r.s, i0 + p.tpt);
      u.lim0 = p.causal ? r.s.len - r.s.n + i0 + 1 : r.s.len;
      u.len = r.s.len;
      u.slot = u.j0 > 0 ? 0 : (u.j1 < nt ? 1 : -1);
      u.pre = r.s.j > 0;
      u.j0 += r.s.j;
      u.j1 += r.s.j;
    }
    r.t += cost - r.at.off;
    // on to the next unit: of the head, the next head, the next sequence with new tokens
    r.at.off = 0;
    if (r.t < r.t1 && ++r.at.q == units_of(p, r.s)) {
      r.at.q = 0;
      if (++r.at.head == p.Hkv) {
        r.at.head = 0;
        do {
          r.s = seq_of<MODE>(p, ++r.at.b, false);
        } while (r.s.n == 0 && r.at.b + 1 < seqs_of<MODE>(p));
      }
    }
  }
  return u;
}

// --------------------------------------------------------------- main kernel
template <int D, int MODE>
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
  for (int b = threadIdx.x; b < seqs_of<MODE>(p); b += THREADS)
    sums[b] = head_cost(p, seq_of<MODE>(p, b, blockIdx.x == 0));
  fence_proxy_async_smem();  // the ring's first copies come after these writes and their reads
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();  // the join may be launched; it waits for this grid

  // The scheduler warp finds where the block's run begins.
  Run run;
  if (warp == 10) {
    const bool work = begin_run<CTAS, MODE>(p, sums, run, lane);
    if (lane == 0) *has_work = work;
  }
  __syncthreads();
  if (!*has_work) {
    if (warp == 9) tmem_dealloc(tmem, 512);
    if (MODE == OWN) pdl_wait();
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
      const Unit u = next_of<MODE>(p, run, lane);
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
      // A sequence that has nothing behind its prefix still has one tile, and the page that the prefix ends in may hold
      // anything there: no page of it has keys.  (A tile that the sequence's end falls into: see `tail`.)
      const int len = u.j0 * BN < u.len ? u.len : 0;
      auto keys_at = [&](int at) { return ((long long)at << p.s.page_shift) < len; };
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
  // mixed sequences no faster, and every buffer freed by two warps that run apart.  At d = 128: halves of 64 keys, a
  // half's next S behind its product, while the softmax is at the other half: twice the exchanges, 1,030 us -> 1,450.
  // One elected lane goes through a unit's steps by itself: the pipe holds few products, so that what lies between a
  // step's last and the next one's first shows whole.  (Elected step by step, the waits by a lane and their outcome
  // exchanged, the chunk at d = 128 959 us that takes 867.)
  auto role_mma = [&]() {
    const uint32_t idS = idesc_bf16_f32(BM, BN, 0, 0), idO = idesc_bf16_f32(BM, D, 0, 1);
    const SDesc dQ = sdesc_make(smem_u32(smem + L::OFF_Q), 16, 1024);
    const SDesc dK = sdesc_make(smem_u32(smem + L::OFF_RING), 16, 1024);
    const SDesc dV = sdesc_make(smem_u32(smem + L::OFF_RING), BN * 128, 1024);
    Unit u;
    int k = 0;
    uint32_t q_uses[2] = {0, 0}, qsel = 0;
    uint32_t base = 0;             // ring number of the unit's first K tile
    uint32_t steps[2] = {0, 0};    // P V products of each stream before the unit
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return mbar_wait_warp(bar, parity, p.wc, abort_flag, SITE_PAGED_MMA);
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
      auto there = [&](uint32_t seq) {
        return mbar_wait(&full[seq % NS], (seq / NS) & 1, p.wc, abort_flag, SITE_PAGED_MMA);
      };
      // The last page may hold anything behind the sequence's end, and 0 times a NaN is not 0: those rows of the
      // last tile's V become zeros, by the warp, before the unit's last steps.
      const int valid = u.len - (u.j1 - 1) * BN, count = two ? n : (n + 1) / 2;
      const bool tail = valid > 0 && valid < BN;
#pragma unroll 1
      for (int last = 0; ok && last < (tail ? 2 : 1); ++last) {
        if (last) {
          const uint32_t seq = base + 2 * n - 1, st = seq % NS;
          ok = wait(&full[st], (seq / NS) & 1);
          if (!ok) break;
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
        if (elect_one()) {
          if (!last)
#pragma unroll
            for (int t = 0; t < 2; ++t)
              if (ok && ns[t] > 0 && (ok = there(k_seq(t, 0)))) {
                tc_fence_after();
                put_s(t, 0);
              }
          const int end = tail && !last ? count - 1 : count;
#pragma unroll 1
          for (int i = last ? count - 1 : 0; ok && i < end; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || i >= ns[t]) continue;
              // O_t += P_hi V + P_lo V of step i; stream 1 finds the tiles there that stream 0 has waited for
              const uint32_t seq = k_seq(t, i) + 1, st = seq % NS, vo = st * L::TILE;
              const bool seen = two && t == 1 && i < ns[0];
              ok = (seen || there(seq)) &&
                   mbar_wait(&p_ready[t], (steps[t] + i) & 1, p.wc, abort_flag, SITE_PAGED_MMA);
              if (!ok) continue;
              tc_fence_after();
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                  umma_f16_ts(tmem + L::o_col(t), tmem + t * BN + kk * 16 + part * 8, sdesc_at(dV, vo + kk * 2048), idO,
                              i > 0 || part > 0 || kk > 0);
              umma_commit(&pv_done[t]);
              if (last_reader(t)) umma_commit(&empty[st]);
              if (i + 1 < ns[t] && (ok = (seen && i + 1 < ns[0]) || there(k_seq(t, i + 1)))) {
                tc_fence_after();
                put_s(t, i + 1);
              }
            }
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, ok);
      }
      steps[0] += ns[0];
      steps[1] += ns[1];
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
          // In loops, S read twice from tensor memory, the first time for its maximum, which the load brings (the
          // chunk 868 us, 858 so; 32 chunks behind 16,384 shared positions 333 and 324): straight through the 128
          // columns the instructions came from memory at a launch's start and not all of them stayed beside the other
          // stream's.  Other loops of 32 to 128 columns, or with the next load under way: 2% slower to 2% faster on
          // long runs, 2 to 6% slower on 24 mixed sequences.
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < BN; c += 64) {
            if (__any_sync(0xffffffffu, kv0 + c + 64 > lim)) {
#pragma unroll 1
              for (int d = c; d < c + 64; d += 32) {
                uint32_t s[32];
                tmem_ld32(tS + d, s);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (kv0 + d + e >= lim) s[e] = __float_as_uint(-INFINITY);
                __syncwarp();  // the lanes' limits differ, the store is the whole warp's
                tmem_st32(tS + d, s);
              }
              tmem_wait_st();
            }
            uint32_t s[2][32];
            const float a = tmem_ld32_max(tS + c, s[0]), b = tmem_ld32_max(tS + c + 32, s[1]);
            tmem_wait_ld();
            mx = fmax3(mx, a, b);
          }
          mx *= p.scale_log2;
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
#pragma unroll 1
          for (int c = 0; c < BN; c += 32) {
            uint32_t s[32];
            tmem_ld32(tS + c, s);
            tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < 2; ++g) {
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
                float y0, y1;
                f32x2_split(fma_f32x2(f32x2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u)), f32x2(-1.0f, -1.0f), f32x2(p0, p1)), y0, y1);
                pk[8 + (e >> 1)] = pack_bf16(y0, y1);
              }
              tmem_st16(tS + c + g * 16, pk);
            }
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
        } else {
          l += o.y;  // 0 or NaN
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
        const bool sums_out = MODE == SHARED || !whole;
        // the row's sums over its group's prefix
        const int64_t pre_pitch = (int64_t)p.total * p.G;
        const int64_t pre_row = ((int64_t)u.tok0 + tok) * p.G + rhead;
        float4 *pre = reinterpret_cast<float4 *>(p.pre_o) + u.head * (D / 4) * pre_pitch + pre_row;
        float wp = 0.0f;
        if (MODE == OWN && whole && u.pre) {
          pdl_wait();
          if (valid) {
            const float2 x = p.pre_ml[u.head * pre_pitch + pre_row];
            const float top = fmaxf(m, x.x), f = top == -INFINITY ? 0.0f : ex2(m - top);
            wp = top == -INFINITY ? 0.0f : ex2(x.x - top);
            w[0] *= f;
            w[1] *= f;
            l = l * f + x.y * wp;
            m = top;
          }
          __syncwarp();
        }
        if (!sums_out) {
          const float inv = inverse(l);
          w[0] *= inv;
          w[1] *= inv;
          wp *= inv;
          __syncwarp();  // the division may part the lanes; the loads below are the whole warp's
        }
        const int64_t qhead = (int64_t)u.head * p.G + rhead;
        __nv_bfloat16 *orow = p.O + ((int64_t)u.tok0 + tok) * p.o_stok + qhead * p.o_shead;
        // a slot's O is [D / 4][2 BM][4], so that lanes, which hold rows, write side by side
        const int64_t slot = (int64_t)blockIdx.x * 2 + u.slot;
        float4 *prow = MODE == SHARED && whole
                           ? pre
                           : reinterpret_cast<float4 *>(p.part_o) + slot * (2 * BM * D / 4) + t * BM + row;
        const int64_t pitch = MODE == SHARED && whole ? pre_pitch : 2 * BM;
#pragma unroll 1
        for (int c = 0; c < D / 32 && (has[0] || has[1]); ++c) {
          uint32_t x[32];
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.0f;
          if (MODE == OWN && whole && u.pre) {
            if (valid) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 x = pre[(c * 8 + e) * pre_pitch];
                o[4 * e] = x.x * wp;
                o[4 * e + 1] = x.y * wp;
                o[4 * e + 2] = x.z * wp;
                o[4 * e + 3] = x.w * wp;
              }
            }
            __syncwarp();
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (!has[y]) continue;
            tmem_ld32(tmem + lane_off + L::o_col(y) + c * 32, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(x[e]), w[y], o[e]);
          }
          if (!sums_out) {
            uint4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
            store_rows(v, orow + c * 32, valid, lane);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (valid) prow[(c * 8 + e) * pitch] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          __syncwarp();
        }
        if (valid) {
          if (!sums_out)
            p.LSE[qhead * p.lse_shead + u.tok0 + tok] = lse_of(m, l);
          else if (MODE == SHARED && whole)
            p.pre_ml[u.head * pre_pitch + pre_row] = make_float2(m, l);
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
  // the join behind this kernel reads the prefixes' sums: this grid does not end before they are there
  if (MODE == OWN) pdl_wait();
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
// the kernel above.  Two stages of 8 KB a warp; a third, or more blocks, made the memory slower (64 sequences
// of up to 16,384: 356 us with two stages, 374 with three).  A unit is joined while the next one's first stage and Q
// are under way, through shared memory of its own (that batch 364 -> 329 us, one sequence of 131,072 102 -> 92).
constexpr int TOK_ROWS = 16;
template <int D, int WARPS>
struct TokenLayout {
  static constexpr int BLOCKS = 8 / WARPS, RUNS = CTAS * BLOCKS;
  static constexpr int KEYS = BN / WARPS;                       // of a key tile, a warp's
  static constexpr int KS = KEYS < 2048 / D ? KEYS : 2048 / D;  // of a stage: 8 KB of K and V at most
  static constexpr int STAGES = 2;
  static constexpr uint32_t HALF = KS * D * 2, STAGE = 2 * HALF;
  static constexpr uint32_t WARP = STAGES * STAGE;  // a warp's ring
  static constexpr int OPITCH = D + 4;
  static constexpr uint32_t SHARE = TOK_ROWS * OPITCH * 4;  // a warp's O, beside the rings: the next unit's keys are
                                                            // under way while a unit is joined
  static constexpr uint32_t ALLOC = WARPS * (WARP + SHARE);
  static constexpr int COST = 4, OVERHEAD = D == 128 ? 4 : 8;
  static_assert(MAX_BATCH * 8 <= ALLOC, "the schedule's sums use the rings");
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

template <int D, int WARPS, int MODE>
__global__ void __launch_bounds__(32 * WARPS, TokenLayout<D, WARPS>::BLOCKS) paged_token_kernel(const Params p) {
  using L = TokenLayout<D, WARPS>;
  constexpr int CH = D / 8;             // 16-byte chunks of a row
  constexpr int RPC = 32 / CH;          // rows that a copy of the warp covers
  constexpr int PER = L::KEYS / L::KS;  // stages of a key tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ Unit next[2];
  __shared__ float2 ml[WARPS][TOK_ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long *sums = reinterpret_cast<long long *>(smem_raw);
  for (int b = threadIdx.x; b < seqs_of<MODE>(p); b += 32 * WARPS)
    sums[b] = head_cost(p, seq_of<MODE>(p, b, blockIdx.x == 0));
  __syncthreads();
  pdl_launch_dependents();  // the join may be launched; it waits for this grid
  Run run;
  if (warp == 0) begin_run<L::RUNS, MODE>(p, sums, run, lane);
  const uint32_t ring = smem_u32(smem_raw) + warp * L::WARP;
  const int page = 1 << p.s.page_shift, pool = (int)p.s.num_pages;
  float *mine = reinterpret_cast<float *>(smem_raw + WARPS * L::WARP + warp * L::SHARE);
  auto publish = [&](Unit &to) {  // by warp 0
    const Unit n = next_of<MODE>(p, run, lane);
    if (lane == 0) to = n;
  };
  if (warp == 0) publish(next[0]);
  __syncthreads();
  Unit u = next[0], done = {};
  bool first = true;
  for (int turn = 0;; turn ^= 1) {
    // What the unit needs first: its first stage and Q, asked for while the unit before is joined.
    const int steps = u.head < 0 ? 0 : (u.j1 - u.j0) * PER;
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
    if (!first) {  // joins the warps' shares of the unit before
      constexpr int COLS = D / 8;  // a thread's, of row threadIdx.x / 8
      const int row = threadIdx.x >> 3, c0 = (threadIdx.x & 7) * COLS, tok = row / p.G;
      if (row < TOK_ROWS && tok < done.ntok && tok < p.tpt) {
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
              reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem_raw + WARPS * L::WARP + w * L::SHARE) + row * L::OPITCH + c0);
#pragma unroll
          for (int c = 0; c < COLS / 4; ++c) {
            const float4 y = src[c];
            x[4 * c] = fmaf(y.x, f, x[4 * c]);
            x[4 * c + 1] = fmaf(y.y, f, x[4 * c + 1]);
            x[4 * c + 2] = fmaf(y.z, f, x[4 * c + 2]);
            x[4 * c + 3] = fmaf(y.w, f, x[4 * c + 3]);
          }
        }
        const int64_t pre_pitch = (int64_t)p.total * p.G, pre_row = (int64_t)done.tok0 * p.G + row;
        float4 *pre = reinterpret_cast<float4 *>(p.pre_o) + (done.head * (D / 4) + c0 / 4) * pre_pitch + pre_row;
        if (MODE == OWN && done.slot < 0 && done.pre) {  // the row's sums over its group's prefix
          pdl_wait();
          const float2 v = p.pre_ml[done.head * pre_pitch + pre_row];
          const float high = fmaxf(top, v.x), f = high == -INFINITY ? 0.0f : ex2(top - high);
          const float g = high == -INFINITY ? 0.0f : ex2(v.x - high);
          top = high;
          sum = fmaf(sum, f, v.y * g);
#pragma unroll
          for (int c = 0; c < COLS / 4; ++c) {
            const float4 y = pre[c * pre_pitch];
            x[4 * c] = fmaf(x[4 * c], f, y.x * g);
            x[4 * c + 1] = fmaf(x[4 * c + 1], f, y.y * g);
            x[4 * c + 2] = fmaf(x[4 * c + 2], f, y.z * g);
            x[4 * c + 3] = fmaf(x[4 * c + 3], f, y.w * g);
          }
        }
        if (MODE == SHARED && done.slot < 0) {
#pragma unroll
          for (int c = 0; c < COLS / 4; ++c)
            pre[c * pre_pitch] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
          if ((threadIdx.x & 7) == 0) p.pre_ml[done.head * pre_pitch + pre_row] = make_float2(top, sum);
        } else if (done.slot < 0) {
          const float inv = inverse(sum);
          const int64_t qhead = (int64_t)done.head * p.G + row - tok * p.G;
          uint4 *dst = reinterpret_cast<uint4 *>(p.O + ((int64_t)done.tok0 + tok) * p.o_stok + qhead * p.o_shead + c0);
#pragma unroll
          for (int c = 0; c < COLS / 8; ++c)
            dst[c] = make_uint4(pack_bf16(x[8 * c] * inv, x[8 * c + 1] * inv), pack_bf16(x[8 * c + 2] * inv, x[8 * c + 3] * inv),
                                pack_bf16(x[8 * c + 4] * inv, x[8 * c + 5] * inv),
                                pack_bf16(x[8 * c + 6] * inv, x[8 * c + 7] * inv));
          if ((threadIdx.x & 7) == 0)
            p.LSE[qhead * p.lse_shead + done.tok0 + tok] = lse_of(top, sum);
        } else {
          const int64_t slot = (int64_t)blockIdx.x * 2 + done.slot;
          float4 *dst = reinterpret_cast<float4 *>(p.part_o) + slot * (TOK_ROWS * D / 4) + row;
#pragma unroll
          for (int c = 0; c < COLS / 4; ++c)
            dst[(c0 / 4 + c) * TOK_ROWS] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
          if ((threadIdx.x & 7) == 0) p.part_ml[slot * TOK_ROWS + row] = make_float2(top, sum);
        }
      }
      __syncthreads();  // the shares and ml are free
    }
    first = false;
    if (u.head < 0) break;
    if (warp == 0) publish(next[turn ^ 1]);
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
    // the warps' shares
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
    done = u;
    u = next[turn ^ 1];
  }
  if (MODE == OWN) pdl_wait();  // as above
}

// Whether a call's rows may be few: with a query head's group that fits 16 rows, no more new
// tokens than sequences, or so few that they fit one tile.  Single tokens, 32 heads on 8, this kernel
// and the one above: 64 sequences of 300 at d = 64 16.2 us and 36.3, at d = 128 22.6 and 42.6; of
// 1,000 53 and 70, of 4,000 167 and 191, of 8,192 324 and 355 (d = 64 184 and 215); 200 of 300 59 and 110.
// One sequence of 100: 6.7 and 11.5, of 4,096: 13.1 and 16.6, of 131,072: 89 and 102.
bool few_rows(const PagedAttnArgs &a, int G) {
  return G <= TOK_ROWS && (a.total <= a.seqs.batch || (int64_t)a.total * G <= TOK_ROWS);
}
// The counts themselves are on the device.  As many tokens as sequences are single tokens but for a
// coincidence; fewer may be a chunk in a batch that is padded with empty sequences, whose keys 16-row
// tiles would read once for every 16 rows.  Then sequences of more than two tiles are left to a launch
// of the kernel above, which finds nothing to do where there are none (32 heads on 8, d = 128, a batch
// of 256 padded with empty sequences: 200 tokens over 8,192 keys 52 us, 158 without that launch; 64 single
// tokens over 300 keys 27 and 23).
bool may_have_chunks(const PagedAttnArgs &a, int G) {
  return a.total < a.seqs.batch && (int64_t)a.total * G > 2 * TOK_ROWS;
}

// Joins a unit that runs' ends cut into parts: block (c, y) the unit that
// boundary c + 1 falls into, if that is the unit's first boundary.  A block takes
// `ROWS` rows and a warp D / 8 columns of them; a lane takes a row, as in the
// parts, and every GROUPS-th part of it, PB loaded at once: the kernel is a
// few dependent loads long.  Rows go out through shared memory.
template <int D, int RUNS, int SLOT, int MODE, int ROWS>
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
  // OWN: where runs are shorter than a key tile, by the unit's tiles and the runs that hold them: of 152 runs over
  // four tiles four have a part (84 rows 34 us by runs, 8 by tiles)
  const bool by_tile = MODE == OWN && tiny;
  auto run_of = [&](int j) {
    return run_from<RUNS>(bd.total, bd.u0 + p.overhead + (long long)bd.w * (j + 1)) - 1;
  };
  for (int k0 = by_tile ? 0 : c - 1; by_tile ? k0 < bd.nt : in_unit(k0); k0 += PB * GROUPS) {
    float2 x[PB];
    float4 v[PB][Q];
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      int k = k0 + i * GROUPS + group;
      bool part;
      if (by_tile) {
        const int j = k;
        k = run_of(j);
        part = j < bd.nt && (j == 0 || run_of(j - 1) != k);
      } else {
        part = has_part(k);
      }
      x[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int q = 0; q < Q; ++q) v[i][q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (valid && part) {
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
    if (top == -INFINITY) {
#pragma unroll
      for (int i = 0; i < PB; ++i) l += x[i].y;  // 0 or NaN
      continue;
    }
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
  const int64_t pre_pitch = (int64_t)p.total * p.G;
  const int64_t pre_row = ((int64_t)bd.tok0 + tok) * p.G + r % BM - rt * p.G;
  float4 *pre = reinterpret_cast<float4 *>(p.pre_o) + (bd.head * (D / 4) + warp * Q) * pre_pitch + pre_row;
  if (MODE == OWN && bd.pre && valid) {  // the row's sums over its group's prefix
    const float2 x = p.pre_ml[bd.head * pre_pitch + pre_row];
    const float top = fmaxf(m, x.x);
    const float w0 = top == -INFINITY ? 0.0f : ex2(m - top), w1 = top == -INFINITY ? 0.0f : ex2(x.x - top);
    m = top;
    l = l * w0 + x.y * w1;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float4 y = pre[q * pre_pitch];
      o[q].x = o[q].x * w0 + y.x * w1;
      o[q].y = o[q].y * w0 + y.y * w1;
      o[q].z = o[q].z * w0 + y.z * w1;
      o[q].w = o[q].w * w0 + y.w * w1;
    }
  }
  const float inv = inverse(l);
  if (group == 0) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      rows[lane % ROWS][warp * Q + q] =
          make_uint2(pack_bf16(o[q].x * inv, o[q].y * inv), pack_bf16(o[q].z * inv, o[q].w * inv));
    if (warp == 0 && valid)
      p.LSE[((int64_t)bd.head * p.G + r % BM - rt * p.G) * p.lse_shead + bd.tok0 + tok] = lse_of(m, l);
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

template <int D, int RUNS, int SLOT, int MODE>
__global__ void __launch_bounds__(256, 4) paged_combine_kernel(const Params p) {
  static_assert(MODE != SHARED, "the prefix's parts are joined by shared_join_kernel");
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
    combine_rows<D, RUNS, SLOT, MODE, 8>(p, bd, c, 0, rows);
  else
    combine_rows<D, RUNS, SLOT, MODE, 32>(p, bd, c, y * 32, rows);
}

// The same with SHARED, whose units have many rows and may have many parts, into the sums that OWN joins.
// A block takes ROWS rows, a lane a row, as in the parts (with 16 rows, half a warp's lanes take other parts).  Of a few
// parts a warp takes COLS float4 of every row, and the unit's first boundary all columns; many parts are dealt to the
// warps, PB loaded at once, and the unit's boundaries share its columns out.  The groups' sums are joined
// through shared memory.  With a warp to each D / 8 columns and the parts one after another, as above, 48 rows of 76 parts
// took 38 us, 8 now; 256 rows of 19 parts 13.7, 10 now (each launch by itself, second-level cache cold).  As one block an SM
// that loops, so that OWN's first blocks run beside it, the whole call was 3% slower.
template <int ROWS>
struct JoinShared {
  static constexpr int COLS = 4, GROUPS = 8 * (32 / ROWS);
  float4 part[GROUPS][COLS][ROWS];
  float2 ml[GROUPS][ROWS];
};

// A lane's share of its row: parts first, first + step, ... below last, columns [col0, col0 + COLS).
template <int D, int SLOT, int PB, int COLS, typename F>
__device__ __forceinline__ void join_parts(const Params &p, int c, int first, int step, int last, int r, int col0,
                                           const F &has_part, float &m, float &l, float4 (&o)[COLS]) {
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int q = 0; q < COLS; ++q) o[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k0 = first; k0 < last; k0 += PB * step) {
    float2 x[PB];
    float4 v[PB][COLS];
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const int k = k0 + i * step;
      x[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int q = 0; q < COLS; ++q) v[i][q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (k < last && has_part(k)) {
        const int64_t slot = (int64_t)k * 2 + (k < c ? 1 : 0);
        const float4 *po = reinterpret_cast<const float4 *>(p.part_o) + (slot * (D / 4) + col0) * SLOT + r;
        x[i] = p.part_ml[slot * SLOT + r];
#pragma unroll
        for (int q = 0; q < COLS; ++q) v[i][q] = po[q * SLOT];
      }
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < PB; ++i) top = fmaxf(top, x[i].x);
    if (top == -INFINITY) {
#pragma unroll
      for (int i = 0; i < PB; ++i) l += x[i].y;  // 0 or NaN
      continue;
    }
    const float w0 = ex2(m - top);
    m = top;
    l *= w0;
#pragma unroll
    for (int q = 0; q < COLS; ++q) {
      o[q].x *= w0;
      o[q].y *= w0;
      o[q].z *= w0;
      o[q].w *= w0;
    }
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const float w = ex2(x[i].x - top);
      l = fmaf(w, x[i].y, l);
#pragma unroll
      for (int q = 0; q < COLS; ++q) {
        o[q].x = fmaf(w, v[i][q].x, o[q].x);
        o[q].y = fmaf(w, v[i][q].y, o[q].y);
        o[q].z = fmaf(w, v[i][q].z, o[q].z);
        o[q].w = fmaf(w, v[i][q].w, o[q].w);
      }
    }
  }
}

template <int D, int RUNS, int SLOT>
__global__ void __launch_bounds__(256, 2) shared_join_kernel(const Params p) {
  constexpr int ROWS = SLOT < 32 ? SLOT : 32, HALVES = 32 / ROWS;
  using J = JoinShared<ROWS>;
  constexpr int COLS = J::COLS, GROUPS = J::GROUPS, CHUNKS = D / 4 / COLS, FEW = 8;
  __shared__ J sh;
  pdl_launch_dependents();  // the pass over the sequences' own keys, which waits where it joins
  pdl_wait();               // the parts and boundaries
  const int first_row = blockIdx.y * ROWS;
  const Boundary bd = p.bounds[blockIdx.x + 1];
  const int tiles = bd.ntok > p.tpt ? 2 : 1;
  if (!bd.cut || (SLOT > ROWS && first_row >= tiles * BM)) return;
  const int left = bd.ntok - first_row / BM * p.tpt;
  if (first_row % BM >= min(left, p.tpt) * p.G) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane / ROWS;
  const long long end = bd.u0 + p.overhead + (long long)bd.w * bd.nt;
  auto tile_of = [&](int k) { return tile_at(p, run_start<RUNS>(bd.total, k) - bd.u0, bd.w); };
  // the unit's first boundary, its first part being run c - 1's, and the end of its parts
  const int c = run_from<RUNS>(bd.total, bd.u0 + p.overhead + bd.w), last = run_from<RUNS>(bd.total, end);
  const int before = (int)blockIdx.x + 1 - c;
  if (before >= CHUNKS) return;
  const bool few = last - c + 1 <= FEW;
  if (few && before > 0) return;
  // a run shorter than a key tile may hold none of the unit, and then no part
  const bool tiny = bd.total < (long long)RUNS * (bd.w + 1);
  auto row_at = [&](int r, int &tok) {  // whether row r of the unit's tiles is a token's
    const int rt = r % BM / p.G;
    tok = r / BM * p.tpt + rt;
    return rt < p.tpt && tok < bd.ntok;
  };
  const int64_t pitch = (int64_t)p.total * p.G;
  auto put = [&](int r, int tok, int col, const float4 &v, float m, float l) {
    const int64_t at = ((int64_t)bd.tok0 + tok) * p.G + r % BM % p.G;
    reinterpret_cast<float4 *>(p.pre_o)[(bd.head * (D / 4) + col) * pitch + at] = v;
    if (col == 0) p.pre_ml[bd.head * pitch + at] = make_float2(m, l);
  };
  const int r = first_row + lane % ROWS;
  int tok;
  const bool valid = row_at(r, tok);
  auto has_part = [&](int k) {
    return valid && (!tiny || run_start<RUNS>(bd.total, k + 1) >= end || tile_of(k + 1) > tile_of(k));
  };
  float m, l;
  float4 o[COLS];
  if (few) {
    for (int col0 = (warp * HALVES + half) * COLS; col0 < D / 4; col0 += 8 * HALVES * COLS) {
      join_parts<D, SLOT, 2, COLS>(p, c, c - 1, 1, last, r, col0, has_part, m, l, o);
      if (!valid) continue;
#pragma unroll
      for (int q = 0; q < COLS; ++q) put(r, tok, col0 + q, o[q], m, l);
    }
    return;
  }
  const int group = warp * HALVES + half;
  for (int col0 = before * COLS; col0 < D / 4; col0 += (last - c) * COLS) {
    join_parts<D, SLOT, 4, COLS>(p, c, c - 1 + group, GROUPS, last, r, col0, has_part, m, l, o);
    sh.ml[group][lane % ROWS] = make_float2(m, l);
#pragma unroll
    for (int q = 0; q < COLS; ++q) sh.part[group][q][lane % ROWS] = o[q];
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * COLS; i += 256) {
      const int y = i % ROWS, q = i / ROWS;
      int ty;
      if (!row_at(first_row + y, ty)) continue;
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) top = fmaxf(top, sh.ml[g][y].x);
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const float2 x = sh.ml[g][y];
        const float w = x.x == -INFINITY ? 0.0f : ex2(x.x - top);
        const float4 v = sh.part[g][q][y];
        sum = fmaf(w, x.y, sum);
        s.x = fmaf(w, v.x, s.x);
        s.y = fmaf(w, v.y, s.y);
        s.z = fmaf(w, v.z, s.z);
        s.w = fmaf(w, v.w, s.w);
      }
      put(first_row + y, ty, col0 + q, s, top, sum);
    }
    __syncthreads();
  }
}

size_t part_bytes(int d) { return (size_t)CTAS * 2 * 2 * BM * d * sizeof(float); }
size_t ml_bytes() { return (size_t)CTAS * 2 * 2 * BM * sizeof(float2); }

// A launch; where `early`, one that may begin before the kernel before it has ended.
template <typename... Args>
cudaError_t launch_kernel(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, bool early, cudaStream_t st,
                          const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Behind the kernel that made the parts: a boundary is a block's, 32 rows of it at a time.
template <int D, int RUNS, int SLOT, int MODE>
cudaError_t launch_join(const PagedAttnArgs &a, const Params &p, cudaStream_t st) {
  // no sequence is longer than a key tile: no unit is cut
  if (((int64_t)a.seqs.max_pages << a.seqs.page_shift) <= BN) return cudaSuccess;
  const dim3 grid(RUNS - 1, SLOT < 32 ? 1 : SLOT / 32);
  if constexpr (MODE == SHARED)
    return launch_kernel(shared_join_kernel<D, RUNS, SLOT>, grid, 256, 0, true, st, p);
  else
    return launch_kernel(paged_combine_kernel<D, RUNS, SLOT, MODE>, grid, 256, 0, true, st, p);
}

template <int D, int WARPS, int MODE>
cudaError_t launch_tokens(const PagedAttnArgs &a, Params p, bool chunks, bool early, cudaStream_t st) {
  using L = TokenLayout<D, WARPS>;
  p.tpt = p.utok = TOK_ROWS / p.G;
  if (chunks) p.upto = 2 * p.utok;
  p.cost1 = p.cost2 = L::COST;
  p.overhead = L::OVERHEAD;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  constexpr size_t SLOTS = (size_t)L::RUNS * 2 * TOK_ROWS;
  static_assert(SLOTS * (D * 4 + 8) + L::RUNS * sizeof(Boundary) <= (size_t)CTAS * 4 * BM * D * 4, "workspace");
  p.part_o = reinterpret_cast<float *>(ws);
  p.part_ml = reinterpret_cast<float2 *>(ws + SLOTS * D * 4);
  p.bounds = reinterpret_cast<Boundary *>(ws + SLOTS * (D * 4 + 8));
  auto kernel = paged_token_kernel<D, WARPS, MODE>;
  static std::atomic<uint64_t> allowed{0};  // devices on which the kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  if (MODE == ALONE) timing_mark(st, 0);
  if ((e = launch_kernel(kernel, dim3(L::RUNS), 32 * WARPS, L::ALLOC, early, st, p)) != cudaSuccess) return e;
  if (MODE == ALONE) timing_mark(st, 1);
  return launch_join<D, L::RUNS, TOK_ROWS, MODE>(a, p, st);
}

template <int D>
Params params_of(const PagedAttnArgs &a, const WaitCfg &wc) {
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
  return p;
}

// One pass over the work that `p` describes, of `seqs` sequences: by tiles of 16 rows where `few`, by
// those of 128 where not, and for what is longer among the few where `chunks`.
template <int D, int MODE>
cudaError_t launch_pass(const PagedAttnArgs &a, Params p, int seqs, bool few, bool chunks, bool early, cudaStream_t st) {
  using L = Layout<D>;
  // Few units are spread over the warps of one block an SM, more over two blocks, whose starts and
  // ends overlap (1,000 keys a sequence, 8 K/V heads: 2 sequences 11.4 us, 13.3 with two blocks;
  // 4 sequences 11.8 and 12.3; 8 15.0 and 13.5; 16 19.7 and 17.6)
  cudaError_t e;
  int mark = 0;  // kernel boundaries so far
  if (few) {
    e = (int64_t)seqs * p.Hkv <= CTAS / 3 ? launch_tokens<D, 8, MODE>(a, p, chunks, early, st)
                                          : launch_tokens<D, 4, MODE>(a, p, chunks, early, st);
    if (e != cudaSuccess || !chunks) return e;
    p.above = 2 * (TOK_ROWS / p.G);
    mark = 1;
    early = false;  // the workspace is the kernels' before
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
  // nothing (single tokens of 64 sequences of 8,192 keys, 64 heads on 2: 75 us, 79 with 256, by tiles of 128 rows).  At
  // d = 128 the row is the 256 bytes.
  const CUtensorMapL2promotion promote =
      D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  if ((e = make_tmap(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.Q, dq, sq, bq)) != cudaSuccess ||
      (e = make_tmap(&mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.kc.ptr, dk, sk, bk, promote)) != cudaSuccess ||
      (e = make_tmap(&mv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.vc.ptr, dk, sv, bk, promote)) != cudaSuccess)
    return e;
  e = cudaFuncSetAttribute(paged_attn_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
  if (e != cudaSuccess) return e;
  if (MODE == ALONE && mark == 0) timing_mark(st, 0);
  if ((e = launch_kernel(paged_attn_kernel<D, MODE>, dim3(CTAS), THREADS, L::ALLOC, early, st, mq, mk, mv, p)) !=
      cudaSuccess)
    return e;
  if (MODE == ALONE) timing_mark(st, mark + 1);
  return launch_join<D, CTAS, 2 * BM, MODE>(a, p, st);
}

size_t pass_workspace(int d) { return part_bytes(d) + ml_bytes() + CTAS * sizeof(Boundary) + 256; }

}  // namespace
}  // namespace chain
