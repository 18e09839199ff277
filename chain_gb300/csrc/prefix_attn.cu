// prefix_attn.cu -- attention over a paged cache for a batch whose sequences share long prefixes.
//
// Softmax attention of a row over keys in two sets is the join of its sums over each: with m the
// largest score of a set, l = sum exp(s - m) and A = sum exp(s - m) v,
//   m = max(m1, m2),  O = (A1 e^(m1 - m) + A2 e^(m2 - m)) / (l1 e^(m1 - m) + l2 e^(m2 - m)).
// The first set is the group's prefix, whole key tiles of it.  It is the same for every row of the group, and
// the packed rows of a group's sequences lie together, so the group is one long sequence of new tokens without
// a mask over it: its keys are read once for 128 rows instead of once for each sequence, and
// multiplied in full tiles.  The second is what each sequence has behind, masked as ever.
//
// Two passes of the kernels of paged_attn.cuh, then: SHARED writes (m, l, A) in 32 bits, [head][column / 4][row][4],
// lanes side by side as in the parts of a cut unit; OWN joins them where it would have
// written O, in a unit's end or in the join of a cut one, so that O is rounded once.  Each pass deals its work as a
// call alone does.  OWN begins while SHARED ends, and waits for it only where it joins.
//
// Bounds, and what was measured (in a graph, again and again; by itself, second-level cache cold, in brackets):
//   64 tokens, 32 heads on 8, d = 128, behind 8,192 positions, up to 512 of their own: 60 us [SHARED 25, its join 10,
//   OWN 24, its join 6], of which 16 are its bytes.  SHARED is a start (8 us to the first S, 5 to the first softmax's
//   end, both instructions and tables from memory), three steps of 2 us and 128 KB of sums a block;
//   128 tokens behind 32,768, up to 1,024 of their own: 143 us [72, 14, 55, 7], bytes 60, operations 37: the
//   128-row tiles, whose tensor pipe is 66% busy, then memory;
//   6 tokens of 8 heads to a K/V head behind 131,072: 58 us [34, 8, 10, 7], bytes 20: the chain of copies
//   and products at one query tile, and three starts;
//   32 chunks of up to 64 tokens behind 16,384: 325 us [280, 14, 32, 3], operations 181 and, with P's low part, 271;
//   without a mask the same within 2%; at d = 64 274 to 283 us, operations 91 (136 with the low part).
// Measured for SHARED and dropped, each right: V turned into f16 in shared memory by warps of its own, so that P
// enters as one f16 (322 us -> 336 then: what passes between the warps counts; without P's low part at all the 32
// chunks would take 273 of 325 now); 32- and 64-row tiles in
// the kernel of few rows (one group of 32 rows 57 us -> 53, eight 61 -> 65, 48 rows 60 -> 72).
#include "paged_attn.cuh"

namespace chain {
namespace {

// Two passes and one, 32 heads on 8, d = 128, second-level cache cold: single tokens, 64 sequences of 512
// positions (128 MB in all) 44 us and 34, of 1,024 44 and 46, of 2,048 46 and 69; 16 of 2,048 35 and 31, of 4,096 37
// and 43.  32 sequences of 1,024 (128 MB), 16 new tokens each 66 and 50, 64 each 98 and 70.  Query tiles that are
// full: 4 sequences of 16,128 (252 MB), 128 new tokens each 177 and 151.  What a table can name stands for what the
// lengths are, which only the device knows: 5 tokens behind 600 positions take 20 us with a table of ten pages and 36 with one of 512.
constexpr int64_t ALONE_BYTES = int64_t(1) << 27;

size_t rows_bytes(int64_t rows, int d) { return (size_t)rows * d * sizeof(float); }

template <int D>
cudaError_t launch(const PrefixAttnArgs &x, const WaitCfg &wc, cudaStream_t st) {
  const PagedAttnArgs &a = x.a;
  Params own = params_of<D>(a, wc);
  own.group_cu = x.group_cu;
  own.group_lens = x.group_lens;
  own.groups = x.groups;
  // One pass where two would not pay: with few keys (the most that the table can name, since the lengths are on
  // the device), and with so many tokens a sequence that each fills its own query tiles: they are multiplied as
  // often, and read from the second-level cache.
  const int64_t keys = (int64_t)a.seqs.batch * a.seqs.max_pages << a.seqs.page_shift;
  if (keys * a.Hkv * D * 4 <= ALONE_BYTES || a.total >= 2 * (int64_t)own.utok * a.seqs.batch) {
    timing_mark(st, 0);
    const cudaError_t e = launch_pass<D, OWN>(a, own, a.seqs.batch, few_rows(a, own.G), may_have_chunks(a, own.G), false, st);
    timing_mark(st, 1);
    return e;
  }
  timing_mark(st, 0);
  const int64_t rows = (int64_t)a.total * a.H;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace) + 2 * pass_workspace(D);
  own.pre_o = reinterpret_cast<float *>(ws);
  own.pre_ml = reinterpret_cast<float2 *>(ws + rows_bytes(rows, D));
  Params shared = own;
  shared.causal = 0;
  PagedAttnArgs b = a;  // the passes' workspaces are apart: they overlap
  b.workspace = static_cast<uint8_t *>(a.workspace) + pass_workspace(D);
  shared.part_o = reinterpret_cast<float *>(b.workspace);
  shared.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(b.workspace) + part_bytes(D));
  shared.bounds = reinterpret_cast<Boundary *>(static_cast<uint8_t *>(b.workspace) + part_bytes(D) + ml_bytes());
  // Tiles of 16 rows where the groups' rows fit one on the average; what is longer than two of them then goes to a launch
  // of its own, as with single tokens.  (Two tiles to a group: 16 groups of 24 rows at d = 64 62 us, 59 with tiles of
  // 128; one of 32 behind 32,768 73 and 58.)
  const int64_t group_rows = (int64_t)a.total * own.G;
  const bool few = own.G <= TOK_ROWS && group_rows <= (int64_t)TOK_ROWS * x.groups;
  cudaError_t e = launch_pass<D, SHARED>(b, shared, x.groups, few, x.groups > 1 && group_rows > 2 * TOK_ROWS, false, st);
  if (e != cudaSuccess) return e;
  timing_mark(st, 1);
  e = launch_pass<D, OWN>(a, own, a.seqs.batch, few_rows(a, own.G), may_have_chunks(a, own.G), true, st);
  timing_mark(st, 2);
  return e;
}

}  // namespace

size_t prefix_attn_workspace(int d, int64_t total, int H) {
  return 2 * pass_workspace(d) + rows_bytes(total * H, d) + (size_t)total * H * sizeof(float2);
}

cudaError_t launch_prefix_attn(const PrefixAttnArgs &x, const WaitCfg &wc, cudaStream_t st) {
  return x.a.d == 128 ? launch<128>(x, wc, st) : launch<64>(x, wc, st);
}

}  // namespace chain
