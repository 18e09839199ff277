// qk_norm_rope.cu -- per-head RMS norm of queries and keys with the rotary
// position embedding in the same pass: forward, backward, and the form that
// writes new keys and values into a paged cache.
//
// One row is one head of one token, x in R^d at position p, with a weight g
// in R^d and frequencies w_i, i < rot/2:
//   forward   r = 1 / sqrt(mean(x^2) + eps),  u = x r g,  y = R(p) u,
//             R(p) rotating the pair (i, i + rot/2), or (2i, 2i + 1), by the
//             angle p w_i and leaving elements from rot on alone;
//   backward  a = R(p)^T dy,  dg = sum over rows of a x r,  h = a g,
//             dx = r (h - x r^2 mean(h x)).
// Everything between the load and the store is fp32; the one rounding to
// bf16 is the store's.  Both passes read each input once and write each
// output once, so memory bandwidth bounds them: 32 + 8 heads of d = 128, 32,768
// tokens, bf16: the forward 103 us (0.67 GB, 6.5 TB/s; a copy of the same bytes takes 100),
// the backward 157 us (1.01 GB, 6.4 TB/s), 16 prompts of 18,632 tokens in all into the
// cache 77 us (0.46 GB, 5.9 TB/s).  At d = 64 a token's angles are shared by half as many
// bytes and the arithmetic shows: backward 80 us of 0.46 GB.  A few tokens take what a
// launch takes: 3 to 4 us, two launches with the sums of a weight's gradient 6 to 8.  With few heads
// the angles bound it: 32,768 tokens of 3 + 1 heads of 128 26 us, where the bytes take 10.
//
// Angles.  p w_i mod 2 pi keeps no fp32 accuracy at far positions, and fp64
// is slow here, so angles are kept in turns as 64-bit fixed point: w_i / 2 pi
// is formed once per block as an integer U_i = w_i / (2 pi) 2^64 (mod 2^64,
// exact to one unit), and p U_i mod 2^64 is the angle of position p: exact
// modular arithmetic whose error is |p| 2^-64 turns.  Its low 32 bits are dropped (2^-32 turns); the
// rest, less its quarter turns, becomes an fp32 number of radians by one conversion (2^-28 turns) and
// one product (2^-27 with the constant's own rounding).
#include <algorithm>

#include "internal.h"

namespace chain {
namespace {

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_FREQ = 64;  // rot / 2 at d = 128
constexpr int SMS = 152;
using std::min;

// 1 / (2 pi) = 0.159154943... as a 128-bit binary fraction
constexpr unsigned long long INV_2PI_HI = 0x28be60db9391054aull;
constexpr unsigned long long INV_2PI_LO = 0x7f09d5f47d4d3770ull;

// w / (2 pi) in units of 2^-64 turns, mod 2^64.  w = m 2^e with an integer m
// of 24 bits; m times the 128-bit fraction, shifted by e.  (From w = 2^24 on,
// bits past the fraction's end would be needed: accuracy falls there.)
__device__ __forceinline__ unsigned long long turns_per_position(float w) {
  const uint32_t b = __float_as_uint(w);
  const int ex = (int)((b >> 23) & 0xff);
  if (ex == 255) return 0;  // infinite or NaN: see put_turns
  const unsigned long long m = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int sh = 150 - (ex ? ex : 1);  // -e
  const unsigned __int128 hi = (unsigned __int128)m * INV_2PI_HI;
  const unsigned __int128 lo = (unsigned __int128)m * INV_2PI_LO;
  const unsigned __int128 p = hi + (lo >> 64);
  unsigned long long u;
  if (sh >= 0)
    u = sh < 128 ? (unsigned long long)(p >> sh) : 0ull;
  else
    u = (unsigned long long)(p << -sh);
  return (b >> 31) ? 0ull - u : u;
}

// (cos, sin) of position p and frequency U.  The angle's nearest quarter turn
// comes off exactly, in integers; what is left, |x| <= pi/4, goes through the Taylor
// series (to x^9 and x^8: their next terms are below 2^-25).  CUDA's sincospif in
// their place made up a fifth of the forward's instructions.
__device__ __forceinline__ float2 angle(int p, unsigned long long u) {
  const unsigned long long a = u * (unsigned long long)(long long)p;
  const uint32_t t = (uint32_t)(a >> 32);         // turns in units of 2^-32
  const uint32_t q = (t + 0x20000000u) >> 30;     // quarter turns, mod 4
  const float x = (float)(int)(t - (q << 30)) * 1.46291807926715969e-9f;  // 2 pi 2^-32
  const float z = x * x;
  float s = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, -1/7!
  s = fmaf(z, s, 8.33333333e-3f);                      // 1/5!
  s = fmaf(z, s, -1.66666667e-1f);                     // -1/3!
  s = fmaf(x * z, s, x);
  float c = fmaf(z, 2.48015873e-5f, -1.38888889e-3f);  // 1/8!, -1/6!
  c = fmaf(z, c, 4.16666667e-2f);                      // 1/4!
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  if (q & 1) {
    const float w = s;
    s = c;
    c = -w;
  }
  return q & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// The block's frequencies as turns, and whether one of them is infinite or NaN.  That has to show in
// the result, so the weights of its pairs become NaN then: a test at the angles themselves cost
// the kernels of few heads 2 to 35% of their time.  Holds the block's barrier.
__device__ __forceinline__ bool put_turns(unsigned long long *turns, const float *inv_freq, int rot) {
  bool odd = false;
  for (int f = threadIdx.x; f < rot / 2; f += THREADS) {
    const float w = __ldg(inv_freq + f);
    turns[f] = turns_per_position(w);
    odd = odd || !isfinite(w);
  }
  return __syncthreads_or(odd);
}

// ------------------------------------------------------ sixteen elements a lane
// A lane holds sixteen elements of a row as eight pairs, in parts of 16 bytes (eight bf16,
// four f32), and the lanes' parts lie side by side: with n lanes, lane l's part j is the
// (j n + l)th, so that a warp's access covers whole sectors.  (Sixteen elements in a row a
// lane, forward of 40 heads of d = 128: pairs (2i, 2i + 1) of 32,768 tokens in bf16 150 us,
// 102 so; 16,384 tokens in f32 149 us, 108 so.  The f32 backward of as many takes 160.)  The lanes
// of the rotated elements and those of the others are dealt apart; pairs (i, i + rot/2)
// then lie in one lane, as pairs (2i, 2i + 1) do, and a rotation needs no other lane.  (With
// eight elements a lane, the reduction, the addressing and the loop cost twice as much for
// each element, and the instruction issue bounded the kernels.)
constexpr int EPL = 16;
template <typename T>
constexpr int part_of() { return 16 / (int)sizeof(T); }  // elements
struct Lane {
  int at, step;  // its first part, from one part to the next; its elements rotate if at < rot
};
template <typename T, int D>
__device__ __forceinline__ Lane lane_of(int lane, int rot) {
  constexpr int W = part_of<T>();
  const int l = lane % (D / EPL), n = rot / EPL;
  Lane r;
  r.at = l < n ? l * W : rot + (l - n) * W;
  r.step = (l < n ? n : D / EPL - n) * W;
  return r;
}
// Where a lane's element k lies in the row: k < 8 the firsts of the pairs, from 8 on their seconds
template <typename T, bool NEIGHBOUR>
__device__ __forceinline__ int element(const Lane &ln, int k) {
  constexpr int W = part_of<T>();
  const int i = NEIGHBOUR ? 2 * (k % 8) + k / 8 : k;
  return ln.at + i / W * ln.step + i % W;
}

// Asynchronous copy of 16 bytes into shared memory
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_async() {  // all but the newest N groups have arrived
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A lane's sixteen elements, as its parts lie in memory; get() gives the pairs' firsts in
// f[0..7] and their seconds in f[8..15].  In a ring slot each 16-byte part of a
// warp's lanes lies side by side, 512 bytes a part.
template <typename T>
struct Row;
template <>
struct Row<__nv_bfloat16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, int step) {
    a = *reinterpret_cast<const uint4 *>(p);
    b = *reinterpret_cast<const uint4 *>(p + step);
  }
  static __device__ __forceinline__ void fetch(uint32_t slot, const __nv_bfloat16 *p, int step) {
    copy_async(slot, p);
    copy_async(slot + 512, p + step);
  }
  __device__ __forceinline__ void take(const uint8_t *slot) {
    a = *reinterpret_cast<const uint4 *>(slot);
    b = *reinterpret_cast<const uint4 *>(slot + 512);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  template <bool NEIGHBOUR>
  __device__ __forceinline__ void get(float (&f)[16]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[NEIGHBOUR ? k : 2 * k] = lo(w[k]);
      f[NEIGHBOUR ? 8 + k : 2 * k + 1] = hi(w[k]);
    }
  }
  template <bool NEIGHBOUR>
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, int step, const float (&f)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      w[k] = NEIGHBOUR ? pack_bf16(f[k], f[8 + k]) : pack_bf16(f[2 * k], f[2 * k + 1]);
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(p + step) = make_uint4(w[4], w[5], w[6], w[7]);
  }
};
template <>
struct Row<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float *p, int step) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const float4 *>(p + k * step);
  }
  static __device__ __forceinline__ void fetch(uint32_t slot, const float *p, int step) {
#pragma unroll
    for (int k = 0; k < 4; ++k) copy_async(slot + 512 * k, p + k * step);
  }
  __device__ __forceinline__ void take(const uint8_t *slot) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const float4 *>(slot + 512 * k);
  }
  template <bool NEIGHBOUR>
  __device__ __forceinline__ void get(float (&f)[16]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float m[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) f[NEIGHBOUR ? 2 * k + e / 2 + 8 * (e & 1) : 4 * k + e] = m[e];
    }
  }
  template <bool NEIGHBOUR>
  static __device__ __forceinline__ void store(float *p, int step, const float (&f)[16]) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<float4 *>(p + k * step) =
          NEIGHBOUR ? make_float4(f[2 * k], f[8 + 2 * k], f[2 * k + 1], f[9 + 2 * k])
                    : make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
  }
};

template <typename T, bool NEIGHBOUR>
__device__ __forceinline__ void load_weight(const NormRopeWeight &g, const Lane &ln, float (&f)[16]) {
  if ((g.bf16 != 0) == (sizeof(T) == 2)) {  // of the heads' type: part by part
    Row<T> r;
    r.load(static_cast<const T *>(g.ptr) + ln.at, ln.step);
    r.template get<NEIGHBOUR>(f);
    return;
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int e = element<T, NEIGHBOUR>(ln, k);
    f[k] = g.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(g.ptr)[e]) : static_cast<const float *>(g.ptr)[e];
  }
}

// NaN in place of what belongs to a pair whose frequency is infinite or NaN
template <typename T, bool NEIGHBOUR>
__device__ __forceinline__ void spoil(const float *inv_freq, int rot, const Lane &ln, float (&f)[16]) {
  if (ln.at >= rot) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = element<T, NEIGHBOUR>(ln, k);
    if (!isfinite(__ldg(inv_freq + (NEIGHBOUR ? e / 2 : e)))) f[k] = f[8 + k] = __int_as_float(0x7fffffff);
  }
}

// Cosines and sines of a lane's eight pairs at one token
struct Angles {
  float c[8], s[8];
};

// Every frequency's (cos, sin) at position p into the warp's table, each
// computed once.
__device__ __forceinline__ void put_angles(int lane, int rot, int p, const unsigned long long *turns,
                                           float2 *table) {
  __syncwarp();  // the table's last readers are done
  for (int f = lane; f < rot / 2; f += 32) table[f] = angle(p, turns[f]);
  __syncwarp();
}
// The lane's own out of it; elements that do not rotate get (1, 0).
template <typename T, bool NEIGHBOUR>
__device__ __forceinline__ void take_angles(Angles &an, const Lane &ln, int rot, const float2 *table) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float4 cs = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
    const int e = element<T, NEIGHBOUR>(ln, 2 * k);  // pairs 2k and 2k + 1 have frequencies side by side
    if (ln.at < rot) cs = *reinterpret_cast<const float4 *>(table + (NEIGHBOUR ? e / 2 : e));
    an.c[2 * k] = cs.x;
    an.s[2 * k] = cs.y;
    an.c[2 * k + 1] = cs.z;
    an.s[2 * k + 1] = cs.w;
  }
}

// R^T u: u[0..7] the firsts, u[8..15] the seconds of the pairs
__device__ __forceinline__ void rotate_back(const Angles &an, float (&u)[16]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float x = u[k], y = u[8 + k];
    u[k] = fmaf(y, an.s[k], x * an.c[k]);
    u[8 + k] = fmaf(-x, an.s[k], y * an.c[k]);
  }
}

// Norm weight and rotation in one matrix for each pair: R(p) diag(g).  The row's
// 1 / rms, a scalar, is multiplied in afterwards.
struct Turn {
  float xx[8], xy[8], yx[8], yy[8];
};
__device__ __forceinline__ void turn_of(Turn &t, const Angles &an, const float (&g)[16]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    t.xx[k] = an.c[k] * g[k];
    t.xy[k] = -an.s[k] * g[8 + k];
    t.yx[k] = an.s[k] * g[k];
    t.yy[k] = an.c[k] * g[8 + k];
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Offset in elements of token t: t = b n + i of [B][n][H][d].
__device__ __forceinline__ int64_t token_off(const NormRopeSide &x, int t, int n) {
  if (x.s_batch == n * x.s_tok) return t * x.s_tok;
  const int b = t / n;
  return b * x.s_batch + (t - b * n) * x.s_tok;
}

template <int D>
__device__ __forceinline__ void fwd_row(float (&f)[16], float eps, const Turn &t) {
  float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 16; ++k) q[k & 3] = fmaf(f[k], f[k], q[k & 3]);
  const float r = rsqrtf(row_sum<D / EPL>((q[0] + q[1]) + (q[2] + q[3])) * (1.0f / D) + eps);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float x = f[k] * r, y = f[8 + k] * r;
    f[k] = fmaf(y, t.xy[k], x * t.xx[k]);
    f[8 + k] = fmaf(x, t.yx[k], y * t.yy[k]);
  }
}

// ------------------------------------------------------------ walk and ring
// A warp takes the rows of a token in batches of U passes (32 / (D / 16) heads a
// pass), queries' batches first, then keys', then (cache writes) values'; `run`
// batches in a row are one warp's, all of the token's where there are tokens
// enough.
//
// The rows of the next STAGES - 1 batches are on their way, by asynchronous
// copies into shared memory, while a batch is worked on.  Every lane copies
// the very bytes that it will read, so nothing but its own copies is waited for.
// No more bytes in flight than hide the latency: beyond that the memory serves them worse.
// At d = 128, bf16, a warp's one pass of 1 KB with five blocks an SM makes 20 KB an SM (40 heads
// x 32,768 tokens, forward: 105 us; four blocks 112, six 109; two passes or a third stage 120).
// At d = 64 a token's angles serve half as many bytes, and two passes hide that
// arithmetic better (60,011 tokens of 32 heads: 86 us, 92 with one).
constexpr int STAGES = 2;
constexpr int FWD_BLOCKS = 5, BWD_BLOCKS = kNormRopeBwdMaxGrid / SMS, ROW_BLOCKS = 5;  // an SM

template <typename T, int D>
constexpr int fwd_passes() { return sizeof(T) == 2 && D == 64 ? 2 : 1; }  // U
template <typename T>
constexpr int bwd_passes() { return 1; }  // of x and of dy
template <typename T>
constexpr int pass_bytes() { return 32 * EPL * (int)sizeof(T); }
template <int D>
constexpr int rows_per_pass() { return 32 / (D / EPL); }

struct Plan {
  int batches;      // of a token
  int run, chunks;  // batches a warp takes in a row; of a token, how many such runs
  int bq, bk;       // batches of queries, of keys
};

struct Walk {
  uint32_t c;    // run: tokens times runs of a token stay below 2^31
  int t, j, j1;  // token (-1: done), its batch, end of the run
};
__device__ __forceinline__ void walk_to(Walk &w, const Plan &pl, uint32_t tokens, uint32_t c) {
  w.c = c;
  w.t = -1;
  if (pl.chunks == 1) {
    if (c < tokens) w.t = (int)c;
    w.j = 0;
    w.j1 = pl.batches;
  } else if (c < tokens * pl.chunks) {
    w.t = (int)(c / (uint32_t)pl.chunks);
    w.j = (int)(c - (uint32_t)w.t * pl.chunks) * pl.run;
    w.j1 = min(w.j + pl.run, pl.batches);
  }
}
__device__ __forceinline__ void walk_on(Walk &w, const Plan &pl, uint32_t tokens) {
  if (++w.j == w.j1) walk_to(w, pl, tokens, w.c + gridDim.x * WARPS);
}

__device__ __forceinline__ int position(const NormRopeArgs &a, int t) {
  return a.positions ? __ldg(a.positions + t) : t % (int)a.n;
}
// The position of run c's token, looked up while the token before it is worked on
__device__ __forceinline__ void look_ahead(int &p, const NormRopeArgs &a, const Plan &pl, uint32_t c) {
  const uint32_t t = pl.chunks == 1 ? c : c / (uint32_t)pl.chunks;
  if (t < (uint32_t)a.tokens) p = position(a, (int)t);
}

__device__ __forceinline__ uint32_t walk_start() { return blockIdx.x * WARPS + (threadIdx.x >> 5); }

// A lane's place in the batches of one side at one token; set at a change of token
// or side, moved on from batch to batch in between (the 64-bit arithmetic of a
// place made up half of the instructions when every batch computed its own).
template <typename T>
struct Cursor {
  T *p;          // the lane's first part in its row of the next pass
  int64_t pass;  // elements to the next pass
  int left;      // rows below the side's last, from the lane's on
  int batches;   // of this side, from here to the end of the run
};
template <typename T, int D>
__device__ __forceinline__ void aim(Cursor<T> &c, const NormRopeSide &x, int64_t off, int heads, int j, int batches,
                                    int passes, const Lane &ln, int lane) {
  constexpr int RPW = rows_per_pass<D>();
  const int h = j * passes * RPW + lane / (D / EPL);
  c.p = static_cast<T *>(x.ptr) + off + h * x.s_head + ln.at;
  c.pass = RPW * x.s_head;
  c.left = heads - h;
  c.batches = batches;
}

// Starts the copies of the next batch into a ring slot.
template <typename T, int D, int U>
__device__ __forceinline__ void fetch_rows(uint32_t slot, Cursor<T> &c, const Lane &ln, int lane) {
  constexpr int RPW = rows_per_pass<D>();
#pragma unroll
  for (int u = 0; u < U; ++u, c.p += c.pass)
    if (c.left > u * RPW) Row<T>::fetch(slot + u * pass_bytes<T>() + lane * 16, c.p, ln.step);
  c.left -= U * RPW;
}

// The batch's rows: norm, rotation, store.
template <typename T, int D, bool NEIGHBOUR, int U>
__device__ __forceinline__ void fwd_batch(const uint8_t *slot, Cursor<T> &c, float eps, const Turn &turn,
                                          const Lane &ln, int lane) {
  constexpr int RPW = rows_per_pass<D>();
  const int first = c.left + lane / (D / EPL);  // of the warp's first row
#pragma unroll
  for (int u = 0; u < U; ++u, c.p += c.pass) {
    if (first <= u * RPW) break;  // warp-uniform: no row of this pass is there
    // a lane beyond the last head works on what its slot holds and stores nothing: sums stay within a row
    Row<T> x;
    x.take(slot + u * pass_bytes<T>() + lane * 16);
    float f[16];
    x.template get<NEIGHBOUR>(f);
    fwd_row<D>(f, eps, turn);
    if (c.left > u * RPW) Row<T>::template store<NEIGHBOUR>(c.p, ln.step, f);
  }
  c.left -= U * RPW;
}

// The queries' and the keys' weights as a lane's pairs; kept in shared memory, a
// lane's part of it read at each change of side.
struct Weights {
  float g[2][16][8];  // [side][k][lane of a row]
};
template <typename T, int D, bool NEIGHBOUR>
__device__ __forceinline__ void put_weights(Weights &w, const NormRopeWeight &gq, const NormRopeWeight &gk, int rot) {
  constexpr int LPR = D / EPL;
  if ((int)threadIdx.x < 2 * LPR) {
    const int side = threadIdx.x / LPR, l = threadIdx.x % LPR;
    float g[16];
    load_weight<T, NEIGHBOUR>(side ? gk : gq, lane_of<T, D>(l, rot), g);
#pragma unroll
    for (int k = 0; k < 16; ++k) w.g[side][k][l] = g[k];
  }
}
template <typename T, int D, bool NEIGHBOUR>
__device__ __forceinline__ void spoil_weights(Weights &w, const float *inv_freq, int rot) {
  constexpr int LPR = D / EPL;
  if ((int)threadIdx.x < 2 * LPR) {
    const int side = threadIdx.x / LPR, l = threadIdx.x % LPR;
    float g[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) g[k] = w.g[side][k][l];
    spoil<T, NEIGHBOUR>(inv_freq, rot, lane_of<T, D>(l, rot), g);
#pragma unroll
    for (int k = 0; k < 16; ++k) w.g[side][k][l] = g[k];
  }
  __syncthreads();
}
template <typename T, int D, bool NEIGHBOUR>
__device__ __forceinline__ void turn_for(Turn &t, const Weights &w, int side, const Lane &ln, int rot, const float2 *table,
                                         int lane) {
  Angles an;
  take_angles<T, NEIGHBOUR>(an, ln, rot, table);
  float g[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) g[k] = w.g[side][k][lane % (D / EPL)];
  turn_of(t, an, g);
}

template <typename T, int D, bool NEIGHBOUR>
__global__ void __launch_bounds__(THREADS, FWD_BLOCKS) norm_rope_kernel(const NormRopeArgs a, const Plan pl) {
  constexpr int U = fwd_passes<T, D>(), BYTES = U * pass_bytes<T>();
  __shared__ unsigned long long turns[MAX_FREQ];
  __shared__ __align__(16) float2 table[WARPS][MAX_FREQ];
  __shared__ Weights weights;
  __shared__ __align__(16) uint8_t ring[WARPS][STAGES][BYTES];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane ln = lane_of<T, D>(lane, a.rot);
  Walk ahead, now;
  walk_to(ahead, pl, (uint32_t)a.tokens, walk_start());
  now = ahead;
  int put = 0, got = 0;
  // a side's cursor at batch w.j of token w.t
  auto aim_at = [&](Cursor<T> &c, const Walk &w, const NormRopeSide &q, const NormRopeSide &k) {
    const bool key = w.j >= pl.bq;
    const NormRopeSide &x = key ? k : q;
    aim<T, D>(c, x, token_off(x, w.t, (int)a.n), key ? a.Hkv : a.H, key ? w.j - pl.bq : w.j,
              (key ? w.j1 : min(w.j1, pl.bq)) - w.j, U, ln, lane);
  };
  Cursor<T> in, out;
  in.batches = out.batches = 0;
  auto fetch = [&]() {
    if (ahead.t >= 0) {
      if (in.batches == 0) aim_at(in, ahead, a.q, a.k);
      --in.batches;
      fetch_rows<T, D, U>(smem_u32(ring[warp][put]), in, ln, lane);
      walk_on(ahead, pl, (uint32_t)a.tokens);
      put = put + 1 == STAGES ? 0 : put + 1;
    }
    commit_async();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch();
  put_weights<T, D, NEIGHBOUR>(weights, a.gq, a.gk, a.rot);
  const bool odd = put_turns(turns, a.inv_freq, a.rot);
  if (odd) spoil_weights<T, D, NEIGHBOUR>(weights, a.inv_freq, a.rot);
  Turn turn;
  int of = -1;  // the token of `table`
  int pos = 0;
  look_ahead(pos, a, pl, now.c);
  while (now.t >= 0) {
    fetch();
    if (out.batches == 0) {
      aim_at(out, now, a.qo, a.ko);
      if (now.t != of) {
        put_angles(lane, a.rot, pos, turns, table[warp]);
        of = now.t;
        look_ahead(pos, a, pl, now.c + gridDim.x * WARPS);
      }
      turn_for<T, D, NEIGHBOUR>(turn, weights, now.j >= pl.bq, ln, a.rot, table[warp], lane);
    }
    --out.batches;
    wait_async<STAGES - 1>();
    fwd_batch<T, D, NEIGHBOUR, U>(ring[warp][got], out, a.eps, turn, ln, lane);
    walk_on(now, pl, (uint32_t)a.tokens);
    got = got + 1 == STAGES ? 0 : got + 1;
  }
}

// ------------------------------------------------------------------- few heads
// With few heads a token's angles and addresses cost more than its rows.  There a pass
// takes its 32 / (D / 16) rows from the row of all tokens' heads, each lane works out the
// eight angles of its own row, and a warp takes passes of the queries first, then of the keys.
template <typename T, int D>
struct RowPass {
  int t, h;    // the lane's token and head
  bool there;
  __device__ __forceinline__ void at(uint32_t pass, uint32_t tokens, uint32_t heads, int lane) {
    const uint32_t row = pass * rows_per_pass<D>() + lane / (D / EPL), tok = row / heads;
    t = (int)tok;
    h = (int)(row - tok * heads);
    there = tok < tokens;
  }
  __device__ __forceinline__ T *in(const NormRopeSide &x, int n, const Lane &ln) const {
    return static_cast<T *>(x.ptr) + token_off(x, t, n) + h * x.s_head + ln.at;
  }
};
template <typename T, bool NEIGHBOUR>
__device__ __forceinline__ void own_angles(Angles &an, const Lane &ln, int rot, int p, const unsigned long long *turns) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = element<T, NEIGHBOUR>(ln, k);
    float2 cs = make_float2(1.0f, 0.0f);
    if (ln.at < rot) cs = angle(p, turns[NEIGHBOUR ? e / 2 : e]);
    an.c[k] = cs.x;
    an.s[k] = cs.y;
  }
}

template <typename T, int D, bool NEIGHBOUR>
__global__ void __launch_bounds__(THREADS, ROW_BLOCKS)
    norm_rows_kernel(const NormRopeArgs a, const uint32_t qpasses, const uint32_t passes) {
  __shared__ unsigned long long turns[MAX_FREQ];
  const int lane = threadIdx.x & 31;
  const Lane ln = lane_of<T, D>(lane, a.rot);
  const bool odd = put_turns(turns, a.inv_freq, a.rot);
  float g[16];
  int of = -1;  // the side of g
  for (uint32_t pass = walk_start(); pass < passes; pass += gridDim.x * WARPS) {
    const int side = pass >= qpasses;
    RowPass<T, D> r;
    r.at(side ? pass - qpasses : pass, (uint32_t)a.tokens, side ? a.Hkv : a.H, lane);
    Row<T> x = {};
    int p = 0;
    if (r.there) {
      x.load(r.in(side ? a.k : a.q, (int)a.n, ln), ln.step);
      p = position(a, r.t);
    }
    if (side != of) {
      load_weight<T, NEIGHBOUR>(side ? a.gk : a.gq, ln, g);
      if (odd) spoil<T, NEIGHBOUR>(a.inv_freq, a.rot, ln, g);
    }
    of = side;
    Angles an;
    own_angles<T, NEIGHBOUR>(an, ln, a.rot, p, turns);
    Turn turn;
    turn_of(turn, an, g);
    float f[16];
    x.template get<NEIGHBOUR>(f);
    fwd_row<D>(f, a.eps, turn);
    if (r.there) Row<T>::template store<NEIGHBOUR>(r.in(side ? a.ko : a.qo, (int)a.n, ln), ln.step, f);
  }
}

// ------------------------------------------------------------------ backward
// f = x in, dx out; v = dy
template <int D>
__device__ __forceinline__ void bwd_row(float (&f)[16], float (&v)[16], const float (&g)[16], float (&dg)[16],
                                        float eps, const Angles &an) {
  rotate_back(an, v);
  float q[2] = {0.0f, 0.0f}, w[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    q[k & 1] = fmaf(f[k], f[k], q[k & 1]);
    w[k & 1] = fmaf(v[k] * g[k], f[k], w[k & 1]);
  }
  const float sq = row_sum<D / EPL>(q[0] + q[1]), sw = row_sum<D / EPL>(w[0] + w[1]);
  const float r = rsqrtf(sq * (1.0f / D) + eps);
  const float c = -(sw * (1.0f / D)) * r * r * r;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float a = v[k] * r;
    dg[k] = fmaf(a, f[k], dg[k]);
    f[k] = fmaf(a, g[k], f[k] * c);
  }
}

// The lanes' sums to the block's, in one order: rows of a warp, then warps of the block.
template <typename T, int D, bool NEIGHBOUR>
__device__ __forceinline__ void sum_block(const float (&dg)[16], const Lane &ln, float (*sums)[D], float *part) {
  constexpr int LPR = D / EPL;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 16; ++k) {  // firsts, then seconds
    float v = dg[k];
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane < LPR) sums[warp][element<T, NEIGHBOUR>(ln, k)] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += THREADS) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) s += sums[w][i];
    part[i] = s;
  }
  __syncthreads();
}

// One side (queries or keys) of the backward: `heads` heads of every token;
// the block's sum of a x r into part[D].
template <typename T, int D, bool NEIGHBOUR>
__device__ __forceinline__ void bwd_side(const NormRopeArgs &a, const NormRopeSide &x, const NormRopeSide &dy,
                                         const NormRopeSide &dx, const NormRopeWeight &weight, int heads,
                                         const Plan &pl, const unsigned long long *turns, bool odd, float2 *table,
                                         uint8_t *ring, float (*sums)[D], float *part) {
  constexpr int LPR = D / EPL, RPW = rows_per_pass<D>();
  constexpr int U = bwd_passes<T>(), BYTES = U * pass_bytes<T>();  // of x, and of dy
  const int lane = threadIdx.x & 31, sub = lane / LPR;
  const Lane ln = lane_of<T, D>(lane, a.rot);
  Walk ahead, now;
  walk_to(ahead, pl, (uint32_t)a.tokens, walk_start());
  now = ahead;
  int put = 0, got = 0;
  Cursor<T> in_x, in_dy, out;
  in_x.batches = in_dy.batches = out.batches = 0;
  auto aim_at = [&](Cursor<T> &c, const Walk &w, const NormRopeSide &s) {
    aim<T, D>(c, s, token_off(s, w.t, (int)a.n), heads, w.j, w.j1 - w.j, U, ln, lane);
  };
  auto fetch = [&]() {
    if (ahead.t >= 0) {
      if (in_x.batches == 0) {
        aim_at(in_x, ahead, x);
        aim_at(in_dy, ahead, dy);
      }
      --in_x.batches;
      const uint32_t slot = smem_u32(ring) + put * 2 * BYTES;
      in_dy.left = in_x.left;  // one register for both
      fetch_rows<T, D, U>(slot, in_x, ln, lane);
      fetch_rows<T, D, U>(slot + BYTES, in_dy, ln, lane);
      walk_on(ahead, pl, (uint32_t)a.tokens);
      put = put + 1 == STAGES ? 0 : put + 1;
    }
    commit_async();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch();
  float g[16], dg[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) dg[k] = 0.0f;
  load_weight<T, NEIGHBOUR>(weight, ln, g);
  if (odd) {
    spoil<T, NEIGHBOUR>(a.inv_freq, a.rot, ln, g);
    spoil<T, NEIGHBOUR>(a.inv_freq, a.rot, ln, dg);
  }
  Angles an;
  int of = -1;  // the token of `an`
  int pos = 0;
  look_ahead(pos, a, pl, now.c);
  while (now.t >= 0) {
    fetch();
    if (out.batches == 0) {
      aim_at(out, now, dx);
      if (now.t != of) {
        put_angles(lane, a.rot, pos, turns, table);
        look_ahead(pos, a, pl, now.c + gridDim.x * WARPS);
        take_angles<T, NEIGHBOUR>(an, ln, a.rot, table);
        of = now.t;
      }
    }
    --out.batches;
    wait_async<STAGES - 1>();
    const uint8_t *slot = ring + got * 2 * BYTES + lane * 16;
    const int first = out.left + sub;  // of the warp's first row
#pragma unroll
    for (int u = 0; u < U; ++u, out.p += out.pass) {
      if (first <= u * RPW) break;  // warp-uniform
      float f[16], v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) f[k] = v[k] = 0.0f;
      if (out.left > u * RPW) {  // a row that is not there adds nothing to dg
        Row<T> r;
        r.take(slot + u * pass_bytes<T>());
        r.template get<NEIGHBOUR>(f);
        r.take(slot + BYTES + u * pass_bytes<T>());
        r.template get<NEIGHBOUR>(v);
      }
      bwd_row<D>(f, v, g, dg, a.eps, an);
      if (out.left > u * RPW) Row<T>::template store<NEIGHBOUR>(out.p, ln.step, f);
    }
    out.left -= U * RPW;
    walk_on(now, pl, (uint32_t)a.tokens);
    got = got + 1 == STAGES ? 0 : got + 1;
  }
  wait_async<0>();
  sum_block<T, D, NEIGHBOUR>(dg, ln, sums, part);
}

// The same with few heads: passes over the rows of all tokens
template <typename T, int D, bool NEIGHBOUR>
__device__ __forceinline__ void bwd_rows(const NormRopeArgs &a, const NormRopeSide &x, const NormRopeSide &dy,
                                         const NormRopeSide &dx, const NormRopeWeight &weight, int heads,
                                         const unsigned long long *turns, bool odd, float (*sums)[D], float *part) {
  const int lane = threadIdx.x & 31;
  const Lane ln = lane_of<T, D>(lane, a.rot);
  float g[16], dg[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) dg[k] = 0.0f;
  load_weight<T, NEIGHBOUR>(weight, ln, g);
  if (odd) {
    spoil<T, NEIGHBOUR>(a.inv_freq, a.rot, ln, g);
    spoil<T, NEIGHBOUR>(a.inv_freq, a.rot, ln, dg);
  }
  const uint32_t passes = ((uint32_t)a.tokens * heads + rows_per_pass<D>() - 1) / rows_per_pass<D>();
  for (uint32_t pass = walk_start(); pass < passes; pass += gridDim.x * WARPS) {
    RowPass<T, D> r;
    r.at(pass, (uint32_t)a.tokens, heads, lane);
    Row<T> xr = {}, dr = {};  // a row that is not there adds nothing to dg
    int p = 0;
    if (r.there) {
      xr.load(r.in(x, (int)a.n, ln), ln.step);
      dr.load(r.in(dy, (int)a.n, ln), ln.step);
      p = position(a, r.t);
    }
    Angles an;
    own_angles<T, NEIGHBOUR>(an, ln, a.rot, p, turns);
    float f[16], v[16];
    xr.template get<NEIGHBOUR>(f);
    dr.template get<NEIGHBOUR>(v);
    bwd_row<D>(f, v, g, dg, a.eps, an);
    if (r.there) Row<T>::template store<NEIGHBOUR>(r.in(dx, (int)a.n, ln), ln.step, f);
  }
  sum_block<T, D, NEIGHBOUR>(dg, ln, sums, part);
}

// part[block][2][D]: the block's sums of a x r over its query rows and its
// key rows.  No atomics: rows are dealt to warps by their number and every
// sum has one order.  Queries first, then keys: a weight and its sums take 16
// registers, and holding both sides' at once would cost a third of the warps.
template <typename T, int D, bool NEIGHBOUR>
__global__ void __launch_bounds__(THREADS, BWD_BLOCKS) norm_rows_bwd_kernel(const NormRopeBwdArgs b,
                                                                            float *__restrict__ part) {
  __shared__ unsigned long long turns[MAX_FREQ];
  __shared__ float sums[WARPS][D];
  const NormRopeArgs &a = b.fwd;
  pdl_launch_dependents();
  const bool odd = put_turns(turns, a.inv_freq, a.rot);
  part += (int64_t)blockIdx.x * 2 * D;
  bwd_rows<T, D, NEIGHBOUR>(a, a.q, b.dqo, a.qo, a.gq, a.H, turns, odd, sums, part);
  bwd_rows<T, D, NEIGHBOUR>(a, a.k, b.dko, a.ko, a.gk, a.Hkv, turns, odd, sums, part + D);
}

template <typename T, int D, bool NEIGHBOUR>
__global__ void __launch_bounds__(THREADS, BWD_BLOCKS) norm_rope_bwd_kernel(const NormRopeBwdArgs b, const Plan plq,
                                                                   const Plan plk, float *__restrict__ part) {
  constexpr int BYTES = bwd_passes<T>() * pass_bytes<T>();
  __shared__ unsigned long long turns[MAX_FREQ];
  __shared__ __align__(16) float2 table[WARPS][MAX_FREQ];
  __shared__ float sums[WARPS][D];
  __shared__ __align__(16) uint8_t ring[WARPS][STAGES * 2 * BYTES];
  const NormRopeArgs &a = b.fwd;
  const int warp = threadIdx.x >> 5;
  pdl_launch_dependents();  // the sums over blocks may be launched; they wait for this grid
  const bool odd = put_turns(turns, a.inv_freq, a.rot);
  part += (int64_t)blockIdx.x * 2 * D;
  bwd_side<T, D, NEIGHBOUR>(a, a.q, b.dqo, a.qo, a.gq, a.H, plq, turns, odd, table[warp], ring[warp], sums, part);
  bwd_side<T, D, NEIGHBOUR>(a, a.k, b.dko, a.ko, a.gk, a.Hkv, plk, turns, odd, table[warp], ring[warp], sums, part + D);
}

// dgq, dgk [D] from the blocks' sums: a block for 8 of the 2 D columns, its warps
// four blocks' sums each at a time, all loaded at once.  (A block for 32 columns, a warp a
// row, read them in rounds of dependent loads.)
constexpr int DG_WARPS = 32, DG_COLS = 8, DG_ROWS = 32 / DG_COLS * DG_WARPS;
__global__ void __launch_bounds__(32 * DG_WARPS) norm_rope_dg_kernel(const float *__restrict__ part, int blocks,
                                                                     int d, float *__restrict__ dgq,
                                                                     float *__restrict__ dgk) {
  constexpr int LOADS = (kNormRopeBwdMaxGrid + DG_ROWS - 1) / DG_ROWS;
  __shared__ float sums[DG_WARPS][DG_COLS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = warp * (32 / DG_COLS) + lane / DG_COLS, col = blockIdx.x * DG_COLS + lane % DG_COLS;
  pdl_wait();
  float v[LOADS], s = 0.0f;
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int r = row + i * DG_ROWS;
    v[i] = r < blocks ? part[(int64_t)r * 2 * d + col] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < LOADS; ++i) s += v[i];
#pragma unroll
  for (int o = DG_COLS; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane < DG_COLS) sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < DG_WARPS; w += 32 / DG_COLS) s += sums[w + lane / DG_COLS][lane % DG_COLS];
#pragma unroll
    for (int o = DG_COLS; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane < DG_COLS) (col < d ? dgq : dgk - d)[col] = s;
  }
}

// -------------------------------------------------------------- cache writes
template <int D>
__device__ __forceinline__ void copy_rows(const __nv_bfloat16 *src, int64_t s_head, __nv_bfloat16 *dst,
                                          int64_t d_head, int h0, int h1, int lane) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
  const int e0 = (lane % LPR) * 8;
  for (int h = h0 + lane / LPR; h < h1; h += RPW * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * RPW < h1) v[u] = *reinterpret_cast<const uint4 *>(src + (h + u * RPW) * s_head + e0);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * RPW < h1) *reinterpret_cast<uint4 *>(dst + (h + u * RPW) * d_head + e0) = v[u];
  }
}

// The sequence of token t, the last b with cu[b] <= t: 32 places at a time.
__device__ __forceinline__ int sequence_of(const int *cu, int batch, int t, int lane) {
  int b = 0, n = batch;  // it lies in [b, b + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const uint32_t below = __ballot_sync(0xffffffffu, at < n && __ldg(cu + b + at) <= t);
    // cu is nondecreasing: the lanes below form a run from 0 (none: t lies before the first)
    const int k = below ? 31 - __clz(below) : 0;
    b += k * step;
    n = min(step, n - k * step);
  }
  return b;
}

// Where token t goes: its position, and the element offsets of its row in the
// pools' first head, or ok = 0 with what is out of range reported.
struct Spot {
  int64_t pos, k, v;
  int in, ok;  // in: it belongs to a sequence
};
__device__ __forceinline__ Spot spot_in(const AppendArgs &a, int t, int b, bool report) {
  const PagedSeqs &s = a.seqs;
  Spot sp = {0, 0, 0, 0, 0};
  const int first = __ldg(s.cu + b), len = __ldg(s.lens + b);
  const int end = min(__ldg(s.cu + b + 1), (int)a.tokens);
  if (t < first || t >= end) return sp;  // a row behind the last sequence
  sp.in = 1;
  sp.pos = (int64_t)len - end + t;
  int page = -1;
  if (sp.pos >= 0 && sp.pos < ((int64_t)s.max_pages << s.page_shift))
    page = __ldg(s.table + b * s.table_stride + (sp.pos >> s.page_shift));
  if (page < 0 || page >= s.num_pages) {
    if (report) atomicExch(&a.status->reserved[0], 1);
    return sp;
  }
  const int64_t slot = sp.pos & ((1 << s.page_shift) - 1);
  sp.k = page * a.kc.s_page + slot * a.kc.s_slot;
  sp.v = page * a.vc.s_page + slot * a.vc.s_slot;
  sp.ok = 1;
  return sp;
}

__device__ __forceinline__ Spot spot_of(const AppendArgs &a, int t, int lane) {
  return spot_in(a, t, sequence_of(a.seqs.cu, a.seqs.batch, t, lane), lane == 0);
}
// The same for a lane's own token
__device__ __forceinline__ Spot spot_of(const AppendArgs &a, int t) {
  int b = 0;
  for (int n = a.seqs.batch; n > 1;) {
    const int half = n / 2;
    const bool up = __ldg(a.seqs.cu + b + half) <= t;
    b += up ? half : 0;
    n = up ? n - half : half;
  }
  return spot_in(a, t, b, true);
}

// Q normed, rotated and written to qo, K normed, rotated and written into its
// page, V copied into its page.
template <int D, bool NEIGHBOUR>
__global__ void __launch_bounds__(THREADS, FWD_BLOCKS) norm_append_kernel(const AppendArgs a, const Plan pl) {
  using T = __nv_bfloat16;
  constexpr int RPW = rows_per_pass<D>(), U = fwd_passes<T, D>(), BYTES = U * pass_bytes<T>();
  __shared__ unsigned long long turns[MAX_FREQ];
  __shared__ __align__(16) float2 table[WARPS][MAX_FREQ];
  __shared__ Weights weights;
  __shared__ __align__(16) uint8_t ring[WARPS][STAGES][BYTES];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane ln = lane_of<T, D>(lane, a.rot);
  Walk ahead, now;
  walk_to(ahead, pl, (uint32_t)a.tokens, walk_start());
  now = ahead;
  int put = 0, got = 0;
  // of batch w.j: its side (queries, keys, values), and the batches of the side before and up to it
  auto side_of = [&](const Walk &w, int &from, int &to) {
    const int side = w.j < pl.bq ? 0 : (w.j < pl.bq + pl.bk ? 1 : 2);
    from = side == 0 ? 0 : (side == 1 ? pl.bq : pl.bq + pl.bk);
    to = min(w.j1, side == 0 ? pl.bq : (side == 1 ? pl.bq + pl.bk : pl.batches));
    return side;
  };
  Cursor<T> in, out;
  in.batches = out.batches = 0;
  auto fetch = [&]() {
    if (ahead.t >= 0) {
      if (in.batches == 0) {
        int from, to;
        const int side = side_of(ahead, from, to);
        const NormRopeSide &x = side == 0 ? a.q : (side == 1 ? a.k : a.v);
        aim<T, D>(in, x, ahead.t * x.s_tok, side ? a.Hkv : a.H, ahead.j - from, to - ahead.j, U, ln, lane);
      }
      --in.batches;
      fetch_rows<T, D, U>(smem_u32(ring[warp][put]), in, ln, lane);
      walk_on(ahead, pl, (uint32_t)a.tokens);
      put = put + 1 == STAGES ? 0 : put + 1;
    }
    commit_async();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch();
  put_weights<T, D, NEIGHBOUR>(weights, a.gq, a.gk, a.rot);
  const bool odd = put_turns(turns, a.inv_freq, a.rot);
  if (odd) spoil_weights<T, D, NEIGHBOUR>(weights, a.inv_freq, a.rot);
  Turn turn;
  Spot sp = {0, 0, 0, 0, 0};
  int of = -1, side = 0;  // the token of `table` and `sp`, the side of `out` and `turn`
  while (now.t >= 0) {
    fetch();
    if (out.batches == 0) {
      if (now.t != of) {
        sp = spot_of(a, now.t, lane);
        put_angles(lane, a.rot, (int)sp.pos, turns, table[warp]);
        of = now.t;
      }
      int from, to;
      side = side_of(now, from, to);
      NormRopeSide y = a.qo;
      int64_t off = now.t * y.s_tok;
      if (side) {
        y.ptr = side == 1 ? a.kc.ptr : a.vc.ptr;
        y.s_head = side == 1 ? a.kc.s_head : a.vc.s_head;
        off = side == 1 ? sp.k : sp.v;
      }
      aim<T, D>(out, y, off, (side ? sp.ok : sp.in) ? (side ? a.Hkv : a.H) : 0, now.j - from, to - now.j, U, ln, lane);
      if (side < 2) turn_for<T, D, NEIGHBOUR>(turn, weights, side, ln, a.rot, table[warp], lane);
    }
    --out.batches;
    wait_async<STAGES - 1>();
    const uint8_t *slot = ring[warp][got];
    if (side < 2) {
      fwd_batch<T, D, NEIGHBOUR, U>(slot, out, a.eps, turn, ln, lane);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u, out.p += out.pass)
        if (out.left > u * RPW) {
          Row<T> r;
          r.take(slot + u * pass_bytes<T>() + lane * 16);
          *reinterpret_cast<uint4 *>(out.p) = r.a;
          *reinterpret_cast<uint4 *>(out.p + ln.step) = r.b;
        }
      out.left -= U * RPW;
    }
    walk_on(now, pl, (uint32_t)a.tokens);
    got = got + 1 == STAGES ? 0 : got + 1;
  }
}

// The same with few heads: passes over the rows of all tokens, queries, keys, then values.
template <int D, bool NEIGHBOUR>
__global__ void __launch_bounds__(THREADS, ROW_BLOCKS)
    norm_append_rows_kernel(const AppendArgs a, const uint32_t qpasses, const uint32_t kpasses) {
  using T = __nv_bfloat16;
  __shared__ unsigned long long turns[MAX_FREQ];
  const int lane = threadIdx.x & 31;
  const Lane ln = lane_of<T, D>(lane, a.rot);
  const bool odd = put_turns(turns, a.inv_freq, a.rot);
  float g[16];
  int of = -1;  // the side of g
  for (uint32_t pass = walk_start(); pass < qpasses + 2 * kpasses; pass += gridDim.x * WARPS) {
    const int side = pass < qpasses ? 0 : (pass < qpasses + kpasses ? 1 : 2);
    RowPass<T, D> r;
    r.at(side == 0 ? pass : pass - qpasses - (side - 1) * kpasses, (uint32_t)a.tokens, side ? a.Hkv : a.H, lane);
    Row<T> x = {};
    Spot sp = {0, 0, 0, 0, 0};
    if (r.there) {
      const NormRopeSide &y = side == 0 ? a.q : (side == 1 ? a.k : a.v);
      x.load(r.in(y, (int)a.tokens, ln), ln.step);
      sp = spot_of(a, r.t);
    }
    T *out = r.in(a.qo, (int)a.tokens, ln);
    if (side == 1) out = static_cast<T *>(a.kc.ptr) + sp.k + r.h * a.kc.s_head + ln.at;
    if (side == 2) out = static_cast<T *>(a.vc.ptr) + sp.v + r.h * a.vc.s_head + ln.at;
    const bool write = side == 0 ? sp.in : sp.ok;
    if (side == 2) {
      if (write) {
        *reinterpret_cast<uint4 *>(out) = x.a;
        *reinterpret_cast<uint4 *>(out + ln.step) = x.b;
      }
      continue;
    }
    if (side != of) {
      load_weight<T, NEIGHBOUR>(side ? a.gk : a.gq, ln, g);
      if (odd) spoil<T, NEIGHBOUR>(a.inv_freq, a.rot, ln, g);
    }
    of = side;
    Angles an;
    own_angles<T, NEIGHBOUR>(an, ln, a.rot, (int)sp.pos, turns);
    Turn turn;
    turn_of(turn, an, g);
    float f[16];
    x.template get<NEIGHBOUR>(f);
    fwd_row<D>(f, a.eps, turn);
    if (write) Row<T>::template store<NEIGHBOUR>(out, ln.step, f);
  }
}

// K and V copied into their pages, a token to a warp.
template <int D>
__global__ void __launch_bounds__(THREADS) append_kernel(const AppendArgs a) {
  using T = __nv_bfloat16;
  const int lane = threadIdx.x & 31;
  for (int64_t t = walk_start(); t < a.tokens; t += gridDim.x * WARPS) {
    const Spot sp = spot_of(a, (int)t, lane);
    if (!sp.ok) continue;
    copy_rows<D>(static_cast<const T *>(a.k.ptr) + t * a.k.s_tok, a.k.s_head, static_cast<T *>(a.kc.ptr) + sp.k,
                 a.kc.s_head, 0, a.Hkv, lane);
    copy_rows<D>(static_cast<const T *>(a.v.ptr) + t * a.v.s_tok, a.v.s_head, static_cast<T *>(a.vc.ptr) + sp.v,
                 a.vc.s_head, 0, a.Hkv, lane);
  }
}

// Batches a warp takes in a row: all of a token's once the tokens give every
// SM its warps, fewer below that.
Plan plan(int64_t tokens, int bq, int bk, int bv) {
  Plan pl;
  pl.bq = bq;
  pl.bk = bk;
  pl.batches = bq + bk + bv;
  const int64_t want = (int64_t)SMS * 24;
  const int64_t runs = tokens >= want ? 1 : min((want + tokens - 1) / tokens, (int64_t)pl.batches);
  pl.run = (int)((pl.batches + runs - 1) / runs);
  pl.chunks = (pl.batches + pl.run - 1) / pl.run;
  return pl;
}
unsigned blocks_for(int64_t tokens, const Plan &pl, int per_sm) {
  return (unsigned)min((tokens * pl.chunks + WARPS - 1) / WARPS, (int64_t)SMS * per_sm);
}
int batches_of(int heads, int b) { return (heads + b - 1) / b; }

// Few heads: a token's rows take no more bytes than this.  32,768 tokens, by tokens and by rows, in us.
// Forward, bf16: 30.2 and 8.6 (1 + 1 heads of 64), 30.8 and 30.3 (5 + 5: 1,280 bytes), 31.5 and 34.2
// (7 + 4), 35.4 and 25.8 (3 + 1 of 128), 35.6 and 31.7 (4 + 1: 1,280), 35.7 and 36.8 (4 + 2).  f32, whose
// rows hold half the angles a byte: 30.6 and 23.4 (4 + 2 of 64), 31.1 and 29.5 (5 + 3: 2,048), 31.1 and 32.1
// (6 + 3), 33.1 and 29.2 (3 + 1 of 128: 2,048), 33.7 and 35.6 (4 + 1).  Backward, bf16: 46.4 and 37.1 (8 + 1 of
// 64), 59.4 and 63.7 (16 + 1), 63.6 and 60.8 (6 + 2 of 128: 2,048), 63.8 and 67.9 (8 + 1).  f32: 45.8 and 23.0
// (3 + 1 of 64), 67.1 and 63.1 (10 + 4: 3,584), 70.6 and 70.9 (12 + 4), 68.1 and 63.4 (5 + 2 of 128: 3,584), 70.2 and
// 71.2 (6 + 2).  Into the cache, bf16 with the values: 16 prompts of 18,600 tokens in all, 28.8 and 24.7
// (8 + 2 of 64), 32.5 and 24.7 (4 + 1 of 128), 37 and 41 (8 + 1).
constexpr int FEW_FWD[2] = {1280, 2048}, FEW_BWD[2] = {2048, 3584}, FEW_APPEND = 2048;  // bf16, f32
bool few_heads(int64_t tokens, int heads, int head_bytes, int most) {
  return (int64_t)heads * head_bytes <= most && tokens * heads < (int64_t(1) << 31);
}
bool few_heads(const NormRopeArgs &a, const int (&most)[2]) {
  return few_heads(a.tokens, a.H + a.Hkv, a.d * (a.f32 ? 4 : 2), most[a.f32 ? 1 : 0]);
}
template <int D>
uint32_t row_passes(int64_t tokens, int heads) {
  return (uint32_t)((tokens * heads + rows_per_pass<D>() - 1) / rows_per_pass<D>());
}

template <typename T, int D, bool NEIGHBOUR>
cudaError_t launch_fwd(const NormRopeArgs &a, cudaStream_t st) {
  if (few_heads(a, FEW_FWD)) {
    const uint32_t q = row_passes<D>(a.tokens, a.H), all = q + row_passes<D>(a.tokens, a.Hkv);
    const unsigned blocks = min((all + WARPS - 1) / WARPS, (uint32_t)SMS * ROW_BLOCKS);
    norm_rows_kernel<T, D, NEIGHBOUR><<<blocks, THREADS, 0, st>>>(a, q, all);
    return cudaGetLastError();
  }
  constexpr int B = fwd_passes<T, D>() * rows_per_pass<D>();
  const Plan pl = plan(a.tokens, batches_of(a.H, B), batches_of(a.Hkv, B), 0);
  norm_rope_kernel<T, D, NEIGHBOUR><<<blocks_for(a.tokens, pl, FWD_BLOCKS), THREADS, 0, st>>>(a, pl);
  return cudaGetLastError();
}

template <typename T, int D, bool NEIGHBOUR>
cudaError_t launch_bwd(const NormRopeBwdArgs &b, cudaStream_t st) {
  constexpr int B = bwd_passes<T>() * rows_per_pass<D>();
  float *part = static_cast<float *>(b.workspace);
  unsigned blocks = 0;  // no tokens: no sums, dg = 0
  if (b.fwd.tokens > 0 && few_heads(b.fwd, FEW_BWD)) {
    const uint32_t most = row_passes<D>(b.fwd.tokens, b.fwd.H > b.fwd.Hkv ? b.fwd.H : b.fwd.Hkv);
    blocks = min((most + WARPS - 1) / WARPS, (uint32_t)kNormRopeBwdMaxGrid);
    norm_rows_bwd_kernel<T, D, NEIGHBOUR><<<blocks, THREADS, 0, st>>>(b, part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  } else if (b.fwd.tokens > 0) {
    const Plan plq = plan(b.fwd.tokens, batches_of(b.fwd.H, B), 0, 0);
    const Plan plk = plan(b.fwd.tokens, batches_of(b.fwd.Hkv, B), 0, 0);
    blocks = blocks_for(b.fwd.tokens, plq, BWD_BLOCKS);
    norm_rope_bwd_kernel<T, D, NEIGHBOUR><<<blocks, THREADS, 0, st>>>(b, plq, plk, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * D / DG_COLS);
  cfg.blockDim = dim3(32 * DG_WARPS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = blocks > 0;  // behind this call's own kernel only
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_dg_kernel, (const float *)part, (int)blocks, D, b.dgq, b.dgk);
}

template <int D>
cudaError_t launch_app(const AppendArgs &a, cudaStream_t st) {
  constexpr int B = fwd_passes<__nv_bfloat16, D>() * rows_per_pass<D>();
  if (a.norm && few_heads(a.tokens, a.H + 2 * a.Hkv, D * 2, FEW_APPEND)) {
    const uint32_t q = row_passes<D>(a.tokens, a.H), k = row_passes<D>(a.tokens, a.Hkv);
    const unsigned n = min((q + 2 * k + WARPS - 1) / WARPS, (uint32_t)SMS * ROW_BLOCKS);
    if (a.neighbour)
      norm_append_rows_kernel<D, true><<<n, THREADS, 0, st>>>(a, q, k);
    else
      norm_append_rows_kernel<D, false><<<n, THREADS, 0, st>>>(a, q, k);
    return cudaGetLastError();
  }
  const int kv = batches_of(a.Hkv, B);
  const Plan pl = a.norm ? plan(a.tokens, batches_of(a.H, B), kv, kv) : plan(a.tokens, 1, 0, 0);
  const unsigned blocks = blocks_for(a.tokens, pl, a.norm ? FWD_BLOCKS : 16);
  if (!a.norm)
    append_kernel<D><<<blocks, THREADS, 0, st>>>(a);
  else if (a.neighbour)
    norm_append_kernel<D, true><<<blocks, THREADS, 0, st>>>(a, pl);
  else
    norm_append_kernel<D, false><<<blocks, THREADS, 0, st>>>(a, pl);
  return cudaGetLastError();
}

// kernel<type, d, pairs> of the arguments
template <typename T>
cudaError_t fwd_of(const NormRopeArgs &a, cudaStream_t st) {
  if (a.d == 128) return a.neighbour ? launch_fwd<T, 128, true>(a, st) : launch_fwd<T, 128, false>(a, st);
  return a.neighbour ? launch_fwd<T, 64, true>(a, st) : launch_fwd<T, 64, false>(a, st);
}
template <typename T>
cudaError_t bwd_of(const NormRopeBwdArgs &b, cudaStream_t st) {
  if (b.fwd.d == 128)
    return b.fwd.neighbour ? launch_bwd<T, 128, true>(b, st) : launch_bwd<T, 128, false>(b, st);
  return b.fwd.neighbour ? launch_bwd<T, 64, true>(b, st) : launch_bwd<T, 64, false>(b, st);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, cudaStream_t st) {
  timing_mark(st, 0);
  const cudaError_t e = a.f32 ? fwd_of<float>(a, st) : fwd_of<__nv_bfloat16>(a, st);
  timing_mark(st, 1);
  return e;
}

cudaError_t launch_norm_rope_bwd(const NormRopeBwdArgs &b, cudaStream_t st) {
  timing_mark(st, 0);
  const cudaError_t e = b.fwd.f32 ? bwd_of<float>(b, st) : bwd_of<__nv_bfloat16>(b, st);
  timing_mark(st, 1);
  return e;
}

cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
  timing_mark(st, 0);
  const cudaError_t e = a.d == 128 ? launch_app<128>(a, st) : launch_app<64>(a, st);
  timing_mark(st, 1);
  return e;
}

}  // namespace chain
