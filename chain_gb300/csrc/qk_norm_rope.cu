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
// output once, so memory bandwidth bounds them.
//
// Angles.  p w_i mod 2 pi keeps no fp32 accuracy at far positions, and fp64
// is slow here, so angles are kept in turns as 64-bit fixed point: w_i / 2 pi
// is formed once per block as an integer U_i = w_i / (2 pi) 2^64 (mod 2^64,
// exact to one unit), and p U_i mod 2^64 is the angle of position p: exact
// modular arithmetic whose error is |p| 2^-64 turns.  Its top 32 bits go to
// sincospif.
#include "internal.h"

namespace chain {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_FREQ = 64;  // rot / 2 at d = 128

// 1 / (2 pi) = 0.159154943... as a 128-bit binary fraction
constexpr unsigned long long INV_2PI_HI = 0x28be60db9391054aull;
constexpr unsigned long long INV_2PI_LO = 0x7f09d5f47d4d3770ull;

// w / (2 pi) in units of 2^-64 turns, mod 2^64.  w = m 2^e with an integer m
// of 24 bits; m times the 128-bit fraction, shifted by e.  (From w = 2^24 on,
// bits past the fraction's end would be needed: accuracy falls there.)
__device__ __forceinline__ unsigned long long turns_per_position(float w) {
  const uint32_t b = __float_as_uint(w);
  const int ex = (int)((b >> 23) & 0xff);
  if (ex == 255) return 0;  // infinite or NaN frequency: no rotation
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

// (cos, sin) of position p and frequency U
__device__ __forceinline__ float2 angle(int p, unsigned long long u) {
  const unsigned long long a = u * (unsigned long long)(long long)p;
  const float t = (float)(int)(a >> 32) * 0x1p-31f;  // twice the turns, in [-1, 1]
  float2 cs;
  sincospif(t, &cs.y, &cs.x);
  return cs;
}

// ------------------------------------------------------- eight elements a lane
template <typename T>
struct Row8;
template <>
struct Row8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    v = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                               pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
};
template <>
struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float *p, const float (&f)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

__device__ __forceinline__ void load_weight(const NormRopeWeight &g, int e0, float (&f)[8]) {
  if (g.bf16) {
    Row8<__nv_bfloat16> r;
    r.load(static_cast<const __nv_bfloat16 *>(g.ptr) + e0);
    r.get(f);
  } else {
    Row8<float> r;
    r.load(static_cast<const float *>(g.ptr) + e0);
    r.get(f);
  }
}

// What a lane knows of the rotation of its eight elements at one token.
// Pairs (i, i + rot/2): all eight lie in one half and their partners in
// lane `src`; pairs (2i, 2i + 1) lie within the lane.
struct LaneRope {
  float c[8], s[8];
  int src;     // partner lane (pairs of halves)
  bool on;     // the elements rotate
  bool second; // they are the second of their pairs (pairs of halves)
};

template <int D>
__device__ __forceinline__ void lane_rope_setup(LaneRope &lr, int lane, int rot, int neighbour) {
  constexpr int LPR = D / 8;  // lanes a row
  const int l = lane % LPR;
  lr.on = l * 8 < rot;
  lr.second = !neighbour && l * 16 >= rot;
  const int half = rot / 16;  // lanes of half the rotated elements
  lr.src = neighbour || !lr.on ? lane : (lr.second ? lane - half : lane + half);
}

// The token's (cos, sin) of each frequency into the warp's table, then the
// lane's own into registers.  Elements that do not rotate get (1, 0).
template <int D>
__device__ __forceinline__ void lane_rope_token(LaneRope &lr, int lane, int rot, int neighbour, int p,
                                                const unsigned long long *turns, float2 *table) {
  constexpr int LPR = D / 8;
  const int l = lane % LPR;
  __syncwarp();  // the table's last readers are done
  for (int f = lane; f < rot / 2; f += 32) table[f] = angle(p, turns[f]);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float2 cs = make_float2(1.0f, 0.0f);
    if (lr.on) {
      const int e = l * 8 + k;
      cs = table[neighbour ? e / 2 : (lr.second ? e - rot / 2 : e)];
    }
    lr.c[k] = cs.x;
    lr.s[k] = cs.y;
  }
}

// y = R u (SIGN = 1) or R^T u (SIGN = -1).  Every lane of the warp calls it.
template <int SIGN>
__device__ __forceinline__ void rotate(const LaneRope &lr, int neighbour, float (&u)[8]) {
  if (neighbour) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float a = u[k], b = u[k + 1], s = SIGN * lr.s[k];
      u[k] = a * lr.c[k] - b * s;
      u[k + 1] = a * s + b * lr.c[k];
    }
  } else {
    const float sg = lr.second ? (float)SIGN : -(float)SIGN;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float o = __shfl_sync(0xffffffffu, u[k], lr.src);
      u[k] = u[k] * lr.c[k] + o * (sg * lr.s[k]);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Offset in elements of token t: t = b n + i of [B][n][H][d].
__device__ __forceinline__ int64_t token_off(const NormRopeSide &x, int64_t t, int64_t n) {
  if (x.s_batch == n * x.s_tok) return t * x.s_tok;
  const int64_t b = t / n;
  return b * x.s_batch + (t - b * n) * x.s_tok;
}

// Rows [h0, h1) of one token: norm, rotation, store.
template <typename T, int D>
__device__ __forceinline__ void fwd_rows(const T *src, int64_t s_head, T *dst, int64_t d_head, int h0,
                                         int h1, const float (&g)[8], float eps, int neighbour,
                                         const LaneRope &lr, int lane) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
  const int sub = lane / LPR, e0 = (lane % LPR) * 8;
  for (int h = h0 + sub; h - sub < h1; h += RPW * U) {
    Row8<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hh = h + u * RPW;
      if (hh < h1) x[u].load(src + hh * s_head + e0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hh = h + u * RPW;
      if (hh - sub >= h1) break;  // warp-uniform
      float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (hh < h1) x[u].get(f);
      float q = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) q = fmaf(f[k], f[k], q);
      const float r = rsqrtf(row_sum<LPR>(q) * (1.0f / D) + eps);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = f[k] * r * g[k];
      rotate<1>(lr, neighbour, f);
      if (hh < h1) Row8<T>::store(dst + hh * d_head + e0, f);
    }
  }
}

// Heads [c per, (c + 1) per) of `heads`, clipped
__device__ __forceinline__ void clip(int lo, int hi, int from, int heads, int &h0, int &h1) {
  h0 = max(lo - from, 0);
  h1 = min(hi - from, heads);
}

template <typename T, int D>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const NormRopeArgs a, int per) {
  __shared__ unsigned long long turns[MAX_FREQ];
  __shared__ float2 table[WARPS][MAX_FREQ];
  for (int f = threadIdx.x; f < a.rot / 2; f += THREADS) turns[f] = turns_per_position(__ldg(a.inv_freq + f));
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  LaneRope lr;
  lane_rope_setup<D>(lr, lane, a.rot, a.neighbour);
  float gq[8], gk[8];
  load_weight(a.gq, (lane % (D / 8)) * 8, gq);
  load_weight(a.gk, (lane % (D / 8)) * 8, gk);
  const int heads = a.H + a.Hkv, chunks = (heads + per - 1) / per;
  const int64_t items = a.tokens * chunks, step = (int64_t)gridDim.x * WARPS;
  for (int64_t it = blockIdx.x * (int64_t)WARPS + warp; it < items; it += step) {
    const int64_t t = it / chunks;
    const int lo = (int)(it - t * chunks) * per, hi = min(lo + per, heads);
    const int p = a.positions ? __ldg(a.positions + t) : (int)(t % a.n);
    lane_rope_token<D>(lr, lane, a.rot, a.neighbour, p, turns, table[warp]);
    int h0, h1;
    clip(lo, hi, 0, a.H, h0, h1);
    fwd_rows<T, D>(static_cast<const T *>(a.q.ptr) + token_off(a.q, t, a.n), a.q.s_head,
                   static_cast<T *>(a.qo.ptr) + token_off(a.qo, t, a.n), a.qo.s_head, h0, h1, gq, a.eps,
                   a.neighbour, lr, lane);
    clip(lo, hi, a.H, a.Hkv, h0, h1);
    fwd_rows<T, D>(static_cast<const T *>(a.k.ptr) + token_off(a.k, t, a.n), a.k.s_head,
                   static_cast<T *>(a.ko.ptr) + token_off(a.ko, t, a.n), a.ko.s_head, h0, h1, gk, a.eps,
                   a.neighbour, lr, lane);
  }
}

// ------------------------------------------------------------------ backward
template <typename T, int D>
__device__ __forceinline__ void bwd_rows(const T *src, int64_t s_head, const T *dsrc, int64_t g_head,
                                         T *dst, int64_t d_head, int h0, int h1, const float (&g)[8],
                                         float (&dg)[8], float eps, int neighbour, const LaneRope &lr,
                                         int lane) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 2;
  const int sub = lane / LPR, e0 = (lane % LPR) * 8;
  for (int h = h0 + sub; h - sub < h1; h += RPW * U) {
    Row8<T> x[U], dy[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hh = h + u * RPW;
      if (hh < h1) {
        x[u].load(src + hh * s_head + e0);
        dy[u].load(dsrc + hh * g_head + e0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hh = h + u * RPW;
      if (hh - sub >= h1) break;  // warp-uniform
      float f[8] = {0, 0, 0, 0, 0, 0, 0, 0}, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (hh < h1) {
        x[u].get(f);
        dy[u].get(v);
      }
      rotate<-1>(lr, neighbour, v);
      float q = 0.0f, w = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        q = fmaf(f[k], f[k], q);
        w = fmaf(v[k] * g[k], f[k], w);
      }
      q = row_sum<LPR>(q);
      w = row_sum<LPR>(w);
      const float r = rsqrtf(q * (1.0f / D) + eps);
      const float c = w * (1.0f / D) * r * r;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dg[k] = fmaf(v[k] * f[k], r, dg[k]);
        f[k] = r * (v[k] * g[k] - f[k] * c);
      }
      if (hh < h1) Row8<T>::store(dst + hh * d_head + e0, f);
    }
  }
}

// part[block][2][D]: the block's sums of a x r over its query rows and its
// key rows.  No atomics: rows are dealt to warps by their number and every
// sum has one order.
template <typename T, int D>
__global__ void __launch_bounds__(THREADS) norm_rope_bwd_kernel(const NormRopeBwdArgs b, int per,
                                                                float *__restrict__ part) {
  __shared__ unsigned long long turns[MAX_FREQ];
  __shared__ float2 table[WARPS][MAX_FREQ];
  __shared__ float sums[WARPS][2][D];
  const NormRopeArgs &a = b.fwd;
  for (int f = threadIdx.x; f < a.rot / 2; f += THREADS) turns[f] = turns_per_position(__ldg(a.inv_freq + f));
  __syncthreads();
  constexpr int LPR = D / 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  LaneRope lr;
  lane_rope_setup<D>(lr, lane, a.rot, a.neighbour);
  float gq[8], gk[8], dgq[8] = {0, 0, 0, 0, 0, 0, 0, 0}, dgk[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  load_weight(a.gq, (lane % LPR) * 8, gq);
  load_weight(a.gk, (lane % LPR) * 8, gk);
  const int heads = a.H + a.Hkv, chunks = (heads + per - 1) / per;
  const int64_t items = a.tokens * chunks, step = (int64_t)gridDim.x * WARPS;
  for (int64_t it = blockIdx.x * (int64_t)WARPS + warp; it < items; it += step) {
    const int64_t t = it / chunks;
    const int lo = (int)(it - t * chunks) * per, hi = min(lo + per, heads);
    const int p = a.positions ? __ldg(a.positions + t) : (int)(t % a.n);
    lane_rope_token<D>(lr, lane, a.rot, a.neighbour, p, turns, table[warp]);
    int h0, h1;
    clip(lo, hi, 0, a.H, h0, h1);
    bwd_rows<T, D>(static_cast<const T *>(a.q.ptr) + token_off(a.q, t, a.n), a.q.s_head,
                   static_cast<const T *>(b.dqo.ptr) + token_off(b.dqo, t, a.n), b.dqo.s_head,
                   static_cast<T *>(a.qo.ptr) + token_off(a.qo, t, a.n), a.qo.s_head, h0, h1, gq, dgq,
                   a.eps, a.neighbour, lr, lane);
    clip(lo, hi, a.H, a.Hkv, h0, h1);
    bwd_rows<T, D>(static_cast<const T *>(a.k.ptr) + token_off(a.k, t, a.n), a.k.s_head,
                   static_cast<const T *>(b.dko.ptr) + token_off(b.dko, t, a.n), b.dko.s_head,
                   static_cast<T *>(a.ko.ptr) + token_off(a.ko, t, a.n), a.ko.s_head, h0, h1, gk, dgk,
                   a.eps, a.neighbour, lr, lane);
  }
  // rows of a warp, then warps of the block
#pragma unroll
  for (int k = 0; k < 8; ++k) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      dgq[k] += __shfl_xor_sync(0xffffffffu, dgq[k], o);
      dgk[k] += __shfl_xor_sync(0xffffffffu, dgk[k], o);
    }
    if (lane < LPR) {
      sums[warp][0][lane * 8 + k] = dgq[k];
      sums[warp][1][lane * 8 + k] = dgk[k];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += THREADS) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) s += sums[w][i / D][i % D];
    part[(int64_t)blockIdx.x * 2 * D + i] = s;
  }
}

// dgq, dgk [D] from the blocks' sums: one block for 32 of the 2 D columns,
// warp w adding the blocks w, w + 8, ...
__global__ void __launch_bounds__(THREADS) norm_rope_dg_kernel(const float *__restrict__ part, int blocks,
                                                               int d, float *__restrict__ dgq,
                                                               float *__restrict__ dgk) {
  __shared__ float sums[WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s = 0.0f;
  for (int i = warp; i < blocks; i += WARPS) s += part[(int64_t)i * 2 * d + col];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < WARPS; ++w) s += sums[w][lane];
    (col < d ? dgq : dgk - d)[col] = s;
  }
}

// -------------------------------------------------------------- cache writes
template <int D>
__device__ __forceinline__ void copy_rows(const __nv_bfloat16 *src, int64_t s_head, __nv_bfloat16 *dst,
                                          int64_t d_head, int h0, int h1, int lane) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int e0 = (lane % LPR) * 8;
  for (int h = h0 + lane / LPR; h < h1; h += RPW)
    *reinterpret_cast<uint4 *>(dst + h * d_head + e0) =
        *reinterpret_cast<const uint4 *>(src + h * s_head + e0);
}

// NORM: Q normed, rotated and written to qo, K normed, rotated and written
// into its page, V copied into its page.  Otherwise K and V copied.
template <int D, bool NORM>
__global__ void __launch_bounds__(THREADS) append_kernel(const AppendArgs a, int per) {
  __shared__ unsigned long long turns[MAX_FREQ];
  __shared__ float2 table[WARPS][MAX_FREQ];
  using T = __nv_bfloat16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  LaneRope lr;
  float gq[8], gk[8];
  if constexpr (NORM) {
    for (int f = threadIdx.x; f < a.rot / 2; f += THREADS)
      turns[f] = turns_per_position(__ldg(a.inv_freq + f));
    __syncthreads();
    lane_rope_setup<D>(lr, lane, a.rot, a.neighbour);
    load_weight(a.gq, (lane % (D / 8)) * 8, gq);
    load_weight(a.gk, (lane % (D / 8)) * 8, gk);
  }
  const PagedSeqs &s = a.seqs;
  const int qh = NORM ? a.H : 0;
  const int heads = qh + 2 * a.Hkv, chunks = (heads + per - 1) / per;
  const int64_t items = a.tokens * chunks, step = (int64_t)gridDim.x * WARPS;
  for (int64_t it = blockIdx.x * (int64_t)WARPS + warp; it < items; it += step) {
    const int t = (int)(it / chunks);
    const int lo = (int)(it - (int64_t)t * chunks) * per, hi = min(lo + per, heads);
    // the sequence of token t: the last b with cu[b] <= t
    int b = 0, e = s.batch;
    while (e - b > 1) {
      const int m = (b + e) >> 1;
      if (__ldg(s.cu + m) <= t)
        b = m;
      else
        e = m;
    }
    const int first = __ldg(s.cu + b), end = __ldg(s.cu + b + 1);
    if (t < first || t >= end) continue;  // a row behind the last sequence
    const int64_t len = __ldg(s.lens + b), pos = len - end + t;
    // its place; out of the table's or the pool's range: reported, not written
    int64_t page = -1;
    int slot = 0;
    if (pos >= 0 && pos < ((int64_t)s.max_pages << s.page_shift)) {
      page = __ldg(s.table + b * s.table_stride + (pos >> s.page_shift));
      slot = (int)(pos & ((1 << s.page_shift) - 1));
    }
    if (page < 0 || page >= s.num_pages) {
      if (lane == 0) atomicExch(&a.status->reserved[0], 1);
      page = -1;
    }
    int h0, h1;
    if constexpr (NORM) {
      lane_rope_token<D>(lr, lane, a.rot, a.neighbour, (int)pos, turns, table[warp]);
      clip(lo, hi, 0, a.H, h0, h1);
      fwd_rows<T, D>(static_cast<const T *>(a.q.ptr) + t * a.q.s_tok, a.q.s_head,
                     static_cast<T *>(a.qo.ptr) + t * a.qo.s_tok, a.qo.s_head, h0, h1, gq, a.eps,
                     a.neighbour, lr, lane);
    }
    if (page < 0) continue;
    T *kd = static_cast<T *>(a.kc.ptr) + page * a.kc.s_page + slot * a.kc.s_slot;
    T *vd = static_cast<T *>(a.vc.ptr) + page * a.vc.s_page + slot * a.vc.s_slot;
    clip(lo, hi, qh, a.Hkv, h0, h1);
    if constexpr (NORM)
      fwd_rows<T, D>(static_cast<const T *>(a.k.ptr) + t * a.k.s_tok, a.k.s_head, kd, a.kc.s_head, h0, h1,
                     gk, a.eps, a.neighbour, lr, lane);
    else
      copy_rows<D>(static_cast<const T *>(a.k.ptr) + t * a.k.s_tok, a.k.s_head, kd, a.kc.s_head, h0, h1,
                   lane);
    clip(lo, hi, qh + a.Hkv, a.Hkv, h0, h1);
    copy_rows<D>(static_cast<const T *>(a.v.ptr) + t * a.v.s_tok, a.v.s_head, vd, a.vc.s_head, h0, h1,
                 lane);
  }
}

// Rows a warp takes at once, and blocks: one warp to a token once the tokens
// fill the card by themselves, fewer heads to a warp below that.
struct Split {
  int per;
  unsigned grid;
};
Split split(int64_t tokens, int heads, int rows_per_pass, int max_grid) {
  int64_t chunks = 1;
  const int most = (heads + rows_per_pass - 1) / rows_per_pass;
  const int64_t want = (int64_t)152 * 16;  // warps that keep the memory busy
  if (tokens < want) {
    chunks = (want + tokens - 1) / tokens;
    if (chunks > most) chunks = most;
  }
  Split s;
  s.per = (int)((heads + chunks - 1) / chunks);
  s.per = (s.per + rows_per_pass - 1) / rows_per_pass * rows_per_pass;
  const int64_t items = tokens * ((heads + s.per - 1) / s.per);
  const int64_t blocks = (items + WARPS - 1) / WARPS;
  s.grid = (unsigned)(blocks < max_grid ? blocks : max_grid);
  return s;
}

template <typename T, int D>
cudaError_t launch_fwd(const NormRopeArgs &a, cudaStream_t st) {
  const Split s = split(a.tokens, a.H + a.Hkv, 32 / (D / 8), 152 * 8);
  norm_rope_kernel<T, D><<<s.grid, THREADS, 0, st>>>(a, s.per);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_bwd(const NormRopeBwdArgs &b, cudaStream_t st) {
  float *part = static_cast<float *>(b.workspace);
  unsigned blocks = 0;  // no tokens: no sums, dg = 0
  if (b.fwd.tokens > 0) {
    const Split s = split(b.fwd.tokens, b.fwd.H + b.fwd.Hkv, 32 / (D / 8), kNormRopeBwdMaxGrid);
    blocks = s.grid;
    norm_rope_bwd_kernel<T, D><<<blocks, THREADS, 0, st>>>(b, s.per, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  norm_rope_dg_kernel<<<2 * D / 32, THREADS, 0, st>>>(part, (int)blocks, D, b.dgq, b.dgk);
  return cudaGetLastError();
}

template <int D, bool NORM>
cudaError_t launch_app(const AppendArgs &a, cudaStream_t st) {
  const Split s = split(a.tokens, (NORM ? a.H : 0) + 2 * a.Hkv, 32 / (D / 8), 152 * 8);
  append_kernel<D, NORM><<<s.grid, THREADS, 0, st>>>(a, s.per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, cudaStream_t st) {
  timing_mark(st, 0);
  cudaError_t e;
  if (a.f32)
    e = a.d == 128 ? launch_fwd<float, 128>(a, st) : launch_fwd<float, 64>(a, st);
  else
    e = a.d == 128 ? launch_fwd<__nv_bfloat16, 128>(a, st) : launch_fwd<__nv_bfloat16, 64>(a, st);
  timing_mark(st, 1);
  return e;
}

cudaError_t launch_norm_rope_bwd(const NormRopeBwdArgs &b, cudaStream_t st) {
  timing_mark(st, 0);
  cudaError_t e;
  if (b.fwd.f32)
    e = b.fwd.d == 128 ? launch_bwd<float, 128>(b, st) : launch_bwd<float, 64>(b, st);
  else
    e = b.fwd.d == 128 ? launch_bwd<__nv_bfloat16, 128>(b, st) : launch_bwd<__nv_bfloat16, 64>(b, st);
  timing_mark(st, 1);
  return e;
}

cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
  timing_mark(st, 0);
  cudaError_t e;
  if (a.norm)
    e = a.d == 128 ? launch_app<128, true>(a, st) : launch_app<64, true>(a, st);
  else
    e = a.d == 128 ? launch_app<128, false>(a, st) : launch_app<64, false>(a, st);
  timing_mark(st, 1);
  return e;
}

}  // namespace chain
