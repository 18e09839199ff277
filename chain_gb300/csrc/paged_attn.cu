// paged_attn.cu -- softmax attention of a chunk of new tokens over a paged
// K/V cache (the unit O = f(A B) C with f = row softmax, K and V read from
// the pages that a sequence's table names).
//
// New token i of sequence b, with n_b new tokens and lens[b] cached
// positions (the new ones included), sees the keys j < lens[b], and of those
// only j <= lens[b] - n_b + i under the causal mask.  A row that sees none
// gets O = 0 and LSE = -inf.
//
// One block per (token, head): its four warps take every fourth key, each
// with the running maximum and sum of its keys' softmax, and join at the end.
#include "internal.h"

namespace chain {
namespace {

template <int D>
__global__ void __launch_bounds__(128) paged_attn_kernel(const PagedAttnArgs a, DevStatus *status) {
  constexpr int E = D / 32;  // elements a lane
  __shared__ float sm[4], sl[4], so[4][D];
  const PagedSeqs &s = a.seqs;
  const int t = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int b = 0, e = s.batch;
  while (e - b > 1) {
    const int m = (b + e) >> 1;
    if (__ldg(s.cu + m) <= t)
      b = m;
    else
      e = m;
  }
  const int first = __ldg(s.cu + b), end = __ldg(s.cu + b + 1);
  if (t < first || t >= end) return;
  const int64_t most = (int64_t)s.max_pages << s.page_shift;
  int64_t len = __ldg(s.lens + b);
  if (len < 0 || len > most) {
    if (threadIdx.x == 0) atomicExch(&status->reserved[0], 1);
    len = len < 0 ? 0 : most;
  }
  const int64_t seen = a.causal ? len - end + t + 1 : len;
  const int hk = h / (a.H / a.Hkv);
  float q[E], o[E], m = -INFINITY, l = 0.0f;
  const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.Q) + t * a.q_stok + h * a.q_shead;
#pragma unroll
  for (int k = 0; k < E; ++k) {
    q[k] = __bfloat162float(qp[lane + 32 * k]) * a.scale * 1.4426950408889634f;
    o[k] = 0.0f;
  }
  for (int64_t j = warp; j < seen; j += 4) {
    const int page = __ldg(s.table + b * s.table_stride + (j >> s.page_shift));
    if (page < 0 || page >= s.num_pages) {  // reported; the key counts as zeros
      if (lane == 0) atomicExch(&status->reserved[0], 1);
    }
    const bool ok = page >= 0 && page < s.num_pages;
    const int64_t slot = j & ((1 << s.page_shift) - 1);
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(a.kc.ptr) + page * a.kc.s_page +
                              slot * a.kc.s_slot + hk * a.kc.s_head;
    const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(a.vc.ptr) + page * a.vc.s_page +
                              slot * a.vc.s_slot + hk * a.vc.s_head;
    float x = 0.0f;
#pragma unroll
    for (int k = 0; k < E; ++k) x += ok ? q[k] * __bfloat162float(kp[lane + 32 * k]) : 0.0f;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
    const float mn = fmaxf(m, x), f = ex2(m - mn), w = ex2(x - mn);
    l = l * f + w;
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] = o[k] * f + (ok ? w * __bfloat162float(vp[lane + 32 * k]) : 0.0f);
    m = mn;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int k = 0; k < E; ++k) so[warp][lane + 32 * k] = o[k];
  __syncthreads();
  const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float w[4], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = top == -INFINITY ? 0.0f : ex2(sm[i] - top);
    sum += w[i] * sl[i];
  }
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  __nv_bfloat16 *op = static_cast<__nv_bfloat16 *>(a.O) + t * a.o_stok + h * a.o_shead;
  for (int i = threadIdx.x; i < D; i += 128)
    op[i] = __float2bfloat16((w[0] * so[0][i] + w[1] * so[1][i] + w[2] * so[2][i] + w[3] * so[3][i]) * inv);
  if (threadIdx.x == 0)
    a.LSE[h * a.lse_shead + t] = sum > 0.0f ? (top + lg2(sum)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

size_t paged_attn_workspace(int) { return 256; }

cudaError_t launch_paged_attn(const PagedAttnArgs &a, const WaitCfg &wc, cudaStream_t st) {
  timing_mark(st, 0);
  const dim3 grid((unsigned)a.total, (unsigned)a.H);
  if (a.d == 128)
    paged_attn_kernel<128><<<grid, 128, 0, st>>>(a, wc.status);
  else
    paged_attn_kernel<64><<<grid, 128, 0, st>>>(a, wc.status);
  timing_mark(st, 1);
  return cudaGetLastError();
}

}  // namespace chain
