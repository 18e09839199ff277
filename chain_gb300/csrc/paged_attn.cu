// paged_attn.cu -- attention of new tokens over a paged cache, each sequence by itself; the kernels
// stand in paged_attn.cuh.
#include "paged_attn.cuh"

namespace chain {
namespace {

template <int D>
cudaError_t launch(const PagedAttnArgs &a, const WaitCfg &wc, cudaStream_t st) {
  const Params p = params_of<D>(a, wc);
  return launch_pass<D, ALONE>(a, p, a.seqs.batch, few_rows(a, p.G), may_have_chunks(a, p.G), false, st);
}

}  // namespace

size_t paged_attn_workspace(int d) { return pass_workspace(d); }

cudaError_t launch_paged_attn(const PagedAttnArgs &a, const WaitCfg &wc, cudaStream_t st) {
  return a.d == 128 ? launch<128>(a, wc, st) : launch<64>(a, wc, st);
}

}  // namespace chain
