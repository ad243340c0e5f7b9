// paged_tc_kernel over an 8-bit cache.
#define TV_UNIT 18
#include "tv_attn_paged_tc.cuh"

namespace tv {
namespace paged {

cudaError_t launch_tc_q8(const PagedPlan& pl, int D, bool f16, bool bias, const CUtensorMap& tmQ,
                         const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedAttnParams& p,
                         cudaStream_t stream) {
  return launch_any<false, true>(pl, D, f16, bias, tmQ, tmK, tmV, p, stream);
}

}  // namespace paged
}  // namespace tv
