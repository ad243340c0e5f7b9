// paged_tc_kernel, of calls without shared prefixes.
#define TV_UNIT 13
#include "tv_attn_paged_tc.cuh"

namespace tv {
namespace paged {

cudaError_t launch_tc(const PagedPlan& pl, int D, bool f16, bool bias, const CUtensorMap& tmQ,
                      const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedAttnParams& p,
                      cudaStream_t stream) {
  return launch_any<false, false>(pl, D, f16, bias, tmQ, tmK, tmV, p, stream);
}

}  // namespace paged
}  // namespace tv
