// paged_rows_kernel, of calls without shared prefixes.
#define TV_UNIT 12
#include "tv_attn_paged_rows.cuh"

namespace tv {
namespace paged {

cudaError_t launch_rows(const PagedPlan& pl, int D, bool f16, bool mod, const CUtensorMap& tmK,
                        const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream) {
  return launch_any<false>(pl, D, f16, mod, tmK, tmV, p, stream);
}

}  // namespace paged
}  // namespace tv
