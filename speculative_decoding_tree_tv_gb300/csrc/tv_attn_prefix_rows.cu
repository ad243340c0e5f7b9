// paged_rows_kernel, of the passes of calls with shared prefixes.
#define TV_UNIT 17
#include "tv_attn_paged_rows.cuh"

namespace tv {
namespace paged {

cudaError_t launch_rows_prefix(const PagedPlan& pl, int D, bool f16, bool mod, const CUtensorMap& tmK,
                               const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream) {
  return launch_any<true>(pl, D, f16, mod, tmK, tmV, p, stream);
}

}  // namespace paged
}  // namespace tv
