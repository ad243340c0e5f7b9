// paged_rows_q8_kernel over e4m3 codes.
#define TV_UNIT 15
#include "tv_attn_q8_rows.cuh"

namespace tv {
namespace paged {

cudaError_t launch_rows_e4m3(const PagedPlan& pl, int D, bool mod, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream) {
  return launch_format<true>(pl, D, mod, tmK, tmV, p, stream);
}

}  // namespace paged
}  // namespace tv
