// paged_rows_q8_kernel over int8 codes.
#define TV_UNIT 16
#include "tv_attn_q8_rows.cuh"

namespace tv {
namespace paged {

cudaError_t launch_rows_int8(const PagedPlan& pl, int D, bool mod, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream) {
  return launch_format<false>(pl, D, mod, tmK, tmV, p, stream);
}

}  // namespace paged
}  // namespace tv
