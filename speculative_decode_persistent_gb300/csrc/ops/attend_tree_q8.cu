// The attention kernels over a q8 pool, rows being nodes of trees.
#include "attend.cuh"

namespace mk {
namespace ops {
cudaError_t launch_attend_tree_q8(int ns, int cg, const AttendParams& a, const CUtensorMap& tk, const CUtensorMap& tv,
                                   int device, cudaStream_t stream) {
  return launch_any<true, true>(ns, cg, a, tk, tv, device, stream);
}
}  // namespace ops
}  // namespace mk
