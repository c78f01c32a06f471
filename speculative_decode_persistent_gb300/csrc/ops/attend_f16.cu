// The attention kernels over a binary16 pool.
#include "attend.cuh"

namespace mk {
namespace ops {
cudaError_t launch_attend_f16(int ns, int cg, const AttendParams& a, const CUtensorMap& tk, const CUtensorMap& tv,
                              int device, cudaStream_t stream) {
  return launch_any<false>(ns, cg, a, tk, tv, device, stream);
}
}  // namespace ops
}  // namespace mk
