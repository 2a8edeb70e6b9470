// fp32 rows of the head norms and position rotation (tq_append.cuh).
#include "tq_append.cuh"

namespace tq {

cudaError_t launch_append_f32(const AppendPlan& p, cudaStream_t stream) {
  return launch_append_typed<float, false>(p, stream);
}

}  // namespace tq
