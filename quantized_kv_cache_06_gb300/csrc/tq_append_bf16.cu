// bf16 rows of the head norms and position rotation (tq_append.cuh).
#include "tq_append.cuh"

namespace tq {

cudaError_t launch_append_bf16(const AppendPlan& p, cudaStream_t stream) {
  return launch_append_typed<__nv_bfloat16, false>(p, stream);
}

}  // namespace tq
