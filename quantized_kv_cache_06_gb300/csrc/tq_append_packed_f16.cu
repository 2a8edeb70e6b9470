// fp16 rows of the append into packed pages (tq_append.cuh).
#include "tq_append.cuh"

namespace tq {

cudaError_t launch_append_packed_f16(const AppendPlan& p, cudaStream_t stream) {
  return launch_append_typed<__half, true>(p, stream);
}

}  // namespace tq
