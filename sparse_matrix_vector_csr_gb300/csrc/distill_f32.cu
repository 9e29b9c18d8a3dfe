// The distillation kernels for logits of type float.
#include "distill.cuh"

namespace spmv {
namespace rows {

cudaError_t launch_distill_f32(DistillMode mode, const DistillArgs &a, cudaStream_t s) {
    return launch_distill<float>(mode, a, s);
}

}  // namespace rows
}  // namespace spmv
