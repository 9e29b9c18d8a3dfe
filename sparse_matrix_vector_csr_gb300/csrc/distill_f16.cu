// The distillation kernels for logits of type __half.
#include "distill.cuh"

namespace spmv {
namespace rows {

cudaError_t launch_distill_f16(DistillMode mode, const DistillArgs &a, cudaStream_t s) {
    return launch_distill<__half>(mode, a, s);
}

}  // namespace rows
}  // namespace spmv
