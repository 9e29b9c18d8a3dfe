// The distillation kernels for logits of type __nv_bfloat16.
#include "distill.cuh"

namespace spmv {
namespace rows {

cudaError_t launch_distill_bf16(DistillMode mode, const DistillArgs &a, cudaStream_t s) {
    return launch_distill<__nv_bfloat16>(mode, a, s);
}

}  // namespace rows
}  // namespace spmv
