// The feed-forward block's products by the tensor cores for bfloat16 values.
#include "ffn_tc.cuh"

namespace spmv {
namespace ffn {
int launch_tc_bf16(int kind, const Block &b, bool follows, cudaStream_t s) { return tc::launch_kind<__nv_bfloat16>(kind, b, follows, s); }
cudaError_t tc_flag_bf16(int *value) { return tc::take_flag(value); }
}  // namespace ffn
}  // namespace spmv
