// The feed-forward block's products by the tensor cores for half values.
#include "ffn_tc.cuh"

namespace spmv {
namespace ffn {
int launch_tc_f16(int kind, const Block &b, bool follows, cudaStream_t s) { return tc::launch_kind<__half>(kind, b, follows, s); }
cudaError_t tc_flag_f16(int *value) { return tc::take_flag(value); }
}  // namespace ffn
}  // namespace spmv
