// What the tensor-core products share: when they can be used, the driver's description of matrices to the copy
// engine, and the report of waits that ran out.
#include "ffn_tc.cuh"

namespace spmv {
namespace ffn {
namespace {

// rows (and matrices) that start at multiples of 16 bytes
bool describable(const Matrix &m, int64_t count) {
    return !m.p || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.ld % 8 == 0 && (count < 2 || m.expert % 8 == 0));
}

}  // namespace

namespace tc {

Encode encoder() {
    static const Encode fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess) {
            (void)cudaGetLastError();
            return static_cast<Encode>(nullptr);
        }
        return found == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(p) : nullptr;
    }();
    return fn;
}

}  // namespace tc

bool tc_supported(const Block &b, int dtype) {
    if (dtype == SPMV_F32 || !tc::encoder()) return false;
    const int64_t n = b.seg.count;
    for (const Matrix *m : {&b.x, &b.gate, &b.up, &b.h, &b.h2, &b.y, &b.dy, &b.dgate, &b.dup, &b.dx})
        if (!describable(*m, 1)) return false;
    for (const Matrix *m : {&b.wg, &b.wu, &b.wd, &b.dwg, &b.dwu, &b.dwd})
        if (!describable(*m, n)) return false;
    return true;
}

int launch_tc(int kind, const Block &b, int dtype, bool follows, cudaStream_t s) {
    return dtype == SPMV_F16 ? launch_tc_f16(kind, b, follows, s) : launch_tc_bf16(kind, b, follows, s);
}

}  // namespace ffn
}  // namespace spmv

using namespace spmv;

extern "C" SPMV_API int spmv_feed_forward_status(void *stream) {
    SPMV_TRY_CUDA(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
    int first = 0, second = 0;
    SPMV_TRY_CUDA(ffn::tc_flag_bf16(&first));
    SPMV_TRY_CUDA(ffn::tc_flag_f16(&second));
    if (!first && !second) return SPMV_OK;
    return set_error(SPMV_ERR_TIMEOUT, "a kernel of the feed-forward block gave up a wait: the results of the calls since the last report are invalid");
}
