// Whose memory a pointer is, for the entry points that are called for microseconds of work.
#include <cuda.h>

#include "rows_common.cuh"

namespace spmv {
namespace rows {
namespace {

using PointerGetAttribute = CUresult (*)(void *, CUpointer_attribute, CUdeviceptr);

// The driver's query of one attribute, or nullptr where it cannot be had; then, and where the
// process sees several devices, the runtime's full query answers.
PointerGetAttribute one_device_query() {
    int devices = 0;
    if (cudaGetDeviceCount(&devices) != cudaSuccess) {
        (void)cudaGetLastError();
        return nullptr;
    }
    if (devices != 1) return nullptr;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuPointerGetAttribute", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess) {
        (void)cudaGetLastError();
        return nullptr;
    }
    return found == cudaDriverEntryPointSuccess ? reinterpret_cast<PointerGetAttribute>(fn) : nullptr;
}

}  // namespace

bool memory_here(const void *p) {
    static const PointerGetAttribute query = one_device_query();
    if (query) {
        unsigned int type = 0;
        if (query(&type, CU_POINTER_ATTRIBUTE_MEMORY_TYPE, reinterpret_cast<CUdeviceptr>(p)) == CUDA_SUCCESS &&
            type == CU_MEMORYTYPE_DEVICE)
            return true;
    }
    return device_memory_here(p);
}

}  // namespace rows
}  // namespace spmv
