// Arguments of the kernels behind spmv_topk_rows and its gradient (topk.cu, gate.cu).
#pragma once

#include "rows_common.cuh"

namespace spmv {
namespace rows {

struct TopArgs {
    int64_t rows, n, ldx;
    int k, weighting;
    float scale, inv_temperature;  // scale = log2(e) / temperature
    const void *x;
    int32_t *ids;
    float *vals, *weights, *lse;
};

struct TopGradArgs {
    int64_t rows, n, ldx, lddx, pieces;
    int k, weighting;
    float inv_temperature;
    const int32_t *ids;
    const float *weights, *dweights, *lse;
    const void *x;
    void *dx;
};

// Short rows and few entries, a router's choice (gate.cu): rows of up to kGateMaxN values, k up to
// kGateMaxK.
constexpr int kGateMaxN = 512;
constexpr int kGateMaxK = 16;
cudaError_t launch_gate(const TopArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_gate_grad(const TopGradArgs &a, int dtype, cudaStream_t s);

}  // namespace rows
}  // namespace spmv
