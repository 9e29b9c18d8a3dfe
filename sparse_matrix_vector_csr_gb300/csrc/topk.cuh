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
    const float *weights, *dweights;
    const void *x;
    void *dx;
};

// The share of a row's values in its softmax, from the largest of them: q_i = w_0 exp((x_i - x_0) / T)
// with x_0 the first chosen entry, which is the row's maximum, and w_0 its weight.  A difference first, then
// the scale: the row's log-sum in 32 bits would take its own rounding, relative to the distance from 0, into
// every exponent (q of values near 1e4 off by 5e-4, of a row at the type's lowest value n times too large).
struct RowShare {
    float x0, w0, scale;  // scale = log2(e) / T
    __device__ __forceinline__ float of(float x) const { return w0 * ex2((x - x0) * scale); }
};

// Short rows and few entries, a router's choice (gate.cu): rows of up to kGateMaxN values, k up to
// kGateMaxK.
constexpr int kGateMaxN = 512;
constexpr int kGateMaxK = 16;
cudaError_t launch_gate(const TopArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_gate_grad(const TopGradArgs &a, int dtype, cudaStream_t s);

}  // namespace rows
}  // namespace spmv
