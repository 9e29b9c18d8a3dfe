// Entry points of the gated feed-forward block over segments of rows.
#include "ffn.cuh"

namespace spmv {
namespace ffn {
namespace {

constexpr int64_t kMaxWidth = int64_t(1) << 20;

int64_t padded(int64_t f) { return ceil_div(f, 8) * 8; }

int check_sizes(int64_t rows, int64_t d, int64_t f, int dtype) {
    // (a tile's first row and the rows of its copies are 32-bit coordinates)
    if (rows < 0 || rows > (int64_t(1) << 31) - 4096) return refuse("rows must lie in [0, 2^31 - 4096]");
    if (d < 1 || d > kMaxWidth || f < 1 || f > kMaxWidth) return refuse("d and f must lie in [1, 2^20]");
    if (!row_dtype_ok(dtype)) return refuse("dtype must be SPMV_F32, SPMV_F16 or SPMV_BF16");
    return SPMV_OK;
}
// `count` matrices of n rows of m values
int check_weights(const void *p, const char *name, int64_t count, int64_t n, int64_t m, int64_t ld, int64_t expert, int dtype) {
    SPMV_TRY(check_shape(n, m, ld, name));
    if (count > 1 && (expert < (n - 1) * ld + m || expert >= int64_t(1) << 40))
        return refuse(std::string(name) + ": the experts' matrices overlap or are too far apart");
    return check_array(p, name, row_value_bytes(dtype));
}
size_t weight_bytes(int64_t count, int64_t n, int64_t m, int64_t ld, int64_t expert, int dtype) {
    return (static_cast<size_t>(count - 1) * expert + (n - 1) * ld + m) * row_value_bytes(dtype);
}
struct Array {
    const void *p;
    size_t bytes;
    const char *name;
};
// No output shares a byte with another array of the call.
int check_outputs(std::initializer_list<Array> outputs, std::initializer_list<Array> inputs) {
    for (const Array *a = outputs.begin(); a != outputs.end(); ++a) {
        for (const Array &b : inputs) SPMV_TRY(check_apart(a->p, a->bytes, a->name, b.p, b.bytes, b.name));
        for (const Array *b = outputs.begin(); b != a; ++b) SPMV_TRY(check_apart(a->p, a->bytes, a->name, b->p, b->bytes, b->name));
    }
    return SPMV_OK;
}
int check_experts(int32_t experts) {
    return experts < 1 || experts > kMaxSegments ? refuse("experts must lie in [1, " + std::to_string(kMaxSegments) + "]") : SPMV_OK;
}
// h is held in two parts
bool two_parts(int64_t rows, int32_t experts, int dtype) { return dtype != SPMV_F32 && short_rows(rows, experts) != 0; }
int check_segments(int32_t experts, const int32_t *offsets) {
    SPMV_TRY(check_experts(experts));
    if (!offsets) return experts == 1 ? SPMV_OK : refuse("offsets is NULL, which means one segment of all rows, with experts not 1");
    return check_array(offsets, "offsets", 4);
}
// Parts of each segment's rows in the weights' gradients: enough tiles for the GPU where the matrices are small, of at
// least 512 rows on average (a backward pass of 65536 rows, d = f = 64: float 7434 -> 343 us, bf16 258 -> 60; 256: bf16 301 -> 128).
int weight_splits(int64_t rows, int64_t d, int64_t f, int32_t experts) {
    const int64_t tiles = 3 * ceil_div(d, 128) * ceil_div(f, 128) * experts, mean = rows / experts;
    int splits = 1;
    while (splits < 64 && tiles * splits < 2 * kSms && mean / (2 * splits) >= 512) splits *= 2;
    return splits;
}
int64_t rows_bytes(int64_t rows, int64_t f, int dtype) { return rows * padded(f) * row_value_bytes(dtype); }

// The parts' sums, in the order of the rows, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) k_join_weights(Block b) {
    const int64_t n = b.d * b.f, all = 3 * b.seg.count * n;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t matrix = i / n;  // which product, then segment
        const int which = static_cast<int>(matrix / b.seg.count), e = static_cast<int>(matrix % b.seg.count);
        T *out = static_cast<T *>((which == 0 ? b.dwg : which == 1 ? b.dwu : b.dwd).p);
        if (!out) continue;
        const float *p = b.part_sums(which, e, 0) + (i - matrix * n);
        float sum = p[0];
#pragma unroll 8
        for (int k = 1; k < b.splits; ++k) sum += p[k * n];
        out[e * n + (i - matrix * n)] = from_f32<T>(sum);
    }
}
int launch_join(const Block &b, int dtype, cudaStream_t s) {
    const int64_t ctas = ceil_div(3 * b.seg.count * b.d * b.f, 256);
    const dim3 grid(static_cast<unsigned>(ctas < 8 * kSms ? ctas : 8 * kSms));
    if (dtype == SPMV_F32) k_join_weights<float><<<grid, 256, 0, s>>>(b);
    else if (dtype == SPMV_F16) k_join_weights<__half><<<grid, 256, 0, s>>>(b);
    else k_join_weights<__nv_bfloat16><<<grid, 256, 0, s>>>(b);
    SPMV_TRY_CUDA(cudaGetLastError());
    return SPMV_OK;
}
using Launch = int (*)(int, const Block &, int, bool, cudaStream_t);
Matrix matrix(const void *p, int64_t ld, int64_t expert = 0) { return Matrix{const_cast<void *>(p), ld, expert}; }

}  // namespace
}  // namespace ffn
}  // namespace spmv

using namespace spmv;
using namespace spmv::ffn;

extern "C" SPMV_API int64_t spmv_feed_forward_workspace(int64_t rows, int64_t d, int64_t f, int32_t experts, int dtype,
                                                        int gradient) {
    SPMV_TRY(check_sizes(rows, d, f, dtype));
    SPMV_TRY(check_experts(experts));
    const int64_t each = rows_bytes(rows, f, dtype);
    if (!gradient) return each * (two_parts(rows, experts, dtype) ? 2 : 1);
    const int splits = weight_splits(rows, d, f, experts);
    return 3 * each + (splits > 1 ? splits * 3 * experts * d * f * static_cast<int64_t>(sizeof(float)) : 0);
}

extern "C" SPMV_API int spmv_feed_forward(int64_t rows, int64_t d, int64_t f, int32_t experts, const int32_t *offsets,
                                          const void *x, int64_t ldx, const void *w_gate, const void *w_up, int64_t ldw,
                                          int64_t w_expert, const void *w_down, int64_t ldwd, int64_t wd_expert,
                                          int activation, void *gate, void *up, int64_t ldg, void *y, int64_t ldy, int dtype,
                                          void *workspace, int64_t workspace_bytes, void *stream) {
    SPMV_TRY(check_sizes(rows, d, f, dtype));
    if (activation < SPMV_ACT_SILU || activation > SPMV_ACT_RELU) return refuse("activation is not one of spmv_activation");
    if (!gate != !up) return refuse("gate and up are kept both or not at all");
    SPMV_TRY(check_segments(experts, offsets));
    if (rows == 0) return SPMV_OK;
    const int64_t need = spmv_feed_forward_workspace(rows, d, f, experts, dtype, 0);
    if (workspace_bytes < need) return refuse("the workspace has fewer bytes than spmv_feed_forward_workspace says");
    SPMV_TRY(check_matrix(x, "x", rows, d, ldx, dtype));
    SPMV_TRY(check_weights(w_gate, "w_gate", experts, f, d, ldw, w_expert, dtype));
    SPMV_TRY(check_weights(w_up, "w_up", experts, f, d, ldw, w_expert, dtype));
    SPMV_TRY(check_weights(w_down, "w_down", experts, d, f, ldwd, wd_expert, dtype));
    if (gate) {
        SPMV_TRY(check_matrix(gate, "gate", rows, f, ldg, dtype));
        SPMV_TRY(check_matrix(up, "up", rows, f, ldg, dtype));
    }
    SPMV_TRY(check_matrix(y, "y", rows, d, ldy, dtype));
    SPMV_TRY(check_array(workspace, "workspace", 16));
    const int vb = row_value_bytes(dtype);
    const size_t w_bytes = weight_bytes(experts, f, d, ldw, w_expert, dtype);
    SPMV_TRY(check_outputs({{gate, span_bytes(rows, f, ldg, vb), "gate"}, {up, span_bytes(rows, f, ldg, vb), "up"},
                            {y, span_bytes(rows, d, ldy, vb), "y"}, {workspace, static_cast<size_t>(need), "workspace"}},
                           {{x, span_bytes(rows, d, ldx, vb), "x"}, {w_gate, w_bytes, "w_gate"}, {w_up, w_bytes, "w_up"},
                            {w_down, weight_bytes(experts, d, f, ldwd, wd_expert, dtype), "w_down"},
                            {offsets, static_cast<size_t>(experts + 1) * 4, "offsets"}}));
    Block b = {};
    b.seg = Segments{offsets, experts, rows};
    b.d = d;
    b.f = f;
    b.act = activation;
    b.x = matrix(x, ldx);
    b.wg = matrix(w_gate, ldw, w_expert);
    b.wu = matrix(w_up, ldw, w_expert);
    b.wd = matrix(w_down, ldwd, wd_expert);
    b.gate = matrix(gate, ldg);
    b.up = matrix(up, ldg);
    b.h = matrix(workspace, padded(f), rows * padded(f));
    if (two_parts(rows, experts, dtype)) b.h2 = matrix(static_cast<char *>(workspace) + need / 2, padded(f));
    b.y = matrix(y, ldy);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Launch run = tc_supported(b, dtype) ? launch_tc : launch_simt;
    SPMV_TRY(run(kGated, b, dtype, false, s));
    SPMV_TRY(run(kDown, b, dtype, true, s));
    return SPMV_OK;
}

extern "C" SPMV_API int spmv_feed_forward_grad(int64_t rows, int64_t d, int64_t f, int32_t experts, const int32_t *offsets,
                                               const void *x, int64_t ldx, const void *w_gate, const void *w_up, int64_t ldw,
                                               int64_t w_expert, const void *w_down, int64_t ldwd, int64_t wd_expert,
                                               int activation, const void *gate, const void *up, int64_t ldg, const void *dy,
                                               int64_t lddy, void *dx, int64_t lddx, void *dw_gate, void *dw_up, void *dw_down,
                                               int dtype, void *workspace, int64_t workspace_bytes, void *stream) {
    SPMV_TRY(check_sizes(rows, d, f, dtype));
    if (activation < SPMV_ACT_SILU || activation > SPMV_ACT_RELU) return refuse("activation is not one of spmv_activation");
    SPMV_TRY(check_segments(experts, offsets));
    const int64_t need = spmv_feed_forward_workspace(rows, d, f, experts, dtype, 1);
    if (workspace_bytes < need) return refuse("the workspace has fewer bytes than spmv_feed_forward_workspace says");
    SPMV_TRY(check_matrix(x, "x", rows, d, ldx, dtype));
    SPMV_TRY(check_weights(w_gate, "w_gate", experts, f, d, ldw, w_expert, dtype));
    SPMV_TRY(check_weights(w_up, "w_up", experts, f, d, ldw, w_expert, dtype));
    SPMV_TRY(check_weights(w_down, "w_down", experts, d, f, ldwd, wd_expert, dtype));
    SPMV_TRY(check_matrix(gate, "gate", rows, f, ldg, dtype));
    SPMV_TRY(check_matrix(up, "up", rows, f, ldg, dtype));
    SPMV_TRY(check_matrix(dy, "dy", rows, d, lddy, dtype));
    if (dx) SPMV_TRY(check_matrix(dx, "dx", rows, d, lddx, dtype));
    const struct { const void *p; const char *name; } grads[] = {{dw_gate, "dw_gate"}, {dw_up, "dw_up"}, {dw_down, "dw_down"}};
    for (const auto &g : grads)
        if (g.p) SPMV_TRY(check_array(g.p, g.name, row_value_bytes(dtype)));
    if (rows) SPMV_TRY(check_array(workspace, "workspace", 16));
    const int vb = row_value_bytes(dtype);
    const size_t w_bytes = weight_bytes(experts, f, d, ldw, w_expert, dtype), dw_bytes = static_cast<size_t>(experts) * f * d * vb;
    SPMV_TRY(check_outputs({{dx, dx ? span_bytes(rows, d, lddx, vb) : 0, "dx"}, {dw_gate, dw_bytes, "dw_gate"}, {dw_up, dw_bytes, "dw_up"},
                            {dw_down, dw_bytes, "dw_down"}, {workspace, static_cast<size_t>(need), "workspace"}},
                           {{x, span_bytes(rows, d, ldx, vb), "x"}, {w_gate, w_bytes, "w_gate"}, {w_up, w_bytes, "w_up"},
                            {w_down, weight_bytes(experts, d, f, ldwd, wd_expert, dtype), "w_down"},
                            {gate, span_bytes(rows, f, ldg, vb), "gate"}, {up, span_bytes(rows, f, ldg, vb), "up"},
                            {dy, span_bytes(rows, d, lddy, vb), "dy"}, {offsets, static_cast<size_t>(experts + 1) * 4, "offsets"}}));
    Block b = {};
    b.seg = Segments{offsets, experts, rows};
    b.d = d;
    b.f = f;
    b.act = activation;
    b.x = matrix(x, ldx);
    b.wg = matrix(w_gate, ldw, w_expert);
    b.wu = matrix(w_up, ldw, w_expert);
    b.wd = matrix(w_down, ldwd, wd_expert);
    b.gate = matrix(gate, ldg);
    b.up = matrix(up, ldg);
    b.dy = matrix(dy, lddy);
    char *space = static_cast<char *>(workspace);
    const int64_t each = rows_bytes(rows, f, dtype);
    b.dgate = matrix(space, padded(f));
    b.dup = matrix(space + each, padded(f));
    b.h = matrix(space + 2 * each, padded(f));
    b.splits = weight_splits(rows, d, f, experts);
    b.partial = reinterpret_cast<float *>(space + 3 * each);
    b.dx = matrix(dx, lddx);
    b.dwg = matrix(dw_gate, d, f * d);
    b.dwu = matrix(dw_up, d, f * d);
    b.dwd = matrix(dw_down, f, d * f);
    const bool weights = dw_gate || dw_up || dw_down;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // (no rows: the weights' gradients are 0, by the products that need no map of the rows)
    const Launch run = rows && tc_supported(b, dtype) ? launch_tc : launch_simt;
    if (rows && (dx || weights)) SPMV_TRY(run(kBack, b, dtype, false, s));
    if (rows && dx) SPMV_TRY(run(kInput, b, dtype, true, s));
    if (weights) SPMV_TRY(run(kWeights, b, dtype, rows > 0, s));
    if (weights && b.splits > 1) SPMV_TRY(launch_join(b, dtype, s));
    return SPMV_OK;
}
