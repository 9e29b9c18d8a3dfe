// Entry points of the distillation loss (kernels: distill.cuh).
#include "distill.cuh"

namespace spmv {
namespace {

using namespace rows;

// One call in the form of spmv_distill_loss_grad; what a form does not use is NULL.
struct DistillCall {
    int64_t rows, vocab;
    int32_t k;
    const void *z;
    int64_t ldz;
    int dtype;
    const int32_t *ids;
    const void *teacher;
    int teacher_dtype;
    const float *teacher_lse;
    double temperature;
    float *loss;
    const float *stats;
    double scale;
    const float *row_scale;
    void *dz;
    int64_t lddz;
};

int distill(DistillMode mode, const DistillCall &c, void *stream) {
    SPMV_TRY(check_shape(c.rows, c.vocab, c.ldz, "z"));
    if (mode != kLoss) SPMV_TRY(check_shape(c.rows, c.vocab, c.lddz, "dz"));
    if (!row_dtype_ok(c.dtype) || !row_dtype_ok(c.teacher_dtype))
        return refuse("dtype and teacher_dtype must be SPMV_F32, SPMV_F16 or SPMV_BF16");
    if (c.k < 1 || c.k > kMaxEntries) return refuse("k must lie in [1, " + std::to_string(kMaxEntries) + "]");
    if (c.vocab < 1) return refuse("vocab must be at least 1");
    if (c.vocab > kMaxVocab) return set_error(SPMV_ERR_TOO_LARGE, "vocab must be at most 2^22");
    if (!(c.temperature >= 1e-6 && c.temperature <= 1e6)) return refuse("temperature must lie in [1e-6, 1e6]");
    if (mode != kLoss && !std::isfinite(c.scale)) return refuse("scale must be finite");
    if (c.rows == 0) return SPMV_OK;
    const int vb = row_value_bytes(c.dtype), tb = row_value_bytes(c.teacher_dtype);
    SPMV_TRY(check_array(c.z, "z", vb));
    SPMV_TRY(check_array(c.ids, "ids", 4));
    SPMV_TRY(check_array(c.teacher, "teacher", tb));
    if (c.teacher_lse) SPMV_TRY(check_array(c.teacher_lse, "teacher_lse", 4));
    if (mode != kGrad) SPMV_TRY(check_array(c.loss, "loss", 4));
    if (c.stats || mode == kGrad) SPMV_TRY(check_array(c.stats, "stats", 16));
    if (c.row_scale) SPMV_TRY(check_array(c.row_scale, "row_scale", 4));
    const size_t n = static_cast<size_t>(c.rows), m = n * c.k;
    const size_t zb = span_bytes(c.rows, c.vocab, c.ldz, vb);
    struct Span { const void *p; size_t bytes; const char *name; };
    const Span in[] = {{c.z, zb, "z"}, {c.ids, m * 4, "ids"}, {c.teacher, m * tb, "teacher"},
                       {c.teacher_lse, n * 4, "teacher_lse"}, {c.row_scale, n * 4, "row_scale"},
                       {mode == kGrad ? c.stats : nullptr, n * 16, "stats"}};
    Span out[] = {{mode != kGrad ? c.loss : nullptr, n * 4, "loss"}, {mode != kGrad ? c.stats : nullptr, n * 16, "stats"},
                  {nullptr, 0, "dz"}};
    if (mode != kLoss) {
        SPMV_TRY(check_array(c.dz, "dz", vb));
        out[2] = {c.dz, span_bytes(c.rows, c.vocab, c.lddz, vb), "dz"};
    }
    for (int o = 0; o < 3; ++o) {
        if (!out[o].p) continue;
        for (const Span &i : in) {
            if (!i.p || (o == 2 && i.p == c.z && c.dz == c.z && c.lddz == c.ldz)) continue;  // in place is fine
            if (spans_overlap(out[o].p, out[o].bytes, i.p, i.bytes))
                return refuse(std::string(out[o].name) + " overlaps " + i.name);
        }
        for (int q = 0; q < o; ++q)
            if (out[q].p && spans_overlap(out[o].p, out[o].bytes, out[q].p, out[q].bytes))
                return refuse(std::string(out[o].name) + " overlaps " + out[q].name);
    }
    DistillArgs a{};
    a.rows = c.rows;
    a.n = c.vocab;
    a.ldz = c.ldz;
    a.lddz = c.lddz;
    a.k = c.k;
    a.teacher_dtype = c.teacher_dtype;
    a.inv_temperature = static_cast<float>(1.0 / c.temperature);
    a.scale2 = static_cast<float>(1.4426950408889634 / c.temperature);
    a.scale = static_cast<float>(c.scale);
    a.z = c.z;
    a.ids = c.ids;
    a.teacher = c.teacher;
    a.teacher_lse = c.teacher_lse;
    a.row_scale = c.row_scale;
    a.loss = c.loss;
    a.stats = reinterpret_cast<float4 *>(const_cast<float *>(c.stats));
    a.dz = c.dz;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    SPMV_TRY_CUDA(c.dtype == SPMV_F32   ? launch_distill_f32(mode, a, s)
                  : c.dtype == SPMV_F16 ? launch_distill_f16(mode, a, s)
                                        : launch_distill_bf16(mode, a, s));
    return SPMV_OK;
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" SPMV_API int spmv_distill_loss(int64_t rows, int64_t vocab, int32_t k, const void *z, int64_t ldz, int dtype,
                                          const int32_t *ids, const void *teacher, int teacher_dtype,
                                          const float *teacher_lse, double temperature, float *loss, float *stats,
                                          void *stream) {
    return distill(rows::kLoss, {rows, vocab, k, z, ldz, dtype, ids, teacher, teacher_dtype, teacher_lse, temperature,
                                 loss, stats, 0.0, nullptr, nullptr, 0}, stream);
}

extern "C" SPMV_API int spmv_distill_grad(int64_t rows, int64_t vocab, int32_t k, const void *z, int64_t ldz, int dtype,
                                          const int32_t *ids, const void *teacher, int teacher_dtype,
                                          const float *teacher_lse, double temperature, const float *stats,
                                          double scale, const float *row_scale, void *dz, int64_t lddz, void *stream) {
    return distill(rows::kGrad, {rows, vocab, k, z, ldz, dtype, ids, teacher, teacher_dtype, teacher_lse, temperature,
                                 nullptr, stats, scale, row_scale, dz, lddz}, stream);
}

extern "C" SPMV_API int spmv_distill_loss_grad(int64_t rows, int64_t vocab, int32_t k, const void *z, int64_t ldz,
                                               int dtype, const int32_t *ids, const void *teacher, int teacher_dtype,
                                               const float *teacher_lse, double temperature, float *loss, double scale,
                                               const float *row_scale, void *dz, int64_t lddz, void *stream) {
    return distill(rows::kLossGrad, {rows, vocab, k, z, ldz, dtype, ids, teacher, teacher_dtype, teacher_lse,
                                     temperature, loss, nullptr, scale, row_scale, dz, lddz}, stream);
}
