// The gated feed-forward block over segments of rows: shared declarations.
//
//   h = act(x Wg^T) * (x Wu^T),   y = h Wd^T          (Wg, Wu: f x d, Wd: d x f, one of each a segment)
//
// and back, with gate = x Wg^T and up = x Wu^T kept by the forward call:
//
//   dh = dy Wd,   dgate = dh * up * act'(gate),   dup = dh * act(gate),   h as above (not kept),
//   dx = dgate Wg + dup Wu,   dWg = dgate^T x,   dWu = dup^T x,   dWd = dy^T h    (sums over the segment's rows).
//
// Five kinds of product D[m][n] = sum over k of A[m][k] B[n][k], told apart by how they read A and B and
// by what is done with D.  Two implementations have the same kinds: products by the tensor cores
// (16-bit types whose matrices a tensor map can describe), and by the ordinary units (float, and
// 16-bit values at any address).
#pragma once

#include "device_util.cuh"
#include "rows_common.cuh"

namespace spmv {
namespace ffn {

using namespace rows;

enum Kind {
    kGated = 0,    // A = x, B = Wg and Wu side by side; D becomes h (and gate and up)
    kDown = 1,     // A = h, B = Wd; D becomes y
    kBack = 2,     // A = dy, B = Wd transposed; D = dh becomes dgate, dup and h
    kInput = 3,    // A = dgate, then dup; B = Wg, then Wu, transposed; D becomes dx
    kWeights = 4,  // A = dgate (dup; dy) and B = x (x; h), both transposed, sums over rows; D becomes dWg (dWu; dWd)
};
// how the operands lie: along k (false) or along m, n (true)
__host__ __device__ constexpr bool a_transposed(int kind) { return kind == kWeights; }
__host__ __device__ constexpr bool b_transposed(int kind) { return kind >= kBack; }

constexpr int kMaxSegments = 4096;
// Rows of a tile for segments that wait for their weights and not for products: 8 or 16, or 0 where they are longer.  A
// segment beyond the tile takes its weights through L2 once more, so that several are taken as up to twice their mean
// (32 experts of 8 rows on average, d = 2048, f = 1024: 81 us forward with tiles of 8 rows, 70 with tiles of 128).
constexpr int kShortRows = 16;
__host__ __device__ inline int short_rows(int64_t rows, int64_t segments) {
    const int64_t most = segments == 1 ? rows : 2 * ((rows + segments - 1) / segments);
    return most <= 8 ? 8 : most <= kShortRows ? kShortRows : 0;
}

// rows in segments; offsets == nullptr: one segment of all rows.  Whatever offsets holds, spans lie in [0, rows).
struct Segments {
    const int32_t *offsets;
    int32_t count;
    int64_t rows;
    struct Span {
        int64_t begin, end;
    };
    // segment e, or (e == count) the rows behind the last segment
    __device__ __forceinline__ Span span(int e) const {
        if (!offsets) return e == 0 ? Span{0, rows} : Span{rows, rows};
        const auto at = [&](int i) {
            const int64_t o = offsets[i];
            return o < 0 ? 0 : o > rows ? rows : o;
        };
        Span s{at(e), e == count ? rows : at(e + 1)};
        if (s.end < s.begin) s.end = s.begin;
        return s;
    }
};

// matrices of the call, strides in values
struct Matrix {
    void *p;
    int64_t ld;
    int64_t expert;  // from one segment's matrix to the next (weights)
};

// All operands of one call; a kind looks at its own.
struct Block {
    Segments seg;
    int64_t d, f;
    int act;
    Matrix x, wg, wu, wd;        // rows x d; experts x f x d; experts x d x f
    Matrix gate, up, h;          // rows x f (gate.p and up.p may be null forward)
    Matrix h2;                   // rows x f: what h's rounding left out (tensor cores, short segments)
    Matrix y;                    // rows x d
    Matrix dy, dgate, dup, dx;   // rows x d; rows x f; rows x d
    Matrix dwg, dwu, dwd;        // as wg, wu, wd (any may be null)
    // kWeights of few tiles and many rows: each segment's rows in `splits` parts, whose sums go to `partial`
    // (which product, segment, part, then its matrix) and are joined by k_join_weights
    int splits;
    float *partial;
    // segment e's rows of part `p`: multiples of 64 but for the last
    __device__ __forceinline__ Segments::Span part(int e, int p) const {
        Segments::Span s = seg.span(e);
        const int64_t each = ((s.end - s.begin + splits - 1) / splits + 63) / 64 * 64;
        s.begin = s.begin + p * each < s.end ? s.begin + p * each : s.end;
        if (s.begin + each < s.end) s.end = s.begin + each;
        return s;
    }
    __device__ __forceinline__ float *part_sums(int which, int e, int p) const {
        return partial + ((static_cast<int64_t>(which) * seg.count + e) * splits + p) * d * f;
    }
};

// ----------------------------------------------------------------------------
// activations
// ----------------------------------------------------------------------------
// s = 1 / (1 + exp(-x)) and 1 - s.  Float rows: both within 5 2^-23 of their value (the exponential of -|x| and the
// quotient within two units in the last place each; no difference is taken; a rounded division costs the products
// registers: 4096 rows, d = 2048, f = 4096, forward 5.55 ms instead of 5.32).  16-bit rows, whose type rounds far
// more and whose writing warps the instructions count in: s within about 2^-21 + |x| 2^-23 of its value (x log2(e) is
// rounded), 0 below -87.3, and 1 - s their difference.
struct Logistic {
    float s, rest;
};
template <typename T>
__device__ __forceinline__ Logistic logistic(float x) {
    if constexpr (sizeof(T) == 4) {
        const float e = expf(-fabsf(x)), large = __fdividef(1.0f, 1.0f + e), small = e * large;
        return x < 0.0f ? Logistic{small, large} : Logistic{large, small};
    } else {
        const float s = __fdividef(1.0f, 1.0f + ex2(-x * kLog2e));
        return {s, 1.0f - s};
    }
}
// act(x) and act'(x), for rows of type T.  gelu_tanh: x (1 + tanh z) / 2 = x / (1 + exp(-2z)), z = sqrt(2 / pi) (x + 0.044715 x^3); the
// rounding of 2z, 3 2^-23 of it, adds as much times |2z| to the error of float rows where 2z is below 0.
struct Activated {
    float value, slope;
};
template <typename T, bool kSlope>
__device__ __forceinline__ Activated activate(float x, int act) {
    if (act == SPMV_ACT_RELU) return {x < 0.0f ? 0.0f : x, x > 0.0f ? 1.0f : 0.0f};
    if (act == SPMV_ACT_SILU) {
        const Logistic l = logistic<T>(x);
        return {x * l.s, kSlope ? l.s * fmaf(x, l.rest, 1.0f) : 0.0f};
    }
    constexpr float kTwoRoot = 1.5957691216057308f, kCube = 0.044715f;  // 2 sqrt(2 / pi)
    const Logistic l = logistic<T>(kTwoRoot * x * fmaf(kCube * x, x, 1.0f));
    const float rest = x * l.s * l.rest;
    // (where s has reached 0 or 1 the rest of the slope is 0, however large its factor)
    return {x * l.s, kSlope ? (rest == 0.0f ? l.s : fmaf(rest, kTwoRoot * fmaf(3.0f * kCube * x, x, 1.0f), l.s)) : 0.0f};
}

// ----------------------------------------------------------------------------
// what becomes of a product
// ----------------------------------------------------------------------------
// kG consecutive values of row `p` (column 0 at p[0]), those below `left`; whole groups as one piece where
// the matrix's rows allow it.
template <typename T, int kG>
__device__ __forceinline__ void put(T *p, const float *v, int64_t left, bool whole) {
    if (whole && left >= kG) {
        constexpr int kBytes = kG * static_cast<int>(sizeof(T)) > 16 ? 16 : kG * static_cast<int>(sizeof(T));
        using U = typename Unit<kBytes>::type;
        constexpr int kEach = kBytes / static_cast<int>(sizeof(T));
#pragma unroll
        for (int i = 0; i < kG; i += kEach) *reinterpret_cast<U *>(p + i) = unit_from_f32<T, U>(v + i);
    } else {
#pragma unroll
        for (int i = 0; i < kG; ++i)
            if (i < left) p[i] = from_f32<T>(v[i]);
    }
}
template <typename T, int kG>
__device__ __forceinline__ void get(const T *p, float *v, int64_t left, bool whole) {
    if (whole && left >= kG) {
        constexpr int kBytes = kG * static_cast<int>(sizeof(T)) > 16 ? 16 : kG * static_cast<int>(sizeof(T));
        using U = typename Unit<kBytes>::type;
        constexpr int kEach = kBytes / static_cast<int>(sizeof(T));
#pragma unroll
        for (int i = 0; i < kG; i += kEach) unit_to_f32<T>(*reinterpret_cast<const U *>(p + i), v + i);
    } else {
#pragma unroll
        for (int i = 0; i < kG; ++i) v[i] = i < left ? to_f32(p[i]) : 0.0f;
    }
}

// kG values of D from column `col` of row `row` on (kGated: `v` is x Wg^T, `w` is x Wu^T); `whole`: rows of
// every matrix written or read start at multiples of the pieces' size.  kWeights: `which` of the three
// products, `e` its segment, `p` the part of its rows, `row` and `col` in the segment's matrix.
template <typename T, int kKind, int kG>
__device__ __forceinline__ void finish(const Block &b, int which, int e, int p, int64_t row, int64_t col, float *v, float *w,
                                       bool whole) {
    const auto at = [&](const Matrix &m) { return static_cast<T *>(m.p) + row * m.ld + col; };
    if constexpr (kKind == kGated) {
        const int64_t left = b.f - col;
        if (b.gate.p) {
            put<T, kG>(at(b.gate), v, left, whole);
            put<T, kG>(at(b.up), w, left, whole);
        }
#pragma unroll
        for (int i = 0; i < kG; ++i) v[i] = activate<T, false>(v[i], b.act).value * w[i];
        // rounded to the type: the next product takes it so (one rounding of each term of y's sums)
        put<T, kG>(at(b.h), v, left, whole);
    } else if constexpr (kKind == kDown) {
        put<T, kG>(at(b.y), v, b.d - col, whole);
    } else if constexpr (kKind == kBack) {
        const int64_t left = b.f - col;
        float g[kG], u[kG];
        get<T, kG>(at(b.gate), g, left, whole);
        get<T, kG>(at(b.up), u, left, whole);
#pragma unroll
        for (int i = 0; i < kG; ++i) {
            const Activated a = activate<T, true>(g[i], b.act);
            g[i] = v[i] * u[i] * a.slope;
            w[i] = v[i] * a.value;
            u[i] = a.value * u[i];
        }
        // each rounded once, to the type that the next products take
        put<T, kG>(at(b.dgate), g, left, whole);
        put<T, kG>(at(b.dup), w, left, whole);
        put<T, kG>(at(b.h), u, left, whole);
    } else if constexpr (kKind == kInput) {
        put<T, kG>(at(b.dx), v, b.d - col, whole);
    } else {
        const Matrix &m = which == 0 ? b.dwg : which == 1 ? b.dwu : b.dwd;
        const int64_t n = which == 2 ? b.f : b.d;
        if (b.splits > 1) put<float, kG>(b.part_sums(which, e, p) + row * n + col, v, n - col, n % 4 == 0);
        else put<T, kG>(static_cast<T *>(m.p) + e * m.expert + row * m.ld + col, v, n - col, whole);
    }
}
template <int kKind>
__host__ __device__ inline int64_t product_columns(const Block &b, int which) {
    if (kKind == kGated || kKind == kBack) return b.f;
    if (kKind == kDown || kKind == kInput) return b.d;
    return which == 2 ? b.f : b.d;
}
// rows of a kWeights product
__host__ __device__ inline int64_t weight_rows(const Block &b, int which) { return which == 2 ? b.d : b.f; }

// ----------------------------------------------------------------------------
// implementations
// ----------------------------------------------------------------------------
// `follows`: behind a kernel of the same call, on whose results it depends.
// ffn_simt.cu: any type and address
int launch_simt(int kind, const Block &b, int dtype, bool follows, cudaStream_t s);
// ffn_tc.cu: 16-bit values in rows that start at multiples of 16 bytes
bool tc_supported(const Block &b, int dtype);
int launch_tc(int kind, const Block &b, int dtype, bool follows, cudaStream_t s);
int launch_tc_f16(int kind, const Block &b, bool follows, cudaStream_t s);
int launch_tc_bf16(int kind, const Block &b, bool follows, cudaStream_t s);
// whether a wait of their kernels has run out since the last question
cudaError_t tc_flag_f16(int *value);
cudaError_t tc_flag_bf16(int *value);

}  // namespace ffn
}  // namespace spmv
