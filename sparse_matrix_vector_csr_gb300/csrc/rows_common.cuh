// Shared device code of the sparse-row operators (topk.cu, route.cu, distill*.cu): value
// types of 16 and 32 bits, rows at any address read in 16-byte vectors, clusters of CTAs
// that share a row, and the argument checks of their entry points.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <string>
#include <utility>

#include "spmv_internal.cuh"

namespace spmv {
namespace rows {

constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxCluster = 8;  // portable cluster size

__host__ __device__ inline int row_value_bytes(int dtype) { return dtype == SPMV_F32 ? 4 : 2; }
inline bool row_dtype_ok(int dtype) { return dtype == SPMV_F32 || dtype == SPMV_F16 || dtype == SPMV_BF16; }

// ----------------------------------------------------------------------------
// value types
// ----------------------------------------------------------------------------
template <typename T>
struct Vec {
    static constexpr int kN = 16 / static_cast<int>(sizeof(T));  // values in 16 bytes
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The values of one 32-bit word (one float, two halves or two bfloat16s).
__device__ __forceinline__ void unpack_word(uint32_t w, float *out, float) { out[0] = __uint_as_float(w); }
__device__ __forceinline__ void unpack_word(uint32_t w, float *out, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    out[0] = f.x;
    out[1] = f.y;
}
__device__ __forceinline__ void unpack_word(uint32_t w, float *out, __nv_bfloat16) {
    out[0] = __uint_as_float(w << 16);
    out[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack_word(const float *in, float) { return __float_as_uint(in[0]); }
__device__ __forceinline__ uint32_t pack_word(const float *in, __half) {
    const __half2 h = __floats2half2_rn(in[0], in[1]);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_word(const float *in, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(in[0], in[1]);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T>
__device__ __forceinline__ void unpack(const uint4 &v, float *out) {
    constexpr int kW = Vec<T>::kN / 4;
    unpack_word(v.x, out, T());
    unpack_word(v.y, out + kW, T());
    unpack_word(v.z, out + 2 * kW, T());
    unpack_word(v.w, out + 3 * kW, T());
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float *in) {
    constexpr int kW = Vec<T>::kN / 4;
    return make_uint4(pack_word(in, T()), pack_word(in + kW, T()), pack_word(in + 2 * kW, T()),
                      pack_word(in + 3 * kW, T()));
}

template <typename T>
__device__ __forceinline__ uint4 splat(float v) {
    float f[Vec<T>::kN];
#pragma unroll
    for (int i = 0; i < Vec<T>::kN; ++i) f[i] = v;
    return pack<T>(f);
}
// The largest of a vector's values: a NaN is passed over, or (nan_max) is the result.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
template <typename H2>
__device__ __forceinline__ H2 as_pair(uint32_t w) { return *reinterpret_cast<const H2 *>(&w); }
// value by value
__device__ __forceinline__ uint4 vec_max2(const uint4 &a, const uint4 &b, float) {
    return make_uint4(__float_as_uint(fmaxf(__uint_as_float(a.x), __uint_as_float(b.x))),
                      __float_as_uint(fmaxf(__uint_as_float(a.y), __uint_as_float(b.y))),
                      __float_as_uint(fmaxf(__uint_as_float(a.z), __uint_as_float(b.z))),
                      __float_as_uint(fmaxf(__uint_as_float(a.w), __uint_as_float(b.w))));
}
template <typename H2>
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
    const H2 m = __hmax2(as_pair<H2>(a), as_pair<H2>(b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
__device__ __forceinline__ uint4 vec_max2(const uint4 &a, const uint4 &b, __half) {
    return make_uint4(pair_max<__half2>(a.x, b.x), pair_max<__half2>(a.y, b.y), pair_max<__half2>(a.z, b.z),
                      pair_max<__half2>(a.w, b.w));
}
__device__ __forceinline__ uint4 vec_max2(const uint4 &a, const uint4 &b, __nv_bfloat16) {
    return make_uint4(pair_max<__nv_bfloat162>(a.x, b.x), pair_max<__nv_bfloat162>(a.y, b.y),
                      pair_max<__nv_bfloat162>(a.z, b.z), pair_max<__nv_bfloat162>(a.w, b.w));
}
__device__ __forceinline__ float vec_max(const uint4 &v, float) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}
__device__ __forceinline__ float vec_max_nan(const uint4 &v, float) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
}
__device__ __forceinline__ float vec_max(const uint4 &v, __half) {
    const float2 f = __half22float2(__hmax2(__hmax2(as_pair<__half2>(v.x), as_pair<__half2>(v.y)),
                                            __hmax2(as_pair<__half2>(v.z), as_pair<__half2>(v.w))));
    return fmaxf(f.x, f.y);
}
__device__ __forceinline__ float vec_max_nan(const uint4 &v, __half) {
    const float2 f = __half22float2(__hmax2_nan(__hmax2_nan(as_pair<__half2>(v.x), as_pair<__half2>(v.y)),
                                                __hmax2_nan(as_pair<__half2>(v.z), as_pair<__half2>(v.w))));
    return max_nan(f.x, f.y);
}
__device__ __forceinline__ float vec_max(const uint4 &v, __nv_bfloat16) {
    const float2 f = __bfloat1622float2(__hmax2(__hmax2(as_pair<__nv_bfloat162>(v.x), as_pair<__nv_bfloat162>(v.y)),
                                                __hmax2(as_pair<__nv_bfloat162>(v.z), as_pair<__nv_bfloat162>(v.w))));
    return fmaxf(f.x, f.y);
}
__device__ __forceinline__ float vec_max_nan(const uint4 &v, __nv_bfloat16) {
    const float2 f =
        __bfloat1622float2(__hmax2_nan(__hmax2_nan(as_pair<__nv_bfloat162>(v.x), as_pair<__nv_bfloat162>(v.y)),
                                       __hmax2_nan(as_pair<__nv_bfloat162>(v.z), as_pair<__nv_bfloat162>(v.w))));
    return max_nan(f.x, f.y);
}

// The value a teacher array of any of the three types holds at i.
__device__ __forceinline__ float load_any(const void *p, int64_t i, int dtype) {
    if (dtype == SPMV_F32) return static_cast<const float *>(p)[i];
    if (dtype == SPMV_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// ----------------------------------------------------------------------------
// a row as 16-byte vectors
// ----------------------------------------------------------------------------
// A row may start at any multiple of its value size.  Vector v covers the values
// [v * N - head, v * N - head + N) of the row, head = the values between the 16-byte
// boundary at or below the row's start and the start, so every whole vector is aligned.
// The first and the last vector may reach over the row's ends: those go value by value
// and touch nothing outside the row.
template <typename T>
struct RowView {
    static constexpr int kN = Vec<T>::kN;
    const T *p;
    int64_t n;
    int head;
    __device__ __forceinline__ RowView(const T *row, int64_t n_values)
        : p(row), n(n_values), head(static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T))) {}
    __device__ __forceinline__ int64_t vectors() const { return (head + n + kN - 1) / kN; }
    __device__ __forceinline__ int64_t first(int64_t v) const { return v * kN - head; }
};
// The consecutive vectors of a row that one CTA has: `count` of them, of which [lo, hi) lie
// inside the row; only the row's own first and last vector can be others.
template <typename T>
struct Share {
    static constexpr int kN = Vec<T>::kN;
    const T *p;        // the row
    const uint4 *vec;  // its vector 0 of this share (which may begin in front of the row)
    int64_t n, e0;     // the row's length; the first value of vector 0 (negative in front of the row)
    int count, lo, hi;
    // the rank-th of 2^log2_ctas equal shares (the last may be shorter)
    __device__ __forceinline__ Share(const RowView<T> &row, uint32_t rank, int log2_ctas)
        : Share(row, static_cast<int64_t>(rank) * ((row.vectors() + (1 << log2_ctas) - 1) >> log2_ctas), (row.vectors() + (1 << log2_ctas) - 1) >> log2_ctas) {}
    // up to `per` vectors from v0 on
    __device__ __forceinline__ Share(const RowView<T> &row, int64_t v0, int64_t per) : p(row.p), n(row.n) {
        const int64_t nv = row.vectors();
        if (v0 > nv) v0 = nv;
        const int64_t v1 = v0 + per < nv ? v0 + per : nv;
        e0 = row.first(v0);
        vec = reinterpret_cast<const uint4 *>(p + e0);
        count = static_cast<int>(v1 - v0);
        lo = e0 < 0 ? 1 : 0;
        hi = e0 + static_cast<int64_t>(count) * kN > n ? count - 1 : count;
        if (lo > count) lo = count;
    }
    __device__ __forceinline__ bool whole(int v) const { return v >= lo && v < hi; }
    __device__ __forceinline__ int64_t first(int v) const { return e0 + static_cast<int64_t>(v) * kN; }
    __device__ __forceinline__ bool owns(int64_t e) const { return e >= e0 && e < first(count); }
    __device__ __forceinline__ uint4 load_whole(int v) const { return vec[v]; }
    __device__ __forceinline__ uint4 load_last(int v) const { return __ldcs(vec + v); }
    // any vector of the share; values outside the row read as -inf
    __device__ __forceinline__ uint4 load(int v) const {
        if (whole(v)) return load_whole(v);
        const int64_t e = first(v);
        float f[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) f[i] = (e + i >= 0 && e + i < n) ? to_f32(p[e + i]) : kNegInf;
        return pack<T>(f);
    }
    // one vector of a row of the same length; `congruent`: it starts at the same offset from
    // a 16-byte boundary as this one (otherwise values go one by one)
    __device__ __forceinline__ void store(T *row, int v, const uint4 &x, bool congruent) const {
        if (congruent && whole(v)) {
            __stcs(reinterpret_cast<uint4 *>(row + e0) + v, x);
        } else {
            const int64_t e = first(v);
            float f[kN];
            unpack<T>(x, f);
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (e + i >= 0 && e + i < n) row[e + i] = from_f32<T>(f[i]);
        }
    }
};

// Vectors t, t + workers, t + 2 workers, ... of the share, thread t's of `workers`, in
// registers: all loads are issued before the few threads with a vector at the row's ends look
// at theirs.  What is not there is -inf.
template <typename T, int kR>
__device__ __forceinline__ void load_share(const Share<T> &sh, int t, int workers, uint4 *reg) {
    const uint4 none = splat<T>(kNegInf);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        const int v = i * workers + t;
        reg[i] = none;
        if (sh.whole(v)) reg[i] = sh.load_whole(v);
    }
    if (sh.lo != 0 || sh.hi != sh.count) {
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            const int v = i * workers + t;
            if (v < sh.count && !sh.whole(v)) reg[i] = sh.load(v);
        }
    }
}
// the vectors at the row's ends, threads 0's and 1's (one vector may be both)
template <typename T, int kU, typename F>
__device__ __forceinline__ void stream_ends(const Share<T> &sh, int t, F f) {
    const bool first = t == 0 && sh.lo == 1 && sh.count > 0, last = t == 1 && sh.hi < sh.count && sh.hi >= sh.lo;
    if (first || last) {
        const int edge = first ? 0 : sh.hi;
        uint4 x[kU];
        const uint4 none = splat<T>(kNegInf);
#pragma unroll
        for (int i = 1; i < kU; ++i) x[i] = none;
        x[0] = sh.load(edge);
        f(x, edge, 1);
    }
}
// f(vectors[kU], index of the first, how many) over thread t's vectors, `workers` apart, read
// from memory kU at a time (those past the count are -inf), the vectors inside the row first.
// Rows that are read twice: the first kKeep whole batches go to slots of the thread's own in
// shared memory (kKeep * kU of them, `workers` apart) for stream_back.
template <typename T, int kU, bool kLast, int kKeep, typename F>
__device__ __forceinline__ void stream_share(const Share<T> &sh, int t, int workers, uint4 *keep, F f) {
    uint4 x[kU];
    const int step = kU * workers;
    int v = sh.lo + t;
    if constexpr (kKeep > 0) {
#pragma unroll 1
        for (int q = 0; q < kKeep && v + (kU - 1) * workers < sh.hi; ++q, v += step) {
#pragma unroll
            for (int i = 0; i < kU; ++i) x[i] = sh.load_whole(v + i * workers);
#pragma unroll
            for (int i = 0; i < kU; ++i) keep[(q * kU + i) * workers] = x[i];
            f(x, v, kU);
        }
    }
    for (; v + (kU - 1) * workers < sh.hi; v += step) {
#pragma unroll
        for (int i = 0; i < kU; ++i) x[i] = kLast ? sh.load_last(v + i * workers) : sh.load_whole(v + i * workers);
        f(x, v, kU);
    }
    const uint4 none = splat<T>(kNegInf);
    if (v < sh.hi) {
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            x[i] = none;
            if (v + i * workers < sh.hi) x[i] = sh.load_whole(v + i * workers);
        }
        f(x, v, (sh.hi - v + workers - 1) / workers);
    }
    stream_ends<T, kU>(sh, t, f);
}
// the same vectors from the end: what was read last is likeliest to be in L2 still, what was read
// first comes from the slots
template <typename T, int kU, int kKeep, typename F>
__device__ __forceinline__ void stream_back(const Share<T> &sh, int t, int workers, const uint4 *keep, F f) {
    uint4 x[kU];
    const int step = kU * workers, first = sh.lo + t;
    int v = first + (sh.hi > first ? (sh.hi - first - 1) / step * step : -step), q = (v - first) / step;  // the last batch
    const uint4 none = splat<T>(kNegInf);
    if (v >= first && v + (kU - 1) * workers >= sh.hi) {
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            x[i] = none;
            if (v + i * workers < sh.hi) x[i] = sh.load_whole(v + i * workers);
        }
        f(x, v, (sh.hi - v + workers - 1) / workers);
        v -= step;
        --q;
    }
#pragma unroll 1
    for (; q >= kKeep; --q, v -= step) {
#pragma unroll
        for (int i = 0; i < kU; ++i) x[i] = sh.load_last(v + i * workers);
        f(x, v, kU);
    }
#pragma unroll 1
    for (; q >= 0; --q, v -= step) {
#pragma unroll
        for (int i = 0; i < kU; ++i) x[i] = keep[(q * kU + i) * workers];
        f(x, v, kU);
    }
    stream_ends<T, kU>(sh, t, f);
}

// ----------------------------------------------------------------------------
// a row as units: the widest loads and stores that every row's address allows
// ----------------------------------------------------------------------------
template <int kBytes>
struct Unit;
template <>
struct Unit<16> { using type = uint4; };
template <>
struct Unit<8> { using type = uint2; };
template <>
struct Unit<4> { using type = uint32_t; };
template <>
struct Unit<2> { using type = uint16_t; };

// values of one unit of type T (kBytes >= sizeof(T)) as floats
template <typename T, typename U>
__device__ __forceinline__ void unit_to_f32(const U &u, float *out) {
    constexpr int kN = sizeof(U) / sizeof(T);
    const T *p = reinterpret_cast<const T *>(&u);
#pragma unroll
    for (int i = 0; i < kN; ++i) out[i] = to_f32(p[i]);
}
template <typename T, typename U>
__device__ __forceinline__ U unit_from_f32(const float *in) {
    constexpr int kN = sizeof(U) / sizeof(T);
    U u;
    T *p = reinterpret_cast<T *>(&u);
#pragma unroll
    for (int i = 0; i < kN; ++i) p[i] = from_f32<T>(in[i]);
    return u;
}

// ----------------------------------------------------------------------------
// arithmetic
// ----------------------------------------------------------------------------
// 2^x by the hardware unit: relative error about 2^-22, below the rounding of an argument of
// a few units in 32 bits; 0 for -inf, NaN for NaN.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two floats at a time: one instruction for both.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long &>(d))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long &>(d))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long &>(d))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)),
          "l"(reinterpret_cast<unsigned long long &>(c)));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// acc + the vector's exp2((x - m) scale): the difference first, so that values and maxima near
// the type's limits (masks) neither overflow nor meet an infinity of their own
template <typename T>
__device__ __forceinline__ float2 exp_sum(const uint4 &v, float m, float scale, float2 acc) {
    float x[Vec<T>::kN];
    unpack<T>(v, x);
#pragma unroll
    for (int i = 0; i < Vec<T>::kN; i += 2) {
        const float2 d = mul2(add2(make_float2(x[i], x[i + 1]), both(-m)), both(scale));
        acc = add2(acc, make_float2(ex2(d.x), ex2(d.y)));
    }
    return acc;
}
// Maximum and sum of exponentials of a thread's values, as they come.
struct Running {
    float m = kNegInf;
    float2 s = {0.0f, 0.0f};
    // kU vectors more
    template <typename T, int kU>
    __device__ __forceinline__ void add(const uint4 *x, float scale) {
        float top = vec_max(x[0], T());
#pragma unroll
        for (int i = 1; i < kU; ++i) top = fmaxf(top, vec_max(x[i], T()));
        add<T, kU>(x, top, scale);
    }
    // with their maximum at hand (a NaN where they have one: the sum becomes NaN whatever m is)
    template <typename T, int kU>
    __device__ __forceinline__ void add(const uint4 *x, float top, float scale) {
        if (top > m) {
            if (m != kNegInf) s = mul2(s, both(ex2((m - top) * scale)));
            m = top;
        }
        const float m0 = m == kNegInf ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < kU; ++i) s = exp_sum<T>(x[i], m0, scale, s);
    }
    __device__ __forceinline__ float sum() const { return s.x + s.y; }
};
// The reference point of a sum of exponentials: the maximum, or 0 if nothing is above -inf
// (so that -inf - m is -inf and never NaN).
__device__ __forceinline__ float reference_of(float m) { return m == kNegInf ? 0.0f : m; }
// The log of a row's sum of exponentials from its reference point and its sum relative to that; +inf
// where the row's largest value is (whose difference from itself makes the relative sum a NaN).
__device__ __forceinline__ float log_sum(float m, float sum, float inv_temperature) {
    return m == INFINITY ? INFINITY : fmaf(m, inv_temperature, logf(sum));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// Unsigned keys in the order of the numbers: -0 and +0 are equal, a NaN is above +inf.
__device__ __forceinline__ uint32_t order_key(float f) {
    if (f != f) return 0xff800001u;
    const uint32_t b = __float_as_uint(f + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// ----------------------------------------------------------------------------
// clusters
// ----------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// Address of the same shared variable in the CTA of rank `rank` of this cluster.
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void peer_store(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void peer_store2(uint32_t a, float x, float y) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void peer_store4(uint32_t a, float x, float y, float z, float w) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
__device__ __forceinline__ void peer_store64(uint32_t a, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t peer_load(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t peer_add(uint32_t a, uint32_t v) {
    uint32_t old;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(a), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Every thread of the cluster (of the CTA where it is alone) has arrived and its writes to
// shared memory are visible.
__device__ __forceinline__ void cluster_sync(int ctas) {
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------
// Launch `grid` CTAs of `threads` in clusters of `cluster` CTAs (grid a multiple of it).
template <typename... Params, typename... Args>
cudaError_t launch_rows(void (*kernel)(Params...), int64_t grid, int threads, int cluster, size_t smem, cudaStream_t s,
                        Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// 16-byte vectors that a row of n values reaches into, wherever the matrix's rows start.
template <typename T>
int64_t row_vectors(int64_t n, const void *p, int64_t ld) {
    const bool aligned = (reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(ld) * sizeof(T)) % 16 == 0;
    return ceil_div(n + (aligned ? 0 : Vec<T>::kN - 1), Vec<T>::kN);
}
// How a row of `vectors` 16-byte vectors is shared out: `ctas` CTAs (a cluster) of `threads`
// threads, one warp of each not taking part in the row itself; with `regs` vectors in registers
// each, or 0: read a batch at a time.
struct RowShape {
    int ctas, threads, regs;
    int log2_ctas() const { return ctas == 1 ? 0 : ctas == 2 ? 1 : ctas == 4 ? 2 : 3; }
};
constexpr int kRowRegs = 8;  // 32 registers of data
constexpr int kSms = 152;  // of this GPU
inline RowShape row_shape(int64_t rows, int64_t vectors, bool read_twice) {
    RowShape s{1, 512, 0};
    if (rows < kSms) {
        // few rows: more CTAs a row while SMs would be idle and each thread still has a vector;
        // in registers where they hold it, which is one reading and no loop
        while (s.ctas < kMaxCluster && rows * s.ctas < kSms && vectors > s.ctas * 480) s.ctas *= 2;
        if (vectors > s.ctas * 480 * kRowRegs) return s;
        const int64_t share = ceil_div(vectors, s.ctas);
        s.threads = share <= 192 ? 128 : share <= 896 ? 256 : 512;
        s.regs = 2;
        while (static_cast<int64_t>(s.regs) * (s.threads - 32) < share) s.regs *= 2;
        return s;
    }
    // Many rows: CTAs small enough to hide each other's barriers (3000 x 16000 bf16 values, loss
    // and gradient: 49 us with 128 threads, 54 with 256, 72 with 512; in registers, 288 threads:
    // 50), but large where the rows in flight would not stay in L2 for a second reading
    // (8192 x 131072 bf16 values: 950 us with 256, 761 with 512).  The rule looks at the row alone: from
    // 151 rows of 32000 bf16 values to 152, 8.1 us become 11.9 (loss and gradient; 304 rows 13.3, 1024 26.6).
    if (vectors <= 4096) {
        s.threads = 128;
    } else if (vectors <= 8192 || !read_twice) {
        s.threads = 256;
    } else {
        // two CTAs an SM: a few waves of long rows end evenly where a cluster takes each (400 x
        // 150000 float values: 125 us with one CTA a row, 99 with two)
        double best = 1e30;
        for (int c = 1; c <= 4; c *= 2) {
            const double waves = static_cast<double>(ceil_div(rows * c, 2 * kSms)) / c * (c == 1 ? 1.0 : c == 2 ? 1.05 : 1.15);
            if (waves < best && (c == 1 || vectors > c * 8192)) {
                best = waves;
                s.ctas = c;
            }
        }
    }
    return s;
}

inline int refuse(const std::string &what) { return set_error(SPMV_ERR_INVALID_ARG, what); }

// p is memory of the current device: device_memory_here's answer, in a fifth of its time where
// the process sees one device (rows_check.cu).
bool memory_here(const void *p);

// An array that a kernel reads or writes: there, aligned to its values and
// in the current device's memory.
inline int check_array(const void *p, const char *name, size_t align) {
    if (!p) return refuse(std::string(name) + " is NULL");
    if (reinterpret_cast<uintptr_t>(p) % align)
        return refuse(std::string(name) + " is not aligned to its " + std::to_string(align) + "-byte values");
    if (!memory_here(p))
        return refuse(std::string(name) + " is not device memory of the current device");
    return SPMV_OK;
}
// Bytes from the first to behind the last value of a rows x n matrix of leading dimension ld.
inline size_t span_bytes(int64_t rows, int64_t n, int64_t ld, int value_size) {
    return rows == 0 || n == 0 ? 0 : static_cast<size_t>((rows - 1) * ld + n) * static_cast<size_t>(value_size);
}
// rows, n in [0, 2^31) and ld >= n, with a span that 63 bits hold.
inline int check_shape(int64_t rows, int64_t n, int64_t ld, const char *name) {
    if (rows < 0 || n < 0 || rows >= (int64_t(1) << 31) || n >= (int64_t(1) << 31))
        return refuse(std::string(name) + ": the number of rows and their length must lie in [0, 2^31)");
    if (ld < n || ld >= (int64_t(1) << 31)) return refuse(std::string(name) + ": the leading dimension is below the row length or too large");
    return SPMV_OK;
}

// The widest unit (16, 8, 4 or 2 bytes, at least the value size) that every row of every
// array starts on and that divides a row's bytes.
inline int unit_bytes(int value_size, int64_t d, std::initializer_list<std::pair<const void *, int64_t>> arrays) {
    uint64_t bits = static_cast<uint64_t>(d) * value_size;
    for (const auto &a : arrays)
        bits |= reinterpret_cast<uintptr_t>(a.first) | static_cast<uint64_t>(a.second) * value_size;
    for (int b = 16; b > value_size; b /= 2)
        if (bits % b == 0) return b;
    return value_size;
}

inline int check_matrix(const void *p, const char *name, int64_t rows, int64_t d, int64_t ld, int dtype) {
    SPMV_TRY(check_shape(rows, d, ld, name));
    return rows && d ? check_array(p, name, row_value_bytes(dtype)) : SPMV_OK;
}

// An output shares no byte with an input (both matrices of rows, or plain arrays).
inline int check_apart(const void *out, size_t out_bytes, const char *out_name, const void *in, size_t in_bytes,
                const char *in_name) {
    if (out && in && out_bytes && in_bytes && spans_overlap(out, out_bytes, in, in_bytes))
        return refuse(std::string(out_name) + " overlaps " + in_name);
    return SPMV_OK;
}

#define SPMV_UNIT_SWITCH(bytes, CALL)      \
    switch (bytes) {                       \
        case 16: CALL(16); break;          \
        case 8: CALL(8); break;            \
        case 4: CALL(4); break;            \
        default: CALL(2); break;           \
    }

}  // namespace rows
}  // namespace spmv
