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
#include <string>

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
    __device__ __forceinline__ bool whole(int64_t e) const { return e >= 0 && e + kN <= n; }
    // values outside the row read as -inf
    __device__ __forceinline__ uint4 load(int64_t v) const {
        const int64_t e = first(v);
        if (whole(e)) return *reinterpret_cast<const uint4 *>(p + e);
        float f[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) f[i] = (e + i >= 0 && e + i < n) ? to_f32(p[e + i]) : kNegInf;
        return pack<T>(f);
    }
};
// Store one vector of a row whose geometry is that of `at` (same head) or not (`congruent`
// false: the row starts at another offset from a 16-byte boundary, values go one by one).
template <typename T>
__device__ __forceinline__ void store_vec(T *row, const RowView<T> &at, int64_t v, const float *f, bool congruent) {
    const int64_t e = at.first(v);
    if (congruent && at.whole(e)) {
        *reinterpret_cast<uint4 *>(row + e) = pack<T>(f);
    } else {
#pragma unroll
        for (int i = 0; i < Vec<T>::kN; ++i)
            if (e + i >= 0 && e + i < at.n) row[e + i] = from_f32<T>(f[i]);
    }
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
// The reference point of a sum of exponentials: the maximum, or 0 if nothing is above -inf
// (so that -inf - m is -inf and never NaN).
__device__ __forceinline__ float reference_of(float m) { return m == kNegInf ? 0.0f : m; }

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

inline int refuse(const std::string &what) { return set_error(SPMV_ERR_INVALID_ARG, what); }

// An array of `bytes` bytes that a kernel reads or writes: there, aligned to its values and
// in the current device's memory.
inline int check_array(const void *p, const char *name, size_t align) {
    if (!p) return refuse(std::string(name) + " is NULL");
    if (reinterpret_cast<uintptr_t>(p) % align)
        return refuse(std::string(name) + " is not aligned to its " + std::to_string(align) + "-byte values");
    if (!device_memory_here(p))
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

}  // namespace rows
}  // namespace spmv
