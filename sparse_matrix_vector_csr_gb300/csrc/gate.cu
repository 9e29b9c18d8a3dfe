// A router's choice: the k <= 16 largest of short rows, with softmax weights, and the weights' gradient.
//
// Eight lanes share a row (with four, a fifth fewer instructions a row but half the warps: 32768 rows
// of 256 bf16 values, 8 chosen, with gradient, 20.8 us against 18.7).  Each sorts its values in blocks of kK
// (a sorting network on keys that hold the value's order and its column, so that no two are equal and ties
// go to the lowest column) and merges the blocks, keeping the kK
// largest; exchanges with the lanes 1, 2 and 4 away merge the lanes' lists.  Every operation is a
// minimum or maximum on registers that four rows a warp share: rounds of "largest of
// the warp" cost five times as many instructions a row (256 bf16 values, 8 of them: 780).  The
// row is read once, its sum of exponentials taken along.
#include "topk.cuh"

namespace spmv {
namespace rows {
namespace {

constexpr int kThreads = 128;
constexpr int kLanes = 8;  // per row

// Keys in the order of (value, lower column first): the value's order above the complement of its
// column, so 0 (no value) is below all.  Adding +0 makes one zero of both and the one positive NaN
// of any (above +inf), so nothing but 0 orders below -inf, which is dropped at the end.
template <typename T>
struct Key;
template <>
struct Key<float> {
    using type = unsigned long long;
    static constexpr uint32_t kNone = 0x007fffffu;  // order of -inf
    // the keys of a vector whose first value has column col
    static __device__ __forceinline__ void make(const uint4 &v, int col, type *k) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t b = __float_as_uint(__uint_as_float(w[i]) + 0.0f);
            const uint32_t o = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
            k[i] = static_cast<unsigned long long>(o) << 32 | (0xffffffffu - static_cast<uint32_t>(col + i));
        }
    }
    static __device__ __forceinline__ bool some(type k) { return static_cast<uint32_t>(k >> 32) > kNone; }
    static __device__ __forceinline__ float value(type k) { return some(k) ? key_value(static_cast<uint32_t>(k >> 32)) : kNegInf; }
    static __device__ __forceinline__ int col(type k) { return some(k) ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)) : -1; }
};
// 16-bit values: order in the upper half, kFirst - column in the lower (the vector at a row's
// start may begin up to 7 columns in front of it, and no half may borrow from the other).
template <typename T, typename T2, uint32_t kInfBits>
struct Key16 {
    using type = uint32_t;
    static constexpr int kFirst = 0xffff - 8;
    static __device__ __forceinline__ void make(const uint4 &v, int col, type *k) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        // two columns' complements in a word; the next two are 2 lower in each half
        uint32_t c = static_cast<uint32_t>(kFirst - col) | static_cast<uint32_t>(kFirst - col - 1) << 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const T2 h = __hadd2(as_pair<T2>(w[i]), as_pair<T2>(0u));
            const uint32_t b = *reinterpret_cast<const uint32_t *>(&h);
            const uint32_t o = b ^ ((b >> 15 & 0x00010001u) * 0xffffu | 0x80008000u);
            k[2 * i] = __byte_perm(o, c, 0x1054);
            k[2 * i + 1] = __byte_perm(o, c, 0x3276);
            c -= 0x00020002u;
        }
    }
    static __device__ __forceinline__ bool some(type k) { return k >> 16 > 0x7fffu - kInfBits; }
    static __device__ __forceinline__ float value(type k) {
        const uint32_t o = k >> 16;
        const uint16_t b = static_cast<uint16_t>(o & 0x8000u ? o ^ 0x8000u : ~o);
        return some(k) ? to_f32(*reinterpret_cast<const T *>(&b)) : kNegInf;
    }
    static __device__ __forceinline__ int col(type k) { return some(k) ? kFirst - static_cast<int>(k & 0xffffu) : -1; }
};
template <>
struct Key<__half> : Key16<__half, __half2, 0x7c00u> {};
template <>
struct Key<__nv_bfloat16> : Key16<__nv_bfloat16, __nv_bfloat162, 0x7f80u> {};

template <typename K>
__device__ __forceinline__ void order_pair(K &a, K &b) {  // a >= b
    const K hi = a > b ? a : b, lo = a > b ? b : a;
    a = hi;
    b = lo;
}
// a bitonic sequence to descending order
template <int kK, typename K>
__device__ __forceinline__ void merge_down(K *x) {
#pragma unroll
    for (int d = kK / 2; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < kK; ++i)
            if ((i & d) == 0) order_pair(x[i], x[i + d]);
}
// Batcher's odd-even merge sort: 5, 19, 63 pairs for 4, 8, 16 values
template <int kK, typename K>
__device__ __forceinline__ void sort_down(K *x) {
#pragma unroll
    for (int p = 1; p < kK; p *= 2)
#pragma unroll
        for (int k = p; k > 0; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < kK; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < kK && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order_pair(x[i + j], x[i + j + k]);
}
// the kK largest of two descending lists, descending
template <int kK, typename K>
__device__ __forceinline__ void keep_largest(K *x, const K *y) {
#pragma unroll
    for (int i = 0; i < kK; ++i) x[i] = x[i] > y[kK - 1 - i] ? x[i] : y[kK - 1 - i];
    merge_down<kK>(x);
}

template <typename V>
__device__ __forceinline__ V from_lane_away(V v, int d) { return __shfl_xor_sync(0xffffffffu, v, d); }

// kV vectors a lane at a time, lists of kK.
template <typename T, int kV, int kK>
__global__ void __launch_bounds__(kThreads) k_gate(TopArgs a) {
    using K = typename Key<T>::type;
    constexpr int kN = Vec<T>::kN;
    const int lane = threadIdx.x & (kLanes - 1);
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
    const bool there = r < a.rows;  // lanes of no row go along with the exchanges
    const RowView<T> row(static_cast<const T *>(a.x) + (there ? r : 0) * a.ldx, there ? a.n : 0);
    const Share<T> share(row, uint32_t(0), 0);
    const bool whole_row = a.lse || a.weighting == SPMV_WEIGHTS_ROW;
    K best[kK];
    Running run;
    constexpr int kValues = kV * kN, kBlocks = (kValues + kK - 1) / kK;
    for (int v0 = 0; v0 == 0 || v0 < share.count; v0 += kV * kLanes) {
        uint4 vec[kV];
        load_share<T, kV>(share, v0 + lane, kLanes, vec);
        K key[kBlocks * kK];
#pragma unroll
        for (int i = 0; i < kV; ++i)  // (what is not there is -inf, whatever column it says)
            Key<T>::make(vec[i], static_cast<int>(share.first(v0 + i * kLanes + lane)), key + i * kN);
#pragma unroll
        for (int i = kValues; i < kBlocks * kK; ++i) key[i] = 0;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            sort_down<kK>(key + b * kK);
            if (b > 0) keep_largest<kK>(key, key + b * kK);
        }
        if (v0 == 0) {
#pragma unroll
            for (int i = 0; i < kK; ++i) best[i] = key[i];
        } else {
            keep_largest<kK>(best, key);
        }
        if (whole_row) run.add<T, kV>(vec, Key<T>::value(key[0]), a.scale);
    }
    float m_lane = run.m, sum = run.sum();
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) {
        K other[kK];
#pragma unroll
        for (int i = 0; i < kK; ++i) other[i] = from_lane_away(best[i], d);
        keep_largest<kK>(best, other);
    }
    const float m = reference_of(Key<T>::value(best[0]));
    if (whole_row) {
        if (m_lane != kNegInf) sum *= ex2((m_lane - m) * a.scale);
#pragma unroll
        for (int d = 1; d < kLanes; d *= 2) sum += from_lane_away(sum, d);
        if (a.lse && lane == 0 && there) a.lse[r] = Key<T>::some(best[0]) ? log_sum(m, sum, a.inv_temperature) : kNegInf;
    }
    // entries lane, lane + kLanes, ... of the row are this lane's
    constexpr int kMine = (kK + kLanes - 1) / kLanes;
    float e[kMine], chosen = 0.0f;
    K mine[kMine];
#pragma unroll
    for (int t = 0; t < kMine; ++t) {
        mine[t] = 0;
#pragma unroll
        for (int i = 0; i < kLanes && t * kLanes + i < kK; ++i)
            if (lane == i && t * kLanes + i < a.k) mine[t] = best[t * kLanes + i];
        e[t] = Key<T>::some(mine[t]) ? ex2((Key<T>::value(mine[t]) - m) * a.scale) : 0.0f;
        chosen += e[t];
    }
    if (a.weighting == SPMV_WEIGHTS_SELECTED) {
#pragma unroll
        for (int d = 1; d < kLanes; d *= 2) chosen += from_lane_away(chosen, d);
        sum = chosen;
    }
    if (!there) return;
#pragma unroll
    for (int t = 0; t < kMine; ++t) {
        const int j = t * kLanes + lane;
        if (j < a.k) {
            a.ids[r * a.k + j] = Key<T>::col(mine[t]);
            if (a.vals) a.vals[r * a.k + j] = Key<T>::value(mine[t]);
            if (a.weighting != SPMV_WEIGHTS_NONE) a.weights[r * a.k + j] = Key<T>::some(mine[t]) ? e[t] / sum : 0.0f;
        }
    }
}

// The gradient (see topk.cu for the formulas): the lanes write a row's vectors, then, after
// __syncwarp has ordered the stores, its chosen columns.  8 of 256 for 32768 bf16 rows, over the row: 5.5 us
// one after the other, 9.3 with cold caches, bound by the latency of its loads.
template <typename T, int kV>
__global__ void __launch_bounds__(kThreads) k_gate_grad(TopGradArgs a) {
    constexpr int kN = Vec<T>::kN;
    const int lane = threadIdx.x & (kLanes - 1);
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
    const bool there = r < a.rows, whole_row = a.weighting == SPMV_WEIGHTS_ROW;
    T *out = static_cast<T *>(a.dx) + (there ? r : 0) * a.lddx;
    const T *x = whole_row ? static_cast<const T *>(a.x) + (there ? r : 0) * a.ldx : out;
    const Share<T> share(RowView<T>(x, there ? a.n : 0), uint32_t(0), 0);  // x's vectors, or without it dx's
    const bool congruent = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
    uint4 vec[kV];
    if (whole_row) load_share<T, kV>(share, lane, kLanes, vec);
    constexpr int kMine = kGateMaxK / kLanes;
    int32_t id[kMine];
    float w[kMine], dw[kMine], s = 0.0f;
#pragma unroll
    for (int t = 0; t < kMine; ++t) {
        const int j = t * kLanes + lane;
        id[t] = -1;
        w[t] = dw[t] = 0.0f;
        if (there && j < a.k) {
            id[t] = a.ids[r * a.k + j];
            w[t] = a.weights[r * a.k + j];
            dw[t] = a.dweights[r * a.k + j];
            if (id[t] >= a.n) id[t] = -1;  // outside: no entry
            if (id[t] >= 0) s = fmaf(w[t], dw[t], s);
        }
    }
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) s += from_lane_away(s, d);
    // (a row without entries has nothing above -inf: 0 everywhere)
    const int32_t first = __shfl_sync(0xffffffffu, id[0], 0, kLanes);
    const float w0 = __shfl_sync(0xffffffffu, w[0], 0, kLanes);
    const bool some = whole_row && first >= 0;
    const RowShare q{some ? to_f32(x[first]) : 0.0f, some ? w0 * (-s * a.inv_temperature) : 0.0f,
                     a.inv_temperature * kLog2e};
    for (int v0 = 0; v0 < share.count; v0 += kV * kLanes) {
        if (v0 && whole_row) load_share<T, kV>(share, v0 + lane, kLanes, vec);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int v = v0 + i * kLanes + lane;
            if (v < share.count) {
                uint4 o = splat<T>(0.0f);
                if (some) {
                    float f[kN];
                    unpack<T>(vec[i], f);
#pragma unroll
                    for (int j = 0; j < kN; j += 2) {
                        float2 d = mul2(add2(make_float2(f[j], f[j + 1]), both(-q.x0)), both(q.scale));
                        d = mul2(make_float2(ex2(d.x), ex2(d.y)), both(q.w0));
                        f[j] = d.x;
                        f[j + 1] = d.y;
                    }
                    o = pack<T>(f);
                }
                share.store(out, v, o, congruent);
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < kMine; ++t)
        if (id[t] >= 0) out[id[t]] = from_f32<T>(w[t] * (dw[t] - s) * a.inv_temperature);
}

template <typename T, int kV>
cudaError_t launch(const TopArgs &a, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(ceil_div(a.rows, kThreads / kLanes));
    if (a.k <= 4) k_gate<T, kV, 4><<<grid, kThreads, 0, s>>>(a);
    else if (a.k <= 8) k_gate<T, kV, 8><<<grid, kThreads, 0, s>>>(a);
    else k_gate<T, kV, 16><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int kV>
cudaError_t launch(const TopGradArgs &a, cudaStream_t s) {
    k_gate_grad<T, kV><<<static_cast<unsigned>(ceil_div(a.rows, kThreads / kLanes)), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// by the vectors that a row of the matrix p may reach into
template <typename T, typename Args>
cudaError_t launch_by_vectors(const Args &a, const void *p, int64_t ld, cudaStream_t s) {
    const int64_t vectors = row_vectors<T>(a.n, p, ld);
    if (vectors <= kLanes) return launch<T, 1>(a, s);
    if (vectors <= 2 * kLanes) return launch<T, 2>(a, s);
    return launch<T, 4>(a, s);
}

template <typename Args>
cudaError_t launch_by_type(const Args &a, int dtype, const void *p, int64_t ld, cudaStream_t s) {
    if (dtype == SPMV_F32) return launch_by_vectors<float>(a, p, ld, s);
    if (dtype == SPMV_F16) return launch_by_vectors<__half>(a, p, ld, s);
    return launch_by_vectors<__nv_bfloat16>(a, p, ld, s);
}

}  // namespace

cudaError_t launch_gate(const TopArgs &a, int dtype, cudaStream_t s) { return launch_by_type(a, dtype, a.x, a.ldx, s); }

cudaError_t launch_gate_grad(const TopGradArgs &a, int dtype, cudaStream_t s) {
    const bool whole_row = a.weighting == SPMV_WEIGHTS_ROW;
    return launch_by_type(a, dtype, whole_row ? a.x : a.dx, whole_row ? a.ldx : a.lddx, s);
}

}  // namespace rows
}  // namespace spmv
