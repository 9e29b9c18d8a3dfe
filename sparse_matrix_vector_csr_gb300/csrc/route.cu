// Rows sorted by expert and back.  The routing of `tokens` tokens to k of E experts each is a
// sparse tokens x E matrix R with k entries a row; a plan is its transposed order (a stable
// counting sort by column), dispatch is the product of the transposed pattern with a dense
// matrix of rows, combine the product of the weighted matrix with the experts' rows, and the
// gradient of combine is the transposed product together with the sampled products
// <dy[t], ys[slot]> that are the gradient of R's values.  Every kernel is bound by its rows'
// bytes, so each row is read once and written once, tokens first: a token's row sits in
// registers while its k sorted copies are written (or its k sorted rows are summed).
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "device_util.cuh"
#include "rows_common.cuh"

namespace spmv {
namespace {

using namespace rows;

constexpr int kPlanThreads = 512;
constexpr int kMaxExperts = 4096;
constexpr int64_t kPlanChunk = 1024;  // entries per CTA of the plan, at least
constexpr int64_t kPlanCtas = 128;    // CTAs of the plan, at most
constexpr int kPlanSmem = 128 * 1024; // limit of its shared memory (4096 experts: 96 KB)

struct PlanShape {
    int64_t entries, chunk;
    int ctas, warps;  // warps that rank entries: their counters share the CTA's memory
    size_t smem;
};

PlanShape plan_shape(int64_t tokens, int32_t k, int32_t experts) {
    PlanShape p;
    p.entries = tokens * k;
    p.chunk = kPlanChunk;
    if (ceil_div(p.entries, p.chunk) > kPlanCtas) p.chunk = ceil_div(p.entries, kPlanCtas);
    p.ctas = static_cast<int>(ceil_div(p.entries, p.chunk));
    if (p.ctas < 1) p.ctas = 1;
    p.warps = kPlanThreads / 32;
    const int64_t most = p.entries < p.chunk ? p.entries : p.chunk;
    while (p.warps > 1 && p.warps * 16 >= most) p.warps /= 2;  // no more than there are 32s of entries
    while (p.warps > 1 && static_cast<int64_t>(p.warps) * experts > 16384) p.warps /= 2;
    // all of it dynamic, the scan's partial sums too, so that p.smem is what the default limit is held against
    p.smem = (static_cast<size_t>(p.warps + 2) * static_cast<size_t>(experts) + kPlanThreads / 32) * sizeof(int32_t);
    return p;
}

__device__ __forceinline__ int32_t expert_of(const int32_t *ids, int64_t i, int32_t experts) {
    const int32_t e = ids[i];
    return static_cast<uint32_t>(e) < static_cast<uint32_t>(experts) ? e : -1;
}

// hist[e * CTAs + b] = entries of expert e in CTA b's share
__global__ void __launch_bounds__(kPlanThreads) k_route_hist(int64_t entries, int64_t chunk, int32_t experts,
                                                            const int32_t *__restrict__ ids, int32_t *__restrict__ hist) {
    extern __shared__ int32_t count[];
    for (int e = threadIdx.x; e < experts; e += kPlanThreads) count[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * chunk, end = begin + chunk < entries ? begin + chunk : entries;
    for (int64_t i = begin + threadIdx.x; i < end; i += kPlanThreads) {
        const int32_t e = expert_of(ids, i, experts);
        if (e >= 0) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kPlanThreads)
        hist[static_cast<int64_t>(e) * gridDim.x + blockIdx.x] = count[e];
    dev::allow_dependents();
}

// Every CTA takes its share of the entries in order, each of its ranking warps a run of
// consecutive ones, so the sort is stable: an entry's place is its expert's start, plus the
// expert's entries in earlier CTAs, in earlier warps of the CTA, and earlier in the warp
// (by match_any).  The integer counters make the order independent of timing.
// hist: the counts of every CTA, or nullptr when one CTA does it all.  Latency bound: 131072 entries
// of 128 experts 12 us with k_route_hist, 32 entries 6 us in one CTA.
__global__ void __launch_bounds__(kPlanThreads) k_route_place(int64_t entries, int64_t chunk, int32_t experts,
                                                             int32_t align, int64_t rows, int n_warps,
                                                             const int32_t *__restrict__ ids,
                                                             const int32_t *__restrict__ hist,
                                                             int32_t *__restrict__ offsets, int32_t *__restrict__ slots,
                                                             int32_t *__restrict__ sources) {
    extern __shared__ int32_t shared[];
    int32_t *wcount = shared;                       // [n_warps][experts]: counts, then next places
    int32_t *total = wcount + n_warps * experts;    // [experts]
    int32_t *start = total + experts;               // [experts]: first row of the expert's segment
    int32_t *warp_part = start + experts;           // [kPlanThreads / 32]: the scan's, one a warp
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t begin = blockIdx.x * chunk, end = begin + chunk < entries ? begin + chunk : entries;
    // runs of whole 32s
    const int64_t run = ((end > begin ? end - begin : 0) + 32 * n_warps - 1) / (32 * n_warps) * 32;
    const int64_t r0 = begin + warp * run, r1 = r0 + run < end ? r0 + run : end;

    for (int i = tid; i < n_warps * experts; i += kPlanThreads) wcount[i] = 0;
    __syncthreads();
    if (warp < n_warps)
        for (int64_t i = r0 + lane; i < r1; i += 32) {
            const int32_t e = expert_of(ids, i, experts);
            if (e >= 0) atomicAdd(&wcount[warp * experts + e], 1);
        }
    __syncthreads();

    // per expert: entries in all and in earlier CTAs (a warp per expert, at most four counts a
    // lane); then the warps' counts become places relative to the expert's segment
    if (hist) {
        dev::grid_wait();
        for (int e = warp; e < experts; e += kPlanThreads / 32) {
            int32_t before = 0, sum = 0;
#pragma unroll
            for (int i = 0; i < kPlanCtas / 32; ++i) {
                const int b = i * 32 + lane;
                const int32_t c = b < gridDim.x ? hist[static_cast<int64_t>(e) * gridDim.x + b] : 0;
                before += b < blockIdx.x ? c : 0;
                sum += c;
            }
            before = warp_sum(before);
            sum = warp_sum(sum);
            if (lane == 0) {
                start[e] = before;
                total[e] = sum;
            }
        }
        __syncthreads();
    }
    for (int e = tid; e < experts; e += kPlanThreads) {
        int32_t at = hist ? start[e] : 0;
        for (int w = 0; w < n_warps; ++w) {
            const int32_t c = wcount[w * experts + e];
            wcount[w * experts + e] = at;
            at += c;
        }
        if (!hist) total[e] = at;
    }
    __syncthreads();

    // exclusive scan of the padded segment lengths (unsigned: a padded length is below 2^31, a length
    // plus align - 1 need not be)
    const auto padded = [&](int e) {
        const uint32_t tile = static_cast<uint32_t>(align);
        return static_cast<int32_t>((static_cast<uint32_t>(total[e]) + tile - 1) / tile * tile);
    };
    const int per = (experts + kPlanThreads - 1) / kPlanThreads;
    int32_t mine = 0;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e < experts) mine += padded(e);
    }
    int32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_part[warp] = incl;
    __syncthreads();
    int32_t at = incl - mine;
    for (int w = 0; w < warp; ++w) at += warp_part[w];
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e < experts) {
            start[e] = at;
            if (blockIdx.x == 0) offsets[e] = at;
            at += padded(e);
            if (blockIdx.x == 0 && e == experts - 1) offsets[experts] = at;
        }
    }
    __syncthreads();
    int32_t used = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) used += warp_part[w];

    // padding rows have no source
    const int n_cta = gridDim.x;
    for (int e = blockIdx.x * (kPlanThreads / 32) + warp; e < experts; e += n_cta * (kPlanThreads / 32)) {
        const int64_t a = static_cast<int64_t>(start[e]) + total[e];
        const int64_t b = static_cast<int64_t>(start[e]) + padded(e);
        for (int64_t s = a + lane; s < b; s += 32) sources[s] = -1;
    }
    for (int64_t s = used + static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid; s < rows;
         s += static_cast<int64_t>(n_cta) * kPlanThreads)
        sources[s] = -1;

    if (warp < n_warps)
        for (int64_t i0 = r0; i0 < r1; i0 += 32) {
            const int64_t i = i0 + lane;
            const int32_t e = i < r1 ? expert_of(ids, i, experts) : -1;
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            const int rank = __popc(same & ((1u << lane) - 1));
            int32_t *next = &wcount[warp * experts + (e >= 0 ? e : 0)];
            const int32_t place = e >= 0 ? start[e] + *next + rank : -1;
            __syncwarp();
            if (e >= 0 && rank == 0) *next += __popc(same);
            __syncwarp();
            if (i < r1) {
                slots[i] = place;
                if (e >= 0) sources[place] = static_cast<int32_t>(i);
            }
        }
}

// ----------------------------------------------------------------------------
// rows out and back
// ----------------------------------------------------------------------------

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

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

// Zero the sorted rows without a source among 32 that the CTA looks at: padding comes in runs
// (behind each segment, and behind the last), so the CTA's warps take turns.
constexpr int kPadRows = 32;  // per CTA
template <typename U>
__device__ void zero_padding(int64_t first, int64_t rows, const int32_t *sources, int64_t units, U *out, int64_t ld) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
    const uint32_t pad = __ballot_sync(0xffffffffu, first + lane < rows && sources[first + lane] < 0);
    for (int i = warp; i < 32; i += n_warps)
        if (pad >> i & 1) {
            U *row = out + (first + i) * ld;
            for (int64_t u = lane; u < units; u += 32) row[u] = U{};
        }
}
// A token's entries 32 at a time, a lane each: sorted row (-1: none) and weight.
struct Entries {
    int32_t slot;
    float weight;
    __device__ __forceinline__ Entries(int64_t t, int k, int j0, int64_t rows, const int32_t *slots, const float *weights) {
        const int j = j0 + (threadIdx.x & 31);
        slot = j < k ? slots[t * k + j] : -1;
        if (slot >= rows) slot = -1;
        weight = weights && slot >= 0 ? weights[t * k + j] : 1.0f;
    }
    __device__ __forceinline__ int32_t row(int j) const { return __shfl_sync(0xffffffffu, slot, j); }
    __device__ __forceinline__ float of(int j) const { return __shfl_sync(0xffffffffu, weight, j); }
};

// 16384 tokens x 8 of 4096 bf16 values, segments of 128: 200 us, 6.7 TB/s (DRAM's writes).
// xs[slots[t, j]] = x[t] for every entry; xs[s] = 0 for rows without a source.  A warp
// takes kU x 32 units of one token's row (units: the widest loads that the alignment of
// every row allows); the first CTAs zero the padding.
template <typename U, int kU>
__global__ void __launch_bounds__(kRowThreads) k_dispatch(int64_t tokens, int k, int64_t rows, int64_t units,
                                                         int64_t parts, int64_t pad_ctas,
                                                         const int32_t *__restrict__ slots,
                                                         const int32_t *__restrict__ sources, const U *__restrict__ x,
                                                         int64_t ldx, U *__restrict__ xs, int64_t ldxs) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x < pad_ctas) {
        zero_padding(static_cast<int64_t>(blockIdx.x) * kPadRows, rows, sources, units, xs, ldxs);
        return;
    }
    const int64_t item = (blockIdx.x - pad_ctas) * kRowWarps + warp;
    const int64_t t = item / parts;
    if (t >= tokens) return;
    const int64_t u0 = (item - t * parts) * (32 * kU) + lane;
    const U *src = x + t * ldx;
    U v[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i)
        if (u0 + i * 32 < units) v[i] = src[u0 + i * 32];
    for (int j0 = 0; j0 < k; j0 += 32) {
        const Entries entries(t, k, j0, rows, slots, nullptr);
        const int n = min(k - j0, 32);
        for (int j = 0; j < n; ++j) {
            const int64_t s = entries.row(j);
            if (s < 0) continue;
            U *dst = xs + s * ldxs;
#pragma unroll
            for (int i = 0; i < kU; ++i)
                if (u0 + i * 32 < units) dst[u0 + i * 32] = v[i];
        }
    }
}

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

// y[t] = sum over j of weights[t, j] ys[slots[t, j]], j ascending, in 32 bits, rounded once.  A
// warp has kU x 32 units of kJ entries' rows in flight.  Many tokens: 2 x 2 keeps 40 warps on an
// SM (16384 tokens x 8 rows of 4096 bf16 values 197 us; 4 x 2 with 20 warps 277 us).  Few tokens:
// one load's latency for four entries (4 tokens x 8 rows 4.9 us; one by one 8.8 us).  Narrower
// units: as many bytes in flight as the registers of their sums allow (8192 tokens x 4 rows of
// 4095 bf16 values 86 us, of 2047 float values 62; 16-byte rows 62 and 56).
template <typename T, typename U, int kJ, int kU>
__global__ void __launch_bounds__(kRowThreads) k_combine(int64_t tokens, int k, int64_t rows, int64_t units,
                                                        int64_t parts, const int32_t *__restrict__ slots,
                                                        const float *__restrict__ weights, const U *__restrict__ ys,
                                                        int64_t ldys, U *__restrict__ y, int64_t ldy) {
    constexpr int kN = sizeof(U) / sizeof(T);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp;
    const int64_t t = item / parts;
    if (t >= tokens) return;
    const int64_t u0 = (item - t * parts) * (32 * kU) + lane;
    float acc[kU][kN] = {};
    for (int j0 = 0; j0 < k; j0 += 32) {
        const Entries entries(t, k, j0, rows, slots, weights);
        const int n = min(k - j0, 32);
        for (int j = 0; j < n; j += kJ) {
            U v[kJ][kU];
            float w[kJ];
            bool some[kJ];
#pragma unroll
            for (int q = 0; q < kJ; ++q) {
                const int64_t s = entries.row(j + q);  // (-1 past the last)
                w[q] = entries.of(j + q);
                some[q] = s >= 0;
                if (some[q]) {
                    const U *src = ys + s * ldys;
#pragma unroll
                    for (int i = 0; i < kU; ++i)
                        if (u0 + i * 32 < units) v[q][i] = src[u0 + i * 32];
                }
            }
#pragma unroll
            for (int q = 0; q < kJ; ++q)
                if (some[q]) {
#pragma unroll
                    for (int i = 0; i < kU; ++i)
                        if (u0 + i * 32 < units) {
                            float f[kN];
                            unit_to_f32<T>(v[q][i], f);
#pragma unroll
                            for (int p = 0; p < kN; ++p) acc[i][p] = fmaf(w[q], f[p], acc[i][p]);
                        }
                }
        }
    }
    U *dst = y + t * ldy;
#pragma unroll
    for (int i = 0; i < kU; ++i)
        if (u0 + i * 32 < units) dst[u0 + i * 32] = unit_from_f32<T, U>(acc[i]);
}

// dys[slots[t, j]] = weights[t, j] dy[t] and dweights[t, j] = <dy[t], ys[slots[t, j]]>: one CTA
// per token (of one warp to eight, by the row's length), so that its products reduce inside the CTA in a
// fixed order (no atomics); entries are taken four at a time, dy coming from L1 from the second time on.  Rows of dys without
// a source are zeroed by the first CTAs.  16384 tokens x 4 of 2048 bf16 values: 94 us, 6.4 TB/s of
// dy, ys and dys.
template <typename T, typename U>
__global__ void __launch_bounds__(kRowThreads) k_combine_grad(int64_t pad_ctas, int k, int64_t rows, int64_t units,
                                                             const int32_t *__restrict__ slots,
                                                             const int32_t *__restrict__ sources,
                                                             const float *__restrict__ weights, const U *__restrict__ dy,
                                                             int64_t lddy, const U *__restrict__ ys, int64_t ldys,
                                                             U *__restrict__ dys, int64_t lddys,
                                                             float *__restrict__ dweights) {
    constexpr int kN = sizeof(U) / sizeof(T);
    constexpr int kJ = 4;
    __shared__ float part[kJ][kRowWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_threads = blockDim.x, n_warps = n_threads >> 5;
    if (blockIdx.x < pad_ctas) {
        zero_padding(static_cast<int64_t>(blockIdx.x) * kPadRows, rows, sources, units, dys, lddys);
        return;
    }
    const int64_t t = blockIdx.x - pad_ctas;
    const U *g = dy + t * lddy;
    for (int j0 = 0; j0 < k; j0 += kJ) {
        int64_t s[kJ];
        float w[kJ], acc[kJ] = {};
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            s[j] = j0 + j < k ? slots[t * k + j0 + j] : -1;
            if (s[j] >= rows) s[j] = -1;
            w[j] = s[j] >= 0 ? weights[t * k + j0 + j] : 0.0f;
        }
        for (int64_t u = threadIdx.x; u < units; u += n_threads) {
            U v[kJ];
            const U gu = g[u];
#pragma unroll
            for (int j = 0; j < kJ; ++j)
                if (s[j] >= 0) v[j] = ys[s[j] * ldys + u];
            float gf[kN];
            unit_to_f32<T>(gu, gf);
#pragma unroll
            for (int j = 0; j < kJ; ++j)
                if (s[j] >= 0) {
                    float f[kN], o[kN];
                    unit_to_f32<T>(v[j], f);
#pragma unroll
                    for (int q = 0; q < kN; ++q) {
                        acc[j] = fmaf(gf[q], f[q], acc[j]);
                        o[q] = w[j] * gf[q];
                    }
                    dys[s[j] * lddys + u] = unit_from_f32<T, U>(o);
                }
        }
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const float sum = warp_sum(acc[j]);
            if (lane == 0) part[j][warp] = sum;
        }
        if (n_warps > 1) __syncthreads();
        else __syncwarp();
        if (threadIdx.x < kJ && j0 + static_cast<int>(threadIdx.x) < k) {
            float sum = 0.0f;
            for (int i = 0; i < n_warps; ++i) sum += part[threadIdx.x][i];
            dweights[t * k + j0 + threadIdx.x] = sum;
        }
        if (n_warps > 1) __syncthreads();
        else __syncwarp();
    }
}

// The widest unit (16, 8, 4 or 2 bytes, at least the value size) that every row of every
// array starts on and that divides a row's bytes.
int unit_bytes(int value_size, int64_t d, std::initializer_list<std::pair<const void *, int64_t>> arrays) {
    uint64_t bits = static_cast<uint64_t>(d) * value_size;
    for (const auto &a : arrays)
        bits |= reinterpret_cast<uintptr_t>(a.first) | static_cast<uint64_t>(a.second) * value_size;
    for (int b = 16; b > value_size; b /= 2)
        if (bits % b == 0) return b;
    return value_size;
}

int check_route(int64_t tokens, int32_t k, int64_t rows) {
    if (tokens < 0 || tokens >= (int64_t(1) << 31)) return refuse("tokens must lie in [0, 2^31)");
    if (k < 1) return refuse("k must be at least 1");
    if (tokens * k >= (int64_t(1) << 31)) return set_error(SPMV_ERR_TOO_LARGE, "tokens * k must be below 2^31");
    if (rows < 0 || rows >= (int64_t(1) << 31)) return refuse("rows must lie in [0, 2^31)");
    return SPMV_OK;
}

int check_matrix(const void *p, const char *name, int64_t rows, int64_t d, int64_t ld, int dtype) {
    SPMV_TRY(check_shape(rows, d, ld, name));
    return rows && d ? check_array(p, name, row_value_bytes(dtype)) : SPMV_OK;
}

// An output shares no byte with an input (both matrices of rows, or plain arrays).
int check_apart(const void *out, size_t out_bytes, const char *out_name, const void *in, size_t in_bytes,
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

// Units of a row that a lane of k_dispatch holds: 64 bytes where they are 16 (16384 tokens x 4 of 2048 bf16
// values: 53.4 us; with two 52.6, with eight 55.6), else eight (8192 x 4 of 4095 bf16 values:
// 65.9 us; with four 65.7, with sixteen 68.3): enough in flight, few copies of a row's slots.
constexpr int units_per_lane(int bytes) { return bytes == 16 ? 4 : 8; }

template <typename T>
void launch_combine(int unit, int64_t tokens, int k, int64_t rows, int64_t d, const int32_t *slots,
                    const float *weights, const void *ys, int64_t ldys, void *y, int64_t ldy, cudaStream_t s) {
    auto go = [&](auto tag, auto entries, auto per_lane) {
        using U = decltype(tag);
        constexpr int kJ = decltype(entries)::value, kU = decltype(per_lane)::value;
        constexpr int64_t kN = sizeof(U) / sizeof(T);
        const int64_t units = d / kN, parts = ceil_div(units, 32 * kU);
        k_combine<T, U, kJ, kU><<<static_cast<unsigned>(ceil_div(tokens * parts, kRowWarps)), kRowThreads, 0, s>>>(
            tokens, k, rows, units, parts, slots, weights, static_cast<const U *>(ys), ldys / kN, static_cast<U *>(y),
            ldy / kN);
    };
    constexpr std::integral_constant<int, 1> one;
    constexpr std::integral_constant<int, 2> two;
    constexpr std::integral_constant<int, 4> four;
    constexpr std::integral_constant<int, 8> eight;
    constexpr std::integral_constant<int, 16> sixteen;
    // few tokens: as many warps as there are 512-byte pieces
    const bool few = tokens * d * static_cast<int64_t>(sizeof(T)) < int64_t(152) * 16 * 1024;
    if (unit == 16) few ? go(uint4{}, four, one) : go(uint4{}, two, two);
    else if (unit == 8) sizeof(T) == 4 ? go(uint2{}, two, eight) : go(uint2{}, one, four);
    else if (unit == 4) go(uint32_t{}, two, eight);
    else if constexpr (sizeof(T) == 2) go(uint16_t{}, two, sixteen);
}

template <typename T>
void launch_combine_grad(int unit, int64_t tokens, int k, int64_t rows, int64_t d, const int32_t *slots,
                         const int32_t *sources, const float *weights, const void *dy, int64_t lddy, const void *ys,
                         int64_t ldys, void *dys, int64_t lddys, float *dweights, cudaStream_t s) {
    auto go = [&](auto tag) {
        using U = decltype(tag);
        constexpr int64_t kN = sizeof(U) / sizeof(T);
        const int64_t units = d / kN;
        // two to eight units a thread: fewer leave warps without work behind the sums' barriers, more
        // leave too little in flight.  us with 32, 64, 128, 256 threads for 4 rows a token of
        //   8 units (16384 bf16 tokens)     11.8  17.3  20.8  41.6
        //   64                              25.2  26.8  37.2  70.1
        //   128                             48.1  47.6  50.8  79.5
        //   256                             93.2  91.3  90.5  104
        //   1024 (4096 tokens)              102   94.8  92.8  91.4
        //   4095 of 2 bytes (8192 tokens)   230   170   154   149
        const int threads = units >= 512 ? 256 : units >= 128 ? 128 : units > 64 ? 64 : 32;
        k_combine_grad<T, U><<<static_cast<unsigned>(tokens + ceil_div(rows, kPadRows)), threads, 0, s>>>(
            ceil_div(rows, kPadRows), k, rows, units, slots, sources, weights, static_cast<const U *>(dy), lddy / kN,
            static_cast<const U *>(ys), ldys / kN, static_cast<U *>(dys), lddys / kN, dweights);
    };
    if (unit == 16) go(uint4{});
    else if (unit == 8) go(uint2{});
    else if (unit == 4) go(uint32_t{});
    else if constexpr (sizeof(T) == 2) go(uint16_t{});
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" SPMV_API int64_t spmv_route_rows(int64_t tokens, int32_t k, int32_t experts, int32_t align) {
    SPMV_TRY(check_route(tokens, k, 0));
    if (experts < 1 || experts > kMaxExperts) return refuse("experts must lie in [1, " + std::to_string(kMaxExperts) + "]");
    if (align < 1 || align > 65536) return refuse("align must lie in [1, 65536]");
    const int64_t m = tokens * k, used = m < experts ? m : experts;
    const int64_t rows = (m + used * (align - 1)) / align * align;
    if (rows >= (int64_t(1) << 31)) return set_error(SPMV_ERR_TOO_LARGE, "the sorted matrix would have 2^31 rows or more");
    return rows;
}

extern "C" SPMV_API int64_t spmv_route_workspace(int64_t tokens, int32_t k, int32_t experts) {
    const int64_t rows = spmv_route_rows(tokens, k, experts, 1);
    if (rows < 0) return rows;
    const PlanShape p = plan_shape(tokens, k, experts);
    return p.ctas > 1 ? static_cast<int64_t>(p.ctas) * experts * static_cast<int64_t>(sizeof(int32_t)) : 0;
}

extern "C" SPMV_API int spmv_route_plan(int64_t tokens, int32_t k, int32_t experts, int32_t align, const int32_t *ids,
                                        int32_t *offsets, int32_t *slots, int32_t *sources, void *workspace,
                                        int64_t workspace_bytes, void *stream) {
    const int64_t rows = spmv_route_rows(tokens, k, experts, align);
    if (rows < 0) return static_cast<int>(rows);
    const int64_t need = spmv_route_workspace(tokens, k, experts);
    if (workspace_bytes < need) return refuse("the workspace has fewer bytes than spmv_route_workspace says");
    const int64_t m = tokens * k;
    SPMV_TRY(check_array(offsets, "offsets", 4));
    if (m) {
        SPMV_TRY(check_array(ids, "ids", 4));
        SPMV_TRY(check_array(slots, "slots", 4));
        SPMV_TRY(check_array(sources, "sources", 4));
    }
    if (need) SPMV_TRY(check_array(workspace, "workspace", 4));
    const struct { const void *p; size_t bytes; const char *name; } arrays[] = {
        {ids, static_cast<size_t>(m) * 4, "ids"}, {offsets, static_cast<size_t>(experts + 1) * 4, "offsets"},
        {slots, static_cast<size_t>(m) * 4, "slots"}, {sources, static_cast<size_t>(rows) * 4, "sources"},
        {workspace, static_cast<size_t>(need), "workspace"}};
    for (int a = 1; a < 5; ++a)
        for (int b = 0; b < a; ++b)
            SPMV_TRY(check_apart(arrays[a].p, arrays[a].bytes, arrays[a].name, arrays[b].p, arrays[b].bytes, arrays[b].name));
    const PlanShape p = plan_shape(tokens, k, experts);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int32_t *hist = p.ctas > 1 ? static_cast<int32_t *>(workspace) : nullptr;
    if (p.smem > 48 * 1024)
        SPMV_TRY_CUDA(cudaFuncSetAttribute(k_route_place, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanSmem));
    if (hist) {
        k_route_hist<<<p.ctas, kPlanThreads, static_cast<size_t>(experts) * 4, s>>>(m, p.chunk, experts, ids, hist);
        SPMV_TRY_CUDA(cudaGetLastError());
    }
    // the second kernel counts its own share while the first one ends
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ctas));
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = hist ? 1 : 0;
    SPMV_TRY_CUDA(cudaLaunchKernelEx(&cfg, k_route_place, m, p.chunk, experts, align, rows, p.warps, ids,
                                     static_cast<const int32_t *>(hist), offsets, slots, sources));
    return SPMV_OK;
}

extern "C" SPMV_API int spmv_route_dispatch(int64_t tokens, int32_t k, int64_t rows, int64_t d, const int32_t *slots,
                                            const int32_t *sources, const void *x, int64_t ldx, void *xs, int64_t ldxs,
                                            int dtype, void *stream) {
    SPMV_TRY(check_route(tokens, k, rows));
    if (!row_dtype_ok(dtype)) return refuse("dtype must be SPMV_F32, SPMV_F16 or SPMV_BF16");
    SPMV_TRY(check_matrix(x, "x", tokens, d, ldx, dtype));
    SPMV_TRY(check_matrix(xs, "xs", rows, d, ldxs, dtype));
    if (rows == 0 || d == 0) return SPMV_OK;
    if (tokens) SPMV_TRY(check_array(slots, "slots", 4));
    SPMV_TRY(check_array(sources, "sources", 4));
    const int vb = row_value_bytes(dtype);
    const size_t out = span_bytes(rows, d, ldxs, vb);
    SPMV_TRY(check_apart(xs, out, "xs", x, span_bytes(tokens, d, ldx, vb), "x"));
    SPMV_TRY(check_apart(xs, out, "xs", slots, static_cast<size_t>(tokens * k) * 4, "slots"));
    SPMV_TRY(check_apart(xs, out, "xs", sources, static_cast<size_t>(rows) * 4, "sources"));
    const int unit = unit_bytes(vb, d, {{x, ldx}, {xs, ldxs}});
    cudaStream_t s = static_cast<cudaStream_t>(stream);
#define SPMV_DISPATCH(B)                                                                                       \
    do {                                                                                                       \
        using U = Unit<B>::type;                                                                               \
        constexpr int kU = units_per_lane(B);                                                                  \
        const int64_t units = d * vb / B, parts = ceil_div(units, 32 * kU);                                    \
        const int64_t pads = ceil_div(rows, kPadRows), ctas = ceil_div(tokens * parts, kRowWarps);             \
        k_dispatch<U, kU><<<static_cast<unsigned>(pads + ctas), kRowThreads, 0, s>>>(                          \
            tokens, k, rows, units, parts, pads, slots, sources, static_cast<const U *>(x), ldx * vb / B,      \
            static_cast<U *>(xs), ldxs * vb / B);                                                              \
    } while (0)
    SPMV_UNIT_SWITCH(unit, SPMV_DISPATCH)
#undef SPMV_DISPATCH
    SPMV_TRY_CUDA(cudaGetLastError());
    return SPMV_OK;
}

extern "C" SPMV_API int spmv_route_combine(int64_t tokens, int32_t k, int64_t rows, int64_t d, const int32_t *slots,
                                           const float *weights, const void *ys, int64_t ldys, void *y, int64_t ldy,
                                           int dtype, void *stream) {
    SPMV_TRY(check_route(tokens, k, rows));
    if (!row_dtype_ok(dtype)) return refuse("dtype must be SPMV_F32, SPMV_F16 or SPMV_BF16");
    SPMV_TRY(check_matrix(ys, "ys", rows, d, ldys, dtype));
    SPMV_TRY(check_matrix(y, "y", tokens, d, ldy, dtype));
    if (tokens == 0 || d == 0) return SPMV_OK;
    SPMV_TRY(check_array(slots, "slots", 4));
    if (weights) SPMV_TRY(check_array(weights, "weights", 4));
    const int vb = row_value_bytes(dtype);
    const size_t out = span_bytes(tokens, d, ldy, vb), m = static_cast<size_t>(tokens * k) * 4;
    SPMV_TRY(check_apart(y, out, "y", ys, span_bytes(rows, d, ldys, vb), "ys"));
    SPMV_TRY(check_apart(y, out, "y", slots, m, "slots"));
    SPMV_TRY(check_apart(y, out, "y", weights, m, "weights"));
    const int unit = unit_bytes(vb, d, {{ys, ldys}, {y, ldy}});
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SPMV_F32) launch_combine<float>(unit, tokens, k, rows, d, slots, weights, ys, ldys, y, ldy, s);
    else if (dtype == SPMV_F16) launch_combine<__half>(unit, tokens, k, rows, d, slots, weights, ys, ldys, y, ldy, s);
    else launch_combine<__nv_bfloat16>(unit, tokens, k, rows, d, slots, weights, ys, ldys, y, ldy, s);
    SPMV_TRY_CUDA(cudaGetLastError());
    return SPMV_OK;
}

extern "C" SPMV_API int spmv_route_combine_grad(int64_t tokens, int32_t k, int64_t rows, int64_t d,
                                                const int32_t *slots, const int32_t *sources, const float *weights,
                                                const void *dy, int64_t lddy, const void *ys, int64_t ldys, void *dys,
                                                int64_t lddys, float *dweights, int dtype, void *stream) {
    SPMV_TRY(check_route(tokens, k, rows));
    if (!row_dtype_ok(dtype)) return refuse("dtype must be SPMV_F32, SPMV_F16 or SPMV_BF16");
    SPMV_TRY(check_matrix(dy, "dy", tokens, d, lddy, dtype));
    SPMV_TRY(check_matrix(ys, "ys", rows, d, ldys, dtype));
    SPMV_TRY(check_matrix(dys, "dys", rows, d, lddys, dtype));
    if (tokens + ceil_div(rows, kPadRows) >= int64_t(1) << 31)  // CTAs
        return set_error(SPMV_ERR_TOO_LARGE, "tokens + rows / " + std::to_string(kPadRows) + " must be below 2^31");
    if (rows) SPMV_TRY(check_array(sources, "sources", 4));
    if (tokens) {
        SPMV_TRY(check_array(slots, "slots", 4));
        SPMV_TRY(check_array(weights, "weights", 4));
        SPMV_TRY(check_array(dweights, "dweights", 4));
    }
    if (tokens == 0 && rows == 0) return SPMV_OK;
    const int vb = row_value_bytes(dtype);
    const size_t m = static_cast<size_t>(tokens * k) * 4;
    const struct { const void *p; size_t bytes; const char *name; } in[] = {
        {dy, span_bytes(tokens, d, lddy, vb), "dy"}, {ys, span_bytes(rows, d, ldys, vb), "ys"},
        {slots, m, "slots"}, {sources, static_cast<size_t>(rows) * 4, "sources"}, {weights, m, "weights"}};
    const size_t out = span_bytes(rows, d, lddys, vb);
    for (const auto &a : in) {
        SPMV_TRY(check_apart(dys, out, "dys", a.p, a.bytes, a.name));
        SPMV_TRY(check_apart(dweights, m, "dweights", a.p, a.bytes, a.name));
    }
    SPMV_TRY(check_apart(dys, out, "dys", dweights, m, "dweights"));
    const int unit = unit_bytes(vb, d, {{dy, lddy}, {ys, ldys}, {dys, lddys}});
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SPMV_F32)
        launch_combine_grad<float>(unit, tokens, k, rows, d, slots, sources, weights, dy, lddy, ys, ldys, dys, lddys, dweights, s);
    else if (dtype == SPMV_F16)
        launch_combine_grad<__half>(unit, tokens, k, rows, d, slots, sources, weights, dy, lddy, ys, ldys, dys, lddys, dweights, s);
    else
        launch_combine_grad<__nv_bfloat16>(unit, tokens, k, rows, d, slots, sources, weights, dy, lddy, ys, ldys, dys, lddys, dweights, s);
    SPMV_TRY_CUDA(cudaGetLastError());
    return SPMV_OK;
}
