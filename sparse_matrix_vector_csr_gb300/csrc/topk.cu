// The k largest entries of every row of a dense matrix: dense rows to sparse rows.  Values
// descend, ties go to the lowest column, -inf is never taken.  With them the row's
// log-sum-exp (the same pass over the row) and softmax weights, and the weights' gradient.
#include <type_traits>

#include "topk.cuh"

namespace spmv {
namespace {

using namespace rows;

constexpr int kMaxTop = 256;
constexpr int kWarpMaxN = 512;    // rows up to this length are taken by one warp each
constexpr int kWarpMaxK = 32;     // ... with one lane per chosen entry
constexpr int kMaxCand = 640;     // candidates that one CTA sorts
constexpr int kMaxPieces = 512;  // pieces that are read again
constexpr int kMaxGroups = 512;   // maxima that set the threshold

// (key of the value, column) as one number: unique within a row, larger = taken earlier.
__device__ __forceinline__ unsigned long long composite(float v, int64_t col) {
    return (static_cast<unsigned long long>(order_key(v)) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ int32_t composite_col(unsigned long long c) {
    return static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(c));
}

// ----------------------------------------------------------------------------
// short rows: one warp per row
// ----------------------------------------------------------------------------
// The row sits in registers, value i * 32 + lane in register i.  k rounds: the warp's
// largest key (redux), the lowest column that has it (redux), the owner drops it.
template <typename T, int kR>
__global__ void __launch_bounds__(256) k_topk_warp(TopArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= a.rows) return;
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    const int n = static_cast<int>(a.n);
    uint32_t key[kR];  // 0 = taken, or not there, or -inf
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        const int c = i * 32 + lane;
        const float v = c < n ? to_f32(x[c]) : kNegInf;
        key[i] = v == kNegInf ? 0u : order_key(v);
    }
    float sum = 0.0f, m = 0.0f;
    if (a.lse || a.weighting == SPMV_WEIGHTS_ROW) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < kR; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        m = best ? key_value(best) : 0.0f;
#pragma unroll
        for (int i = 0; i < kR; ++i)
            if (key[i]) sum += ex2((key_value(key[i]) - m) * a.scale);
        sum = warp_sum(sum);
    }
    int32_t my_id = -1;
    uint32_t my_key = 0;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kR; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top == 0) break;
        const uint32_t mine = best == top ? static_cast<uint32_t>(at * 32 + lane) : 0xffffffffu;
        const uint32_t col = __reduce_min_sync(0xffffffffu, mine);
        if (mine == col) {
#pragma unroll
            for (int i = 0; i < kR; ++i)
                if (i == at) key[i] = 0;
        }
        if (lane == j) {
            my_id = static_cast<int32_t>(col);
            my_key = top;
        }
    }
    const float v = my_key ? key_value(my_key) : kNegInf;
    if (a.weighting == SPMV_WEIGHTS_SELECTED) {
        const float m0 = reference_of(__shfl_sync(0xffffffffu, v, 0));
        const float e = my_key ? ex2((v - m0) * a.scale) : 0.0f;
        const float s = warp_sum(e);
        if (lane < a.k) a.weights[row * a.k + lane] = my_key ? e / s : 0.0f;
    } else if (a.weighting == SPMV_WEIGHTS_ROW) {
        if (lane < a.k) a.weights[row * a.k + lane] = my_key ? ex2((v - m) * a.scale) / sum : 0.0f;
    }
    if (lane < a.k) {
        a.ids[row * a.k + lane] = my_id;
        if (a.vals) a.vals[row * a.k + lane] = v;
    }
    if (a.lse && lane == 0) a.lse[row] = log_sum(m, sum, a.inv_temperature);
}

// ----------------------------------------------------------------------------
// long rows: a CTA, or a cluster of CTAs, per row
// ----------------------------------------------------------------------------
// 1. Every thread reads its share once, a few vectors at a time, and keeps its maximum and the maxima
//    of pieces of 16 values (in shared memory).  The k-th largest of the maxima of groups of
//    threads is a lower bound of the row's k-th largest entry that passes few others; a warp
//    finds it to 20 bits of its order, which keeps it one.
// 2. The few pieces that reach it are listed and read again (from L2), all at once, and their
//    entries at or above it go to the first CTA's candidate list.
// 3. If a list overflows (values bunched in one group, or many ties), the threshold is
//    bisected on (value, column) numbers, which are unique, until between k and kMaxCand
//    pass: at most 64 counting passes, whatever the row holds.  They cost: a row of 50021 equal fp16
//    values takes 310 us, and a twentieth of 4096 such rows makes 99 us of a call 1610.
// 4. The first CTA ranks the candidates by counting and writes the k largest.
// 32 of 4096 x 50021 fp16 values with the log-sum: 99 us, 4.1 TB/s, the reading itself about 75; the
// rest is the chain threshold - pieces - candidates, which six CTAs an SM overlap in part, and
// instructions (70 % of the issue slots).  One reading kept in registers or shared memory would
// need a cluster's barriers per row (372 us for the first such kernel).
constexpr int kBatch = 4;        // vectors a thread loads at a time
constexpr int kPieceMaxima = 15; // a thread's pieces share this many maxima (and one for the row's ends)

struct TopShared {
    unsigned long long cand[kMaxCand];
    uint32_t group_max[kMaxGroups];  // as order keys
    float2 sums[kMaxCluster * 16];  // per warp of the cluster: maximum, sum of exponentials
    float top_vals[kMaxTop];
    uint32_t piece[kMaxPieces];  // listed: thread and slot of the maximum
    uint32_t count[5];  // [0] candidates (first CTA's), [1..3] the bisection's counts, [4] listed pieces
    float thr, lse_m, lse_sum;
};

// Thread t's vectors of a share: lo + t + i w inside the row, and, for threads 0 and 1, the vector at
// the row's start and end.
template <typename T>
struct Batches {
    const Share<T> share;
    int t, w;
    __device__ __forceinline__ Batches(const Share<T> &s, int t_, int w_) : share(s), t(t_), w(w_) {}
    __device__ __forceinline__ int edge() const {
        if (t == 0 && share.lo == 1 && share.count > 0) return 0;
        if (t == 1 && share.hi < share.count && share.hi >= share.lo) return share.hi;
        return -1;
    }
    // f(vector, its index) over all of the thread's vectors
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll 1
        for (int v = share.lo + t; v < share.hi; v += w) f(share.load_whole(v), v);
        if (edge() >= 0) f(share.load(edge()), edge());
    }
};
// f(value, column) over the values of a vector
template <typename T, typename F>
__device__ __forceinline__ void each_value(const Share<T> &share, const uint4 &vec, int v, F f) {
    float x[Vec<T>::kN];
    unpack<T>(vec, x);
    const int64_t e = share.first(v);
#pragma unroll
    for (int q = 0; q < Vec<T>::kN; ++q) f(x[q], e + q);
}

// The list overflowed: candidates by bisection on (value, column); returns how many.  Out of line, by
// values that are at hand (a reference to the caller's would keep them in memory all along).
template <typename T>
__device__ __noinline__ uint32_t collect_by_bisection(const T *x, int64_t n, int k, uint32_t rank, int log2_ctas, float thr,
                                                      uint32_t shared) {
    TopShared &sh = *static_cast<TopShared *>(__cvta_shared_to_generic(shared));
    const Share<T> share(RowView<T>(x, n), rank, log2_ctas);
    const Batches<T> batches(share, threadIdx.x, blockDim.x);
    const int tid = threadIdx.x, lane = tid & 31, ctas = 1 << log2_ctas;
    unsigned long long lo = static_cast<unsigned long long>(order_key(thr)) << 32, hi = ~0ull, cut = lo;
    uint32_t found = kMaxCand + 1;
    for (int step = 0; step < 64 && found > kMaxCand; ++step) {
        cut = lo + (hi - lo) / 2;
        int mine = 0;
        batches.each([&](const uint4 &x, int v) {
            each_value<T>(batches.share, x, v, [&](float f, int64_t e) { mine += f != kNegInf && composite(f, e) >= cut; });
        });
        __syncwarp();
        mine = warp_sum(mine);
        const int slot = 1 + step % 3;
        if (lane < ctas && mine) {
            if (ctas > 1) peer_add(peer_addr(&sh.count[slot], lane), mine);
            else atomicAdd(&sh.count[slot], mine);
        }
        cluster_sync(ctas);
        found = sh.count[slot];
        if (tid == 0) sh.count[1 + (step + 2) % 3] = 0;  // last read before the previous barrier
        if (found > kMaxCand) lo = cut;
        else if (found < static_cast<uint32_t>(k)) {
            hi = cut;
            found = kMaxCand + 1;
        }
    }
    if (tid == 0) sh.count[0] = 0;
    cluster_sync(ctas);
    batches.each([&](const uint4 &x, int v) {
        each_value<T>(batches.share, x, v, [&](float f, int64_t e) {
            if (f == kNegInf || composite(f, e) < cut) return;
            if (ctas > 1) {
                const uint32_t at = peer_add(peer_addr(&sh.count[0], 0), 1);
                if (at < kMaxCand) peer_store64(peer_addr(&sh.cand[at], 0), composite(f, e));
            } else {
                const uint32_t at = atomicAdd(&sh.count[0], 1u);
                if (at < kMaxCand) sh.cand[at] = composite(f, e);
            }
        });
    });
    __syncwarp();
    cluster_sync(ctas);
    return ctas > 1 ? peer_load(peer_addr(&sh.count[0], 0)) : sh.count[0];
}

// A piece's maximum in 16 bits, 32-bit values rounded up: shared memory is what L1 has less of for
// loads in flight (32 largest of 4096 x 50021 fp16 rows: 99 us so, 106 with 32-bit maxima).
template <typename T>
struct PieceMax {
    using type = T;
    static __device__ __forceinline__ T of(float v) { return from_f32<T>(v); }
};
template <>
struct PieceMax<float> {
    using type = __nv_bfloat16;
    static __device__ __forceinline__ __nv_bfloat16 of(float v) { return __float2bfloat16_ru(v); }
};

// 2^log2_per pieces share a maximum; slots: maxima a thread has for its whole vectors.
template <typename T>
__global__ void __launch_bounds__(512, 3) k_topk_row(TopArgs a, int log2_ctas, int log2_group, int log2_per, int slots) {
    constexpr int kN = Vec<T>::kN, kPiece = 16 / kN;  // vectors of a piece
    __shared__ __align__(16) TopShared sh;
    extern __shared__ __align__(16) unsigned char piece_mem[];
    using Bound = typename PieceMax<T>::type;
    Bound *piece_max = reinterpret_cast<Bound *>(piece_mem);  // [slots + 1][threads]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_threads = blockDim.x, n_warps = n_threads >> 5;
    const int ctas = 1 << log2_ctas, group = 1 << log2_group, per = 1 << log2_per;
    const int64_t r = blockIdx.x >> log2_ctas;
    const uint32_t rank = blockIdx.x & (ctas - 1);
    const RowView<T> row(static_cast<const T *>(a.x) + r * a.ldx, a.n);
    const Share<T> share(row, rank, log2_ctas);
    const Batches<T> batches(share, tid, n_threads);
    const bool want_lse = a.lse || a.weighting == SPMV_WEIGHTS_ROW;
    if (ctas > 1) cluster_arrive();  // the peers' shared memory may be written from here on ...
    if (tid < 5) sh.count[tid] = 0;

    Running run;  // its maximum passes over NaNs; the pieces' maxima hand them on
    const auto note = [&](const uint4 *x, float top, auto n) {
        if (want_lse) run.add<T, decltype(n)::value>(x, top, a.scale);
        else if (top > run.m) run.m = top;
    };
    int left = per;
    float so_far = kNegInf;
    Bound *next = piece_max + tid, *const last = next + slots * n_threads;
    const auto piece = [&](float top) {
        so_far = max_nan(so_far, top);
        if (--left == 0) {
            *next = PieceMax<T>::of(so_far);
            next += n_threads;
            so_far = kNegInf;
            left = per;
        }
    };
    int v = share.lo + tid;
    for (; v + (kBatch - 1) * n_threads < share.hi; v += kBatch * n_threads) {
        uint4 x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) x[i] = share.load_whole(v + i * n_threads);
        float all = kNegInf;
#pragma unroll
        for (int i = 0; i < kBatch; i += kPiece) {
            float top = vec_max_nan(x[i], T());
#pragma unroll
            for (int q = 1; q < kPiece; ++q) top = max_nan(top, vec_max_nan(x[i + q], T()));
            piece(top);
            all = max_nan(all, top);
        }
        note(x, all, std::integral_constant<int, kBatch>());
    }
    {
        uint4 x[kBatch - 1];
#pragma unroll
        for (int i = 0; i < kBatch - 1; ++i)
            if (v + i * n_threads < share.hi) x[i] = share.load_whole(v + i * n_threads);
        float top = kNegInf;
#pragma unroll
        for (int i = 0; i < kBatch - 1; ++i) {
            if (v + i * n_threads < share.hi) {
                const float one = vec_max_nan(x[i], T());
                top = max_nan(top, one);
                note(x + i, one, std::integral_constant<int, 1>());
            }
            if (i % kPiece == kPiece - 1 || i == kBatch - 2) {  // the last piece may lack vectors, or have none
                if (next < last) piece(top);
                top = kNegInf;
            }
        }
        for (; next < last; next += n_threads, so_far = kNegInf) *next = PieceMax<T>::of(so_far);
        if (batches.edge() >= 0) {
            x[0] = share.load(batches.edge());
            top = vec_max_nan(x[0], T());
            note(x, top, std::integral_constant<int, 1>());
        }
        *last = PieceMax<T>::of(top);
    }
    float g = run.m;
    for (int o = 1; o < group; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    const float m = warp_max(run.m);
    float sum = 0.0f;
    if (want_lse) {
        sum = run.sum();
        if (run.m != kNegInf) sum *= ex2((run.m - m) * a.scale);
        sum = warp_sum(sum);
    }
    if (ctas > 1) cluster_wait();  // ... once they have all started
    const int per_cta = n_threads >> log2_group, n_groups = per_cta * ctas;
    if ((tid & (group - 1)) == 0)
        for (int c = 0; c < ctas; ++c) {
            uint32_t *at = &sh.group_max[rank * per_cta + (tid >> log2_group)];
            if (ctas > 1) peer_store(peer_addr(at, c), __uint_as_float(order_key(g)));
            else *at = order_key(g);
        }
    if (want_lse && lane < ctas) {
        float2 *at = &sh.sums[rank * n_warps + warp];
        if (ctas > 1) peer_store2(peer_addr(at, lane), m, sum);
        else *at = make_float2(m, sum);
    }
    if (tid == 0) sh.thr = kNegInf;
    cluster_sync(ctas);

    if (n_groups <= (ctas > 1 ? 128 : 64)) {  // few, or little else to do: by counting, a thread each
        for (int i = tid; i < n_groups; i += n_threads) {
            const uint32_t key = sh.group_max[i];
            int above = 0;
            for (int j = 0; j < n_groups; j += 4) {  // (a multiple of 4)
                const uint4 w = *reinterpret_cast<const uint4 *>(&sh.group_max[j]);
                above += (w.x > key || (w.x == key && j < i)) + (w.y > key || (w.y == key && j + 1 < i)) +
                         (w.z > key || (w.z == key && j + 2 < i)) + (w.w > key || (w.w == key && j + 3 < i));
            }
            if (above == a.k - 1) sh.thr = key_value(key);
        }
    } else if (warp == 0) {  // by bits of the order, a count for each
        uint32_t key[kMaxGroups / 32];
#pragma unroll
        for (int i = 0; i < kMaxGroups / 32; ++i) key[i] = i * 32 + lane < n_groups ? sh.group_max[i * 32 + lane] : 0;
        uint32_t found_key = 0;
        for (int bit = 31; bit >= 12; --bit) {
            const uint32_t cut = found_key | 1u << bit;
            int n = 0;
#pragma unroll
            for (int i = 0; i < kMaxGroups / 32; ++i)
                if (i * 32 < n_groups) n += key[i] >= cut;
            if (warp_sum(n) >= a.k) found_key = cut;
        }
        if (lane == 0) sh.thr = key_value(found_key);  // (a NaN below -inf's key: no bound)
    }
    __syncthreads();
    const float thr = fmaxf(sh.thr, -FLT_MAX);  // above -inf: masked entries are never candidates

    for (int s = 0; s <= slots; ++s)
        if (!(to_f32(piece_max[s * n_threads + tid]) < thr)) {
            const uint32_t at = atomicAdd(&sh.count[4], 1u);
            if (at < kMaxPieces) sh.piece[at] = static_cast<uint32_t>(s) << 16 | tid;
        }
    __syncthreads();
    const uint32_t listed = sh.count[4];
    if (listed <= kMaxPieces) {
        // half a warp a piece, a value a lane, four loads in flight
        const int in = lane & 15, half = tid >> 4, halves = n_threads >> 4;
        const int64_t at_lane = static_cast<int64_t>(in / kN) * n_threads * kN + in % kN;  // from the piece's first value
        const int items = static_cast<int>(listed) << log2_per;  // pieces, a slot's one after the other
        for (int i0 = half; i0 < items; i0 += 4 * halves) {
            float f[4];
            int64_t e[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u * halves;
                f[u] = kNegInf;
                e[u] = -1;
                if (i < items) {
                    const uint32_t b = sh.piece[i >> log2_per];
                    const int owner = static_cast<int>(b & 0xffff), s = static_cast<int>(b >> 16), sub = i & (per - 1);
                    if (s == slots) {  // the owner's vector at the row's start or end
                        e[u] = share.first(owner == 0 && share.lo == 1 ? 0 : share.hi) + in;
                        if (sub == 0 && in < kN && e[u] >= 0 && e[u] < a.n) f[u] = to_f32(share.p[e[u]]);
                    } else {
                        const int first = share.lo + owner + ((s << log2_per) + sub) * kPiece * n_threads;
                        e[u] = share.first(first) + at_lane;
                        if (first + in / kN * n_threads < share.hi) f[u] = to_f32(share.p[e[u]]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (!(f[u] < thr)) {
                    const uint32_t at = ctas > 1 ? peer_add(peer_addr(&sh.count[0], 0), 1) : atomicAdd(&sh.count[0], 1u);
                    if (at < kMaxCand) {
                        if (ctas > 1) peer_store64(peer_addr(&sh.cand[at], 0), composite(f[u], e[u]));
                        else sh.cand[at] = composite(f[u], e[u]);
                    }
                }
        }
    } else if (tid == 0) {
        if (ctas > 1) peer_add(peer_addr(&sh.count[0], 0), kMaxCand + 1);
        else atomicAdd(&sh.count[0], kMaxCand + 1);
    }
    __syncwarp();
    cluster_sync(ctas);
    uint32_t found = ctas > 1 ? peer_load(peer_addr(&sh.count[0], 0)) : sh.count[0];
    if (found > kMaxCand) found = collect_by_bisection<T>(row.p, a.n, a.k, rank, log2_ctas, thr, smem_addr(&sh));
    // the first CTA stays until the others have read its count; they have nothing left to do
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
    }

    // rank 0: the candidates in order, the row's sum (by the last warp)
    if (warp == n_warps - 1 && want_lse) {
        float mm = kNegInf;
        for (int i = lane; i < n_warps * ctas; i += 32) mm = fmaxf(mm, sh.sums[i].x);
        mm = reference_of(warp_max(mm));
        float s = 0.0f;
        for (int i = lane; i < n_warps * ctas; i += 32) {
            const float2 w = sh.sums[i];  // a warp without a value above -inf adds its 0 (or a NaN)
            s += w.x == kNegInf ? w.y : w.y * ex2((w.x - mm) * a.scale);
        }
        s = warp_sum(s);
        if (lane == 0) {
            sh.lse_m = mm;
            sh.lse_sum = s;
            if (a.lse && s == s) a.lse[r] = fmaf(mm, a.inv_temperature, logf(s));
        }
    }
    const int n_cand = static_cast<int>(found < kMaxCand ? found : kMaxCand);
    for (int i = tid; i < n_cand; i += n_threads) {
        const unsigned long long c = sh.cand[i];
        int above = 0;
        for (int j = 0; j < n_cand; ++j) above += sh.cand[j] > c;
        if (above < a.k) {
            const float v = key_value(static_cast<uint32_t>(c >> 32));
            sh.top_vals[above] = v;
            a.ids[r * a.k + above] = composite_col(c);
            if (a.vals) a.vals[r * a.k + above] = v;
            // a sum that is NaN comes from the row's largest entry, and so does its log: +inf or NaN
            if (above == 0 && !(v < INFINITY) && a.lse) a.lse[r] = v;
        }
    }
    for (int j = n_cand + tid; j < a.k; j += n_threads) {
        sh.top_vals[j] = kNegInf;
        a.ids[r * a.k + j] = -1;
        if (a.vals) a.vals[r * a.k + j] = kNegInf;
    }
    if (a.weighting == SPMV_WEIGHTS_NONE) return;
    __syncthreads();
    if (warp == 0) {
        float mm = sh.lse_m, s = sh.lse_sum;
        if (a.weighting == SPMV_WEIGHTS_SELECTED) {
            mm = reference_of(sh.top_vals[0]);
            s = 0.0f;
            for (int j = lane; j < a.k; j += 32) s += ex2((sh.top_vals[j] - mm) * a.scale);
            s = warp_sum(s);
        }
        for (int j = lane; j < a.k; j += 32) {
            const float v = sh.top_vals[j];
            a.weights[r * a.k + j] = v == kNegInf ? 0.0f : ex2((v - mm) * a.scale) / s;
        }
    }
}

// ----------------------------------------------------------------------------
// gradient of the weights
// ----------------------------------------------------------------------------
// With s = sum over j of w_j dw_j, both weightings give dx[id_j] = w_j (dw_j - s) / temperature;
// elsewhere dx is 0 (weights over the chosen entries) or -q s / temperature with q the softmax of
// the row (weights over the whole row; see RowShare).  A warp writes a piece of a
// row; __syncwarp orders its plain stores before the stores to the chosen columns.  32 entries of 4096 x
// 50021 bf16 rows, over the row: 199 us, 4.1 TB/s; x is read a value at a time, which is what bounds it.
constexpr int kGradPiece = 1024;  // values per warp

template <typename T>
__global__ void __launch_bounds__(256) k_topk_grad(TopGradArgs a) {
    constexpr int kN = Vec<T>::kN;
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t r = a.pieces == 1 ? item : item / a.pieces;
    if (r >= a.rows) return;
    T *out = static_cast<T *>(a.dx) + r * a.lddx;
    const RowView<T> view(out, a.n);
    const Share<T> piece(view, (item - r * a.pieces) * (kGradPiece / kN), int64_t(kGradPiece / kN));
    const int32_t *ids = a.ids + r * a.k;
    const float *w = a.weights + r * a.k, *dw = a.dweights + r * a.k;
    float s = 0.0f;
    for (int j = lane; j < a.k; j += 32)
        if (ids[j] >= 0 && ids[j] < a.n) s = fmaf(w[j], dw[j], s);
    s = warp_sum(s);
    const bool whole_row = a.weighting == SPMV_WEIGHTS_ROW;
    const T *x = static_cast<const T *>(a.x) + (whole_row ? r * a.ldx : 0);
    // (a row without entries has nothing above -inf: 0 everywhere)
    const bool some = whole_row && ids[0] >= 0 && ids[0] < a.n;
    const RowShare q{some ? to_f32(x[ids[0]]) : 0.0f, some ? w[0] * (-s * a.inv_temperature) : 0.0f,
                     a.inv_temperature * kLog2e};
    for (int v = lane; v < piece.count; v += 32) {
        float f[kN] = {};
        if (some) {
            const int64_t e = piece.first(v);
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (e + i >= 0 && e + i < a.n) f[i] = q.of(to_f32(x[e + i]));
        }
        piece.store(out, v, pack<T>(f), true);
    }
    __syncwarp();
    for (int j = lane; j < a.k; j += 32) {
        const int32_t id = ids[j];
        if (id >= 0 && id < a.n && piece.owns(id)) out[id] = from_f32<T>(w[j] * (dw[j] - s) * a.inv_temperature);
    }
}

template <typename T>
cudaError_t launch_topk_warp(const TopArgs &a, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(ceil_div(a.rows, 8));
    if (a.n <= 64) k_topk_warp<T, 2><<<grid, 256, 0, s>>>(a);
    else if (a.n <= 128) k_topk_warp<T, 4><<<grid, 256, 0, s>>>(a);
    else if (a.n <= 256) k_topk_warp<T, 8><<<grid, 256, 0, s>>>(a);
    else k_topk_warp<T, 16><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_topk_row(const TopArgs &a, cudaStream_t s) {
    const int64_t vectors = row_vectors<T>(a.n, a.x, a.ldx);
    // few rows: more CTAs a row while SMs would be idle and each thread still has a batch
    int ctas = 1;
    while (ctas < kMaxCluster && a.rows * ctas < kSms && vectors > ctas * 512 * kBatch) ctas *= 2;
    const int64_t share = ceil_div(vectors, ctas);
    // many rows: CTAs small enough to hide each other's barriers
    const int threads = share <= 512 && a.k <= 64 ? 128 : (share <= 2048 || a.rows * ctas >= 4 * kSms) && a.k <= 128 ? 256 : 512;
    // at least twice as many groups as entries wanted, so that the threshold passes few others
    int log2_group = 5, log2_ctas = 0;
    while (log2_group > 0 && ctas * threads >> log2_group < 2 * a.k) --log2_group;
    while (1 << log2_ctas < ctas) ++log2_ctas;
    const int64_t pieces = ceil_div(share, static_cast<int64_t>(threads) * (16 / Vec<T>::kN));
    int log2_per = 0;
    while (ceil_div(pieces, int64_t(1) << log2_per) > kPieceMaxima) ++log2_per;
    const int slots = static_cast<int>(ceil_div(pieces, int64_t(1) << log2_per));
    const size_t smem = static_cast<size_t>(slots + 1) * threads * sizeof(typename PieceMax<T>::type);
    return launch_rows(k_topk_row<T>, a.rows * ctas, threads, ctas, smem, s, a, log2_ctas, log2_group, log2_per, slots);
}

template <typename T>
cudaError_t launch_topk(const TopArgs &a, cudaStream_t s) {
    return a.n <= kWarpMaxN && a.k <= kWarpMaxK ? launch_topk_warp<T>(a, s) : launch_topk_row<T>(a, s);
}

int check_top(int64_t rows, int64_t n, int32_t k, int dtype, double temperature) {
    if (!row_dtype_ok(dtype)) return refuse("dtype must be SPMV_F32, SPMV_F16 or SPMV_BF16");
    if (k < 1 || k > kMaxTop || k > n)
        return refuse("k must lie in [1, min(n, " + std::to_string(kMaxTop) + ")]");
    if (!(temperature > 0.0) || !(temperature <= 1e6) || temperature < 1e-6)
        return refuse("temperature must lie in [1e-6, 1e6]");
    if (rows * static_cast<int64_t>(k) >= (int64_t(1) << 40)) return set_error(SPMV_ERR_TOO_LARGE, "rows * k is too large");
    return SPMV_OK;
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" SPMV_API int spmv_topk_rows(int64_t rows, int64_t n, int32_t k, const void *x, int64_t ldx, int dtype,
                                       double temperature, int weighting, int32_t *ids, float *vals, float *weights,
                                       float *lse, void *stream) {
    SPMV_TRY(check_shape(rows, n, ldx, "x"));
    SPMV_TRY(check_top(rows, n, k, dtype, temperature));
    if (weighting < SPMV_WEIGHTS_NONE || weighting > SPMV_WEIGHTS_ROW) return refuse("no such weighting");
    if (rows == 0) return SPMV_OK;
    const int vb = row_value_bytes(dtype);
    SPMV_TRY(check_array(x, "x", vb));
    SPMV_TRY(check_array(ids, "ids", 4));
    if (vals) SPMV_TRY(check_array(vals, "vals", 4));
    if (weighting != SPMV_WEIGHTS_NONE) SPMV_TRY(check_array(weights, "weights", 4));
    if (lse) SPMV_TRY(check_array(lse, "lse", 4));
    const size_t xb = span_bytes(rows, n, ldx, vb), m = static_cast<size_t>(rows) * k * 4;
    const struct { const void *p; size_t bytes; const char *name; } out[] = {
        {ids, m, "ids"}, {vals, m, "vals"}, {weighting ? weights : nullptr, m, "weights"}, {lse, static_cast<size_t>(rows) * 4, "lse"}};
    for (int i = 0; i < 4; ++i) {
        if (out[i].p && spans_overlap(out[i].p, out[i].bytes, x, xb)) return refuse(std::string(out[i].name) + " overlaps x");
        for (int j = 0; j < i; ++j)
            if (out[i].p && out[j].p && spans_overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return refuse(std::string(out[i].name) + " overlaps " + out[j].name);
    }
    const TopArgs a{rows, n, ldx, k, weighting, static_cast<float>(1.4426950408889634 / temperature),
                    static_cast<float>(1.0 / temperature), x, ids, vals, weights, lse};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n <= kGateMaxN && k <= kGateMaxK) {
        SPMV_TRY_CUDA(launch_gate(a, dtype, s));
        return SPMV_OK;
    }
    SPMV_TRY_CUDA(dtype == SPMV_F32   ? launch_topk<float>(a, s)
                  : dtype == SPMV_F16 ? launch_topk<__half>(a, s)
                                      : launch_topk<__nv_bfloat16>(a, s));
    return SPMV_OK;
}

extern "C" SPMV_API int spmv_topk_rows_grad(int64_t rows, int64_t n, int32_t k, const int32_t *ids,
                                            const float *weights, const float *dweights, int weighting,
                                            double temperature, const void *x, int64_t ldx, const float *lse, void *dx,
                                            int64_t lddx, int dtype, void *stream) {
    SPMV_TRY(check_shape(rows, n, lddx, "dx"));
    SPMV_TRY(check_top(rows, n, k, dtype, temperature));
    if (weighting != SPMV_WEIGHTS_SELECTED && weighting != SPMV_WEIGHTS_ROW) return refuse("no such weighting, or none");
    const bool whole_row = weighting == SPMV_WEIGHTS_ROW;
    if (whole_row) SPMV_TRY(check_shape(rows, n, ldx, "x"));
    if (rows == 0) return SPMV_OK;
    const int vb = row_value_bytes(dtype);
    SPMV_TRY(check_array(ids, "ids", 4));
    SPMV_TRY(check_array(weights, "weights", 4));
    SPMV_TRY(check_array(dweights, "dweights", 4));
    SPMV_TRY(check_array(dx, "dx", vb));
    if (whole_row) {
        SPMV_TRY(check_array(x, "x", vb));
        if (lse) SPMV_TRY(check_array(lse, "lse", 4));
    }
    const size_t out = span_bytes(rows, n, lddx, vb), m = static_cast<size_t>(rows) * k * 4;
    const struct { const void *p; size_t bytes; const char *name; } in[] = {
        {ids, m, "ids"}, {weights, m, "weights"}, {dweights, m, "dweights"},
        {whole_row ? x : nullptr, span_bytes(rows, n, ldx, vb), "x"}, {whole_row ? lse : nullptr, static_cast<size_t>(rows) * 4, "lse"}};
    for (const auto &i : in)
        if (i.p && spans_overlap(dx, out, i.p, i.bytes)) return refuse(std::string("dx overlaps ") + i.name);
    // a row may start up to 15 bytes behind a 16-byte boundary: one vector more
    const int64_t pieces = ceil_div(n + 16 / vb - 1, kGradPiece);
    const TopGradArgs a{rows, n, ldx, lddx, pieces, k, weighting,
                        static_cast<float>(1.0 / temperature), ids, weights, dweights, x, dx};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n <= kGateMaxN && k <= kGateMaxK) {
        SPMV_TRY_CUDA(launch_gate_grad(a, dtype, s));
        return SPMV_OK;
    }
    const unsigned grid = static_cast<unsigned>(ceil_div(rows * pieces, 8));
    if (dtype == SPMV_F32) k_topk_grad<float><<<grid, 256, 0, s>>>(a);
    else if (dtype == SPMV_F16) k_topk_grad<__half><<<grid, 256, 0, s>>>(a);
    else k_topk_grad<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
    SPMV_TRY_CUDA(cudaGetLastError());
    return SPMV_OK;
}
