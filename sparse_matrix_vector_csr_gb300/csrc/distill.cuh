// Distillation from a teacher's top logits: the loss of a dense row of logits z against a
// target that is a sparse row of at most k entries, and its gradient.
//
//   q_i = exp(z_i / T - Z), Z = log sum exp(z / T); p_j from the teacher's logits t_j:
//   without the teacher's log-sum   p = softmax(t / T) over the entries
//       KL = sum p_j (log p_j - log q_j),  dKL/dz_i = (q_i - p_i) / T
//   with it (lse)                   p_j = exp(t_j / T - lse), r = 1 - sum p_j, one more class
//       that holds every other column, of probability r and 1 - S (S = sum of the entries' q):
//       KL + r (log r - log(1 - S)),  dKL/dz_i = (q_i - p_i) / T at the entries,
//       q_i (1 - r / (1 - S)) / T elsewhere.
// 1 - S is the sum of q over the other columns, never a difference, and has a maximum of its own
// (the student may put nearly everything on the entries): a bit per value of the row marks the
// entries' columns, which the row's sums then leave out; the entries' own sum joins at the end.
//
// The row is what costs: V values read, V written.  Long rows pass through the registers twice,
// once for the sums (maximum and sum together, rescaled when a thread's maximum grows) and once for
// the gradient, the second time from L2 and from the end.  Few rows are shared by a cluster of CTAs
// each, in registers where they fit, which exchange their warps' sums through distributed shared
// memory; many short rows take a warp each.  The entries (at most kMaxEntries) are the business of each CTA's
// last warp while the others read the row.
#pragma once

#include "rows_common.cuh"

namespace spmv {
namespace rows {

constexpr int kMaxEntries = 512;
constexpr int64_t kMaxVocab = int64_t(1) << 22;
// A remainder of the teacher's mass below this is the rounding of 32-bit logits and of lse; it
// only matters where the student's mass on the other columns is 0 in 32 bits (masked by -inf or by the
// type's lowest value: 1e-7 of 1e38 would be the loss), and counts as 0 there (see rest_of).
constexpr float kRestRounding = 1e-5f;

enum DistillMode { kLoss = 0, kLossGrad = 1, kGrad = 2 };

struct DistillArgs {
    int64_t rows, n, ldz, lddz;
    int k, teacher_dtype;
    float inv_temperature, scale2;  // scale2 = log2(e) / T
    float scale;                    // of the gradient, with row_scale
    const void *z;
    const int32_t *ids;
    const void *teacher;
    const float *teacher_lse, *row_scale;
    float *loss;
    float4 *stats;  // per row, for the gradient: see RowFactors
    void *dz;
};

// What a row's entries give: sum p log p, sum p, r (0 without lse), how many there are (0: no target).
struct EntryScalars {
    float entropy, mass, rest;
    int valid;
};

// A CTA's shared memory (dynamic, no larger than the call needs: L1 has the rest for the loads in
// flight).  With slots for the batches that a row read twice keeps; per warp of the cluster its
// columns' maximum and sum (with lse: of those that are no entries, and in z, w of its CTA's entries,
// from its last warp); the entries' columns (-1: none), probabilities and z (see load_entries);
// with lse a byte per vector of the CTA's share, a bit per value.
struct DistillShared {
    uint4 *keep;
    float4 *part;
    EntryScalars *sc;
    int32_t *id;
    float *p, *z;
    uint32_t *marks;
    __host__ __device__ static int padded(int k) { return (k + 3) & ~3; }
    __device__ DistillShared(unsigned char *mem, int keep_slots, int parts, int k) {
        keep = reinterpret_cast<uint4 *>(mem);
        part = reinterpret_cast<float4 *>(keep + keep_slots);
        sc = reinterpret_cast<EntryScalars *>(part + parts);
        id = reinterpret_cast<int32_t *>(sc + 1);
        p = reinterpret_cast<float *>(id + padded(k));
        z = p + padded(k);
        marks = reinterpret_cast<uint32_t *>(z + padded(k));
    }
    static size_t bytes(int64_t keep_slots, int parts, int k, int64_t marks) {
        return static_cast<size_t>(16 * (keep_slots + parts + 1) + 12 * padded(k) + (marks + 3) / 4 * 4);
    }
};

// One warp: the entries' probabilities, and z at those of columns [e0, e1) (the CTA's own, or all
// for the CTA that sums the loss).
template <typename T>
__device__ __forceinline__ void load_entries(const DistillArgs &a, int32_t *sid, float *sp, float *sz, EntryScalars &sc,
                                             int64_t r, const T *z, int64_t e0, int64_t e1) {
    const int lane = threadIdx.x & 31;
    const int32_t *ids = a.ids + r * a.k;
    float top = kNegInf;
    int valid = 0;
    for (int j = lane; j < a.k; j += 32) {
        int32_t id = ids[j];
        float t = kNegInf;
        if (id >= 0 && id < a.n) {
            t = load_any(a.teacher, r * a.k + j, a.teacher_dtype);
            ++valid;
            if (id >= e0 && id < e1) sz[j] = to_f32(z[id]);
        } else {
            id = -1;
        }
        sid[j] = id;
        sp[j] = t;
        top = fmaxf(top, t);
    }
    valid = warp_sum(valid);
    top = reference_of(warp_max(top));
    float log_norm, shift;
    if (a.teacher_lse) {
        shift = 0.0f;
        log_norm = a.teacher_lse[r];
    } else {
        float s = 0.0f;
        for (int j = lane; j < a.k; j += 32) s += expf((sp[j] - top) * a.inv_temperature);
        shift = top;
        log_norm = logf(warp_sum(s));
    }
    float entropy = 0.0f, mass = 0.0f;
    for (int j = lane; j < a.k; j += 32) {
        const float lp = fmaf(sp[j] - shift, a.inv_temperature, -log_norm);
        const float p = sp[j] == kNegInf ? 0.0f : expf(lp);
        if (p > 0.0f || p != p) entropy = fmaf(p, lp, entropy);
        mass += p;
        sp[j] = p;
    }
    entropy = warp_sum(entropy);
    mass = warp_sum(mass);
    if (lane == 0) {
        // no entry, or (without lse) none above -inf: no target, nothing to learn
        sc.valid = valid && (a.teacher_lse || log_norm != kNegInf) ? valid : 0;
        sc.entropy = entropy;
        sc.mass = mass;
        sc.rest = a.teacher_lse && valid < a.n ? fmaxf(0.0f, 1.0f - mass) : 0.0f;
    }
}

// -inf in the places of the marked values
template <typename T>
__device__ __forceinline__ void mask_vec(uint4 &v, uint32_t marked) {
    if (marked) {
        float x[Vec<T>::kN];
        unpack<T>(v, x);
#pragma unroll
        for (int i = 0; i < Vec<T>::kN; ++i)
            if (marked >> i & 1) x[i] = kNegInf;
        v = pack<T>(x);
    }
}

// scale_signed * exp2((x - ref) scale2) of a vector.  16-bit results take the factor's logarithm
// into the exponent (one operation less a value, its rounding far below theirs).
template <typename T>
struct GradOf {
    float ref, scale2, factor, log_factor;
    uint32_t flip;  // the factor's sign, for both values of a word
    __device__ __forceinline__ GradOf(float ref_, float scale2_, float factor_)
        : ref(ref_), scale2(scale2_), factor(factor_), log_factor(log2f(fabsf(factor_))), flip(factor_ < 0.0f ? 0x80008000u : 0u) {}
    __device__ __forceinline__ uint4 operator()(const uint4 &v) const {
        float x[Vec<T>::kN];
        unpack<T>(v, x);
#pragma unroll
        for (int i = 0; i < Vec<T>::kN; i += 2) {
            float2 d = add2(make_float2(x[i], x[i + 1]), both(-ref));
            if constexpr (sizeof(T) == 2) {
                d = fma2(d, both(scale2), both(log_factor));
                x[i] = ex2(d.x);
                x[i + 1] = ex2(d.y);
            } else {
                d = mul2(d, both(scale2));
                d = mul2(make_float2(ex2(d.x), ex2(d.y)), both(factor));
                x[i] = d.x;
                x[i + 1] = d.y;
            }
        }
        uint4 o = pack<T>(x);
        if constexpr (sizeof(T) == 2) o = make_uint4(o.x ^ flip, o.y ^ flip, o.z ^ flip, o.w ^ flip);
        return o;
    }
};

// A row's maximum and sum of exponentials (of z / T): of all columns, and with lse of those that
// are no entries.
struct RowSums {
    float m, sum, m_rest, rest_sum;
};

// A warp joins the parts of all warps that share the row; a part without a value above -inf adds
// its 0 (or a NaN).
__device__ __forceinline__ RowSums join_parts(const DistillArgs &a, const float4 *parts, int n) {
    const int lane = threadIdx.x & 31;
    const bool tail = a.teacher_lse != nullptr;
    const auto scaled = [&](float part, float from, float to) {
        return from == kNegInf ? part : part * ex2((from - to) * a.scale2);
    };
    RowSums s;
    s.m_rest = kNegInf;
    float em = kNegInf;
    for (int i = lane; i < n; i += 32) {
        s.m_rest = fmaxf(s.m_rest, parts[i].x);
        em = fmaxf(em, parts[i].z);
    }
    s.m_rest = warp_max(s.m_rest);
    s.m = reference_of(fmaxf(s.m_rest, tail ? warp_max(em) : kNegInf));
    s.m_rest = reference_of(s.m_rest);
    float es = 0.0f;
    s.rest_sum = 0.0f;
    for (int i = lane; i < n; i += 32) {
        const float4 w = parts[i];
        s.rest_sum += scaled(w.y, w.x, s.m_rest);
        es += scaled(w.w, w.z, s.m);
    }
    s.rest_sum = warp_sum(s.rest_sum);
    s.sum = s.rest_sum;
    if (tail) s.sum = warp_sum(es) + (s.rest_sum != 0.0f ? scaled(s.rest_sum, s.m_rest, s.m) : 0.0f);
    return s;
}

// the same for one warp that has the whole row: its columns (with lse: the others), the entries
__device__ __forceinline__ RowSums join_two(const DistillArgs &a, float m_rest, float rest_sum, float em, float es) {
    const bool tail = a.teacher_lse != nullptr;
    RowSums s;
    s.m = reference_of(fmaxf(m_rest, em));
    s.rest_sum = rest_sum;
    s.sum = rest_sum;
    if (tail) s.sum = (em == kNegInf ? es : es * ex2((em - s.m) * a.scale2)) + (m_rest == kNegInf ? rest_sum : rest_sum * ex2((m_rest - s.m) * a.scale2));
    s.m_rest = reference_of(m_rest);
    return s;
}

// The remainder that counts.  A rest_sum is relative to m_rest, so it is 0 under a mask of -inf alone.
__device__ __forceinline__ float rest_of(const DistillArgs &a, const EntryScalars &sc, const RowSums &s) {
    const bool none = s.rest_sum == 0.0f || ex2((s.m_rest - s.m) * a.scale2) == 0.0f;
    return sc.rest < kRestRounding && none ? 0.0f : sc.rest;
}

// What a row's gradient takes of it: q_i = inv_sum exp((z_i - m) / T) at the entries (less p_i), and
// elsewhere other exp((z_i - ref) / T): q_i, and with lse q_i - r q'_i, q' the softmax over the
// other columns.  All factors 0: no target, no gradient.  The loss leaves it for a gradient
// that is taken later, which so need not wait for the row's entries.
struct RowFactors {
    float ref, other, m, inv_sum;
    __device__ __forceinline__ explicit RowFactors(const float4 &s) : ref(s.x), other(s.y), m(s.z), inv_sum(s.w) {}
    __device__ __forceinline__ RowFactors(const DistillArgs &a, const EntryScalars &sc, const RowSums &s)
        : ref(s.m), other(0.0f), m(s.m), inv_sum(0.0f) {
        if (!sc.valid) return;
        other = inv_sum = 1.0f / s.sum;
        if (a.teacher_lse) {
            ref = s.m_rest;
            other = s.rest_sum != 0.0f ? ex2((s.m_rest - s.m) * a.scale2) / s.sum - rest_of(a, sc, s) / s.rest_sum : 0.0f;
        }
    }
    __device__ __forceinline__ bool live() const { return inv_sum != 0.0f || other != 0.0f; }
    __device__ __forceinline__ float at_entry(const DistillArgs &a, float g, float p, float z) const {
        return g * fmaf(ex2((z - m) * a.scale2), inv_sum, -p);
    }
};
__device__ __forceinline__ float row_gain(const DistillArgs &a, int64_t r) {
    return a.scale * (a.row_scale ? a.row_scale[r] : 1.0f) * a.inv_temperature;
}

// One warp sums the loss over the entries (z: all of them).
__device__ __forceinline__ void write_loss(const DistillArgs &a, int64_t r, const int32_t *id, const float *p,
                                           const float *z, const EntryScalars &sc, const RowSums &s) {
    const int lane = threadIdx.x & 31;
    float cross = 0.0f;  // sum p (z - m)
    for (int j = lane; j < a.k; j += 32)
        if (id[j] >= 0 && p[j] != 0.0f) cross = fmaf(p[j], z[j] - s.m, cross);
    cross = warp_sum(cross);
    if (lane == 0) {
        const float log_sum = logf(s.sum);
        float loss = sc.entropy - cross * a.inv_temperature + sc.mass * log_sum;
        const float rest = rest_of(a, sc, s);
        if (rest > 0.0f)  // (the distance times rest first: a mask's may be near the largest float)
            loss += rest * (logf(rest) - logf(s.rest_sum) + log_sum) + rest * (s.m - s.m_rest) * a.inv_temperature;
        a.loss[r] = sc.valid ? loss : 0.0f;
        if (a.stats) {
            const RowFactors f(a, sc, s);
            a.stats[r] = make_float4(f.ref, f.other, f.m, f.inv_sum);
        }
    }
}

constexpr int kBatchVectors = 4;  // in flight per thread where the row does not fit its registers
constexpr int kPrefetch = 8;      // vectors of a thread that L2 fetches first (16: no faster)
constexpr int kKeepBatches = 2;   // of a row that is read twice: 61 KB of a CTA's shared memory

// kR: vectors of a thread in registers, 0: batches from memory.  Bound by DRAM: 8192 x 131072 bf16 rows,
// 64 entries, loss and gradient in 752 us, 5.7 TB/s of z and dz (a copy runs at 6.7); with its
// arithmetic left out the same reads and writes took 95 % of the time.  What misses is the part
// of the rows in flight that L2 has dropped before the second reading (7 % of z).  The gradient
// alone 5.1 TB/s, the loss alone 5.2: the chain of loads behind a row's entries and the barrier,
// which other CTAs of the SM hide in part, so as many are resident as registers allow (loss 61 us
// at 64 registers, 52 at 32; two readings want fewer rows in flight: 900 us at 40, 813 at 64).
template <typename T, int kR, int kMode>
__global__ void __launch_bounds__(512, kR > 0 || kMode == kLossGrad ? 2 : kMode == kGrad ? 3 : 4) k_distill(DistillArgs a, int log2_ctas) {
    constexpr int kN = Vec<T>::kN;
    constexpr int kU = kBatchVectors;
    constexpr int kKeep = kR == 0 && kMode == kLossGrad ? kKeepBatches : 0;
    extern __shared__ __align__(16) unsigned char dynamic_mem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
    const int workers = blockDim.x - 32;
    const bool entry_warp = tid >= workers;
    const int ctas = 1 << log2_ctas;
    const DistillShared sh(dynamic_mem, kU * kKeep * workers, ctas * n_warps, a.k);
    uint4 *const keep = sh.keep + tid;
    uint32_t *const marks_mem = sh.marks;
    const int64_t r = blockIdx.x >> log2_ctas;
    const uint32_t rank = blockIdx.x & (ctas - 1);
    const T *z = static_cast<const T *>(a.z) + r * a.ldz;
    const RowView<T> row(z, a.n);
    const Share<T> share(row, rank, log2_ctas);
    const bool tail = a.teacher_lse != nullptr;
    const auto own = [&](int32_t id) { return id >= 0 && share.owns(id); };
    uint4 reg[kR > 0 ? kR : 1];
    if constexpr (kR > 0)
        if (!entry_warp) load_share<T, kR>(share, tid, workers, reg);
    if (kR == 0 && kMode == kGrad && !entry_warp) {
        // the row waits for its factors: L2 meanwhile fetches
#pragma unroll
        for (int i = 0; i < kPrefetch; ++i)
            if (share.whole(i * workers + tid)) asm volatile("prefetch.global.L2 [%0];" ::"l"(share.vec + i * workers + tid));
    }
    if (kMode != kGrad && ctas > 1) cluster_arrive();  // the peers' shared memory may be written ...
    const uint8_t *marks = reinterpret_cast<const uint8_t *>(marks_mem);
    if (kMode != kGrad && tail) {
        // marked from the ids alone: the row waits for nothing else of its entries
        int32_t id = tid < a.k ? a.ids[r * a.k + tid] : -1;
        for (int i = tid; i < (share.count + 3) / 4; i += blockDim.x) marks_mem[i] = 0;
        __syncthreads();
        for (int j = tid; j < a.k; j += blockDim.x) {
            if (j != tid) id = a.ids[r * a.k + j];
            if (id < a.n && own(id)) {
                const uint32_t at = static_cast<uint32_t>(id - share.e0), byte = at / kN;
                atomicOr(&marks_mem[byte / 4], 1u << (byte % 4 * 8 + at % kN));
            }
        }
        __syncthreads();
    }
    if (entry_warp) {
        const bool sums_loss = kMode != kGrad && rank == 0;
        load_entries<T>(a, sh.id, sh.p, sh.z, *sh.sc, r, z, sums_loss ? 0 : share.e0, sums_loss ? a.n : share.first(share.count));
    }

    RowSums sums;
    if constexpr (kMode != kGrad) {
        float wm = kNegInf, ws = 0.0f, em = kNegInf, es = 0.0f;
        if (!entry_warp) {
            if constexpr (kR > 0) {
                if (tail) {
#pragma unroll
                    for (int i = 0; i < kR; ++i)
                        if (i * workers + tid < share.count) mask_vec<T>(reg[i], marks[i * workers + tid]);
                }
#pragma unroll
                for (int i = 0; i < kR; ++i) wm = fmaxf(wm, vec_max(reg[i], T()));
                wm = warp_max(wm);
                const float w0 = reference_of(wm);
                float2 s2 = both(0.0f);
#pragma unroll
                for (int i = 0; i < kR; ++i) s2 = exp_sum<T>(reg[i], w0, a.scale2, s2);
                ws = s2.x + s2.y;
            } else {
                Running run;
                stream_share<T, kU, kMode == kLoss, kKeep>(share, tid, workers, keep, [&](uint4 *x, int v, int have) {
                    if (tail) {
#pragma unroll
                        for (int i = 0; i < kU; ++i)
                            if (i < have) mask_vec<T>(x[i], marks[v + i * workers]);
                    }
                    run.add<T, kU>(x, a.scale2);
                });
                wm = warp_max(run.m);
                ws = run.sum();
                if (run.m != kNegInf) ws *= ex2((run.m - wm) * a.scale2);
            }
        } else if (tail) {
            for (int j = lane; j < a.k; j += 32)
                if (own(sh.id[j])) em = fmaxf(em, sh.z[j]);
            em = warp_max(em);
            const float m0 = reference_of(em);
            for (int j = lane; j < a.k; j += 32)
                if (own(sh.id[j])) es += ex2((sh.z[j] - m0) * a.scale2);
            es = warp_sum(es);
        }
        ws = warp_sum(ws);
        if (ctas > 1) cluster_wait();  // ... once they have started
        if (lane < ctas) {
            float4 *slot = &sh.part[rank * n_warps + warp];
            if (ctas > 1) peer_store4(peer_addr(slot, lane), wm, ws, em, es);
            else *slot = make_float4(wm, ws, em, es);
        }
        cluster_sync(ctas);
        sums = join_parts(a, sh.part, n_warps * ctas);
        if (rank == 0 && entry_warp) write_loss(a, r, sh.id, sh.p, sh.z, *sh.sc, sums);
    } else if (a.dz == a.z) {
        __syncthreads();  // in place: z at the entries is read before any of the row is written
    }

    if constexpr (kMode != kLoss) {
        const RowFactors rf = kMode == kGrad ? RowFactors(a.stats[r]) : RowFactors(a, *sh.sc, sums);
        const bool live = rf.live();
        const float g = row_gain(a, r);
        T *dz = static_cast<T *>(a.dz) + r * a.lddz;
        const bool congruent = ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
        if (!entry_warp) {
            if (!live) {
                const uint4 zero = splat<T>(0.0f);
                for (int v = tid; v < share.count; v += workers) share.store(dz, v, zero, congruent);
            } else {
                const GradOf<T> grad(rf.ref, a.scale2, g * rf.other);
                if constexpr (kR > 0) {
#pragma unroll
                    for (int i = 0; i < kR; ++i)
                        if (i * workers + tid < share.count) share.store(dz, i * workers + tid, grad(reg[i]), congruent);
                } else {
                    const auto put = [&](uint4 *x, int v, int have) {
#pragma unroll
                        for (int i = 0; i < kU; ++i)
                            if (i < have) share.store(dz, v + i * workers, grad(x[i]), congruent);
                    };
                    if constexpr (kMode == kGrad) stream_share<T, kU, true, 0>(share, tid, workers, keep, put);
                    else stream_back<T, kU, kKeep>(share, tid, workers, keep, put);
                }
            }
        }
        __syncthreads();  // the entries' columns are written after the plain stores
        if (live)
            for (int j = tid; j < a.k; j += blockDim.x) {
                const int32_t id = sh.id[j];
                if (own(id)) dz[id] = from_f32<T>(rf.at_entry(a, g, sh.p[j], sh.z[j]));
            }
    }
}

// Many short rows: a warp per row, its registers hold it, no barrier.  12832 rows of 500 float values
// with 127 entries, loss and gradient: 31 us (a CTA per row spends 6 to 8 us on a row's latencies:
// 84 us).  Bound by the instructions of the entries and of the row's sums.
constexpr int kWarpRows = 4;  // per CTA
template <typename T, int kR, int kMode>
__global__ void __launch_bounds__(32 * kWarpRows, kR == 4 ? 8 : kR == 8 ? 5 : 3) k_distill_warp(DistillArgs a, int k_padded, int mark_words) {
    constexpr int kN = Vec<T>::kN;
    extern __shared__ __align__(16) unsigned char dynamic_mem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarpRows + warp;
    if (r >= a.rows) return;
    EntryScalars &sc = reinterpret_cast<EntryScalars *>(dynamic_mem)[warp];
    int32_t *id = reinterpret_cast<int32_t *>(reinterpret_cast<EntryScalars *>(dynamic_mem) + kWarpRows) + warp * k_padded;
    float *p = reinterpret_cast<float *>(id + (kWarpRows - warp) * k_padded) + warp * k_padded, *zk = p + kWarpRows * k_padded;
    uint32_t *marks = reinterpret_cast<uint32_t *>(zk + (kWarpRows - warp) * k_padded) + warp * mark_words;
    const T *z = static_cast<const T *>(a.z) + r * a.ldz;
    const Share<T> share(RowView<T>(z, a.n), uint32_t(0), 0);
    const bool tail = a.teacher_lse != nullptr;
    uint4 reg[kR];
    load_share<T, kR>(share, lane, 32, reg);
    if (kMode != kGrad && tail)
        for (int i = lane; i < mark_words; i += 32) marks[i] = 0;
    load_entries<T>(a, id, p, zk, sc, r, z, 0, a.n);
    __syncwarp();
    RowSums sums;
    if constexpr (kMode != kGrad) {
        float em = kNegInf, es = 0.0f;
        if (tail) {
            for (int j = lane; j < a.k; j += 32)
                if (id[j] >= 0) {
                    const uint32_t at = static_cast<uint32_t>(id[j] - share.e0), byte = at / kN;
                    atomicOr(&marks[byte / 4], 1u << (byte % 4 * 8 + at % kN));
                    em = fmaxf(em, zk[j]);
                }
            em = warp_max(em);
            const float m0 = reference_of(em);
            for (int j = lane; j < a.k; j += 32)
                if (id[j] >= 0) es += ex2((zk[j] - m0) * a.scale2);
            es = warp_sum(es);
            __syncwarp();
            const uint8_t *bytes = reinterpret_cast<const uint8_t *>(marks);
#pragma unroll
            for (int i = 0; i < kR; ++i)
                if (i * 32 + lane < share.count) mask_vec<T>(reg[i], bytes[i * 32 + lane]);
        }
        uint4 top = reg[0];
#pragma unroll
        for (int i = 1; i < kR; ++i) top = vec_max2(top, reg[i], T());
        const float wm = warp_max(vec_max(top, T()));
        const float w0 = reference_of(wm);
        float2 s2 = both(0.0f);
#pragma unroll
        for (int i = 0; i < kR; ++i) s2 = exp_sum<T>(reg[i], w0, a.scale2, s2);
        sums = join_two(a, wm, warp_sum(s2.x + s2.y), em, es);
        write_loss(a, r, id, p, zk, sc, sums);
    }
    if constexpr (kMode != kLoss) {
        const RowFactors rf = kMode == kGrad ? RowFactors(a.stats[r]) : RowFactors(a, sc, sums);
        const float g = row_gain(a, r);
        T *dz = static_cast<T *>(a.dz) + r * a.lddz;
        const bool live = rf.live(), congruent = ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
        const GradOf<T> grad(rf.ref, a.scale2, g * rf.other);
#pragma unroll
        for (int i = 0; i < kR; ++i)
            if (i * 32 + lane < share.count) share.store(dz, i * 32 + lane, live ? grad(reg[i]) : splat<T>(0.0f), congruent);
        __syncwarp();  // the entries' columns are written after the plain stores
        if (live)
            for (int j = lane; j < a.k; j += 32)
                if (id[j] >= 0) dz[id[j]] = from_f32<T>(rf.at_entry(a, g, p[j], zk[j]));
    }
}

constexpr int kWarpVectors = 512;  // a warp's registers hold up to this
template <typename T, int kMode>
cudaError_t launch_distill_warp(int64_t vectors, const DistillArgs &a, cudaStream_t s) {
    const int k_padded = (a.k + 3) / 4 * 4;
    const int mark_words = kMode != kGrad && a.teacher_lse ? static_cast<int>(ceil_div(vectors, 4)) : 0;
    const size_t smem = kWarpRows * (sizeof(EntryScalars) + static_cast<size_t>(12) * k_padded + static_cast<size_t>(4) * mark_words);
    const int64_t grid = ceil_div(a.rows, kWarpRows);
    if (vectors <= 4 * 32) return launch_rows(k_distill_warp<T, 4, kMode>, grid, 32 * kWarpRows, 1, smem, s, a, k_padded, mark_words);
    if (vectors <= 8 * 32) return launch_rows(k_distill_warp<T, 8, kMode>, grid, 32 * kWarpRows, 1, smem, s, a, k_padded, mark_words);
    return launch_rows(k_distill_warp<T, 16, kMode>, grid, 32 * kWarpRows, 1, smem, s, a, k_padded, mark_words);
}

template <typename T, int kR, int kMode>
cudaError_t launch_distill_shape(const RowShape &shape, int64_t vectors, const DistillArgs &a, cudaStream_t s) {
    auto *kernel = k_distill<T, kR, kMode>;
    const int64_t keep = kR == 0 && kMode == kLossGrad ? static_cast<int64_t>(kBatchVectors) * kKeepBatches * (shape.threads - 32) : 0;
    const int64_t marks = kMode != kGrad && a.teacher_lse ? ceil_div(vectors, shape.ctas) : 0;
    const size_t smem = DistillShared::bytes(keep, shape.ctas * shape.threads / 32, a.k, marks);
    if (smem > 48 * 1024) {  // (always the same limit: another thread's call may set it at the same time)
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
    }
    // the gradient alone needs no exchange: its CTAs are no cluster
    return launch_rows(kernel, a.rows * shape.ctas, shape.threads, kMode == kGrad ? 1 : shape.ctas, smem, s, a, shape.log2_ctas());
}

template <typename T, int kMode>
cudaError_t launch_distill_mode(const DistillArgs &a, cudaStream_t s) {
    const int64_t vectors = row_vectors<T>(a.n, a.z, a.ldz);
    // Many rows are eight an SM or more.  us for loss and gradient, the loss alone, with a warp / a
    // CTA (below 152 rows a cluster) a row, 32 entries:
    //   rows    500 floats               4000 bf16 values
    //   608     4.8, 3.4 / 5.8, 4.2      8.5, 3.8 / 7.1, 4.6
    //   1215    4.9, 3.6 / 6.8, 5.0      8.9, 4.4 / 9.9, 5.9
    //   1824    5.1, 3.8 / 10.2, 6.2     9.5, 4.9 / 15.0, 7.5
    //   16384   19.8, 12.4 / 70.8, 32.7  76.4, 33.9 / 103, 44.2
    if (vectors <= kWarpVectors && a.rows >= 1216) return launch_distill_warp<T, kMode>(vectors, a, s);
    RowShape shape = row_shape(a.rows, vectors, kMode == kLossGrad);
    // with lse a CTA keeps a byte per vector of its share (2^22 float values: a cluster of 8)
    if (kMode != kGrad && a.teacher_lse)
        while (shape.ctas < kMaxCluster && ceil_div(vectors, shape.ctas) > 140 * 1024) shape.ctas *= 2;
    switch (shape.regs) {
        case 2: return launch_distill_shape<T, 2, kMode>(shape, vectors, a, s);
        case 4: return launch_distill_shape<T, 4, kMode>(shape, vectors, a, s);
        case 8: return launch_distill_shape<T, 8, kMode>(shape, vectors, a, s);
        default: return launch_distill_shape<T, 0, kMode>(shape, vectors, a, s);
    }
}

template <typename T>
cudaError_t launch_distill(DistillMode mode, const DistillArgs &a, cudaStream_t s) {
    if (mode == kLoss) return launch_distill_mode<T, kLoss>(a, s);
    if (mode == kLossGrad) return launch_distill_mode<T, kLossGrad>(a, s);
    return launch_distill_mode<T, kGrad>(a, s);
}

cudaError_t launch_distill_f32(DistillMode mode, const DistillArgs &a, cudaStream_t s);
cudaError_t launch_distill_f16(DistillMode mode, const DistillArgs &a, cudaStream_t s);
cudaError_t launch_distill_bf16(DistillMode mode, const DistillArgs &a, cudaStream_t s);

}  // namespace rows
}  // namespace spmv
