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
// the gradient, the second time from L2; rows that fit the registers of a CTA stay there.  Few
// rows are shared by a cluster of CTAs each, which exchange their warps' sums through
// distributed shared memory.  The entries (at most kMaxEntries) are the business of each CTA's
// last warp while the others read the row.
#pragma once

#include "rows_common.cuh"

namespace spmv {
namespace rows {

constexpr int kMaxEntries = 512;
constexpr int64_t kMaxVocab = int64_t(1) << 22;
// A remainder of the teacher's mass below this is the rounding of 32-bit logits and of lse; it
// only matters where the student has no mass on the other columns at all, and counts as 0 there.
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
    float4 *stats;  // per row: m, sum exp((z - m) / T) over all columns; with lse the same of the others
    void *dz;
};

struct DistillShared {
    // per warp of the cluster: maximum and sum of its columns (with lse: of those that are no
    // entries, and in z, w of its CTA's entries, from its last warp)
    float4 warp_part[kMaxCluster * 16];
    int32_t id[kMaxEntries];             // column, or -1
    float p[kMaxEntries], z[kMaxEntries];  // z: see load_entries
    float entropy, mass, rest;           // sum p log p, sum p, r (0 without lse)
    int valid;
};

// One warp: the entries' probabilities, and z at those of columns [e0, e1) (the CTA's own, or all
// for the CTA that sums the loss).
template <typename T>
__device__ __forceinline__ void load_entries(const DistillArgs &a, DistillShared &sh, int64_t r, const T *z, int64_t e0,
                                             int64_t e1) {
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
            if (id >= e0 && id < e1) sh.z[j] = to_f32(z[id]);
        } else {
            id = -1;
        }
        sh.id[j] = id;
        sh.p[j] = t;
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
        for (int j = lane; j < a.k; j += 32) s += expf((sh.p[j] - top) * a.inv_temperature);
        shift = top;
        log_norm = logf(warp_sum(s));
    }
    float entropy = 0.0f, mass = 0.0f;
    for (int j = lane; j < a.k; j += 32) {
        const float lp = fmaf(sh.p[j] - shift, a.inv_temperature, -log_norm);
        const float p = sh.p[j] == kNegInf ? 0.0f : expf(lp);
        if (p > 0.0f || p != p) entropy = fmaf(p, lp, entropy);
        mass += p;
        sh.p[j] = p;
    }
    entropy = warp_sum(entropy);
    mass = warp_sum(mass);
    if (lane == 0) {
        // no entry, or (without lse) none above -inf: no target, nothing to learn
        sh.valid = valid && (a.teacher_lse || log_norm != kNegInf) ? valid : 0;
        sh.entropy = entropy;
        sh.mass = mass;
        sh.rest = a.teacher_lse && valid < a.n ? fmaxf(0.0f, 1.0f - mass) : 0.0f;
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

constexpr int kBatchVectors = 4;  // in flight per thread where the row does not fit its registers
constexpr int kKeepBatches = 2;   // of a row that is read twice: 92 KB of a CTA's shared memory

template <typename T, int kR, int kMode>
__global__ void __launch_bounds__(512, kR > 0 || kMode == kLossGrad ? 2 : kMode == kGrad ? 3 : 4) k_distill(DistillArgs a, int log2_ctas) {
    constexpr int kN = Vec<T>::kN;
    constexpr int kU = kBatchVectors;
    __shared__ DistillShared sh;
    constexpr int kKeep = kR == 0 && kMode == kLossGrad ? kKeepBatches : 0;
    extern __shared__ __align__(16) unsigned char dynamic_mem[];
    uint4 *keep = reinterpret_cast<uint4 *>(dynamic_mem) + threadIdx.x;
    // with lse: a byte per vector of the CTA's share, a bit per value
    uint32_t *marks_mem = reinterpret_cast<uint32_t *>(dynamic_mem + static_cast<size_t>(16) * kU * kKeep * (blockDim.x - 32));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
    const int workers = blockDim.x - 32;
    const bool entry_warp = tid >= workers;
    const int ctas = 1 << log2_ctas;
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
        load_entries<T>(a, sh, r, z, sums_loss ? 0 : share.e0, sums_loss ? a.n : share.first(share.count));
    }

    // of all columns; of the others (with lse)
    float m, sum, m_rest = 0.0f, rest_sum = 0.0f;
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
            float4 *slot = &sh.warp_part[rank * n_warps + warp];
            if (ctas > 1) peer_store4(peer_addr(slot, lane), wm, ws, em, es);
            else *slot = make_float4(wm, ws, em, es);
        }
        cluster_sync(ctas);
        // every warp joins all warps' sums; a part without a value above -inf adds its 0 (or a NaN)
        const auto scaled = [&](float part, float from, float to) {
            return from == kNegInf ? part : part * ex2((from - to) * a.scale2);
        };
        m_rest = kNegInf;
        em = kNegInf;
        for (int i = lane; i < n_warps * ctas; i += 32) {
            m_rest = fmaxf(m_rest, sh.warp_part[i].x);
            em = fmaxf(em, sh.warp_part[i].z);
        }
        m_rest = warp_max(m_rest);
        m = reference_of(fmaxf(m_rest, tail ? warp_max(em) : kNegInf));
        m_rest = reference_of(m_rest);
        es = 0.0f;
        for (int i = lane; i < n_warps * ctas; i += 32) {
            const float4 w = sh.warp_part[i];
            rest_sum += scaled(w.y, w.x, m_rest);
            es += scaled(w.w, w.z, m);
        }
        rest_sum = warp_sum(rest_sum);
        sum = rest_sum;
        if (tail) sum = warp_sum(es) + (rest_sum != 0.0f ? scaled(rest_sum, m_rest, m) : 0.0f);
        if (rank == 0 && entry_warp) {
            float cross = 0.0f;  // sum p (z - m)
            for (int j = lane; j < a.k; j += 32)
                if (sh.id[j] >= 0 && sh.p[j] != 0.0f) cross = fmaf(sh.p[j], sh.z[j] - m, cross);
            cross = warp_sum(cross);
            if (lane == 0) {
                const float log_sum = logf(sum), rest = sh.rest;
                float loss = sh.entropy - cross * a.inv_temperature + sh.mass * log_sum;
                if (rest > 0.0f && !(rest < kRestRounding && rest_sum == 0.0f))
                    loss += rest * (logf(rest) - logf(rest_sum) + log_sum + (m - m_rest) * a.inv_temperature);
                a.loss[r] = sh.valid ? loss : 0.0f;
                if (a.stats) a.stats[r] = make_float4(m, sum, m_rest, rest_sum);
            }
        }
    } else {
        __syncthreads();
        const float4 st = a.stats[r];
        m = st.x;
        sum = st.y;
        m_rest = st.z;
        rest_sum = st.w;
    }

    if constexpr (kMode != kLoss) {
        const bool live = sh.valid != 0;
        const float g = a.scale * (a.row_scale ? a.row_scale[r] : 1.0f) * a.inv_temperature;
        const float q_scale = g / sum;
        // elsewhere than at the entries: g q, and with lse g (q - r q_other), q_other the softmax
        // over the other columns; both are multiples of exp((z - m_rest) / T)
        float ref = m, o_scale = q_scale;
        if (tail) {
            ref = m_rest;
            o_scale = rest_sum != 0.0f ? g * (ex2((m_rest - m) * a.scale2) / sum - sh.rest / rest_sum) : 0.0f;
        }
        T *dz = static_cast<T *>(a.dz) + r * a.lddz;
        const bool congruent = ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
        if (!entry_warp) {
            if (!live) {
                const uint4 zero = splat<T>(0.0f);
                for (int v = tid; v < share.count; v += workers) share.store(dz, v, zero, congruent);
            } else {
                const GradOf<T> grad(ref, a.scale2, o_scale);
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
                if (own(id)) dz[id] = from_f32<T>(fmaf(ex2((sh.z[j] - m) * a.scale2), q_scale, -sh.p[j] * g));
            }
    }
}

template <typename T, int kR, int kMode>
cudaError_t launch_distill_shape(const RowShape &shape, int64_t vectors, const DistillArgs &a, cudaStream_t s) {
    auto *kernel = k_distill<T, kR, kMode>;
    size_t smem = kR == 0 && kMode == kLossGrad ? static_cast<size_t>(16) * kBatchVectors * kKeepBatches * (shape.threads - 32) : 0;
    if (kMode != kGrad && a.teacher_lse) smem += static_cast<size_t>(ceil_div(ceil_div(vectors, shape.ctas), 4) * 4);
    if (smem + sizeof(DistillShared) > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    // the gradient alone needs no exchange: its CTAs are no cluster
    return launch_rows(kernel, a.rows * shape.ctas, shape.threads, kMode == kGrad ? 1 : shape.ctas, smem, s, a, shape.log2_ctas());
}

template <typename T, int kMode>
cudaError_t launch_distill_mode(const DistillArgs &a, cudaStream_t s) {
    const int64_t vectors = row_vectors<T>(a.n, a.z, a.ldz);
    const RowShape shape = row_shape(a.rows, vectors);
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
