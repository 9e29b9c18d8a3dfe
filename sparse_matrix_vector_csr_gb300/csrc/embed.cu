// Rows of a table by token, and the gradient of that lookup.  The tokens of a batch are a sparse
// tokens x vocab matrix P with one entry of value `scale` a row (none where the token is padding);
// the lookup is P times the table, its gradient the transposed product P^T dx.  For the latter the
// entries are put in the order of their columns (a stable radix sort), equal shares of that order go
// to the warps whatever the columns' lengths, and a column that reaches over several shares is joined
// from their partial sums, as the merge-path product joins its rows.  Both are bound by their rows'
// bytes.
#include <type_traits>

#include "device_util.cuh"
#include "rows_common.cuh"

namespace spmv {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ bool is_entry(int32_t id, int64_t vocab) { return id >= 0 && id < vocab; }

// ----------------------------------------------------------------------------
// lookup
// ----------------------------------------------------------------------------
// A warp takes kU x 32 units of one token's row: 64 bytes a lane in flight where there are many tokens, 16 where few would
// leave SMs idle.  Bound by DRAM: 32768 tokens of 131072, 4096 bf16 values a row, scaled: 60 us, 6.1 TB/s; 8 tokens 1.7 us.
template <typename T, typename U, int kU, bool kScaled>
__global__ void __launch_bounds__(kThreads) k_embed(int64_t tokens, int64_t vocab, int64_t units, int64_t parts,
                                                   float scale, const int32_t *__restrict__ ids,
                                                   const U *__restrict__ table, int64_t ldt, U *__restrict__ x,
                                                   int64_t ldx) {
    constexpr int kN = sizeof(U) / sizeof(T);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int64_t t = item / parts;
    if (t >= tokens) return;
    const int64_t u0 = (item - t * parts) * (32 * kU) + lane;
    const int32_t id = ids[t];
    const bool there = is_entry(id, vocab);
    const U *src = table + static_cast<int64_t>(there ? id : 0) * ldt;
    U *dst = x + t * ldx;
    U v[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
        v[i] = U{};
        if (there && u0 + i * 32 < units) v[i] = src[u0 + i * 32];
    }
#pragma unroll
    for (int i = 0; i < kU; ++i)
        if (u0 + i * 32 < units) {
            if constexpr (kScaled) {
                float f[kN];
                unit_to_f32<T>(v[i], f);
#pragma unroll
                for (int j = 0; j < kN; ++j) f[j] *= scale;
                if (there) v[i] = unit_from_f32<T, U>(f);  // (0 without a token, whatever the scale)
            }
            dst[u0 + i * 32] = v[i];
        }
}

template <typename T>
void launch_embed(int unit, int64_t tokens, int64_t vocab, int64_t d, float scale, const int32_t *ids, const void *table,
                  int64_t ldt, void *x, int64_t ldx, cudaStream_t s) {
    auto go = [&](auto tag, auto per_lane, auto scaled) {
        using U = decltype(tag);
        constexpr int kU = decltype(per_lane)::value;
        constexpr int64_t kN = sizeof(U) / sizeof(T);
        const int64_t units = d / kN, parts = ceil_div(units, 32 * kU);
        k_embed<T, U, kU, decltype(scaled)::value><<<static_cast<unsigned>(ceil_div(tokens * parts, kWarps)), kThreads, 0, s>>>(
            tokens, vocab, units, parts, scale, ids, static_cast<const U *>(table), ldt / kN, static_cast<U *>(x), ldx / kN);
    };
    auto either = [&](auto tag, auto per_lane) {
        scale == 1.0f ? go(tag, per_lane, std::false_type{}) : go(tag, per_lane, std::true_type{});
    };
    constexpr std::integral_constant<int, 1> one;
    constexpr std::integral_constant<int, 4> four;
    constexpr std::integral_constant<int, 8> eight;
    const bool few = tokens * d * static_cast<int64_t>(sizeof(T)) < int64_t(kSms) * 16 * 1024;
    if (unit == 16) few ? either(uint4{}, one) : either(uint4{}, four);
    else if (unit == 8) either(uint2{}, four);
    else if (unit == 4) either(uint32_t{}, eight);
    else if constexpr (sizeof(T) == 2) either(uint16_t{}, eight);
}

// ----------------------------------------------------------------------------
// tokens in the order of their rows
// ----------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int64_t kSortShare = 1024;  // tokens a CTA sorts, at least, while the cluster has room
constexpr int kHeld = 8;              // times 32: of a warp's tokens in registers

struct SortShape {
    int ctas;    // a cluster
    int passes;  // digits of the row number, lowest first
    int bits;    // of a digit
    size_t smem;
};
SortShape sort_shape(int64_t tokens, int64_t vocab) {
    SortShape s;
    s.ctas = 1;
    while (s.ctas < kMaxCluster && tokens > s.ctas * kSortShare) s.ctas *= 2;
    int bits = 1;
    while ((int64_t(1) << bits) < vocab) ++bits;
    s.passes = static_cast<int>(ceil_div(bits, kDigitBits));
    s.bits = static_cast<int>(ceil_div(bits, s.passes));
    s.smem = ((kSortWarps + kMaxCluster + 1) * (size_t(1) << s.bits) + kSortWarps) * sizeof(int32_t);
    return s;
}

struct SortArgs {
    int64_t tokens, vocab;
    int passes, bits;
    const int32_t *ids;
    int2 *sorted[2];           // row and token; the last pass writes the first
    int32_t *count;            // tokens that are entries; chunks in whose end a row stays open (0, for k_embed_sum)
};
struct ZeroArgs {  // rows x row_bytes at a distance of ld bytes
    char *p;
    int64_t rows, row_bytes, ld;
    const char *ahead;  // and then to L2: this many lines from here on
    int64_t ahead_lines;
};

__device__ __forceinline__ void zero_bytes(char *p, int64_t n, int64_t worker, int64_t workers) {
    // 2-byte values up to the first 16-byte boundary and behind the last one
    int64_t head = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15);
    if (head > n) head = n;
    const int64_t vecs = (n - head) / 16, tail = head + vecs * 16;
    uint4 *v = reinterpret_cast<uint4 *>(p + head);
    for (int64_t i = worker; i < vecs; i += workers) __stcs(v + i, make_uint4(0, 0, 0, 0));
    if (worker < head / 2) reinterpret_cast<uint16_t *>(p)[worker] = 0;
    if (worker < (n - tail) / 2) reinterpret_cast<uint16_t *>(p + tail)[worker] = 0;
}

// The first cluster sorts the entries by row, stably (tokens of a row stay in their order, so sums over
// them do not depend on timing); the other CTAs meanwhile write zeros over the whole gradient, of
// which most rows have no token.  Every pass counts each warp's run of tokens by digit, exchanges
// the CTAs' counts through the cluster's shared memory, and writes each token to its place.  Bound by latency where it is alone
// (5003 tokens, two passes: 15 us, of which 3 us are the clusters' barriers a pass; with shares of 4096 tokens 21; 65536
// tokens, one pass: 19 us, half of it the stores, each to a place of its own), and by DRAM's writes beside them: 537 MB of zeros
// and 16384 tokens 92 us.
__global__ void __launch_bounds__(kSortThreads) k_embed_sort(SortArgs a, ZeroArgs z, int ctas) {
    extern __shared__ int32_t shared[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x >= ctas) {
        const int64_t worker = (static_cast<int64_t>(blockIdx.x) - ctas) * kSortThreads + tid;
        const int64_t workers = (static_cast<int64_t>(gridDim.x) - ctas) * kSortThreads;
        if (z.ld == z.row_bytes) {
            zero_bytes(z.p, z.rows * z.row_bytes, worker, workers);
        } else {
            for (int64_t r = worker / 32; r < z.rows; r += workers / 32) zero_bytes(z.p + r * z.ld, z.row_bytes, lane, 32);
        }
        for (int64_t i = worker; i < z.ahead_lines; i += workers) asm volatile("prefetch.global.L2 [%0];" ::"l"(z.ahead + i * 128));
            return;
    }
    const int bins = 1 << a.bits, rank = blockIdx.x;
    int32_t *wcount = shared;                         // [warps][bins]: counts, then next places
    int32_t *hist = wcount + kSortWarps * bins;       // [kMaxCluster][bins]: the CTAs' counts
    int32_t *place0 = hist + kMaxCluster * bins;      // [bins]: this CTA's first place
    int32_t *warp_part = place0 + bins;               // [warps]
    int64_t n = a.tokens;
    if (ctas > 1) cluster_sync(ctas);  // every CTA is there before its shared memory is written
    for (int p = 0; p < a.passes; ++p) {
        const int2 *in = p == 0 ? nullptr : a.sorted[(a.passes - p) & 1];
        int2 *out = a.sorted[(a.passes - 1 - p) & 1];
        const int shift = p * a.bits;
        const int64_t share = (n + ctas - 1) / ctas, begin = min(n, rank * share), end = min(n, begin + share);
        // as few warps as hold their tokens in registers: their counts have to be cleared and added up (one where no
        // token is left)
        const int n_warps = static_cast<int>(min(max((share + 32 * kHeld - 1) / (32 * kHeld), int64_t(1)), int64_t(kSortWarps)));
        const int64_t run = (end - begin + 32 * n_warps - 1) / (32 * n_warps) * 32;
        const int64_t r0 = begin + warp * run, r1 = warp < n_warps ? min(end, r0 + run) : r0;
        int32_t *mine = wcount + warp * bins;
        // kHeld times 32 keys of the warp's run and where their tokens are, all loads at once (from L2: other SMs of
        // the cluster wrote them in the pass before)
        int32_t key[kHeld], src[kHeld], found[kHeld];
        const auto load = [&](int64_t i0) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int64_t at = i0 + i * 32 + lane;
                key[i] = -1;
                src[i] = static_cast<int32_t>(at);
                if (at < r1 && in) {
                    const int2 v = __ldcg(in + at);
                    key[i] = v.x;
                    src[i] = v.y;
                } else if (at < r1) {
                    key[i] = a.ids[at];
                }
            }
        };
        // a key's digit, the entries of the same digit in lower lanes and how many have it; -1: no entry.  (By a vote a bit:
        // 65536 tokens of 300 rows 22.7 us; by __match_any_sync 23.8.)
        const auto match = [&](int32_t k) {
            const bool entry = is_entry(k, a.vocab);
            const int dig = (k >> shift) & (bins - 1);
            uint32_t same = __ballot_sync(0xffffffffu, entry);
#pragma unroll
            for (int b = 0; b < kDigitBits; ++b) {
                const uint32_t ones = __ballot_sync(0xffffffffu, dig >> b & 1);
                same &= dig >> b & 1 ? ones : ~ones;
            }
            return entry ? dig | __popc(same & ((1u << lane) - 1)) << 10 | __popc(same) << 16 : -1;
        };
        load(r0);
        for (int i = tid; i < n_warps * bins; i += kSortThreads) wcount[i] = 0;
        __syncthreads();
        for (int64_t i0 = r0; i0 < r1; i0 += 32 * kHeld) {
            if (i0 != r0) load(i0);
#pragma unroll
            for (int i = 0; i < kHeld; ++i) found[i] = i0 + i * 32 < r1 ? match(key[i]) : -1;
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                if (found[i] >= 0 && (found[i] >> 10 & 63) == 0) mine[found[i] & 1023] += found[i] >> 16;
                __syncwarp();
            }
        }
        __syncthreads();
        for (int b = tid; b < bins; b += kSortThreads) {  // (at most one a thread)
            int32_t at = 0;
#pragma unroll 8
            for (int w = 0; w < n_warps; ++w) {
                const int32_t c = wcount[w * bins + b];
                wcount[w * bins + b] = at;
                at += c;
            }
            if (ctas == 1) {
                hist[b] = at;
            } else {
                for (int r = 0; r < ctas; ++r)
                    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer_addr(hist + rank * bins + b, r)), "r"(at)
                                 : "memory");
            }
        }
        cluster_sync(ctas);
        int32_t before = 0, total = 0;
        if (tid < bins)
            for (int r = 0; r < ctas; ++r) {
                const int32_t c = hist[r * bins + tid];
                before += r < rank ? c : 0;
                total += c;
            }
        int32_t incl = total;  // scan over the digits
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_part[warp] = incl;
        __syncthreads();
        const int32_t of_warp = warp_part[lane];
        const int32_t at = incl - total + __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0);
        const int32_t all = __reduce_add_sync(0xffffffffu, of_warp);
        if (tid < bins) place0[tid] = at + before;
        __syncthreads();
        for (int64_t i0 = r0; i0 < r1; i0 += 32 * kHeld) {
            if (run > 32 * kHeld) {
                load(i0);
#pragma unroll
                for (int i = 0; i < kHeld; ++i) found[i] = i0 + i * 32 < r1 ? match(key[i]) : -1;
            }
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int dig = found[i] & 1023, earlier = found[i] >> 10 & 63;
                const int32_t to = found[i] >= 0 ? place0[dig] + mine[dig] + earlier : -1;
                __syncwarp();
                if (found[i] >= 0 && earlier == 0) mine[dig] += found[i] >> 16;
                __syncwarp();
                if (to >= 0) out[to] = make_int2(key[i], src[i]);  // (stores to places of their own: one of 8 bytes, not two)
            }
        }
        n = all;
        cluster_sync(ctas);  // the places are written, the counts read
    }
    if (rank == 0 && tid == 0) {
        a.count[0] = static_cast<int32_t>(n);
        a.count[1] = 0;
    }
    dev::allow_dependents();
}

// ----------------------------------------------------------------------------
// sums over each row's tokens
// ----------------------------------------------------------------------------
// Entries that one warp sums: as few as leave no more than `warps` of them for the pieces of a row that go to warps
// of their own (a chunk's entries follow one another, so fewer are faster where they fill the GPU), 8 to 64,
// and more where the carries of 8192 chunks would not do.
int64_t chunk_entries(int64_t tokens, int64_t d) {
    int64_t c = 8;
    while (c < 64 && ceil_div(tokens, c) * ceil_div(d, 256) > 5000) c *= 2;
    while (ceil_div(tokens, c) > 8192) c *= 2;
    return c;
}
constexpr int kJoinCols = 4 * 32;  // of a row, per item of k_embed_join
constexpr int kJoinAlone = 16;     // carries that one warp adds up

struct SumArgs {
    int64_t d, chunk, parts;
    float scale;
    int accumulate;
    const int2 *sorted;
    int32_t *count, *open;  // open: the chunks in whose end a row begun in them stays open
    uint8_t *through;       // [chunks]: a row comes from the chunk in front and goes on behind
    float *carry;  // [chunks][2][ldc]: sum up to the end of a row begun in front of the chunk; from the start of a row open at its end
    int64_t ldc;
};

template <typename O, int kN>
__device__ __forceinline__ void load_values(const O *p, float *f) {
    constexpr int kBytes = kN * static_cast<int>(sizeof(O)) > 16 ? 16 : kN * static_cast<int>(sizeof(O));
    using U = typename Unit<kBytes>::type;
    constexpr int kEach = kBytes / static_cast<int>(sizeof(O));
#pragma unroll
    for (int i = 0; i < kN; i += kEach) unit_to_f32<O>(*reinterpret_cast<const U *>(p + i), f + i);
}
template <typename O, int kN>
__device__ __forceinline__ void store_values(O *p, const float *f) {
    constexpr int kBytes = kN * static_cast<int>(sizeof(O)) > 16 ? 16 : kN * static_cast<int>(sizeof(O));
    using U = typename Unit<kBytes>::type;
    constexpr int kEach = kBytes / static_cast<int>(sizeof(O));
#pragma unroll
    for (int i = 0; i < kN; i += kEach) *reinterpret_cast<U *>(p + i) = unit_from_f32<O, U>(f + i);
}

// A warp sums kU x 32 units of kN values of the rows of one chunk of sorted entries, kR rows' loads in
// flight (and, where they are added to, the gradient's), in 32 bits, in the tokens' order.  Bound by the loads in flight: 16 bytes
// a lane and four rows keep 32 warps on an SM (65536 tokens of 300 rows of 1024 fp16 values: 33 us, 4.1 TB/s; 32 bytes a lane 34,
// eight rows 47).  Adding to a gradient, its rows' loads go with dx's (5003 odd float rows: 20 us; one after the other 62).
template <typename T, typename O, int kN, int kU, int kR, bool kAdd>
__global__ void __launch_bounds__(kThreads, kAdd ? 2 : 4) k_embed_sum(SumArgs a, const T *__restrict__ dx, int64_t lddx, O *out, int64_t ldo) {
    using U = typename Unit<kN * static_cast<int>(sizeof(T))>::type;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    dev::grid_wait();
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp, c = item / a.parts;
    const int64_t total = *a.count, lo = c * a.chunk, hi = min(lo + a.chunk, total);
    if (lo >= total) return;
    const int64_t col0 = ((item - c * a.parts) * (32 * kU) + lane) * kN;  // unit i's values: from col0 + i * 32 * kN
    float acc[kU][kN] = {};
    const auto flush = [&](int32_t row, float *carry, const float (*old)[kN]) {
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            const int64_t col = col0 + i * 32 * kN;
            if (col < a.d) {
                if (carry) {
#pragma unroll
                    for (int j = 0; j < kN; ++j) carry[col + j] = acc[i][j];
                } else {
                    float f[kN];
#pragma unroll
                    for (int j = 0; j < kN; ++j) f[j] = kAdd ? fmaf(acc[i][j], a.scale, old[i][j]) : acc[i][j] * a.scale;
                    store_values<O, kN>(out + static_cast<int64_t>(row) * ldo + col, f);
                }
            }
#pragma unroll
            for (int j = 0; j < kN; ++j) acc[i][j] = 0.0f;
        }
    };
    float *carry = a.carry + 2 * c * a.ldc;
    bool carried = lo > 0 && a.sorted[lo - 1].x == a.sorted[lo].x;
    for (int64_t g = lo; g < hi; g += 32) {
        const int n = static_cast<int>(min(hi - g, int64_t(32)));
        const int2 mine = lane < n ? a.sorted[g + lane] : make_int2(-1, 0);
        const int32_t key = mine.x, src = mine.y, behind = g + n < total ? a.sorted[g + n].x : -1;
        for (int q0 = 0; q0 < n; q0 += kR) {
            U v[kR][kU];
            float old[kAdd ? kR : 1][kU][kN];
#pragma unroll
            for (int q = 0; q < kR; ++q) {
                const int64_t t = __shfl_sync(0xffffffffu, src, q0 + q);
                const int32_t row = __shfl_sync(0xffffffffu, key, q0 + q), later = __shfl_sync(0xffffffffu, key, (q0 + q + 1) & 31);
                if (q0 + q < n) {
                    const bool ends = (q0 + q + 1 < n ? later : behind) != row;
#pragma unroll
                    for (int i = 0; i < kU; ++i) {
                        const int64_t col = col0 + i * 32 * kN;
                        if (col < a.d) {
                            v[q][i] = __ldcs(reinterpret_cast<const U *>(dx + t * lddx + col));
                            if constexpr (kAdd)
                                if (ends) load_values<O, kN>(out + static_cast<int64_t>(row) * ldo + col, old[q][i]);
                        }
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < kR; ++q) {
                const int32_t row = __shfl_sync(0xffffffffu, key, q0 + q);
                const int32_t later = __shfl_sync(0xffffffffu, key, (q0 + q + 1) & 31);
                if (q0 + q < n) {
#pragma unroll
                    for (int i = 0; i < kU; ++i)
                        if (col0 + i * 32 * kN < a.d) {
                            float f[kN];
                            unit_to_f32<T>(v[q][i], f);
#pragma unroll
                            for (int j = 0; j < kN; ++j) acc[i][j] += f[j];
                        }
                    if ((q0 + q + 1 < n ? later : behind) != row) {
                        flush(row, carried ? carry : nullptr, old[kAdd ? q : 0]);
                        carried = false;
                    } else if (q0 + q + 1 == n && g + n == hi) {  // the row goes on in the next chunk
                        flush(row, carried ? carry : carry + a.ldc, old[0]);
                        if (item == c * a.parts && lane == 0) {
                            if (!carried) a.open[atomicAdd(a.count + 1, 1)] = static_cast<int32_t>(c);
                            a.through[c] = carried;
                        }
                    }
                    if (q0 + q + 1 == n && g + n == hi && behind != row) {
                        if (item == c * a.parts && lane == 0) a.through[c] = 0;
                    }
                }
            }
        }
    }
    dev::allow_dependents();
}

// The rows that reach over several chunks: the sum of the open end of the first chunk and what the next
// chunks have of the row, in a fixed order: one after the other by one warp where they are few, else each warp
// of the CTA an eighth of them.  An item is kJoinCols columns of one of the rows that k_embed_sum listed.
template <typename O>
__global__ void __launch_bounds__(kThreads) k_embed_join(SumArgs a, O *out, int64_t ldo) {
    __shared__ float4 part[kWarps][32];
    __shared__ int many[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    dev::grid_wait();
    const int64_t total = a.count[0], opened = a.count[1], items = (a.d + kJoinCols - 1) / kJoinCols * opened;
    struct Run {
        int64_t c, n, col;  // first chunk, carries, column
        int32_t row;
    };
    const auto find = [&](int64_t item) {
        Run r;
        const int64_t piece = item / opened;  // (a long row's pieces go to CTAs far from one another)
        r.c = a.open[item - piece * opened];
        r.col = piece * kJoinCols + lane * 4;
        r.row = a.sorted[(r.c + 1) * a.chunk - 1].x;
        int64_t end = r.c + 1;  // the row's last chunk: the first behind r.c through which it does not go
        for (;;) {
            const bool through = (end + lane + 1) * a.chunk < total && a.through[end + lane];
            const bool through2 = (end + lane + 33) * a.chunk < total && a.through[end + lane + 32];
            const uint32_t stops = ~__ballot_sync(0xffffffffu, through), stops2 = ~__ballot_sync(0xffffffffu, through2);
            if (stops | stops2) {
                end += stops ? __ffs(stops) - 1 : 31 + __ffs(stops2);
                break;
            }
            end += 64;
        }
        r.n = end - r.c + 1;
        return r;
    };
    // carries q0, q0 + every, ...: the row's start in its first chunk, then the heads of the next ones
    const auto add = [&](const Run &r, int64_t q0, int64_t every) {
        float4 sum = make_float4(0, 0, 0, 0);
        constexpr int kLoads = 16;
        if (r.col < a.d)
            for (; q0 < r.n; q0 += every * kLoads) {
                float4 v[kLoads];
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const int64_t q = q0 + i * every;
                    v[i] = make_float4(0, 0, 0, 0);
                    if (q < r.n) v[i] = *reinterpret_cast<const float4 *>(a.carry + (2 * (r.c + q) + (q == 0 ? 1 : 0)) * a.ldc + r.col);
                }
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    sum.x += v[i].x;
                    sum.y += v[i].y;
                    sum.z += v[i].z;
                    sum.w += v[i].w;
                }
            }
        return sum;
    };
    const auto write = [&](const Run &r, const float4 &sum) {
        const float f[4] = {sum.x, sum.y, sum.z, sum.w};
        O *p = out + static_cast<int64_t>(r.row) * ldo + r.col;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r.col + j < a.d) p[j] = from_f32<O>(a.accumulate ? fmaf(f[j], a.scale, to_f32(p[j])) : f[j] * a.scale);
    };
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kWarps; i0 < items; i0 += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t item = i0 + warp;
        bool long_one = false;
        if (item < items) {
            const Run r = find(item);
            long_one = r.n > kJoinAlone;
            if (!long_one) write(r, add(r, 0, 1));
        }
        if (lane == 0) many[warp] = long_one;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) {
            if (!many[w]) continue;
            const Run r = find(i0 + w);
            part[warp][lane] = add(r, warp, kWarps);
            __syncthreads();
            if (warp == 0) {
                float4 sum = part[0][lane];
                for (int k = 1; k < kWarps; ++k) {
                    sum.x += part[k][lane].x;
                    sum.y += part[k][lane].y;
                    sum.z += part[k][lane].z;
                    sum.w += part[k][lane].w;
                }
                write(r, sum);
            }
            __syncthreads();
        }
        __syncthreads();
    }
}

template <typename T, typename O>
cudaError_t launch_sums(int values, const SumArgs &a, int64_t chunks, const void *dx, int64_t lddx, void *out, int64_t ldo,
                        cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto go = [&](auto n_values, auto per_lane, auto in_flight, auto add) {
        constexpr int kN = decltype(n_values)::value, kU = decltype(per_lane)::value;
        SumArgs b = a;
        b.parts = ceil_div(a.d, 32 * kU * kN);
        cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(chunks * b.parts, kWarps)));
        return cudaLaunchKernelEx(&cfg, k_embed_sum<T, O, kN, kU, decltype(in_flight)::value, decltype(add)::value>, b,
                                  static_cast<const T *>(dx), lddx, static_cast<O *>(out), ldo);
    };
    constexpr std::integral_constant<int, 1> one;
    constexpr std::integral_constant<int, 2> two;
    constexpr std::integral_constant<int, 4> four;
    constexpr std::integral_constant<int, 8> eight;
    // rows in flight
    auto either = [&](auto n_values, auto per_lane) {
        if (!a.accumulate) return go(n_values, per_lane, four, std::false_type{});
        return go(n_values, per_lane, four, std::true_type{});
    };
    cudaError_t e;
    if (values == 1) e = either(one, four);
    else if (values == 2) e = either(two, four);
    else if (values == 4) e = either(four, two);
    else if constexpr (sizeof(T) == 2) e = either(eight, one);
    else e = cudaErrorInvalidValue;
    if (e != cudaSuccess || chunks < 2) return e;
    const int64_t items = ceil_div(chunks * ceil_div(a.d, kJoinCols), kWarps);
    cfg.gridDim = dim3(static_cast<unsigned>(items < 4 * kSms ? items : 4 * kSms));
    return cudaLaunchKernelEx(&cfg, k_embed_join<O>, a, static_cast<O *>(out), ldo);
}

constexpr int64_t kMaxEmbedWidth = int64_t(1) << 23;

int check_embed(int64_t tokens, int64_t vocab, int64_t d) {
    if (tokens < 0 || tokens >= int64_t(1) << 31) return refuse("tokens must lie in [0, 2^31)");
    if (vocab < 1 || vocab >= int64_t(1) << 31) return refuse("vocab must lie in [1, 2^31)");
    if (d < 0 || d > kMaxEmbedWidth) return refuse("d must lie in [0, " + std::to_string(kMaxEmbedWidth) + "]");
    if (tokens * ceil_div(d, 128) >= int64_t(1) << 33) return set_error(SPMV_ERR_TOO_LARGE, "tokens * d must be below 2^40");
    return SPMV_OK;
}

// The parts of the gradient's workspace, each at a multiple of 16 bytes.
struct EmbedSpace {
    int64_t sorted[2], count, open, through, carry, bytes;
    int64_t chunks, ldc;
};
EmbedSpace embed_space(int64_t tokens, int64_t vocab, int64_t d) {
    EmbedSpace w;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += ceil_div(bytes, 16) * 16;
        return here;
    };
    const bool one = sort_shape(tokens, vocab).passes == 1;
    w.sorted[0] = take(tokens * 8);
    w.sorted[1] = one ? 0 : take(tokens * 8);
    w.count = take(8);
    w.chunks = ceil_div(tokens, chunk_entries(tokens, d));
    w.open = take(w.chunks * 4);
    w.through = take(w.chunks);
    w.ldc = ceil_div(d, 4) * 4;
    w.carry = take(w.chunks > 1 ? w.chunks * 2 * w.ldc * 4 : 0);
    w.bytes = at;
    return w;
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" SPMV_API int spmv_embed_rows(int64_t tokens, int64_t vocab, int64_t d, const int32_t *ids, const void *table,
                                        int64_t ldtable, double scale, void *x, int64_t ldx, int dtype, void *stream) {
    SPMV_TRY(check_embed(tokens, vocab, d));
    if (!row_dtype_ok(dtype)) return refuse("dtype must be SPMV_F32, SPMV_F16 or SPMV_BF16");
    if (tokens == 0 || d == 0) return SPMV_OK;
    SPMV_TRY(check_array(ids, "ids", 4));
    SPMV_TRY(check_matrix(table, "table", vocab, d, ldtable, dtype));
    SPMV_TRY(check_matrix(x, "x", tokens, d, ldx, dtype));
    const int vb = row_value_bytes(dtype);
    const size_t out = span_bytes(tokens, d, ldx, vb);
    SPMV_TRY(check_apart(x, out, "x", table, span_bytes(vocab, d, ldtable, vb), "table"));
    SPMV_TRY(check_apart(x, out, "x", ids, static_cast<size_t>(tokens) * 4, "ids"));
    const int unit = unit_bytes(vb, d, {{table, ldtable}, {x, ldx}});
    const float f = static_cast<float>(scale);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SPMV_F32) launch_embed<float>(unit, tokens, vocab, d, f, ids, table, ldtable, x, ldx, s);
    else if (dtype == SPMV_F16) launch_embed<__half>(unit, tokens, vocab, d, f, ids, table, ldtable, x, ldx, s);
    else launch_embed<__nv_bfloat16>(unit, tokens, vocab, d, f, ids, table, ldtable, x, ldx, s);
    SPMV_TRY_CUDA(cudaGetLastError());
    return SPMV_OK;
}

extern "C" SPMV_API int64_t spmv_embed_workspace(int64_t tokens, int64_t vocab, int64_t d) {
    SPMV_TRY(check_embed(tokens, vocab, d));
    return embed_space(tokens, vocab, d).bytes;
}

extern "C" SPMV_API int spmv_embed_rows_grad(int64_t tokens, int64_t vocab, int64_t d, const int32_t *ids, const void *dx,
                                             int64_t lddx, int dtype, double scale, int accumulate, void *dtable,
                                             int64_t lddtable, int out_dtype, void *workspace, int64_t workspace_bytes,
                                             void *stream) {
    SPMV_TRY(check_embed(tokens, vocab, d));
    if (!row_dtype_ok(dtype)) return refuse("dtype must be SPMV_F32, SPMV_F16 or SPMV_BF16");
    if (out_dtype != dtype && out_dtype != SPMV_F32) return refuse("out_dtype must be dtype or SPMV_F32");
    if (d == 0 || (tokens == 0 && accumulate)) return SPMV_OK;
    const EmbedSpace w = embed_space(tokens, vocab, d);
    if (workspace_bytes < w.bytes) return refuse("the workspace has fewer bytes than spmv_embed_workspace says");
    SPMV_TRY(check_matrix(dtable, "dtable", vocab, d, lddtable, out_dtype));
    SPMV_TRY(check_array(workspace, "workspace", 16));
    SPMV_TRY(check_matrix(dx, "dx", tokens, d, lddx, dtype));
    if (tokens) SPMV_TRY(check_array(ids, "ids", 4));
    const int vb = row_value_bytes(dtype), vo = row_value_bytes(out_dtype);
    const struct { const void *p; size_t bytes; const char *name; } arrays[] = {
        {ids, static_cast<size_t>(tokens) * 4, "ids"}, {dx, span_bytes(tokens, d, lddx, vb), "dx"},
        {dtable, span_bytes(vocab, d, lddtable, vo), "dtable"}, {workspace, static_cast<size_t>(w.bytes), "workspace"}};
    for (int i = 2; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            SPMV_TRY(check_apart(arrays[i].p, arrays[i].bytes, arrays[i].name, arrays[j].p, arrays[j].bytes, arrays[j].name));

    char *base = static_cast<char *>(workspace);
    const SortShape shape = sort_shape(tokens, vocab);
    SortArgs sort{tokens, vocab, shape.passes, shape.bits, ids, {}, reinterpret_cast<int32_t *>(base + w.count)};
    for (int i = 0; i < 2; ++i) {
        sort.sorted[i] = reinterpret_cast<int2 *>(base + w.sorted[i]);
    }
    ZeroArgs zero{static_cast<char *>(dtable), accumulate ? 0 : vocab, d * vo, lddtable * vo, static_cast<const char *>(dx), 0};
    // The sort alone takes about 15 us, in which 96 MB can be written and read: as much of dx as that leaves room for
    // waits in L2 for the sums.
    const int64_t zeros = zero.rows * zero.row_bytes, dx_bytes = static_cast<int64_t>(span_bytes(tokens, d, lddx, vb));
    if (zeros < 96000000) {
        zero.ahead = reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(dx) & ~uintptr_t(127));
        const int64_t room = 96000000 - zeros;
        zero.ahead_lines = (dx_bytes < room ? dx_bytes : room) / 128;
    }
    // CTAs that do that: two fit an SM; at least 64 KB each
    int64_t fill = ceil_div(zeros + zero.ahead_lines * 128, 64 * 1024);
    if (fill > 2 * kSms - shape.ctas) fill = 2 * kSms - shape.ctas;
    fill = ceil_div(fill, shape.ctas) * shape.ctas;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (shape.smem > 48 * 1024)
        SPMV_TRY_CUDA(cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(shape.smem)));
    SPMV_TRY_CUDA(launch_rows(k_embed_sort, shape.ctas + fill, kSortThreads, shape.ctas, shape.smem, s, sort, zero, shape.ctas));
    if (tokens == 0) return SPMV_OK;
    // values of a lane's unit: what the alignment of both matrices' rows allows
    const int in = unit_bytes(vb, d, {{dx, lddx}}) / vb, to = unit_bytes(vo, d, {{dtable, lddtable}});
    const int values = to == 16 ? in : (in < to / vo ? in : to / vo);
    const SumArgs sum{d, chunk_entries(tokens, d), 1, static_cast<float>(scale), accumulate, sort.sorted[0], sort.count,
                      reinterpret_cast<int32_t *>(base + w.open), reinterpret_cast<uint8_t *>(base + w.through), reinterpret_cast<float *>(base + w.carry), w.ldc};
    cudaError_t e;
    if (dtype == SPMV_F32) e = launch_sums<float, float>(values, sum, w.chunks, dx, lddx, dtable, lddtable, s);
    else if (dtype == SPMV_F16 && out_dtype == SPMV_F16) e = launch_sums<__half, __half>(values, sum, w.chunks, dx, lddx, dtable, lddtable, s);
    else if (dtype == SPMV_F16) e = launch_sums<__half, float>(values, sum, w.chunks, dx, lddx, dtable, lddtable, s);
    else if (out_dtype == SPMV_BF16) e = launch_sums<__nv_bfloat16, __nv_bfloat16>(values, sum, w.chunks, dx, lddx, dtable, lddtable, s);
    else e = launch_sums<__nv_bfloat16, float>(values, sum, w.chunks, dx, lddx, dtable, lddtable, s);
    SPMV_TRY_CUDA(e);
    return SPMV_OK;
}
