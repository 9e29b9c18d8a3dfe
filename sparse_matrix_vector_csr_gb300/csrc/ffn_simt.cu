// The products of the feed-forward block by the ordinary units: float, and 16-bit values at any address.
// A CTA of 256 threads has 128 x 128 values of D, 8 x 8 a thread (32 x 128 where segments are short), in 32 bits; pieces of A
// and B of 16 along k go through shared memory, k first, two of each so that one is filled while the other is
// multiplied.  Sums of 256 of k join totals in shared memory, so that their rounding does not grow with k (28 rows, d = 3781,
// f = 9793: 5e-7 from 64 bits, 3e-6 before), and where the tiles would leave SMs without one, up to eight CTAs share a tile's k (2
// rows, d = 3089, f = 8394: 1468 us forward, 341 with that and tiles of 32 rows).  Bound by the ordinary units' arithmetic (two
// multiply-adds an instruction) and the reads of shared memory that feed it, an equal share of cycles: 4096 rows, d = 2048, f =
// 4096, float: 38.7 TFLOP/s forward, 35.9 back (43.6 and 44.5 without the totals).  Tried without them: pieces of 8 along k 34.9
// forward; A's values twice in shared memory, to be a pair's operand as they are, 34.4; 128 x 256 values, 8 x 16 a thread, 41.3.
#include "ffn.cuh"

namespace spmv {
namespace ffn {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;  // columns of D; rows: 16 kR (128 or 32)
constexpr int kDepth = 16;
constexpr int kFold = 16;   // pieces of k (256 of k) that are summed before the sum joins a total

// fours of a piece (kRows x kDepth) that a thread has
template <int kRows>
constexpr int kFours = (kRows * kDepth / 4 + kThreads - 1) / kThreads;
// A thread's values of a piece of an operand whose (0, 0) is at p: along k, four threads a row; along m or n, kRows / 4 a
// row.  Along k the two halves of the rows may be of two matrices (p2: the second half's).
template <typename T, bool kAcross, int kRows>
__device__ __forceinline__ void fetch(const T *p, const T *p2, int64_t ld, int64_t mn_left, int64_t mn_left2, int64_t k_left, bool quads,
                                      float (&v)[4 * kFours<kRows>]) {
#pragma unroll
    for (int i = 0; i < kFours<kRows>; ++i) {
        float *out = v + 4 * i;
        const int q = threadIdx.x + kThreads * i;
        const int mn = kAcross ? q % (kRows / 4) * 4 : q / 4, k = kAcross ? q / (kRows / 4) : (q & 3) * 4;
        const bool second = !kAcross && mn >= kRows / 2;
        const int in_half = second ? mn - kRows / 2 : mn;
        const T *at = kAcross ? p + k * ld + mn : (second ? p2 : p) + in_half * ld + k;
        const int64_t rows = q * 4 >= kRows * kDepth ? 0 : kAcross ? k_left - k : (second ? mn_left2 : mn_left) - in_half;
        const int64_t run = kAcross ? mn_left - mn : k_left - k;  // values that follow on
        if (rows > 0 && run >= 4 && quads) {
            using U = typename Unit<4 * sizeof(T)>::type;
            unit_to_f32<T>(*reinterpret_cast<const U *>(at), out);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) out[j] = rows > 0 && j < run ? to_f32(at[j]) : 0.0f;
        }
    }
}
template <bool kAcross, int kRows>
__device__ __forceinline__ void stage(float (*s)[kRows + 4], const float (&v)[4 * kFours<kRows>]) {
#pragma unroll
    for (int i = 0; i < kFours<kRows>; ++i) {
        const int q = threadIdx.x + kThreads * i;
        if (q * 4 >= kRows * kDepth) continue;
        if (kAcross) {
            *reinterpret_cast<float4 *>(&s[q / (kRows / 4)][q % (kRows / 4) * 4]) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[(q & 3) * 4 + j][q / 4] = v[4 * i + j];
        }
    }
}

// The tile of `rows` rows that blockIdx.x counts over all segments, and behind them the rows in none.
struct Place {
    int e;
    int64_t row, end;  // its first row, the segment's end
};
template <int kRows>
__device__ bool find_tile(const Segments &seg, Place &place) {
    __shared__ int32_t part[kThreads / 32];
    __shared__ Place found;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int per = (seg.count + 1 + kThreads - 1) / kThreads;
    const auto tiles = [&](int e) {
        const Segments::Span s = seg.span(e);
        return static_cast<int32_t>((s.end - s.begin + kRows - 1) / kRows);
    };
    int32_t mine = 0;
    for (int i = 0; i < per; ++i)
        if (t * per + i <= seg.count) mine += tiles(t * per + i);
    int32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) part[warp] = incl;
    if (t == 0) found.e = -1;
    __syncthreads();
    int32_t at = incl - mine;
    for (int w = 0; w < warp; ++w) at += part[w];
    const int32_t want = static_cast<int32_t>(blockIdx.x);
    if (want >= at && want < at + mine)
        for (int i = 0; i < per; ++i) {
            const int e = t * per + i, n = e <= seg.count ? tiles(e) : 0;
            if (want >= at && want < at + n) {
                const Segments::Span s = seg.span(e);
                found = Place{e, s.begin + static_cast<int64_t>(want - at) * kRows, s.end};
            }
            at += n;
        }
    __syncthreads();
    place = found;
    return place.e >= 0;
}

// D's tile of the CTA.  grid: x tiles of rows (kWeights: of the segment's matrix), y tiles of columns
// (kWeights: segments and their parts), z which of the three products (kWeights), or which part of k: a cluster of up to
// eight CTAs has the parts of one tile, whose sums each of them joins for its share of the rows, in the parts' order.
template <typename T, int kKind, int kR>
__global__ void __launch_bounds__(kThreads, 2) k_ffn_simt(Block b, unsigned quads_in, bool quads_out) {
    constexpr int kRows = 16 * kR;
    __shared__ __align__(16) float sa[2][kDepth][kRows + 4], sb[2][kDepth][kTile + 4];
    extern __shared__ __align__(16) uint8_t more[];
    float4 *totals = reinterpret_cast<float4 *>(more) + threadIdx.x;  // [2 kR], kThreads apart
    const int parts = kKind == kWeights ? 1 : static_cast<int>(gridDim.z), rank = kKind == kWeights ? 0 : static_cast<int>(blockIdx.z);
    constexpr bool kAcrossA = a_transposed(kKind), kAcrossB = b_transposed(kKind);
    constexpr int kCols = kKind == kGated ? kTile / 2 : kTile;  // gate's and up's beside each other
    const int which = kKind == kWeights ? blockIdx.z : 0;
    Place place;
    int64_t col0, m_left, depth, k0 = 0;
    int part = 0;
    if constexpr (kKind == kWeights) {
        const int64_t n_cols = product_columns<kKind>(b, which), n_rows = weight_rows(b, which);
        const int64_t tiles_n = (n_cols + kTile - 1) / kTile;
        place = Place{static_cast<int>(blockIdx.y / b.splits), blockIdx.x / tiles_n * kTile, n_rows};
        part = static_cast<int>(blockIdx.y % b.splits);
        col0 = (blockIdx.x % tiles_n) * kTile;
        if (place.row >= n_rows || !(which == 0 ? b.dwg : which == 1 ? b.dwu : b.dwd).p) return;
        const Segments::Span s = b.part(place.e, part);
        depth = s.end - s.begin;
        k0 = s.begin;
    } else {
        if (!find_tile<kRows>(b.seg, place)) return;
        col0 = static_cast<int64_t>(blockIdx.y) * kCols;
        depth = kKind == kGated || kKind == kBack ? b.d : b.f;
        if (place.e == b.seg.count) {
            if (kKind == kBack) return;
            depth = 0;  // rows in no segment: 0
        }
    }
    m_left = place.end - place.row;
    const int64_t n_left = product_columns<kKind>(b, which) - col0;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float2 acc[kR][4] = {};
    bool folded = false;

    for (int pass = 0; pass < (kKind == kInput ? 2 : 1); ++pass) {
        // A's and B's first value of the tile
        const T *pa, *pb, *pb2 = nullptr;
        int64_t lda, ldb;
        const auto start = [&](const Matrix &m, int64_t row, int64_t col, int64_t &ld) {
            ld = m.ld;
            return static_cast<const T *>(m.p) + row * m.ld + col;
        };
        const auto weight = [&](const Matrix &m, int64_t row, int64_t col, int64_t &ld) {
            return start(m, row, col, ld) + place.e * m.expert;
        };
        if (depth == 0) break;
        if constexpr (kKind == kGated) {
            pa = start(b.x, place.row, 0, lda);
            pb = weight(b.wg, col0, 0, ldb);
            pb2 = weight(b.wu, col0, 0, ldb);  // (the same leading dimension)
        } else if constexpr (kKind == kDown) {
            pa = start(b.h, place.row, 0, lda);
            pb = weight(b.wd, col0, 0, ldb);
            pb2 = pb + 64 * ldb;
        } else if constexpr (kKind == kBack) {
            pa = start(b.dy, place.row, 0, lda);
            pb = weight(b.wd, 0, col0, ldb);
        } else if constexpr (kKind == kInput) {
            pa = start(pass == 0 ? b.dgate : b.dup, place.row, 0, lda);
            pb = weight(pass == 0 ? b.wg : b.wu, 0, col0, ldb);
        } else {
            pa = start(which == 0 ? b.dgate : which == 1 ? b.dup : b.dy, k0, place.row, lda);
            pb = start(which == 2 ? b.h : b.x, k0, col0, ldb);
        }
        // this CTA's part of k, a multiple of the pieces' depth
        const int64_t each = ((depth + parts - 1) / parts + kDepth - 1) / kDepth * kDepth, k_first = rank * each;
        const int64_t mine = depth - k_first < each ? depth - k_first : each;
        if (mine <= 0) break;  // (of every pass)
        pa += kAcrossA ? k_first * lda : k_first;
        pb += kAcrossB ? k_first * ldb : k_first;
        if (!kAcrossB && pb2) pb2 += k_first;
        const bool qa = quads_in & 1, qb = quads_in & 2;
        const int64_t step_a = kAcrossA ? kDepth * lda : kDepth, step_b = kAcrossB ? kDepth * ldb : kDepth;
        const int64_t n2 = kKind == kGated ? n_left : n_left - 64;
        const int64_t steps = (mine + kDepth - 1) / kDepth;
        float va[4 * kFours<kRows>], vb[4 * kFours<kTile>];
        const auto load = [&](int64_t i) {
            const int64_t k_left = mine - i * kDepth;
            fetch<T, kAcrossA, kRows>(pa + i * step_a, pa + i * step_a + kRows / 2 * lda, lda, m_left, m_left - kRows / 2, k_left, qa, va);
            fetch<T, kAcrossB, kTile>(pb + i * step_b, pb2 + i * step_b, ldb, n_left, n2, k_left, qb, vb);
        };
        load(0);
        __syncthreads();  // (the pass before may still read)
        stage<kAcrossA, kRows>(sa[0], va);
        stage<kAcrossB, kTile>(sb[0], vb);
        __syncthreads();
        for (int64_t i = 0; i < steps; ++i) {
            const int now = i & 1;
            if (i + 1 < steps) load(i + 1);
#pragma unroll
            for (int k = 0; k < kDepth; ++k) {
                float a[kR];
                float2 c[4];
                if constexpr (kR == 8) {
                    *reinterpret_cast<float4 *>(a) = *reinterpret_cast<const float4 *>(&sa[now][k][ty * 4]);
                    *reinterpret_cast<float4 *>(a + 4) = *reinterpret_cast<const float4 *>(&sa[now][k][64 + ty * 4]);
                } else {
                    *reinterpret_cast<float2 *>(a) = *reinterpret_cast<const float2 *>(&sa[now][k][ty * 2]);
                }
                *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(&sb[now][k][tx * 4]);
                *reinterpret_cast<float4 *>(c + 2) = *reinterpret_cast<const float4 *>(&sb[now][k][64 + tx * 4]);
#pragma unroll
                for (int r = 0; r < kR; ++r)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[r][j] = fma2(both(a[r]), c[j], acc[r][j]);
            }
            if (i + 1 < steps) {
                stage<kAcrossA, kRows>(sa[now ^ 1], va);
                stage<kAcrossB, kTile>(sb[now ^ 1], vb);
            }
            // long sums in parts, so that their rounding does not grow with k
            if ((i & (kFold - 1)) == kFold - 1 && i + 1 < steps) {
#pragma unroll
                for (int q = 0; q < 2 * kR; ++q) {
                    float4 sum = folded ? totals[q * kThreads] : make_float4(0, 0, 0, 0);
                    float2 *two = &acc[q / 2][q % 2 * 2];
                    totals[q * kThreads] = make_float4(sum.x + two[0].x, sum.y + two[0].y, sum.z + two[1].x, sum.w + two[1].y);
                    two[0] = two[1] = make_float2(0, 0);
                }
                folded = true;
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int q = 0; q < 2 * kR; ++q) {
        float2 *two = &acc[q / 2][q % 2 * 2];
        if (folded) {
            const float4 sum = totals[q * kThreads];
            two[0] = add2(two[0], make_float2(sum.x, sum.y));
            two[1] = add2(two[1], make_float2(sum.z, sum.w));
        }
        if (parts > 1) totals[q * kThreads] = make_float4(two[0].x, two[0].y, two[1].x, two[1].y);
    }
    if (parts > 1) cluster_sync(parts);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        const int m = kR == 8 ? (r < 4 ? 0 : 60) + ty * 4 + r : ty * kR + r;
        if (parts > 1) {  // the parts' sums of every parts-th row
            if (r % parts != rank) continue;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float4 sum = make_float4(0, 0, 0, 0);
                for (int p = 0; p < parts; ++p) {
                    float4 v;
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                                 : "r"(peer_addr(totals + (2 * r + q) * kThreads, p))
                                 : "memory");
                    sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
                }
                acc[r][2 * q] = make_float2(sum.x, sum.y);
                acc[r][2 * q + 1] = make_float2(sum.z, sum.w);
            }
        }
        if (m >= m_left) continue;
        const int64_t row = place.row + m;
        float v[4] = {acc[r][0].x, acc[r][0].y, acc[r][1].x, acc[r][1].y};
        float w[4] = {acc[r][2].x, acc[r][2].y, acc[r][3].x, acc[r][3].y};
        if constexpr (kKind == kGated) {
            if (tx * 4 < n_left) finish<T, kKind, 4>(b, which, place.e, part, row, col0 + tx * 4, v, w, quads_out);
        } else {
            float spare[4];
            if (tx * 4 < n_left) finish<T, kKind, 4>(b, which, place.e, part, row, col0 + tx * 4, v, spare, quads_out);
            if (64 + tx * 4 < n_left) finish<T, kKind, 4>(b, which, place.e, part, row, col0 + 64 + tx * 4, w, spare, quads_out);
        }
    }
    if (parts > 1) cluster_sync(parts);  // the other CTAs have read this one's sums
}

template <typename T, int kKind, int kR>
int launch(const Block &b, int parts, cudaStream_t s) {
    constexpr int kRows = 16 * kR;
    // every row (and every segment's matrix) of these starts at a multiple of four values
    const auto quads = [&](std::initializer_list<const Matrix *> ms) {
        for (const Matrix *m : ms)
            if (m->p && ((reinterpret_cast<uintptr_t>(m->p) / sizeof(T) | static_cast<uint64_t>(m->ld) | static_cast<uint64_t>(m->expert)) % 4 ||
                         reinterpret_cast<uintptr_t>(m->p) % (4 * sizeof(T))))
                return false;
        return true;
    };
    bool qa, qb, qo;
    if (kKind == kGated) qa = quads({&b.x}), qb = quads({&b.wg, &b.wu}), qo = quads({&b.h, &b.gate, &b.up});
    else if (kKind == kDown) qa = quads({&b.h}), qb = quads({&b.wd}), qo = quads({&b.y});
    else if (kKind == kBack) qa = quads({&b.dy}), qb = quads({&b.wd}), qo = quads({&b.gate, &b.up, &b.dgate, &b.dup, &b.h});
    else if (kKind == kInput) qa = quads({&b.dgate, &b.dup}), qb = quads({&b.wg, &b.wu}), qo = quads({&b.dx});
    else qa = quads({&b.dgate, &b.dup, &b.dy}), qb = quads({&b.x, &b.h}), qo = quads({&b.dwg, &b.dwu, &b.dwd});
    int64_t gx, gy, gz = parts;
    if (kKind == kWeights) {
        gx = ceil_div(b.d, kTile) * ceil_div(b.f, kTile);
        gy = static_cast<int64_t>(b.seg.count) * b.splits;
        gz = 3;
    } else {
        gx = b.seg.rows / kRows + (b.seg.count < b.seg.rows ? b.seg.count : b.seg.rows) + 1;
        gy = ceil_div(product_columns<kKind>(b, 0), kKind == kGated ? kTile / 2 : kTile);
    }
    if (gx >= int64_t(1) << 31 || gy > 65535) return set_error(SPMV_ERR_TOO_LARGE, "the feed-forward block has too many tiles");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), static_cast<unsigned>(gz));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 2 * kR * kThreads * sizeof(float4);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = static_cast<unsigned>(parts);
    cfg.attrs = attr;
    cfg.numAttrs = parts > 1 ? 1 : 0;
    SPMV_TRY_CUDA(cudaFuncSetAttribute(k_ffn_simt<T, kKind, kR>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(cfg.dynamicSmemBytes)));
    SPMV_TRY_CUDA(cudaLaunchKernelEx(&cfg, k_ffn_simt<T, kKind, kR>, b, (qa ? 1u : 0u) | (qb ? 2u : 0u), qo));
    return SPMV_OK;
}
// Tiles of 32 rows for segments of up to that (taken as up to twice their mean, where there are several), and k in parts where
// the tiles would leave SMs without one.
template <typename T, int kKind>
int launch_shape(const Block &b, cudaStream_t s) {
    if constexpr (kKind == kWeights) {
        return launch<T, kKind, 8>(b, 1, s);
    } else {
        const int64_t rows = b.seg.rows, count = b.seg.count, used = count < rows ? count : rows;
        const bool few = (count == 1 ? rows : 2 * ceil_div(rows, count)) <= 32;
        const int64_t high = few ? 32 : 128, row_tiles = ceil_div(rows, high) > used ? ceil_div(rows, high) : used;
        const int64_t tiles = row_tiles * ceil_div(product_columns<kKind>(b, 0), kKind == kGated ? kTile / 2 : kTile);
        const int64_t depth = kKind == kGated || kKind == kBack ? b.d : b.f;
        int parts = 1;
        while (parts < kMaxCluster && tiles * parts < 2 * kSms && depth / (2 * parts) >= 4 * kDepth) parts *= 2;
        return few ? launch<T, kKind, 2>(b, parts, s) : launch<T, kKind, 8>(b, parts, s);
    }
}
template <typename T>
int launch_kind(int kind, const Block &b, cudaStream_t s) {
    switch (kind) {
        case kGated: return launch_shape<T, kGated>(b, s);
        case kDown: return launch_shape<T, kDown>(b, s);
        case kBack: return launch_shape<T, kBack>(b, s);
        case kInput: return launch_shape<T, kInput>(b, s);
        default: return launch_shape<T, kWeights>(b, s);
    }
}

}  // namespace

int launch_simt(int kind, const Block &b, int dtype, bool, cudaStream_t s) {
    if (dtype == SPMV_F32) return launch_kind<float>(kind, b, s);
    if (dtype == SPMV_F16) return launch_kind<__half>(kind, b, s);
    return launch_kind<__nv_bfloat16>(kind, b, s);
}

}  // namespace ffn
}  // namespace spmv
