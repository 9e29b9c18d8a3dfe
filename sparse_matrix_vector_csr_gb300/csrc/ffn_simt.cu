// The products of the feed-forward block by the ordinary units: float, and 16-bit values at any address.
// A CTA of 256 threads has 128 x 128 values of D, 8 x 8 a thread, in 32 bits; pieces of A and B of 16
// along k go through shared memory, k first, two of each so that one is filled while the other is
// multiplied.  Bound by the ordinary units' arithmetic (two multiply-adds an instruction) and the reads of shared memory that
// feed it, an equal share of cycles: 4096 rows, d = 2048, f = 4096, float: 43.6 TFLOP/s forward, 44.5 back.  Pieces of 8 along k:
// 34.9; A's values twice in shared memory, to be a pair's operand as they are: 34.4; 128 x 256 values, 8 x 16 a thread, one
// CTA an SM: 41.3.
#include "ffn.cuh"

namespace spmv {
namespace ffn {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;
constexpr int kDepth = 16;
constexpr int kPitch = kTile + 4;  // floats of a row in shared memory

// Thread t's eight values of a piece (kTile x kDepth) of an operand whose (0, 0) is at p.
// Along k: four of rows t / 4 and t / 4 + 64; along m or n: four of k = t / 32 and t / 32 + 8.
template <typename T, bool kAcross>
__device__ __forceinline__ void fetch(const T *p, const T *p2, int64_t ld, int64_t mn_left, int64_t mn_left2, int64_t k_left, bool quads,
                                      float (&v)[8]) {
    const int t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float *out = v + 4 * i;
        const int mn = kAcross ? (t & 31) * 4 : t / 4 + 64 * i, k = kAcross ? t / 32 + 8 * i : (t & 3) * 4;
        // along k the two halves of the rows may be of two matrices (p2: the second half's)
        const T *q = kAcross ? p + k * ld + mn : (i == 0 ? p : p2) + (t / 4) * ld + k;
        const int64_t rows = kAcross ? k_left - k : (i == 0 ? mn_left - mn : mn_left2 - (mn - 64));
        const int64_t run = kAcross ? mn_left - mn : k_left - k;  // values that follow on
        if (rows > 0 && run >= 4 && quads) {
            using U = typename Unit<4 * sizeof(T)>::type;
            unit_to_f32<T>(*reinterpret_cast<const U *>(q), out);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) out[j] = rows > 0 && j < run ? to_f32(q[j]) : 0.0f;
        }
    }
}
template <bool kAcross>
__device__ __forceinline__ void stage(float (*s)[kPitch], const float (&v)[8]) {
    const int t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (kAcross) {
            *reinterpret_cast<float4 *>(&s[t / 32 + 8 * i][(t & 31) * 4]) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[(t & 3) * 4 + j][t / 4 + 64 * i] = v[4 * i + j];
        }
    }
}

// The tile of `rows` rows that blockIdx.x counts over all segments, and behind them the rows in none.
struct Place {
    int e;
    int64_t row, end;  // its first row, the segment's end
};
__device__ bool find_tile(const Segments &seg, Place &place) {
    __shared__ int32_t part[kThreads / 32];
    __shared__ Place found;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int per = (seg.count + 1 + kThreads - 1) / kThreads;
    const auto tiles = [&](int e) {
        const Segments::Span s = seg.span(e);
        return static_cast<int32_t>((s.end - s.begin + kTile - 1) / kTile);
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
                found = Place{e, s.begin + static_cast<int64_t>(want - at) * kTile, s.end};
            }
            at += n;
        }
    __syncthreads();
    place = found;
    return place.e >= 0;
}

// D's tile of the CTA.  grid: x tiles of rows (kWeights: of the segment's matrix), y tiles of columns
// (kWeights: segments), z (kWeights) which of the three products.
template <typename T, int kKind>
__global__ void __launch_bounds__(kThreads, 2) k_ffn_simt(Block b, unsigned quads_in, bool quads_out) {
    __shared__ __align__(16) float sa[2][kDepth][kPitch], sb[2][kDepth][kPitch];
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
        if (!find_tile(b.seg, place)) return;
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
    float2 acc[8][4] = {};

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
        const bool qa = quads_in & 1, qb = quads_in & 2;
        const int64_t step_a = kAcrossA ? kDepth * lda : kDepth, step_b = kAcrossB ? kDepth * ldb : kDepth;
        const int64_t n2 = kKind == kGated ? n_left : n_left - 64;
        const int64_t steps = (depth + kDepth - 1) / kDepth;
        float va[8], vb[8];
        const auto load = [&](int64_t i) {
            const int64_t k_left = depth - i * kDepth;
            fetch<T, kAcrossA>(pa + i * step_a, pa + i * step_a + 64 * lda, lda, m_left, m_left - 64, k_left, qa, va);
            fetch<T, kAcrossB>(pb + i * step_b, pb2 + i * step_b, ldb, n_left, n2, k_left, qb, vb);
        };
        load(0);
        __syncthreads();  // (the pass before may still read)
        stage<kAcrossA>(sa[0], va);
        stage<kAcrossB>(sb[0], vb);
        __syncthreads();
        for (int64_t i = 0; i < steps; ++i) {
            const int now = i & 1;
            if (i + 1 < steps) load(i + 1);
#pragma unroll
            for (int k = 0; k < kDepth; ++k) {
                float a[8];
                float2 c[4];
                *reinterpret_cast<float4 *>(a) = *reinterpret_cast<const float4 *>(&sa[now][k][ty * 4]);
                *reinterpret_cast<float4 *>(a + 4) = *reinterpret_cast<const float4 *>(&sa[now][k][64 + ty * 4]);
                *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(&sb[now][k][tx * 4]);
                *reinterpret_cast<float4 *>(c + 2) = *reinterpret_cast<const float4 *>(&sb[now][k][64 + tx * 4]);
#pragma unroll
                for (int r = 0; r < 8; ++r)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[r][j] = fma2(both(a[r]), c[j], acc[r][j]);
            }
            if (i + 1 < steps) {
                stage<kAcrossA>(sa[now ^ 1], va);
                stage<kAcrossB>(sb[now ^ 1], vb);
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int m = (r < 4 ? 0 : 60) + ty * 4 + r;
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
}

template <typename T, int kKind>
int launch(const Block &b, cudaStream_t s) {
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
    int64_t gx, gy, gz = 1;
    if (kKind == kWeights) {
        gx = ceil_div(b.d, kTile) * ceil_div(b.f, kTile);
        gy = static_cast<int64_t>(b.seg.count) * b.splits;
        gz = 3;
    } else {
        gx = b.seg.rows / kTile + (b.seg.count < b.seg.rows ? b.seg.count : b.seg.rows) + 1;
        gy = ceil_div(product_columns<kKind>(b, 0), kKind == kGated ? kTile / 2 : kTile);
    }
    if (gx >= int64_t(1) << 31 || gy > 65535) return set_error(SPMV_ERR_TOO_LARGE, "the feed-forward block has too many tiles");
    k_ffn_simt<T, kKind><<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), static_cast<unsigned>(gz)), kThreads, 0, s>>>(
        b, (qa ? 1u : 0u) | (qb ? 2u : 0u), qo);
    SPMV_TRY_CUDA(cudaGetLastError());
    return SPMV_OK;
}
template <typename T>
int launch_kind(int kind, const Block &b, cudaStream_t s) {
    switch (kind) {
        case kGated: return launch<T, kGated>(b, s);
        case kDown: return launch<T, kDown>(b, s);
        case kBack: return launch<T, kBack>(b, s);
        case kInput: return launch<T, kInput>(b, s);
        default: return launch<T, kWeights>(b, s);
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
