// The products of the feed-forward block by the tensor cores: 16-bit values in matrices whose rows start at
// multiples of 16 bytes.
//
// A CTA an SM, which takes tiles of D in turn.  One warp has the tiles of A and B brought to shared memory
// (64 of k at a time, a ring of stages), one issues the products of a stage into an accumulator in tensor
// memory, four read a finished accumulator and write what becomes of it (ffn.cuh, finish) while the next
// tile's products go to the other accumulator.  Rows of a tile behind its segment's end are read (they
// belong to the next segment, or lie behind the matrix and read as 0) and their values of D not written;
// where sums run over rows (kWeights), they are replaced by 0 in shared memory, in A and in B, because 0
// times a NaN is none.
//
// Every wait ends after a second or two at the latest: the kernel then sets a flag that
// spmv_feed_forward_status reports, lets its copies and products in flight end, gives its tensor memory
// back and returns.
#pragma once

#include <cuda.h>

#include "ffn.cuh"

namespace spmv {
namespace ffn {
namespace tc {

constexpr int kThreads = 192;     // four warps that write D, one that copies, one that multiplies
constexpr int kWriters = 4;
constexpr int kRows = 128;        // of a tile of D: the accumulator's lanes
constexpr int kDepth = 64;        // of a stage: 128 bytes, the width of the swizzle
constexpr int kRowBytes = 128;
constexpr int kGroup = 16;        // row tiles that take turns before the next column tile, so that both stay in L2
constexpr unsigned long long kWaitNs = 2000000000ull;

struct Args {
    CUtensorMap a[3], b[3];
    Block block;
    int products;      // kWeights: how many of the three, and
    int which[3];      // which
    int *failed;
};

// ----------------------------------------------------------------------------
// barriers, copies, products
// ----------------------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
// false after kWaitNs, or when another warp has given up
static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int *gave_up, int *failed) {
    const unsigned long long t0 = now_ns();
    while (!bar_try(bar, parity)) {
        if (*gave_up) return false;
        if (now_ns() - t0 > kWaitNs) {
            *gave_up = 1;
            atomicExch(failed, 1);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *gave_up, int *failed) {
    return bar_try(bar, parity) || bar_wait_slow(bar, parity, gave_up, failed);
}
// the same by a whole warp, one answer for all lanes
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *gave_up, int *failed) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, gave_up, failed));
}
// one box of a tensor map to shared memory; the first coordinate is a multiple of 64 values
__device__ __forceinline__ void copy2(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void copy3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// An operand's tile in shared memory, 128-byte swizzle: along k, rows of 128 bytes (64 of k), eight rows
// 1024 bytes; along m or n, blocks of 64 of m or n, each of 64 rows (of k) of 128 bytes, so the next eight
// of k follow 1024 bytes on and the next block 8192.
template <bool kAcross>
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
    constexpr uint64_t kBlock = kAcross ? kDepth * kRowBytes : 16, kEight = 1024;
    return (static_cast<uint64_t>(addr >> 4) & 0x3fff) | (kBlock >> 4) << 16 | (kEight >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}
// 16 of k further on
template <bool kAcross>
constexpr uint32_t kStep = (kAcross ? 16 * kRowBytes : 32) >> 4;

// float accumulator, both operands of one 16-bit type
template <typename T, int kKind, int kN>
__device__ __forceinline__ constexpr uint32_t product_shape() {
    constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    return 1u << 4 | type << 7 | type << 10 | (a_transposed(kKind) ? 1u << 15 : 0u) | (b_transposed(kKind) ? 1u << 16 : 0u) |
           static_cast<uint32_t>(kN >> 3) << 17 | static_cast<uint32_t>(kRows >> 4) << 24;
}
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(shape), "r"(add ? 1u : 0u)
        : "memory");
}
// arrives when the products issued so far have been made
__device__ __forceinline__ void signal_done(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 16 columns of the warp's 32 lanes of the accumulator
__device__ __forceinline__ void read16(uint32_t addr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void read_done() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ----------------------------------------------------------------------------
// tiles
// ----------------------------------------------------------------------------
struct Tile {
    int e, which;
    int64_t row, end;   // of D: first row and where its rows end
    int64_t col;
    int64_t first, depth;  // kWeights: the segment's rows; else depth is k's extent (0: D is 0)
};

// Tiles of kTileRows x kCols columns; row tiles of the segments counted in `prefix` (its last entry: all).
template <int kKind, int kTileRows, int kCols>
struct Tiles {
    const Block &b;
    const Args &args;
    const int32_t *prefix;
    int64_t columns, total;
    __device__ __forceinline__ Tiles(const Args &a, const int32_t *p) : b(a.block), args(a), prefix(p) {
        if constexpr (kKind == kWeights) {
            total = 0;
            for (int i = 0; i < a.products; ++i) total += of(a.which[i]);
            columns = total;  // of one segment
            total *= b.seg.count;
        } else {
            columns = (product_columns<kKind>(b, 0) + kCols - 1) / kCols;
            total = columns * prefix[b.seg.count + (kKind == kBack ? 0 : 1)];
        }
    }
    __device__ __forceinline__ int64_t of(int which) const {
        return (weight_rows(b, which) + kTileRows - 1) / kTileRows * ((product_columns<kKind>(b, which) + kCols - 1) / kCols);
    }
    __device__ __forceinline__ Tile operator[](int64_t t) const {
        Tile r;
        r.which = 0;
        r.first = 0;
        if constexpr (kKind == kWeights) {
            r.e = static_cast<int>(t / columns);
            int64_t i = t - r.e * columns;
            for (int p = 0;; ++p) {
                r.which = args.which[p];
                const int64_t n = of(r.which);
                if (i < n) break;
                i -= n;
            }
            r.end = weight_rows(b, r.which);
            const int64_t m = (r.end + kTileRows - 1) / kTileRows;
            r.row = i % m * kTileRows;
            r.col = i / m * kCols;
            const Segments::Span s = b.seg.span(r.e);
            r.first = s.begin;
            r.depth = s.end - s.begin;
        } else {
            int lo = 0, hi = b.seg.count + 1;  // prefix[lo] * columns <= t < prefix[hi] * columns
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (prefix[mid] * columns <= t) lo = mid;
                else hi = mid;
            }
            r.e = lo;
            const int64_t i = t - prefix[lo] * columns;
            const int m = prefix[lo + 1] - prefix[lo];
            const int64_t g = i / (kGroup * columns), j = i - g * kGroup * columns;
            const int64_t in_group = min(static_cast<int64_t>(m) - g * kGroup, static_cast<int64_t>(kGroup));
            const Segments::Span s = b.seg.span(lo);
            r.row = s.begin + (g * kGroup + j % in_group) * kTileRows;
            r.end = s.end;
            r.col = j / in_group * kCols;
            r.depth = lo == b.seg.count ? 0 : kKind == kGated || kKind == kBack ? b.d : b.f;
        }
        return r;
    }
};

// prefix[e] = row tiles of the segments in front of e, e = 0 .. count + 1 (segment `count`: the rows behind the last)
template <int kTileRows>
__device__ void count_tiles(const Segments &seg, int32_t *prefix) {
    __shared__ int32_t part[kThreads / 32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int per = (seg.count + 1 + kThreads - 1) / kThreads;
    const auto tiles = [&](int e) {
        const Segments::Span s = seg.span(e);
        return static_cast<int32_t>((s.end - s.begin + kTileRows - 1) / kTileRows);
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
    __syncthreads();
    int32_t at = incl - mine;
    for (int w = 0; w < warp; ++w) at += part[w];
    for (int i = 0; i < per; ++i)
        if (t * per + i <= seg.count) {
            prefix[t * per + i] = at;
            at += tiles(t * per + i);
            if (t * per + i == seg.count) prefix[seg.count + 1] = at;
        }
    __syncthreads();
}

// ----------------------------------------------------------------------------
// the kernel
// ----------------------------------------------------------------------------
// kN columns of the accumulator (kGated: kN / 2 of gate, then as many of up); kLoaded rows of A's tile are
// copied where segments are short (the accumulator's other lanes then hold sums of whatever lies behind
// them in the ring, which nothing reads).
template <int kKind, int kN, int kLoaded>
struct Shape {
    static constexpr int kCols = kKind == kGated ? kN / 2 : kN;
    static constexpr int kTileRows = kKind == kWeights ? kRows : kLoaded;
    static constexpr int kABytes = kTileRows * kRowBytes, kBBytes = kN * kRowBytes;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kSlack = kRows * kRowBytes - kABytes;  // behind the ring: what the last stage's product reads
    static constexpr int kRoom = 200 * 1024 - kSlack;
    static constexpr int kStages = kRoom / kStageBytes > 16 ? 16 : kRoom / kStageBytes;
    static constexpr int kColumns = 2 * kN;  // of tensor memory: two accumulators
    static size_t smem(int segments) { return 1024 + kStages * kStageBytes + kSlack + (2 * kStages + 5) * 8 + (segments + 2) * 4; }
};

template <typename T, int kKind, int kN, int kLoaded>
__global__ void __launch_bounds__(kThreads, 1) k_ffn(const __grid_constant__ Args args, bool whole) {
    using S = Shape<kKind, kN, kLoaded>;
    constexpr bool kAcrossA = a_transposed(kKind), kAcrossB = b_transposed(kKind);
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t raw[];
    __shared__ uint32_t tmem_at;
    __shared__ int gave_up_at;
    const uint32_t ring_b = (smem_addr(raw) + 1023) & ~1023u;       // B's stages, then A's: each a multiple of 1024 bytes
    const uint32_t ring_a = ring_b + kStages * S::kBBytes;
    const uint32_t bars = ring_a + kStages * S::kABytes + S::kSlack;
    const auto full = [&](int s) { return bars + 8 * s; };
    const auto empty = [&](int s) { return bars + 8 * (kStages + s); };
    const auto acc_full = [&](int i) { return bars + 8 * (2 * kStages + i); };
    const auto acc_empty = [&](int i) { return bars + 8 * (2 * kStages + 2 + i); };
    const uint32_t drained = bars + 8 * (2 * kStages + 4);
    int32_t *prefix = reinterpret_cast<int32_t *>(raw + (bars + 8 * (2 * kStages + 5) - smem_addr(raw)));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *gave_up = &gave_up_at;
    int *failed = args.failed;

    if (threadIdx.x == 0) {
        gave_up_at = 0;
        for (int s = 0; s < kStages; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(acc_full(i), 1);
            bar_init(acc_empty(i), kWriters);
        }
        bar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWriters + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_at)), "n"(S::kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        fence_before();
    }
    if constexpr (kKind != kWeights) count_tiles<S::kTileRows>(args.block.seg, prefix);
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_at;
    const Tiles<kKind, S::kTileRows, S::kCols> tiles(args, prefix);
    const auto stages_of = [&](const Tile &t) { return static_cast<int>((t.depth + kDepth - 1) / kDepth) * (kKind == kInput ? 2 : 1); };

    if (warp == kWriters) {
        if (lane == 0) {
            int s = 0, round = 0;
            bool ok = true;
            for (int64_t i = blockIdx.x; ok && i < tiles.total; i += gridDim.x) {
                const Tile t = tiles[i];
                const int n = stages_of(t), once = kKind == kInput ? n / 2 : n;
                for (int q = 0; q < n; ++q) {
                    if (!(ok = bar_wait(empty(s), (round & 1) ^ 1, gave_up, failed))) break;
                    bar_expect(full(s), S::kStageBytes);
                    const int pass = q >= once, k = (pass ? q - once : q) * kDepth;
                    const uint32_t a = ring_a + s * S::kABytes, b = ring_b + s * S::kBBytes;
                    const int row = static_cast<int>(t.row), col = static_cast<int>(t.col);
                    if constexpr (kAcrossA) {
                        const int k0 = static_cast<int>(t.first) + k;
#pragma unroll
                        for (int j = 0; j < S::kTileRows / 64; ++j)
                            copy2(a + j * (kDepth * kRowBytes), &args.a[t.which], row + j * 64, k0, full(s));
#pragma unroll
                        for (int j = 0; j < kN / 64; ++j)
                            copy2(b + j * (kDepth * kRowBytes), &args.b[t.which], col + j * 64, k0, full(s));
                    } else {
                        copy2(a, &args.a[pass], k, row, full(s));
                        if constexpr (kKind == kGated) {
                            copy3(b, &args.b[0], k, col, t.e, full(s));
                            copy3(b + kN / 2 * kRowBytes, &args.b[1], k, col, t.e, full(s));
                        } else if constexpr (kAcrossB) {
#pragma unroll
                            for (int j = 0; j < kN / 64; ++j)
                                copy3(b + j * (kDepth * kRowBytes), &args.b[pass], col + j * 64, k, t.e, full(s));
                        } else {
                            copy3(b, &args.b[0], k, col, t.e, full(s));
                        }
                    }
                    if (++s == kStages) {
                        s = 0;
                        ++round;
                    }
                }
            }
            // the ring is empty again (given up: at least every copy has landed)
            for (int j = 0; j < kStages; ++j) {
                const int last = j < s ? round : round - 1;  // the round in which the stage was filled last
                if (last < 0) continue;
                if (ok) ok = bar_wait(empty(j), last & 1, gave_up, failed);
                if (!ok) {
                    const unsigned long long t0 = now_ns();
                    while (!bar_try(full(j), last & 1) && now_ns() - t0 < kWaitNs) {}
                }
            }
        }
        __syncwarp();
    } else if (warp == kWriters + 1) {
        constexpr uint32_t shape = product_shape<T, kKind, kN>();
        int s = 0, round = 0, done = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < tiles.total; i += gridDim.x) {
            const Tile t = tiles[i];
            const int n = stages_of(t);
            if (n == 0) continue;
            const int which = done & 1;
            if (!(ok = warp_wait(acc_empty(which), ((done >> 1) & 1) ^ 1, gave_up, failed))) break;
            fence_after();
            const uint32_t d = tmem + which * kN;
            for (int q = 0; q < n; ++q) {
                if (!(ok = warp_wait(full(s), round & 1, gave_up, failed))) break;
                fence_after();
                const uint32_t a = ring_a + s * S::kABytes, b = ring_b + s * S::kBBytes;
                int steps = kDepth / 16;
                if constexpr (kKind == kWeights) {
                    const int64_t left = t.depth - static_cast<int64_t>(q) * kDepth;
                    if (left < kDepth) {  // rows of other segments, up to a whole 16 of k
                        steps = static_cast<int>((left + 15) / 16);
                        constexpr int kBlocks = kRows / 64 + kN / 64;
                        const int begin = static_cast<int>(left), rows = steps * 16 - begin;
                        for (int j = lane; j < rows * kBlocks * 8; j += 32) {
                            const int piece = j & 7, block = (j >> 3) % kBlocks, row = begin + (j >> 3) / kBlocks;
                            const uint32_t at = (block < kRows / 64 ? a + block * (kDepth * kRowBytes)
                                                                    : b + (block - kRows / 64) * (kDepth * kRowBytes)) +
                                                row * kRowBytes + piece * 16;
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                }
                if (lane == 0) {
                    uint64_t da = operand<kAcrossA>(a), db = operand<kAcrossB>(b);
                    for (int k = 0; k < steps; ++k) {
                        multiply(d, da, db, shape, q > 0 || k > 0);
                        da += kStep<kAcrossA>;
                        db += kStep<kAcrossB>;
                    }
                    signal_done(empty(s));
                    if (q == n - 1) signal_done(acc_full(which));
                }
                __syncwarp();
                if (++s == kStages) {
                    s = 0;
                    ++round;
                }
            }
            ++done;
        }
        if (!ok && lane == 0) {  // given up: the products in flight end before their memory is given back
            signal_done(drained);
            const unsigned long long t0 = now_ns();
            while (!bar_try(drained, 0) && now_ns() - t0 < kWaitNs) {}
        }
        __syncwarp();
    } else {
        int done = 0;
        const Block &b = args.block;
        for (int64_t i = blockIdx.x; i < tiles.total; i += gridDim.x) {
            const Tile t = tiles[i];
            const bool zero = stages_of(t) == 0;
            const int which = done & 1;
            if (!zero) {
                if (!warp_wait(acc_full(which), (done >> 1) & 1, gave_up, failed)) break;
                fence_after();
                ++done;
            }
            const int64_t row = t.row + warp * 32 + lane;
            const bool mine = row < t.end && warp * 32 + lane < S::kTileRows;
            const uint32_t from = tmem + which * kN + (static_cast<uint32_t>(warp * 32) << 16);
            const int64_t columns = product_columns<kKind>(b, t.which);
            if (warp * 32 < S::kTileRows) {
#pragma unroll 1
                for (int c = 0; c < S::kCols && t.col + c < columns; c += 16) {
                    float v[16], w[16];
                    if (!zero) {
                        read16(from + c, v);
                        if constexpr (kKind == kGated) read16(from + kN / 2 + c, w);
                        read_done();
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = w[j] = 0.0f;
                    }
                    if (mine) {
#pragma unroll
                        for (int j = 0; j < 16; j += 8)
                            if (t.col + c + j < columns) finish<T, kKind, 8>(b, t.which, t.e, row, t.col + c + j, v + j, w + j, whole);
                    }
                }
            }
            if (!zero) {
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(acc_empty(which));
            }
        }
    }
    __syncthreads();
    if (warp == kWriters + 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kColumns) : "memory");
    }
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------
// ffn_tc.cu
using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                            const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder();  // nullptr where the driver has none
int *failure_flag();

// `count` matrices (0: one, as a map of two dimensions) of `rows` rows of `n` values; boxes of 64 values x box_rows
template <typename T>
bool make_map(CUtensorMap *map, const Matrix &m, int64_t n, int64_t rows, int64_t count, int box_rows) {
    const cuuint64_t sizes[3] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(count ? count : 1)};
    // (one matrix: its distance to the next is not used, but has to be a valid one)
    const int64_t apart = count > 1 ? m.expert : ceil_div((rows - 1) * m.ld + n, 8) * 8;
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(m.ld) * sizeof(T), static_cast<cuuint64_t>(apart) * sizeof(T)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, step[3] = {1, 1, 1};
    return encoder()(map, std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     count ? 3 : 2, m.p, sizes, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int kKind, int kN, int kLoaded>
int launch(const Block &b, cudaStream_t s) {
    using S = Shape<kKind, kN, kLoaded>;
    Args args;
    args.block = b;
    args.failed = failure_flag();
    args.products = 0;
    const int64_t rows = b.seg.rows, d = b.d, f = b.f, count = b.seg.count;
    const auto activation = [&](CUtensorMap *map, const Matrix &m, int64_t n) {
        return make_map<T>(map, m, n, rows, 0, kKind == kWeights ? kDepth : S::kTileRows);
    };
    bool ok = true;
    int64_t tiles = 0;
    if (kKind == kWeights) {
        const Matrix *out[3] = {&b.dwg, &b.dwu, &b.dwd}, *in[3] = {&b.dgate, &b.dup, &b.dy};
        for (int i = 0; i < 3; ++i) {
            if (!out[i]->p) continue;
            args.which[args.products++] = i;
            ok = ok && activation(&args.a[i], *in[i], weight_rows(b, i)) && activation(&args.b[i], i == 2 ? b.h : b.x, i == 2 ? f : d);
            tiles += ceil_div(weight_rows(b, i), kRows) * ceil_div(product_columns<kKind>(b, i), kN) * count;
        }
    } else if (kKind == kGated) {
        ok = activation(&args.a[0], b.x, d) && make_map<T>(&args.b[0], b.wg, d, f, count, kN / 2) && make_map<T>(&args.b[1], b.wu, d, f, count, kN / 2);
    } else if (kKind == kDown) {
        ok = activation(&args.a[0], b.h, f) && make_map<T>(&args.b[0], b.wd, f, d, count, kN);
    } else if (kKind == kBack) {
        ok = activation(&args.a[0], b.dy, d) && make_map<T>(&args.b[0], b.wd, f, d, count, kDepth);
    } else {
        ok = activation(&args.a[0], b.dgate, f) && activation(&args.a[1], b.dup, f) && make_map<T>(&args.b[0], b.wg, d, f, count, kDepth) &&
             make_map<T>(&args.b[1], b.wu, d, f, count, kDepth);
    }
    if (!ok) return set_error(SPMV_ERR_CUDA, "the feed-forward block's matrices could not be described to the copy engine");
    if (kKind != kWeights)
        tiles = ceil_div(product_columns<kKind>(b, 0), S::kCols) * (rows / S::kTileRows + (count < rows ? count : rows) + 1);
    const size_t smem = S::smem(static_cast<int>(count));
    SPMV_TRY_CUDA(cudaFuncSetAttribute(k_ffn<T, kKind, kN, kLoaded>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
    k_ffn<T, kKind, kN, kLoaded><<<static_cast<unsigned>(tiles < kSms ? tiles : kSms), kThreads, smem, s>>>(args, true);
    SPMV_TRY_CUDA(cudaGetLastError());
    return SPMV_OK;
}

template <typename T>
int launch_kind(int kind, const Block &b, cudaStream_t s) {
    // rows of a segment that a tile has at least, taking segments as equally long
    const int64_t rows = ceil_div(b.seg.rows, b.seg.count);
    const bool few = rows <= 16;
    const auto small = [&](int64_t columns) { return (b.seg.rows / kRows + 1) * columns < kSms; };
    switch (kind) {
        case kGated: return few ? launch<T, kGated, 64, 16>(b, s) : small(ceil_div(b.f, 128)) ? launch<T, kGated, 64, 128>(b, s) : launch<T, kGated, 256, 128>(b, s);
        case kDown: return few ? launch<T, kDown, 64, 16>(b, s) : small(ceil_div(b.d, 256)) ? launch<T, kDown, 64, 128>(b, s) : launch<T, kDown, 256, 128>(b, s);
        case kBack: return few ? launch<T, kBack, 64, 16>(b, s) : small(ceil_div(b.f, 256)) ? launch<T, kBack, 64, 128>(b, s) : launch<T, kBack, 256, 128>(b, s);
        case kInput: return few ? launch<T, kInput, 64, 16>(b, s) : small(ceil_div(b.d, 256)) ? launch<T, kInput, 64, 128>(b, s) : launch<T, kInput, 256, 128>(b, s);
        default: {
            const int64_t tiles = ceil_div(b.f, kRows) * ceil_div(b.d, 256) * b.seg.count;
            return tiles * 3 < kSms ? launch<T, kWeights, 64, 128>(b, s) : launch<T, kWeights, 256, 128>(b, s);
        }
    }
}

}  // namespace tc
}  // namespace ffn
}  // namespace spmv
