// The products of the feed-forward block by the tensor cores: 16-bit values in matrices whose rows start at
// multiples of 16 bytes.
//
// A CTA an SM (or a pair of CTAs on two SMs), which takes tiles of D in turn.  One warp has the tiles of A and B
// brought to shared memory (64 of k at a time, a ring of stages), one issues the products of a stage into an
// accumulator in tensor memory, eight read a finished accumulator and write what becomes of it while the
// next tile's products go to the other accumulator.  A pair has 256 x 256 values of D, each CTA its 128 rows:
// each brings its rows of A and half of B, and the first CTA's products read both halves, so an SM takes in a
// third less for each product.  Rows of a tile behind its segment's end are read (they belong to the next
// segment, or lie behind the matrix and read as 0) and their values of D not written; where sums run over
// rows (kWeights), they are replaced by 0 in shared memory, in A and in B, because 0 times a NaN is none.
//
// Every wait ends after about two seconds at the latest: the kernel then sets a flag that
// spmv_feed_forward_status reports, lets its copies and products in flight end, gives its tensor memory
// back and returns.
#pragma once

#include <cuda.h>

#include "ffn.cuh"

namespace spmv {
namespace ffn {
namespace tc {

constexpr int kWriters = 8;       // warps that write D; behind them one that copies and one that multiplies
// (kWeights: one more, that clears what is not the segment's)
constexpr int threads_of(int kind) { return (kWriters + (kind == kWeights ? 3 : 2)) * 32; }
constexpr int kThreads = threads_of(kGated);
constexpr int kRows = 128;        // of a tile of D: the accumulator's lanes
constexpr int kDepth = 64;        // of a stage: 128 bytes, the width of the swizzle
constexpr int kRowBytes = 128;
constexpr int kGroupRows = 2048;  // of the row tiles that take turns before the next column tile, so that both stay in L2
constexpr int kSharedBytes = 227 * 1024 - 256;  // dynamic; the rest for the variables of fixed size
constexpr int kMaxStages = 32;
constexpr int kFewRows = kShortRows;  // of a tile where segments are short
constexpr long long kWaitCycles = 4000000000LL;  // about two seconds

struct Args {
    CUtensorMap a[3], b[3];
    Block block;
    int products;      // kWeights: how many of the three, and
    int which[3];      // which
    int stages;        // of the ring
    bool follows;      // launched behind a kernel of the same call that may still run
};

// a wait of one of this file's kernels ran out (each file that includes this has its own)
static __device__ int gave_up_flag;

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
// the same barrier in the pair's first CTA
__device__ __forceinline__ uint32_t bar_first(uint32_t bar) {
    uint32_t there;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(bar));
    return there;
}
// arrives there; kRelease: what the warp wrote to shared memory is seen by whoever waits
template <bool kRelease>
__device__ __forceinline__ void bar_arrive_first(uint32_t bar) {
    if constexpr (kRelease) asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_first(bar)) : "memory");
    else asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_first(bar)) : "memory");
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
// true in one lane of a whole warp.  The copies and products take their operands from registers that a warp
// shares; where the compiler cannot see that one lane alone is there, it walks over the lanes for each of them.
__device__ __forceinline__ bool one_lane() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}
// false after kWaitCycles, or when another warp has given up (the clock and the flag are looked at now and then only:
// a wait's end is seen at once)
template <bool kNap>
static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int *gave_up) {
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i) {
            if (bar_try(bar, parity)) return true;
            if (kNap) __nanosleep(64);
        }
        if (*gave_up) return false;
        if (clock64() - t0 > kWaitCycles) {
            *gave_up = 1;
            atomicExch(&gave_up_flag, 1);
            return false;
        }
    }
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *gave_up) {
    return bar_try(bar, parity) || bar_wait_slow<false>(bar, parity, gave_up);
}
// the same for a whole warp, by one of its lanes; kNap: one that does not mind to see it a little later
template <bool kNap>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *gave_up) {
    bool ok = true;
    if (one_lane()) ok = bar_try(bar, parity) || bar_wait_slow<kNap>(bar, parity, gave_up);
    return __all_sync(0xffffffffu, ok);
}
// one box of a tensor map to shared memory, counted on a barrier of this CTA or (kPair) of either of the pair; the
// first coordinate is a multiple of 64 values
template <bool kPair>
__device__ __forceinline__ void copy2(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    if constexpr (kPair)
        asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                     "l"(map), "r"(x), "r"(y), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                     "l"(map), "r"(x), "r"(y), "r"(bar)
                     : "memory");
}
template <bool kPair>
__device__ __forceinline__ void copy3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    if constexpr (kPair)
        asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                     "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
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
template <typename T, int kKind, int kN, bool kPair>
__device__ __forceinline__ constexpr uint32_t product_shape() {
    constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    return 1u << 4 | type << 7 | type << 10 | (a_transposed(kKind) ? 1u << 15 : 0u) | (b_transposed(kKind) ? 1u << 16 : 0u) |
           static_cast<uint32_t>(kN >> 3) << 17 | static_cast<uint32_t>((kPair ? 2 : 1) * kRows >> 4) << 24;
}
template <bool kPair>
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(shape), "r"(add ? 1u : 0u)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(shape), "r"(add ? 1u : 0u)
            : "memory");
}
// arrives (at the barrier of both CTAs of a pair) when the products issued so far have been made
template <bool kPair>
__device__ __forceinline__ void signal_done(uint32_t bar) {
    if constexpr (kPair)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                     "h"(static_cast<uint16_t>(3))
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 columns of the warp's 32 lanes of the accumulator
__device__ __forceinline__ void read32(uint32_t addr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void read_done() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ----------------------------------------------------------------------------
// tiles
// ----------------------------------------------------------------------------
struct Tile {
    int e, which, part;
    int64_t row, end;   // of D: first row and where its rows end
    int64_t col;
    int64_t first, depth;  // kWeights: the segment's rows; else depth is k's extent (0: D is 0)
};

// Tiles of kTileRows x kCols columns; row tiles of the segments counted in `prefix` (its last entry: all).  Fewer than
// 2^31, so that a tile's place takes divisions of 32 bits: it is worked out between two tiles' copies, and the ring has
// to cover what that takes (weights' gradients of 64 experts, 6144 tiles: 597 us, with divisions of 64 bits 615).
template <int kKind, int kTileRows, int kCols>
struct Tiles {
    const Block &b;
    const Args &args;
    const int32_t *prefix;
    uint32_t columns, total;
    int e = 0;  // the segment of the last tile asked for: those asked for next lie in it or behind
    __device__ __forceinline__ Tiles(const Args &a, const int32_t *p) : b(a.block), args(a), prefix(p) {
        if constexpr (kKind == kWeights) {
            columns = 0;  // of one part of a segment
            for (int i = 0; i < a.products; ++i) columns += of(a.which[i]);
            total = columns * static_cast<uint32_t>(b.seg.count * b.splits);
        } else {
            columns = static_cast<uint32_t>((product_columns<kKind>(b, 0) + kCols - 1) / kCols);
            total = columns * static_cast<uint32_t>(prefix[b.seg.count + (kKind == kBack ? 0 : 1)]);
        }
    }
    __device__ __forceinline__ uint32_t of(int which) const {
        return static_cast<uint32_t>((weight_rows(b, which) + kTileRows - 1) / kTileRows * ((product_columns<kKind>(b, which) + kCols - 1) / kCols));
    }
    __device__ __forceinline__ Tile operator[](uint32_t t) {
        Tile r;
        r.which = r.part = 0;
        r.first = 0;
        if constexpr (kKind == kWeights) {
            const uint32_t parts = t / columns, splits = static_cast<uint32_t>(b.splits);
            uint32_t i = t - parts * columns;
            r.e = static_cast<int>(parts / splits);
            r.part = static_cast<int>(parts - r.e * splits);
            for (int p = 0;; ++p) {
                r.which = args.which[p];
                const uint32_t n = of(r.which);
                if (i < n) break;
                i -= n;
            }
            r.end = weight_rows(b, r.which);
            const uint32_t m = static_cast<uint32_t>((r.end + kTileRows - 1) / kTileRows), col = i / m;
            r.row = static_cast<int64_t>(i - col * m) * kTileRows;
            r.col = static_cast<int64_t>(col) * kCols;
            const Segments::Span s = b.part(r.e, r.part);
            r.first = s.begin;
            r.depth = s.end - s.begin;
        } else {
            while (e < b.seg.count && static_cast<uint32_t>(prefix[e + 1]) * columns <= t) ++e;
            r.e = e;
            constexpr uint32_t kGroup = kGroupRows / kTileRows;
            const uint32_t i = t - static_cast<uint32_t>(prefix[e]) * columns, m = static_cast<uint32_t>(prefix[e + 1] - prefix[e]);
            const uint32_t g = i / (kGroup * columns), j = i - g * kGroup * columns;
            const uint32_t in_group = min(m - g * kGroup, kGroup), col = j / in_group;
            const Segments::Span s = b.seg.span(e);
            r.row = s.begin + static_cast<int64_t>(g * kGroup + j - col * in_group) * kTileRows;
            r.end = s.end;
            r.col = static_cast<int64_t>(col) * kCols;
            r.depth = e == b.seg.count ? 0 : kKind == kGated || kKind == kBack ? b.d : b.f;
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
// D's way out
// ----------------------------------------------------------------------------
// A warp's 32 rows x 32 columns of 16-bit values in shared memory: rows of 64 bytes, the 16-byte pieces of two
// rows placed so that neither a row a lane nor four lanes a row meet in a bank.
constexpr int kPatchBytes = 32 * 64;
__device__ __forceinline__ uint32_t patch_piece(uint32_t patch, int row, int piece) {
    return patch + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint4 patch_load(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void patch_store(uint32_t at, const uint4 &v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// the patch's first `rows` rows to p, `left` of a row's columns there; four lanes a row, 64 bytes
template <typename T>
__device__ __forceinline__ void patch_out(uint32_t patch, T *p, int64_t ld, int rows, int64_t left) {
    const int lane = threadIdx.x & 31, piece = lane & 3;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + lane / 4;
        const uint4 v = patch_load(patch_piece(patch, r, piece));
        if (r < rows) {
            T *q = p + r * ld + piece * 8;
            if (left >= piece * 8 + 8) {
                *reinterpret_cast<uint4 *>(q) = v;
            } else {
                const T *values = reinterpret_cast<const T *>(&v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (piece * 8 + j < left) q[j] = values[j];
            }
        }
    }
    __syncwarp();
}
// the lane's row of the patch, rounded to the type
template <typename T>
__device__ __forceinline__ void patch_row(uint32_t patch, const float *v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) patch_store(patch_piece(patch, lane, i), pack<T>(v + 8 * i));
}
// asks for a patch's values from p (rows and columns outside: 0)
template <typename T>
__device__ __forceinline__ void patch_in(uint32_t patch, const T *p, int64_t ld, int rows, int64_t left) {
    const int lane = threadIdx.x & 31, piece = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + lane / 4;
        const int64_t n = r < rows ? min(max(left - piece * 8, int64_t(0)), int64_t(8)) : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(patch_piece(patch, r, piece)),
                     "l"(n ? p + r * ld + piece * 8 : p), "r"(static_cast<int>(n) * 2)
                     : "memory");
    }
}

// A whole warp: the rows (of k) from `left` to the next multiple of 16 of a stage of kWeights become 0 in A's tile and
// in kColumns of B's.
template <int kColumns>
__device__ __forceinline__ void clear_rows(uint32_t a, uint32_t b, int left) {
    constexpr int kBlocks = kRows / 64 + kColumns / 64;
    const int rows = (left + 15) / 16 * 16 - left;
    for (int j = threadIdx.x & 31; j < rows * kBlocks * 8; j += 32) {
        const int piece = j & 7, block = (j >> 3) % kBlocks, row = left + (j >> 3) / kBlocks;
        const uint32_t at = (block < kRows / 64 ? a + block * (kDepth * kRowBytes) : b + (block - kRows / 64) * (kDepth * kRowBytes)) +
                            row * kRowBytes + piece * 16;
        patch_store(at, make_uint4(0, 0, 0, 0));
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// ----------------------------------------------------------------------------
// the kernel
// ----------------------------------------------------------------------------
// kN columns of the accumulator (kGated: half of them gate's, then as many of up); kLoaded rows of A's tile are
// copied where segments are short (8 or 16; the accumulator's other lanes then hold sums of whatever lies behind
// them in the ring, which nothing reads).  What a stage costs besides its products (two waits and a signal, about
// 160 ns) is shared by several 64s of k where those are short, and tiles of 64 columns take turns with four
// accumulators, so that a product need not wait for the one in front (100 rows, d = f = 2048, forward and back: 94.9 us;
// with one accumulator 110.3, with one 64 of k a stage 99.7; 4 rows, d = 4096, f = 12288, forward: 65.7 us, with four
// accumulators 67.3, with one 64 of k a stage 91.2).
template <int kKind, int kN, int kLoaded, bool kPair>
struct Shape {
    static constexpr bool kTwoParts = kKind == kDown && kLoaded <= kFewRows;  // of h, one behind the other in A's tile
    static constexpr int kCtas = kPair ? 2 : 1;
    static constexpr int kCols = kKind == kGated ? kN / 2 : kN;
    static constexpr int kMine = kKind == kWeights ? kRows : kLoaded;  // rows of D that a CTA has
    static constexpr int kTileRows = kMine * kCtas;
    static constexpr int kAccs = kN == 256 || kLoaded <= kFewRows ? 1 : 4;
    static constexpr int kABytes = (kTwoParts ? 2 : 1) * kMine * kRowBytes, kBBytes = kN / kCtas * kRowBytes;
    static constexpr int kBlocks = kKind == kWeights || kN == 256 ? 1 : kLoaded == kRows ? 2 : 4;  // 64s of k of a stage
    static constexpr int kBlockBytes = kABytes + kBBytes, kStageBytes = kBlocks * kBlockBytes;
    static constexpr int kSlack = kRows * kRowBytes - kABytes;  // behind the ring: what the last stage's product reads
    // (kBack: gate and up, in whose place their gradients and then h go out; a second pair to ask for the next columns earlier
    // costs two of the ring's six stages: 8192 rows, d = f = 4096: 206 us, so 180)
    static constexpr int kWriterBytes = (kKind == kBack ? 2 : 1) * kPatchBytes;
    static constexpr int kFixed = 1024 + kSlack + kWriters * kWriterBytes + (4 * kMaxStages + 5) * 8;
    static constexpr int kColumns = 2 * kN * kAccs;  // of tensor memory: two buffers
    static int stages(int segments) {
        const int n = (kSharedBytes - kFixed - (segments + 2) * 4) / kStageBytes;
        return n > kMaxStages ? kMaxStages : n;
    }
    static size_t smem(int segments, int stages) { return kFixed + stages * kStageBytes + (segments + 2) * 4; }
};

template <typename T, int kKind, int kN, int kLoaded, bool kPair>
__global__ void __launch_bounds__(threads_of(kKind), 1) k_ffn(const __grid_constant__ Args args) {
    using S = Shape<kKind, kN, kLoaded, kPair>;
    constexpr bool kAcrossA = a_transposed(kKind), kAcrossB = b_transposed(kKind);
    extern __shared__ uint8_t raw[];
    __shared__ uint32_t tmem_at;
    __shared__ int gave_up_at;
    const int stages = args.stages;
    const uint32_t ring_b = (smem_addr(raw) + 1023) & ~1023u;       // B's stages, then A's: each a multiple of 1024 bytes
    const uint32_t ring_a = ring_b + stages * S::kBlocks * S::kBBytes;
    const uint32_t patches = ring_a + stages * S::kBlocks * S::kABytes + S::kSlack;
    const uint32_t bars = patches + kWriters * S::kWriterBytes;
    const auto full = [&](int s) { return bars + 8 * s; };
    const auto empty = [&](int s) { return bars + 8 * (kMaxStages + s); };
    // a segment's last rows (kWeights), which every CTA has to clear something in first: here, and cleared in every CTA
    const auto rest_full = [&](int s) { return bars + 8 * (2 * kMaxStages + s); };
    const auto cleared = [&](int s) { return bars + 8 * (3 * kMaxStages + s); };
    const auto acc_full = [&](int i) { return bars + 8 * (4 * kMaxStages + i); };
    const auto acc_empty = [&](int i) { return bars + 8 * (4 * kMaxStages + 2 + i); };
    const uint32_t drained = bars + 8 * (4 * kMaxStages + 4);
    int32_t *prefix = reinterpret_cast<int32_t *>(raw + (bars + 8 * (4 * kMaxStages + 5) - smem_addr(raw)));
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;  // (seen to be the warp's)
    const int rank = kPair ? static_cast<int>(blockIdx.x & 1) : 0;  // in the pair
    const uint32_t first = blockIdx.x / S::kCtas, step = gridDim.x / S::kCtas;
    volatile int *gave_up = &gave_up_at;

    if (threadIdx.x == 0) {
        gave_up_at = 0;
        for (int s = 0; s < stages; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
            bar_init(rest_full(s), 1);
            bar_init(cleared(s), S::kCtas);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(acc_full(i), 1);
            bar_init(acc_empty(i), kWriters * S::kCtas);
        }
        bar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWriters + 1) {
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_at)), "n"(S::kColumns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_at)), "n"(S::kColumns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
        fence_before();
    }
    if constexpr (kKind != kWeights) count_tiles<S::kTileRows>(args.block.seg, prefix);
    __syncthreads();
    if constexpr (kPair) cluster_sync(2);
    fence_after();
    dev::allow_dependents();
    const uint32_t tmem = tmem_at;
    Tiles<kKind, S::kTileRows, S::kCols> tiles(args, prefix);
    const auto blocks_of = [&](const Tile &t) { return static_cast<int>((t.depth + kDepth - 1) / kDepth) * (kKind == kInput ? 2 : 1); };

    if (warp == kWriters) {
        if (one_lane()) {
            int s = 0, round = 0;
            uint32_t full_fills = 0, rest_fills = 0, rest_last = 0;  // a bit a stage: parity of its fills of either kind, kind of the last
            bool ok = true;
            // block q of the tile to place `at` of the ring: B's part, A's part
            const auto copy_b = [&](const Tile &t, int at, int q, int once, uint32_t bar) {
                const uint32_t b = ring_b + at * S::kBBytes;
                const int pass = q >= once, k = (pass ? q - once : q) * kDepth;
                // this CTA's part: half of the columns (kGated: gate or up)
                const int col = static_cast<int>(t.col) + (kKind == kGated ? 0 : rank * (kN / S::kCtas));
                if constexpr (kAcrossA) {
#pragma unroll
                    for (int j = 0; j < kN / S::kCtas / 64; ++j)
                        copy2<kPair>(b + j * (kDepth * kRowBytes), &args.b[t.which], col + j * 64, static_cast<int>(t.first) + k, bar);
                } else if constexpr (kKind == kGated && kPair) {
                    copy3<kPair>(b, &args.b[rank], k, col, t.e, bar);
                } else if constexpr (kKind == kGated) {
                    copy3<kPair>(b, &args.b[0], k, col, t.e, bar);
                    copy3<kPair>(b + kN / 2 * kRowBytes, &args.b[1], k, col, t.e, bar);
                } else if constexpr (kAcrossB) {
#pragma unroll
                    for (int j = 0; j < kN / S::kCtas / 64; ++j)
                        copy3<kPair>(b + j * (kDepth * kRowBytes), &args.b[pass], col + j * 64, k, t.e, bar);
                } else {
                    copy3<kPair>(b, &args.b[0], k, col, t.e, bar);
                }
            };
            const auto copy_a = [&](const Tile &t, int at, int q, int once, uint32_t bar) {
                const uint32_t a = ring_a + at * S::kABytes;
                const int pass = q >= once, k = (pass ? q - once : q) * kDepth, row = static_cast<int>(t.row) + rank * S::kMine;
                if constexpr (kAcrossA) {
#pragma unroll
                    for (int j = 0; j < S::kMine / 64; ++j)
                        copy2<kPair>(a + j * (kDepth * kRowBytes), &args.a[t.which], row + j * 64, static_cast<int>(t.first) + k, bar);
                } else {
                    if constexpr (S::kTwoParts) copy3<kPair>(a, &args.a[0], k, row, 0, bar);
                    else copy2<kPair>(a, &args.a[pass], k, row, bar);
                }
            };
            // Behind a kernel that may still run: its results are A (kWeights: B too).  B's stages of the first tile
            // come before them.
            int ahead = 0;
            if (args.follows) {
                if (kKind != kWeights && first < tiles.total) {
                    const Tile t = tiles[first];
                    const int n = blocks_of(t);
                    for (; ahead < stages && ahead * S::kBlocks < n; ++ahead) {
                        const int q0 = ahead * S::kBlocks, blocks = min(S::kBlocks, n - q0);
                        const uint32_t bar = rank == 0 ? full(ahead) : bar_first(full(ahead));
                        if (rank == 0) bar_expect(full(ahead), S::kCtas * blocks * S::kBlockBytes);
                        for (int j = 0; j < blocks; ++j) copy_b(t, q0 + j, q0 + j, kKind == kInput ? n / 2 : n, bar);
                    }
                }
                dev::grid_wait();
            }
            for (uint32_t i = first; ok && i < tiles.total; i += step) {
                const Tile t = tiles[i];
                const int n = blocks_of(t), once = kKind == kInput ? n / 2 : n;
                for (int q0 = 0; q0 < n; q0 += S::kBlocks) {
                    if (!(ok = bar_wait(empty(s), (round & 1) ^ 1, gave_up))) break;
                    const int blocks = min(S::kBlocks, n - q0);
                    // a pair's copies are counted by its first CTA, but for a segment's last rows, by each CTA
                    const bool rest = kKind == kWeights && t.depth - static_cast<int64_t>(q0) * kDepth < kDepth;
                    const bool own = !kPair || rest;
                    const uint32_t here = rest ? rest_full(s) : full(s), bar = own || rank == 0 ? here : bar_first(here);
                    (rest ? rest_fills : full_fills) ^= 1u << s;
                    rest_last = rest ? rest_last | 1u << s : rest_last & ~(1u << s);
                    if (ahead > 0) {
                        --ahead;
                    } else {
                        if (own || rank == 0) bar_expect(here, (own ? 1 : 2) * blocks * S::kBlockBytes);
                        for (int j = 0; j < blocks; ++j) copy_b(t, s * S::kBlocks + j, q0 + j, once, bar);
                    }
                    for (int j = 0; j < blocks; ++j) copy_a(t, s * S::kBlocks + j, q0 + j, once, bar);
                    if (++s == stages) {
                        s = 0;
                        ++round;
                    }
                }
            }
            // the ring is empty again (given up: at least every copy has landed)
            long long t0 = ok ? 0 : clock64();
            for (int j = 0; j < stages; ++j) {
                const int last = j < s ? round : round - 1;  // the round in which the stage was filled last
                if (last < 0) continue;
                if (ok && !(ok = bar_wait(empty(j), last & 1, gave_up))) t0 = clock64();
                const bool rest = rest_last >> j & 1;
                if (!ok && (rest || rank == 0)) {
                    while (!bar_try(rest ? rest_full(j) : full(j), (~(rest ? rest_fills : full_fills)) >> j & 1) && clock64() - t0 < kWaitCycles) {}
                }
            }
        }
        __syncwarp();
    } else if (warp == kWriters + 1) {
        constexpr uint32_t shape = product_shape<T, kKind, kN, kPair>();
        int s = 0, done = 0;
        uint32_t full_parity = 0, cleared_parity = 0;  // a bit a stage
        bool ok = true;
        // by one lane: stage s of a tile, its blocks from q0 on, the last block `steps` 16s of k
        const auto products = [&](int q0, int n, int steps) {
            fence_after();
            const uint32_t d = tmem + (done & 1) * (kN * S::kAccs);
            const int blocks = min(S::kBlocks, n - q0);
#pragma unroll
            for (int j = 0; j < S::kBlocks; ++j) {
                if (j >= blocks) break;
                const int at = s * S::kBlocks + j;
                uint64_t da = operand<kAcrossA>(ring_a + at * S::kABytes), db = operand<kAcrossB>(ring_b + at * S::kBBytes);
#pragma unroll
                for (int k = 0; k < kDepth / 16; ++k) {
                    if (k < steps) multiply<kPair>(d + k % S::kAccs * kN, da, db, shape, q0 + j > 0 || k >= S::kAccs);
                    da += kStep<kAcrossA>;
                    db += kStep<kAcrossB>;
                }
            }
            signal_done<kPair>(empty(s));
            if (q0 + blocks == n) signal_done<kPair>(acc_full(done & 1));
        };
        if (rank == 0 && one_lane())
            for (uint32_t i = first; ok && i < tiles.total; i += step) {
                const Tile t = tiles[i];
                const int n = blocks_of(t), left = kKind == kWeights ? static_cast<int>(t.depth % kDepth) : 0;
                if (n == 0) continue;
                if (!(ok = bar_wait(acc_empty(done & 1), ((done >> 1) & 1) ^ 1, gave_up))) break;
                for (int q = 0; q < n; q += S::kBlocks) {
                    int steps = kDepth / 16;
                    if (left && q == n - 1) {
                        if (!(ok = bar_wait(cleared(s), cleared_parity >> s & 1, gave_up))) break;
                        if (kPair) asm volatile("fence.acq_rel.cluster;" ::: "memory");
                        cleared_parity ^= 1u << s;
                        steps = (left + 15) / 16;
                    } else {
                        if (!(ok = bar_wait(full(s), full_parity >> s & 1, gave_up))) break;
                        full_parity ^= 1u << s;
                    }
                    products(q, n, steps);
                    if (++s == stages) s = 0;
                }
                ++done;
            }
        __syncwarp();
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && rank == 0 && one_lane()) {  // given up: the products in flight end before their memory is given back
            signal_done<kPair>(drained);
            const long long t0 = clock64();
            while (!bar_try(drained, 0) && clock64() - t0 < kWaitCycles) {}
        }
        __syncwarp();
    } else if (kKind == kWeights && warp == kWriters + 2) {
        // rows of other segments in a tile's last stage, up to a whole 16 of k, as soon as they are there
        int s = 0;
        uint32_t parity = 0;  // a bit a stage
        for (uint32_t i = first; i < tiles.total; i += step) {
            const Tile t = tiles[i];
            const int left = static_cast<int>(t.depth % kDepth);
            if (left == 0) {
                s = (s + blocks_of(t)) % stages;
                continue;
            }
            s = (s + blocks_of(t) - 1) % stages;
            if (!warp_wait<false>(rest_full(s), parity >> s & 1, gave_up)) break;
            parity ^= 1u << s;
            clear_rows<kN / S::kCtas>(ring_a + s * S::kABytes, ring_b + s * S::kBBytes, left);
            if (lane == 0) {
                if (kPair && rank == 1) bar_arrive_first<true>(cleared(s));
                else bar_arrive(cleared(s));
            }
            __syncwarp();
            s = (s + 1) % stages;
        }
    } else {
        int done = 0;
        const Block &b = args.block;
        const uint32_t mine = patches + warp * S::kWriterBytes;
        constexpr int kHalves = S::kCols > 32 ? 2 : 1;  // the two warps of a quarter of the lanes take columns in turn
        const int quarter = warp & 3, half = warp >> 2;
        for (uint32_t i = first; i < tiles.total; i += step) {
            const Tile t = tiles[i];
            const bool zero = blocks_of(t) == 0;
            const int which = done & 1;
            const int64_t row = t.row + rank * S::kMine + quarter * 32;
            const int64_t columns = product_columns<kKind>(b, t.which) - t.col;  // from the tile's first on
            const int rows = half >= kHalves || quarter * 32 >= S::kMine
                                 ? 0
                                 : static_cast<int>(max(min(t.end - row, static_cast<int64_t>(min(32, S::kMine))), int64_t(0)));
            const int width = static_cast<int>(min(columns, static_cast<int64_t>(S::kCols)));
            const auto at = [&](const Matrix &m, int c) { return static_cast<T *>(m.p) + row * m.ld + t.col + c; };
            const auto ask_gate = [&](int c) { patch_in<T>(mine, at(b.gate, c), b.gate.ld, rows, columns - c); };  // kBack
            const auto ask_up = [&](int c) { patch_in<T>(mine + kPatchBytes, at(b.up, c), b.up.ld, rows, columns - c); };
            if constexpr (kKind == kBack)
                if (rows > 0 && half * 32 < width) {
                    ask_gate(half * 32);
                    ask_up(half * 32);
                }
            if (!zero) {
                if (!warp_wait<true>(acc_full(which), (done >> 1) & 1, gave_up)) break;
                fence_after();
                ++done;
            }
            const uint32_t from = tmem + which * (kN * S::kAccs) + (static_cast<uint32_t>(quarter * 32) << 16);
            // accumulators that have been written (kWeights: a segment of few rows leaves the others)
            const int accs = kKind == kWeights && t.depth < 16 * S::kAccs ? static_cast<int>((t.depth + 15) / 16) : S::kAccs;
            const auto take = [&](int c, float *v) {
                read32(from + c, v);
                read_done();
                if constexpr (S::kAccs > 1) {
#pragma unroll 1
                    for (int a = 1; a < accs; ++a) {
                        float w[32];
                        read32(from + a * kN + c, w);
                        read_done();
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] += w[j];
                    }
                }
            };
            const int until = rows > 0 ? width : 0;
#pragma unroll 1
            for (int c = half * 32; c < until; c += 32 * kHalves) {
                float v[32];
                if (zero) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                } else {
                    take(c, v);
                    if constexpr (S::kTwoParts) {  // the sums of h's second parts, kLoaded lanes on
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float rest = __shfl_down_sync(0xffffffffu, v[j], kLoaded);
                            // (a weight that is no number times a second part, which may be 0, is not what it is times h)
                            if (fabsf(v[j]) < INFINITY) v[j] += rest;
                        }
                    }
                }
                const int64_t left = columns - c;
                if constexpr (kKind == kGated) {
                    float w[32];
                    if (zero) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) w[j] = 0.0f;
                    } else {
                        take(kN / 2 + c, w);
                    }
                    if (b.gate.p) {
                        patch_row<T>(mine, v);
                        patch_out<T>(mine, at(b.gate, c), b.gate.ld, rows, left);
                        patch_row<T>(mine, w);
                        patch_out<T>(mine, at(b.up, c), b.up.ld, rows, left);
                    }
                    if (!zero) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = activate<T, false>(v[j], b.act).value * w[j];
                        // rounded to the type: the next product takes it so (one rounding of each term of y's sums); of short
                        // segments, whose products wait for the weights, it takes what the rounding left out, too
                        patch_row<T>(mine, v);
                        patch_out<T>(mine, at(b.h, c), b.h.ld, rows, left);
                        if constexpr (kLoaded <= kFewRows) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const float rest = v[j] - to_f32(from_f32<T>(v[j]));
                                v[j] = fabsf(rest) < INFINITY ? rest : 0.0f;  // (nothing of an infinity, or of a value beyond the type's)
                            }
                            patch_row<T>(mine, v);
                            patch_out<T>(mine, at(b.h2, c), b.h2.ld, rows, left);
                        }
                    }
                } else if constexpr (kKind == kBack) {
                    const uint32_t gate = mine, up = mine + kPatchBytes;
                    uint4 h_row[4];
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    __syncwarp();
                    // each result rounded once, to the type that the next products take
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        float g[8], u[8], h[8];
                        unpack<T>(patch_load(patch_piece(gate, lane, p)), g);
                        unpack<T>(patch_load(patch_piece(up, lane, p)), u);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const Activated a = activate<T, true>(g[j], b.act);
                            g[j] = v[8 * p + j] * u[j] * a.slope;
                            h[j] = a.value * u[j];
                            u[j] = v[8 * p + j] * a.value;
                        }
                        patch_store(patch_piece(gate, lane, p), pack<T>(g));
                        patch_store(patch_piece(up, lane, p), pack<T>(u));
                        h_row[p] = pack<T>(h);
                    }
                    const bool more = c + 32 * kHalves < width;
                    patch_out<T>(up, at(b.dup, c), b.dup.ld, rows, left);
                    if (more) ask_up(c + 32 * kHalves);
                    patch_out<T>(gate, at(b.dgate, c), b.dgate.ld, rows, left);
#pragma unroll
                    for (int p = 0; p < 4; ++p) patch_store(patch_piece(gate, lane, p), h_row[p]);
                    patch_out<T>(gate, at(b.h, c), b.h.ld, rows, left);
                    if (more) ask_gate(c + 32 * kHalves);
                } else {
                    const Matrix &m = kKind == kDown ? b.y : kKind == kInput ? b.dx : t.which == 0 ? b.dwg : t.which == 1 ? b.dwu : b.dwd;
                    if constexpr (kKind == kWeights) {
                        if (b.splits > 1) {
                            const int64_t n = product_columns<kKind>(b, t.which);
                            if (lane < rows) put<float, 32>(b.part_sums(t.which, t.e, t.part) + (row + lane) * n + t.col + c, v, left, n % 4 == 0);
                            continue;
                        }
                    }
                    patch_row<T>(mine, v);
                    patch_out<T>(mine, at(m, c) + (kKind == kWeights ? t.e * m.expert : 0), m.ld, rows, left);
                }
            }
            if (!zero) {
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair && rank == 1) bar_arrive_first<false>(acc_empty(which));
                    else bar_arrive(acc_empty(which));
                }
            }
        }
    }
    __syncthreads();
    if constexpr (kPair) cluster_sync(2);  // the other CTA's copies, products and barriers are done with
    if (warp == kWriters + 1) {
        fence_after();
        if constexpr (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kColumns) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kColumns) : "memory");
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

// reads and clears the flag
inline cudaError_t take_flag(int *value) {
    cudaError_t e = cudaMemcpyFromSymbol(value, gave_up_flag, sizeof(int));
    const int none = 0;
    if (e == cudaSuccess && *value) e = cudaMemcpyToSymbol(gave_up_flag, &none, sizeof(int));
    return e;
}

// `count` matrices (0: one, as a map of two dimensions) of `rows` rows of `n` values; boxes of 64 values x box_rows (of
// box_count matrices)
template <typename T>
bool make_map(CUtensorMap *map, const Matrix &m, int64_t n, int64_t rows, int64_t count, int box_rows, int box_count = 1) {
    const cuuint64_t sizes[3] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(count ? count : 1)};
    // (one matrix: its distance to the next is not used, but has to be a valid one)
    const int64_t apart = count > 1 ? m.expert : ceil_div((rows - 1) * m.ld + n, 8) * 8;
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(m.ld) * sizeof(T), static_cast<cuuint64_t>(apart) * sizeof(T)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_count)}, step[3] = {1, 1, 1};
    return encoder()(map, std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     count ? 3 : 2, m.p, sizes, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int kKind, int kN, int kLoaded, bool kPair>
int launch(const Block &b, bool follows, cudaStream_t s) {
    using S = Shape<kKind, kN, kLoaded, kPair>;
    Args args;
    args.block = b;
    args.products = 0;
    args.follows = follows;
    const int64_t rows = b.seg.rows, d = b.d, f = b.f, count = b.seg.count;
    args.stages = S::stages(static_cast<int>(count));
    const size_t smem = S::smem(static_cast<int>(count), args.stages);
    // (in front of the maps: they are made for the context that is current to this host thread, and this makes the
    // device's that where no call has yet; always the same limit: another thread's call may set it between this and the launch)
    SPMV_TRY_CUDA(cudaFuncSetAttribute(k_ffn<T, kKind, kN, kLoaded, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes));
    const auto activation = [&](CUtensorMap *map, const Matrix &m, int64_t n) {
        return make_map<T>(map, m, n, rows, 0, kKind == kWeights ? kDepth : S::kMine);
    };
    const auto weight = [&](CUtensorMap *map, const Matrix &m, int64_t n, int64_t m_rows, int box) { return make_map<T>(map, m, n, m_rows, count, box); };
    bool ok = true;
    int64_t tiles = 0;
    if (kKind == kWeights) {
        const Matrix *out[3] = {&b.dwg, &b.dwu, &b.dwd}, *in[3] = {&b.dgate, &b.dup, &b.dy};
        for (int i = 0; i < 3; ++i) {
            if (!out[i]->p) continue;
            args.which[args.products++] = i;
            ok = ok && activation(&args.a[i], *in[i], weight_rows(b, i)) && activation(&args.b[i], i == 2 ? b.h : b.x, i == 2 ? f : d);
            tiles += ceil_div(weight_rows(b, i), S::kTileRows) * ceil_div(product_columns<kKind>(b, i), kN) * count * b.splits;
        }
    } else if (kKind == kGated) {
        ok = ok && activation(&args.a[0], b.x, d) && weight(&args.b[0], b.wg, d, f, kN / 2) && weight(&args.b[1], b.wu, d, f, kN / 2);
    } else if (kKind == kDown) {
        // (both parts of h as two matrices)
        ok = ok && (S::kTwoParts ? make_map<T>(&args.a[0], b.h, f, rows, 2, S::kMine, 2) : activation(&args.a[0], b.h, f)) && weight(&args.b[0], b.wd, f, d, kN / S::kCtas);
    } else if (kKind == kBack) {
        ok = ok && activation(&args.a[0], b.dy, d) && weight(&args.b[0], b.wd, f, d, kDepth);
    } else {
        ok = ok && activation(&args.a[0], b.dgate, f) && activation(&args.a[1], b.dup, f) && weight(&args.b[0], b.wg, d, f, kDepth) &&
             weight(&args.b[1], b.wu, d, f, kDepth);
    }
    if (!ok) return set_error(SPMV_ERR_CUDA, "the feed-forward block's matrices could not be described to the copy engine");
    if (kKind != kWeights)
        tiles = ceil_div(product_columns<kKind>(b, 0), S::kCols) * (rows / S::kTileRows + (count < rows ? count : rows) + 1);
    if (tiles >= int64_t(1) << 31) return set_error(SPMV_ERR_TOO_LARGE, "the feed-forward block has too many tiles");
    const int64_t workers = kSms / S::kCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((tiles < workers ? tiles : workers) * S::kCtas));
    cfg.blockDim = dim3(threads_of(kKind));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    if (kPair) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = 2;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (follows) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    cfg.attrs = attr;
    SPMV_TRY_CUDA(cudaLaunchKernelEx(&cfg, k_ffn<T, kKind, kN, kLoaded, kPair>, args));
    return SPMV_OK;
}

// Which tiles (d = f = 2048 unless said; us, forward and then back without weights, of all the call's products):
//   short segments    8 or 16 rows x 64 columns (16 dense rows 17.7 22.1; tiles of 128 x 64 24.9 34.5, of 128 x 256 28.2 43.9)
//   pairs of CTAs     segments of 112 rows on average, enough tiles for 48 pairs (16 experts of 64 rows 84.0 93.3, of 128 87.6 98.7;
//                     2048 dense rows 40.6 50.0)
//   128 x 256         enough tiles for 96 SMs (the same three: 74.3 78.7; 93.3 115.6; 43.0 53.5)
//   128 x 64          the rest (512 dense rows 25.6 27.6; 128 x 256 30.0 49.1, pairs 27.8 43.6)
template <typename T, int kKind>
int launch_shape(const Block &b, bool follows, cudaStream_t s) {
    const int64_t rows = b.seg.rows, count = b.seg.count, used = count < rows ? count : rows;
    const auto row_tiles = [&](int64_t n) { return ceil_div(rows, n) > used ? ceil_div(rows, n) : used; };
    const int64_t columns = product_columns<kKind>(b, 0);
    if constexpr (kKind == kWeights) {
        const int64_t tiles = (2 * ceil_div(b.f, 256) * ceil_div(b.d, 256) + ceil_div(b.d, 256) * ceil_div(b.f, 256)) * count * b.splits;
        if (tiles >= 48) return launch<T, kKind, 256, 128, true>(b, follows, s);
        return launch<T, kKind, 64, 128, false>(b, follows, s);
    } else {
        const int few = short_rows(rows, count);
        if constexpr (kKind == kDown) {
            // tiles of 32 columns where those of 64 would leave SMs without one
            const bool narrow = used * ceil_div(columns, 64) < kSms;
            if (few == 8) return narrow ? launch<T, kKind, 32, 8, false>(b, follows, s) : launch<T, kKind, 64, 8, false>(b, follows, s);
            if (few) return narrow ? launch<T, kKind, 32, kFewRows, false>(b, follows, s) : launch<T, kKind, 64, kFewRows, false>(b, follows, s);
        } else {
            if (kKind == kGated && few == 8) return launch<T, kKind, 64, 8, false>(b, follows, s);
            if (few) return launch<T, kKind, 64, kFewRows, false>(b, follows, s);
        }
        const int64_t wide = ceil_div(columns, kKind == kGated ? 128 : 256);
        if (rows >= 112 * count && row_tiles(256) * wide >= 48) return launch<T, kKind, 256, 128, true>(b, follows, s);
        if (row_tiles(128) * wide >= 96) return launch<T, kKind, 256, 128, false>(b, follows, s);
        return launch<T, kKind, 64, 128, false>(b, follows, s);
    }
}
template <typename T>
int launch_kind(int kind, const Block &b, bool follows, cudaStream_t s) {
    switch (kind) {
        case kGated: return launch_shape<T, kGated>(b, follows, s);
        case kDown: return launch_shape<T, kDown>(b, follows, s);
        case kBack: return launch_shape<T, kBack>(b, follows, s);
        case kInput: return launch_shape<T, kInput>(b, follows, s);
        default: return launch_shape<T, kWeights>(b, follows, s);
    }
}

}  // namespace tc
}  // namespace ffn
}  // namespace spmv
