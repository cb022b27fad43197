// C = A B^T on the tensor cores, with a fused epilogue.
//
// A block (or a pair of blocks on two SMs) owns one tile of C at a time and
// walks the tiles of the launch.  Its roles run at once: two threads fetch 64
// depths of A and of B at a time with TMA into a ring of shared-memory stages,
// one thread multiplies them with tcgen05.mma into TMEM, and eight warps turn a
// finished accumulator (one TMEM lane per row) into the result while the next
// tile is multiplied into the other half of TMEM.
//
// Operands may be contiguous along the depth or along the rows: the tensor
// core reads both from the 128-byte swizzled layout that TMA writes, so the
// transposed products of the gradients need no copy.
//
// A pair of blocks (tcgen05 cta_group::2) multiplies 256 rows by up to 256
// columns: each block holds its own 128 rows of A and half of the columns of
// B, so a stage takes 32 KB instead of 48 KB and six of them fit.
//
// What bounds it (GB300, bf16): large products run at the tensor cores' rate,
// 8192 x 8192 x 8192 in 571 us, 1927 TFLOP/s in short runs, and at the power
// limit in long ones (1638 to 1676 TFLOP/s over 1.5 s); one token to a few
// dozen stream the weights, 16 x 4096 x 14336 in 23 us, 5.1 TB/s.
#include <cuda.h>

#include <algorithm>
#include <array>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "../../include/uzip_debug.h"
#include "product.cuh"

namespace uzip {
namespace {

constexpr uint32_t kRowsTile = 128;  // accumulator rows of a block: the TMEM lanes
constexpr uint32_t kDepthTile = 64;  // depths of a stage: 128 bytes, the swizzle's span
constexpr uint32_t kSliceBytes = kDepthTile * 128;  // 64 rows x 64 depths when rows are contiguous
constexpr uint32_t kAStage = kRowsTile * kDepthTile * 2;
constexpr uint32_t kMaxStages = 24;
constexpr uint32_t kThreads = 352;  // TMA warp for A, MMA warp, 4 epilogue warps, TMA warp for B, 4 epilogue warps
// The tensor core cuts each addition to 24 bits toward zero, which adds up to a
// bias of half a unit an addition: at 4096 depths logits were 1e-5 off and the
// loss 1.4e-6 of itself.  The loss statistics, and the logits of the loss's
// gradient, take the products of 1024 depths at a time into registers, where
// they are added with rounding: both have the same logits, and p - 1 of a token
// whose target has nearly all of the probability is a difference of two near
// numbers (p = 0.9995 at 4096 depths: that token's gradient was off by 45 % of
// itself when its logits were summed in one go).
constexpr uint32_t kLogitChunk = 16;  // stages
// Other products take this many stages in one go: over 32768 depths the same sign
// all the way was 2e-4 short (2^-12, fp16's rounding), over 2^20 6e-3.  Longer
// depths take chunks of 16384 in the same way: 1e-4 and 1.3e-4.  (Chunks of
// 8192 would leave half of that and cost 2048 x 14336 x 4096 143 us instead of
// 139.)
constexpr uint32_t kLongChunk = 256;
constexpr uint32_t kEpilogueWarps = 8;
constexpr uint32_t kPatchCols = 32;  // columns that an epilogue warp takes at a time
constexpr uint32_t kPatchBytes = 32 * kPatchCols * 2, kEpilogueBytes = kPatchBytes + 128 * 4;  // a warp's shared memory
constexpr uint32_t kMaxSplits = 8;  // blocks of a portable cluster
constexpr uint32_t kHeights = 6;    // boxes of 1 to 32 lines for depths that are cut
constexpr uint32_t kWaitLimit = 7630;  // times 2^20 clock cycles: a wait gives up after about four seconds,
constexpr int64_t kDrainLimit = 100000000;  // one for products in flight then after 50 ms

struct Tiling {
    uint32_t bn;       // columns of a tile
    uint32_t stages;
    uint32_t a_stage;  // bytes of A in a stage: fewer rows than 128 leave more stages
    uint32_t stage_bytes;
    uint32_t splits;   // blocks of a cluster that share a tile's depth
    uint32_t pair;     // 2: two blocks share a tile of 256 rows, else 1
    uint32_t a_box, b_box;  // rows of one TMA box (depth-major)
    uint32_t a_slab, b_slab;  // all slices of a stage in one box (rows contiguous)
    uint32_t raster;   // row tiles taken together for the sake of L2
    uint32_t tmem_cols;
    uint32_t idesc;
    uint32_t smem;
    uint32_t out_width, z_width;  // values that rows of 16-bit results are aligned to: 8, 4, 2 or 1
    uint32_t vec;      // bit flags: 16-byte access to out 1, bias 2, residual 4, z 8, sums 16
    uint32_t starve;   // tests: A is never fetched, so that every wait for it runs out
    uint32_t wait_limit;  // 2^20 clock cycles
};

// ---- PTX ------------------------------------------------------------------------

__device__ __forceinline__ uint64_t matrix_descriptor(uint32_t addr, bool depth_major) {
    // start, distance between 64-row slices (rows contiguous), distance between
    // groups of 8 swizzled 128-byte lines, version 1, 128-byte swizzle
    const uint64_t lead = depth_major ? 1 : kSliceBytes / 16;
    return uint64_t((addr & 0x3FFFF) >> 4) | lead << 16 | uint64_t(1024 / 16) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}
template <bool PAIR>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    if (PAIR)  // the barrier may be the other block's
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
            "%3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
            : "memory");
    else
        asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
}
// one arrival once the products issued so far are done (a pair: on both blocks' barriers)
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t leader = 0) {
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(uint16_t(3u << leader))
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t to, uint32_t cols) {
    if (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    if (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 columns of this warp's 32 lanes; each lane gets its row
__device__ __forceinline__ void tmem_load32(uint32_t addr, float v[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (uint32_t i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// True in one lane of a converged warp.  The compiler knows that one lane is
// left, so the TMA and MMA instructions behind it take their operands straight
// from uniform registers; behind `lane == 0` each of them cost 100 cycles more.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_address(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Barriers between the pair's blocks order only TMEM (by the tcgen05 fences)
// and copies, no ordinary memory: without a cluster scope an arrival does not
// wait for the warp's stores to global memory.
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// the operands in boxes of a whole stage, and of 1, 2, 4, ... 32 lines for cut depths
template <bool CUT>
struct Maps {
    CUtensorMap a, b;
};
template <>
struct Maps<true> : Maps<false> {
    CUtensorMap a_lines[kHeights], b_lines[kHeights];
};

// ---- the block's shared state ------------------------------------------------------

struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem;
    volatile uint32_t abort, wait_limit;
};
// behind it, for the grouped schedules: int32 offsets[groups + 1], then (kRows,
// kColumns) the first row or column tile of each group, int32 [groups + 1]

// A wait that is not over at its first try goes on outside the loops of the
// fetching and multiplying threads, whose code the epilogue's warps push out of
// the instruction cache: each line less is felt there.  (With the limit as a plain
// 64-bit value beside `abort` the 48 x 128256 x 4096 loss took 168 us, not 166.)
__device__ __noinline__ bool wait_on(volatile uint32_t* abort, const volatile uint32_t* limit, uint32_t bar, uint32_t parity) {
    const int64_t start = clock64();
    do {
        for (uint32_t i = 0; i < 64; ++i)
            if (try_wait(bar, parity)) return true;
        if (*abort) return false;
    } while (clock64() - start < int64_t(*limit) << 20);
    *abort = 1;
    return false;
}
__device__ __forceinline__ bool wait(Control* c, uint32_t bar, uint32_t parity) {
    return try_wait(bar, parity) || wait_on(&c->abort, &c->wait_limit, bar, parity);
}
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
    const int64_t start = clock64();
    while (!try_wait(smem_u32(bar), parity) && clock64() - start < kDrainLimit) {
    }
}
// A block that has given up lets the copies in flight land before it ends: the
// two fetching threads of its own, and of its pair, may each have got to another
// stage, whose barriers then never complete, so it waits for longer than any copy
// takes (microseconds) instead.
__device__ __noinline__ void settle() {
    const int64_t start = clock64();
    while (clock64() - start < kDrainLimit) __nanosleep(1000);
}

// The next stage of the ring and the parity of its use.
struct Ring {
    uint32_t stages, s = 0, phase = 0, used = 0;
    __device__ __forceinline__ void advance() {
        ++used;
        if (++s == stages) s = 0, phase ^= 1;
    }
};

// A tile of C: its group, first row, the end of its rows, its columns and its depths.
struct Tile {
    uint32_t group, row0, row_end, col0, cols, width;  // width: cols up to what the MMA takes
    uint32_t d0, blocks, depth_end;
};

// The launch's tiles in the order in which this block takes them.  All of its
// numbers are copies: the roles' loops touch no parameter memory.
struct Walk {
    const int32_t *offsets, *first;  // shared memory
    uint32_t schedule, rows, depth, bn, splits, raster;
    uint32_t tile_rows, row_tiles, col_tiles, total, step, next, group, split, columns, unit;

    // rows and depth: how many there are
    __device__ __forceinline__ Walk(const Product& p, const Tiling& t, const int32_t* offsets, const int32_t* first, uint32_t rows,
                                    uint32_t depth)
        : offsets(offsets), first(first), schedule(p.schedule), rows(rows), depth(depth), bn(t.bn), splits(t.splits),
          raster(t.raster) {
        tile_rows = kRowsTile * t.pair;
        col_tiles = (uint32_t(p.n) + bn - 1) / bn;
        columns = uint32_t(p.n);
        unit = 16 * t.pair;
        row_tiles = schedule == kRows ? uint32_t(first[p.groups]) : (rows + tile_rows - 1) / tile_rows;
        if (schedule == kColumns) col_tiles = uint32_t(first[p.groups]);
        total = row_tiles * col_tiles * (schedule == kDepth ? p.groups : 1);
        const uint32_t cluster = splits * t.pair;
        step = gridDim.x / cluster;
        next = blockIdx.x / cluster;
        split = blockIdx.x % cluster / t.pair;
        group = 0;
    }
    __device__ __forceinline__ bool take(Tile& o) {
        if (next >= total) return false;
        uint32_t id = next;
        next += step;
        o.group = 0;
        o.d0 = 0;
        o.depth_end = depth;
        if (schedule == kColumns) {
            // a group's columns in tiles of equal width, all of them before the next rows of A
            while (uint32_t(first[group + 1]) * row_tiles <= id) ++group;
            const uint32_t some = first[group + 1] - first[group], count = offsets[group + 1] - offsets[group];
            id -= first[group] * row_tiles;
            o.group = group;
            o.row0 = id / some * tile_rows;
            o.row_end = rows;
            o.width = ((count + some - 1) / some + unit - 1) / unit * unit;
            const uint32_t c = id % some * o.width;
            o.col0 = offsets[group] + c;
            o.cols = min(o.width, count - c);
            o.blocks = (depth + kDepthTile - 1) / kDepthTile;
            return true;
        }
        uint32_t col_tile;
        if (schedule == kRows) {
            while (uint32_t(first[group + 1]) * col_tiles <= id) ++group;
            const uint32_t some = first[group + 1] - first[group];
            id -= first[group] * col_tiles;
            o.group = group;
            col_tile = id / some;
            o.row0 = offsets[group] + id % some * tile_rows;
            o.row_end = offsets[group + 1];
        } else {
            if (schedule == kDepth) {
                const uint32_t per = row_tiles * col_tiles;
                o.group = id / per;
                id -= o.group * per;
                o.d0 = offsets[o.group];
                o.depth_end = offsets[o.group + 1];
            }
            const uint32_t band = id / (raster * col_tiles), in = id - band * raster * col_tiles;
            const uint32_t some = min(raster, row_tiles - band * raster);
            o.row0 = (band * raster + in % some) * tile_rows;
            col_tile = in / some;
            o.row_end = rows;
        }
        o.col0 = col_tile * bn;
        o.cols = min(bn, columns - o.col0);
        o.width = bn;
        o.blocks = (o.depth_end - o.d0 + kDepthTile - 1) / kDepthTile;
        if (splits > 1) {
            const uint32_t lo = o.blocks * split / splits, hi = o.blocks * (split + 1) / splits;
            o.d0 += lo * kDepthTile;
            o.blocks = hi - lo;
        }
        return true;
    }
};

// ---- epilogues ------------------------------------------------------------------------

// Up to 8 values of a row from 16-bit memory; vec: one 16-byte load.
__device__ __forceinline__ void read8(const void* base, uint64_t at, bool vec, uint32_t cols, int dtype, float v[8]) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    uint32_t w[4] = {};
    if (vec && cols == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
            if (j < cols) w[j / 2] |= uint32_t(p[j]) << (j % 2 * 16);
    }
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
        const float2 f = from16x2(w[j], dtype);
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
    }
}
__device__ __forceinline__ void write8(void* base, uint64_t at, bool vec, uint32_t cols, int dtype, const float v[8]) {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    uint32_t w[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) w[j] = to16x2(v[2 * j], v[2 * j + 1], dtype);
    if (vec && cols == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
            if (j < cols) p[j] = uint16_t(w[j / 2] >> (j % 2 * 16));
    }
}

__device__ __forceinline__ void add_sums8(const StoreEpilogue& e, uint32_t vec, uint64_t row, uint32_t col, uint32_t cols, float v[8]) {
    const float* s = e.sum_in + row * e.ld_sum + col;
    if ((vec & 16) && cols == 8) {
        const float4 lo = *reinterpret_cast<const float4*>(s), hi = *reinterpret_cast<const float4*>(s + 4);
        v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w, v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
            if (j < cols) v[j] += s[j];
    }
}
__device__ __forceinline__ void write_fp32(const StoreEpilogue& e, uint64_t at, uint32_t vec, uint32_t cols, const float v[8]) {
    float* o = static_cast<float*>(e.out) + at;
    if ((vec & 1) && cols == 8) {
        reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
            if (j < cols) o[j] = v[j];
    }
}

// kStore for `cols` (1 to 8) neighbouring values of a row.
__device__ __forceinline__ void store8(const Product& p, uint32_t vec, uint32_t g, uint64_t row, uint32_t col,
                                       uint32_t cols, float alpha, float v[8]) {
    const StoreEpilogue& e = p.st;
    float q[8];
    {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) v[j] *= alpha;
    }
    if (e.sum_in) add_sums8(e, vec, row, col, cols, v);
    if (e.bias) {
        read8(e.bias, g * p.n + col, vec & 2, cols, p.dtype, q);
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) v[j] += q[j];
    }
    if (e.z) write8(e.z, row * e.ldz + col, vec & 8, cols, p.dtype, v);
    if (e.act != UZIP_ACT_NONE) {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) v[j] = act_value(v[j], e.act);
    }
    if (e.residual) {
        read8(e.residual, row * e.ldr + col, vec & 4, cols, p.dtype, q);
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) v[j] += q[j];
    }
    const uint64_t at = g * e.out_group + row * e.ldo + col;
    if (!e.out_fp32) {
        write8(e.out, at, vec & 1, cols, p.dtype, v);
        return;
    }
    write_fp32(e, at, vec, cols, v);
}

// An epilogue warp holds a row in each lane, which would read and write memory
// 16 bytes a row apart.  32 rows x 32 columns of 16-bit values go through 2 KB
// of shared memory instead (16-byte pieces swizzled by the row, free of bank
// conflicts both ways), so that 4 lanes touch 64 contiguous bytes of a row.
// Rows that do not start on 16-byte boundaries go in smaller pieces.
struct Patch {
    uint4* s;  // [32][4]
    uint32_t lane;
    __device__ __forceinline__ uint4& at(uint32_t row, uint32_t piece) const { return s[row * 4 + (piece ^ (row >> 1 & 3))]; }
    __device__ __forceinline__ uint16_t& value(uint32_t row, uint32_t col) const {
        return reinterpret_cast<uint16_t*>(&at(row, col / 8))[col % 8];
    }
    // A value kept for relu's slope keeps its sign: a positive one that the type
    // cannot hold is kept as its smallest.
    template <bool KEPT>
    static __device__ __forceinline__ float kept(float v, float smallest) { return KEPT && v > 0.f ? fmaxf(v, smallest) : v; }
    // this lane's row, rounded
    template <bool KEPT = false>
    __device__ __forceinline__ void put(const float v[32], int dtype) const {
        const auto two = [&](uint32_t i, int type, float smallest) {
            return to16x2(kept<KEPT>(v[i], smallest), kept<KEPT>(v[i + 1], smallest), type);
        };
        __syncwarp();
        if (dtype == UZIP_BF16) {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i)
                at(lane, i) = make_uint4(two(8 * i, UZIP_BF16, 0x1p-133f), two(8 * i + 2, UZIP_BF16, 0x1p-133f),
                                         two(8 * i + 4, UZIP_BF16, 0x1p-133f), two(8 * i + 6, UZIP_BF16, 0x1p-133f));
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i)
                at(lane, i) = make_uint4(two(8 * i, UZIP_FP16, 0x1p-24f), two(8 * i + 2, UZIP_FP16, 0x1p-24f),
                                         two(8 * i + 4, UZIP_FP16, 0x1p-24f), two(8 * i + 6, UZIP_FP16, 0x1p-24f));
        }
        __syncwarp();
    }
    // one value for each of the 32 rows, in this lane's column, rounded
    template <bool KEPT = false>
    __device__ __forceinline__ void put_column(const float v[32], int dtype) const {
        __syncwarp();
        if (dtype == UZIP_BF16) {
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) value(i, lane) = to16(kept<KEPT>(v[i], 0x1p-133f), UZIP_BF16);
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) value(i, lane) = to16(kept<KEPT>(v[i], 0x1p-24f), UZIP_FP16);
        }
        __syncwarp();
    }
    // rows x cols values on their way from p, rows ld apart; vec: 16-byte access
    __device__ __forceinline__ void fetch(const uint16_t* p, uint64_t ld, uint32_t rows, uint32_t cols, bool vec, uint4 q[4]) const {
        if (vec) {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t r = 8 * i + lane / 4;
                q[i] = make_uint4(0, 0, 0, 0);
                if (r < rows && lane % 4 * 8 < cols) q[i] = *reinterpret_cast<const uint4*>(p + r * ld + lane % 4 * 8);
            }
        } else {  // column `lane`, two rows in a word
            uint32_t w[16];
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i) {
                uint32_t lo = 0, hi = 0;
                if (lane < cols && 2 * i < rows) lo = p[2 * i * ld + lane];
                if (lane < cols && 2 * i + 1 < rows) hi = p[(2 * i + 1) * ld + lane];
                w[i] = lo | hi << 16;
            }
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
    __device__ __forceinline__ void place(const uint4 q[4], bool vec) const {
        if (vec) {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) at(8 * i + lane / 4, lane % 4) = q[i];
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    value(8 * i + 2 * j, lane) = uint16_t(w[j]);
                    value(8 * i + 2 * j + 1, lane) = uint16_t(w[j] >> 16);
                }
            }
        }
    }
    // W values a lane: 32 / W lanes to a row, W rows at once
    template <typename T>
    __device__ __forceinline__ void store_by(uint16_t* p, uint64_t ld, uint32_t rows, uint32_t cols) const {
        constexpr uint32_t W = sizeof(T) / 2, kLanes = 32 / W;
        const uint32_t c = lane % kLanes * W, r0 = lane / kLanes;
        if (c >= cols) return;
        p += r0 * ld + c;
#pragma unroll 8
        for (uint32_t r = r0; r < 32; r += W, p += W * ld)
            if (r < rows) *reinterpret_cast<T*>(p) = *reinterpret_cast<const T*>(&value(r, c));
    }
    __device__ __forceinline__ void store(uint16_t* p, uint64_t ld, uint32_t rows, uint32_t cols, uint32_t width) const {
        if (width == 8 && cols % 8 == 0) store_by<uint4>(p, ld, rows, cols);
        else if (width >= 4 && cols % 4 == 0) store_by<uint2>(p, ld, rows, cols);
        else if (width >= 2 && cols % 2 == 0) store_by<uint32_t>(p, ld, rows, cols);
        else store_by<uint16_t>(p, ld, rows, cols);
    }
};

// The product of row `row` of A and column `col` of B (of group g) and a bias
// once more, by one warp, as near as 32 bits hold it.  Two 16-bit values' product
// is exact in 32 bits; what each addition rounds away is summed beside it (the
// error of a sum in six additions, Knuth), and the lanes meet in 64 bits.  Both
// operands lie along the depth, their rows on 16-byte boundaries.
__device__ __noinline__ float dot_again(const Product& p, uint32_t ga, uint32_t gb, uint64_t row, uint64_t col, float bias, uint32_t lane) {
    const uint16_t* a = static_cast<const uint16_t*>(p.a.p) + ga * p.a.group + row * p.a.ld;
    const uint16_t* b = static_cast<const uint16_t*>(p.b.p) + gb * p.b.group + col * p.b.ld;
    float sum = 0.f, lost = 0.f;
    const auto add = [&](float v) {
        const float next = __fadd_rn(sum, v), part = __fsub_rn(next, sum);
        lost = __fadd_rn(lost, __fadd_rn(__fsub_rn(sum, __fsub_rn(next, part)), __fsub_rn(v, part)));
        sum = next;
    };
#pragma unroll 4
    for (uint64_t i = 8 * lane; i + 8 <= p.depth; i += 256) {
        float x[8], y[8];
        read8(a, i, true, 8, p.dtype, x);
        read8(b, i, true, 8, p.dtype, y);
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) add(__fmul_rn(x[j], y[j]));
    }
    const uint64_t rest = p.depth / 8 * 8 + lane;
    if (rest < p.depth) add(__fmul_rn(from16(a[rest], p.dtype), from16(b[rest], p.dtype)));
    double all = double(sum) + double(lost);
#pragma unroll
    for (uint32_t o = 16; o; o /= 2) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    return float(all + double(bias));
}

// A step in the slope, as relu's, turns a value's error into a wrong gradient
// where the error passes zero.  The tensor core's additions cut toward zero,
// so a sum of k products is off by about k 2^-30 of its neighbours' mean size,
// ten times what rounded additions would leave, and by up to twice k 2^-29
// where the partial sums went far from zero on their way.  Where a value to be
// kept for the gradient is nearer to zero than k 2^-28 (and 1024 depths more,
// as the products of one step are cut too; 12 in a million at 4096 depths), it
// is summed again, as good as exactly.  Wrong signs of 690 million values at 520
// to 32768 depths: 17 with half that distance, none with it (32-bit sums: 5 in
// 180 million at 520).  4096 x 4096 x 4096 takes 90 us instead of 83, 2048 x
// 14336 x 4096 200 instead of 137.  v[i] are the lane's 32 values, `count` of
// them real; at most kMended of a patch, so that no input can make this the
// kernel's work.
constexpr uint32_t kMended = 16;
template <typename Again>
__device__ __forceinline__ void mend_near_zero(const Product& p, float v[32], uint32_t count, bool live, uint32_t lane, Again again) {
    float sum = 0.f;  // (past `count` a patch holds whatever was there)
#pragma unroll
    for (uint32_t i = 0; i < 32; ++i) sum += i < count ? fabsf(v[i]) : 0.f;
    float of = float(count);
    if (count < 8) {  // too few say nothing of their size: the whole patch
        if (!live) sum = 0.f;
#pragma unroll
        for (uint32_t o = 16; o; o /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        of *= float(__popc(__ballot_sync(0xFFFFFFFFu, live)));
    }
    const float near = sum / of * float(p.depth + 1024) * 0x1p-28f;
    uint32_t close = 0, zero = 0;
#pragma unroll
    for (uint32_t i = 0; i < 32; ++i) {
        if (fabsf(v[i]) < near) close |= 1u << i;
        if (v[i] == 0.f) zero |= 1u << i;
    }
    if (!live) close = 0;
    if (count < 32) close &= (1u << count) - 1;
    if (__reduce_add_sync(0xFFFFFFFFu, __popc(close & zero)) > kMended) close &= ~zero;  // zeros of a row or a column, not of a sum
    uint32_t lanes = __ballot_sync(0xFFFFFFFFu, close);
    for (uint32_t left = kMended; lanes && left; --left) {
        const uint32_t from = __ffs(lanes) - 1, at = __ffs(__shfl_sync(0xFFFFFFFFu, close, from)) - 1;
        const float mended = again(from, at);
        if (lane == from) {
            close &= close - 1;
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i)
                if (i == at && fabsf(mended) < INFINITY) v[i] = mended;  // (another order's partial sums may pass bf16's range)
        }
        lanes = __ballot_sync(0xFFFFFFFFu, close);
    }
}

// An accumulator of the transposed product: lanes are output columns (features)
// and accumulator columns are output rows (tokens), so a patch is written a
// token a step, 32 neighbouring features at once.  load(c, v) as in finish_tile.
template <bool FORWARD, typename Load>
__device__ __forceinline__ void finish_transposed(const Product& p, const Tiling& t, const Tile& o, uint32_t warp_row, uint32_t half,
                                                  const Patch& patch, Load load) {
    const uint32_t lane = patch.lane, feature0 = o.row0 + warp_row;
    const uint32_t features = feature0 < o.row_end ? min(32u, o.row_end - feature0) : 0;
    const int dtype = p.dtype;
    const StoreEpilogue& e = p.st;
    float bias = 0.f;
    if (e.bias && lane < features) bias = from16(static_cast<const uint16_t*>(e.bias)[o.group * p.m + feature0 + lane], dtype);
    uint16_t* const out = static_cast<uint16_t*>(e.out) + uint64_t(o.col0) * e.ldo + feature0;
    uint16_t* const z = e.z ? static_cast<uint16_t*>(e.z) + uint64_t(o.col0) * e.ldz + feature0 : nullptr;
#pragma unroll 1
    for (uint32_t c = half * kPatchCols; c < o.cols; c += 2 * kPatchCols) {
        const uint32_t tokens = min(32u, o.cols - c);
        float v[32];
        load(c, v);
#pragma unroll
        for (uint32_t i = 0; i < 32; ++i) v[i] += bias;
        if (FORWARD && z && e.act == UZIP_ACT_RELU)
            mend_near_zero(p, v, tokens, lane < features, lane, [&](uint32_t from, uint32_t at) {
                const float b = __shfl_sync(0xFFFFFFFFu, bias, from);
                return dot_again(p, o.group, 0, feature0 + from, o.col0 + c + at, b, lane);
            });
        if (z) {
            if (FORWARD && e.act == UZIP_ACT_RELU) patch.put_column<true>(v, dtype);
            else patch.put_column(v, dtype);
            patch.store(z + uint64_t(c) * e.ldz, e.ldz, tokens, features, t.z_width);
        }
        if (e.act == UZIP_ACT_RELU) {
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) v[i] = act_value(v[i], UZIP_ACT_RELU);
        } else if (e.act == UZIP_ACT_GELU) {
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) v[i] = act_value(v[i], UZIP_ACT_GELU);
        } else if (e.act == UZIP_ACT_SILU) {
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) v[i] = act_value(v[i], UZIP_ACT_SILU);
        }
        patch.put_column(v, dtype);
        patch.store(out + uint64_t(c) * e.ldo, e.ldo, tokens, features, t.out_width);
    }
    __syncwarp();
}

// The loss statistics of a row's logits in one half (128 columns) of a tile.
__device__ __forceinline__ void finish_stats(const Product& p, const Tile& o, uint64_t row, uint32_t half, float v[128]) {
    if (row >= o.row_end) return;
    const uint32_t col0 = o.col0 + half * 128, cols = min(128u, uint32_t(p.n) - col0);
    const int64_t target = p.ls.targets[row] - int64_t(col0);
    if (target >= 0 && target < int64_t(cols)) {
#pragma unroll
        for (uint32_t i = 0; i < 128; ++i)
            if (target == int64_t(i)) p.ls.hit[row] = v[i];
    }
    if (cols < 128) {
#pragma unroll
        for (uint32_t i = 0; i < 128; ++i)
            if (i >= cols) v[i] = -INFINITY;
    }
    float most[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (uint32_t i = 4; i < 128; ++i) most[i % 4] = fmaxf(most[i % 4], v[i]);
    const float top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])), base = top == -INFINITY ? 0.f : top;
    float add[4] = {};
#pragma unroll
    for (uint32_t i = 0; i < 128; ++i) add[i % 4] += fast_exp2((v[i] - base) * kLog2e);
    p.ls.part[row * p.ls.tiles + col0 / 128] = make_float2(top, (add[0] + add[1]) + (add[2] + add[3]));
}

// One finished accumulator of a block: 128 rows, one in each lane of the four
// warps of a column half; warps of half 0 take the patches 0, 2, ... of 32
// columns, those of half 1 the others.  `bias` is the warp's copy of its
// columns' bias.  load(c, v) brings the patch at column c into v.  The loops over
// patches stay rolled: the code of one patch fits the instruction cache, four of
// them did not.
template <int EPI, bool FORWARD, typename Load>
__device__ __forceinline__ void finish_tile(const Product& p, const Tiling& t, const Tile& o, uint32_t warp_row, uint32_t half,
                                            float alpha, const Patch& patch, const float* bias, uint4 ahead[4], Load load) {
    const uint32_t lane = patch.lane;
    const uint64_t row0 = uint64_t(o.row0) + warp_row, row = row0 + lane;
    const bool live = row < o.row_end;
    const uint32_t rows = row0 < o.row_end ? uint32_t(min(uint64_t(32), o.row_end - row0)) : 0;
    const uint32_t cols = o.cols;
    const int dtype = p.dtype;
    const StoreEpilogue& e = p.st;
    int64_t target = -1;
    float lse = 0.f, weight = 0.f;
    if (EPI == kLossGrad && live) {
        target = p.ls.targets[row] - int64_t(p.ls.col0 + o.col0);
        lse = p.ls.lse[row];
        weight = p.ls.g[row];
    }
    const bool wide = EPI == kStore && (e.out_fp32 || e.sum_in);  // partial results in 32 bits: few, after long depths
    const bool has_bias = EPI == kStore && e.bias, has_res = EPI == kStore && e.residual && !wide;
    const uint32_t act = EPI == kStore ? e.act : uint32_t(UZIP_ACT_NONE);
    uint16_t* const out = EPI == kStore ? static_cast<uint16_t*>(e.out) + o.group * e.out_group + row0 * e.ldo + o.col0
                                        : static_cast<uint16_t*>(p.ls.out) + row0 * p.ls.ldo + o.col0;
    const uint64_t ldo = EPI == kStore ? e.ldo : p.ls.ldo;
    const uint16_t* const res = static_cast<const uint16_t*>(e.residual) + row0 * e.ldr + o.col0;
    uint16_t* const z = EPI == kStore && e.z ? static_cast<uint16_t*>(e.z) + row0 * e.ldz + o.col0 : nullptr;
#pragma unroll 1
    for (uint32_t c = half * kPatchCols; c < cols; c += 2 * kPatchCols) {
        const uint32_t here = min(kPatchCols, cols - c);
        float v[32];
        load(c, v);
        if (wide) {
            if (live) {
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
                    if (8 * j < here) {
                        const uint32_t some = min(8u, here - 8 * j), col = o.col0 + c + 8 * j;
                        float* const q = v + 8 * j;
#pragma unroll
                        for (uint32_t i = 0; i < 8; ++i) q[i] *= alpha;
                        if (e.sum_in) add_sums8(e, t.vec, row, col, some, q);
                        const uint64_t at = row * e.ldo + col;
                        if (e.out_fp32) write_fp32(e, at, t.vec, some, q);
                        else write8(e.out, at, t.vec & 1, some, dtype, q);
                    }
            }
            __syncwarp();
            continue;
        }
        if (EPI == kLossGrad) {
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) {
                float d = fast_exp2((v[i] - lse) * kLog2e);  // (near p = 1 the difference is exact)
                if (target == int64_t(c + i)) d -= 1.f;
                v[i] = weight == 0.f ? 0.f : weight * d;
            }
        } else {
            if (e.alpha) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) v[i] *= alpha;
            }
            if (has_bias) {
                const float* const b = bias + c / 2 - half * (kPatchCols / 2);  // this warp's patches one after the other
#pragma unroll
                for (uint32_t i = 0; i < 32; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(b + i);
                    v[i] += f.x, v[i + 1] += f.y, v[i + 2] += f.z, v[i + 3] += f.w;
                }
            }
            if (FORWARD && z && act == UZIP_ACT_RELU)
                mend_near_zero(p, v, here, live, lane, [&](uint32_t from, uint32_t at) {
                    const float b = has_bias ? bias[c / 2 - half * (kPatchCols / 2) + at] : 0.f;
                    return dot_again(p, 0, o.group, row0 + from, uint64_t(o.col0) + c + at, b, lane);
                });
            if (z) {
                if (FORWARD && act == UZIP_ACT_RELU) patch.put<true>(v, dtype);
                else patch.put(v, dtype);
                patch.store(z + c, e.ldz, rows, here, t.z_width);
            }
            if (act == UZIP_ACT_RELU) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) v[i] = act_value(v[i], UZIP_ACT_RELU);
            } else if (act == UZIP_ACT_GELU) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) v[i] = act_value(v[i], UZIP_ACT_GELU);
            } else if (act == UZIP_ACT_SILU) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) v[i] = act_value(v[i], UZIP_ACT_SILU);
            }
            if (has_res) {
                __syncwarp();
                patch.place(ahead, (t.vec & 4) && here % 8 == 0);
                __syncwarp();
                if (c + 2 * kPatchCols < cols) {
                    const uint32_t next = min(kPatchCols, cols - c - 2 * kPatchCols);
                    patch.fetch(res + c + 2 * kPatchCols, e.ldr, rows, next, (t.vec & 4) && next % 8 == 0, ahead);
                }
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) {
                    const uint4 q = patch.at(lane, i);
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        const float2 f = from16x2(w[j], dtype);
                        v[8 * i + 2 * j] += f.x, v[8 * i + 2 * j + 1] += f.y;
                    }
                }
            }
        }
        patch.put(v, dtype);
        patch.store(out + c, ldo, rows, here, t.out_width);
    }
    __syncwarp();
}

// What a block that has given up a wait was to write becomes NaN (a caller that
// gave no status word would not learn of it otherwise).  The next products and
// the loss carry it on.
template <int EPI, bool TURNED>
__device__ __noinline__ void leave_nan(const Product& p, const Tiling& t, const int32_t* offsets) {
    const uint32_t rank = t.pair == 2 ? cluster_rank() & 1 : 0;
    Walk walk(p, t, offsets, offsets + p.groups + 1, p.live_rows ? *p.live_rows : uint32_t(p.m),
              p.live_depth ? *p.live_depth : uint32_t(p.depth));
    const uint16_t nan = p.dtype == UZIP_BF16 ? 0x7FC0 : 0x7E00;
    const StoreEpilogue& e = p.st;
    Tile o;
    while (walk.take(o)) {
        const uint64_t row0 = uint64_t(o.row0) + rank * kRowsTile;
        const uint32_t rows = row0 < o.row_end ? uint32_t(min(uint64_t(kRowsTile), o.row_end - row0)) : 0;
        for (uint32_t i = threadIdx.x; i < rows * o.cols; i += kThreads) {
            uint64_t row = row0 + i / o.cols, col = uint64_t(o.col0) + i % o.cols;
            if (EPI == kLossStats) {
                if (i % o.cols % kStatsCols == 0) p.ls.part[row * p.ls.tiles + col / kStatsCols] = make_float2(0.f, NAN);
            } else if (EPI == kLossGrad) {
                static_cast<uint16_t*>(p.ls.out)[row * p.ls.ldo + col] = nan;
            } else {
                if (TURNED) {
                    const uint64_t r = row;
                    row = col, col = r;
                }
                const uint64_t at = o.group * e.out_group + row * e.ldo + col;
                if (e.out_fp32) static_cast<float*>(e.out)[at] = NAN;
                else static_cast<uint16_t*>(e.out)[at] = nan;
                if (e.z) static_cast<uint16_t*>(e.z)[row * e.ldz + col] = nan;
            }
        }
    }
}

// ---- the kernel -------------------------------------------------------------------------

// MODE: 0 a block by itself, 1 a cluster of blocks splits the depth, 2 a pair of
// blocks, 3 a cluster of pairs splits the depth.
// LAYOUT: 0 both operands contiguous along the depth, 1 only A, 2 neither, 3
// neither, with a depth that only the device knows, 4 and 5 the
// transposed product with ragged columns, A contiguous along the depth or not.
// CHUNKED: a tile's depth is taken in chunks, added up in registers.
template <int EPI, int MODE, int LAYOUT, bool CHUNKED>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ Product p, const __grid_constant__ Tiling t,
                   const __grid_constant__ Maps<LAYOUT == 3> maps) {
    constexpr bool SPLIT = MODE & 1, PAIR = MODE & 2, STATS = EPI == kLossStats;
    constexpr uint32_t kChunk = EPI == kStore ? kLongChunk : kLogitChunk;
    constexpr bool A_DEEP = LAYOUT < 2 || LAYOUT == 4, B_DEEP = LAYOUT == 0 || LAYOUT > 3, CUT = LAYOUT == 3, TURNED = LAYOUT > 3;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    Control* ctl = reinterpret_cast<Control*>(smem + t.stages * t.stage_bytes + kEpilogueWarps * kEpilogueBytes);
    int32_t* offsets = reinterpret_cast<int32_t*>(ctl + 1);
    int32_t* first = offsets + p.groups + 1;
    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t rank = PAIR ? cluster_rank() & 1 : 0;  // the pair's block 0 issues the products,
    const uint32_t leader = MODE == 3 ? cluster_rank() & ~1u : 0;  // and has this rank in the cluster

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < t.stages; ++i) {
            mbar_init(smem_u32(&ctl->full[i]), 2);  // A's and B's bytes announced
            mbar_init(smem_u32(&ctl->empty[i]), 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl->acc_full[i]), 1);
            mbar_init(smem_u32(&ctl->acc_empty[i]), kEpilogueWarps * t.pair);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort = 0;
        ctl->wait_limit = t.wait_limit;
        fence_mbar_init();
    }
    wait_for_launch_before();
    const uint32_t live_rows = p.live_rows ? *p.live_rows : uint32_t(p.m), live_depth = p.live_depth ? *p.live_depth : uint32_t(p.depth);

    // the cut of the rows or depths, checked whole
    if (p.schedule != kDense) {
        const int64_t end = p.schedule == kRows ? p.m : p.schedule == kColumns ? p.n : p.depth;
        bool bad = false;
        for (uint32_t i = threadIdx.x; i <= p.groups; i += kThreads) {
            const int64_t v = p.offsets[i];
            bad |= v < 0 || v > end || (i == 0 && v != 0) || (i == p.groups ? v != end : v > p.offsets[i + 1]);
            offsets[i] = int32_t(v);
        }
        if (__syncthreads_or(bad)) {
            if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) atomicCAS(p.status, 0, int(UZIP_ERR_INVALID_ARG));
            const uint16_t nan = p.dtype == UZIP_BF16 ? 0x7FC0 : 0x7E00;
            const uint64_t out_rows = TURNED ? p.n : p.m, out_cols = TURNED ? p.m : p.n;
            const uint64_t total = p.m * p.n * (p.schedule == kDepth ? p.groups : 1);
            for (uint64_t i = blockIdx.x * uint64_t(kThreads) + threadIdx.x; i < total; i += uint64_t(gridDim.x) * kThreads) {
                const uint64_t r = i / out_cols, g = r / out_rows;
                static_cast<uint16_t*>(p.st.out)[g * p.st.out_group + (r - g * out_rows) * p.st.ldo + i % out_cols] = nan;
                if (p.st.z) static_cast<uint16_t*>(p.st.z)[r * p.st.ldz + i % out_cols] = nan;
            }
            return;
        }
        if (p.schedule != kDepth && warp == 0) {
            const uint32_t unit = TURNED ? t.bn : kRowsTile * t.pair;
            int32_t before = 0;
            for (uint32_t i = 0; i < p.groups; i += 32) {
                const uint32_t g = i + lane;
                int32_t v = 0;
                if (g < p.groups) v = int32_t((uint32_t(offsets[g + 1] - offsets[g]) + unit - 1) / unit);
#pragma unroll
                for (uint32_t d = 1; d < 32; d *= 2) {
                    const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, d);
                    if (lane >= d) v += u;
                }
                if (g < p.groups) first[g + 1] = before + v;
                before += __shfl_sync(0xFFFFFFFFu, v, 31);
            }
            if (lane == 0) first[0] = 0;
        }
    }
    if (warp == 1) tmem_alloc<PAIR>(smem_u32(&ctl->tmem), t.tmem_cols);
    tmem_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = ctl->tmem;
    const uint32_t buffer_cols = t.tmem_cols / 2;

    // One thread fetches A, another B: issuing a copy takes about 100 cycles, more while the epilogue's warps are busy,
    // and up to four to a stage would take longer than the stage's products.
    const auto fetch = [&](auto which) {
        constexpr bool IS_A = decltype(which)::value, DEEP = IS_A ? A_DEEP : B_DEEP;
        Walk walk(p, t, offsets, first, live_rows, live_depth);
        Tile o;
        Ring ring{t.stages};
        bool ok = true;
        const uint32_t b_cols = t.bn / (PAIR ? 2 : 1), slices = IS_A ? 2 : (b_cols + 63) / 64;
        const bool by_group = TURNED ? IS_A : walk.schedule == kRows && !IS_A;
        const bool slab = !DEEP && (IS_A ? t.a_slab : t.b_slab);
        const uint32_t box = IS_A ? t.a_box : t.b_box, stage_bytes = t.stage_bytes;
        [[maybe_unused]] const uint32_t beyond = uint32_t(p.depth);
        const uint32_t base = smem_u32(smem) + (IS_A ? 0 : t.a_stage), full = smem_u32(ctl->full), empty = smem_u32(ctl->empty);
        const uint32_t leader_full = PAIR ? cluster_address(full, leader) : full;
        const CUtensorMap* const map = IS_A ? &maps.a : &maps.b;
        while (ok && walk.take(o)) {
            const uint32_t half_width = o.width / (PAIR ? 2 : 1);
            const uint32_t row0 = IS_A ? o.row0 + rank * kRowsTile : o.col0 + rank * (TURNED ? half_width : b_cols);
            // rows in whole boxes (a pair's A: always 128)
            const uint32_t rows = IS_A ? (PAIR ? kRowsTile : min(kRowsTile, (o.row_end - row0 + box - 1) / box * box))
                                       : (half_width + box - 1) / box * box;
            const uint32_t bytes = (DEEP ? rows * 128 : slices * kSliceBytes) * (PAIR ? 2 : 1);
            const int group = by_group ? int(o.group) : 0;
            uint32_t d = o.d0;
            for (uint32_t i = 0; i < o.blocks; ++i, d += kDepthTile, ring.advance()) {
                if (!(ok = wait(ctl, empty + 8 * ring.s, ring.phase ^ 1))) break;
                const uint32_t mine = full + 8 * ring.s, bar = leader_full + 8 * ring.s;
                const uint32_t to = base + ring.s * stage_bytes;
                if constexpr (CUT) {
                    const uint32_t left = o.depth_end - d;
                    if (left < kDepthTile) {
                        // Depths past the end belong to the group's neighbour, or to nobody, and may hold anything: their
                        // lines are read from beyond the tensor's end, where TMA gives zeros.  (Both operands have
                        // contiguous rows here: a depth is one line of each slice.)
                        const uint32_t lines = (left + 15) / 16 * 16;
                        if (rank == 0) mbar_expect_tx(mine, slices * 128 * lines * (PAIR ? 2 : 1));
                        const CUtensorMap* const heights = IS_A ? maps.a_lines : maps.b_lines;
                        for (uint32_t l = 0; l < lines;) {  // kept and cleared lines, in powers of two
                            const uint32_t run = l < left ? left - l : lines - l, h = min(31u - __clz(run), kHeights - 1);
                            const int from = int(l < left ? d + l : beyond);
                            for (uint32_t r = 0; r < slices; ++r)
                                tma_load<PAIR>(to + r * kSliceBytes + l * 128, &heights[h], int(row0 + 64 * r), from, 0, bar);
                            l += 1u << h;
                        }
                        continue;
                    }
                }
                if (rank == 0) mbar_expect_tx(mine, bytes);
                if constexpr (DEEP) {
                    tma_load<PAIR>(to, map, int(d), int(row0), group, bar);
                    for (uint32_t r = box; r < rows; r += box) tma_load<PAIR>(to + r * 128, map, int(d), int(row0 + r), group, bar);
                } else if (slab) {
                    tma_load<PAIR>(to, map, 0, int(d), int(row0 / 64), bar);
                } else {
                    tma_load<PAIR>(to, map, int(row0), int(d), group, bar);
                    for (uint32_t r = 1; r < slices; ++r)
                        tma_load<PAIR>(to + r * kSliceBytes, map, int(row0 + 64 * r), int(d), group, bar);
                }
            }
        }
    };

    if (warp == 0) {
        if (elect_one() && !t.starve) fetch(std::true_type{});
        __syncwarp();
    } else if (warp == 6) {
        if (elect_one()) fetch(std::false_type{});
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            Walk walk(p, t, offsets, first, live_rows, live_depth);
            Tile o;
            Ring ring{t.stages};
            uint32_t used = 0;  // accumulators
            bool ok = true;
            // 16 depths further: 32 bytes along the depth, or 16 lines
            constexpr uint32_t kStepA = A_DEEP ? 2 : 128, kStepB = B_DEEP ? 2 : 128;
            const uint32_t idesc = t.idesc, stage_step = t.stage_bytes >> 4, full = smem_u32(ctl->full), empty = smem_u32(ctl->empty);
            const uint64_t desc_a = matrix_descriptor(smem_u32(smem), A_DEEP);
            // (the tensor core reads 128 rows of A also where a stage holds fewer: those accumulator rows are never
            // stored, and what lies there, the stage's B, later stages or the epilogue's patches, is shared memory of
            // this block)
            const uint64_t desc_b = matrix_descriptor(smem_u32(smem) + t.a_stage, B_DEEP);
            while (ok && walk.take(o)) {
                const uint32_t shape = TURNED ? idesc | o.width >> 3 << 17 : idesc;
                for (uint32_t i = 0; ok && (i < o.blocks || i == 0); ++used) {
                    const uint32_t buf = used & 1;
                    if (!(ok = wait(ctl, smem_u32(&ctl->acc_empty[buf]), (used >> 1 & 1) ^ 1))) break;
                    tmem_fence_after();
                    const uint32_t acc = tmem + buf * buffer_cols;
                    const uint32_t first_block = i, end = CHUNKED ? min(o.blocks, i + kChunk) : o.blocks;
                    if (end == 0) {  // nothing to add up: the epilogues take zeros
                        if (PAIR) {
                            cluster_arrive(cluster_address(smem_u32(&ctl->acc_full[buf]), leader));
                            cluster_arrive(cluster_address(smem_u32(&ctl->acc_full[buf]), leader + 1));
                        } else {
                            mbar_arrive(smem_u32(&ctl->acc_full[buf]));
                        }
                        ++i;
                        continue;
                    }
                    for (; i < end; ++i, ring.advance()) {
                        if (!(ok = wait(ctl, full + 8 * ring.s, ring.phase))) break;
                        tmem_fence_after();
                        const uint64_t a = desc_a + ring.s * stage_step, b = desc_b + ring.s * stage_step;
                        const uint32_t steps = CUT ? (o.depth_end - (o.d0 + i * kDepthTile) + 15) / 16 : 4;
                        mma<PAIR>(acc, a, b, shape, i != first_block);
                        if (!CUT || steps > 1) mma<PAIR>(acc, a + kStepA, b + kStepB, shape, 1);
                        if (!CUT || steps > 2) mma<PAIR>(acc, a + 2 * kStepA, b + 2 * kStepB, shape, 1);
                        if (!CUT || steps > 3) mma<PAIR>(acc, a + 3 * kStepA, b + 3 * kStepB, shape, 1);
                        mma_commit<PAIR>(empty + 8 * ring.s, leader);
                    }
                    if (!ok) break;  // not finished: the epilogues give up too, those of the pair's other block among them
                    mma_commit<PAIR>(smem_u32(&ctl->acc_full[buf]), leader);
                }
            }
            if (ctl->abort) {  // products in flight end before TMEM is freed
                mma_commit<PAIR>(smem_u32(&ctl->drain), leader);
                drain(&ctl->drain, 0);
            }
        }
        __syncwarp();
    } else if (STATS) {
        Walk walk(p, t, offsets, first, live_rows, live_depth);
        Tile o;
        uint32_t used = 0;
        bool ok = true;
        const uint32_t quarter = warp % 4, half = warp > 6;
        while (ok && walk.take(o)) {
            const uint32_t cols = o.cols, mine = cols > half * 128 ? cols - half * 128 : 0;
            float v[128];
#pragma unroll
            for (uint32_t i = 0; i < 128; ++i) v[i] = 0.f;
            for (uint32_t i = 0; i < max(o.blocks, 1u); i += kChunk, ++used) {
                const uint32_t buf = used & 1;
                if (!(ok = __all_sync(0xFFFFFFFFu, wait(ctl, smem_u32(&ctl->acc_full[buf]), used >> 1 & 1)))) break;
                tmem_fence_after();
                const uint32_t acc = tmem + buf * buffer_cols + half * 128 + (quarter * 32 << 16);
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c)
                    if (32 * c < mine && o.blocks) {
                        float add[32];
                        tmem_load32(acc + 32 * c, add);
#pragma unroll
                        for (uint32_t k = 0; k < 32; ++k) v[32 * c + k] += add[k];
                    }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) cluster_arrive(cluster_address(smem_u32(&ctl->acc_empty[buf]), leader));
                    else mbar_arrive(smem_u32(&ctl->acc_empty[buf]));
                }
            }
            if (ok && mine) finish_stats(p, o, uint64_t(o.row0) + rank * kRowsTile + quarter * 32 + lane, half, v);
            __syncwarp();
        }
    } else {
        Walk walk(p, t, offsets, first, live_rows, live_depth);
        Tile o;
        uint32_t used = 0;  // accumulators
        const uint32_t quarter = warp % 4, half = warp > 6;  // the TMEM lanes that this warp may read, its columns
        const float alpha = EPI == kStore && p.st.alpha ? *p.st.alpha : 1.f;
        uint8_t* const mine = reinterpret_cast<uint8_t*>(ctl) - (kEpilogueWarps - 4 * half - quarter) * kEpilogueBytes;
        const Patch patch{reinterpret_cast<uint4*>(mine), lane};
        float* const bias = reinterpret_cast<float*>(mine + kPatchBytes);
        while (walk.take(o)) {
            uint4 ahead[4] = {};
            if (!SPLIT) {
                // what the epilogue reads besides the products is fetched while they run
                o.row0 += rank * kRowsTile;
                const uint32_t cols = o.cols, c0 = half * kPatchCols;
                if (EPI == kStore && !TURNED && p.st.bias) {
                    const uint16_t* from = static_cast<const uint16_t*>(p.st.bias) + o.group * p.n + o.col0 + c0 + lane;
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i)
                        if (c0 + 2 * kPatchCols * i + lane < cols) bias[kPatchCols * i + lane] = from16(from[2 * kPatchCols * i], p.dtype);
                }
                if (EPI == kStore && !TURNED && p.st.residual && c0 < cols) {
                    const uint64_t row0 = uint64_t(o.row0) + quarter * 32;
                    const uint32_t rows = row0 < o.row_end ? uint32_t(min(uint64_t(32), o.row_end - row0)) : 0;
                    const uint32_t some = min(kPatchCols, cols - c0);
                    patch.fetch(static_cast<const uint16_t*>(p.st.residual) + row0 * p.st.ldr + o.col0 + c0, p.st.ldr, rows, some,
                                (t.vec & 4) && some % 8 == 0, ahead);
                }
                __syncwarp();
            }
            // the next accumulator, and the way to give it back once this warp has read its last column
            const auto arrived = [&] {
                const bool ok = __all_sync(0xFFFFFFFFu, wait(ctl, smem_u32(&ctl->acc_full[used & 1]), used >> 1 & 1));
                tmem_fence_after();
                return ok;
            };
            const auto release = [&](uint32_t buf) {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) cluster_arrive(cluster_address(smem_u32(&ctl->acc_empty[buf]), leader));
                    else mbar_arrive(smem_u32(&ctl->acc_empty[buf]));
                }
            };
            [[maybe_unused]] float sum[4][32] = {};  // CHUNKED: this warp's patches, the next one always in sum[0]
            if constexpr (CHUNKED) {
                bool ok = true;
                for (uint32_t i = 0; i < max(o.blocks, 1u); i += kChunk, ++used) {
                    if (!(ok = arrived())) break;
                    const uint32_t acc = tmem + (used & 1) * buffer_cols + half * kPatchCols + (quarter * 32 << 16);
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j)
                        if (half * kPatchCols + 2 * kPatchCols * j < o.cols && o.blocks) {
                            float add[32];
                            tmem_load32(acc + 2 * kPatchCols * j, add);
#pragma unroll
                            for (uint32_t k = 0; k < 32; ++k) sum[j][k] += add[k];
                        }
                    release(used & 1);
                }
                if (!ok) break;
            } else {
                if (!arrived()) break;
                if (!SPLIT && o.cols <= half * kPatchCols) release(used & 1);  // nothing of this tile is this warp's
            }
            const uint32_t buf = used & 1, acc = tmem + buf * buffer_cols + (quarter * 32 << 16);
            const bool empty = o.blocks == 0;
            const auto load = [&, buf, acc, empty](uint32_t c, float v[32]) {
                if constexpr (CHUNKED) {
#pragma unroll
                    for (uint32_t k = 0; k < 32; ++k) v[k] = sum[0][k], sum[0][k] = sum[1][k], sum[1][k] = sum[2][k], sum[2][k] = sum[3][k];
                } else {
                    if (empty) {
#pragma unroll
                        for (uint32_t i = 0; i < 32; ++i) v[i] = 0.f;
                    } else {
                        tmem_load32(acc + c, v);
                    }
                    if (!SPLIT && c + 2 * kPatchCols >= o.cols) release(buf);
                }
            };
            if constexpr (TURNED) {
                finish_transposed<LAYOUT == 4>(p, t, o, quarter * 32, half, patch, load);
            } else if constexpr (!SPLIT) {
                finish_tile<EPI, LAYOUT == 0>(p, t, o, quarter * 32, half, alpha, patch, bias, ahead, load);
            } else {
                const uint32_t lane_row = quarter * 32 + lane, row0 = o.row0 + rank * kRowsTile;
                // partial sums to shared memory, rows bn + 4 floats apart (no bank conflicts for 16-byte access)
                float* part = reinterpret_cast<float*>(smem) + lane_row * (t.bn + 4);
                for (uint32_t c = 32 * half; c < t.bn; c += 64) {
                    float v[32];
                    load(c, v);
#pragma unroll
                    for (uint32_t i = 0; i < 32; i += 4)
                        if (c + i < t.bn && row0 + lane_row < o.row_end)
                            *reinterpret_cast<float4*>(part + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
            if (!CHUNKED) ++used;
        }
    }
    if (SPLIT) {
        // every block of the cluster joins and finishes its share of the tile, in the order of the splits
        __syncthreads();
        cluster_sync();
        Walk walk(p, t, offsets, first, live_rows, live_depth);
        Tile o;
        if (walk.take(o) && o.row0 + rank * kRowsTile < o.row_end) {
            const float alpha = p.st.alpha ? *p.st.alpha : 1.f;
            o.row0 += rank * kRowsTile;
            const uint32_t rows = min(kRowsTile, o.row_end - o.row0), wide = t.bn / 8, items = rows * wide;
            const uint32_t base = smem_u32(smem);
            for (uint32_t i = walk.split * kThreads + threadIdx.x; i < items; i += t.splits * kThreads) {
                const uint32_t r = i / wide, c = i % wide * 8;
                if (o.col0 + c >= p.n) continue;
                const uint32_t at = base + (r * (t.bn + 4) + c) * 4;
                float4 lo[kMaxSplits], hi[kMaxSplits];
#pragma unroll
                for (uint32_t s = 0; s < kMaxSplits; ++s)  // all in flight at once
                    if (s < t.splits) {
                        const uint32_t from = cluster_address(at, PAIR ? 2 * s + rank : s);
                        lo[s] = cluster_load4(from), hi[s] = cluster_load4(from + 16);
                    }
                float v[8] = {};
#pragma unroll
                for (uint32_t s = 0; s < kMaxSplits; ++s)
                    if (s < t.splits) {
                        v[0] += lo[s].x, v[1] += lo[s].y, v[2] += lo[s].z, v[3] += lo[s].w;
                        v[4] += hi[s].x, v[5] += hi[s].y, v[6] += hi[s].z, v[7] += hi[s].w;
                    }
                store8(p, t.vec, 0, uint64_t(o.row0) + r, o.col0 + c, min(8u, uint32_t(p.n) - o.col0 - c), alpha, v);
            }
        }
        cluster_sync();
    }
    tmem_fence_before();
    __syncthreads();
    if (ctl->abort) {
        settle();
        leave_nan<EPI, TURNED>(p, t, offsets);
    }
    if (PAIR) cluster_sync();  // no arrival reaches a block that has ended
    tmem_fence_after();
    if (warp == 1) tmem_free<PAIR>(tmem, t.tmem_cols);
    if (threadIdx.x == 0 && ctl->abort && p.status) atomicCAS(p.status, 0, int(UZIP_ERR_TIMEOUT));
}

// ---- host side ----------------------------------------------------------------------------

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// rows x depth x groups of 16-bit values, read in swizzled boxes of 64 contiguous values
// (outer: rows of a box along the depth, else its depths); with slices, rows are contiguous, a multiple of 64, and a box
// holds that many slices of 64
cudaError_t make_map(CUtensorMap* map, const Operand& o, uint64_t rows, uint64_t depth, uint64_t groups, uint32_t box_outer,
                     int dtype, uint32_t slices = 0) {
    const uint64_t inner = o.depth_major ? depth : rows, outer = o.depth_major ? rows : depth;
    if (inner == 0 || outer == 0) {  // nothing to load
        *map = CUtensorMap{};
        return cudaSuccess;
    }
    EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {slices ? 64 : inner, outer, slices ? rows / 64 : groups};
    const uint64_t group = slices ? 128 : groups > 1 ? o.group * 2 : std::min<uint64_t>(o.ld * 2 * outer, uint64_t(1) << 39);
    const cuuint64_t strides[2] = {o.ld * 2, group};
    const cuuint32_t box[3] = {64, box_outer, slices ? slices : 1}, ones[3] = {1, 1, 1};
    const CUresult r = fn(map, dtype == UZIP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                          const_cast<void*>(o.p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

uint32_t row_width(const void* p, uint64_t ld) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(p) / 2 | ld;
    return bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
}
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

constexpr uint32_t kSmemMost = 227 * 1024;
std::atomic<uint32_t> g_starved_wait{0};  // 2^20 clock cycles (uzip_debug_starve_products)

bool cut(const Product& p) { return p.schedule == kDepth || p.live_depth; }  // the depths end where the device says
uint64_t col_tiles_of(const Product& p, uint32_t bn) {
    return p.schedule == kColumns ? p.n / bn + p.groups : (p.n + bn - 1) / bn;  // grouped: at most
}
uint64_t row_tiles_of(const Product& p, uint32_t pair) {
    const uint64_t unit = kRowsTile * pair;
    return p.schedule == kRows ? p.m / unit + p.groups : (p.m + unit - 1) / unit;  // grouped: at most
}
// grouped: what ragged groups take on average, with rows spread at random
double mean_row_tiles(const Product& p, uint32_t pair) {
    const uint64_t unit = kRowsTile * pair;
    if (p.schedule != kRows) return double((p.m + unit - 1) / unit);
    const double used = p.groups * (1 - std::exp(-double(p.m) / p.groups));
    return std::max(used, double(p.m) / unit + 0.5 * used);
}
uint64_t most_tiles(const Product& p, const Tiling& t) {
    return row_tiles_of(p, t.pair) * col_tiles_of(p, t.bn) * (p.schedule == kDepth ? p.groups : 1);
}

// Blocks that run at once in clusters of `size` (a GPC's odd SMs stay idle).
uint32_t cluster_blocks(uint32_t size, int sms);

// Tile width, split of the depth and pairing: the smallest estimate in clock
// cycles, from rates measured on a GB300 (1.9 GHz).  A stage of 64 depths
// costs the longest of its multiplication (2 cycles a column and 35), its way
// into shared memory (78 bytes a cycle for a block, 62 where only four stages
// fit: 128-column tiles of a single block ran at 385 to 410 cycles a stage,
// 256-column tiles at 640 to 770, pairs of 256 x 256 at 523) and the issue of
// its copies (350 cycles).  A wave of tiles costs its stages or, where that is
// longer, its epilogue and 1500 cycles; the last epilogue is not hidden, and joining the
// splits took 3.5 us and half a microsecond for every 12 KB of partial sums a
// block.  All bytes pass HBM once at 3500 a cycle; an operand streamed with
// its rows contiguous comes in lines of twice the tile's columns, and below
// 192 columns at three quarters of that rate (16 tokens through 8 experts of
// 4096 x 14336, transposed: 103 us at 256 columns, 132 at 128).  The two times
// overlap, less well the closer they are: they are joined by a cubic mean.
struct Choice {
    Tiling t;
    double cost;
};

// The search takes 2 to 3 us, which a call of a few microseconds feels, so each
// thread remembers its last choices by what they depend on: sizes and kind of
// product, nothing of the operands.
struct Picked {
    uint64_t m, n, depth;
    uint32_t groups, kind;
    uint32_t bn, splits, pair;
    double cost;
};
Picked* picked_slot(const Product& p, uint32_t kind) {
    static thread_local Picked slots[64];  // kind 0: empty
    const uint64_t h = (p.m * 0x9E3779B97F4A7C15ull ^ p.n * 0xC2B2AE3D27D4EB4Full ^ p.depth * 0x165667B19E3779F9ull ^ p.groups ^ kind) *
                       0x9E3779B97F4A7C15ull;
    return &slots[h >> 58];
}

void search_tile(const Product& p, int sms, Picked& best) {
    double best_cost = 1e300;
    const uint64_t rows = p.m, groups = p.schedule == kDepth ? p.groups : 1;
    const double blocks = std::max(1.0, double(p.depth) / (p.schedule == kDepth ? p.groups : 1) / kDepthTile);
    const uint32_t low = uint32_t(std::min<uint64_t>(kRowsTile, (rows + 7) / 8 * 8));
    const uint32_t unit = p.b.depth_major ? 16 : 64;  // whole slices where rows are contiguous
    const uint32_t widest = uint32_t(std::min<uint64_t>(256, (p.n + unit - 1) / unit * unit));
    // (values near zero that are kept for relu's gradient are summed again where one block holds a tile's whole depth)
    const bool may_split = p.epilogue == kStore && p.schedule == kDense && !p.live_depth && !(p.st.z && p.st.act == UZIP_ACT_RELU);
    const double column = (p.st.ldo % 8 ? 40.0 : 14.0) * (p.st.z ? 2 : 1);  // epilogue cycles a column
    const double used = p.schedule == kRows || p.schedule == kColumns  // groups that have rows, when these are spread at random
                            ? p.groups * (1 - std::exp(-double(p.schedule == kRows ? p.m : p.n) / p.groups)) : groups;
    const double a_groups = p.schedule == kColumns ? used : 1, b_groups = p.schedule == kRows ? used : 1;
    const double traffic = 2.0 * (a_groups * p.m * p.depth + b_groups * p.n * p.depth +
                                  groups * p.m * p.n * ((p.st.z ? 2 : 1) + (p.st.residual ? 1 : 0)));
    auto both = [](double x, double y) {  // close to the cube root of the sum of cubes
        const double more = std::max(x, y), share = std::min(x, y) / more;
        return more * (1 + 0.26 * share * share * share);
    };
    const double row_tiles[3] = {0, mean_row_tiles(p, 1), mean_row_tiles(p, 2)};
    auto offer = [&](uint32_t bn, uint32_t splits, uint32_t pair, double waves, double stage, double last) {
        const double work = (waves - 1) * std::max(blocks * stage, last + 1500) + std::ceil(blocks / splits) * stage;
        const double rate = p.schedule != kColumns && !p.b.depth_major && bn < 192 ? 2700 : 3500;
        const double cost = both(work, traffic / rate) + last + 1000.0 * pair;
        if (cost >= best_cost) return;
        best_cost = cost;
        best.bn = bn, best.splits = splits, best.pair = pair;
    };
    auto stage_of = [](double width, double bytes) { return std::max({2 * width + 35, bytes / (bytes > 40960 ? 62 : 78), 350.0}); };
    auto consider = [&](uint32_t bn, uint32_t splits, uint32_t pair) {
        const double tiles = row_tiles[pair] * double((p.n + bn - 1) / bn * groups);
        const double at_once = double(splits > 1 ? cluster_blocks(splits * pair, sms) / (splits * pair) : sms / pair);
        // (how many tiles ragged rows make is not known: half a wave more on average)
        const double waves = p.schedule == kRows ? std::max(1.0, tiles / at_once + 0.5) : std::ceil(tiles / at_once);
        double last = column * bn;
        if (splits > 1) last = std::ceil(low * bn / 8.0 / (kThreads * splits)) * (1000 + 2 * column) + 6500;
        offer(bn, splits, pair, waves, stage_of(bn, ((pair == 2 ? kRowsTile : low) + bn / pair) * 128.0), last);
    };
    // Ragged columns: a group's columns go in tiles of equal width up to bn, so a tile costs what it holds.
    const double mean = p.n / std::max(1.0, used);
    auto consider_turned = [&](uint32_t bn, uint32_t pair) {
        const double each = mean <= 0.8 * bn ? 1.0 : mean / bn + 0.5, width = std::min<double>(bn, mean / each + 8 * pair);
        const double tiles = used * each * double(row_tiles_of(p, pair));
        offer(bn, 1, pair, std::max(1.0, tiles / (sms / pair) + 0.5), stage_of(width, (kRowsTile + bn / pair) * 128.0),
              1.5 * column * width);
    };
    if (p.schedule == kColumns) {
        for (uint32_t bn : {256u, 128u, 64u, 32u})
            if (bn <= widest || bn == 32) consider_turned(bn, 1);
        if (rows > kRowsTile) consider_turned(256, 2);
    } else {
        for (uint32_t bn = widest; bn >= unit; bn -= unit) {
            if (bn < 32 && bn < widest) break;
            if (p.epilogue == kLossStats && bn % 128 && bn < widest) continue;  // statistics are kept for every 128 columns
            consider(bn, 1, 1);
            if (may_split)
                for (uint32_t splits = 2; splits <= kMaxSplits && blocks / splits >= 4; ++splits) consider(bn, splits, 1);
        }
        if (rows > kRowsTile)
            for (uint32_t bn = 256; bn >= 96; bn -= 32)
                if (p.epilogue != kLossStats || bn % 128 == 0) {
                    consider(bn, 1, 2);
                    if (may_split)
                        for (uint32_t splits = 2; splits <= kMaxSplits / 2 && blocks / splits >= 4; ++splits) consider(bn, splits, 2);
                }
    }
    best.cost = best_cost;
}

Choice choose(const Product& p, int sms) {
    const StoreEpilogue& e = p.st;
    const uint32_t kind = 1 | p.schedule << 1 | p.epilogue << 3 | (p.a.depth_major ? 32 : 0) | (p.b.depth_major ? 64 : 0) |
                          (e.z ? 128 : 0) | (e.residual ? 256 : 0) | (e.ldo % 8 ? 512 : 0) |
                          (e.z && e.act == UZIP_ACT_RELU ? 1024 : 0) | (p.live_depth ? 2048 : 0);
    Picked* const slot = picked_slot(p, kind);
    if (slot->kind != kind || slot->m != p.m || slot->n != p.n || slot->depth != p.depth || slot->groups != p.groups) {
        *slot = Picked{p.m, p.n, p.depth, p.groups, kind, 0, 0, 0, 0};
        search_tile(p, sms, *slot);
    }
    Tiling t{};
    t.bn = slot->bn, t.splits = slot->splits, t.pair = slot->pair;
    const uint64_t rows = p.m;
    const uint32_t low = uint32_t(std::min<uint64_t>(kRowsTile, (rows + 7) / 8 * 8));
    const double used = p.groups * (1 - std::exp(-double(p.n) / p.groups)), mean = p.n / std::max(1.0, used);  // kColumns
    const uint32_t b_cols = t.bn / t.pair;
    t.b_box = p.schedule != kColumns ? b_cols : std::min(b_cols, mean >= 96 * t.pair ? 64u : mean >= 24 ? 32u : 16u);
    // the slices of a stage come in one box where they end with the rows (the third dimension is the groups' otherwise)
    const bool one_group = p.schedule == kDense || p.schedule == kDepth;
    t.a_slab = one_group && !p.a.depth_major && p.m % 64 == 0 ? 2 : 0;
    t.b_slab = one_group && !p.b.depth_major && p.n % 64 == 0 && b_cols % 64 == 0 ? b_cols / 64 : 0;
    const uint32_t b_bytes = p.b.depth_major ? b_cols * 128 : (b_cols + 63) / 64 * kSliceBytes;
    const bool few = t.pair == 1 && p.a.depth_major;
    t.a_box = !few ? kRowsTile : p.schedule != kRows || low < 32 ? low : rows / p.groups >= 96 ? kRowsTile : 32;
    t.a_stage = few ? (low + t.a_box - 1) / t.a_box * t.a_box * 128 : kAStage;
    t.stage_bytes = t.a_stage + b_bytes;
    const uint32_t tables = p.schedule == kDense ? 0 : (2 * p.groups + 2) * 4;
    const uint32_t rest = 1024 + kEpilogueWarps * kEpilogueBytes + sizeof(Control) + tables;
    t.stages = std::min<uint32_t>(kMaxStages, (kSmemMost - rest) / t.stage_bytes);
    // (with splits the partial sums, 512 bn + 2 KiB bytes, take the stages' place: always less)
    t.smem = rest + t.stages * t.stage_bytes;
    uint32_t cols = 32;
    while (cols < 2 * ((t.bn + 31) / 32 * 32)) cols *= 2;
    t.tmem_cols = cols;
    t.raster = 16 / t.pair;
    const uint32_t fmt = p.dtype == UZIP_BF16 ? 1 : 0;
    t.idesc = 1u << 4 | fmt << 7 | fmt << 10 | (p.a.depth_major ? 0u : 1u << 15) | (p.b.depth_major ? 0u : 1u << 16) |
              (p.schedule == kColumns ? 0 : t.bn >> 3 << 17) | (kRowsTile * t.pair >> 4) << 24;
    t.out_width = p.epilogue == kLossGrad ? 8 : row_width(e.out, e.ldo | e.out_group);
    t.z_width = row_width(e.z, e.ldz);
    const uint32_t out_unit = e.out_fp32 ? 4 : 8;
    t.vec = (aligned16(e.out) && e.ldo % out_unit == 0 && e.out_group % out_unit == 0 ? 1 : 0) |
            (aligned16(e.bias) && (p.n % 8 == 0 || p.groups == 1) ? 2 : 0) | (aligned16(e.residual) && e.ldr % 8 == 0 ? 4 : 0) |
            (aligned16(e.z) && e.ldz % 8 == 0 ? 8 : 0) | (aligned16(e.sum_in) && e.ld_sum % 4 == 0 ? 16 : 0);
    const uint32_t starved = g_starved_wait.load(std::memory_order_relaxed);
    t.starve = starved != 0;
    t.wait_limit = starved ? starved : kWaitLimit;
    return Choice{t, slot->cost};
}

template <int EPI, int MODE, int LAYOUT, bool CHUNKED>
cudaError_t launch(const Product& p, const Tiling& t, int sms, const Maps<LAYOUT == 3>& maps, cudaStream_t s) {
    auto kern = product_kernel<EPI, MODE, LAYOUT, CHUNKED>;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use all of the shared memory
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemMost));
        if (err != cudaSuccess) return err;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    const uint64_t tiles = most_tiles(p, t);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(uint32_t(MODE & 1    ? tiles * t.splits * t.pair
                                : MODE == 2 ? 2 * std::min<uint64_t>(tiles, sms / 2)
                                            : std::min<uint64_t>(tiles, sms)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = t.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = t.splits * t.pair;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = MODE ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p, t, maps);
}

template <int EPI, int LAYOUT, bool CHUNKED>
cudaError_t launch_mode(const Product& p, const Tiling& t, int sms, cudaStream_t s) {
    constexpr bool kCut = LAYOUT == 3, kTurned = LAYOUT > 3, kMaySplit = EPI == kStore && !kCut && !kTurned;
    Maps<kCut> maps;
    cudaError_t err = make_map(&maps.a, p.a, p.m, p.depth, kTurned ? p.groups : 1, p.a.depth_major ? t.a_box : kDepthTile, p.dtype, t.a_slab);
    if (err == cudaSuccess)
        err = make_map(&maps.b, p.b, p.n, p.depth, p.schedule == kRows ? p.groups : 1, p.b.depth_major ? t.b_box : kDepthTile, p.dtype,
                       t.b_slab);
    if constexpr (kCut) {
        for (uint32_t h = 0; h < kHeights && err == cudaSuccess; ++h) {
            err = make_map(&maps.a_lines[h], p.a, p.m, p.depth, 1, 1u << h, p.dtype);
            if (err == cudaSuccess) err = make_map(&maps.b_lines[h], p.b, p.n, p.depth, 1, 1u << h, p.dtype);
        }
    }
    if (err != cudaSuccess) return err;
    if (kMaySplit && t.pair == 2 && t.splits > 1) return launch<EPI, kMaySplit ? 3 : 2, LAYOUT, CHUNKED>(p, t, sms, maps, s);
    if (t.pair == 2) return launch<EPI, 2, LAYOUT, CHUNKED>(p, t, sms, maps, s);
    if (kMaySplit && t.splits > 1) return launch<EPI, kMaySplit ? 1 : 0, LAYOUT, CHUNKED>(p, t, sms, maps, s);
    return launch<EPI, 0, LAYOUT, CHUNKED>(p, t, sms, maps, s);
}

template <int EPI, int LAYOUT>
cudaError_t launch_layout(const Product& p, const Tiling& t, int sms, cudaStream_t s) {
    if constexpr (EPI != kStore) {
        return launch_mode<EPI, LAYOUT, true>(p, t, sms, s);
    } else {
        // the most depths that a block may meet in one tile (a group may have all of them)
        const bool long_depth = (p.depth + kDepthTile - 1) / kDepthTile > uint64_t(kLongChunk) * t.splits;
        return long_depth ? launch_mode<EPI, LAYOUT, true>(p, t, sms, s) : launch_mode<EPI, LAYOUT, false>(p, t, sms, s);
    }
}

uint32_t cluster_blocks(uint32_t size, int sms) {
    static const std::array<uint32_t, kMaxSplits + 1> most = [sms] {
        std::array<uint32_t, kMaxSplits + 1> v{};
        auto kern = product_kernel<kStore, 1, 0, false>;
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemMost));
        for (uint32_t size = 1; size <= kMaxSplits; ++size) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(size * 64);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = kSmemMost;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = size, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
                cudaGetLastError();
                n = std::max(1, sms / int(size));
            }
            v[size] = uint32_t(n) * size;
        }
        return v;
    }();
    return most[size];
}

}  // namespace

cudaError_t launch_product(const Product& p, int sms, cudaStream_t s) {
    if (p.m == 0 || p.n == 0) return cudaSuccess;
    const Choice c = choose(p, sms);
    const Tiling& t = c.t;
    if (p.epilogue == kLossStats) return launch_layout<kLossStats, 0>(p, t, sms, s);
    if (p.epilogue == kLossGrad) return launch_layout<kLossGrad, 0>(p, t, sms, s);
    if (p.schedule == kRows && !p.st.residual) {
        // Groups' rows as the columns of the transposed product: a tile takes as many as there are instead of 128 or
        // 256, at the price of a slower epilogue, which adds no residual.
        Product q = p;
        q.a = p.b, q.b = p.a, q.m = p.n, q.n = p.m, q.schedule = kColumns;
        const Choice turned = choose(q, sms);
        if (turned.cost < c.cost) {
            return q.a.depth_major ? launch_layout<kStore, 4>(q, turned.t, sms, s) : launch_layout<kStore, 5>(q, turned.t, sms, s);
        }
    }
    if (p.b.depth_major) return launch_layout<kStore, 0>(p, t, sms, s);
    if (p.a.depth_major) return launch_layout<kStore, 1>(p, t, sms, s);
    return cut(p) ? launch_layout<kStore, 3>(p, t, sms, s) : launch_layout<kStore, 2>(p, t, sms, s);
}

}  // namespace uzip

extern "C" void uzip_debug_starve_products(int64_t wait_cycles) {
    uzip::g_starved_wait = uint32_t(std::min<int64_t>((std::max<int64_t>(wait_cycles, 0) + (1 << 20) - 1) >> 20, uzip::kWaitLimit));
}
