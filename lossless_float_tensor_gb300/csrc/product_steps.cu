// The element-wise steps around the matrix products: row packing, the
// activation's gradient with the bias gradient, the checks of offsets and
// targets, and the joining of the loss statistics.  All of them read and
// write each value once and are bound by memory bandwidth or launch latency.
#include <algorithm>

#include "product.cuh"

namespace uzip {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint64_t kSms = 152;  // these steps' grids are sized for a GB300; any other number would do

// A launch whose blocks may be set up while the one before it ends: the kernel starts with wait_for_launch_before().
template <typename... Args, typename... Given>
cudaError_t launch_after(void (*kernel)(Args...), dim3 grid, uint32_t threads, cudaStream_t s, Given... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Args(args)...);
}

uint32_t blocks_for(uint64_t items, uint64_t most) {
    return uint32_t(std::max<uint64_t>(1, std::min<uint64_t>((items + kThreads - 1) / kThreads, most)));
}

// Rows copied to rows on 16-byte boundaries; the last values of a padded row
// are zero.  One thread makes one 16-byte store from eight 2-byte loads.
// blockIdx.y is the matrix.
__global__ void __launch_bounds__(kThreads) pack_kernel(const __grid_constant__ PackJobs jobs) {
    wait_for_launch_before();
    const PackJob& j = jobs.job[blockIdx.y];
    const uint64_t vecs = j.ld_to / 8, total = vecs * j.rows * j.groups;
    for (uint64_t i = blockIdx.x * uint64_t(kThreads) + threadIdx.x; i < total; i += uint64_t(gridDim.x) * kThreads) {
        const uint64_t v = i % vecs, r = i / vecs, g = r / j.rows, row = r - g * j.rows;
        const uint16_t* src = static_cast<const uint16_t*>(j.from) + g * j.group + row * j.ld + 8 * v;
        uint32_t w[4];
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            const uint32_t lo = 8 * v + 2 * k < j.cols ? src[2 * k] : 0u;
            const uint32_t hi = 8 * v + 2 * k + 1 < j.cols ? src[2 * k + 1] : 0u;
            w[k] = lo | hi << 16;
        }
        static_cast<uint4*>(j.to)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

__global__ void __launch_bounds__(kThreads) clear_kernel(uint16_t* p, uint64_t ld, uint64_t cols, uint64_t total) {
    wait_for_launch_before();
    for (uint64_t i = blockIdx.x * uint64_t(kThreads) + threadIdx.x; i < total; i += uint64_t(gridDim.x) * kThreads)
        p[i / cols * ld + i % cols] = 0;
}

// Block (x, y, z): 128 columns, a share of the rows, one group.  Where rows
// start on 16-byte boundaries a thread holds 8 neighbouring columns and walks
// every 16th row; elsewhere it holds columns 32 apart, so that a warp still
// reads neighbouring values, and walks every 8th row.  64 rows of a block are
// in flight; the partial column sums meet in shared memory in a fixed order.
constexpr uint32_t kGradCols = 128;

__device__ __forceinline__ void spread8(const uint4& q, int dtype, float v[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
        const float2 f = from16x2(w[j], dtype);
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
    }
}
template <int N>
__device__ __forceinline__ void times_slope(float d[N], const float z[N], uint32_t act) {
    if (act == UZIP_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) d[j] *= act_slope(z[j], UZIP_ACT_RELU);
    } else if (act == UZIP_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) d[j] *= act_slope(z[j], UZIP_ACT_GELU);
    } else if (act == UZIP_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) d[j] *= act_slope(z[j], UZIP_ACT_SILU);
    }
}

// Whether this thread's share of the offsets breaks the rule: 0, never less, m.
__device__ __forceinline__ bool offsets_bad(const int64_t* offsets, uint32_t groups, uint64_t m) {
    bool bad = false;
    for (uint32_t i = threadIdx.x; i <= groups; i += kThreads) {
        const int64_t v = offsets[i];
        bad |= v < 0 || v > int64_t(m) || (i == 0 && v != 0) || (i == groups ? v != int64_t(m) : v > offsets[i + 1]);
    }
    return bad;
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads) act_grad_kernel(const __grid_constant__ ActGrad a) {
    wait_for_launch_before();
    constexpr uint32_t kAcross = VEC ? 16 : 32, kRows = kThreads / kAcross, kHeld = kGradCols / kAcross;
    constexpr uint32_t kGradAhead = 64 / kRows;
    __shared__ float sums[kRows][kGradCols + 4];
    const uint32_t tx = threadIdx.x % kAcross, ty = threadIdx.x / kAcross, g = blockIdx.z;
    const uint64_t col0 = uint64_t(blockIdx.x) * kGradCols;
    uint64_t r0 = 0, r1 = a.m;
    bool bad = false;
    if (a.offsets) {
        bad = __syncthreads_or(offsets_bad(a.offsets, a.groups, a.m));
        if (bad && a.status && blockIdx.x + blockIdx.y + blockIdx.z + threadIdx.x == 0)
            atomicCAS(a.status, 0, int(UZIP_ERR_INVALID_ARG));
        r0 = bad ? 0 : a.offsets[g], r1 = bad ? 0 : a.offsets[g + 1];
    }
    const uint64_t share = (r1 - r0 + a.splits - 1) / a.splits;
    r0 = min(r0 + blockIdx.y * share, r1);
    r1 = min(r0 + share, r1);
    const bool has_act = a.act != UZIP_ACT_NONE;
    float sum[kHeld] = {};
    const uint16_t* const dy = static_cast<const uint16_t*>(a.dy) + col0;
    const uint16_t* const z = static_cast<const uint16_t*>(a.z) + col0;
    uint16_t* const dz = static_cast<uint16_t*>(a.dz) + col0;
    const uint32_t cols = uint32_t(min(uint64_t(kGradCols), a.n - col0));
    if (!VEC || tx * 8 < cols)
        for (uint64_t r = r0 + ty; r < r1; r += kGradAhead * kRows) {
            uint4 qd[kGradAhead], qz[kGradAhead];
            uint16_t ud[kGradAhead][kHeld], uz[kGradAhead][kHeld];
#pragma unroll
            for (uint32_t i = 0; i < kGradAhead; ++i) {
                const uint64_t row = r + i * kRows;
                if (row >= r1) break;
                if (VEC) {
                    qd[i] = *reinterpret_cast<const uint4*>(dy + row * a.lddy + 8 * tx);
                    if (has_act) qz[i] = *reinterpret_cast<const uint4*>(z + row * a.ldz + 8 * tx);
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < kHeld; ++j) {
                        const uint32_t c = tx + j * kAcross;
                        ud[i][j] = c < cols ? dy[row * a.lddy + c] : 0;
                        uz[i][j] = c < cols && has_act ? z[row * a.ldz + c] : 0;
                    }
                }
            }
#pragma unroll
            for (uint32_t i = 0; i < kGradAhead; ++i) {
                const uint64_t row = r + i * kRows;
                if (row >= r1) break;
                float d[kHeld], f[kHeld];
                if constexpr (VEC) {
                    spread8(qd[i], a.dtype, d);
                    spread8(qz[i], a.dtype, f);
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < kHeld; ++j) d[j] = from16(ud[i][j], a.dtype), f[j] = from16(uz[i][j], a.dtype);
                }
                times_slope<kHeld>(d, f, a.act);
#pragma unroll
                for (uint32_t j = 0; j < kHeld; ++j) sum[j] += d[j];
                if (!a.dz) continue;
                if constexpr (VEC) {
                    *reinterpret_cast<uint4*>(dz + row * a.lddz + 8 * tx) =
                        make_uint4(to16x2(d[0], d[1], a.dtype), to16x2(d[2], d[3], a.dtype), to16x2(d[4], d[5], a.dtype),
                                   to16x2(d[6], d[7], a.dtype));
                } else {  // the work area's rows are padded to 16 bytes: the padding is written too
#pragma unroll
                    for (uint32_t j = 0; j < kHeld; ++j)
                        if (col0 + tx + j * kAcross < a.lddz) dz[row * a.lddz + tx + j * kAcross] = to16(d[j], a.dtype);
                }
            }
        }
    if (!a.db) return;
#pragma unroll
    for (uint32_t j = 0; j < kHeld; ++j) sums[ty][VEC ? kHeld * tx + j : tx + j * kAcross] = sum[j];
    __syncthreads();
    if (threadIdx.x < cols) {
        float total = bad ? NAN : 0.f;
#pragma unroll
        for (uint32_t i = 0; i < kRows; ++i) total += sums[i][threadIdx.x];
        const uint64_t c = col0 + threadIdx.x;
        if (a.splits > 1) a.part[(uint64_t(g) * a.splits + blockIdx.y) * a.n + c] = total;
        else static_cast<uint16_t*>(a.db)[g * a.n + c] = to16(total, a.dtype);
    }
}

__global__ void __launch_bounds__(kThreads) join_columns_kernel(const float* part, uint32_t splits, uint64_t n,
                                                                uint64_t total, uint16_t* db, int dtype) {
    wait_for_launch_before();
    const uint64_t i = blockIdx.x * uint64_t(kThreads) + threadIdx.x;
    if (i >= total) return;
    const uint64_t g = i / n, c = i - g * n;
    float v = 0.f;
    for (uint32_t s = 0; s < splits; ++s) v += part[(g * splits + s) * n + c];
    db[i] = to16(v, dtype);
}

__global__ void __launch_bounds__(kThreads) offset_check_kernel(const int64_t* offsets, uint32_t groups, uint64_t m,
                                                                int32_t* status) {
    wait_for_launch_before();
    if (__syncthreads_or(offsets_bad(offsets, groups, m)) && threadIdx.x == 0) *status = int(UZIP_ERR_INVALID_ARG);
}

// Two (maximum, sum of exponentials) pairs as one; NaN sums stay.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x), base = top == -INFINITY ? 0.f : top;
    return make_float2(top, a.y * exp2f((a.x - base) * kLog2e) + b.y * exp2f((b.x - base) * kLog2e));
}

// One block for each row joins its tiles' pairs: thread i takes tiles i,
// i + 128, ..., then pairs of threads meet, always in the same order.
constexpr uint32_t kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) loss_join_kernel(LossEpilogue e, const uint32_t* token, const uint32_t* count,
                                                                 uint64_t v, uint32_t tiles, float* loss, float* lse,
                                                                 int32_t* status) {
    wait_for_launch_before();
    __shared__ float2 s[kJoinThreads / 32];
    const uint64_t row = blockIdx.x;
    if (count && row >= *count) return;
    const float2* part = e.part + row * tiles;
    float2 q = make_float2(-INFINITY, 0.f);
    for (uint32_t i = threadIdx.x; i < tiles; i += kJoinThreads) q = join(q, part[i]);
#pragma unroll
    for (uint32_t o = 16; o; o /= 2)
        q = join(q, make_float2(__shfl_xor_sync(0xFFFFFFFFu, q.x, o), __shfl_xor_sync(0xFFFFFFFFu, q.y, o)));
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = q;
    __syncthreads();
    if (threadIdx.x) return;
    q = join(join(s[0], s[1]), join(s[2], s[3]));
    const int64_t target = e.targets[row];
    const uint64_t to = token ? token[row] : row;
    if (target == e.ignore) {
        loss[to] = 0.f;
        lse[to] = 0.f;
        return;
    }
    const float l = q.x + logf(q.y);
    lse[to] = l;
    if (target < 0 || target >= int64_t(v)) {
        loss[to] = NAN;
        if (status) atomicCAS(status, 0, int(UZIP_ERR_INVALID_ARG));
        return;
    }
    loss[to] = l - e.hit[row];
}

// Every block counts through all targets (they are few beside the rows), a
// thousand at a time, and copies the rows i with i % gridDim.x == blockIdx.x: the
// places come out the same in each, without a launch in between.
constexpr uint32_t kPickThreads = 1024, kPickList = 2048;
__global__ void __launch_bounds__(kPickThreads) loss_rows_kernel(const __grid_constant__ LossRows a) {
    wait_for_launch_before();
    __shared__ uint32_t list[kPickList][2];  // token, place
    __shared__ uint32_t listed, before[32];
    __shared__ float tops[32];
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (threadIdx.x == 0) listed = 0;
    float up = 1.f;
    if (a.dloss) {
        float top = 0.f;
        for (uint64_t i = threadIdx.x; i < a.t; i += kPickThreads) {
            const float w = fabsf(a.dloss[i]);
            if (a.targets[i] != a.ignore && w < INFINITY) top = fmaxf(top, w);
        }
#pragma unroll
        for (uint32_t o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        top = tops[lane];
#pragma unroll
        for (uint32_t o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        // The largest weight becomes 2^10.  Not merely something between 2^10 and 2^11: equal weights, as in a mean, then
        // all round alike, and a target's g (p - 1), nearly g, would carry one rounding error through the whole gradient.
        up = top > 0.f ? fminf(1024.f / top, 0x1p120f) : 1.f;
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.scale = 1.f / up;
    }
    uint32_t base = 0;
    for (uint64_t start = 0; start < a.t; start += kPickThreads) {
        const uint64_t i = start + threadIdx.x;
        const bool mine = i < a.t && i % gridDim.x == blockIdx.x;
        const int64_t target = i < a.t ? a.targets[i] : a.ignore;
        const bool used = target != a.ignore;
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, used);
        __syncthreads();  // the counts of the last round, and the list, are read
        if (lane == 0) before[warp] = __popc(votes);
        __syncthreads();
        uint32_t sum = before[lane];
#pragma unroll
        for (uint32_t o = 1; o < 32; o *= 2) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += v;
        }
        const uint32_t mine_before = warp ? __shfl_sync(0xFFFFFFFFu, sum, warp - 1) : 0;
        const uint32_t place = base + mine_before + __popc(votes & lanemask_lt());
        base += __shfl_sync(0xFFFFFFFFu, sum, 31);
        if (mine && used) {
            const uint32_t k = atomicAdd(&listed, 1);
            list[k][0] = uint32_t(i), list[k][1] = place;
            a.out_targets[place] = target;
            a.token[place] = uint32_t(i);
            if (a.dloss) {
                const bool bad = target < 0 || target >= int64_t(a.v);
                if (bad && a.status) atomicCAS(a.status, 0, int(UZIP_ERR_INVALID_ARG));
                a.out_g[place] = bad ? NAN : a.dloss[i] * up;
                a.out_lse[place] = a.lse[i];
            }
        }
        if (mine) {
            if (a.place) a.place[i] = used ? place : ~0u;
            if (a.loss && !used) a.loss[i] = 0.f, a.zero_lse[i] = 0.f;
        }
        __syncthreads();
        if (listed + kPickThreads <= kPickList && start + kPickThreads < a.t) continue;
        // four rows at once, 256 threads to each: pieces of 16 bytes, or single values where rows start anywhere
        const bool vec = a.ldh % 8 == 0 && a.d % 8 == 0 && reinterpret_cast<uintptr_t>(a.h) % 16 == 0;
        const uint64_t pieces = vec ? a.d / 8 : a.d;
        for (uint32_t k = threadIdx.x / 256; k < listed; k += kPickThreads / 256) {
            const uint16_t* from = static_cast<const uint16_t*>(a.h) + list[k][0] * a.ldh;
            uint16_t* to = static_cast<uint16_t*>(a.out_h) + list[k][1] * a.ld_out;
            if (vec) {
#pragma unroll 4
                for (uint64_t c = threadIdx.x % 256; c < pieces; c += 256)
                    reinterpret_cast<uint4*>(to)[c] = reinterpret_cast<const uint4*>(from)[c];
            } else {
#pragma unroll 8
                for (uint64_t c = threadIdx.x % 256; c < pieces; c += 256) to[c] = from[c];
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) listed = 0;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.count = base;
}

// A warp for each row.
__global__ void __launch_bounds__(kThreads) spread_rows_kernel(const uint16_t* from, uint64_t ld, const uint32_t* place,
                                                               uint16_t* to, uint64_t ld_to, uint64_t rows, uint64_t cols, bool vec) {
    wait_for_launch_before();
    const uint32_t lane = threadIdx.x % 32;
    for (uint64_t r = blockIdx.x * uint64_t(kThreads / 32) + threadIdx.x / 32; r < rows; r += uint64_t(gridDim.x) * (kThreads / 32)) {
        const uint32_t at = place[r];
        const uint16_t* src = from + uint64_t(at) * ld;
        uint16_t* dst = to + r * ld_to;
        const uint64_t whole = vec ? cols / 8 : 0;
#pragma unroll 4
        for (uint64_t c = lane; c < whole; c += 32)
            reinterpret_cast<uint4*>(dst)[c] = at == ~0u ? make_uint4(0, 0, 0, 0) : reinterpret_cast<const uint4*>(src)[c];
#pragma unroll 4
        for (uint64_t c = 8 * whole + lane; c < cols; c += 32) dst[c] = at == ~0u ? uint16_t(0) : src[c];
    }
}

}  // namespace

cudaError_t launch_pack(const PackJobs& jobs, cudaStream_t s) {
    uint64_t most = 0;
    for (uint32_t i = 0; i < jobs.count; ++i)
        most = std::max(most, jobs.job[i].ld_to / 8 * jobs.job[i].rows * jobs.job[i].groups);
    if (most == 0) return cudaSuccess;
    return launch_after(pack_kernel, dim3(blocks_for(most, kSms * 32), jobs.count), kThreads, s, jobs);
}

cudaError_t launch_clear(void* p, uint64_t ld, uint64_t rows, uint64_t cols, cudaStream_t s) {
    const uint64_t total = rows * cols;
    if (total == 0) return cudaSuccess;
    return launch_after(clear_kernel, blocks_for(total, kSms * 32), kThreads, s, static_cast<uint16_t*>(p), ld, cols, total);
}

// Eight blocks for each SM, a share of at least 64 rows: a block takes 64 rows
// in about 2 us (777 x 1237 in 12 shares: 5.9 us, in 3: 15.1), and a second
// kernel joins the shares.  Experts have rows unevenly: there a share is eight
// rows of the mean.
uint32_t act_grad_splits(uint64_t m, uint64_t n, uint64_t groups) {
    const uint64_t have = (n + kGradCols - 1) / kGradCols * groups;
    const uint64_t want = std::max<uint64_t>(1, kSms * 8 / std::max<uint64_t>(1, have));
    return uint32_t(std::max<uint64_t>(1, std::min(want, m / groups / (groups > 1 ? 8 : 64))));
}

cudaError_t launch_act_grad(const ActGrad& a, cudaStream_t s) {
    if (a.n == 0) return cudaSuccess;
    const dim3 grid(uint32_t((a.n + kGradCols - 1) / kGradCols), a.splits, a.groups);
    const bool vec = a.n % 8 == 0 && a.lddy % 8 == 0 && reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 &&
                     (a.act == UZIP_ACT_NONE || (a.ldz % 8 == 0 && reinterpret_cast<uintptr_t>(a.z) % 16 == 0));
    cudaError_t err = launch_after(vec ? act_grad_kernel<true> : act_grad_kernel<false>, grid, kThreads, s, a);
    if (err == cudaSuccess && a.db && a.splits > 1) {
        const uint64_t total = uint64_t(a.groups) * a.n;
        err = launch_after(join_columns_kernel, uint32_t((total + kThreads - 1) / kThreads), kThreads, s, a.part, a.splits, a.n, total,
                           static_cast<uint16_t*>(a.db), a.dtype);
    }
    return err;
}

cudaError_t launch_offset_check(const int64_t* offsets, uint64_t groups, uint64_t m, int32_t* status, cudaStream_t s) {
    if (!status) return cudaSuccess;
    return launch_after(offset_check_kernel, 1, kThreads, s, offsets, uint32_t(groups), m, status);
}

cudaError_t launch_loss_join(const LossEpilogue& e, const uint32_t* token, const uint32_t* count, uint64_t t, uint64_t v,
                             float* loss, float* lse, int32_t* status, cudaStream_t s) {
    return launch_after(loss_join_kernel, uint32_t(t), kJoinThreads, s, e, token, count, v, e.tiles, loss, lse, status);
}

cudaError_t launch_loss_rows(const LossRows& a, cudaStream_t s) {
    return launch_after(loss_rows_kernel, uint32_t(std::min<uint64_t>(a.t, 2 * kSms)), kPickThreads, s, a);
}

cudaError_t launch_spread_rows(const void* from, uint64_t ld, const uint32_t* place, void* to, uint64_t ld_to, uint64_t rows,
                               uint64_t cols, cudaStream_t s) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    const bool vec = ld_to % 8 == 0 && reinterpret_cast<uintptr_t>(to) % 16 == 0;
    return launch_after(spread_rows_kernel, uint32_t(std::min<uint64_t>((rows + 7) / 8, kSms * 8)), kThreads, s,
                        static_cast<const uint16_t*>(from), ld, place, static_cast<uint16_t*>(to), ld_to, rows, cols, vec);
}

}  // namespace uzip
