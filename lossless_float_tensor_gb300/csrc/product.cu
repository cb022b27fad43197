// C = A B^T with a fused epilogue, the plain way: 64 x 64 tiles of C per
// block, 4 x 4 values per thread, operands staged through shared memory and
// multiplied in 32 bits.
#include "product.cuh"

namespace uzip {
namespace {

constexpr uint32_t kTile = 64, kStep = 16;

__device__ __forceinline__ float load_value(const Operand& o, uint32_t g, uint64_t row, uint64_t depth, int dtype) {
    const uint64_t at = g * o.group + (o.depth_major ? row * o.ld + depth : depth * o.ld + row);
    return from16(static_cast<const uint16_t*>(o.p)[at], dtype);
}

__device__ __forceinline__ void store_value(const Product& p, uint32_t g, uint64_t row, uint64_t col, float acc) {
    const StoreEpilogue& e = p.st;
    if (e.alpha) acc *= *e.alpha;
    if (e.sum_in) acc += e.sum_in[row * e.ld_sum + col];
    if (e.bias) acc += from16(static_cast<const uint16_t*>(e.bias)[g * p.n + col], p.dtype);
    if (e.z) static_cast<uint16_t*>(e.z)[row * e.ldz + col] = to16(acc, p.dtype);
    acc = act_value(acc, e.act);
    if (e.residual) acc += from16(static_cast<const uint16_t*>(e.residual)[row * e.ldr + col], p.dtype);
    const uint64_t at = g * e.out_group + row * e.ldo + col;
    if (e.out_fp32) static_cast<float*>(e.out)[at] = acc;
    else static_cast<uint16_t*>(e.out)[at] = to16(acc, p.dtype);
}

__global__ void __launch_bounds__(256) product_kernel(const __grid_constant__ Product p) {
    __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1], sc[kTile][kTile + 1];
    const uint32_t tid = threadIdx.x, tx = tid % 16, ty = tid / 16, g = blockIdx.z;
    uint64_t row0 = uint64_t(blockIdx.y) * kTile, row_end = p.m, d0 = 0, d_end = p.depth;
    const uint64_t col0 = uint64_t(blockIdx.x) * kTile;
    if (p.schedule != kDense) {
        int64_t lo = p.offsets[g], hi = p.offsets[g + 1];
        const int64_t top = p.schedule == kRows ? p.m : p.depth;
        if (lo < 0 || hi > top || lo > hi) return;  // reported by the offset check
        if (p.schedule == kRows) {
            row0 += lo;
            row_end = hi;
        } else {
            d0 = lo;
            d_end = hi;
        }
    }
    if (row0 >= row_end) return;
    float acc[4][4] = {};
    for (uint64_t d = d0; d < d_end; d += kStep) {
        for (uint32_t i = tid; i < kTile * kStep; i += 256) {
            const uint32_t r = i / kStep, c = i % kStep;
            bool on = d + c < d_end;
            if (on && p.skip_depth) on = !((p.skip_depth[(d + c) / 64] >> ((d + c) % 64)) & 1);
            sa[c][r] = on && row0 + r < row_end ? load_value(p.a, p.schedule == kDepth ? 0 : 0, row0 + r, d + c, p.dtype) : 0.f;
            sb[c][r] = on && col0 + r < p.n ? load_value(p.b, p.schedule == kRows ? g : 0, col0 + r, d + c, p.dtype) : 0.f;
        }
        __syncthreads();
        for (uint32_t c = 0; c < kStep; ++c)
            for (uint32_t i = 0; i < 4; ++i)
                for (uint32_t j = 0; j < 4; ++j) acc[i][j] += sa[c][ty + 16 * i] * sb[c][tx + 16 * j];
        __syncthreads();
    }
    if (p.epilogue == kStore) {
        for (uint32_t i = 0; i < 4; ++i)
            for (uint32_t j = 0; j < 4; ++j) {
                const uint64_t r = row0 + ty + 16 * i, c = col0 + tx + 16 * j;
                if (r < row_end && c < p.n) store_value(p, g, r, c, acc[i][j]);
            }
        return;
    }
    if (p.epilogue == kLossGrad) {
        for (uint32_t i = 0; i < 4; ++i)
            for (uint32_t j = 0; j < 4; ++j) {
                const uint64_t r = row0 + ty + 16 * i, c = col0 + tx + 16 * j;
                if (r >= row_end || c >= p.n) continue;
                const float w = p.ls.g[r];
                float v = exp2f((acc[i][j] - p.ls.lse[r]) * kLog2e);
                if (p.ls.targets[r] == int64_t(p.ls.col0 + c)) v -= 1.f;
                static_cast<uint16_t*>(p.ls.out)[r * p.ls.ldo + c] = to16(w == 0.f ? 0.f : w * v, p.dtype);
            }
        return;
    }
    for (uint32_t i = 0; i < 4; ++i)
        for (uint32_t j = 0; j < 4; ++j) sc[ty + 16 * i][tx + 16 * j] = acc[i][j];
    __syncthreads();
    if (tid < kTile && row0 + tid < row_end) {
        const uint64_t r = row0 + tid;
        float top = -INFINITY, sum = 0.f;
        const uint32_t cols = p.n - col0 < kTile ? uint32_t(p.n - col0) : kTile;
        for (uint32_t c = 0; c < cols; ++c) top = fmaxf(top, sc[tid][c]);
        const float base = top == -INFINITY ? 0.f : top;
        for (uint32_t c = 0; c < cols; ++c) sum += exp2f((sc[tid][c] - base) * kLog2e);
        p.ls.part[blockIdx.x * p.m + r] = make_float2(top, sum);
        const int64_t t = p.ls.targets[r] - int64_t(p.ls.col0 + col0);
        if (t >= 0 && t < int64_t(cols)) p.ls.hit[r] = sc[tid][t];
    }
}

}  // namespace

uint32_t product_tile_columns(const Product&, int) { return kTile; }

cudaError_t launch_product(const Product& p, cudaStream_t s) {
    if (p.m == 0 || p.n == 0) return cudaSuccess;
    const dim3 grid(uint32_t((p.n + kTile - 1) / kTile), uint32_t((p.m + kTile - 1) / kTile), p.groups);
    product_kernel<<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace uzip
