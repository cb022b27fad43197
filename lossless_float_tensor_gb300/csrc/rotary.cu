// Rotary positions: y_a = s (x_a cos - x_b sin), y_b = s (x_a sin + x_b cos) for the
// pairs (a, b) of each head, by the angle position * frequency; backward is the
// opposite angle.  Each value is read and written once, so memory bounds it.
//
// Angles are kept in turns, as 64-bit fractions: position * frequency is one
// integer product modulo 2^64, which is the reduction modulo a full turn, exact
// for any position; its upper 32 bits go to sincospi in 32 bits.  (In 32-bit
// floating point an angle of 10^6 radians would be off by 0.03.)
//
// A warp takes a token and a share of its heads: the cosines and sines of a token
// are computed once a warp, exchanged through shared memory, and kept in
// registers for all of its heads.
#include <algorithm>

#include "cache.cuh"

namespace uzip {
namespace {

constexpr uint32_t kWarps = 4, kThreads = kWarps * 32;
constexpr int kAhead = 4;  // heads whose values are in flight in a lane

// Radians per position as a fraction of a turn, modulo 1, in units of 2^-64.
__device__ __forceinline__ uint64_t turns_of(double radians) {
    double t = radians * 0.15915494309189533577;
    t -= rint(t);
    return uint64_t(__double2ll_rn(t * 18446744073709551616.0));
}

template <int V>
struct Piece;  // V values of 16 bits
template <>
struct Piece<8> {
    using T = uint4;
};
template <>
struct Piece<2> {
    using T = uint32_t;
};
template <>
struct Piece<1> {
    using T = uint16_t;
};

template <int V>
union Values {
    typename Piece<V>::T piece;
    uint16_t v[V];
};

template <bool BF>
__device__ __forceinline__ float value(uint16_t v) {
    return BF ? __uint_as_float(uint32_t(v) << 16) : __half2float(__ushort_as_half(v));
}
template <bool BF>
__device__ __forceinline__ uint16_t rounded(float v) {
    return to16(v, BF ? UZIP_BF16 : UZIP_FP16);
}

template <bool BF>
__device__ __forceinline__ void turn(uint16_t& x, uint16_t& y, float2 cs) {
    const float u = value<BF>(x), w = value<BF>(y);
    x = rounded<BF>(u * cs.x - w * cs.y);
    y = rounded<BF>(u * cs.y + w * cs.x);
}

// An item is two pieces of V neighbouring values of a head with the V pairs
// that they hold: V j.. and half + V j.. (halves), or 2 V j.. and 2 V j + V..
// (interleaved); behind the rotated part, two neighbouring pieces.
template <int V, bool INTER, bool BF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Rotary a, int splits) {
    extern __shared__ float2 shared_cs[];  // [warps][half]
    wait_for_launch_before();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float2* cs = shared_cs + warp * a.half;
    const int turned_items = INTER ? 0 : a.half / V;  // halves: rotated items first
    const int items = INTER ? (a.d + 2 * V - 1) / (2 * V) : turned_items + (a.d - 2 * a.half + 2 * V - 1) / (2 * V);
    const int across = max(1, 32 / items);  // heads that a warp takes at once
    const uint64_t stride = uint64_t(gridDim.x) * kWarps;
    // frequencies of this lane's first pairs are kept; heads of more than 128 pairs convert the others again
    uint64_t freq[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) freq[k] = lane + 32 * k < a.half ? turns_of(a.freqs[lane + 32 * k]) : 0;
    for (uint64_t job = blockIdx.x * uint64_t(kWarps) + warp; job < uint64_t(a.t) * splits; job += stride) {
        const int64_t token = job / splits;
        const int share = int(job % splits);
        const uint64_t pos = uint64_t(a.positions[token]);
        __syncwarp();
        for (int k = 0; k * 32 < a.half; ++k) {
            const int j = k * 32 + lane;
            if (j >= a.half) break;
            const uint64_t f = k == 0 ? freq[0] : k == 1 ? freq[1] : k == 2 ? freq[2] : k == 3 ? freq[3] : turns_of(a.freqs[j]);
            float s, c;
            sincospif(float(int32_t((pos * f + 0x80000000ull) >> 32)) * 0x1p-31f, &s, &c);
            cs[j] = make_float2(c * a.scale, s * a.scale * a.sign);
        }
        __syncwarp();
        int64_t page = -1, off = 0;
        if (a.slots) {
            const int64_t slot = a.slots[token];
            if (slot >= 0 && slot < a.slot_count) {
                page = slot / a.page, off = slot - page * a.page;
            } else if (slot != -1 && a.status && lane == 0) {
                *a.status = UZIP_ERR_INVALID_ARG;
            }
        }
        for (int item = lane % min(items, 32); item < items; item += 32) {
            if (lane >= across * items) break;  // lanes that no whole head is left for
            const bool plain = !INTER && item >= turned_items;
            const int e0 = INTER ? 2 * V * item : plain ? 2 * a.half + 2 * V * (item - turned_items) : V * item;
            const int e1 = INTER || plain ? e0 + V : a.half + V * item;
            const bool both = e1 < a.d;
            const int pair0 = V * item;
            float2 t[V];
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] = !plain && pair0 + i < a.half ? cs[pair0 + i] : make_float2(1.f, 0.f);
            // heads of this warp's share, `across` of them at once; kAhead of those are loaded before the first is
            // stored (an output may be its input, so the compiler would not move a load over a store)
            const int step = splits * across;
            for (int head = share * across + lane / min(items, 32); head < a.heads; head += kAhead * step) {
                Values<V> x[kAhead], y[kAhead];
                uint16_t* to[kAhead];
                bool turned[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    int h = head + u * step, n = 0;
                    to[u] = nullptr;
                    if (h >= a.heads) continue;
                    if (h >= a.seg[0].heads) {
                        h -= a.seg[0].heads, n = 1;
                        if (h >= a.seg[1].heads) h -= a.seg[1].heads, n = 2;
                    }
                    const RotarySegment& g = a.seg[n];
                    if (g.paged && page < 0) continue;
                    turned[u] = g.turned;
                    to[u] = g.to + h * g.to_head + (g.paged ? page * g.to_row + off * g.to_token : token * g.to_row);
                    const uint16_t* from = g.from + token * g.row + h * g.head;
                    x[u].piece = *reinterpret_cast<const typename Piece<V>::T*>(from + e0);
                    if (both) y[u].piece = *reinterpret_cast<const typename Piece<V>::T*>(from + e1);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (!to[u]) continue;
                    if (turned[u] && !plain) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            if (pair0 + i >= a.half) continue;
                            if constexpr (!INTER || V == 1)
                                turn<BF>(x[u].v[i], y[u].v[i], t[i]);
                            else if (i < V / 2)
                                turn<BF>(x[u].v[(2 * i) % V], x[u].v[(2 * i + 1) % V], t[i]);
                            else
                                turn<BF>(y[u].v[(2 * i) % V], y[u].v[(2 * i + 1) % V], t[i]);
                        }
                    }
                    *reinterpret_cast<typename Piece<V>::T*>(to[u] + e0) = x[u].piece;
                    if (both) *reinterpret_cast<typename Piece<V>::T*>(to[u] + e1) = y[u].piece;
                }
            }
        }
    }
}

template <int V, bool INTER, bool BF>
cudaError_t launch_as(const Rotary& r, int sms, cudaStream_t s) {
    const int items = INTER ? (r.d + 2 * V - 1) / (2 * V) : r.half / V + (r.d - 2 * r.half + 2 * V - 1) / (2 * V);
    const int across = std::max(1, 32 / std::max(items, 1));
    const int most = (r.heads + across - 1) / across;  // warps that can share a token's heads
    // enough warps for every SM (16 each): few tokens have their heads split, down to one step of a warp
    const int64_t want = int64_t(sms) * 16;
    const int splits = int(std::max<int64_t>(1, std::min<int64_t>(most, want / std::max<int64_t>(1, r.t))));
    const int64_t blocks = std::min<int64_t>((r.t * splits + kWarps - 1) / kWarps, int64_t(sms) * 16);
    return launch_next(rotary_kernel<V, INTER, BF>, dim3(uint32_t(blocks)), kThreads, uint32_t(kWarps * std::max(1, r.half) * sizeof(float2)), 1,
                       s, r, splits);
}

template <int V>
cudaError_t launch_wide(const Rotary& r, int dtype, bool interleaved, int sms, cudaStream_t s) {
    if (dtype == UZIP_BF16)
        return interleaved ? launch_as<V, true, true>(r, sms, s) : launch_as<V, false, true>(r, sms, s);
    return interleaved ? launch_as<V, true, false>(r, sms, s) : launch_as<V, false, false>(r, sms, s);
}

}  // namespace

cudaError_t launch_rotary(const Rotary& r, int dtype, bool interleaved, int sms, cudaStream_t s) {
    // the widest pieces that every address, and the border of the rotated part, is a multiple of
    uint64_t all = 2 * uint64_t(r.d) | 2 * uint64_t(interleaved ? 2 * r.half : r.half);
    for (const RotarySegment& g : r.seg) {
        if (!g.heads) continue;
        all |= reinterpret_cast<uint64_t>(g.from) | reinterpret_cast<uint64_t>(g.to);
        all |= 2 * uint64_t(g.row) | 2 * uint64_t(g.head) | 2 * uint64_t(g.to_row) | 2 * uint64_t(g.to_head) | 2 * uint64_t(g.to_token);
    }
    if (all % 16 == 0) return launch_wide<8>(r, dtype, interleaved, sms, s);
    if (all % 4 == 0) return launch_wide<2>(r, dtype, interleaved, sms, s);
    return launch_wide<1>(r, dtype, interleaved, sms, s);
}

}  // namespace uzip
