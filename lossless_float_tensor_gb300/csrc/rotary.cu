// Rotary positions: y_a = s (x_a cos - x_b sin), y_b = s (x_a sin + x_b cos) for the
// pairs (a, b) of each head, by the angle position * frequency; backward is the
// opposite angle.  Each value is read and written once, so memory bounds it: 8192
// tokens with 32 + 8 + 8 heads of 128 into pages 35 us, 5.8 TB/s of 6.8 that a copy
// reaches; 8191 tokens with 32 heads of 96, 48 values turned: 20.6 us, 4.9 TB/s.
//
// Angles are kept in turns, as 64-bit fractions: position * frequency is one
// integer product modulo 2^64, which is the reduction modulo a full turn, exact
// for any position (the frequency's fraction is cut to 2^-64, so an angle is off by
// less than 2^-62 of a turn for each position); its upper 32 bits go to sincospi in
// 32 bits.  (In 32-bit
// floating point an angle of 10^6 radians would be off by 0.03.)
//
// A warp takes a token and a share of its heads: the cosines and sines of a token
// are computed once a warp, exchanged through shared memory, and kept in
// registers for all of its heads.  Two heads are in flight in a lane (four: 37.3 and
// 46 us for the two above; eight warps a block instead of four: 39.7 and 55).
#include <algorithm>

#include "cache.cuh"

namespace uzip {
namespace {

constexpr uint32_t kWarps = 4, kThreads = kWarps * 32;
constexpr int kAhead = 2;  // heads whose values are in flight in a lane

// Radians per position as a fraction of a turn, modulo 1, in units of 2^-64: the
// 53 bits of the number times 2^66 / (2 pi) in integers, shifted to its exponent
// (fp64 instructions are slow here).
__device__ __forceinline__ uint64_t turns_of(double radians) {
    constexpr uint64_t kPerTurn = 0xA2F9836E4E44152Aull;  // 2^66 / (2 pi)
    const uint64_t bits = uint64_t(__double_as_longlong(radians));
    const int e = int(bits >> 52 & 0x7FF);
    const uint64_t m = (bits & ((1ull << 52) - 1)) | (e ? 1ull << 52 : 0);
    const uint64_t hi = __umul64hi(m, kPerTurn), lo = m * kPerTurn;
    const int right = 1075 + 2 - max(e, 1);  // radians = m 2^(e - 1075)
    uint64_t t = 0;
    if (right >= 128 || right <= -64)
        t = 0;
    else if (right >= 64)
        t = hi >> (right - 64);
    else if (right > 0)
        t = hi << (64 - right) | lo >> right;
    else
        t = lo << -right;
    return bits >> 63 ? 0 - t : t;
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
    uint32_t w[V > 1 ? V / 2 : 1];
};

template <bool BF>
__device__ __forceinline__ float2 two(uint32_t w) {
    if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF>
__device__ __forceinline__ uint32_t rounded(float lo, float hi) {
    if constexpr (BF) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&b);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Turns the pairs that two pieces hold; pairs from `live` on stay as they are.
template <int V, bool INTER, bool BF>
__device__ __forceinline__ void turn(Values<V>& x, Values<V>& y, const float2 (&t)[V], int live) {
    if constexpr (V == 1) {
        if (live < 1) return;
        const float u = two<BF>(x.v[0]).x, w = two<BF>(y.v[0]).x;
        const uint32_t r = rounded<BF>(u * t[0].x - w * t[0].y, u * t[0].y + w * t[0].x);
        x.v[0] = uint16_t(r), y.v[0] = uint16_t(r >> 16);
    } else if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i >= live) continue;
            uint32_t& word = i < V / 2 ? x.w[i] : y.w[i - V / 2];
            const float2 f = two<BF>(word);
            word = rounded<BF>(f.x * t[i].x - f.y * t[i].y, f.x * t[i].y + f.y * t[i].x);
        }
    } else {
        if (live < V) return;  // pieces are turned as a whole
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 u = two<BF>(x.w[i / 2]), w = two<BF>(y.w[i / 2]);
            x.w[i / 2] = rounded<BF>(u.x * t[i].x - w.x * t[i].y, u.y * t[i + 1].x - w.y * t[i + 1].y);
            y.w[i / 2] = rounded<BF>(u.x * t[i].y + w.x * t[i].x, u.y * t[i + 1].y + w.y * t[i + 1].x);
        }
    }
}

// An item is two pieces of V neighbouring values of a head with the V pairs
// that they hold: V j.. and half + V j.. (halves), or 2 V j.. and 2 V j + V..
// (interleaved); behind the rotated part, two neighbouring pieces.
template <int V, bool INTER, bool BF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Rotary a, int splits) {
    using Word = typename Piece<V>::T;
    extern __shared__ float2 shared_cs[];  // [warps][half]
    wait_for_launch_before();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint64_t job = blockIdx.x * uint64_t(kWarps) + warp;
    if (job >= uint64_t(a.t) * splits) return;
    const int64_t token = job / splits;
    const int share = int(job - token * splits);
    const uint64_t pos = uint64_t(a.positions[token]);
    const int64_t slot = a.slots ? a.slots[token] : -1;
    float2* cs = shared_cs + warp * a.half;
    for (int j = lane; j < a.half; j += 32) {
        const uint64_t turns = pos * turns_of(a.freqs[j]);
        float s, c;
        sincospif(float(int32_t((turns + 0x80000000ull) >> 32)) * 0x1p-31f, &s, &c);
        cs[j] = make_float2(c * a.scale, s * a.scale * a.sign);
    }
    int64_t page = -1, off = 0;
    if (slot >= 0 && slot < a.slot_count) {
        page = slot / a.page, off = slot - page * a.page;
    } else if (slot != -1 && a.status && lane == 0) {
        *a.status = UZIP_ERR_INVALID_ARG;
    }
    __syncwarp();
    const int turned_items = INTER ? 0 : a.half / V;  // halves: rotated items first
    const int items = INTER ? (a.d + 2 * V - 1) / (2 * V) : turned_items + (a.d - 2 * a.half + 2 * V - 1) / (2 * V);
    const int across = max(1, 32 / items), lanes = min(items, 32);  // heads that a warp takes at once
    if (lane >= across * lanes) return;                              // lanes that no whole head is left for
    const int first = share * across + lane / lanes, step = splits * across;
    for (int item = lane % lanes; item < items; item += 32) {
        const bool plain = !INTER && item >= turned_items;
        const int e0 = INTER ? 2 * V * item : plain ? 2 * a.half + 2 * V * (item - turned_items) : V * item;
        const int e1 = INTER || plain ? e0 + V : a.half + V * item;
        const bool both = e1 < a.d;
        const int live = plain ? 0 : min(V, a.half - V * item);
        float2 t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = i < live ? cs[V * item + i] : make_float2(1.f, 0.f);
        // kAhead heads are loaded before the first is stored (an output may be its input, so the compiler would not move
        // a load over a store)
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            const RotarySegment& g = a.seg[n];
            if (g.paged && page < 0) continue;
            const uint16_t* from = g.from + token * g.row + first * g.head;
            uint16_t* to = g.to + (g.paged ? page * g.to_row + off * g.to_token : token * g.to_row) + first * g.to_head;
            for (int head = first; head < g.heads; head += kAhead * step) {
                Values<V> x[kAhead], y[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (head + u * step >= g.heads) continue;
                    const uint16_t* at = from + u * step * g.head;
                    x[u].piece = *reinterpret_cast<const Word*>(at + e0);
                    if (both) y[u].piece = *reinterpret_cast<const Word*>(at + e1);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (head + u * step >= g.heads) continue;
                    if (g.turned) turn<V, INTER, BF>(x[u], y[u], t, live);
                    uint16_t* at = to + u * step * g.to_head;
                    *reinterpret_cast<Word*>(at + e0) = x[u].piece;
                    if (both) *reinterpret_cast<Word*>(at + e1) = y[u].piece;
                }
                from += kAhead * step * g.head, to += kAhead * step * g.to_head;
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
    const int64_t blocks = (r.t * splits + kWarps - 1) / kWarps;
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
