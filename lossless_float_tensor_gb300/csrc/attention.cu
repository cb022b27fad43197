// Attention of one new token of each sequence over a paged cache.
//
// For a key head h, its query heads g = 0.. and the live tokens t of a sequence:
// z_gt = scale q_g . k_t, p = softmax over t, o_g = sum_t p_gt v_t, in one pass
// over the keys and values with a running maximum m and sum l:
//   m' = max(m, z), l' = l 2^(m - m') + 2^(z - m'), o' = o 2^(m - m') + 2^(z - m') v.
// Every key and value is read once for up to 32 query heads that share it (16 where
// heads have over 128 values), once more for each further 32.  A pair of them is 4
// bytes and 4 operations a query head, so 1 to 32 operations a byte: what bounds it is
// memory, and the work of a block is to keep enough of it in flight.  128 sequences of
// 1024 to 12288 tokens, 8 x 4 heads of 128 in bf16: 519 to 533 us, 6.6 to 6.7 TB/s of
// 6.79 that a copy reaches; 131072 tokens of one sequence: 88.7 us, 6.1 TB/s, 8 us of it
// start, end and joining.  The products still need matrix instructions (8 query heads
// would take 54 TFLOP/s of plain ones); they run transposed, tokens or head values as
// the rows and query heads as the 8 columns, so that heads that do not exist cost no
// rows: S^T = K Q^T and O^T = V^T P^T by m16n8k16, which keeps the tensor pipe busy 9 %
// of the time.  tcgen05's rows of 128 tokens would want the tokens of eight tiles in one
// step, two from each of four warps, with the barriers between them that this layout
// does without.
//
// A warp takes tiles of 16 tokens, has a ring of shared memory of its own for
// them (cp.async, 16 bytes a lane, rows 16 bytes apart from a multiple of 128 so
// that ldmatrix finds no bank twice), and running sums of its own: no barrier but
// where a sequence's part ends and the four warps' sums are joined.  A lane each
// looks its token's page up, so pages may end anywhere in a tile.  (One bulk copy a
// row instead, 256 bytes: 663 us for the 128 sequences.)  Rows behind the last
// token are filled with zeros and never read, so what they hold says nothing.
//
// The tokens of all sequences and heads, in tiles, are cut into one equal piece
// for each block, found by every block from the lengths on the device (1.1 us).  A
// row (a sequence's tokens for one head) counts kRowCost tiles more than it has, for
// its queries and its end, so that a block of many short rows has no more to do.
// Where a border falls inside a row the sums go to the workspace and a second launch
// joins them, in the order of the tokens: the same bits each time.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cache.cuh"

namespace uzip {
namespace {

constexpr uint32_t kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 16;  // tokens of a tile: the rows of one matrix instruction

template <int DP, int NT>
struct Shape {
    static constexpr uint32_t kPitch = DP * 2 + 16;         // bytes from token to token
    static constexpr uint32_t kStage = 2 * kTile * kPitch;  // keys, then values
    // blocks on an SM, with the stages that fit: 64 sequences of 16 to 4096 tokens, d = 128, take 92.0 us on three of
    // two stages, 102.6 on two of three.  Where 32 query heads' sums take the registers: two; of up to 64 values they
    // are left three, with 28 words spilled (two blocks there: not measured)
    static constexpr uint32_t kBlocks = NT == 4 && DP > 64 ? 2 : DP <= 128 ? 3 : DP <= 192 ? 2 : 1;
    // queries: in registers up to 32 of them a lane, else in shared memory, read again for each tile (64 sequences of
    // 2000 to 6000 tokens, 4 x 16 heads of 256: 221 us with spilled registers, 181)
    static constexpr bool kShared = NT * DP > 256;
    static constexpr uint32_t kQueries = kShared ? 8 * NT * kPitch : 0;
    static constexpr uint32_t kRoom = 227 * 1024 / kBlocks - 2560 - kQueries;  // 1 KB a block is the system's, 1.4 static
    static constexpr uint32_t kMost = kRoom / (kWarps * kStage);
    static constexpr uint32_t kStages = kMost < 8 ? kMost : 8;
    static constexpr uint32_t kSmem = kWarps * kStages * kStage + kQueries;
    static_assert(kStages >= 2, "one to use, one to fetch into");
};

// 16 bytes into shared memory; 16 zeros where not `there`
__device__ __forceinline__ void fetch16(uint32_t to, uint64_t from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void fetch16(uint32_t to, uint64_t from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void fetch_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void load4(uint32_t r[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void load4_turned(uint32_t r[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ uint32_t turned8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <bool BF>
__device__ __forceinline__ void multiply(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return to16x2(lo, hi, BF ? UZIP_BF16 : UZIP_FP16);
}
// Weights are held times 2^kLift: in fp16 the largest is 2^15, so that those down to 2^-29
// of it are normal numbers and those down to 2^-39 are there (from 1 on, fp16 would lose
// digits at 2^-14 and all at 2^-25, which is what a result consists of where one token
// takes nearly all of the weight and its value is 0).  Sums and parts hold the factor too.
template <bool BF>
constexpr float kLift = BF ? 0.f : 15.f;
// Live tokens [lo, len) of sequence i and its tiles; a sequence without tokens
// has one tile of none, and so has one whose length cannot be (bad).
struct Live {
    int lo, len, tiles;
    bool bad;
};
__device__ __forceinline__ Live live_of(const Attention& a, int i) {
    int n = a.lengths[i];
    Live s;
    s.bad = n < 0 || n > a.most;
    if (s.bad) n = 0;
    s.len = n;
    s.lo = a.window && n > a.window ? n - a.window : 0;
    s.tiles = max(1, int((uint32_t(n - s.lo) + kTile - 1) / kTile));
    return s;
}

// cap tanh(u) by powers of 2, u = score / cap, with the score and the cap times log2 e.
// From |u| = 1/2 on by the exponential, 1 - 2 / (exp(2 |u|) + 1).  Below, that would
// subtract two numbers near 1 and leave an error that goes by the cap (of 10^6: 0.1 of
// a score of 2), so there the score times tanh(u) / u = 1 + w P(w), w = u u: P of degree
// 3, fitted to 1.5e-8 of the result over w to 1/4.  Either is off by less than 2^-20 of
// itself, and a cap far above a score (u may underflow) leaves the score as it is.
__device__ __forceinline__ float capped(float score, float u, float cap) {
    constexpr float kTwoLog2e = 2.8853900817779268f;
    const float w = u * u;
    float p = fmaf(0.01724148f, w, -0.05304549f);
    p = fmaf(p, w, 0.13325879f);
    p = fmaf(p, w, -0.33333144f);
    const float far = fmaf(-2.f * fast_reciprocal(fast_exp2(fabsf(u) * kTwoLog2e) + 1.f), cap, cap);
    return fabsf(u) < 0.5f ? fmaf(score * w, p, score) : copysignf(far, u);
}

// What a row costs beside its tiles, in tiles.  24 sequences of 0 to 6000 tokens in
// windows of 1024, 16 heads: 51.6 us with 0, 28.2 with 4, 23.6 with 8, 23.9 with 14.
constexpr int kRowCost = 8;
// What a block has at least, where rows are cut: over kRowCost, so that it has a
// tile.  37 sequences of 0 to 2777 tokens, 3 heads: 16.8 us with 16, 18.2 with 32.
constexpr int kLeast = 16;
static_assert(kLeast > kRowCost, "");

// Tiles that a block adds up in one go.  The matrix instructions cut their 32-bit
// additions toward zero, so a sum of one sign falls short by 6e-9 of itself for each
// token of a warp (524288 tokens, a row for each block: results off by 8e-4, nearly
// two of fp16's roundings); after 8192 tokens a warp (5e-5) a block's sums are
// joined and rounded to nearest, as at a part's end.
constexpr int kChunk = 2048;
static_assert(kChunk % kWarps == 0, "a warp's tiles are the same whether a part is taken in chunks or not");

// Where a warp is: tiles [j0, j1) of row `row` of sequence i, and its tile of
// them.  `left` counts what the block has from the row's beginning on, kRowCost
// before the first tile (whole rows: unused).
struct Place {
    int i, row, j0, j1, tile, head;
    int64_t left, begin;  // begin: where the row begins among all costs
    const int32_t* pages;  // the sequence's row of the table
    Live s;
    __device__ __forceinline__ void enter(const Attention& a) {
        head = a.blocks == 1 ? row : row / a.blocks;
        pages = a.table + i * a.ldt;
    }
};

// The next part of the block's work; false at its end.
__device__ __forceinline__ bool next_part(const Attention& a, Place& p) {
    if (a.cut) {
        p.left -= kRowCost + p.s.tiles, p.begin += kRowCost + p.s.tiles;
        if (p.left <= kRowCost) return false;
        if (++p.row == a.pairs) {
            p.row = 0;
            p.s = live_of(a, ++p.i);
        }
    } else {  // whole rows, one for each block in turn
        p.row += a.skip_row;
        int i = p.i + a.skip_seq;
        if (p.row >= a.pairs) p.row -= a.pairs, ++i;
        if (i >= a.seqs) return false;
        if (i != p.i) p.s = live_of(a, i);
        p.i = i;
    }
    p.j0 = 0;
    p.j1 = a.cut ? int(min(int64_t(p.s.tiles), p.left - kRowCost)) : p.s.tiles;
    p.enter(a);
    return true;
}

// The first part of this block's work, and the record of the border before it.
// Costs are counted through all sequences; block b has those from b * total /
// blocks on.  Returns false if there is none.
__device__ bool first_part(const Attention& a, Place& p, int64_t& total, int64_t& blocks) {
    if (!a.cut) {
        const int64_t at = blockIdx.x;
        if (at >= int64_t(a.seqs) * a.pairs) return false;
        p.i = int(at / a.pairs), p.row = int(at - int64_t(p.i) * a.pairs);
        p.s = live_of(a, p.i);
        p.j0 = 0, p.j1 = p.s.tiles;
        p.enter(a);
        return true;
    }
    __shared__ int64_t sums[kWarps];
    __shared__ int64_t found[2];  // sequence, tiles before it
    const int each = (a.seqs + int(kThreads) - 1) / int(kThreads);
    const int from = min(a.seqs, int(threadIdx.x) * each), to = min(a.seqs, from + each);
    int64_t mine = 0;
    for (int i = from; i < to; ++i) mine += kRowCost + live_of(a, i).tiles;
    int64_t sum = mine;
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t got = __shfl_up_sync(~0u, sum, o);
        if (lane >= uint32_t(o)) sum += got;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    int64_t before = sum - mine;
    total = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    total *= a.pairs;
    before *= a.pairs;
    blocks = min(int64_t(gridDim.x), max(int64_t(1), total / kLeast));
    const int64_t b = blockIdx.x;
    if (b >= blocks) {
        if (threadIdx.x == 0) a.record[b] = make_int4(-1, 0, 0, 0);
        return false;
    }
    const int64_t begin = b * total / blocks, end = (b + 1) * total / blocks;
    if (begin >= before && begin < before + mine * a.pairs) {  // one thread's sequences hold the beginning
        for (int i = from; i < to; ++i) {
            const int64_t n = int64_t(kRowCost + live_of(a, i).tiles) * a.pairs;
            if (begin < before + n) {
                found[0] = i, found[1] = before;
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    p.i = int(found[0]);
    p.s = live_of(a, p.i);
    const int64_t in = begin - found[1];
    const int span = kRowCost + p.s.tiles;
    p.row = int(in / span);
    const int in_row = int(in - int64_t(p.row) * span);
    p.j0 = max(0, in_row - kRowCost);
    p.left = end - begin + in_row, p.begin = begin - in_row;
    p.j1 = int(min(int64_t(p.s.tiles), p.left - kRowCost));
    p.enter(a);
    if (threadIdx.x == 0) {
        // the first border behind a row's first tile is the one that has its joining done
        const int64_t tile0 = p.begin + kRowCost, row_end = tile0 + p.s.tiles;
        const bool first = p.j0 > 0 && (b - 1) * total / blocks <= tile0;
        a.record[b] = first ? make_int4(p.i, p.row, int(b - 1), int((row_end * blocks - 1) / total)) : make_int4(-1, 0, 0, 0);
    }
    return true;
}

// 2^(z - m) for z <= m: 0 for a score of -inf, also where there is none above it; what is no number stays so.
__device__ __forceinline__ float weight(float z, float m) { return z == -INFINITY ? 0.f : fast_exp2(z - m); }

template <int DP, int NT, bool BF>
__global__ void __launch_bounds__(kThreads, (Shape<DP, NT>::kBlocks)) attention_kernel(const __grid_constant__ Attention a) {
    using S = Shape<DP, NT>;
    constexpr int kSteps = DP / 16;
    constexpr int kStages = int(S::kStages);
    constexpr int kHeads = 8 * NT;
    constexpr int kOut = DP + 4;  // floats from head to head of a warp's sums in shared memory
    constexpr int kRound = NT < 2 ? NT : 2;  // of 8 heads: those whose sums fit one stage
    static_assert(kRound * 8 * kOut * 4 <= int(S::kStage), "a warp's sums fit one stage");
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float2 stat[kWarps + 1][kHeads];  // the warps' maxima and sums, and those of the part's chunks before
    __shared__ uint32_t where[kWarps];
    wait_for_launch_before();

    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t mine = smem_u32(ring) + warp * kStages * S::kStage;
    uint8_t* const queries = ring + kWarps * kStages * S::kStage;
    const uint32_t q_at = smem_u32(queries) + (lane / 16 * 8 + lane % 8) * S::kPitch + lane / 8 % 2 * 16;
    Place ahead;
    int64_t total = 0, blocks = 0;
    if (!first_part(a, ahead, total, blocks)) return;  // the whole block
    Place at = ahead;
    int chunk = at.j0;  // where the part's next tiles to be added up begin
    bool more = true;  // `ahead` is at a tile (or at the end)
    ahead.tile = ahead.j0 + warp;
    auto settle = [&] {
        while (more && ahead.tile >= ahead.j1) {
            more = next_part(a, ahead);
            ahead.tile = ahead.j0 + warp;
        }
    };
    // A tile to fetch: lane l (and l + 16) has token l's page and its place there.
    struct Row {
        int page, off, head, count;  // count: live tokens (the same in all lanes)
    };
    auto row_of = [&]() -> Row {
        Row r{0, 0, 0, 0};
        if (!more) return r;
        const int t0 = ahead.s.lo + ahead.tile * kTile, t = t0 + lane % kTile;
        r.count = min(kTile, ahead.s.len - t0);
        r.head = ahead.head;
        if (lane % kTile < r.count) {
            const uint32_t col = uint32_t(uint64_t(uint32_t(t)) * a.page_by >> a.page_shift);
            r.page = ahead.pages[col];
            r.off = t - int(col) * a.page;
        }
        return r;
    };
    uint32_t poison = 0;  // stages whose tile has a page that does not exist
    // A row's 16-byte pieces lie with neighbouring lanes, as many rows at once as fit a warp.  A lane's place in keys and
    // values differs by a constant where their strides are the same, so one shuffle finds both.  Columns behind d are zeros.
    constexpr int kChunks = DP / 8, kRows = kChunks < 32 ? 32 / kChunks : 1;
    const int col = lane % kChunks * 16, first_row = lane / kChunks;
    const bool col_in = col < 2 * a.d;
    const uint64_t keys_from = reinterpret_cast<uint64_t>(a.k) + (col_in ? col : 0), values_from = reinterpret_cast<uint64_t>(a.v) + (col_in ? col : 0);
    const uint32_t col_to = mine + first_row * S::kPitch + col;
    auto fetch = [&](const Row& r, int stage) {
        const bool in = lane % kTile < r.count;
        int live = r.count;
        poison &= ~(1u << stage);
        if (__any_sync(~0u, in && uint32_t(r.page) >= uint32_t(a.pages))) {
            poison |= 1u << stage;
            if (a.status && lane == 0) *a.status = UZIP_ERR_INVALID_ARG;
            live = 0;
        }
        // bytes from the pool's first value; rows that are not there: its first row, of which nothing is read
        auto place = [&](const PoolStrides& st) -> uint64_t {
            return lane % kTile < live ? uint32_t(r.page) * st.page + uint32_t(r.head) * st.head + uint32_t(r.off) * st.token : 0;
        };
        const uint64_t k_off = place(a.ks);
        const uint32_t to = col_to + stage * S::kStage;
        if (live == kTile && a.alike) {
            if (kRows * kChunks == 32 && a.d == DP) {
#pragma unroll
                for (int n = 0; n < kTile; n += kRows) {
                    const uint64_t off = __shfl_sync(~0u, k_off, n + first_row);
                    fetch16(to + n * S::kPitch, keys_from + off);
                    fetch16(to + (kTile + n) * S::kPitch, values_from + off);
                }
            } else {
#pragma unroll
                for (int n = 0; n < kTile; n += kRows) {
                    const uint64_t off = __shfl_sync(~0u, k_off, n + first_row);
                    if (first_row < kRows) {
                        fetch16(to + n * S::kPitch, keys_from + off, col_in);
                        fetch16(to + (kTile + n) * S::kPitch, values_from + off, col_in);
                    }
                }
            }
        } else {
            const uint64_t v_off = place(a.vs);
#pragma unroll 2
            for (int n = 0; n < kTile; n += kRows) {
                const int row = n + first_row;
                const uint64_t ko = __shfl_sync(~0u, k_off, row), vo = __shfl_sync(~0u, v_off, row);
                if (first_row < kRows) {
                    fetch16(to + n * S::kPitch, keys_from + ko, row < live && col_in);
                    fetch16(to + (kTile + n) * S::kPitch, values_from + vo, row < live && col_in);
                }
            }
        }
    };

    // the first stages; their pages are looked up together
    settle();
    {
        Row r[kStages - 1];
        bool real[kStages - 1];
#pragma unroll
        for (int n = 0; n < kStages - 1; ++n) {
            real[n] = more;
            r[n] = row_of();
            ahead.tile += kWarps;
            settle();
        }
#pragma unroll
        for (int n = 0; n < kStages - 1; ++n) {
            if (real[n]) fetch(r[n], n);
            fetch_end();
        }
    }
    Row row = row_of();
    int stage = 0, refill = kStages - 1;  // stage to use next, stage to fetch into next: the free one

    do {
        const int blk = at.row % a.blocks, head0 = at.row / a.blocks * a.group + blk * kHeads;
        const int heads = min(kHeads, a.group - blk * kHeads);
        // two neighbouring values of a query; zeros where there is no head or column
        auto query = [&](int h, int col) -> uint32_t {
            if (h >= heads || col >= a.d) return 0;
            const uint16_t* at_q = a.q + at.i * a.q_row + int64_t(head0 + h) * a.q_head + col;
            return a.q_pairs ? *reinterpret_cast<const uint32_t*>(at_q) : at_q[0] | uint32_t(at_q[1]) << 16;
        };
        uint32_t q[S::kShared ? 1 : NT][S::kShared ? 1 : kSteps][2];
        if constexpr (S::kShared) {
            for (int x = threadIdx.x; x < kHeads * DP / 2; x += kThreads) {
                const int h = x / (DP / 2), col = x % (DP / 2) * 2;
                *reinterpret_cast<uint32_t*>(queries + h * S::kPitch + col * 2) = query(h, col);
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
                    for (int e = 0; e < 2; ++e) q[nt][ks][e] = query(nt * 8 + lane / 4, ks * 16 + e * 8 + lane % 4 * 2);
        }
        float o[NT][kSteps][4] = {};
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
        bool broken = at.s.bad;
        if (broken && a.status && threadIdx.x == 0) *a.status = UZIP_ERR_INVALID_ARG;

        const int stop = min(at.j1, chunk + kChunk);
        for (at.tile = chunk + warp; at.tile < stop; at.tile += kWarps) {
            fetch_wait<kStages - 2>();
            __syncwarp();
            if (more) {
                fetch(row, refill);
                ahead.tile += kWarps;
                settle();
                row = row_of();
            }
            fetch_end();
            const uint32_t keys = mine + stage * S::kStage, values = keys + kTile * S::kPitch;
            const int count = at.s.len - at.s.lo - at.tile * kTile;  // live tokens of the tile, if fewer than 16
            broken |= poison >> stage & 1;
            refill = stage;
            stage = stage + 1 == kStages ? 0 : stage + 1;

            // two chains of sums, where there are few heads: half the wait for each product's result
            constexpr int kChains = NT < 4 ? 2 : 1;
            float z[NT][4] = {}, z2[kChains == 2 ? NT : 1][4] = {};
            const uint32_t k_at = keys + lane % 16 * S::kPitch + lane / 16 * 16;
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                uint32_t f[4];
                load4(f, k_at + ks * 32);
                if constexpr (S::kShared) {
#pragma unroll
                    for (int nt = 0; nt < NT; nt += 2) {
                        uint32_t b[4];
                        load4(b, q_at + nt * 8 * S::kPitch + ks * 32);
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            multiply<BF>(kChains == 2 && ks % 2 ? z2[(nt + c) % (kChains == 2 ? NT : 1)] : z[nt + c], f, b[2 * c], b[2 * c + 1]);
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        multiply<BF>(kChains == 2 && ks % 2 ? z2[nt % (kChains == 2 ? NT : 1)] : z[nt], f, q[nt][ks][0], q[nt][ks][1]);
                }
            }
            uint32_t p[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float product = kChains == 2 ? z[nt][e] + z2[nt % (kChains == 2 ? NT : 1)][e] : z[nt][e];
                    z[nt][e] = a.cap > 0 ? capped(product * a.scale, product * a.per_cap, a.cap) : product * a.scale;
                }
                if (count < kTile) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (lane / 4 + e / 2 * 8 >= count) z[nt][e] = -INFINITY;
                }
                float top[2] = {fmaxf(z[nt][0], z[nt][2]), fmaxf(z[nt][1], z[nt][3])};
                // most tiles hold no new maximum and need one vote.  It follows at once, so that the largest weight is 1 and
                // loses nothing: letting it lag by 2^8 is no faster and leaves 1.3 times the result's own rounding, not 1.07
                if (__any_sync(~0u, top[0] > m[nt][0] || top[1] > m[nt][1])) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int x = 4; x < 32; x *= 2) top[c] = fmaxf(top[c], __shfl_xor_sync(~0u, top[c], x));
                        const float now = fmaxf(m[nt][c], top[c]), by = weight(m[nt][c], now);
                        m[nt][c] = now;
                        l[nt][c] *= by;
#pragma unroll
                        for (int ks = 0; ks < kSteps; ++ks) o[nt][ks][c] *= by, o[nt][ks][c + 2] *= by;
                    }
                }
                // nothing but -inf so far: weights of 0, by any other maximum
                const float from[2] = {m[nt][0] == -INFINITY ? 0.f : m[nt][0], m[nt][1] == -INFINITY ? 0.f : m[nt][1]};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[nt][e] = fast_exp2(BF ? z[nt][e] - from[e % 2] : z[nt][e] - from[e % 2] + kLift<BF>);
                    l[nt][e % 2] += z[nt][e];
                }
                // rounded to the values' type for the second product, each by half a step of itself at most; the sum l keeps
                // them unrounded.  Where they differ the errors add up, at random, to less than the one rounding of the
                // result; equal weights are off alike, which may be as much as that rounding and no more
                p[nt][0] = turned8x8(pack2<BF>(z[nt][0], z[nt][1]));
                p[nt][1] = turned8x8(pack2<BF>(z[nt][2], z[nt][3]));
            }
            const uint32_t v_at = values + (lane % 8 + lane / 16 * 8) * S::kPitch + lane / 8 % 2 * 16;
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                uint32_t f[4];
                load4_turned(f, v_at + ks * 32);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) multiply<BF>(o[nt][ks], f, p[nt][0], p[nt][1]);
            }
            __syncwarp();
        }

        // the four warps' sums, each in the warp's own free stage, and their maxima; 16 heads at a time
        const bool whole = at.j0 == 0 && at.j1 == at.s.tiles;
        const int64_t part = 2 * int64_t(blockIdx.x) + (at.j0 == 0);
        if (a.row_record && at.j0 == 0 && threadIdx.x == 0) {
            const int last = int(((at.begin + kRowCost + at.s.tiles) * blocks - 1) / total);
            a.row_record[int64_t(at.i) * a.pairs + at.row] = make_int2(whole ? -1 : int(blockIdx.x), last);
        }
        if (lane == 0) where[warp] = (warp * kStages + refill) * S::kStage;
        auto join_warps = [&](auto chunked) {
            constexpr bool CHUNKED = decltype(chunked)::value;
            // the sums of the chunks before lie where the part's will
            if (CHUNKED && chunk > at.j0 && int(threadIdx.x) < heads) stat[kWarps][threadIdx.x] = a.part_ml[part * kHeads + threadIdx.x];
#pragma unroll
            for (int first = 0; first < NT; first += kRound) {
#pragma unroll
                for (int n = 0; n < kRound; ++n) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float& sum = l[first + n][c];
#pragma unroll
                        for (int x = 4; x < 32; x *= 2) sum += __shfl_xor_sync(~0u, sum, x);
                        const int h = n * 8 + lane % 4 * 2 + c;
                        if (lane < 4) stat[warp][first * 8 + h] = make_float2(m[first + n][c], broken ? NAN : sum);
                        float* to = reinterpret_cast<float*>(ring + (warp * kStages + refill) * S::kStage) + h * kOut + lane / 4;
#pragma unroll
                        for (int ks = 0; ks < kSteps; ++ks) to[ks * 16] = o[first + n][ks][c], to[ks * 16 + 8] = o[first + n][ks][c + 2];
                    }
                }
                __syncthreads();
                const int here = min(8 * kRound, heads - first * 8);
                for (int x = threadIdx.x; x < here * (DP / 4); x += kThreads) {  // four results each
                    const int in = x / (DP / 4), e = x % (DP / 4) * 4, h = first * 8 + in;
                    if (e >= a.d) continue;
                    float top = -INFINITY, sum = 0.f;
                    float4 val = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (uint32_t w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w][h].x);
#pragma unroll
                    for (uint32_t w = 0; w < kWarps; ++w) {
                        const float by = weight(stat[w][h].x, top);
                        const float4 v = *reinterpret_cast<const float4*>(ring + where[w] + (in * kOut + e) * 4);
                        sum += stat[w][h].y * by;
                        val.x += v.x * by, val.y += v.y * by, val.z += v.z * by, val.w += v.w * by;
                    }
                    float* const part_o = a.part_o + (part * kHeads + h) * a.d + e;
                    if (CHUNKED && chunk > at.j0) {
                        const float2 ml = stat[kWarps][h];
                        const float4 v = *reinterpret_cast<const float4*>(part_o);
                        const float now = fmaxf(top, ml.x), by = weight(top, now), by2 = weight(ml.x, now);
                        top = now, sum = sum * by + ml.y * by2;
                        val.x = val.x * by + v.x * by2, val.y = val.y * by + v.y * by2, val.z = val.z * by + v.z * by2, val.w = val.w * by + v.w * by2;
                    }
                    if (CHUNKED ? whole && stop == at.j1 : whole) {
                        const bool none = at.s.len == 0 && !at.s.bad;
                        const int hq = head0 + h;
                        const float by = none ? 0.f : 1.f / sum;
                        const uint2 r = none ? make_uint2(0, 0) : make_uint2(pack2<BF>(val.x * by, val.y * by), pack2<BF>(val.z * by, val.w * by));
                        uint16_t* to = a.out + at.i * a.out_row + hq * a.out_head + e;
                        if (a.out_quads)
                            *reinterpret_cast<uint2*>(to) = r;
                        else
                            to[0] = uint16_t(r.x), to[1] = uint16_t(r.x >> 16), to[2] = uint16_t(r.y), to[3] = uint16_t(r.y >> 16);
                        if (a.lse && e == 0)
                            a.lse[int64_t(at.i) * a.q_heads + hq] = none ? -INFINITY : (top + (log2f(sum) - kLift<BF>)) * 0.6931471805599453f;
                    } else {
                        *reinterpret_cast<float4*>(part_o) = val;
                        if (e == 0) a.part_ml[part * kHeads + h] = make_float2(top, sum);
                    }
                }
                __syncthreads();
            }
        };
        if (chunk == at.j0 && stop == at.j1)
            join_warps(std::false_type());
        else
            join_warps(std::true_type());
        chunk = stop;
        if (chunk < at.j1) continue;
        if (!next_part(a, at)) break;
        chunk = at.j0;
    } while (true);
    fetch_wait<0>();
}

// Joins the parts of a row that borders cut, in the order of its tokens: block
// (border, 512 of the row's results), four results a lane.  With SPLIT, where rows
// are few, one has dozens of parts and their loads are what this waits for: block
// (row, 128 results), each warp a quarter of the parts, and the first the warps'
// sums.
template <bool BF, bool SPLIT>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ Attention a, int kept) {
    wait_for_launch_before();
    int4 r;  // sequence, row, first and last block
    if constexpr (SPLIT) {
        const int2 b = a.row_record[blockIdx.x];
        r = make_int4(b.x < 0 ? -1 : int(blockIdx.x) / a.pairs, int(blockIdx.x) % a.pairs, b.x, b.y);
    } else {
        r = a.record[blockIdx.x + 1];
    }
    if (r.x < 0) return;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int blk = r.y % a.blocks, heads = min(kept, a.group - blk * kept);
    const int at = 4 * int(blockIdx.y * (SPLIT ? 32 : kThreads) + (SPLIT ? lane : threadIdx.x)), h = at / a.d, e = at - h * a.d;
    struct Sums {
        float top, sum, val[4];
        __device__ void scale_to(float now) {
            const float by = weight(top, now);
            top = now, sum *= by;
#pragma unroll
            for (int c = 0; c < 4; ++c) val[c] *= by;
        }
        __device__ void add(float m, float l, const float (&o)[4]) {
            const float w = weight(m, top);
            sum += l * w;
#pragma unroll
            for (int c = 0; c < 4; ++c) val[c] += o[c] * w;
        }
    };
    Sums s{-INFINITY, 0.f, {}};
    const int each = SPLIT ? (r.w - r.z + int(kWarps)) / int(kWarps) : r.w + 1 - r.z;
    const int begin = SPLIT ? r.z + warp * each : r.z, end = min(r.w + 1, begin + each);
    constexpr int kAhead = SPLIT ? 8 : 4;
    for (int b0 = begin; h < heads && b0 < end; b0 += kAhead) {
        float2 ml[kAhead];
        float4 o[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
            const int b = b0 + n;
            ml[n] = make_float2(-INFINITY, 0.f), o[n] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (b >= end) continue;
            // the first part lies where its block's last one does, the others where a block's first does
            const int64_t part = (2 * int64_t(b) + (b == r.z)) * kept + h;
            ml[n] = a.part_ml[part];
            o[n] = *reinterpret_cast<const float4*>(a.part_o + part * a.d + e);
        }
        float now = s.top;
#pragma unroll
        for (int n = 0; n < kAhead; ++n) now = fmaxf(now, ml[n].x);
        s.scale_to(now);
#pragma unroll
        for (int n = 0; n < kAhead; ++n) s.add(ml[n].x, ml[n].y, {o[n].x, o[n].y, o[n].z, o[n].w});
    }
    if constexpr (SPLIT) {
        __shared__ Sums of_warp[kWarps][32];
        of_warp[warp][lane] = s;
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (uint32_t w = 1; w < kWarps; ++w) {
            const Sums& t = of_warp[w][lane];
            s.scale_to(fmaxf(s.top, t.top));
            s.add(t.top, t.sum, t.val);
        }
    }
    if (h >= heads) return;
    const int hq = r.y / a.blocks * a.group + blk * kept + h;
    uint16_t* to = a.out + r.x * a.out_row + hq * a.out_head + e;
    const float by = 1.f / s.sum;
    const uint2 v = make_uint2(pack2<BF>(s.val[0] * by, s.val[1] * by), pack2<BF>(s.val[2] * by, s.val[3] * by));
    if (a.out_quads)
        *reinterpret_cast<uint2*>(to) = v;
    else
        to[0] = uint16_t(v.x), to[1] = uint16_t(v.x >> 16), to[2] = uint16_t(v.y), to[3] = uint16_t(v.y >> 16);
    if (a.lse && e == 0) a.lse[int64_t(r.x) * a.q_heads + hq] = (s.top + (log2f(s.sum) - kLift<BF>)) * 0.6931471805599453f;
}

// Blocks on an SM, by head size and query heads kept, as Shape has them.
constexpr int blocks_on_sm(int64_t d, uint32_t heads) {
    if (d > 192) return 1;
    if (d > 128) return 2;
    return heads == 32 && d > 64 ? 2 : 3;
}

template <int DP, int NT, bool BF>
cudaError_t launch_as(const Attention& a, const AttentionPlan& plan, cudaStream_t s) {
    static_assert(blocks_on_sm(DP, 8 * NT) == int(Shape<DP, NT>::kBlocks), "the plan counts on the blocks that there are");
    auto kern = attention_kernel<DP, NT, BF>;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Shape<DP, NT>::kSmem));
        if (err != cudaSuccess) return err;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    err = launch_next(kern, dim3(plan.grid), kThreads, Shape<DP, NT>::kSmem, 1, s, a);
    if (err != cudaSuccess || !plan.cut || plan.grid < 2) return err;
    const uint32_t results = std::min<uint32_t>(plan.heads, a.group) * a.d;
    if (a.row_record)
        return launch_next(join_kernel<BF, true>, dim3(a.seqs * a.pairs, (results + 127) / 128), kThreads, 0, 1, s, a, int(plan.heads));
    return launch_next(join_kernel<BF, false>, dim3(plan.grid - 1, (results + 4 * kThreads - 1) / (4 * kThreads)), kThreads, 0, 1, s, a, int(plan.heads));
}

template <int DP, int NT>
cudaError_t launch_typed(const Attention& a, int dtype, const AttentionPlan& plan, cudaStream_t s) {
    return dtype == UZIP_BF16 ? launch_as<DP, NT, true>(a, plan, s) : launch_as<DP, NT, false>(a, plan, s);
}

template <int DP>
cudaError_t launch_wide(const Attention& a, int dtype, const AttentionPlan& plan, cudaStream_t s) {
    if (plan.heads == 8) return launch_typed<DP, 1>(a, dtype, plan, s);
    if constexpr (DP <= 128)
        if (plan.heads == 32) return launch_typed<DP, 4>(a, dtype, plan, s);
    return launch_typed<DP, 2>(a, dtype, plan, s);
}

}  // namespace

AttentionPlan plan_attention(int64_t seqs, int64_t kv_heads, int64_t group, int64_t d, int64_t most, int sms) {
    AttentionPlan p;
    // more query heads share a key head's pass over memory, up to what registers hold of their sums (64 sequences of 2000
    // to 6000 tokens, 4 x 32 heads of 128: 165 us in two passes, 106 in one)
    p.heads = group <= 8 ? 8 : group <= 16 || d > 128 ? 16 : 32;
    const int64_t rows = seqs * kv_heads * ((group + p.heads - 1) / p.heads);
    const int64_t tiles = std::max<int64_t>(1, (most + kTile - 1) / kTile);
    const int64_t room = int64_t(sms) * blocks_on_sm(d, p.heads);
    // up to 512 tokens a row stays whole: joining would take 2.2 us, as much as four tiles of a warp
    p.cut = tiles > 32;
    p.grid = uint32_t(std::max<int64_t>(1, std::min(room, p.cut ? rows * ((tiles + kRowCost + kLeast - 1) / kLeast) : rows)));
    p.by_row = p.cut && p.grid >= 8 * rows ? rows : 0;  // eight parts a row or more, where it has its full length
    return p;
}

cudaError_t launch_attention(const Attention& a, int dtype, const AttentionPlan& plan, cudaStream_t s) {
    if (a.d <= 64) return launch_wide<64>(a, dtype, plan, s);
    if (a.d <= 96) return launch_wide<96>(a, dtype, plan, s);
    if (a.d <= 128) return launch_wide<128>(a, dtype, plan, s);
    if (a.d <= 192) return launch_wide<192>(a, dtype, plan, s);
    return launch_wide<256>(a, dtype, plan, s);
}

}  // namespace uzip
