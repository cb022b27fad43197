// The pages of a key-value cache: reserving them for new tokens, forking, freeing
// and compacting sequences, and copying pages.
//
// The state (reference counts, tables, lengths) is small and the operations are a
// chain of short dependent steps (prefix sums, then what goes by them), so what
// bounds them is latency.  Each is one launch, of one block or of a cluster whose
// blocks meet at cluster barriers instead of in further launches.  An operation
// first checks everything, and changes the state only after all blocks have agreed
// that nothing is wrong.
#include <algorithm>
#include <atomic>

#include "cache.cuh"

namespace uzip {
namespace {

constexpr uint32_t kThreads = 1024, kWarps = kThreads / 32;
static_assert(kWarps == 32, "prefix() has one warp add up the others' sums, one a lane");
constexpr uint32_t kCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of all blocks; what they wrote before, here and in global memory, is seen after.
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A value in block `rank`'s shared memory, at the place that `here` has in this one's.
__device__ __forceinline__ int64_t peer(const int64_t* here, uint32_t rank) {
    uint32_t at = uint32_t(__cvta_generic_to_shared(here)), far;
    int64_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(far) : "memory");
    return v;
}

// Prefix sums over all threads of the cluster, in the order of blocks and threads.
template <int N>
struct Prefix {
    int64_t before[N], total[N];
};
template <int N>
struct PrefixRoom {
    int64_t warp[N][kWarps];
    int64_t block[N];
};
template <int N>
__device__ Prefix<N> prefix(const int64_t (&mine)[N], PrefixRoom<N>& room, uint32_t rank, uint32_t blocks) {
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int64_t sum[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        sum[n] = mine[n];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t got = __shfl_up_sync(~0u, sum[n], o);
            if (lane >= uint32_t(o)) sum[n] += got;
        }
        if (lane == 31) room.warp[n][warp] = sum[n];
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            int64_t s = room.warp[n][lane];
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int64_t got = __shfl_up_sync(~0u, s, o);
                if (lane >= uint32_t(o)) s += got;
            }
            room.warp[n][lane] = s;  // inclusive
            if (lane == 31) room.block[n] = s;
        }
    }
    if (blocks > 1)
        cluster_meet();
    else
        __syncthreads();
    Prefix<N> p;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        p.before[n] = sum[n] - mine[n] + (warp ? room.warp[n][warp - 1] : 0);
        p.total[n] = 0;
        for (uint32_t b = 0; b < blocks; ++b) {
            const int64_t v = blocks > 1 ? peer(&room.block[n], b) : room.block[n];
            if (b < rank) p.before[n] += v;
            p.total[n] += v;
        }
    }
    return p;
}
// Whether any thread of the cluster says so.
__device__ bool any_of(bool mine, int64_t* flag, uint32_t blocks) {
    const bool here = __syncthreads_or(mine);
    if (blocks == 1) return here;
    if (threadIdx.x == 0) *flag = here;
    cluster_meet();
    bool any = false;
    for (uint32_t b = 0; b < blocks; ++b) any |= peer(flag, b) != 0;
    return any;
}

__device__ __forceinline__ int pages_of(int tokens, int page) { return int((uint32_t(tokens) + uint32_t(page - 1)) / uint32_t(page)); }
__device__ __forceinline__ bool length_ok(const CacheState& c, int n) { return n >= 0 && n <= int64_t(c.width) * c.page; }
// Whether an entry of a row, every 32nd from `col` on, is no page in use.
__device__ __forceinline__ bool pages_bad(const CacheState& c, int64_t row, int col, int end) {
    bool bad = false;
#pragma unroll 4
    for (; col < end; col += 32) {
        const int p = c.table[row * c.ldt + col];
        bad |= uint32_t(p) >= uint32_t(c.pages) || c.refs[p] < 1;
    }
    return bad;
}
__device__ __forceinline__ void report(const CacheState& c, int what) {
    if (c.status && cluster_rank() == 0 && threadIdx.x == 0) *c.status = what;
}

// Last i in [0, n) with v[i] <= x (v ascends, v[0] <= x).
template <typename T>
__device__ __forceinline__ int last_at_most(const T* v, int n, int64_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (v[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Three prefix sums at once: pages that the sequences before need, tokens that
// they have, free pages before.  A thread takes neighbouring sequences and
// neighbouring pages.
__global__ void __launch_bounds__(kThreads) reserve_kernel(const __grid_constant__ Reserve a) {
    wait_for_launch_before();
    __shared__ PrefixRoom<3> room;
    __shared__ int64_t flag;
    extern __shared__ int64_t own[];
    const CacheState& c = a.c;
    const uint32_t blocks = gridDim.x, rank = blocks > 1 ? cluster_rank() : 0;
    const int64_t threads = int64_t(blocks) * kThreads, me = int64_t(rank) * kThreads + threadIdx.x;
    // lists of the sequences and of the pages taken: one block keeps them to itself
    int64_t* const begin_of = a.begin ? a.begin : own;
    int32_t* const first_of = a.begin ? a.first : reinterpret_cast<int32_t*>(own + c.seqs);
    int32_t* const before = a.begin ? a.before : first_of + c.seqs;
    int32_t* const held_of = a.begin ? a.held : before + c.seqs;
    int32_t* const fresh = a.begin ? a.fresh : held_of + c.seqs;
    const int64_t seqs_each = (c.seqs + threads - 1) / threads, pages_each = ((c.pages + threads - 1) / threads + 3) / 4 * 4;
    const int s0 = int(min(int64_t(c.seqs), me * seqs_each)), s1 = int(min(int64_t(c.seqs), s0 + seqs_each));
    const int p0 = int(min(int64_t(c.pages), me * pages_each)), p1 = int(min(int64_t(c.pages), p0 + pages_each));
    int64_t mine[3] = {};
    bool bad = false, wide = false;
    for (int i = s0; i < s1; ++i) {
        const int n = c.lengths[i], count = a.counts[i];
        if (!length_ok(c, n) || count < 0) {
            bad = true;
            continue;
        }
        const int have = pages_of(n, c.page);
        mine[1] += count;
        if (int64_t(n) + count > min(int64_t(c.width) * c.page, int64_t(INT32_MAX))) {
            wide = true;
            continue;
        }
        const int want = pages_of(n + count, c.page);
        int cow = 0;
        if (count && n % c.page) {
            const int last = c.table[i * c.ldt + have - 1];
            if (uint32_t(last) >= uint32_t(c.pages))
                bad = true;
            else if (c.refs[last] < 1)
                bad = true;
            else
                cow = c.refs[last] > 1;
        }
        mine[0] += want - have + cow;
        before[i] = n;
        held_of[i] = cow ? ~have : have;  // pages before; ~ where the last of them is copied
    }
    for (int p = p0; p < p1; ++p) mine[2] += c.refs[p] == 0;
    const Prefix<3> sum = prefix(mine, room, rank, blocks);
    bad = any_of(bad, &flag, blocks) || sum.total[1] > a.tokens;
    if (blocks > 1) cluster_meet();  // the flag is used again
    wide = any_of(wide, &flag, blocks) || sum.total[0] > sum.total[2];
    if (bad || wide) {
        report(c, bad ? UZIP_ERR_INVALID_ARG : UZIP_ERR_CAPACITY);
        for (int64_t t = me; t < a.tokens; t += threads) a.slots[t] = -1, a.positions[t] = 0;
        for (int64_t i = me; i < 2 * int64_t(c.seqs); i += threads) a.copies[i] = -1;
        if (blocks > 1) cluster_meet();  // no block ends while another may read its flag
        return;
    }
    {
        int64_t first = sum.before[0], begin = sum.before[1];
        for (int i = s0; i < s1; ++i) {
            first_of[i] = int32_t(first), begin_of[i] = begin;
            const int n = c.lengths[i], count = a.counts[i], held = held_of[i];
            first += pages_of(n + count, c.page) - (held < 0 ? ~held - 1 : held);
            begin += count;
        }
        int64_t free = sum.before[2];
        for (int p = p0; p < p1 && free < sum.total[0]; ++p)
            if (c.refs[p] == 0) fresh[free++] = p;
    }
    if (blocks > 1)
        cluster_meet();
    else
        __syncthreads();
    // each new page goes to its place
    for (int64_t r = me; r < sum.total[0]; r += threads) {
        const int i = last_at_most(first_of, c.seqs, r);
        const int p = fresh[r], held = held_of[i], cow = held < 0, in = int(r - first_of[i]);
        int32_t* place = c.table + i * c.ldt + (cow ? ~held - 1 : held) + in;
        if (cow && in == 0) {
            const int old = *place;
            a.copies[2 * i] = old, a.copies[2 * i + 1] = p;
            atomicSub(&c.refs[old], 1);
        }
        *place = p;
        c.refs[p] = 1;
    }
    for (int i = s0; i < s1; ++i) {
        c.lengths[i] = before[i] + a.counts[i];
        if (held_of[i] >= 0) a.copies[2 * i] = -1, a.copies[2 * i + 1] = -1;
    }
    for (int64_t t = me; t < a.tokens; t += threads) {
        int64_t slot = -1;
        int pos = 0;
        if (t < sum.total[1]) {
            const int i = last_at_most(begin_of, c.seqs, t);
            pos = before[i] + int(t - begin_of[i]);
            const int col = int(uint32_t(pos) / uint32_t(c.page)), held = held_of[i], kept = held < 0 ? ~held - 1 : held;
            // entries that this call writes are read from the list, the others from the table
            const int p = col >= kept ? fresh[first_of[i] + col - kept] : c.table[i * c.ldt + col];
            slot = int64_t(p) * c.page + (pos - col * c.page);
        }
        a.slots[t] = slot, a.positions[t] = pos;
    }
}

// Fork: children become sequences with the pages of their parents.  Free (no
// parents): the sequences' pages are given back.  mark[s] holds an entry that
// lists sequence s; a second one shows as another's mark.
__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ Fork a) {
    wait_for_launch_before();
    __shared__ int64_t flag;
    const CacheState& c = a.c;
    const uint32_t blocks = gridDim.x, rank = blocks > 1 ? cluster_rank() : 0;
    const int64_t threads = int64_t(blocks) * kThreads, me = int64_t(rank) * kThreads + threadIdx.x;
    const int lane = threadIdx.x % 32;
    extern __shared__ int64_t own[];
    int32_t* const mark = a.mark ? a.mark : reinterpret_cast<int32_t*>(own);  // one block keeps it to itself
    for (int64_t j = me; j < a.n; j += threads) {
        const int s = a.children[j];
        if (s >= 0 && s < c.seqs) mark[s] = int32_t(j);
    }
    if (blocks > 1)
        cluster_meet();
    else
        __syncthreads();
    bool bad = false;
    for (int64_t j = me; j < a.n; j += threads) {
        const int s = a.children[j];
        if (s < -1 || s >= c.seqs) {
            bad = true;
            continue;
        }
        if (s >= 0) bad |= mark[s] != int32_t(j);
        if (a.parents) {
            const int from = a.parents[j];
            if (from < -1 || from >= c.seqs || (from < 0) != (s < 0)) {
                bad = true;
                continue;
            }
            if (s < 0) continue;
            bad |= c.lengths[s] != 0;
            const uint32_t listed = uint32_t(mark[from]);  // says something only where that entry lists it
            bad |= listed < a.n && a.children[listed] == from;
            bad |= !length_ok(c, c.lengths[from]);
        } else if (s >= 0) {
            bad |= !length_ok(c, c.lengths[s]);
        }
    }
    // a warp takes 256 columns of a row at a time
    const int pieces = (c.width + 255) / 256;
    const int64_t jobs = a.n * pieces, warps = threads / 32;
    for (int64_t job = me / 32; job < jobs; job += warps) {
        const int64_t j = job / pieces;
        const int s = a.parents ? a.parents[j] : a.children[j];
        if (s < 0 || s >= c.seqs || !length_ok(c, c.lengths[s])) continue;
        const int begin = int(job % pieces) * 256, end = min(begin + 256, pages_of(c.lengths[s], c.page));
        bad |= pages_bad(c, s, begin + lane, end);
    }
    if (any_of(bad, &flag, blocks)) {
        report(c, UZIP_ERR_INVALID_ARG);
    } else {
        for (int64_t job = me / 32; job < jobs; job += warps) {
            const int64_t j = job / pieces;
            const int s = a.children[j], from = a.parents ? a.parents[j] : s;
            if (s < 0) continue;
            const int begin = int(job % pieces) * 256, used = pages_of(c.lengths[from], c.page);
#pragma unroll 4
            for (int col = begin + lane; col < min(begin + 256, c.width); col += 32) {
                int p = -1;
                if (col < used) {
                    p = c.table[from * c.ldt + col];
                    atomicAdd(&c.refs[p], a.parents ? 1 : -1);
                }
                c.table[s * c.ldt + col] = a.parents ? p : -1;
            }
        }
        // lengths were read by other threads until here
        if (blocks > 1)
            cluster_meet();
        else
            __syncthreads();
        for (int64_t j = me; j < a.n; j += threads)
            if (a.children[j] >= 0) c.lengths[a.children[j]] = a.parents ? c.lengths[a.parents[j]] : 0;
    }
    if (blocks > 1) cluster_meet();  // no block ends while another may read its flag
}

__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ Compact a) {
    wait_for_launch_before();
    __shared__ PrefixRoom<1> room, room2;
    __shared__ int64_t flag;
    const CacheState& c = a.c;
    const uint32_t blocks = gridDim.x, rank = blocks > 1 ? cluster_rank() : 0;
    const int64_t threads = int64_t(blocks) * kThreads, me = int64_t(rank) * kThreads + threadIdx.x;
    const int lane = threadIdx.x % 32;
    const int64_t each = ((c.pages + threads - 1) / threads + 3) / 4 * 4;
    const int p0 = int(min(int64_t(c.pages), me * each)), p1 = int(min(int64_t(c.pages), p0 + each));
    bool bad = false;
    int64_t mine[1] = {0};
    for (int p = p0; p < p1; ++p) {
        const int r = c.refs[p];
        bad |= r < 0;
        mine[0] += r > 0;
    }
    // a warp takes 256 columns of a row at a time
    const int pieces = (c.width + 255) / 256;
    const int64_t jobs = int64_t(c.seqs) * pieces, warps = threads / 32;
    for (int64_t s = me; s < c.seqs; s += threads) bad |= !length_ok(c, c.lengths[s]);
    for (int64_t job = me / 32; job < jobs; job += warps) {
        const int s = int(job / pieces), begin = int(job % pieces) * 256, n = c.lengths[s];
        if (length_ok(c, n)) bad |= pages_bad(c, s, begin + lane, min(begin + 256, pages_of(n, c.page)));
    }
    const Prefix<1> used = prefix(mine, room, rank, blocks);
    const int64_t kept = used.total[0];  // pages used: they end up below this
    int64_t low[1] = {0};  // used pages that lie below already
    for (int p = p0; p < p1 && p < kept; ++p) low[0] += c.refs[p] > 0;
    const Prefix<1> below = prefix(low, room2, rank, blocks);
    if (any_of(bad, &flag, blocks)) {
        report(c, UZIP_ERR_INVALID_ARG);
        for (int64_t i = me; i < c.pages / 2 * 2; i += threads) a.moves[i] = -1;
        if (blocks > 1) cluster_meet();
        return;
    }
    const int64_t count = kept - below.total[0];
    {
        int64_t before = used.before[0];
        for (int p = p0; p < p1; ++p) {
            const bool is = c.refs[p] > 0;
            if (p < kept && !is) a.holes[p - before] = p;
            if (p >= kept && is) a.movers[before - below.total[0]] = p;
            before += is;
        }
    }
    if (blocks > 1)
        cluster_meet();
    else
        __syncthreads();
    for (int64_t i = me; i < c.pages / 2; i += threads) {
        int from = -1, to = -1;
        if (i < count) {
            from = a.movers[i], to = a.holes[i];
            a.to[from] = to;
            c.refs[to] = c.refs[from];
            c.refs[from] = 0;
        }
        a.moves[2 * i] = from, a.moves[2 * i + 1] = to;
    }
    if (blocks > 1)
        cluster_meet();
    else
        __syncthreads();
    for (int64_t job = me / 32; job < jobs; job += warps) {
        const int64_t s = job / pieces;
        const int begin = int(job % pieces) * 256, end = min(begin + 256, pages_of(c.lengths[s], c.page));
#pragma unroll 4
        for (int col = begin + lane; col < end; col += 32) {
            int32_t* place = c.table + s * c.ldt + col;
            if (*place >= kept) *place = a.to[*place];
        }
    }
    if (blocks > 1) cluster_meet();
}

// A chain of short steps on few values: one block has no cluster barriers to
// wait for, eight have eight times the threads: all operations on eight, a step's
// reservation with its copies takes 22.3 us instead of 16.2, but compaction of
// 16384 pages with its copies 364 instead of 377.
uint32_t cluster_for(int64_t items) { return items <= 2 * int64_t(kThreads) ? 1 : kCluster; }

// ---- copies -----------------------------------------------------------------------

constexpr uint32_t kCopyThreads = 256;
constexpr int kCopyAhead = 8;
constexpr int64_t kPiece = int64_t(kCopyThreads) * kCopyAhead;  // 16-byte units of a piece

// Every block first looks all pairs over, with a bit for each page that is
// written: written twice, or read and written, and no block copies anything.
// Then pieces of pages, layers, keys and values are dealt out to the blocks, 32 KB
// at a time.  4096 pages of 4 layers, 2.1 GB read and written: 332 us, 6.5 TB/s.
template <bool FLAT>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ PageCopy a) {
    extern __shared__ uint32_t written[];
    __shared__ int ends[kCopyThreads / 32];
    wait_for_launch_before();
    for (int w = threadIdx.x; w < (a.to_pages + 31) / 32; w += kCopyThreads) written[w] = 0;
    __syncthreads();
    bool bad = false;
    int end = 0;  // pairs up to the last one that is not skipped
    const int2* pairs = reinterpret_cast<const int2*>(a.pairs);
    for (int64_t j = threadIdx.x; j < a.n; j += kCopyThreads) {
        const int2 p = pairs[j];
        if (p.x == -1 || p.y == -1) continue;
        end = int(j) + 1;
        if (uint32_t(p.x) >= uint32_t(a.from_pages) || uint32_t(p.y) >= uint32_t(a.to_pages)) {
            bad = true;
            continue;
        }
        bad |= atomicOr(&written[p.y / 32], 1u << p.y % 32) >> p.y % 32 & 1;
    }
#pragma unroll
    for (int x = 16; x; x /= 2) end = max(end, __shfl_xor_sync(~0u, end, x));
    if (threadIdx.x % 32 == 0) ends[threadIdx.x / 32] = end;
    __syncthreads();
    for (int w = 0; w < int(kCopyThreads / 32); ++w) end = max(end, ends[w]);
    if (a.same)
        for (int64_t j = threadIdx.x; j < end; j += kCopyThreads) {
            const int2 p = pairs[j];
            if (p.x == -1 || p.y == -1 || uint32_t(p.x) >= uint32_t(a.to_pages)) continue;
            bad |= written[p.x / 32] >> p.x % 32 & 1;
        }
    if (__syncthreads_or(bad)) {
        if (a.status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = UZIP_ERR_INVALID_ARG;
        return;
    }
    const int64_t units = int64_t(a.outer) * a.inner * a.run, pieces = (units + kPiece - 1) / kPiece;
    const int64_t per_pair = pieces * a.layers * 2;
    for (int64_t job = blockIdx.x; job < end * per_pair; job += gridDim.x) {
        const int64_t j = job / per_pair;
        const int2 p = pairs[j];
        if (p.x == -1 || p.y == -1) continue;
        const int64_t in = job - j * per_pair, piece = in % pieces, side = in / pieces;
        const int which = int(side % 2), layer = int(side / 2);
        const uint4* from = reinterpret_cast<const uint4*>(which ? a.v : a.k) + layer * a.layer[which] + p.x * a.page[which];
        uint4* to = reinterpret_cast<uint4*>(which ? a.v_to : a.k_to) + layer * a.layer[2 + which] + p.y * a.page[2 + which];
        uint4 held[kCopyAhead];
        int64_t at[kCopyAhead];
#pragma unroll
        for (int u = 0; u < kCopyAhead; ++u) {
            const int64_t x = piece * kPiece + u * kCopyThreads + threadIdx.x;
            at[u] = -1;
            if (x >= units) continue;
            int64_t src = x;
            at[u] = x;
            if constexpr (!FLAT) {
                const int64_t run = x / a.run, o = run / a.inner, i = run - o * a.inner;
                src = x - run * a.run + o * a.outer_step[which] + i * a.inner_step[which];
                at[u] = x - run * a.run + o * a.outer_step[2 + which] + i * a.inner_step[2 + which];
            }
            held[u] = from[src];
        }
#pragma unroll
        for (int u = 0; u < kCopyAhead; ++u)
            if (at[u] >= 0) to[at[u]] = held[u];
    }
}

}  // namespace

// Lists that one block can keep in shared memory need no workspace.
constexpr int64_t kOwn = 40 * 1024;

static uint32_t reserve_blocks(int64_t seqs, int64_t pages, int64_t tokens) {
    return cluster_for(std::max<int64_t>({seqs, pages / 8, tokens}));
}
bool reserve_keeps(int64_t seqs, int64_t pages, int64_t tokens, int64_t list) {
    return reserve_blocks(seqs, pages, tokens) == 1 && 20 * seqs + 4 * list <= kOwn;
}
cudaError_t launch_reserve(const Reserve& r, cudaStream_t s) {
    const uint32_t blocks = reserve_blocks(r.c.seqs, r.c.pages, r.tokens);
    return launch_next(reserve_kernel, dim3(blocks), kThreads, r.begin ? 0 : uint32_t(20 * r.c.seqs + 4 * r.list), blocks, s, r);
}
static uint32_t fork_blocks(int64_t n, int64_t width) { return cluster_for(n * ((width + 255) / 256) * 32); }
bool fork_keeps(int64_t seqs, int64_t n, int64_t width) { return fork_blocks(n, width) == 1 && 4 * seqs <= kOwn; }
cudaError_t launch_fork(const Fork& f, cudaStream_t s) {
    const uint32_t blocks = fork_blocks(f.n, f.c.width);
    return launch_next(fork_kernel, dim3(blocks), kThreads, f.mark ? 0 : uint32_t(4 * f.c.seqs), blocks, s, f);
}
cudaError_t launch_compact(const Compact& m, cudaStream_t s) {
    const uint32_t blocks = cluster_for(std::max<int64_t>(m.c.pages / 4, int64_t(m.c.seqs) * ((m.c.width + 255) / 256) * 32));
    return launch_next(compact_kernel, dim3(blocks), kThreads, 0, blocks, s, m);
}

template <bool FLAT>
static cudaError_t launch_copy_as(const PageCopy& c, uint32_t blocks, uint32_t smem, cudaStream_t s) {
    auto kern = copy_kernel<FLAT>;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use all of the shared memory
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, UZIP_MAX_PAGES / 8);
        if (err != cudaSuccess) return err;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    return launch_next(kern, dim3(blocks), kCopyThreads, smem, 1, s, c);
}

cudaError_t launch_page_copy(const PageCopy& c, int sms, cudaStream_t s) {
    const int64_t units = int64_t(c.outer) * c.inner * c.run, pieces = (units + kPiece - 1) / kPiece;
    const uint32_t smem = uint32_t((c.to_pages + 31) / 32 * 4);
    const int per_sm = int(std::max<uint32_t>(1, std::min<uint32_t>(4, 200 * 1024 / (smem + 1024))));
    const uint32_t blocks = uint32_t(std::max<int64_t>(1, std::min<int64_t>(c.n * pieces * c.layers * 2, int64_t(sms) * per_sm)));
    const bool flat = c.outer == 1 && c.inner == 1;
    return flat ? launch_copy_as<true>(c, blocks, smem, s) : launch_copy_as<false>(c, blocks, smem, s);
}

}  // namespace uzip
