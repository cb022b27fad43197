// C ABI of the key-value cache: argument checks, workspace layout and the order
// of the launches.  Every check that can be made on the host is made before
// anything is enqueued.
#include <algorithm>
#include <array>
#include <cmath>
#include <limits>

#include "cache.cuh"

namespace uzip {
bool device_range_ok(const void* p, uint64_t bytes);  // api.cu
}

namespace {

using namespace uzip;

constexpr int64_t kMost31 = (int64_t(1) << 31) - 1;
constexpr int64_t kMostStride = int64_t(1) << 40;
constexpr int64_t kMostHeads = 65535;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool half_type(int dtype) { return dtype == UZIP_BF16 || dtype == UZIP_FP16; }
bool within(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

uzip_status finish(cudaError_t err) {
    if (err == cudaSuccess) return UZIP_OK;
    cudaGetLastError();
    return UZIP_ERR_CUDA;
}

int sm_count() {
    static const int sms = [] {  // one kind of GPU in a process
        int dev = 0, v = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return 152;
        }
        return v;
    }();
    return sms;
}

// Hands out the workspace in 256-byte steps.  With no base it only measures.
struct Work {
    uint8_t* base;
    uint64_t used = 0;
    template <typename T>
    T* take(uint64_t count) {
        T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
        used += (count * sizeof(T) + 255) / 256 * 256;
        return p;
    }
};

uzip_status check_work(uint64_t need, void* ws, uint64_t bytes, int32_t* d_status) {
    if (need && (!ws || !aligned(ws, 256))) return UZIP_ERR_INVALID_ARG;
    if (bytes < need) return UZIP_ERR_CAPACITY;
    if (!device_range_ok(ws, need)) return UZIP_ERR_INVALID_ARG;
    if (d_status && (!aligned(d_status, 4) || !device_range_ok(d_status, 4))) return UZIP_ERR_INVALID_ARG;
    return UZIP_OK;
}

cudaError_t clear_status(int32_t* d_status, cudaStream_t s) {
    return d_status ? cudaMemsetAsync(d_status, 0, sizeof(int32_t), s) : cudaSuccess;
}

// A tensor of 16-bit values whose last dimension is contiguous: up to three
// outer dimensions with their strides in elements, and the length of the last.
struct Block {
    const void* p;
    std::array<int64_t, 4> count, step;
    int64_t d;

    bool empty() const { return d == 0 || count[0] == 0 || count[1] == 0 || count[2] == 0 || count[3] == 0; }
    // strides of dimensions of one say nothing
    int64_t stride(int n) const { return count[n] > 1 ? step[n] : 0; }
    bool readable(uintptr_t alignment) const {
        if (empty()) return true;
        int64_t last = d;
        for (int n = 0; n < 4; ++n) {
            if (!within(stride(n), 0, kMostStride) || stride(n) * 2 % int64_t(alignment)) return false;
            if (stride(n) && (count[n] - 1) > (int64_t(1) << 58) / stride(n)) return false;
            last += (count[n] - 1) * stride(n);
            if (last > int64_t(1) << 60) return false;
        }
        return p && aligned(p, alignment) && device_range_ok(p, 2 * uint64_t(last));
    }
    // no value lies where another does: sorted by stride, each dimension steps over all of the ones within it
    bool writable(uintptr_t alignment) const {
        if (!readable(alignment)) return false;
        if (empty()) return true;
        std::array<int, 4> order{0, 1, 2, 3};
        std::sort(order.begin(), order.end(), [&](int x, int y) { return stride(x) < stride(y); });
        int64_t within_it = d;
        for (int n : order) {
            if (count[n] <= 1) continue;
            if (stride(n) < within_it) return false;
            within_it = stride(n) * (count[n] - 1) + within_it;
        }
        return true;
    }
};

Block heads_of(const void* p, int64_t rows, int64_t row, int64_t heads, int64_t head, int64_t d) {
    return Block{p, {1, 1, rows, heads}, {0, 0, row, head}, d};
}
Block pool_of(const void* p, int64_t pages, int64_t heads, int64_t page, const PoolStrides& s, int64_t d, int64_t layers = 1,
              int64_t layer = 0) {
    return Block{p, {layers, pages, heads, page}, {layer, s.page, s.head, s.token}, d};
}
PoolStrides bytes_of(const Block& b) { return PoolStrides{2 * b.stride(1), 2 * b.stride(2), 2 * b.stride(3)}; }

template <typename T>
bool list_ok(const T* p, int64_t n) {
    return n == 0 || (p && aligned(p, sizeof(T)) && device_range_ok(p, uint64_t(n) * sizeof(T)));
}

bool pool_sizes_ok(int64_t pages, int64_t heads, int64_t page, int64_t d) {
    return within(pages, 0, kMost31) && within(heads, 1, kMostHeads) && within(page, 1, kMost31) && within(d, 8, UZIP_MAX_HEAD) && d % 8 == 0;
}

// ---- rotary positions ---------------------------------------------------------

uzip_status rotary(const uzip_rotary_args* a, void* ws, uint64_t bytes, int32_t* d_status, cudaStream_t s, bool append) {
    if (!a) return UZIP_ERR_INVALID_ARG;
    if (!half_type(a->dtype)) return UZIP_ERR_UNSUPPORTED_DTYPE;
    if (!within(a->interleaved, 0, 1) || !within(a->backward, 0, 1) || !within(a->t, 0, kMost31) || !within(a->q_heads, 0, kMostHeads) ||
        !within(a->kv_heads, 0, kMostHeads) || !within(a->d, 1, 1024) || !within(a->rot, 0, a->d) || a->rot % 2)
        return UZIP_ERR_INVALID_ARG;
    if (append && (a->backward || !pool_sizes_ok(a->pages, a->kv_heads, a->page, a->d))) return UZIP_ERR_INVALID_ARG;
    if (!append && a->slots) return UZIP_ERR_INVALID_ARG;
    if (append && a->pages && a->k_pages == a->v_pages) return UZIP_ERR_INVALID_ARG;
    const int64_t t = a->t, d = a->d;
    const Block q = heads_of(a->q, t, a->q_row, a->q_heads, a->q_head, d), qo = heads_of(a->q_out, t, a->q_out_row, a->q_heads, a->q_out_head, d),
                k = heads_of(a->k, t, a->k_row, a->kv_heads, a->k_head, d),
                v = heads_of(append ? a->v : nullptr, append ? t : 0, a->v_row, a->kv_heads, a->v_head, d),
                ko = heads_of(append ? nullptr : a->k_out, append ? 0 : t, a->k_out_row, a->kv_heads, a->k_out_head, d);
    const Block kp = pool_of(a->k_pages, append ? a->pages : 0, a->kv_heads, a->page, {a->kp_page, a->kp_head, a->kp_token}, d),
                vp = pool_of(a->v_pages, append ? a->pages : 0, a->kv_heads, a->page, {a->vp_page, a->vp_head, a->vp_token}, d);
    if (!q.readable(2) || !k.readable(2) || !v.readable(2) || !qo.writable(2) || !ko.writable(2) || !kp.writable(16) || !vp.writable(16))
        return UZIP_ERR_INVALID_ARG;
    if (!list_ok(a->positions, t) || (t && !list_ok(a->freqs, a->rot / 2)) || (append && !list_ok(a->slots, t))) return UZIP_ERR_INVALID_ARG;
    uzip_status st = check_work(0, ws, bytes, d_status);
    if (st != UZIP_OK) return st;
    cudaError_t err = clear_status(d_status, s);
    const int64_t heads = a->q_heads + (append ? 2 : 1) * a->kv_heads;
    if (err != cudaSuccess || t == 0 || heads == 0) return finish(err);
    Rotary r{};
    auto segment = [&](int n, const Block& from, void* to, const Block& out, int64_t count, bool turned, bool paged) {
        RotarySegment& g = r.seg[n];
        g.from = static_cast<const uint16_t*>(from.p), g.row = from.stride(2), g.head = from.stride(3);
        g.to = static_cast<uint16_t*>(to);
        if (paged)
            g.to_row = out.stride(1), g.to_head = out.stride(2), g.to_token = out.stride(3);
        else
            g.to_row = out.stride(2), g.to_head = out.stride(3);
        g.heads = int32_t(count), g.turned = turned, g.paged = paged;
    };
    segment(0, q, a->q_out, qo, a->q_heads, true, false);
    if (append) {
        segment(1, k, a->k_pages, kp, a->kv_heads, true, true);
        segment(2, v, a->v_pages, vp, a->kv_heads, false, true);
        r.slots = a->slots, r.slot_count = a->pages * a->page, r.page = int32_t(a->page);
    } else {
        segment(1, k, a->k_out, ko, a->kv_heads, true, false);
    }
    r.positions = a->positions, r.freqs = a->freqs, r.t = t;
    r.heads = int32_t(heads), r.d = int32_t(d), r.half = int32_t(a->rot / 2);
    r.scale = a->scale, r.sign = a->backward ? -1.f : 1.f;
    r.status = d_status;
    return finish(launch_rotary(r, a->dtype, a->interleaved != 0, sm_count(), s));
}

// ---- attention ----------------------------------------------------------------

uzip_status attention_sizes(const uzip_paged_attention_args& a) {
    if (!half_type(a.dtype)) return UZIP_ERR_UNSUPPORTED_DTYPE;
    if (a.reserved || !within(a.seqs, 0, UZIP_MAX_SEQS) || !pool_sizes_ok(a.pages, a.kv_heads, a.page, a.d) ||
        !within(a.q_heads, 1, kMostHeads) || a.q_heads % a.kv_heads || !within(a.width, 0, kMost31))
        return UZIP_ERR_INVALID_ARG;
    return UZIP_OK;
}

int64_t most_tokens(int64_t width, int64_t page) { return std::min(kMost31, width * page); }

Attention plan_work(const uzip_paged_attention_args& a, const AttentionPlan& plan, Work& w) {
    Attention r{};
    if (plan.cut) {
        r.part_o = w.take<float>(2 * uint64_t(plan.grid) * plan.heads * a.d);
        r.part_ml = w.take<float2>(2 * uint64_t(plan.grid) * plan.heads);
        r.record = w.take<int4>(plan.grid);
        if (plan.by_row) r.row_record = w.take<int2>(plan.by_row);
    }
    return r;
}

AttentionPlan plan_of(const uzip_paged_attention_args& a) {
    int64_t most = most_tokens(a.width, a.page);
    if (a.window > 0) most = std::min(most, a.window);
    return plan_attention(a.seqs, a.kv_heads, a.q_heads / a.kv_heads, a.d, most, sm_count());
}

// ---- the cache's state ----------------------------------------------------------

bool state_ok(const uzip_cache_args& a, bool memory) {
    if (!within(a.pages, 0, kMost31 - 8) || !within(a.page, 1, kMost31) || !within(a.seqs, 0, UZIP_MAX_SEQS) ||
        !within(a.width, 0, kMost31 - 256) || (a.seqs > 1 && !within(a.ldt, a.width, kMostStride)))
        return false;
    if (!memory) return true;
    const int64_t entries = a.seqs && a.width ? (a.seqs - 1) * (a.seqs > 1 ? a.ldt : 0) + a.width : 0;
    return list_ok(a.refs, a.pages) && list_ok(a.table, entries) && list_ok(a.lengths, a.seqs);
}

CacheState state_of(const uzip_cache_args& a, int32_t* d_status) {
    return CacheState{a.refs, a.table, a.seqs > 1 ? a.ldt : a.width, a.lengths, int32_t(a.pages), int32_t(a.page), int32_t(a.seqs), int32_t(a.width),
                      d_status};
}

Reserve plan_reserve(const uzip_cache_args& a, Work& w) {
    Reserve r{};
    r.list = std::min(a.pages, 2 * a.tokens);
    if (reserve_keeps(a.seqs, a.pages, a.tokens, r.list)) return r;
    r.first = w.take<int32_t>(a.seqs), r.begin = w.take<int64_t>(a.seqs), r.before = w.take<int32_t>(a.seqs);
    r.held = w.take<int32_t>(a.seqs), r.fresh = w.take<int32_t>(r.list);
    return r;
}

Compact plan_compact(const uzip_cache_args& a, Work& w) {
    Compact m{};
    m.holes = w.take<int32_t>(a.pages / 2), m.movers = w.take<int32_t>(a.pages / 2), m.to = w.take<int32_t>(a.pages);
    return m;
}

uzip_status fork(const uzip_cache_args* a, void* ws, uint64_t bytes, int32_t* d_status, cudaStream_t s, bool with_parents) {
    if (!a || !state_ok(*a, true) || !within(a->n, 0, kMost31) || !list_ok(a->list, a->n) || (with_parents && !list_ok(a->from, a->n)))
        return UZIP_ERR_INVALID_ARG;
    Work need{nullptr};
    if (!fork_keeps(a->seqs, a->n, a->width)) need.take<int32_t>(a->seqs);
    uzip_status st = check_work(need.used, ws, bytes, d_status);
    if (st != UZIP_OK) return st;
    cudaError_t err = clear_status(d_status, s);
    if (err != cudaSuccess || a->n == 0) return finish(err);
    Fork f{};
    f.c = state_of(*a, d_status);
    f.parents = with_parents ? a->from : nullptr, f.children = a->list, f.n = a->n;
    f.mark = need.used ? static_cast<int32_t*>(ws) : nullptr;
    return finish(launch_fork(f, s));
}

}  // namespace

extern "C" {

uint64_t uzip_rotary_workspace_size(const uzip_rotary_args*) { return 0; }
uzip_status uzip_rotary(const uzip_rotary_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status, cudaStream_t s) {
    return rotary(a, d_workspace, workspace_bytes, d_status, s, false);
}
uint64_t uzip_rotary_append_workspace_size(const uzip_rotary_args*) { return 0; }
uzip_status uzip_rotary_append(const uzip_rotary_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status, cudaStream_t s) {
    return rotary(a, d_workspace, workspace_bytes, d_status, s, true);
}

uint64_t uzip_paged_attention_workspace_size(const uzip_paged_attention_args* a) {
    if (!a || attention_sizes(*a) != UZIP_OK || a->seqs == 0) return 0;
    Work w{nullptr};
    plan_work(*a, plan_of(*a), w);
    return w.used;
}

uzip_status uzip_paged_attention(const uzip_paged_attention_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status,
                                 cudaStream_t s) {
    if (!a) return UZIP_ERR_INVALID_ARG;
    uzip_status st = attention_sizes(*a);
    if (st != UZIP_OK) return st;
    if (a->window < 0 || !(a->softcap >= 0.f) || !(a->softcap < std::numeric_limits<float>::infinity())) return UZIP_ERR_INVALID_ARG;
    // a cap so small that the scale over it is no number says nothing
    if (a->softcap > 0.f && std::isfinite(a->scale) && !std::isfinite(4.f * a->scale / a->softcap)) return UZIP_ERR_INVALID_ARG;
    const Block q = heads_of(a->q, a->seqs, a->q_row, a->q_heads, a->q_head, a->d), out = heads_of(a->out, a->seqs, a->out_row, a->q_heads, a->out_head, a->d);
    const Block k = pool_of(a->k_pages, a->pages, a->kv_heads, a->page, {a->kp_page, a->kp_head, a->kp_token}, a->d),
                v = pool_of(a->v_pages, a->pages, a->kv_heads, a->page, {a->vp_page, a->vp_head, a->vp_token}, a->d);
    if (!q.readable(2) || !k.readable(16) || !v.readable(16) || !out.writable(2)) return UZIP_ERR_INVALID_ARG;
    if (a->seqs && a->out == a->q) return UZIP_ERR_INVALID_ARG;  // other blocks may still read a query when its result is written
    if (a->seqs > 1 && !within(a->ldt, 0, kMostStride)) return UZIP_ERR_INVALID_ARG;
    const int64_t ldt = a->seqs > 1 ? a->ldt : 0;
    if (a->seqs && !list_ok(a->table, a->width ? (a->seqs - 1) * ldt + a->width : 0)) return UZIP_ERR_INVALID_ARG;
    if (!list_ok(a->lengths, a->seqs) || (a->lse && !list_ok(a->lse, a->seqs * a->q_heads))) return UZIP_ERR_INVALID_ARG;
    Work need{nullptr};
    AttentionPlan plan{};
    if (a->seqs) {
        plan = plan_of(*a);
        plan_work(*a, plan, need);
    }
    if ((st = check_work(need.used, d_workspace, workspace_bytes, d_status)) != UZIP_OK) return st;
    cudaError_t err = clear_status(d_status, s);
    if (err != cudaSuccess || a->seqs == 0) return finish(err);
    Work work{static_cast<uint8_t*>(d_workspace)};
    Attention r = plan_work(*a, plan, work);
    r.q = static_cast<const uint16_t*>(a->q), r.q_row = q.stride(2), r.q_head = q.stride(3);
    r.k = static_cast<const uint16_t*>(a->k_pages), r.ks = bytes_of(k);
    r.v = static_cast<const uint16_t*>(a->v_pages), r.vs = bytes_of(v);
    r.table = a->table, r.ldt = ldt, r.lengths = a->lengths;
    r.seqs = int32_t(a->seqs), r.q_heads = int32_t(a->q_heads), r.group = int32_t(a->q_heads / a->kv_heads), r.d = int32_t(a->d);
    r.pages = int32_t(a->pages), r.page = int32_t(a->page);
    // with 2^s >= page, ceil(2^(31 + s) / page) is over 2^(31 + s) / page by less than 2^s / page: nothing below 2^31 notices
    int s2 = 0;
    while (int64_t(1) << s2 < a->page) ++s2;
    r.page_shift = 31 + s2;
    r.page_by = uint32_t(((uint64_t(1) << r.page_shift) + a->page - 1) / a->page);
    r.alike = r.ks.page == r.vs.page && r.ks.head == r.vs.head && r.ks.token == r.vs.token;
    r.q_pairs = aligned(a->q, 4) && r.q_row % 2 == 0 && r.q_head % 2 == 0;
    r.blocks = (r.group + int32_t(plan.heads) - 1) / int32_t(plan.heads);
    r.pairs = int32_t(a->kv_heads) * r.blocks;
    r.most = int32_t(most_tokens(a->width, a->page));
    r.window = a->window >= r.most ? 0 : int32_t(a->window);
    r.cut = plan.cut;
    constexpr float kLog2e = 1.4426950408889634f;
    r.scale = a->scale * kLog2e, r.cap = std::min(a->softcap * kLog2e, std::numeric_limits<float>::max());
    r.per_cap = a->softcap > 0.f ? a->scale / a->softcap : 0.f;
    r.out = static_cast<uint16_t*>(a->out), r.out_row = out.stride(2), r.out_head = out.stride(3);
    r.out_quads = aligned(a->out, 8) && r.out_row % 4 == 0 && r.out_head % 4 == 0;
    r.skip_seq = int32_t(plan.grid) / r.pairs, r.skip_row = int32_t(plan.grid) % r.pairs;
    r.lse = a->lse, r.status = d_status;
    return finish(launch_attention(r, a->dtype, plan, s));
}

uint64_t uzip_cache_reserve_workspace_size(const uzip_cache_args* a) {
    if (!a || !state_ok(*a, false) || !within(a->tokens, 0, kMost31)) return 0;
    Work w{nullptr};
    plan_reserve(*a, w);
    return w.used;
}

uzip_status uzip_cache_reserve(const uzip_cache_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status, cudaStream_t s) {
    if (!a || !state_ok(*a, true) || !within(a->tokens, 0, kMost31) || !list_ok(a->list, a->seqs) || !list_ok(a->slots, a->tokens) ||
        !list_ok(a->positions, a->tokens) || !list_ok(a->pairs, 2 * a->seqs))
        return UZIP_ERR_INVALID_ARG;
    Work need{nullptr};
    plan_reserve(*a, need);
    uzip_status st = check_work(need.used, d_workspace, workspace_bytes, d_status);
    if (st != UZIP_OK) return st;
    cudaError_t err = clear_status(d_status, s);
    if (err != cudaSuccess || (a->seqs == 0 && a->tokens == 0)) return finish(err);
    Work work{static_cast<uint8_t*>(d_workspace)};
    Reserve r = plan_reserve(*a, work);
    r.c = state_of(*a, d_status);
    r.counts = a->list, r.tokens = a->tokens, r.slots = a->slots, r.positions = a->positions, r.copies = a->pairs;
    return finish(launch_reserve(r, s));
}

uint64_t uzip_cache_fork_workspace_size(const uzip_cache_args* a) {
    if (!a || !state_ok(*a, false) || a->n < 0 || fork_keeps(a->seqs, a->n, a->width)) return 0;
    Work w{nullptr};
    w.take<int32_t>(a->seqs);
    return w.used;
}
uzip_status uzip_cache_fork(const uzip_cache_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status, cudaStream_t s) {
    return fork(a, d_workspace, workspace_bytes, d_status, s, true);
}
uint64_t uzip_cache_free_workspace_size(const uzip_cache_args* a) { return uzip_cache_fork_workspace_size(a); }
uzip_status uzip_cache_free(const uzip_cache_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status, cudaStream_t s) {
    return fork(a, d_workspace, workspace_bytes, d_status, s, false);
}

uint64_t uzip_cache_compact_workspace_size(const uzip_cache_args* a) {
    if (!a || !state_ok(*a, false)) return 0;
    Work w{nullptr};
    plan_compact(*a, w);
    return w.used;
}
uzip_status uzip_cache_compact(const uzip_cache_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status, cudaStream_t s) {
    if (!a || !state_ok(*a, true) || !list_ok(a->pairs, a->pages / 2 * 2)) return UZIP_ERR_INVALID_ARG;
    Work need{nullptr};
    plan_compact(*a, need);
    uzip_status st = check_work(need.used, d_workspace, workspace_bytes, d_status);
    if (st != UZIP_OK) return st;
    cudaError_t err = clear_status(d_status, s);
    if (err != cudaSuccess || a->pages == 0) return finish(err);
    Work work{static_cast<uint8_t*>(d_workspace)};
    Compact m = plan_compact(*a, work);
    m.c = state_of(*a, d_status);
    m.moves = a->pairs;
    return finish(launch_compact(m, s));
}

uint64_t uzip_cache_copy_workspace_size(const uzip_cache_copy_args*) { return 0; }

uzip_status uzip_cache_copy(const uzip_cache_copy_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status, cudaStream_t s) {
    if (!a) return UZIP_ERR_INVALID_ARG;
    if (!half_type(a->dtype)) return UZIP_ERR_UNSUPPORTED_DTYPE;
    if (a->reserved || !within(a->layers, 0, kMost31) || !pool_sizes_ok(a->from_pages, a->heads, a->page, a->d) ||
        !within(a->to_pages, 0, UZIP_MAX_PAGES) || !within(a->n, 0, kMost31))
        return UZIP_ERR_INVALID_ARG;
    const bool same = a->k == a->k_to && a->v == a->v_to;
    if (!same && (a->k == a->k_to || a->v == a->v_to)) return UZIP_ERR_INVALID_ARG;
    if (a->to_pages && (a->k_to == a->v_to || a->k == a->v_to || a->v == a->k_to)) return UZIP_ERR_INVALID_ARG;
    if (same && a->from_pages != a->to_pages) return UZIP_ERR_INVALID_ARG;
    const Block b[4] = {pool_of(a->k, a->from_pages, a->heads, a->page, {a->k_page, a->k_head, a->k_token}, a->d, a->layers, a->k_layer),
                        pool_of(a->v, a->from_pages, a->heads, a->page, {a->v_page, a->v_head, a->v_token}, a->d, a->layers, a->v_layer),
                        pool_of(a->k_to, a->to_pages, a->heads, a->page, {a->kt_page, a->kt_head, a->kt_token}, a->d, a->layers, a->kt_layer),
                        pool_of(a->v_to, a->to_pages, a->heads, a->page, {a->vt_page, a->vt_head, a->vt_token}, a->d, a->layers, a->vt_layer)};
    if (!b[0].readable(16) || !b[1].readable(16) || !b[2].writable(16) || !b[3].writable(16)) return UZIP_ERR_INVALID_ARG;
    if (same)  // one pool, laid out in one way
        for (int n = 0; n < 4; ++n)
            if (b[0].stride(n) != b[2].stride(n) || b[1].stride(n) != b[3].stride(n)) return UZIP_ERR_INVALID_ARG;
    if (!list_ok(a->pairs, 2 * a->n) || !aligned(a->pairs, 8)) return UZIP_ERR_INVALID_ARG;
    uzip_status st = check_work(0, d_workspace, workspace_bytes, d_status);
    if (st != UZIP_OK) return st;
    cudaError_t err = clear_status(d_status, s);
    if (err != cudaSuccess || a->n == 0) return finish(err);
    PageCopy c{};
    c.k = static_cast<const uint16_t*>(a->k), c.v = static_cast<const uint16_t*>(a->v);
    c.k_to = static_cast<uint16_t*>(a->k_to), c.v_to = static_cast<uint16_t*>(a->v_to);
    // a page as outer x inner runs: the dimension with the larger step outside, dimensions that continue one another
    // in all four pools joined
    const bool token_out = b[0].stride(3) > b[0].stride(2);
    const int out = token_out ? 3 : 2, in = token_out ? 2 : 3;
    int64_t outer = b[0].count[out], inner = b[0].count[in], run = a->d;
    bool inner_joins = true, outer_joins = true;
    for (const Block& x : b) inner_joins &= inner == 1 || x.stride(in) == run;
    if (inner_joins) run *= inner, inner = 1;
    for (const Block& x : b) outer_joins &= outer == 1 || (inner == 1 && x.stride(out) == run);
    if (outer_joins) run *= outer, outer = 1;
    c.outer = int32_t(outer), c.inner = int32_t(inner), c.run = run / 8;
    for (int n = 0; n < 4; ++n) {
        c.layer[n] = b[n].stride(0) / 8, c.page[n] = b[n].stride(1) / 8;
        c.outer_step[n] = b[n].stride(out) / 8, c.inner_step[n] = b[n].stride(in) / 8;
    }
    c.layers = int32_t(a->layers);
    c.pairs = a->pairs, c.n = a->n;
    c.from_pages = int32_t(a->from_pages), c.to_pages = int32_t(a->to_pages);
    c.same = same;
    c.status = d_status;
    return finish(launch_page_copy(c, sm_count(), s));
}

}  // extern "C"
