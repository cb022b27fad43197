// C ABI of the matrix-product operators: argument checks, workspace layout and
// the order of the launches.  Every check that can be made on the host is made
// before anything is enqueued.
#include <algorithm>

#include "product.cuh"

namespace uzip {
bool device_range_ok(const void* p, uint64_t bytes);  // api.cu
}

namespace {

using namespace uzip;

constexpr int64_t kMaxLength = (int64_t(1) << 31) - 1;
// A piece of the vocabulary: at most 512 MiB of softmax gradient, and at most
// 32768 classes, two chunks of a product's depth (product.cu).
constexpr uint64_t kPieceBytes = 512ull << 20, kPieceMost = 32768;

uint64_t round_to(uint64_t v, uint64_t a) { return (v + a - 1) / a * a; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Hands out the workspace in 256-byte steps.  With no base it only measures.
struct Work {
    uint8_t* base;
    uint64_t used = 0;
    template <typename T>
    T* take(uint64_t count) {
        T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
        used += round_to(count * sizeof(T), 256);
        return p;
    }
};

struct Matrix {
    const void* p;
    int64_t ld, group;
    int64_t rows, cols, groups;
    int64_t step() const { return rows > 1 ? ld : int64_t(round_to(cols, 8)); }  // a lone row's stride says nothing
    bool empty() const { return rows == 0 || cols == 0 || groups == 0; }
    uint64_t bytes() const {  // from the first to the last value
        if (empty()) return 0;
        return 2 * (uint64_t(groups - 1) * group + uint64_t(rows - 1) * step() + cols);
    }
    bool shape_ok() const {
        if (rows > 1 && (ld < cols || ld > (int64_t(1) << 36))) return false;
        if (groups > 1 && (group < (rows - 1) * step() + cols || group > (int64_t(1) << 38))) return false;
        return true;
    }
    bool ok() const { return empty() || (p && aligned(p, 2) && shape_ok() && device_range_ok(p, bytes())); }
    // an operand whose rows do not start on 16-byte boundaries is packed first
    bool packed() const {
        return !empty() && (!aligned(p, 16) || step() % 8 != 0 || (groups > 1 && group % 8 != 0));
    }
};

// Operand of a product from matrix `a`, packed in the workspace where needed.
// as_rows: a row of `a` is a row of the operand, else a depth index.
Operand operand(const Matrix& a, bool as_rows, Work& w, PackJobs* packs) {
    const uint64_t group = a.groups > 1 ? a.group : 0;
    if (!a.packed()) return Operand{a.p, uint64_t(a.step()), group, as_rows};
    PackJob& j = packs->job[packs->count++];
    j.from = a.p, j.ld = a.step(), j.group = group;
    j.rows = a.rows, j.cols = a.cols, j.groups = a.groups;
    j.ld_to = round_to(a.cols, 8);
    j.to = w.take<uint16_t>(j.ld_to * j.rows * j.groups);
    return Operand{j.to, j.ld_to, j.ld_to * j.rows, as_rows};
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

bool half_type(int dtype) { return dtype == UZIP_BF16 || dtype == UZIP_FP16; }
bool length_ok(int64_t v) { return v >= 0 && v <= kMaxLength; }

uzip_status finish(cudaError_t err) {
    if (err == cudaSuccess) return UZIP_OK;
    cudaGetLastError();
    return UZIP_ERR_CUDA;
}

uzip_status check_work(const Work& need, void* ws, uint64_t bytes, int32_t* d_status) {
    if (need.used && (!ws || !aligned(ws, 256))) return UZIP_ERR_INVALID_ARG;
    if (bytes < need.used) return UZIP_ERR_CAPACITY;
    if (!device_range_ok(ws, need.used)) return UZIP_ERR_INVALID_ARG;
    if (d_status && (!aligned(d_status, 4) || !device_range_ok(d_status, 4))) return UZIP_ERR_INVALID_ARG;
    return UZIP_OK;
}

// ---- linear -------------------------------------------------------------------

uzip_status check_common(int32_t dtype, int32_t act, int64_t m, int64_t n, int64_t k, int64_t groups,
                         const int64_t* offsets, bool grouped) {
    if (!half_type(dtype)) return UZIP_ERR_UNSUPPORTED_DTYPE;
    if (act < UZIP_ACT_NONE || act > UZIP_ACT_SILU) return UZIP_ERR_INVALID_ARG;
    if (!length_ok(m) || !length_ok(n) || !length_ok(k)) return UZIP_ERR_INVALID_ARG;
    if (!grouped) return groups == 0 && !offsets ? UZIP_OK : UZIP_ERR_INVALID_ARG;
    if (groups < 1 || groups > UZIP_MAX_GROUPS) return UZIP_ERR_INVALID_ARG;
    if (!offsets || !aligned(offsets, 8)) return UZIP_ERR_INVALID_ARG;
    return UZIP_OK;
}

struct Forward {
    Product p{};
    PackJobs packs{};
};

Matrix w_of(const void* w, int64_t ldw, int64_t w_group, int64_t n, int64_t k, int64_t groups) {
    return Matrix{w, ldw, groups ? w_group : 0, n, k, groups ? groups : 1};
}

Forward plan_forward(const uzip_linear_args& a, Work& w, int32_t* d_status) {
    Forward f;
    Product& p = f.p;
    p.a = operand(Matrix{a.x, a.ldx, 0, a.m, a.k, 1}, true, w, &f.packs);
    p.b = operand(w_of(a.w, a.ldw, a.w_group, a.n, a.k, a.groups), true, w, &f.packs);
    p.m = a.m, p.n = a.n, p.depth = a.k;
    p.schedule = a.groups ? kRows : kDense;
    p.groups = a.groups ? uint32_t(a.groups) : 1;
    p.offsets = a.offsets;
    p.epilogue = kStore;
    p.st.out = a.y, p.st.ldo = a.m > 1 ? a.ldy : a.n;
    p.st.bias = a.bias;
    p.st.residual = a.residual, p.st.ldr = a.m > 1 ? a.ldr : a.n;
    p.st.z = a.z, p.st.ldz = a.m > 1 ? a.ldz : a.n;
    p.st.act = a.act;
    p.dtype = a.dtype;
    p.status = d_status;
    return f;
}

uzip_status forward(const uzip_linear_args* a, void* ws, uint64_t bytes, int32_t* d_status, cudaStream_t s,
                    bool grouped) {
    if (!a) return UZIP_ERR_INVALID_ARG;
    uzip_status st = check_common(a->dtype, a->act, a->m, a->n, a->k, a->groups, a->offsets, grouped);
    if (st != UZIP_OK) return st;
    const int64_t g = a->groups ? a->groups : 1;
    const bool some = a->m > 0 && a->n > 0;
    Matrix x{a->x, a->ldx, 0, a->m, a->k, 1}, y{a->y, a->ldy, 0, a->m, a->n, 1}, z{a->z, a->ldz, 0, a->m, a->n, 1},
        r{a->residual, a->ldr, 0, a->m, a->n, 1}, b{a->bias, a->n, a->n, g, a->n, 1};
    if (!x.ok() || !w_of(a->w, a->ldw, a->w_group, a->n, a->k, a->groups).ok() || !y.ok() || (a->z && !z.ok()) ||
        (a->residual && !r.ok()) || (a->bias && !b.ok()) ||
        (grouped && !device_range_ok(a->offsets, 8 * uint64_t(g + 1))))
        return UZIP_ERR_INVALID_ARG;
    Work need{nullptr};
    plan_forward(*a, need, nullptr);
    if ((st = check_work(need, ws, bytes, d_status)) != UZIP_OK) return st;
    Work work{static_cast<uint8_t*>(ws)};
    const Forward f = plan_forward(*a, work, d_status);
    cudaError_t err = cudaSuccess;
    if (d_status) err = cudaMemsetAsync(d_status, 0, sizeof(int32_t), s);
    if (err == cudaSuccess && some) {
        err = launch_pack(f.packs, s);
        if (err == cudaSuccess) err = launch_product(f.p, sm_count(), s);
    } else if (err == cudaSuccess && grouped)
        err = launch_offset_check(a->offsets, g, a->m, d_status, s);
    return finish(err);
}

struct Backward {
    ActGrad grad{};
    Product dx{}, dw{};
    PackJobs packs{};
    bool need_grad;
};

Backward plan_backward(const uzip_linear_grad_args& a, Work& w, int32_t* d_status) {
    Backward f;
    const uint32_t groups = a.groups ? uint32_t(a.groups) : 1;
    const Matrix dy{a.dy, a.lddy, 0, a.m, a.n, 1};
    const bool products = a.dx || a.dw;
    Operand dz_rows{}, dz_depth{};
    f.need_grad = a.db || (products && a.act != UZIP_ACT_NONE);
    if (f.need_grad) {
        ActGrad& q = f.grad;
        q.dy = a.dy, q.lddy = dy.step();
        q.z = a.z, q.ldz = a.m > 1 ? a.ldz : a.n;
        q.m = a.m, q.n = a.n;
        q.act = a.act, q.dtype = a.dtype, q.status = d_status;
        const bool by_group = a.db && a.groups;
        q.groups = by_group ? groups : 1;
        q.offsets = by_group ? a.offsets : nullptr;
        q.splits = act_grad_splits(a.m, a.n, q.groups);
        q.db = a.db;
        if (a.db && q.splits > 1) q.part = w.take<float>(uint64_t(q.groups) * q.splits * a.n);
        if (products && (a.act != UZIP_ACT_NONE || dy.packed())) {
            q.lddz = round_to(a.n, 8);
            q.dz = w.take<uint16_t>(q.lddz * a.m);
            dz_rows = Operand{q.dz, q.lddz, 0, 1};
        }
    }
    if (products && !dz_rows.ld) dz_rows = operand(dy, true, w, &f.packs);
    dz_depth = dz_rows;
    dz_depth.depth_major = 0;
    if (a.dx) {
        Product& p = f.dx;
        p.a = dz_rows;
        p.b = operand(w_of(a.w, a.ldw, a.w_group, a.n, a.k, a.groups), false, w, &f.packs);
        p.m = a.m, p.n = a.k, p.depth = a.n;
        p.schedule = a.groups ? kRows : kDense;
        p.groups = groups, p.offsets = a.offsets;
        p.st.out = a.dx, p.st.ldo = a.m > 1 ? a.lddx : a.k;
        p.dtype = a.dtype, p.status = d_status;
    }
    if (a.dw) {
        Product& p = f.dw;
        p.a = dz_depth;
        p.b = operand(Matrix{a.x, a.ldx, 0, a.m, a.k, 1}, false, w, &f.packs);
        p.m = a.n, p.n = a.k, p.depth = a.m;
        p.schedule = a.groups ? kDepth : kDense;
        p.groups = groups, p.offsets = a.offsets;
        p.st.out = a.dw, p.st.ldo = a.n > 1 ? a.lddw : a.k, p.st.out_group = a.groups ? a.dw_group : 0;
        p.dtype = a.dtype, p.status = d_status;
    }
    return f;
}

uzip_status backward(const uzip_linear_grad_args* a, void* ws, uint64_t bytes, int32_t* d_status, cudaStream_t s,
                     bool grouped) {
    if (!a) return UZIP_ERR_INVALID_ARG;
    uzip_status st = check_common(a->dtype, a->act, a->m, a->n, a->k, a->groups, a->offsets, grouped);
    if (st != UZIP_OK) return st;
    const int64_t g = a->groups ? a->groups : 1;
    const Matrix dy{a->dy, a->lddy, 0, a->m, a->n, 1}, z{a->z, a->ldz, 0, a->m, a->n, 1},
        x{a->x, a->ldx, 0, a->m, a->k, 1}, dx{a->dx, a->lddx, 0, a->m, a->k, 1},
        dw{a->dw, a->lddw, a->dw_group, a->n, a->k, g}, db{a->db, a->n, 0, g, a->n, 1};
    if (!dy.ok() || (a->act != UZIP_ACT_NONE && !z.ok()) || (a->dw && !x.ok()) || (a->dx && !dx.ok()) ||
        (a->dx && !w_of(a->w, a->ldw, a->w_group, a->n, a->k, a->groups).ok()) || (a->dw && !dw.ok()) ||
        (a->db && !db.ok()) || (grouped && !device_range_ok(a->offsets, 8 * uint64_t(g + 1))))
        return UZIP_ERR_INVALID_ARG;
    Work need{nullptr};
    plan_backward(*a, need, nullptr);
    if ((st = check_work(need, ws, bytes, d_status)) != UZIP_OK) return st;
    Work work{static_cast<uint8_t*>(ws)};
    const Backward f = plan_backward(*a, work, d_status);
    cudaError_t err = cudaSuccess;
    if (d_status) err = cudaMemsetAsync(d_status, 0, sizeof(int32_t), s);
    if (err == cudaSuccess && f.need_grad) err = launch_act_grad(f.grad, s);
    if (err == cudaSuccess) err = launch_pack(f.packs, s);
    if (err == cudaSuccess && a->dx) err = launch_product(f.dx, sm_count(), s);
    if (err == cudaSuccess && a->dw) err = launch_product(f.dw, sm_count(), s);
    // the products and the bias gradient check the offsets themselves
    const bool checked = (a->dx && a->m && a->k) || (a->dw && a->n && a->k) || (a->db && a->n);
    if (err == cudaSuccess && grouped && !checked) err = launch_offset_check(a->offsets, g, a->m, d_status, s);
    return finish(err);
}

// ---- cross entropy --------------------------------------------------------------

// Tokens up to one tile of rows are taken as they are: leaving the ignored ones
// out would save nothing.  More are moved together first, which costs one pass
// over h (12 us for 4096 x 4096, against 2.3 ms of products) and saves the
// ignored tokens' share of the products.
constexpr int64_t kMoveAbove = 128;

struct Loss {
    Product p{};
    PackJobs packs{};
    LossRows rows{};
    bool moved;
};

LossRows plan_rows(const void* h, int64_t ldh, const int64_t* targets, int64_t ignore, int64_t t, int64_t v, int64_t d, int dtype,
                   Work& w, int32_t* d_status) {
    LossRows r{};
    r.h = h, r.ldh = t > 1 ? ldh : round_to(d, 8);
    r.targets = targets, r.ignore = ignore;
    r.t = t, r.v = v, r.d = d, r.dtype = dtype, r.status = d_status;
    r.ld_out = round_to(d, 8);
    r.out_h = w.take<uint16_t>(t * r.ld_out);
    r.out_targets = w.take<int64_t>(t);
    r.token = w.take<uint32_t>(t);
    r.count = w.take<uint32_t>(1);
    return r;
}

Loss plan_loss(const uzip_cross_entropy_args& a, Work& w, int32_t* d_status) {
    Loss f;
    Product& p = f.p;
    f.moved = a.t > kMoveAbove;
    if (f.moved) {
        f.rows = plan_rows(a.h, a.ldh, a.targets, a.ignore_index, a.t, a.v, a.d, a.dtype, w, d_status);
        f.rows.loss = a.loss, f.rows.zero_lse = a.lse;
        p.a = Operand{f.rows.out_h, f.rows.ld_out, 0, 1};
        p.live_rows = f.rows.count;
    } else {
        p.a = operand(Matrix{a.h, a.ldh, 0, a.t, a.d, 1}, true, w, &f.packs);
    }
    p.b = operand(Matrix{a.w, a.ldw, 0, a.v, a.d, 1}, true, w, &f.packs);
    p.m = a.t, p.n = a.v, p.depth = a.d;
    p.schedule = kDense, p.groups = 1, p.epilogue = kLossStats;
    p.dtype = a.dtype, p.status = d_status;
    p.ls.tiles = uint32_t((a.v + kStatsCols - 1) / kStatsCols);
    p.ls.targets = f.moved ? f.rows.out_targets : a.targets, p.ls.ignore = a.ignore_index;
    p.ls.part = w.take<float2>(uint64_t(p.ls.tiles) * a.t);
    p.ls.hit = w.take<float>(a.t);
    return f;
}

struct LossGradPlan {
    uint64_t piece, pieces, ld_piece;
    LossRows rows;
    float* sum;
    uint64_t ld_sum;
    void* dl;
    Operand h_rows, w_rows;
    PackJobs packs;
};

LossGradPlan plan_loss_grad(const uzip_cross_entropy_grad_args& a, Work& w, int32_t* d_status) {
    LossGradPlan f{};
    const uint64_t t = a.t, v = a.v;
    uint64_t piece = a.piece;
    if (piece == 0) piece = std::min(kPieceMost, std::max<uint64_t>(256, kPieceBytes / 2 / std::max<uint64_t>(1, t) / 256 * 256));
    if (piece >= v) piece = v;
    else piece = round_to(piece, 8);  // every piece starts on a 16-byte boundary of a gradient row
    f.piece = piece;
    f.pieces = (v + piece - 1) / piece;
    f.ld_piece = round_to(piece, 8);
    f.rows = plan_rows(a.h, a.ldh, a.targets, a.ignore_index, a.t, a.v, a.d, a.dtype, w, d_status);
    f.rows.dloss = a.dloss, f.rows.lse = a.lse;
    f.rows.out_lse = w.take<float>(t);
    f.rows.out_g = w.take<float>(t);
    f.rows.scale = w.take<float>(1);
    f.rows.place = w.take<uint32_t>(t);
    f.h_rows = Operand{f.rows.out_h, f.rows.ld_out, 0, 1};
    f.w_rows = operand(Matrix{a.w, a.ldw, 0, a.v, a.d, 1}, true, w, &f.packs);
    f.dl = w.take<uint16_t>(t * f.ld_piece);
    f.ld_sum = round_to(a.d, 4);
    if (a.dh && f.pieces > 1) f.sum = w.take<float>(t * f.ld_sum);
    return f;
}

cudaError_t run_loss_grad(const uzip_cross_entropy_grad_args& a, const LossGradPlan& f, int32_t* d_status,
                          cudaStream_t s) {
    cudaError_t err = launch_pack(f.packs, s);
    if (err == cudaSuccess) err = launch_loss_rows(f.rows, s);
    for (uint64_t i = 0; i < f.pieces && err == cudaSuccess; ++i) {
        const uint64_t col0 = i * f.piece, cols = std::min<uint64_t>(f.piece, a.v - col0);
        Operand w_rows = f.w_rows;
        w_rows.p = static_cast<const uint16_t*>(w_rows.p) + col0 * w_rows.ld;
        Product p{};
        p.dtype = a.dtype, p.status = d_status, p.groups = 1;
        p.a = f.h_rows, p.b = w_rows;
        p.m = a.t, p.n = cols, p.depth = a.d;
        p.live_rows = f.rows.count;
        p.epilogue = kLossGrad;
        p.ls.targets = f.rows.out_targets, p.ls.ignore = a.ignore_index, p.ls.col0 = col0;
        p.ls.lse = f.rows.out_lse, p.ls.g = f.rows.out_g, p.ls.out = f.dl, p.ls.ldo = f.ld_piece;
        err = launch_product(p, sm_count(), s);
        if (err == cudaSuccess && a.dw) {
            Product q{};
            q.dtype = a.dtype, q.status = d_status, q.groups = 1;
            q.a = Operand{f.dl, f.ld_piece, 0, 0};
            q.b = f.h_rows;
            q.b.depth_major = 0;
            q.m = cols, q.n = a.d, q.depth = a.t;
            q.live_depth = f.rows.count;
            const uint64_t ldo = a.v > 1 ? a.lddw : a.d;
            q.st.out = static_cast<uint16_t*>(a.dw) + col0 * ldo, q.st.ldo = ldo;
            q.st.alpha = f.rows.scale;
            err = launch_product(q, sm_count(), s);
        }
        if (err == cudaSuccess && a.dh) {
            Product q{};
            q.dtype = a.dtype, q.status = d_status, q.groups = 1;
            q.a = Operand{f.dl, f.ld_piece, 0, 1};
            q.b = w_rows;
            q.b.depth_major = 0;
            q.m = a.t, q.n = a.d, q.depth = cols;
            q.live_rows = f.rows.count;
            q.st.sum_in = i ? f.sum : nullptr, q.st.ld_sum = f.ld_sum;
            if (i + 1 < f.pieces) {
                q.st.out = f.sum, q.st.ldo = f.ld_sum, q.st.out_fp32 = 1;
            } else {
                q.st.out = f.rows.out_h, q.st.ldo = f.rows.ld_out;  // h has been read for the last time
            }
            q.st.alpha = f.rows.scale;
            err = launch_product(q, sm_count(), s);
        }
    }
    if (err == cudaSuccess && a.dh)
        err = launch_spread_rows(f.rows.out_h, f.rows.ld_out, f.rows.place, a.dh, a.t > 1 ? a.lddh : a.d, a.t, a.d, s);
    return err;
}

uzip_status check_loss(int32_t dtype, int32_t reserved, int64_t t, int64_t v, int64_t d, const int64_t* targets) {
    if (!half_type(dtype)) return UZIP_ERR_UNSUPPORTED_DTYPE;
    if (reserved != 0 || !length_ok(t) || !length_ok(v) || !length_ok(d) || v == 0) return UZIP_ERR_INVALID_ARG;
    if (t && (!targets || !aligned(targets, 8) || !device_range_ok(targets, 8 * uint64_t(t)))) return UZIP_ERR_INVALID_ARG;
    return UZIP_OK;
}

bool floats_ok(const float* p, int64_t count) {
    return count == 0 || (p && aligned(p, 4) && device_range_ok(p, 4 * uint64_t(count)));
}

}  // namespace

extern "C" {

uint64_t uzip_linear_workspace_size(const uzip_linear_args* a) {
    if (!a || check_common(a->dtype, a->act, a->m, a->n, a->k, a->groups, a->offsets, false) != UZIP_OK) return 0;
    Work w{nullptr};
    plan_forward(*a, w, nullptr);
    return w.used;
}

uzip_status uzip_linear(const uzip_linear_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status,
                        cudaStream_t s) {
    return forward(a, d_workspace, workspace_bytes, d_status, s, false);
}

uint64_t uzip_grouped_linear_workspace_size(const uzip_linear_args* a) {
    if (!a || check_common(a->dtype, a->act, a->m, a->n, a->k, a->groups, a->offsets, true) != UZIP_OK) return 0;
    Work w{nullptr};
    plan_forward(*a, w, nullptr);
    return w.used;
}

uzip_status uzip_grouped_linear(const uzip_linear_args* a, void* d_workspace, uint64_t workspace_bytes,
                                int32_t* d_status, cudaStream_t s) {
    return forward(a, d_workspace, workspace_bytes, d_status, s, true);
}

uint64_t uzip_linear_backward_workspace_size(const uzip_linear_grad_args* a) {
    if (!a || check_common(a->dtype, a->act, a->m, a->n, a->k, a->groups, a->offsets, false) != UZIP_OK) return 0;
    Work w{nullptr};
    plan_backward(*a, w, nullptr);
    return w.used;
}

uzip_status uzip_linear_backward(const uzip_linear_grad_args* a, void* d_workspace, uint64_t workspace_bytes,
                                 int32_t* d_status, cudaStream_t s) {
    return backward(a, d_workspace, workspace_bytes, d_status, s, false);
}

uint64_t uzip_grouped_linear_backward_workspace_size(const uzip_linear_grad_args* a) {
    if (!a || check_common(a->dtype, a->act, a->m, a->n, a->k, a->groups, a->offsets, true) != UZIP_OK) return 0;
    Work w{nullptr};
    plan_backward(*a, w, nullptr);
    return w.used;
}

uzip_status uzip_grouped_linear_backward(const uzip_linear_grad_args* a, void* d_workspace, uint64_t workspace_bytes,
                                         int32_t* d_status, cudaStream_t s) {
    return backward(a, d_workspace, workspace_bytes, d_status, s, true);
}

uint64_t uzip_cross_entropy_workspace_size(const uzip_cross_entropy_args* a) {
    if (!a || !half_type(a->dtype) || a->t <= 0 || !length_ok(a->t) || a->v <= 0 || !length_ok(a->v) || !length_ok(a->d))
        return 0;
    Work w{nullptr};
    plan_loss(*a, w, nullptr);
    return w.used;
}

uzip_status uzip_cross_entropy(const uzip_cross_entropy_args* a, void* d_workspace, uint64_t workspace_bytes,
                               int32_t* d_status, cudaStream_t s) {
    if (!a) return UZIP_ERR_INVALID_ARG;
    uzip_status st = check_loss(a->dtype, a->reserved, a->t, a->v, a->d, a->targets);
    if (st != UZIP_OK) return st;
    const Matrix h{a->h, a->ldh, 0, a->t, a->d, 1}, wm{a->w, a->ldw, 0, a->v, a->d, 1};
    if (!h.ok() || !wm.ok() || !floats_ok(a->loss, a->t) || !floats_ok(a->lse, a->t)) return UZIP_ERR_INVALID_ARG;
    Work need{nullptr};
    if (a->t) plan_loss(*a, need, nullptr);
    if ((st = check_work(need, d_workspace, workspace_bytes, d_status)) != UZIP_OK) return st;
    cudaError_t err = cudaSuccess;
    if (d_status) err = cudaMemsetAsync(d_status, 0, sizeof(int32_t), s);
    if (err != cudaSuccess || a->t == 0) return finish(err);
    Work work{static_cast<uint8_t*>(d_workspace)};
    const Loss f = plan_loss(*a, work, d_status);
    err = launch_pack(f.packs, s);
    if (err == cudaSuccess && f.moved) err = launch_loss_rows(f.rows, s);
    if (err == cudaSuccess) err = launch_product(f.p, sm_count(), s);
    if (err == cudaSuccess)
        err = launch_loss_join(f.p.ls, f.moved ? f.rows.token : nullptr, f.moved ? f.rows.count : nullptr, a->t, a->v, a->loss,
                               a->lse, d_status, s);
    return finish(err);
}

uint64_t uzip_cross_entropy_backward_workspace_size(const uzip_cross_entropy_grad_args* a) {
    if (!a || !half_type(a->dtype) || a->t <= 0 || !length_ok(a->t) || a->v <= 0 || !length_ok(a->v) ||
        !length_ok(a->d) || a->piece < 0)
        return 0;
    Work w{nullptr};
    plan_loss_grad(*a, w, nullptr);
    return w.used;
}

uzip_status uzip_cross_entropy_backward(const uzip_cross_entropy_grad_args* a, void* d_workspace,
                                        uint64_t workspace_bytes, int32_t* d_status, cudaStream_t s) {
    if (!a) return UZIP_ERR_INVALID_ARG;
    uzip_status st = check_loss(a->dtype, a->reserved, a->t, a->v, a->d, a->targets);
    if (st != UZIP_OK) return st;
    const Matrix h{a->h, a->ldh, 0, a->t, a->d, 1}, wm{a->w, a->ldw, 0, a->v, a->d, 1},
        dh{a->dh, a->lddh, 0, a->t, a->d, 1}, dw{a->dw, a->lddw, 0, a->v, a->d, 1};
    if (a->piece < 0 || !h.ok() || !wm.ok() || (a->dh && !dh.ok()) || (a->dw && !dw.ok()) ||
        !floats_ok(a->lse, a->t) || !floats_ok(a->dloss, a->t))
        return UZIP_ERR_INVALID_ARG;
    Work need{nullptr};
    if (a->t) plan_loss_grad(*a, need, nullptr);
    if ((st = check_work(need, d_workspace, workspace_bytes, d_status)) != UZIP_OK) return st;
    cudaError_t err = cudaSuccess;
    if (d_status) err = cudaMemsetAsync(d_status, 0, sizeof(int32_t), s);
    if (err != cudaSuccess) return finish(err);
    if (a->t == 0) {
        if (a->dw) err = launch_clear(a->dw, a->v > 1 ? a->lddw : a->d, a->v, a->d, s);
        return finish(err);
    }
    Work work{static_cast<uint8_t*>(d_workspace)};
    const LossGradPlan f = plan_loss_grad(*a, work, d_status);
    return finish(run_loss_grad(*a, f, d_status, s));
}

}  // extern "C"
