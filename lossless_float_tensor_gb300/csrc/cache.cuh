// Definitions shared by the sources of the paged key-value cache: what each
// launch is given, and how kernels are launched one after another.
#pragma once

#include "../../include/uzip_cache.h"
#include "product.cuh"

namespace uzip {

// A launch whose blocks may be set up while the one before it ends: the kernel
// starts with wait_for_launch_before().
template <typename... Args, typename... Given>
cudaError_t launch_next(void (*kernel)(Args...), dim3 grid, uint32_t threads, uint32_t smem, uint32_t cluster, cudaStream_t s,
                        Given... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, Args(args)...);
}

// Strides of a pool in elements: from page to page, head to head, token to token.
struct PoolStrides {
    int64_t page, head, token;
};

// ---- attention ----------------------------------------------------------------

struct Attention {
    const uint16_t *q, *k, *v;
    int64_t q_row, q_head;
    PoolStrides ks, vs;  // in bytes
    const int32_t* table;
    int64_t ldt;
    const int32_t* lengths;
    int32_t seqs, q_heads, group, d, pages, page;
    int32_t blocks;      // groups of kept heads: a key head's query heads are taken 8, 16 or 32 at a time
    int32_t pairs;       // kv_heads * blocks: rows of work of a sequence
    int32_t most;        // tokens that a sequence's row of the table holds (capped to int32)
    int32_t window;      // 0: none
    uint32_t page_by;    // t / page = t * page_by >> page_shift for t below 2^31
    int32_t page_shift;
    int32_t q_pairs;     // whether neighbouring values of q may be read together
    int32_t alike;       // whether keys and values have the same strides
    int32_t out_quads;   // whether four neighbouring results may be written together
    int32_t skip_seq, skip_row;  // whole rows: from a block's row to its next, in sequences and rows of one
    int32_t cut;         // whether a sequence's tokens may be cut between blocks
    float scale, cap;    // times log2 e: exponentials are powers of 2
    float per_cap;       // the scale over the cap
    uint16_t* out;
    int64_t out_row, out_head;
    float* lse;
    float* part_o;       // [2 grid][kept heads][d] sums over a part of a sequence's tokens
    float2* part_ml;     // [2 grid][kept heads]: largest score (times log2 e), sum of exponentials (fp16: times 2^15)
    int4* record;        // [grid]: what a border between two blocks cuts
    int2* row_record;    // [rows]: first (-1: not cut) and last block; null where there are many rows
    int32_t* status;
};

struct AttentionPlan {
    uint32_t grid;   // blocks
    uint32_t heads;  // kept heads: 8, 16 or 32
    bool cut;
    int64_t by_row;  // rows, where they are few and joined one by one; else 0
};
// what goes by sizes alone, for the workspace and the launch
AttentionPlan plan_attention(int64_t seqs, int64_t kv_heads, int64_t group, int64_t d, int64_t most, int sms);
cudaError_t launch_attention(const Attention& a, int dtype, const AttentionPlan& plan, cudaStream_t s);

// ---- rotary positions -----------------------------------------------------------

struct RotarySegment {  // queries, keys or values of every token
    const uint16_t* from;
    int64_t row, head;
    uint16_t* to;
    int64_t to_row, to_head;  // where paged: strides of the pool
    int64_t to_token;
    int32_t heads;
    int32_t turned, paged;
};

struct Rotary {
    RotarySegment seg[3];
    const int64_t* positions;
    const double* freqs;
    const int64_t* slots;
    int64_t t, slot_count;
    int32_t heads;  // of all segments
    int32_t d, half, page;
    float scale, sign;
    int32_t* status;
};
cudaError_t launch_rotary(const Rotary& r, int dtype, bool interleaved, int sms, cudaStream_t s);

// ---- pages ------------------------------------------------------------------------

struct CacheState {
    int32_t* refs;
    int32_t* table;
    int64_t ldt;
    int32_t* lengths;
    int32_t pages, page, seqs, width;
    int32_t* status;
};
struct Reserve {
    CacheState c;
    const int32_t* counts;
    int64_t tokens;
    int64_t *slots, *positions;
    int32_t* copies;
    // workspace, or null where reserve_keeps()
    int32_t* first;   // [seqs] new pages of the sequences before
    int64_t* begin;   // [seqs] new tokens of the sequences before
    int32_t* before;  // [seqs] length before
    int32_t* held;    // [seqs] pages before, ~ of it where the last is copied
    int32_t* fresh;   // [list] pages taken, ascending
    int64_t list;
};
bool reserve_keeps(int64_t seqs, int64_t pages, int64_t tokens, int64_t list);
cudaError_t launch_reserve(const Reserve& r, cudaStream_t s);
struct Fork {
    CacheState c;
    const int32_t *parents, *children;  // parents null: free the children
    int64_t n;
    int32_t* mark;  // [seqs] workspace, or null where fork_keeps()
};
bool fork_keeps(int64_t seqs, int64_t n, int64_t width);
cudaError_t launch_fork(const Fork& f, cudaStream_t s);
struct Compact {
    CacheState c;
    int32_t* moves;
    int32_t *holes, *movers;  // [pages / 2]
    int32_t* to;              // [pages]
};
cudaError_t launch_compact(const Compact& m, cudaStream_t s);

struct PageCopy {
    const uint16_t *k, *v;
    uint16_t *k_to, *v_to;
    // strides in 16-byte units; a page is `outer` x `inner` runs of `run` units
    int64_t layer[4], page[4], outer_step[4], inner_step[4];  // k, v, k_to, v_to
    int32_t layers, outer, inner;
    int64_t run;
    const int32_t* pairs;
    int64_t n;
    int32_t from_pages, to_pages;
    int32_t same;
    int32_t* status;
};
cudaError_t launch_page_copy(const PageCopy& c, int sms, cudaStream_t s);

}  // namespace uzip
