/*
 * uzip -- the paged key-value cache of a language model (C ABI).
 *
 * What a prompt server sends and a token server reads: keys and values in pages
 * of a pool, a table of pages for each sequence, and reference counts, so that
 * sequences share what they have in common.
 *   uzip_rotary            rotary positions of queries and keys, and (backward) their gradients
 *   uzip_rotary_append     the same, with keys and values stored into the cache's pages
 *   uzip_paged_attention   attention of one new token of each sequence over its pages
 *   uzip_cache_reserve     pages and slots for new tokens, copying shared pages on write
 *   uzip_cache_fork, uzip_cache_free   sequences that share another's pages; sequences given up
 *   uzip_cache_compact     used pages moved to the front of the pool
 *   uzip_cache_copy        pages copied within a pool or to another one (a buffer to compress and send)
 *
 * The cache.  A pool holds `pages` pages of `page` tokens for `heads` heads of
 * `d` values, in bf16 or fp16: token o of page p and head h starts
 * p * *_page + h * *_head + o * *_token elements into the pool.  d is a
 * multiple of 8, at most 256; pools start on 16-byte boundaries and their
 * strides are multiples of 8 elements.  State of a cache, in device memory:
 * refs int32 [pages] (0: free), table int32 [seqs, width] with rows ldt apart,
 * lengths int32 [seqs].  Token t of sequence i lies in page table[i, t / page]
 * at t % page, its slot is table[i, t / page] * page + t % page; the entries of
 * a row behind its last token mean nothing.
 *
 * Common rules, as of uzip_ops.h: the caller gives every buffer; workspaces of
 * uzip_*_workspace_size(args) bytes, 256-byte aligned (NULL where that is 0),
 * used until the call's work on the stream ends; outputs overlap neither inputs
 * nor each other (but see uzip_rotary); calls that share no output and no
 * workspace may overlap; the same inputs give the same bits.  d_status
 * (device i32, nullable) receives 0 or a uzip_status found on the device.
 */
#ifndef UZIP_CACHE_H
#define UZIP_CACHE_H

#include "uzip.h"

#ifdef __cplusplus
extern "C" {
#endif

#define UZIP_MAX_HEAD 256       /* values of a head in a cache */
#define UZIP_MAX_SEQS 65536     /* sequences of a cache */
#define UZIP_MAX_PAGES 1572864  /* pages of a pool that uzip_cache_copy writes */

/* Rotary positions.  The first `rot` (even) values of each head are rotated in
 * pairs, by the angle positions[i] * freqs[j] of token i and pair j, and
 * multiplied by `scale`; the others are copied.  Pair j is (j, j + rot / 2), or
 * (2 j, 2 j + 1) where `interleaved`.  Angles are reduced exactly in 64-bit
 * fixed point from the frequencies in fp64 (radians per position): for
 * frequencies up to a turn they are off by less than 2^-32 + |position| 2^-62 of
 * a turn, so positions of any length of text lose nothing; results are rounded once.  `backward` rotates by the
 * opposite angle: the gradient of the rotation.
 *
 * q is [t, q_heads, d], k and v [t, kv_heads, d], each with any row and head
 * stride (elements), any alignment, d up to 1024 (256 for uzip_rotary_append).  Either of q
 * and k may be absent (q_heads or kv_heads 0 in uzip_rotary).  An output may be
 * its own input (same pointer and strides); other overlap is not allowed.
 *
 * uzip_rotary writes q_out and k_out.  uzip_rotary_append writes q_out, and the
 * rotated k and v into the pages at slots[i] (int64; no two equal).  A slot of
 * -1 stores nothing; one outside [-1, pages * page) stores nothing and is
 * reported as UZIP_ERR_INVALID_ARG in d_status. */
typedef struct {
    int32_t dtype;
    int32_t interleaved; /* 0 or 1 */
    int32_t backward;    /* 0 or 1 */
    float scale;
    int64_t t, q_heads, kv_heads, d, rot;
    const int64_t* positions; /* [t] */
    const double* freqs;      /* [rot / 2], finite */
    const void* q;
    int64_t q_row, q_head;
    const void* k;
    int64_t k_row, k_head;
    const void* v; /* uzip_rotary_append */
    int64_t v_row, v_head;
    void* q_out;
    int64_t q_out_row, q_out_head;
    void* k_out; /* uzip_rotary */
    int64_t k_out_row, k_out_head;
    int64_t pages, page; /* uzip_rotary_append, and what follows */
    void* k_pages;
    int64_t kp_page, kp_head, kp_token;
    void* v_pages;
    int64_t vp_page, vp_head, vp_token;
    const int64_t* slots; /* [t] */
} uzip_rotary_args;

uint64_t uzip_rotary_workspace_size(const uzip_rotary_args* a); /* 0 */
uzip_status uzip_rotary(const uzip_rotary_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status,
                        cudaStream_t s);
uint64_t uzip_rotary_append_workspace_size(const uzip_rotary_args* a); /* 0 */
uzip_status uzip_rotary_append(const uzip_rotary_args* a, void* d_workspace, uint64_t workspace_bytes,
                               int32_t* d_status, cudaStream_t s);

/* Attention of one new token of each sequence: for query head h of sequence i,
 * with z_t = scale q . k_t over the keys of head h / (q_heads / kv_heads),
 * capped to softcap tanh(z_t / softcap) where softcap > 0, and t from
 * max(0, lengths[i] - window) (0 where window is 0) to lengths[i] - 1,
 *   out = sum_t softmax(z)_t v_t,  lse = log sum_t exp(z_t).
 * The new token's own key and value are in the cache and count in its length.
 * A sequence of length 0 gives zeros and an lse of -inf.  Products are summed in
 * 32 bits; the exponentials are rounded to the dtype for the second product, each
 * by half a step of itself (fp16: the largest is 2^15 there, so weights down to
 * 2^-29 of it keep all digits; those below 2^-40 of it are lost).
 * Values of a page behind a sequence's last token, or before its window, are
 * never used, whatever they hold.  A length outside [0, width * page] or a page
 * outside [0, pages) among those used gives NaN for that sequence and is
 * reported as UZIP_ERR_INVALID_ARG. */
typedef struct {
    int32_t dtype;
    int32_t reserved; /* 0 */
    int64_t seqs, q_heads, kv_heads, d;
    int64_t pages, page, width;
    const void* q; /* [seqs, q_heads, d] */
    int64_t q_row, q_head;
    const void* k_pages;
    int64_t kp_page, kp_head, kp_token;
    const void* v_pages;
    int64_t vp_page, vp_head, vp_token;
    const int32_t* table;
    int64_t ldt;
    const int32_t* lengths;
    float scale, softcap;
    int64_t window;
    void* out; /* [seqs, q_heads, d] */
    int64_t out_row, out_head;
    float* lse; /* [seqs, q_heads] contiguous, nullable */
} uzip_paged_attention_args;

uint64_t uzip_paged_attention_workspace_size(const uzip_paged_attention_args* a);
uzip_status uzip_paged_attention(const uzip_paged_attention_args* a, void* d_workspace, uint64_t workspace_bytes,
                                 int32_t* d_status, cudaStream_t s);

/* State of a cache and what an operation on it takes and gives.  Lists hold
 * indexes of sequences; an entry of -1 stands for none.  An operation that is
 * refused on the device (UZIP_ERR_INVALID_ARG for an index, a length, a count, a
 * page or a reference count that cannot be; UZIP_ERR_CAPACITY where pages or
 * columns of the table run out) changes nothing of the state, and its outputs
 * are -1 throughout (positions 0).
 *
 * uzip_cache_reserve: counts[i] new tokens for each sequence (int32, seqs of
 * them).  Their pages are the lowest free ones, in the order of the sequences
 * and of their tokens.  A sequence with new tokens whose last page is part full
 * and shared gets a page in its place first, and copies[i] = {old, new} (else
 * {-1, -1}) for uzip_cache_copy.  slots and positions (int64, `tokens` of them)
 * are those of the new tokens, by sequence; entries behind the last are -1 and 0.
 * Counts that add up to more than `tokens` are refused.
 *
 * uzip_cache_fork: children[j] becomes a sequence with the pages and the length
 * of parents[j] (n of each).  A child is empty before (length 0), is listed once
 * and is nobody's parent in the call.
 *
 * uzip_cache_free: the n sequences listed (each once) become empty.
 *
 * uzip_cache_compact: with K used pages, the i-th used page from K on becomes
 * the i-th free page below K.  moves [pages / 2] of {from, to}, -1 behind the
 * last, are for uzip_cache_copy. */
typedef struct {
    int64_t pages, page, seqs, width;
    int32_t* refs;
    int32_t* table;
    int64_t ldt;
    int32_t* lengths;
    int64_t n;              /* fork, free: entries of the lists */
    const int32_t* from;    /* fork: parents */
    const int32_t* list;    /* fork: children; free: sequences; reserve: counts */
    int64_t tokens;         /* reserve */
    int64_t* slots;         /* reserve */
    int64_t* positions;     /* reserve */
    int32_t* pairs;         /* reserve: copies [seqs, 2]; compact: moves [pages / 2, 2] */
} uzip_cache_args;

uint64_t uzip_cache_reserve_workspace_size(const uzip_cache_args* a);
uzip_status uzip_cache_reserve(const uzip_cache_args* a, void* d_workspace, uint64_t workspace_bytes,
                               int32_t* d_status, cudaStream_t s);
uint64_t uzip_cache_fork_workspace_size(const uzip_cache_args* a);
uzip_status uzip_cache_fork(const uzip_cache_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status,
                            cudaStream_t s);
uint64_t uzip_cache_free_workspace_size(const uzip_cache_args* a);
uzip_status uzip_cache_free(const uzip_cache_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status,
                            cudaStream_t s);
uint64_t uzip_cache_compact_workspace_size(const uzip_cache_args* a);
uzip_status uzip_cache_compact(const uzip_cache_args* a, void* d_workspace, uint64_t workspace_bytes,
                               int32_t* d_status, cudaStream_t s);

/* pairs [n] of int32 {from, to}: page `from` of the source becomes page `to` of
 * the destination, for every layer (layers of a pool *_layer elements apart), in
 * keys and values.  The destination is the source where both pool pointers are
 * equal; else the pools must not overlap.  A pair with a -1 is skipped.  All
 * pairs are refused, as UZIP_ERR_INVALID_ARG in d_status, where a page does not
 * exist, is written twice, or is read and written (within one pool). */
typedef struct {
    int32_t dtype;
    int32_t reserved; /* 0 */
    int64_t layers, heads, page, d;
    int64_t from_pages, to_pages;
    const void* k;
    int64_t k_layer, k_page, k_head, k_token;
    const void* v;
    int64_t v_layer, v_page, v_head, v_token;
    void* k_to;
    int64_t kt_layer, kt_page, kt_head, kt_token;
    void* v_to;
    int64_t vt_layer, vt_page, vt_head, vt_token;
    const int32_t* pairs;
    int64_t n;
} uzip_cache_copy_args;

uint64_t uzip_cache_copy_workspace_size(const uzip_cache_copy_args* a); /* 0 */
uzip_status uzip_cache_copy(const uzip_cache_copy_args* a, void* d_workspace, uint64_t workspace_bytes,
                            int32_t* d_status, cudaStream_t s);

#ifdef __cplusplus
}
#endif
#endif /* UZIP_CACHE_H */
