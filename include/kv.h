/*
 * kv.h -- C ABI of the paged key/value cache that serves the attention layers
 * of a hybrid model, next to the recurrent layers of gdn.h: attention of
 * drafted tokens (a tree, a chain, or one token) over the cache, the commit of
 * an accepted path, the attention weight each entry has gathered, and the
 * eviction of the entries with the least of it.
 *
 * A verify step of a hybrid model reads the recurrent state through
 * gdn_spec_step / gdn_verify_window and the cache through kv_tree_attention.
 * Neither writes what a rejected draft would have to take back: drafted keys
 * and values stay in the caller's activations until kv_commit copies the
 * accepted ones into the cache.
 *
 * The conventions of gdn.h hold: asynchronous on `stream`; nothing
 * synchronises, allocates or logs; the caller owns all memory; device pointers
 * unless noted; GDN_OK or a negative GDN_ERR_* code, described by
 * gdn_last_error_string(); problems only visible on the device set bits in
 * *dev_err. A sequence whose slot is negative is padding: nothing of it is
 * read or written and its outputs are zero (lse: -inf). A sequence with an
 * error bit is treated the same way, but for GDN_DEVERR_TIMEOUT, after which
 * some key heads of a sequence may be refused and others not, and weights
 * that kv_accumulate was to update may be as they were. Slots within a call
 * that writes must be distinct (not checked).
 */
#ifndef GDN_KV_H
#define GDN_KV_H

#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KV_MAX_NODES 64  /* drafted nodes of a sequence in one call */
#define KV_MAX_D 256     /* head size */

/* Device-side error bits beside those of gdn.h (GDN_DEVERR_SLOT, GDN_DEVERR_TIMEOUT). */
#define KV_DEVERR_LENGTH 64  /* a length outside [0, max_pages * page_size], too little room for a commit,
                                or fewer entries than accepted nodes */
#define KV_DEVERR_PAGE 128   /* a page index outside [0, num_pages) within a sequence's length */
#define KV_DEVERR_NODES 256  /* a node count outside [0, T], a path length outside [0, P], or a path node
                                outside [0, T) */

/*
 * One layer's cache. Entry e of a sequence lies in page
 * page_table[slot * max_pages + e / page_size] at place e % page_size; its key
 * of head h starts at k + page * k_page + h * k_head + place * k_token
 * (elements), d consecutive elements; values alike. So pages may be laid out
 * [page][head][place][d], [page][place][head][d], or interleaved. Page table
 * entries past a sequence's length are not read. A page may belong to several
 * sequences as long as no call writes it.
 *
 * max_pages * page_size is at most 2^31 - 65536, d at most KV_MAX_D.
 * dtype      GDN_F32, GDN_BF16 or GDN_F16, of k and v.
 * lengths    [num_slots] int32, entries of each slot's sequence.
 * counts     [num_slots] int32, tokens ever committed to the slot (evicted
 *            ones among them); NULL where only kv_tree_attention is called.
 * weights    [num_pages][Hkv][page_size] fp32, gathered attention weight of
 *            each entry; NULL where neither accumulated nor evicted.
 * stamps     [num_pages][Hkv][page_size] int32, the count at which the entry
 *            was committed (its position in the text); NULL with weights.
 */
typedef struct kv_cache {
    void* k;
    void* v;
    int32_t dtype;
    int32_t Hkv, page_size, d;
    int64_t num_pages;
    int64_t k_page, k_head, k_token;
    int64_t v_page, v_head, v_token;
    const int32_t* page_table;
    int32_t max_pages;
    int64_t num_slots;
    int32_t* lengths;
    int32_t* counts;
    float* weights;
    int32_t* stamps;
} kv_cache;

/* Activations [B][T][heads][d] with strides in elements (d contiguous), so that q, k and v may be
 * parts of one projection's output. Of the cache's dtype. */
typedef struct kv_rows {
    const void* p;
    int64_t seq, node, head;
} kv_rows;

/*
 * kv_tree_attention -- attention of T drafted nodes of each sequence over its
 * cache and over one another. For node i of sequence b and query head h, with
 * key head h / (Hq / Hkv):
 *     out = sum_e e^(scale q.k_e - lse) v_e,  lse = ln sum_e e^(scale q.k_e)
 * over all cache entries and the nodes j with bit j of mask[b][i] set (a tree:
 * its ancestors and itself; any mask is taken, one that leaves nothing too: a
 * row without a key gives out = 0, lse = -inf). T = 1 is the decode step of a
 * single token. Scores, softmax statistics and sums are FP32; on the tensor
 * cores (below) the weights are rounded once to the cache's dtype before they
 * meet the values, in fp16 to no finer than 2^-31 of the row's largest. The
 * cache is not written.
 * slots      [B] int32.
 * q          [B][T][Hq][d];  k_new, v_new  [B][T][Hkv][d]; Hq at most 2^24.
 * mask       [B][T] 64-bit words. Bits >= num_nodes[b] are not looked at.
 * num_nodes  [B] int32, drafted nodes of each sequence (<= T; out and lse of
 *            the others are 0 and -inf); NULL: T for all.
 * out        [B][T][Hq][d] of the cache's dtype, contiguous.
 * lse        [B][T][Hq] fp32, or NULL.
 * workspace  kv_tree_attention_workspace() bytes, 16-byte aligned; of one
 *            call at a time. Its contents need no initialisation.
 * 16-bit caches whose pages hold a multiple of 8 entries, with d a multiple of
 * 8 and bases and strides of 16 bytes, run on the tensor cores; everything
 * else, fp32 caches among it, on the FP32 pipe (a 16-bit decode step takes
 * some fifteen times as long there). How a sequence's keys are
 * split over the device, and so the order of its sums, depends on the sizes
 * of the call and the other sequences' lengths; the same call gives the same
 * bits.
 */
int kv_tree_attention(const kv_cache* cache, int32_t B, int32_t T, int32_t Hq,
                      const int32_t* slots, const kv_rows* q, const kv_rows* k_new,
                      const kv_rows* v_new, const uint64_t* mask, const int32_t* num_nodes,
                      float scale, void* out, float* lse, void* workspace,
                      int64_t workspace_bytes, int32_t* dev_err, void* stream);

/* Bytes of workspace for calls with these sizes on the current device (host query), or a negative
 * GDN_ERR_* code. */
int64_t kv_tree_attention_workspace(const kv_cache* cache, int32_t B, int32_t T, int32_t Hq);

/*
 * kv_commit -- append the accepted path of each sequence to its cache: for
 * j < n_path[b], entry lengths + j takes key and value of node path[b][j], its
 * weight becomes 0 and its stamp counts + j (where the cache has them); then
 * lengths and counts grow by n_path[b]. The pages of the new entries must be
 * in the page table; a sequence that lacks one is left as it was.
 * path       [B][P] int32 node indices;  n_path [B] int32 in [0, P].
 */
int kv_commit(const kv_cache* cache, int32_t B, int32_t T, int32_t P, const int32_t* slots,
              const kv_rows* k_new, const kv_rows* v_new, const int32_t* path,
              const int32_t* n_path, int32_t* dev_err, void* stream);

/*
 * kv_accumulate -- add the attention weight that the accepted nodes gave to
 * each entry, after kv_commit of the same path: with n = n_path[b] and len the
 * sequence's length (its last n entries are the path's own), for key head g
 * and entry e
 *     weights[e] = decay * weights[e]
 *         + sum_{j < n, e <= len - n + j} sum_{h of g} e^(scale q_jh.k_e - lse_jh)
 * q [B][T][Hq][d] and lse [B][T][Hq] (contiguous) as given to and returned by
 * kv_tree_attention; row j is that of node path[b][j]. A row whose lse is
 * -inf adds nothing. n_path[b] = 0 leaves the sequence's weights as they are.
 */
int kv_accumulate(const kv_cache* cache, int32_t B, int32_t T, int32_t P, int32_t Hq,
                  const int32_t* slots, const kv_rows* q, const float* lse, const int32_t* path,
                  const int32_t* n_path, float scale, float decay, int32_t* dev_err, void* stream);

/*
 * kv_evict -- bring every sequence longer than `budget` back to it, key head
 * by key head. Kept are the entries whose stamp is at least counts - recent
 * (the newest tokens), then those of the largest weight, `budget` in all; ties
 * go to the lowest entry, NaN counts as the largest weight. Then the j-th
 * lowest entry below `budget` that was not kept takes key, value, weight and
 * stamp of the j-th lowest kept one at or above it, and lengths becomes
 * `budget`: kept entries below it do not move. 1 <= budget, 0 <= recent <=
 * budget.
 * workspace  kv_evict_workspace() bytes, 16-byte aligned; of one call at a
 *            time. Its contents need no initialisation.
 */
int kv_evict(const kv_cache* cache, int32_t B, const int32_t* slots, int32_t budget,
             int32_t recent, void* workspace, int64_t workspace_bytes, int32_t* dev_err,
             void* stream);

int64_t kv_evict_workspace(const kv_cache* cache, int32_t B, int32_t budget);

#ifdef __cplusplus
}
#endif
#endif
