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

/*
 * ---------------------------------------------------------------- prompts
 *
 * A prompt's way through an attention layer: kv_append turns its queries and
 * keys, and puts keys and values into the cache; kv_prompt_attention attends.
 * The prompts of a call are packed as in gdn_prefill: sequence b owns rows
 * cu_seqlens[b] .. cu_seqlens[b+1]-1 of [total][heads][d] activations, whose
 * kv_rows take `node` as the stride of a row (`seq` is not looked at).
 * cu_seqlens [B + 1] int32 (device), 0 <= cu_seqlens[b] <= cu_seqlens[b+1] <=
 * total. Rows of no sequence are neither read nor written. total may be 0 (a
 * step in which no sequence has a row): q, k, v and the outputs are not looked
 * at then, slots, lengths and offsets are.
 */

/*
 * The norm of each head's row and the position rotation. With x a row of d
 * elements:
 *     y = x / sqrt(mean(x^2) + eps) * (weight + offset)     (no weight: y = x)
 * and pair i < rot / 2 of its first `rot` elements is turned by the angle
 * a = 2 pi turns[i] / 2^64 * position[axis[i]]:
 *     z_1 = y_1 cos a - y_2 sin a,  z_2 = y_1 sin a + y_2 cos a
 * Pairs are elements i and i + rot / 2, or 2i and 2i + 1 (interleaved). FP32
 * arithmetic, one rounding at the end; angles are formed in whole numbers
 * modulo a turn, so that far positions lose nothing of what `turns` says (which
 * is off by 2^-65 turns a position where it is the nearest to a frequency).
 * q_norm, k_norm       FP32 weights of queries and keys, head h's at p + h *
 *                      head stride (0: one row for all heads), d of them;
 *                      NULL: that side is not normed.
 * turns    [rot / 2] 64-bit fractions of a turn a position.
 * axis     [rot / 2] int32, which of the `axes` positions a pair follows
 *          (text: one axis; images and video: time, height, width); NULL: 0.
 *          A value outside [0, axes) counts as 0.
 * rot      even, 0 (no rotation) to d.  axes 1 to KV_MAX_AXES.
 */
#define KV_MAX_AXES 4
typedef struct kv_rotary {
    const float* q_norm;
    const float* k_norm;
    int64_t q_norm_head, k_norm_head;
    float eps, offset;
    const uint64_t* turns;
    const int32_t* axis;
    int32_t rot, axes, interleaved;
} kv_rotary;

/*
 * kv_norm_rotate -- norm and rotation of drafted tokens' queries and keys (a
 * decode step's single ones too), ahead of kv_tree_attention.
 * q, q_out   [B][T][Hq][d], k, k_out [B][T][Hkv][d], of `dtype`; q or k may be
 *            NULL with its output. An output may be its input (the same rows),
 *            else they must not overlap. Hq and Hkv at most 2^24.
 * positions  [axes][B][T] int32; NULL where rot is 0.
 */
int kv_norm_rotate(const kv_rotary* rotary, int32_t dtype, int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t d,
                   const int32_t* positions, const kv_rows* q, const kv_rows* q_out, const kv_rows* k,
                   const kv_rows* k_out, void* stream);

/*
 * kv_append -- the prompts' keys and values into the cache: entry lengths + j
 * of a sequence takes key and value of its row j, its weight becomes 0 and its
 * stamp counts + j (where the cache has them); then lengths and counts grow by
 * the sequence's rows. With `rotary` keys are normed and turned on the way, and
 * so are the rows of q into q_out (both NULL: keys and values alone; without
 * rotary they must be).
 * positions  [axes][total] int32; NULL: counts + j on every axis.
 * The pages of the new entries must be in the page table; a sequence that
 * lacks one (KV_DEVERR_PAGE) keeps its length and count, and what its other
 * new entries' places held is lost. q_out rows of padding and of sequences
 * refused for their slot or length are zero. Offsets that decrease or pass
 * `total` anywhere (GDN_DEVERR_SEQLEN) refuse the whole call. Hq and Hkv are
 * at most 2^24.
 */
int kv_append(const kv_cache* cache, int32_t B, int32_t total, int32_t Hq, const int32_t* slots,
              const int32_t* cu_seqlens, const kv_rows* k, const kv_rows* v, const kv_rotary* rotary,
              const int32_t* positions, const kv_rows* q, const kv_rows* q_out, int32_t* dev_err, void* stream);

/*
 * kv_prompt_attention -- causal attention of packed prompts over the cache,
 * after kv_append of the same rows: with n the sequence's rows and len its
 * length (its last n entries are the rows' own), row j and query head h attend
 * the entries e <= len - n + j of key head h / (Hq / Hkv):
 *     out = sum_e e^(scale q.k_e - lse) v_e,  lse = ln sum_e e^(scale q.k_e)
 * Entries from before the prompt (an earlier chunk, a shared prefix) are
 * attended like the others. Arithmetic as in kv_tree_attention.
 * q          [total][Hq][d].  out [total][Hq][d] of the cache's dtype,
 *            contiguous.  lse [total][Hq] fp32, or NULL.
 * workspace  kv_prompt_attention_workspace() bytes, 16-byte aligned; of one
 *            call at a time. Its contents need no initialisation.
 * A sequence shorter than its rows sets KV_DEVERR_LENGTH; offsets that
 * decrease or pass `total` set GDN_DEVERR_SEQLEN, and the sequence is skipped
 * (its rows are not written). Rows whose entries lie in a page outside the
 * pool are zero, as those of the rows of their block.
 * The tensor cores run what they run in kv_tree_attention, where a key head has
 * at most 128 query heads; above that the FP32 pipe does.
 */
int kv_prompt_attention(const kv_cache* cache, int32_t B, int32_t total, int32_t Hq, const int32_t* slots,
                        const int32_t* cu_seqlens, const kv_rows* q, float scale, void* out, float* lse,
                        void* workspace, int64_t workspace_bytes, int32_t* dev_err, void* stream);

int64_t kv_prompt_attention_workspace(const kv_cache* cache, int32_t B, int32_t total, int32_t Hq);

/*
 * ---------------------------------------------------------------- shared pages
 *
 * kv_fork -- sequences dst[i] become copies of sequences src[i]: for every page
 * j that the source holds, dst's table takes the source's page (shared) where
 * new_pages[i][j] is negative, else that page, into which the entries (keys,
 * values, weights, stamps; up to the source's length) are copied. Lengths and
 * counts are copied; dst's table past the last page stays as it is. Sequences
 * that will grow need their last page, unless it is full, for themselves, and
 * those whose weights will be accumulated or evicted all of them.
 * src, dst   [n] int32 slots; either negative: nothing is done. Destinations
 *            are distinct and no call's sources (not checked, but for src[i]
 *            == dst[i], which sets GDN_DEVERR_SLOT); new pages are distinct
 *            and held by no sequence (not checked).
 * new_pages  [n][max_pages] int32.
 * A fork with an error bit leaves dst as it was.
 */
int kv_fork(const kv_cache* cache, int32_t n, const int32_t* src, const int32_t* dst, const int32_t* new_pages,
            int32_t* dev_err, void* stream);

/*
 * kv_compact -- moves the pages that sequences hold to the front of the pool.
 * A page is held if the table names it within some slot's length (an ended
 * sequence is freed by a length of 0). With U pages held, the j-th lowest page
 * below U that is not held takes the contents (keys, values, weights, stamps)
 * of the j-th lowest held one at or above it, and every table entry within a
 * length follows: afterwards pages U and up are free.
 * used       [1] int32: U, or -1 where a length or a page within one is out of
 *            range (KV_DEVERR_LENGTH, KV_DEVERR_PAGE) and nothing is done.
 * workspace  kv_compact_workspace() bytes, 16-byte aligned; of one call at a
 *            time. Its contents need no initialisation.
 */
int kv_compact(const kv_cache* cache, int32_t* used, void* workspace, int64_t workspace_bytes, int32_t* dev_err,
               void* stream);

int64_t kv_compact_workspace(const kv_cache* cache);

#ifdef __cplusplus
}
#endif
#endif
