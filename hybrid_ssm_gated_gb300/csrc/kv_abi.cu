// kv_abi.cu -- the extern "C" entry points declared in include/kv.h: argument
// validation on the host, then launches on the caller's stream. Nothing here
// allocates, synchronises or logs.
#include <math.h>
#include <stdint.h>

#include "../../include/kv.h"
#include "gdn_error.h"
#include "kv_dispatch.h"

namespace {

using gdn::fail;
using gdn::launched;

// A C++ exception (the launch helpers' tables may run out of memory) ends here, not in the C caller.
int caught(const char* fn) {
    try {
        return fail(GDN_ERR_LAUNCH, "%s: out of host memory", fn);
    } catch (...) {
        return GDN_ERR_LAUNCH;
    }
}

bool aligned_to(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) % (uintptr_t)n) == 0; }

int check_cache(const char* fn, const kv_cache* c, int32_t B) {
    if (!c) return fail(GDN_ERR_NULL, "%s: cache is NULL", fn);
    if (c->dtype != GDN_F32 && c->dtype != GDN_BF16 && c->dtype != GDN_F16)
        return fail(GDN_ERR_DTYPE, "%s: unsupported cache dtype %d", fn, c->dtype);
    if (B < 0 || c->Hkv < 1 || c->page_size < 1 || c->num_pages < 0 || c->max_pages < 0 || c->num_slots < 0)
        return fail(GDN_ERR_SHAPE, "%s: negative or zero sizes (B=%d Hkv=%d page_size=%d num_pages=%lld max_pages=%d)",
                    fn, B, c->Hkv, c->page_size, (long long)c->num_pages, c->max_pages);
    if (c->d < 1 || c->d > KV_MAX_D) return fail(GDN_ERR_SHAPE, "%s: d=%d not in [1, %d]", fn, c->d, KV_MAX_D);
    // (the kernels look a few tiles past a sequence's end in 32 bits)
    if ((int64_t)c->max_pages * c->page_size > 0x7fff0000 || c->num_pages > 0x7fffffff)
        return fail(GDN_ERR_SHAPE, "%s: a sequence's capacity or the page count does not fit 31 bits", fn);
    if (c->k_page < 0 || c->k_head < 0 || c->k_token < 0 || c->v_page < 0 || c->v_head < 0 || c->v_token < 0)
        return fail(GDN_ERR_SHAPE, "%s: negative cache strides", fn);
    if (B == 0) return GDN_OK;
    if (!c->k || !c->v || !c->page_table || !c->lengths)
        return fail(GDN_ERR_NULL, "%s: k, v, page_table or lengths is NULL", fn);
    const int esz = gdn::dtype_size(c->dtype);
    if (!aligned_to(c->k, esz) || !aligned_to(c->v, esz) || !aligned_to(c->page_table, 4) ||
        !aligned_to(c->lengths, 4) || !aligned_to(c->counts, 4) || !aligned_to(c->weights, 4) ||
        !aligned_to(c->stamps, 4))
        return fail(GDN_ERR_ALIGN, "%s: a cache array is misaligned for its element type", fn);
    if (!c->weights != !c->stamps) return fail(GDN_ERR_NULL, "%s: weights and stamps come together", fn);
    return GDN_OK;
}

int check_rows(const char* fn, const char* name, const kv_rows* r, int32_t dtype) {
    if (!r || !r->p) return fail(GDN_ERR_NULL, "%s: %s is NULL", fn, name);
    if (r->seq < 0 || r->node < 0 || r->head < 0) return fail(GDN_ERR_SHAPE, "%s: negative strides of %s", fn, name);
    if (!aligned_to(r->p, gdn::dtype_size(dtype)))
        return fail(GDN_ERR_ALIGN, "%s: %s is misaligned for its element type", fn, name);
    return GDN_OK;
}

int check_call(const char* fn, const int32_t* slots, const int32_t* dev_err) {
    if (!slots || !dev_err) return fail(GDN_ERR_NULL, "%s: slots or dev_err is NULL", fn);
    if (!aligned_to(slots, 4) || !aligned_to(dev_err, 4)) return fail(GDN_ERR_ALIGN, "%s: slots or dev_err misaligned", fn);
    return GDN_OK;
}

int check_heads(const char* fn, const kv_cache* c, int32_t Hq, float scale) {
    if (Hq < 1 || Hq % c->Hkv != 0)
        return fail(GDN_ERR_SHAPE, "%s: Hq=%d is not a positive multiple of Hkv=%d", fn, Hq, c->Hkv);
    // rows of a unit, KV_MAX_NODES x Hq / Hkv at most, are counted in 32 bits
    if (Hq > 1 << 24) return fail(GDN_ERR_SHAPE, "%s: Hq=%d is more than 2^24", fn, Hq);
    if (!isfinite(scale)) return fail(GDN_ERR_SHAPE, "%s: scale is not finite", fn);
    return GDN_OK;
}

int check_nodes(const char* fn, int32_t T, int32_t P) {
    if (T < 1 || T > KV_MAX_NODES) return fail(GDN_ERR_WINDOW, "%s: T=%d not in [1, %d]", fn, T, KV_MAX_NODES);
    if (P < 1 || P > KV_MAX_NODES) return fail(GDN_ERR_WINDOW, "%s: P=%d not in [1, %d]", fn, P, KV_MAX_NODES);
    return GDN_OK;
}

gdn::KvRows rows_of(const kv_rows* r) { return {r->p, r->seq, r->node, r->head}; }

gdn::KvArgs args_of(const kv_cache* c, int32_t B, const int32_t* slots, int32_t* dev_err) {
    gdn::KvArgs a{};
    a.k = {c->k, c->k_page, c->k_head, c->k_token};
    a.v = {c->v, c->v_page, c->v_head, c->v_token};
    a.page_table = c->page_table, a.slots = slots, a.dev_err = dev_err;
    a.lengths = c->lengths, a.counts = c->counts, a.weights = c->weights, a.stamps = c->stamps;
    a.num_pages = c->num_pages, a.num_slots = c->num_slots;
    a.B = B, a.Hkv = c->Hkv, a.d = c->d, a.page_size = c->page_size, a.max_pages = c->max_pages, a.dtype = c->dtype;
    a.row_block = 1;
    return a;
}

// Whether every row that starts at p + multiples of the strides (elements of esz bytes, d of them) can
// be read and written 16 bytes at a time.
bool vec_rows(const void* p, int64_t s0, int64_t s1, int64_t s2, int d, int esz) {
    return aligned_to(p, 16) && s0 * esz % 16 == 0 && s1 * esz % 16 == 0 && s2 * esz % 16 == 0 && d * esz % 16 == 0;
}
// Workspace of either attention kernel: the caller's rows decide at the call which one runs.
cudaError_t attention_workspace(gdn::KvArgs& a, int64_t& bytes) {
    cudaError_t e = gdn::kv_attn_workspace(a, bytes);
    if (e != cudaSuccess || !gdn::kv_tc_fits(a)) return e;
    int64_t more = 0;
    e = gdn::kv_attn_tc_workspace(a, more);
    if (more > bytes) bytes = more;
    return e;
}

// The same for prompts.
cudaError_t prompt_workspace(gdn::KvArgs& a, int64_t& bytes) {
    cudaError_t e = gdn::kv_prompt_workspace(a, bytes);
    if (e != cudaSuccess || !gdn::kv_prompt_tc_fits(a)) return e;
    int64_t more = 0;
    e = gdn::kv_prompt_tc_workspace(a, more);
    if (more > bytes) bytes = more;
    return e;
}

// What the places of a call's units on its line are counted in: rows in 31 bits, keys in 62.
int check_prompt(const char* fn, const kv_cache* c, int32_t B, int32_t total, int32_t Hq) {
    if (total < 0) return fail(GDN_ERR_SHAPE, "%s: total=%d", fn, total);
    const double G = Hq / c->Hkv, room = (double)c->max_pages * c->page_size + 1024, blocks = total * G / 64 + B;
    if (total * G > 0x7fff0000 || blocks * (G * room + total * G + 1024) * c->Hkv > 4e18)
        return fail(GDN_ERR_SHAPE, "%s: total=%d rows of %d query heads are too many", fn, total, Hq);
    return GDN_OK;
}

int check_rotary(const char* fn, const kv_rotary* r, int32_t d, bool positions) {
    if (!r) return fail(GDN_ERR_NULL, "%s: rotary is NULL", fn);
    if (r->rot < 0 || r->rot > d || r->rot % 2 != 0)
        return fail(GDN_ERR_SHAPE, "%s: rot=%d is not an even number in [0, d=%d]", fn, r->rot, d);
    if (r->axes < 1 || r->axes > KV_MAX_AXES) return fail(GDN_ERR_SHAPE, "%s: axes=%d not in [1, %d]", fn, r->axes, KV_MAX_AXES);
    if (r->rot > 0 && (!r->turns || !positions)) return fail(GDN_ERR_NULL, "%s: turns or positions is NULL", fn);
    if (r->q_norm_head < 0 || r->k_norm_head < 0) return fail(GDN_ERR_SHAPE, "%s: negative strides of the norms' weights", fn);
    if (!(r->eps >= 0.f) || !isfinite(r->eps) || !isfinite(r->offset))
        return fail(GDN_ERR_SHAPE, "%s: eps must be a finite number from 0 on, offset finite", fn);
    if (!aligned_to(r->q_norm, 4) || !aligned_to(r->k_norm, 4) || !aligned_to(r->turns, 8) || !aligned_to(r->axis, 4))
        return fail(GDN_ERR_ALIGN, "%s: a norm's weights, turns or axis misaligned", fn);
    return GDN_OK;
}

gdn::KvTurn turn_of(const kv_rows* in, const kv_rows* out, const float* norm, int64_t head) {
    gdn::KvTurn t{};
    if (!in) return t;
    t.in = in->p, t.in_seq = in->seq, t.in_node = in->node, t.in_head = in->head, t.norm = norm, t.norm_head = head;
    if (out) t.out = const_cast<void*>(out->p), t.out_seq = out->seq, t.out_node = out->node, t.out_head = out->head;
    return t;
}
void rotary_of(gdn::KvRotateArgs& a, const kv_rotary* r) {
    a.turns = r->turns, a.axis = r->axis, a.eps = r->eps, a.offset = r->offset;
    a.rot = r->rot, a.axes = r->axes, a.interleaved = r->interleaved != 0;
}
bool vec_norm(const float* p, int64_t head) { return aligned_to(p, 16) && head % 4 == 0; }

bool vec_pages(const gdn::KvPages& c, int d, int esz) { return vec_rows(c.p, c.page, c.head, c.token, d, esz); }
bool vec_rows(const gdn::KvRows& r, int d, int esz) { return vec_rows(r.p, r.seq, r.node, r.head, d, esz); }

}  // namespace

extern "C" {

int64_t kv_tree_attention_workspace(const kv_cache* cache, int32_t B, int32_t T, int32_t Hq) try {
    const char* fn = "kv_tree_attention_workspace";
    int rc = check_cache(fn, cache, 0);
    if (rc) return rc;
    if (B < 0) return fail(GDN_ERR_SHAPE, "%s: B=%d", fn, B);
    if ((rc = check_nodes(fn, T, 1)) || (rc = check_heads(fn, cache, Hq, 1.f))) return rc;
    gdn::KvArgs a = args_of(cache, B, nullptr, nullptr);
    a.T = T, a.Hq = Hq, a.G = Hq / cache->Hkv;
    int64_t bytes = 0;
    const cudaError_t e = attention_workspace(a, bytes);
    if (e != cudaSuccess) return launched(e, fn);
    return bytes;
} catch (...) {
    return caught("kv_tree_attention_workspace");
}

int kv_tree_attention(const kv_cache* cache, int32_t B, int32_t T, int32_t Hq, const int32_t* slots, const kv_rows* q,
                      const kv_rows* k_new, const kv_rows* v_new, const uint64_t* mask, const int32_t* num_nodes,
                      float scale, void* out, float* lse, void* workspace, int64_t workspace_bytes, int32_t* dev_err,
                      void* stream) try {
    const char* fn = "kv_tree_attention";
    int rc = check_cache(fn, cache, B);
    if (rc) return rc;
    if ((rc = check_nodes(fn, T, 1)) || (rc = check_heads(fn, cache, Hq, scale))) return rc;
    if (B == 0) return GDN_OK;
    if ((rc = check_call(fn, slots, dev_err))) return rc;
    if ((rc = check_rows(fn, "q", q, cache->dtype)) || (rc = check_rows(fn, "k_new", k_new, cache->dtype)) ||
        (rc = check_rows(fn, "v_new", v_new, cache->dtype)))
        return rc;
    if (!mask || !out || !workspace) return fail(GDN_ERR_NULL, "%s: mask, out or workspace is NULL", fn);
    if (!aligned_to(mask, 8) || !aligned_to(num_nodes, 4) || !aligned_to(lse, 4) || !aligned_to(workspace, 16) ||
        !aligned_to(out, gdn::dtype_size(cache->dtype)))
        return fail(GDN_ERR_ALIGN, "%s: mask, num_nodes, out, lse or workspace misaligned", fn);
    gdn::KvArgs a = args_of(cache, B, slots, dev_err);
    a.T = T, a.Hq = Hq, a.G = Hq / cache->Hkv;
    a.q = rows_of(q), a.kn = rows_of(k_new), a.vn = rows_of(v_new);
    a.mask = mask, a.num_nodes = num_nodes, a.scale = scale, a.out = out, a.lse = lse;
    a.part = static_cast<float*>(workspace);
    int64_t need = 0;
    cudaError_t e = attention_workspace(a, need);
    if (e != cudaSuccess) return launched(e, fn);
    if (workspace_bytes < need)
        return fail(GDN_ERR_SHAPE, "%s: workspace of %lld bytes, %lld needed", fn, (long long)workspace_bytes,
                    (long long)need);
    const int esz = gdn::dtype_size(cache->dtype);
    const bool vec = vec_pages(a.k, a.d, esz) && vec_pages(a.v, a.d, esz) && vec_rows(a.q, a.d, esz) &&
                     vec_rows(a.kn, a.d, esz) && vec_rows(a.vn, a.d, esz);
    e = vec && gdn::kv_tc_fits(a) ? gdn::launch_kv_attn_tc(a, static_cast<cudaStream_t>(stream)) : cudaErrorNotSupported;
    if (e == cudaErrorNotSupported) e = gdn::launch_kv_attn(a, vec, static_cast<cudaStream_t>(stream));
    return launched(e, fn);
} catch (...) {
    return caught("kv_tree_attention");
}

int kv_commit(const kv_cache* cache, int32_t B, int32_t T, int32_t P, const int32_t* slots, const kv_rows* k_new,
              const kv_rows* v_new, const int32_t* path, const int32_t* n_path, int32_t* dev_err, void* stream) try {
    const char* fn = "kv_commit";
    int rc = check_cache(fn, cache, B);
    if (rc) return rc;
    if ((rc = check_nodes(fn, T, P))) return rc;
    if (B == 0) return GDN_OK;
    if ((rc = check_call(fn, slots, dev_err))) return rc;
    if ((rc = check_rows(fn, "k_new", k_new, cache->dtype)) || (rc = check_rows(fn, "v_new", v_new, cache->dtype)))
        return rc;
    if (!path || !n_path) return fail(GDN_ERR_NULL, "%s: path or n_path is NULL", fn);
    if (!aligned_to(path, 4) || !aligned_to(n_path, 4)) return fail(GDN_ERR_ALIGN, "%s: path or n_path misaligned", fn);
    if (cache->stamps && !cache->counts) return fail(GDN_ERR_NULL, "%s: a cache with stamps needs counts", fn);
    gdn::KvArgs a = args_of(cache, B, slots, dev_err);
    a.T = T, a.P = P, a.kn = rows_of(k_new), a.vn = rows_of(v_new), a.path = path, a.n_path = n_path;
    const int esz = gdn::dtype_size(cache->dtype);
    const bool vec = vec_pages(a.k, a.d, esz) && vec_pages(a.v, a.d, esz) && vec_rows(a.kn, a.d, esz) &&
                     vec_rows(a.vn, a.d, esz);
    return launched(gdn::launch_kv_commit(a, vec, static_cast<cudaStream_t>(stream)), fn);
} catch (...) {
    return caught("kv_commit");
}

int kv_accumulate(const kv_cache* cache, int32_t B, int32_t T, int32_t P, int32_t Hq, const int32_t* slots,
                  const kv_rows* q, const float* lse, const int32_t* path, const int32_t* n_path, float scale,
                  float decay, int32_t* dev_err, void* stream) try {
    const char* fn = "kv_accumulate";
    int rc = check_cache(fn, cache, B);
    if (rc) return rc;
    if ((rc = check_nodes(fn, T, P)) || (rc = check_heads(fn, cache, Hq, scale))) return rc;
    if (!isfinite(decay)) return fail(GDN_ERR_SHAPE, "%s: decay is not finite", fn);
    if (B == 0) return GDN_OK;
    if ((rc = check_call(fn, slots, dev_err))) return rc;
    if ((rc = check_rows(fn, "q", q, cache->dtype))) return rc;
    if (!lse || !path || !n_path || !cache->weights)
        return fail(GDN_ERR_NULL, "%s: lse, path, n_path or the cache's weights is NULL", fn);
    if (!aligned_to(lse, 4) || !aligned_to(path, 4) || !aligned_to(n_path, 4))
        return fail(GDN_ERR_ALIGN, "%s: lse, path or n_path misaligned", fn);
    gdn::KvArgs a = args_of(cache, B, slots, dev_err);
    a.T = T, a.P = P, a.Hq = Hq, a.G = Hq / cache->Hkv, a.q = rows_of(q);
    a.lse_in = lse, a.path = path, a.n_path = n_path, a.scale = scale, a.decay = decay;
    const int esz = gdn::dtype_size(cache->dtype);
    const bool vec = vec_pages(a.k, a.d, esz) && vec_rows(a.q, a.d, esz);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = vec && gdn::kv_tc_fits(a) ? gdn::launch_kv_weights_tc(a, s) : cudaErrorNotSupported;
    if (e == cudaErrorNotSupported) e = gdn::launch_kv_weights(a, vec, s);
    return launched(e, fn);
} catch (...) {
    return caught("kv_accumulate");
}

int64_t kv_evict_workspace(const kv_cache* cache, int32_t B, int32_t budget) try {
    const char* fn = "kv_evict_workspace";
    const int rc = check_cache(fn, cache, 0);
    if (rc) return rc;
    if (B < 0 || budget < 1) return fail(GDN_ERR_SHAPE, "%s: B=%d, budget=%d", fn, B, budget);
    return gdn::kv_moves_at((int64_t)B * cache->Hkv, gdn::kv_moves_cap(cache->max_pages, cache->page_size, budget)) * 4;
} catch (...) {
    return caught("kv_evict_workspace");
}

int kv_evict(const kv_cache* cache, int32_t B, const int32_t* slots, int32_t budget, int32_t recent, void* workspace,
             int64_t workspace_bytes, int32_t* dev_err, void* stream) try {
    const char* fn = "kv_evict";
    int rc = check_cache(fn, cache, B);
    if (rc) return rc;
    if (budget < 1 || recent < 0 || recent > budget)
        return fail(GDN_ERR_SHAPE, "%s: budget=%d must be positive and recent=%d in [0, budget]", fn, budget, recent);
    if (B == 0) return GDN_OK;
    if ((rc = check_call(fn, slots, dev_err))) return rc;
    if (!cache->weights || !cache->stamps || !cache->counts || !workspace)
        return fail(GDN_ERR_NULL, "%s: the cache's weights, stamps or counts, or workspace, is NULL", fn);
    if (!aligned_to(workspace, 16)) return fail(GDN_ERR_ALIGN, "%s: workspace misaligned", fn);
    const int cap = gdn::kv_moves_cap(cache->max_pages, cache->page_size, budget);
    const int64_t need = gdn::kv_moves_at((int64_t)B * cache->Hkv, cap) * 4;
    if (workspace_bytes < need)
        return fail(GDN_ERR_SHAPE, "%s: workspace of %lld bytes, %lld needed", fn, (long long)workspace_bytes,
                    (long long)need);
    if (cap == 0) return GDN_OK;  // no sequence can be longer than the budget
    gdn::KvArgs a = args_of(cache, B, slots, dev_err);
    a.budget = budget, a.recent = recent, a.moves = static_cast<int32_t*>(workspace);
    const int esz = gdn::dtype_size(cache->dtype);
    const bool vec = vec_pages(a.k, a.d, esz) && vec_pages(a.v, a.d, esz);
    return launched(gdn::launch_kv_evict(a, cap, vec, static_cast<cudaStream_t>(stream)), fn);
} catch (...) {
    return caught("kv_evict");
}

int kv_norm_rotate(const kv_rotary* rotary, int32_t dtype, int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t d,
                   const int32_t* positions, const kv_rows* q, const kv_rows* q_out, const kv_rows* k,
                   const kv_rows* k_out, void* stream) try {
    const char* fn = "kv_norm_rotate";
    if (dtype != GDN_F32 && dtype != GDN_BF16 && dtype != GDN_F16) return fail(GDN_ERR_DTYPE, "%s: unsupported dtype %d", fn, dtype);
    if (d < 1 || d > KV_MAX_D) return fail(GDN_ERR_SHAPE, "%s: d=%d not in [1, %d]", fn, d, KV_MAX_D);
    if (B < 0 || T < 0 || (int64_t)B * T > 0x7fffff00) return fail(GDN_ERR_SHAPE, "%s: B=%d, T=%d", fn, B, T);
    if ((q && Hq < 1) || (k && Hkv < 1) || Hq > 1 << 24 || Hkv > 1 << 24)
        return fail(GDN_ERR_SHAPE, "%s: Hq=%d, Hkv=%d", fn, Hq, Hkv);
    if ((!q && !k) || !q != !q_out || !k != !k_out) return fail(GDN_ERR_NULL, "%s: q, k and their outputs come in pairs", fn);
    int rc = check_rotary(fn, rotary, d, positions != nullptr || (int64_t)B * T == 0);
    if (rc || (int64_t)B * T == 0) return rc;
    for (const kv_rows* r : {q, q_out, k, k_out})
        if (r && (rc = check_rows(fn, "q, k or an output", r, dtype))) return rc;
    if (!aligned_to(positions, 4)) return fail(GDN_ERR_ALIGN, "%s: positions misaligned", fn);
    gdn::KvRotateArgs a{};
    rotary_of(a, rotary);
    a.q = turn_of(q, q_out, rotary->q_norm, rotary->q_norm_head);
    a.k = turn_of(k, k_out, rotary->k_norm, rotary->k_norm_head);
    a.positions = positions, a.tokens = B * T, a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.d = d, a.dtype = dtype;
    const int esz = gdn::dtype_size(dtype);
    bool vec = true;
    for (const kv_rows* r : {q, q_out, k, k_out})
        if (r) vec = vec && vec_rows(r->p, r->seq, r->node, r->head, d, esz);
    vec = vec && (!q || vec_norm(rotary->q_norm, rotary->q_norm_head)) && (!k || vec_norm(rotary->k_norm, rotary->k_norm_head));
    return launched(gdn::launch_kv_rotate(a, nullptr, vec, static_cast<cudaStream_t>(stream)), fn);
} catch (...) {
    return caught("kv_norm_rotate");
}

int kv_append(const kv_cache* cache, int32_t B, int32_t total, int32_t Hq, const int32_t* slots, const int32_t* cu_seqlens,
              const kv_rows* k, const kv_rows* v, const kv_rotary* rotary, const int32_t* positions, const kv_rows* q,
              const kv_rows* q_out, int32_t* dev_err, void* stream) try {
    const char* fn = "kv_append";
    int rc = check_cache(fn, cache, B);
    if (rc) return rc;
    if (total < 0 || total > 0x7fffff00) return fail(GDN_ERR_SHAPE, "%s: total=%d", fn, total);
    if (!q != !q_out || (q && !rotary)) return fail(GDN_ERR_NULL, "%s: q, q_out and rotary come together", fn);
    // (rows of a block, up to 16 tokens' heads, are counted in 32 bits)
    if ((q && (Hq < 1 || Hq > 1 << 24)) || cache->Hkv > 1 << 24)
        return fail(GDN_ERR_SHAPE, "%s: Hq=%d, Hkv=%d", fn, Hq, cache->Hkv);
    if (rotary && (rc = check_rotary(fn, rotary, cache->d, true))) return rc;
    if (B == 0) return GDN_OK;
    if ((rc = check_call(fn, slots, dev_err))) return rc;
    if (!cu_seqlens) return fail(GDN_ERR_NULL, "%s: cu_seqlens is NULL", fn);
    if (!aligned_to(cu_seqlens, 4) || !aligned_to(positions, 4)) return fail(GDN_ERR_ALIGN, "%s: cu_seqlens or positions misaligned", fn);
    if (total > 0) {  // (without a row none has an address; slots, lengths and offsets are looked at all the same)
        if ((rc = check_rows(fn, "k", k, cache->dtype)) || (rc = check_rows(fn, "v", v, cache->dtype))) return rc;
        for (const kv_rows* r : {q, q_out})
            if (r && (rc = check_rows(fn, "q or q_out", r, cache->dtype))) return rc;
    }
    if (cache->stamps && !cache->counts) return fail(GDN_ERR_NULL, "%s: a cache with stamps needs counts", fn);
    gdn::KvArgs c = args_of(cache, B, slots, dev_err);
    c.cu = cu_seqlens, c.total = total;
    gdn::KvRotateArgs a{};
    if (rotary) rotary_of(a, rotary);
    else a.axes = 1;
    const kv_rows kp = {cache->k, 0, 0, cache->k_head}, vp = {cache->v, 0, 0, cache->v_head};  // (places: on the device)
    a.q = turn_of(q, q_out, rotary ? rotary->q_norm : nullptr, rotary ? rotary->q_norm_head : 0);
    a.k = turn_of(k, &kp, rotary ? rotary->k_norm : nullptr, rotary ? rotary->k_norm_head : 0);
    a.v = turn_of(v, &vp, nullptr, 0);
    a.positions = positions, a.tokens = total, a.T = 1, a.Hq = Hq, a.Hkv = cache->Hkv, a.d = cache->d, a.dtype = cache->dtype;
    const int esz = gdn::dtype_size(cache->dtype);
    bool vec = vec_pages(c.k, a.d, esz) && vec_pages(c.v, a.d, esz);
    for (const kv_rows* r : {q, q_out, k, v})
        if (r) vec = vec && vec_rows(r->p, 0, r->node, r->head, a.d, esz);
    if (rotary) vec = vec && (!q || vec_norm(rotary->q_norm, rotary->q_norm_head)) && vec_norm(rotary->k_norm, rotary->k_norm_head);
    return launched(gdn::launch_kv_rotate(a, &c, vec, static_cast<cudaStream_t>(stream)), fn);
} catch (...) {
    return caught("kv_append");
}

int64_t kv_prompt_attention_workspace(const kv_cache* cache, int32_t B, int32_t total, int32_t Hq) try {
    const char* fn = "kv_prompt_attention_workspace";
    int rc = check_cache(fn, cache, 0);
    if (rc) return rc;
    if (B < 0) return fail(GDN_ERR_SHAPE, "%s: B=%d", fn, B);
    if ((rc = check_heads(fn, cache, Hq, 1.f)) || (rc = check_prompt(fn, cache, B, total, Hq))) return rc;
    gdn::KvArgs a = args_of(cache, B, nullptr, nullptr);
    a.total = total, a.Hq = Hq, a.G = Hq / cache->Hkv;
    int64_t bytes = 0;
    const cudaError_t e = prompt_workspace(a, bytes);
    if (e != cudaSuccess) return launched(e, fn);
    return bytes;
} catch (...) {
    return caught("kv_prompt_attention_workspace");
}

int kv_prompt_attention(const kv_cache* cache, int32_t B, int32_t total, int32_t Hq, const int32_t* slots,
                        const int32_t* cu_seqlens, const kv_rows* q, float scale, void* out, float* lse, void* workspace,
                        int64_t workspace_bytes, int32_t* dev_err, void* stream) try {
    const char* fn = "kv_prompt_attention";
    int rc = check_cache(fn, cache, B);
    if (rc) return rc;
    if ((rc = check_heads(fn, cache, Hq, scale)) || (rc = check_prompt(fn, cache, B, total, Hq))) return rc;
    if (B == 0) return GDN_OK;
    if ((rc = check_call(fn, slots, dev_err))) return rc;
    if (!cu_seqlens || (total > 0 && !out) || !workspace)
        return fail(GDN_ERR_NULL, "%s: cu_seqlens, out or workspace is NULL", fn);
    if (total > 0 && (rc = check_rows(fn, "q", q, cache->dtype))) return rc;
    if (!aligned_to(cu_seqlens, 4) || !aligned_to(lse, 4) || !aligned_to(workspace, 16) ||
        !aligned_to(out, gdn::dtype_size(cache->dtype)))
        return fail(GDN_ERR_ALIGN, "%s: cu_seqlens, out, lse or workspace misaligned", fn);
    gdn::KvArgs a = args_of(cache, B, slots, dev_err);
    a.cu = cu_seqlens, a.total = total, a.Hq = Hq, a.G = Hq / cache->Hkv;
    if (total > 0) a.q = rows_of(q);
    a.scale = scale, a.out = out, a.lse = lse, a.part = static_cast<float*>(workspace);
    int64_t need = 0;
    cudaError_t e = prompt_workspace(a, need);
    if (e != cudaSuccess) return launched(e, fn);
    if (workspace_bytes < need)
        return fail(GDN_ERR_SHAPE, "%s: workspace of %lld bytes, %lld needed", fn, (long long)workspace_bytes,
                    (long long)need);
    const int esz = gdn::dtype_size(cache->dtype);
    const bool vec = vec_pages(a.k, a.d, esz) && vec_pages(a.v, a.d, esz) && vec_rows(a.q.p, 0, a.q.node, a.q.head, a.d, esz);
    e = vec && gdn::kv_prompt_tc_fits(a) ? gdn::launch_kv_prompt_tc(a, static_cast<cudaStream_t>(stream)) : cudaErrorNotSupported;
    if (e == cudaErrorNotSupported) e = gdn::launch_kv_prompt(a, vec, static_cast<cudaStream_t>(stream));
    return launched(e, fn);
} catch (...) {
    return caught("kv_prompt_attention");
}

int kv_fork(const kv_cache* cache, int32_t n, const int32_t* src, const int32_t* dst, const int32_t* new_pages,
            int32_t* dev_err, void* stream) try {
    const char* fn = "kv_fork";
    int rc = check_cache(fn, cache, n);
    if (rc) return rc;
    if (n == 0) return GDN_OK;
    if ((rc = check_call(fn, src, dev_err))) return rc;
    if (!dst || !new_pages) return fail(GDN_ERR_NULL, "%s: dst or new_pages is NULL", fn);
    if (!aligned_to(dst, 4) || !aligned_to(new_pages, 4)) return fail(GDN_ERR_ALIGN, "%s: dst or new_pages misaligned", fn);
    const gdn::KvArgs a = args_of(cache, n, src, dev_err);
    const int esz = gdn::dtype_size(cache->dtype);
    return launched(gdn::launch_kv_fork(a, src, dst, new_pages, vec_pages(a.k, a.d, esz) && vec_pages(a.v, a.d, esz),
                                        static_cast<cudaStream_t>(stream)), fn);
} catch (...) {
    return caught("kv_fork");
}

int64_t kv_compact_workspace(const kv_cache* cache) try {
    const int rc = check_cache("kv_compact_workspace", cache, 0);
    if (rc) return rc;
    return gdn::kv_plan_ints(cache->num_pages) * 4;
} catch (...) {
    return caught("kv_compact_workspace");
}

int kv_compact(const kv_cache* cache, int32_t* used, void* workspace, int64_t workspace_bytes, int32_t* dev_err,
               void* stream) try {
    const char* fn = "kv_compact";
    const int rc = check_cache(fn, cache, 1);
    if (rc) return rc;
    if (!used || !workspace || !dev_err) return fail(GDN_ERR_NULL, "%s: used, workspace or dev_err is NULL", fn);
    if (!aligned_to(used, 4) || !aligned_to(workspace, 16) || !aligned_to(dev_err, 4))
        return fail(GDN_ERR_ALIGN, "%s: used, workspace or dev_err misaligned", fn);
    const int64_t need = gdn::kv_plan_ints(cache->num_pages) * 4;
    if (workspace_bytes < need)
        return fail(GDN_ERR_SHAPE, "%s: workspace of %lld bytes, %lld needed", fn, (long long)workspace_bytes,
                    (long long)need);
    const gdn::KvArgs a = args_of(cache, 1, nullptr, dev_err);
    const int esz = gdn::dtype_size(cache->dtype);
    return launched(gdn::launch_kv_compact(a, static_cast<int32_t*>(workspace), used,
                                           vec_pages(a.k, a.d, esz) && vec_pages(a.v, a.d, esz),
                                           static_cast<cudaStream_t>(stream)), fn);
} catch (...) {
    return caught("kv_compact");
}

}  // extern "C"
