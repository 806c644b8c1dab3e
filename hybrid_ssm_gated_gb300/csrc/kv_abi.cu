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

}  // extern "C"
