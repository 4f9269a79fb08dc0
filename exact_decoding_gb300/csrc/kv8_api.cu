// Entry points of the paged 8-bit KV cache (la_kv8_*, include/la.h): argument
// checks on the host, then launches on the caller's stream.
#include <atomic>
#include <cstdio>

#include "abi_guard.h"
#include "kv8.h"

using namespace la;

namespace {

int bad(const char *where, const char *what, int code = LA_ERR_INVALID_ARG) {
    char msg[256];
    std::snprintf(msg, sizeof(msg), "%s: %s", where, what);
    return set_last_error(code, msg);
}
int cuda_failed(const char *where, cudaError_t e) { return bad(where, cudaGetErrorString(e), LA_ERR_CUDA); }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int la::kv8_check_cache(const la_kv8_cache *c, const char *where) {
    if (!c) return bad(where, "null cache");
    if (c->head_dim != 64 && c->head_dim != 128) return bad(where, "head_dim must be 64 or 128", LA_ERR_UNSUPPORTED);
    if (c->page != 32 && c->page != 64 && c->page != 128) return bad(where, "page must be 32, 64 or 128", LA_ERR_UNSUPPORTED);
    if (c->n_layers < 1 || c->n_layers > 32767 || c->n_pages < 1 || c->n_pages > (1 << 24) || c->n_kv_heads < 1 ||
        c->n_kv_heads > 1024 || c->n_seqs < 1 || c->n_seqs > LA_KV8_MAX_SEQS || c->max_pages < 1 ||
        static_cast<int64_t>(c->max_pages) * c->page > (1 << 30))
        return bad(where, "cache sizes out of range (n_layers 1..32767, n_pages 1..2^24, n_kv_heads 1..1024, n_seqs 1..2048, "
                          "max_pages * page <= 2^30)");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->table || !c->lens || !c->refs || !c->status)
        return bad(where, "null cache array");
    if (!aligned16(c->k) || !aligned16(c->v)) return bad(where, "k and v must be 16-byte aligned");
    return LA_OK;
}

namespace {

int sm_count(int *n) {
    static std::atomic<int> cached[64] = {};   // 0: not asked yet; any thread writes the same value
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_failed("cudaGetDevice", e);
    if (dev >= 0 && dev < 64 && cached[dev]) {
        *n = cached[dev];
        return LA_OK;
    }
    e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_failed("cudaDeviceGetAttribute", e);
    if (dev >= 0 && dev < 64) cached[dev] = *n;
    return LA_OK;
}

int check_workspace(const la_kv8_cache *c, const void *ws, int64_t bytes, int *nsm, const char *where) {
    const int rc = sm_count(nsm);
    if (rc != LA_OK) return rc;
    if (!ws || !aligned16(ws)) return bad(where, "workspace must be 16-byte aligned device memory");
    if (bytes < kv8_workspace_bytes(*c, *nsm)) return bad(where, "workspace too small (see la_kv8_workspace)", LA_ERR_CAPACITY);
    return LA_OK;
}

int workspace_body(const la_kv8_cache *c, int64_t *bytes) {
    int rc = kv8_check_cache(c, "la_kv8_workspace"), nsm = 0;
    if (rc != LA_OK) return rc;
    if (!bytes) return bad("la_kv8_workspace", "null argument");
    if ((rc = sm_count(&nsm)) != LA_OK) return rc;
    *bytes = kv8_workspace_bytes(*c, nsm);
    return LA_OK;
}

int attention_body(const la_kv8_cache *c, const la_kv8_attn *args, void *ws, int64_t ws_bytes, void *stream) {
    const char *where = "la_kv8_attention";
    int rc = kv8_check_cache(c, where);
    if (rc != LA_OK) return rc;
    if (!args) return bad(where, "null arguments");
    la_kv8_attn a = *args;
    if (a.layer < 0 || a.layer >= c->n_layers) return bad(where, "layer out of range");
    if (a.n_heads < 1 || a.n_heads % c->n_kv_heads) return bad(where, "n_heads must be a multiple of n_kv_heads");
    if (a.n_heads / c->n_kv_heads > 256) return bad(where, "more than 256 query heads per KV head", LA_ERR_UNSUPPORTED);
    if (a.n_rows < 0 || a.n_rows > (1 << 22)) return bad(where, "n_rows out of range (0 .. 2^22)");
    if (!a.row_start && a.n_rows != c->n_seqs) return bad(where, "without row_start every slot has one row: n_rows must be n_seqs");
    if (!a.k != !a.v) return bad(where, "k and v come together or not at all");
    if (!(a.scale >= 0.f) || a.scale > 3e38f) return bad(where, "scale must be a finite number, not negative");
    const int64_t qd = static_cast<int64_t>(a.n_heads) * c->head_dim, kd = static_cast<int64_t>(c->n_kv_heads) * c->head_dim;
    if (a.n_rows > 0) {
        if (!a.q || !a.out) return bad(where, "null q or out");
        if (!aligned16(a.q) || !aligned16(a.out) || !aligned16(a.k) || !aligned16(a.v))
            return bad(where, "q, k, v and out must be 16-byte aligned");
        if (a.q_stride < qd || a.out_stride < qd || a.q_stride % 8 || a.out_stride % 8)
            return bad(where, "q_stride and out_stride must be multiples of 8 and at least n_heads * head_dim");
        if (a.k && (a.k_stride < kd || a.v_stride < kd || a.k_stride % 8 || a.v_stride % 8))
            return bad(where, "k_stride and v_stride must be multiples of 8 and at least n_kv_heads * head_dim");
    }
    if (a.scale == 0.f) a.scale = c->head_dim == 128 ? 0.08838834764831845f : 0.125f;
    int nsm = 0;
    if ((rc = check_workspace(c, ws, ws_bytes, &nsm, where)) != LA_OK) return rc;
    const cudaError_t e = kv8_attention_launch(*c, a, ws, nsm, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LA_OK : cuda_failed(where, e);
}

int append_body(const la_kv8_cache *c, const la_kv8_rows *rows, void *ws, int64_t ws_bytes, void *stream) {
    const char *where = "la_kv8_append";
    int rc = kv8_check_cache(c, where);
    if (rc != LA_OK) return rc;
    if (!rows) return bad(where, "null arguments");
    la_kv8_rows r = *rows;
    if (r.n_rows < 0 || r.n_rows > (1 << 24)) return bad(where, "n_rows out of range (0 .. 2^24)");
    if (!r.row_start && r.n_rows != c->n_seqs) return bad(where, "without row_start every slot gets one row: n_rows must be n_seqs");
    if (!r.stored) return bad(where, "null stored");
    if (r.n_src <= 0) r.n_src = r.n_rows;
    if (!r.row_idx && r.n_src < r.n_rows) return bad(where, "n_src is less than n_rows");
    const int64_t kd = static_cast<int64_t>(c->n_kv_heads) * c->head_dim;
    if (r.n_rows > 0) {
        if (!r.k || !r.v || !aligned16(r.k) || !aligned16(r.v)) return bad(where, "k and v must be 16-byte aligned device memory");
        if (r.k_stride < kd || r.v_stride < kd || r.k_stride % 8 || r.v_stride % 8)
            return bad(where, "k_stride and v_stride must be multiples of 8 and at least n_kv_heads * head_dim");
        if (c->n_layers > 1 && (r.k_layer_stride < 0 || r.v_layer_stride < 0 || r.k_layer_stride % 8 || r.v_layer_stride % 8))
            return bad(where, "layer strides must be multiples of 8 and not negative");
    }
    if (!r.row_start) r.max_rows = 1;
    if (r.max_rows <= 0 || r.max_rows > r.n_rows) r.max_rows = r.n_rows;
    if (r.max_rows < 1) r.max_rows = 1;
    if (static_cast<int64_t>(c->n_seqs) * kv8_touched(r.max_rows, c->page) > 0x7fffffffll)
        return bad(where, "n_seqs * max_rows too large for one call");
    int nsm = 0;
    if ((rc = check_workspace(c, ws, ws_bytes, &nsm, where)) != LA_OK) return rc;
    const cudaError_t e = kv8_append_launch(*c, r, static_cast<int *>(ws), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LA_OK : cuda_failed(where, e);
}

int fork_body(const la_kv8_cache *c, const int32_t *src, const int32_t *dst, int32_t n, void *stream) {
    const char *where = "la_kv8_fork";
    const int rc = kv8_check_cache(c, where);
    if (rc != LA_OK) return rc;
    if (n < 0 || n > LA_KV8_MAX_SEQS) return bad(where, "n out of range (0 .. LA_KV8_MAX_SEQS)");
    if (n > 0 && (!src || !dst)) return bad(where, "null src or dst");
    const cudaError_t e = kv8_fork_launch(*c, src, dst, n, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LA_OK : cuda_failed(where, e);
}

int free_body(const la_kv8_cache *c, const int32_t *slots, const int32_t *keep, int32_t n, void *stream) {
    const char *where = "la_kv8_free";
    const int rc = kv8_check_cache(c, where);
    if (rc != LA_OK) return rc;
    if (n < 0 || n > (1 << 20)) return bad(where, "n out of range (0 .. 2^20)");
    if (n > 0 && !slots) return bad(where, "null slots");
    const cudaError_t e = kv8_free_launch(*c, slots, keep, n, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LA_OK : cuda_failed(where, e);
}

int compact_body(const la_kv8_cache *c, int32_t *table_out, int32_t *refs_out, int32_t *n_live, void *ws, int64_t ws_bytes,
                 void *stream) {
    const char *where = "la_kv8_compact";
    int rc = kv8_check_cache(c, where), nsm = 0;
    if (rc != LA_OK) return rc;
    if (!table_out || !refs_out) return bad(where, "null table_out or refs_out");
    if ((rc = check_workspace(c, ws, ws_bytes, &nsm, where)) != LA_OK) return rc;
    const cudaError_t e = kv8_compact_launch(*c, table_out, refs_out, n_live, static_cast<int *>(ws), nsm,
                                             static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LA_OK : cuda_failed(where, e);
}

int status_body(const la_kv8_cache *c, uint32_t *out, void *stream) {
    const char *where = "la_kv8_status";
    const int rc = kv8_check_cache(c, where);
    if (rc != LA_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t bits = 0;
    cudaError_t e = cudaMemcpyAsync(&bits, c->status, sizeof(bits), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(c->status, 0, sizeof(bits), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_failed(where, e);
    if (out) *out = bits;
    if (bits & LA_KV8_TIMEOUT) return bad(where, "a bounded wait gave up; that call's output is void", LA_ERR_DEVICE_TIMEOUT);
    if (bits & LA_KV8_BAD) return bad(where, "a page, slot, length or row outside the cache, or a refused fork", LA_ERR_STATE);
    if (bits & LA_KV8_FULL) return bad(where, "no free page or table entry left for a sequence's rows", LA_ERR_CAPACITY);
    return LA_OK;
}

}  // namespace

extern "C" {

int la_kv8_workspace(const la_kv8_cache *c, int64_t *bytes) {
    return abi_guard("la_kv8_workspace", [&] { return workspace_body(c, bytes); });
}
int la_kv8_attention(const la_kv8_cache *c, const la_kv8_attn *a, void *workspace, int64_t workspace_bytes, void *stream) {
    return abi_guard("la_kv8_attention", [&] { return attention_body(c, a, workspace, workspace_bytes, stream); });
}
int la_kv8_append(const la_kv8_cache *c, const la_kv8_rows *r, void *workspace, int64_t workspace_bytes, void *stream) {
    return abi_guard("la_kv8_append", [&] { return append_body(c, r, workspace, workspace_bytes, stream); });
}
int la_kv8_fork(const la_kv8_cache *c, const int32_t *src, const int32_t *dst, int32_t n, void *stream) {
    return abi_guard("la_kv8_fork", [&] { return fork_body(c, src, dst, n, stream); });
}
int la_kv8_free(const la_kv8_cache *c, const int32_t *slots, const int32_t *keep, int32_t n, void *stream) {
    return abi_guard("la_kv8_free", [&] { return free_body(c, slots, keep, n, stream); });
}
int la_kv8_compact(const la_kv8_cache *c, int32_t *table_out, int32_t *refs_out, int32_t *n_live, void *workspace,
                   int64_t workspace_bytes, void *stream) {
    return abi_guard("la_kv8_compact",
                     [&] { return compact_body(c, table_out, refs_out, n_live, workspace, workspace_bytes, stream); });
}
int la_kv8_status(const la_kv8_cache *c, uint32_t *bits, void *stream) {
    return abi_guard("la_kv8_status", [&] { return status_body(c, bits, stream); });
}

}  // extern "C"
