// The paged 8-bit KV cache: what its kernels share, and the launch functions
// behind la_kv8_* (include/la.h).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "../../include/la.h"
#include "la_common.cuh"

namespace la {

constexpr int kKv8MinExp = -60, kKv8MaxExp = 60;

// One page's number, checked: -1 (and the BAD bit) when the table entry names no page.
__device__ __forceinline__ int kv8_page(const la_kv8_cache &c, int slot, int j) {
    if (j >= c.max_pages) return -1;
    const int p = c.table[static_cast<long long>(slot) * c.max_pages + j];
    if (static_cast<unsigned>(p) < static_cast<unsigned>(c.n_pages)) return p;
    atomicOr(c.status, LA_KV8_BAD);
    return -1;
}
// Tokens of a slot, checked against the table's room.
__device__ __forceinline__ int kv8_len(const la_kv8_cache &c, int slot) {
    const int n = c.lens[slot];
    if (n >= 0 && n <= static_cast<long long>(c.max_pages) * c.page) return n;
    atomicOr(c.status, LA_KV8_BAD);
    return 0;
}
// Rows [*first, *first + count) of a slot, 0 rows (and the BAD bit) if row_start is out of order.
__device__ __forceinline__ int kv8_rows(const la_kv8_cache &c, const int *row_start, int n_rows, int slot, int *first) {
    if (!row_start) {
        *first = slot;
        return slot < n_rows ? 1 : 0;
    }
    const int a = row_start[slot], b = row_start[slot + 1];
    *first = a;
    if (a >= 0 && a <= b && b <= n_rows) return b - a;
    atomicOr(c.status, LA_KV8_BAD);
    return 0;
}
// Byte offset of (layer, page, KV head) in k or v, and its index in the scales.
__device__ __forceinline__ long long kv8_block(const la_kv8_cache &c, int layer, int page, int head) {
    return (static_cast<long long>(layer) * c.n_pages + page) * c.n_kv_heads + head;
}

// Pages that m >= 1 consecutive tokens can touch.
__host__ __device__ inline int kv8_touched(int m, int page) { return m == 1 ? 1 : (m - 2) / page + 2; }

// Workspace of one cache: the attention's partial results, or the plans of
// append and compact (calls that overlap need a workspace each).
int64_t kv8_workspace_bytes(const la_kv8_cache &c, int nsm);
// *launched (or nullptr) grows by the kernels launched.
cudaError_t kv8_attention_launch(const la_kv8_cache &c, const la_kv8_attn &a, void *ws, int nsm, cudaStream_t s,
                                 int64_t *launched = nullptr);
cudaError_t kv8_append_launch(const la_kv8_cache &c, const la_kv8_rows &r, int *ws, cudaStream_t s);
cudaError_t kv8_fork_launch(const la_kv8_cache &c, const int *src, const int *dst, int n, cudaStream_t s);
cudaError_t kv8_free_launch(const la_kv8_cache &c, const int *slots, const int *keep, int n, cudaStream_t s);
cudaError_t kv8_compact_launch(const la_kv8_cache &c, int *table_out, int *refs_out, int *n_live, int *ws, int nsm,
                               cudaStream_t s);

// Checks of a cache's sizes and pointers (an error code, with the message set).
int kv8_check_cache(const la_kv8_cache *c, const char *where);

// ------------------------------------------------------------------ decoders over the cache
struct SpecState;
// Step-state error bits: the cache had no room for a pass's rows; the slot
// does not hold the decoder's tokens, or the cache's status word has
// LA_KV8_BAD or LA_KV8_TIMEOUT.
constexpr unsigned kErrKv8Full = 128u, kErrKv8Bad = 256u;
cudaError_t kv8_qkv_launch(const float *part, const int *planes, long long sstride, int ldp, int nrows, int nh, int nkv, int hd, int k_off,
                           int v_off, const float2 *rope, const int *P_dev, int P, const int *depth, __nv_bfloat16 *q, __nv_bfloat16 *k,
                           __nv_bfloat16 *v, cudaStream_t s);
cudaError_t kv8_rows_of_launch(int *row_start, int n_seqs, int slot, int n, const SpecState *st, int W, int N, int *row_idx, cudaStream_t s);
// tokens: the slot's length afterwards, or -1: the step state's P.
cudaError_t kv8_check_launch(const la_kv8_cache &c, const int *row_start, const int *stored, int slot, int tokens, SpecState *st,
                             cudaStream_t s);

}  // namespace la
