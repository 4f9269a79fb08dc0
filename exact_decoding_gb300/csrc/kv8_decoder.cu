// What a decoder over the paged 8-bit KV cache (la_create_kv8) runs besides
// the attention and the append: the QKV projection's rows turned into the
// attention's inputs, and the row lists of a pass and of a step's accepted
// rows (the winning candidate of "The Verification Branch", paper-graph-ui
// page, section 3.4).
#include "kv8.h"
#include "la_kernels.h"

namespace la {

// Sums the QKV GEMM's partial planes, rotates q and k, and writes bf16 rows
// q [nrows][nh * hd], k and v [nrows][nkv * hd].  One thread per 4 rotary
// pairs of q or k, or 8 dims of v.  Row r sits at position P + depth[r]
// (P + r when depth is null).  The sums and the rotation are fp32; the one
// rounding to bf16 (at most 2^-8 of the value) is what the attention over this cache
// takes, and for k and v it is far below the e4m3 step (2^-4) that they meet
// when they are appended.
__global__ void __launch_bounds__(256) k_kv8_qkv(const float *part, const int *planes, long long sstride, int ldp, int nh, int nkv,
                                                 int hd, int k_off, int v_off, const float2 *rope, const int *P_dev, int P0,
                                                 const int *depth, __nv_bfloat16 *q, __nv_bfloat16 *k, __nv_bfloat16 *v) {
    pdl_trigger();
    pdl_wait();
    const int r = blockIdx.y, t = blockIdx.x * 256 + threadIdx.x;
    const int half = hd / 2, per = half / 4, nq = nh * per, nk = nkv * per, nv = nkv * hd / 8;
    const float *pr = part + static_cast<long long>(r) * ldp;
    auto store4 = [](__nv_bfloat16 *dst, float a, float b, float c, float d) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
        *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    };
    float4 x, y;
    if (t < nq + nk) {
        const bool isq = t < nq;
        const int u = isq ? t : t - nq, head = u / per, j = 4 * (u % per);
        const int col = (isq ? 0 : k_off) + head * hd + j, np = planes ? planes[col >> 7] : 1;
        sum_planes4x2(pr + col, np, pr + col + half, np, sstride, x, y);
        const int pos = (P_dev ? *P_dev : P0) + (depth ? depth[r] : r);
        const float2 *c = rope + static_cast<long long>(pos) * half + j;
        const float4 c01 = *reinterpret_cast<const float4 *>(c), c23 = *reinterpret_cast<const float4 *>(c + 2);
        __nv_bfloat16 *dst = (isq ? q + static_cast<long long>(r) * nh * hd : k + static_cast<long long>(r) * nkv * hd) + head * hd + j;
        store4(dst, x.x * c01.x - y.x * c01.y, x.y * c01.z - y.y * c01.w, x.z * c23.x - y.z * c23.y, x.w * c23.z - y.w * c23.w);
        store4(dst + half, x.x * c01.y + y.x * c01.x, x.y * c01.w + y.y * c01.z, x.z * c23.y + y.z * c23.x, x.w * c23.w + y.w * c23.z);
    } else if (t < nq + nk + nv) {
        const int d = 8 * (t - nq - nk), col = v_off + d, np = planes ? planes[col >> 7] : 1;
        sum_planes4x2(pr + col, np, pr + col + 4, np, sstride, x, y);
        __nv_bfloat16 *dst = v + static_cast<long long>(r) * nkv * hd + d;
        store4(dst, x.x, x.y, x.z, x.w);
        store4(dst + 4, y.x, y.y, y.z, y.w);
    }
}

cudaError_t kv8_qkv_launch(const float *part, const int *planes, long long sstride, int ldp, int nrows, int nh, int nkv, int hd, int k_off,
                           int v_off, const float2 *rope, const int *P_dev, int P, const int *depth, __nv_bfloat16 *q, __nv_bfloat16 *k,
                           __nv_bfloat16 *v, cudaStream_t s) {
    const int items = (nh + nkv) * (hd / 8) + nkv * hd / 8;
    return launch_k(k_kv8_qkv, dim3((items + 255) / 256, nrows), dim3(256), 0, s, part, planes, sstride, ldp, nh, nkv, hd, k_off, v_off, rope,
                    P_dev, P, depth, q, k, v);
}

// row_start of a pass in which one slot has n rows; with a step's state, of
// its accepted rows (row 0, then the winning candidate's), whose numbers go
// to row_idx.
__global__ void __launch_bounds__(256) k_kv8_rows_of(int *row_start, int n_seqs, int slot, int n, const SpecState *st, int W, int N,
                                                     int *row_idx) {
    pdl_trigger();
    pdl_wait();
    const int rows = st ? st->A : n;
    for (int i = threadIdx.x; i <= n_seqs; i += 256) row_start[i] = i <= slot ? 0 : rows;
    if (st && threadIdx.x < rows && threadIdx.x < N)
        row_idx[threadIdx.x] = threadIdx.x == 0 ? 0 : 1 + (N - 1) * W + st->cstar * (N - 1) + static_cast<int>(threadIdx.x) - 1;
}
cudaError_t kv8_rows_of_launch(int *row_start, int n_seqs, int slot, int n, const SpecState *st, int W, int N, int *row_idx, cudaStream_t s) {
    return launch_k(k_kv8_rows_of, dim3(1), dim3(256), 0, s, row_start, n_seqs, slot, n, st, W, N, row_idx);
}

// After an append: were all rows stored, and does the slot hold the decoder's
// tokens?
__global__ void k_kv8_check(const int *row_start, const int *stored, const int *lens, const uint32_t *status, int slot, int tokens,
                            SpecState *st) {
    pdl_trigger();
    pdl_wait();
    if (stored[slot] != row_start[slot + 1] - row_start[slot]) st->err |= kErrKv8Full;
    else if (lens[slot] != (tokens < 0 ? st->P : tokens) || (*status & (LA_KV8_BAD | LA_KV8_TIMEOUT))) st->err |= kErrKv8Bad;
}
cudaError_t kv8_check_launch(const la_kv8_cache &c, const int *row_start, const int *stored, int slot, int tokens, SpecState *st,
                             cudaStream_t s) {
    return launch_k(k_kv8_check, dim3(1), dim3(1), 0, s, row_start, stored, static_cast<const int *>(c.lens),
                    static_cast<const uint32_t *>(c.status), slot, tokens, st);
}

}  // namespace la
