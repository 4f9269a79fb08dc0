// Rows for the paged 8-bit KV cache out of a projection (la_kv8_norm_rope):
// norm of each query and key head, its gain, the rotation by the position, one
// rounding to bf16; values are rounded alone.
//
//   n = x * rsqrt(mean(x^2) + eps) * w               (without w: n = x)
//   y_i = n_i cos a - n_{i+h} sin a,  y_{i+h} = n_{i+h} cos a + n_i sin a,  a = p f_i,  h = head_dim / 2
//
// Angles are kept as turns in 64-bit fixed point: p * (f / 2 pi) modulo 1 is one
// integer product whose high bits fall off, so far positions cost no accuracy
// and no reduction by 2 pi.
//
// A block takes some rows and some of their heads.  Its threads find the rows'
// positions and compute a row's sines and cosines once, for all of its heads,
// into shared memory; then HD / 16 lanes share a head, 8 rotary pairs each, so
// both halves of a pair are one lane's.
#include <algorithm>
#include <cmath>

#include "kv8.h"

namespace la {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 16;   // most rows of a block

struct RopeArgs {
    la_kv8_qkv a;
    const int *lens;
    uint32_t *status;
    int n_seqs, n_kv_heads;
    long long room;            // tokens a slot can hold
    int rows, heads;           // of a block
    uint64_t turn[64];         // f_i / 2 pi * 2^64, where inv_freq is not given
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int HD, typename T>
__global__ void __launch_bounds__(kRopeThreads) k_kv8_norm_rope(const __grid_constant__ RopeArgs p) {
    constexpr int H2 = HD / 2, L = HD / 16, ITEMS = kRopeThreads / L;   // lanes of a head; heads at a time
    __shared__ int sh_pos[kRopeRows];
    __shared__ int sh_on[kRopeRows];
    __shared__ __align__(16) float2 sh_cs[kRopeRows][H2];   // cos, sin; pair 8 j + 2 c (+ 1) of lane j at 2 (c L + j) (+ 1)
    __shared__ __align__(16) float sh_w[2][HD];
    const la_kv8_qkv &a = p.a;
    const int tid = threadIdx.x, r0 = blockIdx.x * p.rows, nr = min(p.rows, a.n_rows - r0);
    const int h_all = a.n_heads + p.n_kv_heads * (a.v ? 2 : 1), h0 = blockIdx.y * p.heads, nh = min(p.heads, h_all - h0);
    pdl_trigger();
    pdl_wait();
    // Positions of the block's rows
    if (tid < kRopeRows) {
        sh_on[tid] = tid < nr && (a.pos || (!a.row_start && r0 + tid < p.n_seqs));
        sh_pos[tid] = 0;
    }
    __syncthreads();
    if (a.pos) {
        if (tid < nr) sh_pos[tid] = a.pos[r0 + tid];
    } else {
        const int s_first = a.row_start ? tid : r0 + tid, s_last = a.row_start ? p.n_seqs : min(r0 + nr, p.n_seqs);
        for (int s = s_first; s < s_last; s += kRopeThreads) {
            int first = s, count = 1;
            if (a.row_start) {
                const int b = a.row_start[s + 1];
                first = a.row_start[s];
                count = first >= 0 && first <= b && b <= a.n_rows ? b - first : -1;
            }
            if (count < 0) atomicOr(p.status, LA_KV8_BAD);
            const int from = max(first, r0), to = min(first + count, r0 + nr);
            if (from >= to) continue;
            int len = p.lens[s];
            if (len < 0 || len > p.room) {
                atomicOr(p.status, LA_KV8_BAD);
                len = 0;
            }
            for (int r = from; r < to; ++r) {
                sh_pos[r - r0] = static_cast<int>(static_cast<unsigned>(len) + static_cast<unsigned>(a.depth ? a.depth[r] : r - first));
                sh_on[r - r0] = 1;
            }
        }
    }
    for (int i = tid; i < 2 * HD; i += kRopeThreads) {
        const void *w = i < HD ? a.q_weight : a.k_weight;
        const int d = i & (HD - 1);
        if (w) sh_w[i / HD][d] = a.weight_type == LA_F32 ? static_cast<const float *>(w)[d] : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[d]);
    }
    __syncthreads();
    for (int i = tid; i < nr * H2; i += kRopeThreads) {
        const int r = i / H2, k = i % H2;
        uint64_t f = p.turn[k];
        if (a.inv_freq) {
            const double x = static_cast<double>(a.inv_freq[k]) * 0.15915494309189533577;   // 1 / 2 pi
            f = __double2ull_rd((x - floor(x)) * 18446744073709551616.0);
        }
        const uint64_t t = f * static_cast<uint64_t>(static_cast<int64_t>(sh_pos[r]));   // turns * 2^64, modulo 2^64
        float s, c;
        sincospif(static_cast<float>(static_cast<int>(t >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns, -1 .. 1
        const int j = k >> 3, e = k & 7;
        sh_cs[r][2 * ((e >> 1) * L + j) + (e & 1)] = make_float2(c, s);
    }
    __syncthreads();

    const int j = tid % L;
#pragma unroll 2
    for (int i = tid / L; i < nr * nh; i += ITEMS) {   // whole groups of L lanes
        const int r = i / nh, head = h0 + i % nh, row = r0 + r;
        if (!sh_on[r]) continue;                       // rows of no slot stay as they are
        const int kind = head < a.n_heads ? 0 : head < a.n_heads + p.n_kv_heads ? 1 : 2;
        const int h = kind == 0 ? head : head - a.n_heads - (kind - 1) * p.n_kv_heads;
        const T *src = static_cast<const T *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + row * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + h * HD + 8 * j;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out) +
                             row * (kind == 0 ? a.q_out_stride : kind == 1 ? a.k_out_stride : a.v_out_stride) + h * HD + 8 * j;
        float x[8], y[8];
        load8(src, x);
        load8(src + H2, y);
        if (kind < 2) {
            if (kind == 0 ? a.q_weight : a.k_weight) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], fmaf(y[e], y[e], sum));
                const unsigned lanes = (L == 8 ? 0xffu : 0xfu) << (tid & 31 & ~(L - 1));
#pragma unroll
                for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(lanes, sum, o);
                const float n = rsqrtf(sum * (1.f / HD) + a.eps);
                const float4 *w = reinterpret_cast<const float4 *>(sh_w[kind] + 8 * j), *u = reinterpret_cast<const float4 *>(sh_w[kind] + H2 + 8 * j);
                const float4 w0 = w[0], w1 = w[1], u0 = u[0], u1 = u[1];
                const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w}, uu[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= n * ww[e];
                    y[e] *= n * uu[e];
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 t = *reinterpret_cast<const float4 *>(&sh_cs[r][2 * (c * L + j)]);
                const float a0 = x[2 * c], b0 = y[2 * c], a1 = x[2 * c + 1], b1 = y[2 * c + 1];
                x[2 * c] = a0 * t.x - b0 * t.y;
                y[2 * c] = b0 * t.x + a0 * t.y;
                x[2 * c + 1] = a1 * t.z - b1 * t.w;
                y[2 * c + 1] = b1 * t.z + a1 * t.w;
            }
        }
        store8(dst, x);
        store8(dst + H2, y);
    }
}

cudaError_t kv8_norm_rope_launch(const la_kv8_cache &c, const la_kv8_qkv &a, int nsm, cudaStream_t s) {
    if (a.n_rows < 1) return cudaSuccess;
    RopeArgs p{};
    p.a = a;
    p.lens = c.lens;
    p.status = c.status;
    p.n_seqs = c.n_seqs;
    p.n_kv_heads = c.n_kv_heads;
    p.room = static_cast<long long>(c.max_pages) * c.page;
    if (!a.inv_freq) {
        // f_i = base^(-2 i / head_dim); in turns, its part below one
        for (int i = 0; i < c.head_dim / 2; ++i) {
            const double x = std::pow(static_cast<double>(a.rope_base), -2.0 * i / c.head_dim) * 0.15915494309189533577;
            const double t = (x - std::floor(x)) * 18446744073709551616.0;
            p.turn[i] = t < 18446744073709549568.0 ? static_cast<uint64_t>(t) : ~0ull;
        }
    }
    const int items = kRopeThreads / (c.head_dim / 16), h_all = a.n_heads + c.n_kv_heads * (a.v ? 2 : 1);
    const long long all = static_cast<long long>(a.n_rows) * h_all, per = std::max<long long>(1, std::min<long long>(8, all / (static_cast<long long>(items) * nsm * 4)));
    // `per` passes of `items` heads for a block: as many rows as that takes, or a part of one row's heads
    p.rows = static_cast<int>(std::max<long long>(1, std::min<long long>(kRopeRows, per * items / h_all)));
    p.heads = p.rows > 1 || h_all <= per * items ? h_all : static_cast<int>(per * items);
    const dim3 grid((a.n_rows + p.rows - 1) / p.rows, (h_all + p.heads - 1) / p.heads);
    if (c.head_dim == 128)
        return a.type == LA_F32 ? launch_k(k_kv8_norm_rope<128, float>, grid, dim3(kRopeThreads), 0, s, p)
                                : launch_k(k_kv8_norm_rope<128, __nv_bfloat16>, grid, dim3(kRopeThreads), 0, s, p);
    return a.type == LA_F32 ? launch_k(k_kv8_norm_rope<64, float>, grid, dim3(kRopeThreads), 0, s, p)
                            : launch_k(k_kv8_norm_rope<64, __nv_bfloat16>, grid, dim3(kRopeThreads), 0, s, p);
}

}  // namespace la
