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
// both halves of a pair are one lane's, 16 bytes a load, and the norm is one
// reduction over 4 or 8 lanes.
//
// Memory bounds a prompt: 4096 rows of 72 heads of 128, bf16 (151 MB): 30.2 us,
// 5.0 TB/s, 74 % of a copy's rate (29.8 without the check of the mean); fp32 (226 MB)
// 39.9 us, 84 %.  What is left: a block finds positions and
// angles before its first load.  Hidden by other blocks of the SM, so registers
// are held to 48 (five blocks; four 32.1 us, eight with spills 39.7) and a lane
// has one head in flight (two: 30.7).  Up to 16 passes of heads a block (8:
// 30.2, 4: 32.4) while that leaves four blocks for every SM.  Tables lie so that the lanes
// of a head read 16 bytes side by side.  A single token (32 + 2 * 32 heads,
// fp32): 3.7 us, latency.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv8.h"

namespace la {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 16;   // most rows of a block
// Means of squares (with eps) between these are sums of fp32 squares that lose nothing: HD of
// them stay below 2^127, and a square that is not a normal number is below 2^-26 of them all.
constexpr float kLeastMean = 7.888609052210118e-31f, kMostMean = 1.329227995784916e36f;   // 2^-100, 2^120

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
// Two fp32 operations in one instruction
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float2 one_by_one(uint64_t v) {
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(v));
    return y;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
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

// 2^-e for x >= 0 in 2^e .. 2^(e + 1), within fp32's normal numbers
__device__ __forceinline__ float power_below(float x) { return __uint_as_float(min(max(254 - static_cast<int>(__float_as_uint(x) >> 23), 1), 254) << 23); }

template <int HD, typename T>
__global__ void __launch_bounds__(kRopeThreads, 5) k_kv8_norm_rope(const __grid_constant__ RopeArgs p) {
    constexpr int H2 = HD / 2, L = HD / 16, ITEMS = kRopeThreads / L;   // lanes of a head; heads at a time
    __shared__ int sh_pos[kRopeRows];
    __shared__ int sh_on[kRopeRows];
    // cos and sin of the pairs: pairs 8 j + 2 c and + 1 of lane j at [c][j]
    __shared__ __align__(16) ulonglong2 sh_cs[kRopeRows][4][L];
    // gains of q and of k: values 8 j + 2 c and + 1 of a head's two halves at [c][j]
    __shared__ __align__(16) ulonglong2 sh_w[2][4][L];
    const la_kv8_qkv &a = p.a;
    const int tid = threadIdx.x, r0 = blockIdx.x * p.rows, nr = min(p.rows, a.n_rows - r0);
    const int h_all = a.n_heads + p.n_kv_heads * (a.v ? 2 : 1), h0 = blockIdx.y * p.heads, nh = min(p.heads, h_all - h0);
    const int j = tid % L;
    // The block's heads of q, of k and of v: heads h0 .. h0 + nh - 1 of them all in a row
    auto part = [&](int from, int count, int &first) {
        first = min(max(h0 - from, 0), count);
        return max(min(h0 + nh - from, count), first) - first;
    };
    int q_first, k_first, v_first;
    const int q_heads = part(0, a.n_heads, q_first), k_heads = part(a.n_heads, p.n_kv_heads, k_first),
              v_heads = part(a.n_heads + p.n_kv_heads, a.v ? p.n_kv_heads : 0, v_first);
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
        const int e = d & 7, half = d / H2;
        float *to = reinterpret_cast<float *>(&sh_w[i / HD][e >> 1][(d - half * H2) >> 3]) + 2 * half + (e & 1);
        if (w) *to = a.weight_type == LA_F32 ? static_cast<const float *>(w)[d] : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[d]);
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
        const int e = k & 7;
        float *to = reinterpret_cast<float *>(&sh_cs[r][e >> 1][k >> 3]) + (e & 1);
        to[0] = c;
        to[2] = s;
    }
    __syncthreads();

    // Heads of one kind: `heads` of every row from `first` on, a group of L lanes
    // (whole in its warp) for each.
    auto heads_of = [&](auto rotated, const T *src, __nv_bfloat16 *dst, long long src_stride, long long dst_stride, int heads, int first, const void *weight, int kind) {
        if (heads < 1) return;
        const float per_row = 1.f / static_cast<float>(heads);
        src += r0 * src_stride + first * HD + 8 * j;
        dst += r0 * dst_stride + first * HD + 8 * j;
#pragma unroll 1
        for (int i = tid / L; i < nr * heads; i += ITEMS) {
            // i / heads: below 16 rows the quotient is off by less than the half that was added
            const int r = static_cast<int>((static_cast<float>(i) + 0.5f) * per_row), at = (i - r * heads) * HD;
            if (!sh_on[r]) continue;   // rows of no slot stay as they are
            float x[8], y[8];
            load8(src + r * src_stride + at, x);
            load8(src + r * src_stride + at + H2, y);
            if constexpr (decltype(rotated)::value) {
                uint64_t x2[4], y2[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    x2[c] = two(x[2 * c], x[2 * c + 1]);
                    y2[c] = two(y[2 * c], y[2 * c + 1]);
                }
                if (weight) {
                    uint64_t s2 = mul2(x2[0], x2[0]);
#pragma unroll
                    for (int c = 1; c < 4; ++c) s2 = fma2(x2[c], x2[c], s2);
#pragma unroll
                    for (int c = 0; c < 4; ++c) s2 = fma2(y2[c], y2[c], s2);
                    const float2 halves = one_by_one(s2);
                    float sum = halves.x + halves.y;
                    const unsigned lanes = (L == 8 ? 0xffu : 0xfu) << (tid & 31 & ~(L - 1));
#pragma unroll
                    for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(lanes, sum, o);
                    float mean = sum * (1.f / HD) + a.eps;
                    if (!(mean > kLeastMean && mean < kMostMean)) {
                        // The squares leave fp32's range: all by a power of two that brings the
                        // largest value, or the root of eps, near 1.  (A NaN or infinity stays one.)
                        float top = 0.f;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float2 u = one_by_one(x2[c]), v = one_by_one(y2[c]);
                            top = fmaxf(fmaxf(top, fmaxf(fabsf(u.x), fabsf(u.y))), fmaxf(fabsf(v.x), fabsf(v.y)));
                        }
#pragma unroll
                        for (int o = 1; o < L; o <<= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, o));
                        const float f = power_below(fmaxf(top, sqrtf(a.eps)));
                        const uint64_t f2 = two(f, f);
                        sum = 0.f;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            x2[c] = mul2(x2[c], f2);
                            y2[c] = mul2(y2[c], f2);
                            const float2 s = one_by_one(fma2(x2[c], x2[c], mul2(y2[c], y2[c])));
                            sum += s.x + s.y;
                        }
#pragma unroll
                        for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(lanes, sum, o);
                        mean = sum * (1.f / HD) + a.eps * f * f;
                    }
                    const float n = rsqrtf(mean);
                    const uint64_t n2 = two(n, n);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const ulonglong2 w = sh_w[kind][c][j];
                        x2[c] = mul2(mul2(x2[c], n2), w.x);
                        y2[c] = mul2(mul2(y2[c], n2), w.y);
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const ulonglong2 t = sh_cs[r][c][j];   // cosines, sines
                    const float2 p0 = one_by_one(fma2(y2[c], t.y ^ 0x8000000080000000ull, mul2(x2[c], t.x))),
                                 p1 = one_by_one(fma2(x2[c], t.y, mul2(y2[c], t.x)));
                    x[2 * c] = p0.x, x[2 * c + 1] = p0.y;
                    y[2 * c] = p1.x, y[2 * c + 1] = p1.y;
                }
            }
            store8(dst + r * dst_stride + at, x);
            store8(dst + r * dst_stride + at + H2, y);
        }
    };
    heads_of(std::true_type{}, static_cast<const T *>(a.q), static_cast<__nv_bfloat16 *>(a.q_out), a.q_stride, a.q_out_stride, q_heads, q_first, a.q_weight, 0);
    heads_of(std::true_type{}, static_cast<const T *>(a.k), static_cast<__nv_bfloat16 *>(a.k_out), a.k_stride, a.k_out_stride, k_heads, k_first, a.k_weight, 1);
    heads_of(std::false_type{}, static_cast<const T *>(a.v), static_cast<__nv_bfloat16 *>(a.v_out), a.v_stride, a.v_out_stride, v_heads, v_first, nullptr, 0);
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
        // f_i = base^(-2 i / head_dim), a power for i / 8 times one for i % 8 (a
        // quarter of the powers, two roundings more); in turns, its part below one
        double low[8], high = 1.;
        for (int i = 0; i < c.head_dim / 2; ++i) {
            const auto power = [&](int n) { return std::pow(static_cast<double>(a.rope_base), -2.0 * n / c.head_dim); };
            if (i < 8) low[i] = power(i) * 0.15915494309189533577;
            if (i % 8 == 0 && i) high = power(i);
            const double x = high * low[i % 8];
            const double t = (x - std::floor(x)) * 18446744073709551616.0;
            p.turn[i] = t < 18446744073709549568.0 ? static_cast<uint64_t>(t) : ~0ull;
        }
    }
    const int items = kRopeThreads / (c.head_dim / 16), h_all = a.n_heads + c.n_kv_heads * (a.v ? 2 : 1);
    const long long all = static_cast<long long>(a.n_rows) * h_all, per = std::max<long long>(1, std::min<long long>(16, all / (static_cast<long long>(items) * nsm * 4)));
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
