// Appending to the paged 8-bit KV cache, and the bookkeeping of its pages:
// forking, freeing and compacting sequences.
//
// A step's accepted rows (the lookahead window's winners, "The Verification
// Branch" of the paper-graph-ui page, section 3.4) enter the cache here as
// e4m3 bytes; the pages say nothing of 8-bit or paged caches.
#include <algorithm>

#include "kv8.h"

namespace la {

// ------------------------------------------------------------------ scans
// Exclusive prefix of v over the block in thread order; the block's sum in *tot.
__device__ __forceinline__ int block_scan(int v, int *warp_tot, int *tot) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_tot[w] = incl;
    __syncthreads();
    if (w == 0) {
        int x = lane < nw ? warp_tot[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        warp_tot[lane] = x;
    }
    __syncthreads();
    *tot = warp_tot[nw - 1];
    const int r = incl - v + (w ? warp_tot[w - 1] : 0);
    __syncthreads();
    return r;
}

// ------------------------------------------------------------------ append: pages
constexpr int kPlanThreads = 1024;

// One CTA decides for every sequence which pages its new rows need, before
// any byte moves.  Whether a page is free or shared is taken from refs as
// they stand at the start, so a page that one sequence copies away from is
// neither written nor handed out again within the call, and the answer does
// not depend on the order in which threads run.
//   ws: record[n_seqs] for the kernels that write the bytes (rows, length
//       before them, page that holds the stored tokens of the first touched
//       page or -1, that page's new place), take[n_seqs] pages wanted (bit 30:
//       the last page is copied), base[n_seqs] first of them in the list,
//       list[] free pages.
__global__ void __launch_bounds__(kPlanThreads) k_kv8_plan(la_kv8_cache c, const int *row_start, int n_rows,
                                                           int max_rows, int *stored, int *ws) {
    pdl_trigger();
    pdl_wait();
    constexpr int kCopy = 1 << 30;
    __shared__ int warp_tot[32];
    int4 *record = reinterpret_cast<int4 *>(ws);
    int *take = ws + 4 * c.n_seqs, *base = take + c.n_seqs, *list = base + c.n_seqs;
    const int tid = threadIdx.x;
    // What each sequence wants; base: its place in the list if all fit.
    int wanted = 0;
    for (int s0 = 0; s0 < c.n_seqs; s0 += kPlanThreads) {
        const int s = s0 + tid;
        int need = 0, copy = 0;
        if (s < c.n_seqs) {
            int first, from = -1;
            int n = kv8_rows(c, row_start, n_rows, s, &first);
            const int len = kv8_len(c, s);
            if (n > max_rows || c.lens[s] != len) {
                atomicOr(c.status, LA_KV8_BAD);
                n = 0;
            }
            if (n > 0) {
                const long long held = (len + c.page - 1) / c.page, want = (static_cast<long long>(len) + n + c.page - 1) / c.page;
                if (want > c.max_pages) {
                    atomicOr(c.status, LA_KV8_FULL);
                    n = 0;
                } else {
                    need = static_cast<int>(want - held);
                    if (len % c.page) {
                        from = kv8_page(c, s, len / c.page);
                        if (from < 0) n = need = 0;
                        else if (c.refs[from] > 1) copy = 1;
                    }
                }
            }
            stored[s] = n;
            record[s] = make_int4(n, len, from, -1);
        }
        int tot;
        const int at = block_scan(need + copy, warp_tot, &tot);
        if (s < c.n_seqs) {
            take[s] = (need + copy) | (copy ? kCopy : 0);
            base[s] = wanted + at;
        }
        wanted += tot;
    }
    // The lowest free pages, as many as are wanted.
    int found = 0;
    for (int p0 = 0; p0 < c.n_pages && found < wanted; p0 += 4 * kPlanThreads) {
        int free4 = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + 4 * tid + i;
            if (p < c.n_pages && c.refs[p] == 0) free4 |= 1 << i;
        }
        int tot;
        int at = found + block_scan(__popc(free4), warp_tot, &tot);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((free4 >> i) & 1) {
                if (at < wanted) list[at] = p0 + 4 * tid + i;
                ++at;
            }
        found += tot;
    }
    __syncthreads();
    // Too few: in the order of the slots, those that still fit.
    if (found < wanted && tid == 0) {
        int used = 0;
        for (int s = 0; s < c.n_seqs; ++s) {
            const int t = take[s] & ~kCopy;
            if (!stored[s]) continue;
            if (t > found - used) {
                stored[s] = 0;
                atomicOr(c.status, LA_KV8_FULL);
                continue;
            }
            base[s] = used;
            used += t;
        }
    }
    __syncthreads();
    // Table, references and lengths: one warp per sequence.
    const int lane = tid & 31;
    for (int s = tid >> 5; s < c.n_seqs; s += kPlanThreads / 32) {
        const int n = stored[s];
        if (!n) {
            if (lane == 0) record[s].x = 0;
            continue;
        }
        const int t = take[s] & ~kCopy, len = record[s].y, from = record[s].z;
        const bool copy = take[s] & kCopy;
        const int begin = copy ? len / c.page : (len + c.page - 1) / c.page;
        int *row = c.table + static_cast<long long>(s) * c.max_pages;
        for (int i = lane; i < t; i += 32) {
            const int p = list[base[s] + i];
            row[begin + i] = p;
            c.refs[p] = 1;
        }
        if (lane == 0) {
            if (copy) atomicSub(&c.refs[from], 1);
            record[s].w = copy || from < 0 ? list[base[s]] : from;
            c.lens[s] = len + n;
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------ append: bytes
__device__ __forceinline__ int kv8_exponent(float amax) {
    const unsigned b = __float_as_uint(amax);
    const int e = static_cast<int>(b >> 23) - ((b & 0x7fffffu) <= 0x600000u ? 135 : 134);   // amax <= 448 * 2^e
    return min(max(e, kKv8MinExp), kKv8MaxExp);
}
__device__ __forceinline__ int kv8_scale_exponent(float scale) {
    const int e = static_cast<int>((__float_as_uint(scale) >> 23) & 255u) - 127;
    return min(max(e, kKv8MinExp), kKv8MaxExp);
}
__device__ __forceinline__ float kv8_power(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }
__device__ __forceinline__ bool finite_f(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }
// Nearest e4m3 (ties to even); magnitudes past 448 clamp, NaN and infinities become NaN.
__device__ __forceinline__ uint32_t kv8_byte(float x) {
    return finite_f(x) ? static_cast<uint32_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3)) : 0x7fu;
}
__device__ __forceinline__ float kv8_value(uint32_t b) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3)));
}
// A stored byte at a scale 2^-shift of what it was, shift >= 0.
__device__ __forceinline__ uint32_t kv8_shrink(uint32_t b, float f) {
    return (b & 0x7fu) == 0x7fu ? b : kv8_byte(kv8_value(b) * f);
}

// Two elements to two bytes, both finite (e4m3 of lo in the low byte).
__device__ __forceinline__ uint32_t kv8_pair(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// Largest magnitude of bf16 pairs, NaN if any is NaN.
__device__ __forceinline__ uint32_t kv8_max2(uint32_t m, uint32_t x) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
    return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// The same among finite elements only, where the fast maximum met others.
__device__ __forceinline__ float kv8_finite_max(float m, uint32_t w) {
    if (finite_f(bf16_lo(w))) m = fmaxf(m, fabsf(bf16_lo(w)));
    if (finite_f(bf16_hi(w))) m = fmaxf(m, fabsf(bf16_hi(w)));
    return m;
}

constexpr int kStoreThreads = 128;

// One CTA per (sequence, touched page, KV head, layer, K or V): the page's
// new rows go through shared memory once, for the largest magnitude and then
// for the bytes (V is transposed on the way).  Bound by memory: 2048 rows x 40
// layers x 8 heads, 336 MB in and 168 MB out, take 91.5 us (5.5 TB/s) with 128
// threads and 8 loads of each in flight; 256 threads, 4 loads: 109; 64 threads, 8
// loads: 104.5; 256 threads, 8 loads: 131 (too few CTAs on an SM).
template <int HD>
__global__ void __launch_bounds__(kStoreThreads) k_kv8_store(la_kv8_cache c, la_kv8_rows r, const int4 *record, int touched) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ __align__(16) __nv_bfloat16 sm[];            // [page] rows, 16 elements more after every 16: see V below
    __shared__ float red[kStoreThreads / 32];
    const int s = blockIdx.x / touched, j = blockIdx.x % touched;
    const int head = blockIdx.y, layer = blockIdx.z >> 1, isv = blockIdx.z & 1;
    const int4 rec = record[s];
    const int first = r.row_start ? r.row_start[s] : s;
    const int n = rec.x, len = rec.y;
    if (n <= 0) return;
    const int pj = len / c.page + j;
    const int a = j == 0 ? len % c.page : 0;                       // tokens of this page that are stored already
    const long long left = static_cast<long long>(len) + n - static_cast<long long>(pj) * c.page;
    if (left <= 0) return;
    const int b = static_cast<int>(min(left, static_cast<long long>(c.page)));
    const int to = j == 0 ? rec.w : kv8_page(c, s, pj), from = a > 0 ? rec.z : -1;
    if (to < 0) return;
    const int row0 = first + pj * c.page + a - len;
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(isv ? r.v : r.k) +
                             layer * (isv ? r.v_layer_stride : r.k_layer_stride) + static_cast<long long>(head) * HD;
    const long long stride = isv ? r.v_stride : r.k_stride;
    const int tid = threadIdx.x, n_src = r.n_src;
    auto place = [](int t, int d) { return t * HD + (t >> 4) * 16 + d; };

    uint32_t top = 0;
    constexpr int C = HD / 8, RT = kStoreThreads / C, B = 8;       // 16-byte pieces of a row; rows of a sweep; loads in flight
    const int d0 = (tid % C) * 8;
    for (int t0 = tid / C; t0 < b - a; t0 += B * RT) {
        uint4 w[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int t = t0 + k * RT;
            w[k] = make_uint4(0, 0, 0, 0);
            if (t >= b - a) continue;
            const int row = r.row_idx ? r.row_idx[row0 + t] : row0 + t;
            if (static_cast<unsigned>(row) < static_cast<unsigned>(n_src)) w[k] = *reinterpret_cast<const uint4 *>(x + row * stride + d0);
            else atomicOr(c.status, LA_KV8_BAD);                   // stored as zeros
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int t = t0 + k * RT;
            if (t < b - a) *reinterpret_cast<uint4 *>(sm + place(a + t, d0)) = w[k];
            top = kv8_max2(kv8_max2(kv8_max2(kv8_max2(top, w[k].x), w[k].y), w[k].z), w[k].w);
        }
    }
    // Every element finite?  Else the maximum is taken again among those that are.
    float amax = fmaxf(bf16_lo(top), bf16_hi(top));
    const bool odd = __syncthreads_or(!finite_f(bf16_lo(top)) || !finite_f(bf16_hi(top)));
    if (odd) {
        amax = 0.f;
        for (int i = tid; i < (b - a) * (HD / 2); i += kStoreThreads)
            amax = kv8_finite_max(amax, *reinterpret_cast<const uint32_t *>(sm + place(a + i / (HD / 2), 2 * (i % (HD / 2)))));
    }
    amax = warp_max(amax);
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kStoreThreads / 32; ++w) amax = fmaxf(amax, red[w]);

    float *scales = isv ? c.v_scale : c.k_scale;
    uint8_t *pool = static_cast<uint8_t *>(isv ? c.v : c.k);
    const long long blk = kv8_block(c, layer, to, head), old = from >= 0 ? kv8_block(c, layer, from, head) : 0;
    const long long bytes = static_cast<long long>(c.page) * HD;
    const int e_old = from >= 0 ? kv8_scale_exponent(scales[old]) : kKv8MinExp;
    const int e = max(e_old, kv8_exponent(amax));
    uint8_t *out = pool + blk * bytes;
    __syncthreads();                                               // every thread has read the old scale
    if (tid == 0) scales[blk] = kv8_power(e);
    // Stored tokens: in a new place, or at a grown scale.
    if (from >= 0 && (e > e_old || from != to)) {
        const uint8_t *was = pool + old * bytes;
        const float f = kv8_power(e_old - e);
        for (int i = tid; i < a * HD; i += kStoreThreads) {
            const int at = isv ? (i / a) * c.page + i % a : i;
            out[at] = static_cast<uint8_t>(kv8_shrink(was[at], f));
        }
    }
    // New tokens.
    const float f = kv8_power(-e);
    if (!isv) {
        auto put = [&](auto pair) {
            for (int i = tid; i < (b - a) * (HD / 16); i += kStoreThreads) {
                const int t = a + i / (HD / 16), d = (i % (HD / 16)) * 16;
                const uint4 lo = *reinterpret_cast<const uint4 *>(sm + place(t, d)), hi = *reinterpret_cast<const uint4 *>(sm + place(t, d + 8));
                *reinterpret_cast<uint4 *>(out + t * HD + d) = make_uint4(pair(lo.x) | pair(lo.y) << 16, pair(lo.z) | pair(lo.w) << 16,
                                                                          pair(hi.x) | pair(hi.y) << 16, pair(hi.z) | pair(hi.w) << 16);
            }
        };
        if (odd) put([f](uint32_t w) { return kv8_byte(bf16_lo(w) * f) | kv8_byte(bf16_hi(w) * f) << 8; });
        else put([f](uint32_t w) { return kv8_pair(bf16_lo(w) * f, bf16_hi(w) * f); });
    } else {
        // 16 tokens of two neighbouring dims per thread; a warp covers whole
        // runs of a dim's tokens, and the padding spreads their reads over the banks.
        const int log2 = c.page == 32 ? 1 : c.page == 64 ? 2 : 3;  // 16-token pieces of a page
        for (int i = tid; i < HD / 2 << log2; i += kStoreThreads) {
            const int d = 2 * (i >> log2), t0 = (i & ((1 << log2) - 1)) * 16;
            uint8_t *dst = out + static_cast<long long>(d) * c.page + t0;
            if (t0 >= a && t0 + 16 <= b && !odd) {
                uint32_t w[2][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t u[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) u[q] = *reinterpret_cast<const uint32_t *>(sm + place(t0 + 4 * k + q, d));
                    w[0][k] = kv8_pair(bf16_lo(u[0]) * f, bf16_lo(u[1]) * f) | kv8_pair(bf16_lo(u[2]) * f, bf16_lo(u[3]) * f) << 16;
                    w[1][k] = kv8_pair(bf16_hi(u[0]) * f, bf16_hi(u[1]) * f) | kv8_pair(bf16_hi(u[2]) * f, bf16_hi(u[3]) * f) << 16;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4 *>(dst + h * c.page) = make_uint4(w[h][0], w[h][1], w[h][2], w[h][3]);
            } else {
                for (int t = max(t0, a); t < min(t0 + 16, b); ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        dst[h * c.page + t - t0] = static_cast<uint8_t>(kv8_byte(__bfloat162float(sm[place(t, d + h)]) * f));
            }
        }
    }
}

// A decoding step appends a row or a few to each sequence: one warp per
// (sequence, touched page, KV head, layer, K or V), a CTA for the heads of one
// (sequence, page, layer).  A CTA per block, as above, spends its time on
// launching and barriers for 256 bytes of input.  What bounds it are V's bytes:
// a token has one byte in each dim's row, so a sector of 32 bytes is read and
// written for each (64 sequences x 32 layers x 8 heads, one row each: 33.9 us
// and 205 MB for 16 MB of new bytes).
// Against k_kv8_store, with la_kv8_free behind: 64 sequences, 2, 4 and 8 rows
// 55 us, 85 and 150 against 84, 110 and 161; 32 sequences x 8 layers x 4 heads, 4
// and 8 rows 10.6 and 14.3 against 11.2 and 12.6; but 4 sequences x 32 layers x 8
// heads, 2 and 4 rows 14.0 and 21.5 against 11.3 and 14.0: there each SM has a CTA
// at most, and stored tokens that are rounded again occupy one warp instead of
// four.  (One row: 9.3.)
constexpr int kFewRows = 4, kFewWarps = 8, kFewCtas = 256;

template <int HD>
__global__ void __launch_bounds__(32 * kFewWarps, 4) k_kv8_store_few(la_kv8_cache c, la_kv8_rows r, const int4 *record, int touched) {
    constexpr int E = HD / 32;                                     // a lane's elements of a row
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int s = blockIdx.x / touched, j = blockIdx.x % touched, layer = blockIdx.y;
    const int4 rec = record[s];
    const int first = r.row_start ? r.row_start[s] : s;
    const int n = rec.x, len = rec.y;
    if (n <= 0) return;
    const int pj = len / c.page + j;
    const int a = j == 0 ? len % c.page : 0;
    const long long left = static_cast<long long>(len) + n - static_cast<long long>(pj) * c.page;
    if (left <= 0) return;
    const int b = static_cast<int>(min(left, static_cast<long long>(c.page)));
    const int to = j == 0 ? rec.w : kv8_page(c, s, pj), from = a > 0 ? rec.z : -1;
    if (to < 0) return;
    const int row0 = first + pj * c.page + a - len;
    const int bytes = c.page * HD;
    const long long blk0 = kv8_block(c, layer, to, 0), old0 = from >= 0 ? kv8_block(c, layer, from, 0) : 0;
    for (int hv = blockIdx.z * (blockDim.x >> 5) + (threadIdx.x >> 5); hv < 2 * c.n_kv_heads; hv += gridDim.z * (blockDim.x >> 5)) {
        const int isv = hv >= c.n_kv_heads, head = isv ? hv - c.n_kv_heads : hv;
        const long long blk = blk0 + head, old = old0 + head;
        float *scales = isv ? c.v_scale : c.k_scale;
        uint8_t *pool = static_cast<uint8_t *>(isv ? c.v : c.k), *out = pool + blk * bytes;
        const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(isv ? r.v : r.k) + layer * (isv ? r.v_layer_stride : r.k_layer_stride) +
                                 head * HD + lane * E;
        const long long stride = isv ? r.v_stride : r.k_stride;
        const float was = from >= 0 ? scales[old] : 0.f;
        // This lane's elements of row i, as bf16 pairs.
        uint32_t w[E / 2];
        auto load = [&](int i) {
            const int row = r.row_idx ? r.row_idx[row0 + i] : row0 + i;
            const bool in = static_cast<unsigned>(row) < static_cast<unsigned>(r.n_src);
            if (!in && lane == 0) atomicOr(c.status, LA_KV8_BAD);  // stored as zeros
            if constexpr (E == 4) {
                const uint2 u = in ? *reinterpret_cast<const uint2 *>(x + row * stride) : make_uint2(0, 0);
                w[0] = u.x;
                w[1] = u.y;
            } else {
                w[0] = in ? *reinterpret_cast<const uint32_t *>(x + row * stride) : 0u;
            }
        };
        float amax = 0.f;
        for (int i = 0; i < b - a; ++i) {
            load(i);
#pragma unroll
            for (int k = 0; k < E / 2; ++k) amax = kv8_finite_max(amax, w[k]);
        }
        const int e_old = from >= 0 ? kv8_scale_exponent(was) : kKv8MinExp;
        const int e = max(e_old, kv8_exponent(warp_max(amax)));
        __syncwarp();                                              // every lane has the old scale
        if (lane == 0) scales[blk] = kv8_power(e);
        if (from >= 0 && (e > e_old || from != to)) {              // stored tokens: a grown scale, or a copy
            const uint8_t *in = pool + old * bytes;
            const float f = kv8_power(e_old - e);
            // 16 bytes at a time: of K from token t0's dims, of V's dim d from
            // token t0.  A piece that ends behind the stored tokens keeps the
            // bytes there (this warp alone writes the block).
            const int pieces = (a + 15) / 16, total = isv ? HD * pieces : a * (HD / 16);
            constexpr int B = 2;
            for (int i0 = lane; i0 < total; i0 += 32 * B) {
                uint4 o[B], v[B];
                int at[B], keep[B];                                // place; bytes of the piece that belong to stored tokens
#pragma unroll
                for (int k = 0; k < B; ++k) {
                    const int i = i0 + 32 * k, d = i / pieces, t0 = (i - d * pieces) * 16;
                    at[k] = isv ? d * c.page + t0 : 16 * i;
                    keep[k] = i >= total ? 0 : isv ? min(a - t0, 16) : 16;
                    if (keep[k] > 0) v[k] = *reinterpret_cast<const uint4 *>(in + at[k]);
                    if (keep[k] > 0 && keep[k] < 16) o[k] = *reinterpret_cast<const uint4 *>(out + at[k]);
                }
#pragma unroll
                for (int k = 0; k < B; ++k) {
                    if (keep[k] == 0) continue;
                    uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                    if (e > e_old) {
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            u[y] = kv8_shrink(u[y] & 255u, f) | kv8_shrink(u[y] >> 8 & 255u, f) << 8 | kv8_shrink(u[y] >> 16 & 255u, f) << 16 |
                                   kv8_shrink(u[y] >> 24, f) << 24;
                    }
                    if (keep[k] < 16) {
                        const uint32_t q[4] = {o[k].x, o[k].y, o[k].z, o[k].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int m = keep[k] - 4 * y;
                            const uint32_t mask = m >= 4 ? 0xffffffffu : m <= 0 ? 0u : (1u << (8 * m)) - 1u;
                            u[y] = (u[y] & mask) | (q[y] & ~mask);
                        }
                    }
                    *reinterpret_cast<uint4 *>(out + at[k]) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
            __syncwarp();                                          // a kept piece may hold bytes that new tokens replace
        }
        const float f = kv8_power(-e);
        for (int i = 0; i < b - a; ++i) {
            if (b - a > 1) load(i);                                // a single row is still in registers
            uint32_t q[E];
#pragma unroll
            for (int k = 0; k < E; ++k) q[k] = kv8_byte((k & 1 ? bf16_hi(w[k >> 1]) : bf16_lo(w[k >> 1])) * f);
            if (!isv) {
                uint8_t *dst = out + (a + i) * HD + lane * E;
                if constexpr (E == 4) *reinterpret_cast<uint32_t *>(dst) = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24;
                else *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(q[0] | q[1] << 8);
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k) out[(lane * E + k) * c.page + a + i] = static_cast<uint8_t>(q[k]);
            }
        }
    }
}

cudaError_t kv8_append_launch(const la_kv8_cache &c, const la_kv8_rows &r, int *ws, cudaStream_t s) {
    cudaError_t e = launch_k(k_kv8_plan, dim3(1), dim3(kPlanThreads), 0, s, c, r.row_start, r.n_rows, r.max_rows, r.stored, ws);
    if (e != cudaSuccess) return e;
    const int touched = kv8_touched(r.max_rows, c.page);
    const int4 *record = reinterpret_cast<const int4 *>(ws);
    const unsigned blocks = static_cast<unsigned>(c.n_seqs) * touched;
    // At most this many (sequence, layer) have rows; below kFewCtas the SMs are not full.
    const bool small = static_cast<int64_t>(std::min(c.n_seqs, r.n_rows)) * c.n_layers < kFewCtas;
    if (r.max_rows == 1 || (r.max_rows <= kFewRows && !small)) {
        // Not full: a warp for each head (1 sequence x 32 layers x 32 heads 9.3 us
        // against 16.6); else the warps take several (64 sequences 33.9 against 39.2).
        const int split = small ? (2 * c.n_kv_heads + kFewWarps - 1) / kFewWarps : 1;
        const dim3 grid(blocks, c.n_layers, split), block(32 * std::min(kFewWarps, 2 * c.n_kv_heads));
        if (c.head_dim == 128) return launch_k(k_kv8_store_few<128>, grid, block, 0, s, c, r, record, touched);
        return launch_k(k_kv8_store_few<64>, grid, block, 0, s, c, r, record, touched);
    }
    const dim3 grid(blocks, c.n_kv_heads, 2 * c.n_layers);
    const size_t smem = static_cast<size_t>(c.page) * (c.head_dim + 1) * 2;   // 16 elements for every 16 rows
    if (c.head_dim == 128) return launch_k(k_kv8_store<128>, grid, dim3(kStoreThreads), smem, s, c, r, record, touched);
    return launch_k(k_kv8_store<64>, grid, dim3(kStoreThreads), smem, s, c, r, record, touched);
}

// ------------------------------------------------------------------ fork, free
// One CTA per pair.  Pairs are judged by the call's start: a dst that is some
// pair's src, or that an earlier pair names, is refused, so no CTA reads what
// another writes but refs, which only grow, atomically.
__global__ void __launch_bounds__(256) k_kv8_fork(la_kv8_cache c, const int *src, const int *dst, int n) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x, tid = threadIdx.x;
    const int a = src[i], b = dst[i];
    bool clash = false;
    for (int k = tid; k < n; k += 256) clash |= src[k] == b || (k < i && dst[k] == b) || dst[k] == a;
    clash = __syncthreads_or(clash);
    const bool ok = !clash && static_cast<unsigned>(a) < static_cast<unsigned>(c.n_seqs) &&
                    static_cast<unsigned>(b) < static_cast<unsigned>(c.n_seqs);
    const int lb = ok ? c.lens[b] : 0;
    const int len = ok ? kv8_len(c, a) : 0;
    __syncthreads();                                               // lens[b] is read before it is written below
    if (!ok || lb != 0 || len != c.lens[a]) {
        if (tid == 0) atomicOr(c.status, LA_KV8_BAD);
        return;
    }
    const int *ra = c.table + static_cast<long long>(a) * c.max_pages;
    int *rb = c.table + static_cast<long long>(b) * c.max_pages;
    for (int k = tid; k < c.max_pages; k += 256) {
        const int p = ra[k];
        const bool real = static_cast<unsigned>(p) < static_cast<unsigned>(c.n_pages);
        if (real) atomicAdd(&c.refs[p], 1);
        rb[k] = real ? p : -1;
    }
    if (tid == 0) c.lens[b] = len;
}

// One CTA per entry of slots.  The exchange gives each table entry to one CTA,
// so a slot that occurs twice loses every reference once.
__global__ void __launch_bounds__(256) k_kv8_free(la_kv8_cache c, const int *slots, const int *keep) {
    pdl_trigger();
    pdl_wait();
    const int s = slots[blockIdx.x], tid = threadIdx.x;
    if (static_cast<unsigned>(s) >= static_cast<unsigned>(c.n_seqs)) {
        if (tid == 0) atomicOr(c.status, LA_KV8_BAD);
        return;
    }
    const int k = keep ? max(keep[blockIdx.x], 0) : 0;
    int *row = c.table + static_cast<long long>(s) * c.max_pages;
    const int first = k / c.page + (k % c.page ? 1 : 0);
    for (int j = first + tid; j < c.max_pages; j += 256) {
        const int p = atomicExch(&row[j], -1);
        if (static_cast<unsigned>(p) < static_cast<unsigned>(c.n_pages)) atomicSub(&c.refs[p], 1);
    }
    if (tid == 0) atomicMin(&c.lens[s], k);
}

cudaError_t kv8_fork_launch(const la_kv8_cache &c, const int *src, const int *dst, int n, cudaStream_t s) {
    return n > 0 ? launch_k(k_kv8_fork, dim3(n), dim3(256), 0, s, c, src, dst, n) : cudaSuccess;
}
cudaError_t kv8_free_launch(const la_kv8_cache &c, const int *slots, const int *keep, int n, cudaStream_t s) {
    return n > 0 ? launch_k(k_kv8_free, dim3(n), dim3(256), 0, s, c, slots, keep) : cudaSuccess;
}

// ------------------------------------------------------------------ compact
// One CTA counts the used pages and pairs the used ones above that count with
// the free ones below it, in ascending order.
//   ws: [0] pairs, [1] used pages, then src[n_pages], dst[n_pages] and
//       count[n_pages] (references) of the pairs, ascending, and to[n_pages],
//       the new number of each used page.
__global__ void __launch_bounds__(kPlanThreads) k_kv8_pair(la_kv8_cache c, int *n_live, int *ws) {
    pdl_trigger();
    pdl_wait();
    __shared__ int warp_tot[32];
    const int tid = threadIdx.x;
    int *src = ws + 4, *dst = src + c.n_pages, *count = dst + c.n_pages, *to = count + c.n_pages;
    int live = 0;
    for (int p0 = 0; p0 < c.n_pages; p0 += kPlanThreads) {
        const int p = p0 + tid;
        int tot;
        block_scan(p < c.n_pages && c.refs[p] > 0, warp_tot, &tot);
        live += tot;
    }
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < c.n_pages; p0 += kPlanThreads) {
        const int p = p0 + tid;
        const bool in = p < c.n_pages, used = in && c.refs[p] > 0;
        const bool hole = in && !used && p < live, mover = used && p >= live;
        int tot;                                                   // a chunk's holes and movers in one scan of two halves
        const int at = block_scan((hole ? 1 : 0) | (mover ? 1 << 16 : 0), warp_tot, &tot);
        if (hole) dst[holes + (at & 0xffff)] = p;
        if (mover) {
            src[movers + (at >> 16)] = p;
            count[movers + (at >> 16)] = c.refs[p];
        }
        if (in) to[p] = p;
        holes += tot & 0xffff;
        movers += tot >> 16;
    }
    __syncthreads();
    for (int i = tid; i < movers; i += kPlanThreads) to[src[i]] = dst[i];
    if (tid == 0) {
        ws[0] = movers;
        ws[1] = live;
        if (n_live) *n_live = live;
    }
}

constexpr int kMoveThreads = 256;

// Copies the pairs' pages, layer by layer, and rewrites the table and refs.
// A (layer, page)'s K (or V) is one run of n_kv_heads * page * head_dim bytes.
// Bound by memory: half of 500 pages x 32 layers x 8 heads in 333 us (6.4 TB/s)
// with 8 loads of each thread in flight, 387 with one.
__global__ void __launch_bounds__(kMoveThreads) k_kv8_move(la_kv8_cache c, int *table_out, int *refs_out, const int *ws) {
    pdl_trigger();
    pdl_wait();
    const int movers = ws[0], live = ws[1];
    const int *src = ws + 4, *dst = src + c.n_pages, *count = dst + c.n_pages, *to = count + c.n_pages;
    const long long thread = static_cast<long long>(blockIdx.x) * kMoveThreads + threadIdx.x;
    const long long threads = static_cast<long long>(gridDim.x) * kMoveThreads;
    const long long cells = static_cast<long long>(c.n_seqs) * c.max_pages;
    for (long long i = thread; i < cells; i += threads) {
        const int p = c.table[i];
        table_out[i] = static_cast<unsigned>(p) < static_cast<unsigned>(c.n_pages) ? to[p] : -1;
    }
    // refs_out may be refs: a page moved into (0 there, or its new count
    // already) and a page moved away from are told apart by number alone.
    for (long long i = thread; i < c.n_pages; i += threads) {
        const int n = c.refs[i];
        if (i >= live) refs_out[i] = 0;
        else if (n > 0) refs_out[i] = n;
    }
    for (long long i = thread; i < movers; i += threads) refs_out[dst[i]] = count[i];
    const int run = c.n_kv_heads * c.page * c.head_dim;            // bytes, a multiple of 2048
    const long long items = 2ll * movers * c.n_layers;
    for (long long i = blockIdx.x; i < items; i += gridDim.x) {
        const int pair = static_cast<int>(i >> 1) % movers, layer = static_cast<int>((i >> 1) / movers);
        uint8_t *pool = static_cast<uint8_t *>(i & 1 ? c.v : c.k);
        float *scales = i & 1 ? c.v_scale : c.k_scale;
        const long long a = kv8_block(c, layer, src[pair], 0), b = kv8_block(c, layer, dst[pair], 0);
        const long long bytes = static_cast<long long>(c.page) * c.head_dim;
        const uint4 *x = reinterpret_cast<const uint4 *>(pool + a * bytes);
        uint4 *y = reinterpret_cast<uint4 *>(pool + b * bytes);
        constexpr int B = 8;                                           // loads in flight
        for (int k0 = threadIdx.x; k0 < run / 16; k0 += B * kMoveThreads) {
            uint4 w[B];
#pragma unroll
            for (int q = 0; q < B; ++q)
                if (k0 + q * kMoveThreads < run / 16) w[q] = x[k0 + q * kMoveThreads];
#pragma unroll
            for (int q = 0; q < B; ++q)
                if (k0 + q * kMoveThreads < run / 16) y[k0 + q * kMoveThreads] = w[q];
        }
        for (int k = threadIdx.x; k < c.n_kv_heads; k += kMoveThreads) scales[b + k] = scales[a + k];
    }
}

cudaError_t kv8_compact_launch(const la_kv8_cache &c, int *table_out, int *refs_out, int *n_live, int *ws, int nsm,
                               cudaStream_t s) {
    cudaError_t e = launch_k(k_kv8_pair, dim3(1), dim3(kPlanThreads), 0, s, c, n_live, ws);
    if (e != cudaSuccess) return e;
    return launch_k(k_kv8_move, dim3(8 * nsm), dim3(kMoveThreads), 0, s, c, table_out, refs_out, ws);
}

}  // namespace la
