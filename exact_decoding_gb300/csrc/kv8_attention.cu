// Attention of new rows over the paged 8-bit KV cache (la_kv8_attention).
//
// For a query vector q (one row, one head) and the keys j it sees,
//   z_j = scale * q . K_j,   o = sum_j e^(z_j) V_j / sum_j e^(z_j),
// computed in one pass over the keys with the running maximum of the softmax.
// With a power-of-two scale 2^kx on a page's K and 2^vx on its V (kx, vx its
// scales' exponents), the kernels keep, in base 2,
//   t_j = z_j log2(e) + vx,  m = max t_j,  w_j = 2^(t_j - m)  (fp16, <= 1),
//   O = sum_j w_j V8_j,      L = sum_j w_j 2^-vx,   o = O / L,
// so the weights that meet the 8-bit values carry V's scale and stay in
// fp16's range, whatever the pages' scales are.
//
// The work is the list of (sequence, KV head, tile of query vectors) units,
// each a run of key tiles: the cached tokens, then the sequence's new rows.
// Every worker (CTA) takes an equal share of the flattened key tiles of all
// units, read off the device-side lengths, so ragged batches and single long
// sequences fill the GPU alike.  A unit that one worker does not cover leaves
// partial (O, m, L) in the workspace, and k_kv8_join adds them in key order.
#include <algorithm>
#include <atomic>

#include "kv8.h"

namespace la {

constexpr float kKv8Log2e = 1.4426950408889634f;

struct Kv8Args {
    la_kv8_cache c;
    la_kv8_attn a;
    int gq;            // query heads per KV head
    int q_tile;        // query vectors per unit
    int k_tile;        // keys per tile
    int whole;         // 1: worker w runs units w, w + workers, ... whole, and nothing is joined
    int workers;
    float scale_log2;  // scale * log2(e)
    float *part;       // [workers][2][q_tile][head_dim] unnormalised sums
    float *part_ml;    // [workers][2][q_tile][2] running maximum and L
};

// ------------------------------------------------------------------ work list
struct Kv8Seq {
    int first, rows;         // rows of the slot
    int len;                 // cached tokens
    int qtiles;              // tiles of query vectors
    int ctiles, ntiles;      // key tiles of the cache and of the new rows
    __device__ int ktiles() const { return max(ctiles + ntiles, 1); }
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8Args &p, int s) {
    Kv8Seq q;
    q.rows = kv8_rows(p.c, p.a.row_start, p.a.n_rows, s, &q.first);
    q.len = kv8_len(p.c, s);
    q.qtiles = static_cast<int>((static_cast<long long>(q.rows) * p.gq + p.q_tile - 1) / p.q_tile);
    q.ctiles = (q.len + p.k_tile - 1) / p.k_tile;
    q.ntiles = p.a.k ? (q.rows + p.k_tile - 1) / p.k_tile : 0;
    return q;
}

// tiles[s] for s = 0 .. n_seqs; every thread of the CTA calls it.
__device__ __forceinline__ void kv8_plan(const Kv8Args &p, long long *tiles, long long *warp_sum) {
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int per = (p.c.n_seqs + nt - 1) / nt;
    const int s0 = min(tid * per, p.c.n_seqs), s1 = min(s0 + per, p.c.n_seqs);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
        const Kv8Seq q = kv8_seq(p, s);
        const long long t = static_cast<long long>(q.qtiles) * p.c.n_kv_heads * q.ktiles();
        tiles[s + 1] = t;
        mine += t;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[w] = incl;
    __syncthreads();
    long long at = incl - mine;
    for (int i = 0; i < w; ++i) at += warp_sum[i];
    for (int s = s0; s < s1; ++s) {
        at += tiles[s + 1];
        tiles[s + 1] = at;
    }
    if (tid == 0) tiles[0] = 0;
    __syncthreads();
}

// The slot that holds key tile t of the flattened list.
__device__ __forceinline__ int kv8_find(const long long *tiles, int n, long long t) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (tiles[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Workers that get tiles: each at least one, so that every piece of a split unit is written.
__device__ __forceinline__ int kv8_workers(const Kv8Args &p, long long total) {
    return static_cast<int>(min(static_cast<long long>(p.workers), total));
}
// First tile of worker w.
__device__ __forceinline__ long long kv8_share(long long total, int w, int workers) { return total * w / workers; }

// ------------------------------------------------------------------ mma
// D (16 x 8, fp32) += A (16 x 16, fp16) * B (16 x 8, fp16).
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 bytes as two pairs of fp16.
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float bf16_bits(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ int exponent_of(float scale) { return static_cast<int>((__float_as_uint(scale) >> 23) & 255u) - 127; }
__device__ __forceinline__ float power_of(int e) { return __uint_as_float(static_cast<unsigned>(min(max(e + 127, 1), 254)) << 23); }
__device__ __forceinline__ bool is_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }
// Exponent x such that |v| < 2^(x + 15) for the largest finite |v| = amax: v * 2^-x fits fp16.
__device__ __forceinline__ int fit_f16(float amax) { return max(exponent_of(amax) - 14, kKv8MinExp); }

// ------------------------------------------------------------------ few query vectors per KV head
// k_kv8_rows: 16 query vectors per unit (all heads of a KV head's group for
// one row, or some rows), 8 warps that take the unit's 64-key tiles in turn,
// each with its own running softmax; joined through shared memory at the end
// of the unit.  No tile is shared, so nothing waits on a barrier inside a
// unit.  K and V bytes go from global memory to registers in the order in
// which mma.m16n8k16 wants its B operand: the products are sums over dims
// (keys), so any order will do as long as q (the weights) has the same one.
//   K: column n of product j is key 16 (n >> 1) + 2 j + (n & 1); lane (n, t)
//      reads HD / 4 consecutive bytes of that key's row from byte t HD / 4.
//   V: lane (n, t) reads keys 16 t .. 16 t + 15 of dim 8 i + n: one 16-byte load.
// Then the weights of product j's columns 2 t, 2 t + 1 are this lane's keys
// 16 t + 2 j, + 1: already the A operand of the second product.
constexpr int kRowsWarps = 8;
constexpr int kRowsQ = 16, kRowsK = 64;

template <int HD>
struct RowsShared {
    long long tiles[LA_KV8_MAX_SEQS + 1];
    long long warp_sum[kRowsWarps];
    float m[kRowsWarps][kRowsQ], l[kRowsWarps][kRowsQ];
    alignas(16) float o[kRowsWarps][kRowsQ][HD + 4];   // read as float4
};

template <int HD>
__global__ void __launch_bounds__(32 * kRowsWarps, 1) k_kv8_rows(const __grid_constant__ Kv8Args p) {
    constexpr int NI = HD / 8;    // 8-dim groups of the output
    constexpr int KS = HD / 16;   // steps of the first product
    extern __shared__ __align__(16) uint8_t smem_raw[];
    RowsShared<HD> &sh = *reinterpret_cast<RowsShared<HD> *>(smem_raw);
    pdl_trigger();
    pdl_wait();
    const la_kv8_cache &c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    kv8_plan(p, sh.tiles, sh.warp_sum);
    const long long total = sh.tiles[c.n_seqs];
    const int workers = kv8_workers(p, total);
    if (!p.whole && static_cast<int>(blockIdx.x) >= workers) return;
    long long at = p.whole ? 0 : kv8_share(total, blockIdx.x, workers);
    const long long end = p.whole ? total : kv8_share(total, blockIdx.x + 1, workers);
    long long skip = blockIdx.x;   // whole: units to pass over
    const uint8_t *kp = static_cast<const uint8_t *>(c.k), *vp = static_cast<const uint8_t *>(c.v);
    const long long bytes = static_cast<long long>(c.page) * HD;

    while (at < end) {
        const int s = kv8_find(sh.tiles, c.n_seqs, at);
        const Kv8Seq sq = kv8_seq(p, s);
        const int kt = sq.ktiles();
        if (p.whole) {
            // units of this slot from `at` on
            const long long units = (sh.tiles[s + 1] - at) / kt;
            if (skip >= units) {
                skip -= units;
                at = sh.tiles[s + 1];
                continue;
            }
            at += skip * kt;
            skip = p.workers - 1;
        }
        const int unit = static_cast<int>((at - sh.tiles[s]) / kt), k0 = static_cast<int>((at - sh.tiles[s]) % kt);
        const int k1 = static_cast<int>(min(static_cast<long long>(kt), k0 + (end - at)));
        const int head = unit / sq.qtiles, qv0 = (unit % sq.qtiles) * kRowsQ;
        const int nqv = min(kRowsQ, sq.rows * p.gq - qv0);

        // q as fp16 A operands, each vector scaled by a power of two to fit.
        uint32_t q[KS][4];
        float qf[2];
        int myrow[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int qv = qv0 + g + 8 * h;
            const bool in = g + 8 * h < nqv;
            myrow[h] = in ? qv / p.gq : -1;
            uint4 w[KS / 2];
            float amax = 0.f;
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.a.q) + (sq.first + max(myrow[h], 0)) * p.a.q_stride +
                                       (head * p.gq + (in ? qv % p.gq : 0)) * HD + t * (HD / 4);
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) {
                w[i] = in ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float lo = bf16_bits(u[k] & 0xffffu), hi = bf16_bits(u[k] >> 16);
                    if (is_finite(lo)) amax = fmaxf(amax, fabsf(lo));
                    if (is_finite(hi)) amax = fmaxf(amax, fabsf(hi));
                }
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int qx = fit_f16(amax);
            const float f = power_of(-qx);
            qf[h] = power_of(qx) * p.scale_log2;
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {   // word k: dims 2k, 2k + 1 of 8; step 2 i + k / 2, half k & 1
                    q[2 * i + (k >> 1)][h + 2 * (k & 1)] = pack_f16(bf16_bits(u[k] & 0xffffu) * f, bf16_bits(u[k] >> 16) * f);
                }
            }
        }

        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[NI][4];
#pragma unroll
        for (int i = 0; i < NI; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

        const int k_end = min(k1, sq.ctiles + sq.ntiles);   // a unit without keys has one empty tile
        for (int kt0 = k0 + warp; kt0 < k_end; kt0 += kRowsWarps) {
            float sc[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
            float kf;      // factor on this lane's scores (columns: keys of its 16-key piece t)
            int vx;        // exponent of V's scale for those keys
            uint32_t see[2];   // bit 2 j + e: key 16 t + 2 j + e is seen by row h
            const bool cached = kt0 < sq.ctiles;
            const int key0 = (cached ? kt0 : kt0 - sq.ctiles) * kRowsK;
            long long vblk = 0;
            int vlive = 0;     // keys of this lane's piece that count
            int nx = 0;
            if (cached) {
                const int ck = key0 + 16 * (g >> 1), cv = key0 + 16 * t;   // first keys of the pieces this lane reads
                const int pk = ck < sq.len ? kv8_page(c, s, ck / c.page) : -1, kk = ck % c.page;
                const int pv = cv < sq.len ? kv8_page(c, s, cv / c.page) : -1;
                const long long kblk = kv8_block(c, p.a.layer, max(pk, 0), head);
                vblk = kv8_block(c, p.a.layer, max(pv, 0), head);
                kf = c.k_scale[vblk];
                vx = exponent_of(c.v_scale[vblk]);
                vlive = pv < 0 ? 0 : min(max(sq.len - key0 - 16 * t, 0), 16);
                see[0] = see[1] = vlive == 16 ? 0xffffu : (1u << vlive) - 1u;
                const uint8_t *row = kp + kblk * bytes + static_cast<long long>(kk + (g & 1)) * HD + t * (HD / 4);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint4 w[HD / 64];
#pragma unroll
                    for (int i = 0; i < HD / 64; ++i) w[i] = __ldcg(reinterpret_cast<const uint4 *>(row + 2 * j * HD) + i);
#pragma unroll
                    for (int i = 0; i < HD / 64; ++i) {
                        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t b0, b1;
                            e4m3x4_f16(u[k], b0, b1);
                            mma_f16(sc[j], q[4 * i + k], b0, b1);
                        }
                    }
                }
            } else {
                // New rows: bf16, scaled by a power of two for the whole tile.
                const int nkeys = min(kRowsK, sq.rows - key0);
                const __nv_bfloat16 *kn = static_cast<const __nv_bfloat16 *>(p.a.k) + (sq.first + key0) * p.a.k_stride + head * HD;
                const __nv_bfloat16 *vn = static_cast<const __nv_bfloat16 *>(p.a.v) + (sq.first + key0) * p.a.v_stride + head * HD;
                float ak = 0.f, av = 0.f;
                for (int i = lane; i < nkeys * (HD / 2); i += 32) {
                    const int r = i / (HD / 2), d = 2 * (i % (HD / 2));
                    const uint32_t a = *reinterpret_cast<const uint32_t *>(kn + r * p.a.k_stride + d);
                    const uint32_t b = *reinterpret_cast<const uint32_t *>(vn + r * p.a.v_stride + d);
                    const float x[4] = {bf16_bits(a & 0xffffu), bf16_bits(a >> 16), bf16_bits(b & 0xffffu), bf16_bits(b >> 16)};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (is_finite(x[k])) ak = fmaxf(ak, fabsf(x[k]));
                        if (is_finite(x[2 + k])) av = fmaxf(av, fabsf(x[2 + k]));
                    }
                }
                ak = warp_max(ak);
                av = warp_max(av);
                const int kx = fit_f16(ak);
                nx = fit_f16(av);
                kf = power_of(kx);
                vx = nx;
                vlive = min(max(nkeys - 16 * t, 0), 16);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int first = key0 + 16 * t;   // this lane's keys, as rows of the sequence
                    if (myrow[h] < 0 || first >= sq.rows) see[h] = 0;
                    else if (p.a.vis)
                        see[h] = first < 256 ? p.a.vis[(static_cast<long long>(sq.first) + myrow[h]) * 8 + first / 32] >> (first % 32) & 0xffffu : 0;
                    else see[h] = myrow[h] >= first + 15 ? 0xffffu : myrow[h] < first ? 0u : (2u << (myrow[h] - first)) - 1u;
                    if (vlive < 16) see[h] &= (1u << vlive) - 1u;
                }
                const float f = power_of(-kx);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = 16 * (g >> 1) + 2 * j + (g & 1);
                    const __nv_bfloat16 *row = kn + r * p.a.k_stride + t * (HD / 4);
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        const uint2 w = r < nkeys ? *reinterpret_cast<const uint2 *>(row + 4 * i) : make_uint2(0, 0);
                        mma_f16(sc[j], q[i], pack_f16(bf16_bits(w.x & 0xffffu) * f, bf16_bits(w.x >> 16) * f),
                                pack_f16(bf16_bits(w.y & 0xffffu) * f, bf16_bits(w.y >> 16) * f));
                    }
                }
            }
            // Softmax: rows g (elements 0, 1 of a product) and g + 8 (2, 3).
            uint32_t w16[8][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float f = kf * qf[h], add = static_cast<float>(vx);
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = sc[j][2 * h + e];
                        x = (see[h] >> (2 * j + e)) & 1u ? fmaf(x, f, add) : -INFINITY;
                        mx = fmaxf(mx, x);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[h], mx), base = mn == -INFINITY ? 0.f : mn;
                const float alpha = exp2f(m[h] - base);
                m[h] = mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float a = exp2f(sc[j][2 * h] - base), b = exp2f(sc[j][2 * h + 1] - base);
                    sum += a + b;
                    w16[j][h] = pack_f16(a, b);
                }
                l[h] = l[h] * alpha + sum * power_of(-vx);
                if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        o[i][2 * h] *= alpha;
                        o[i][2 * h + 1] *= alpha;
                    }
                }
            }
            // O += w V
            if (cached) {
                const uint8_t *col = vp + vblk * bytes + static_cast<long long>(g) * c.page + (key0 + 16 * t) % c.page;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    uint4 w = __ldcg(reinterpret_cast<const uint4 *>(col + static_cast<long long>(8 * i) * c.page));
                    uint32_t u[4] = {w.x, w.y, w.z, w.w};
                    if (vlive < 16) {   // bytes behind the last token may be anything
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int n = vlive - 4 * k;
                            u[k] = n >= 4 ? u[k] : n <= 0 ? 0u : u[k] & ((1u << (8 * n)) - 1u);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t b0, b1;
                        e4m3x4_f16(u[k], b0, b1);
                        const uint32_t a[4] = {w16[2 * k][0], w16[2 * k][1], w16[2 * k + 1][0], w16[2 * k + 1][1]};
                        mma_f16(o[i], a, b0, b1);
                    }
                }
            } else {
                // V of the new rows.  A NaN or infinity counts 0 in the product
                // (0 * inf would reach rows that do not see it) and is added
                // for the rows that do.
                const int nkeys = min(kRowsK, sq.rows - key0);
                const __nv_bfloat16 *vn = static_cast<const __nv_bfloat16 *>(p.a.v) + (sq.first + key0) * p.a.v_stride + head * HD;
                const float f = power_of(-nx);
                bool odd = false;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = 16 * t + 4 * k + e;
                            x[e] = r < nkeys ? __bfloat162float(vn[r * p.a.v_stride + 8 * i + g]) : 0.f;
                            odd |= !is_finite(x[e]);
                            x[e] = is_finite(x[e]) ? x[e] * f : 0.f;
                        }
                        const uint32_t a[4] = {w16[2 * k][0], w16[2 * k][1], w16[2 * k + 1][0], w16[2 * k + 1][1]};
                        mma_f16(o[i], a, pack_f16(x[0], x[1]), pack_f16(x[2], x[3]));
                    }
                }
                if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        for (int r = 0; r < nkeys; ++r) {
                            const uint32_t b0 = __shfl_sync(0xffffffffu, see[0], 4 * g + (r >> 4)), b1 = __shfl_sync(0xffffffffu, see[1], 4 * g + (r >> 4));
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float x = __bfloat162float(vn[r * p.a.v_stride + 8 * i + 2 * t + e]);
                                if (is_finite(x)) continue;
                                if ((b0 >> (r & 15)) & 1u) o[i][e] += x;
                                if ((b1 >> (r & 15)) & 1u) o[i][2 + e] += x;
                            }
                        }
                }
            }
        }

        // Join the warps: weights 2^(m_w - M), then the sum in warp order.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (t == 0) {
                sh.m[warp][g + 8 * h] = m[h];
                sh.l[warp][g + 8 * h] = l[h];
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
                *reinterpret_cast<float2 *>(&sh.o[warp][g + 8 * h][8 * i + 2 * t]) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
        }
        __syncthreads();
        const bool all = k0 == 0 && k1 == kt;
        const int slot = 2 * blockIdx.x + (k0 == 0 ? 1 : 0);
        for (int i = tid; i < nqv * (HD / 4); i += 32 * kRowsWarps) {
            const int r = i / (HD / 4), d = 4 * (i % (HD / 4));
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w) mx = fmaxf(mx, sh.m[w][r]);
            float L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w) {
                if (sh.l[w][r] == 0.f) continue;   // saw no key
                const float f = exp2f(sh.m[w][r] - mx);
                const float4 x = *reinterpret_cast<const float4 *>(&sh.o[w][r][d]);
                L += f * sh.l[w][r];
                acc.x += f * x.x;
                acc.y += f * x.y;
                acc.z += f * x.z;
                acc.w += f * x.w;
            }
            if (all) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
                const int qv = qv0 + r;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) + (sq.first + qv / p.gq) * p.a.out_stride +
                                     (head * p.gq + qv % p.gq) * HD + d;
                const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
                *reinterpret_cast<uint2 *>(out) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
            } else {
                *reinterpret_cast<float4 *>(p.part + (static_cast<long long>(slot) * kRowsQ + r) * HD + d) = acc;
                if (d == 0) *reinterpret_cast<float2 *>(p.part_ml + (static_cast<long long>(slot) * kRowsQ + r) * 2) = make_float2(mx, L);
            }
        }
        __syncthreads();
        at += k1 - k0;
    }
}

// ------------------------------------------------------------------ join
// A unit that several workers share: worker ranges are contiguous, so the
// unit's pieces are those of consecutive workers, the first in its slot 1
// (the piece begins the unit), the others in their slot 0.  One CTA per unit,
// pieces added in key order.
constexpr int kJoinThreads = 128;

template <int HD>
__global__ void __launch_bounds__(kJoinThreads) k_kv8_join(const __grid_constant__ Kv8Args p) {
    __shared__ long long tiles[LA_KV8_MAX_SEQS + 1];
    __shared__ long long warp_sum[kJoinThreads / 32];
    pdl_trigger();
    pdl_wait();
    kv8_plan(p, tiles, warp_sum);
    const long long total = tiles[p.c.n_seqs];
    // unit blockIdx.x: its slot by walking the slots' unit counts
    long long u = blockIdx.x;
    int s = 0;
    Kv8Seq sq;
    for (;; ++s) {
        if (s == p.c.n_seqs) return;
        if (tiles[s + 1] == tiles[s]) continue;
        sq = kv8_seq(p, s);
        const long long units = static_cast<long long>(sq.qtiles) * p.c.n_kv_heads;
        if (u < units) break;
        u -= units;
    }
    const int kt = sq.ktiles();
    const long long t0 = tiles[s] + u * kt, t1 = t0 + kt;
    // first and last worker: the largest w with share(w) <= tile
    const int workers = kv8_workers(p, total);
    auto owner = [&](long long tile) {
        long long w = tile * workers / total;
        while (w + 1 < workers && kv8_share(total, static_cast<int>(w) + 1, workers) <= tile) ++w;
        while (w > 0 && kv8_share(total, static_cast<int>(w), workers) > tile) --w;
        return static_cast<int>(w);
    };
    const int w0 = owner(t0), w1 = owner(t1 - 1);
    if (w0 == w1) return;
    const int head = static_cast<int>(u) / sq.qtiles, qv0 = (static_cast<int>(u) % sq.qtiles) * p.q_tile;
    const int nqv = min(p.q_tile, sq.rows * p.gq - qv0);
    for (int i = threadIdx.x; i < nqv * (HD / 4); i += kJoinThreads) {
        const int r = i / (HD / 4), d = 4 * (i % (HD / 4));
        float mx = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = w0; w <= w1; ++w) {
            const long long rec = static_cast<long long>(2 * w + (w == w0 ? 1 : 0)) * p.q_tile + r;
            const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + rec * 2);
            if (ml.y == 0.f) continue;
            const float4 x = *reinterpret_cast<const float4 *>(p.part + rec * HD + d);
            const float mn = fmaxf(mx, ml.x), a = exp2f(mx - mn), b = exp2f(ml.x - mn);
            L = L * a + ml.y * b;
            acc.x = acc.x * a + x.x * b;
            acc.y = acc.y * a + x.y * b;
            acc.z = acc.z * a + x.z * b;
            acc.w = acc.w * a + x.w * b;
            mx = mn;
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int qv = qv0 + r;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) + (sq.first + qv / p.gq) * p.a.out_stride + (head * p.gq + qv % p.gq) * HD + d;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(out) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
}

// ------------------------------------------------------------------ launch
constexpr int kRowsPerSm = 1;

int64_t kv8_workspace_bytes(const la_kv8_cache &c, int nsm) {
    const int64_t part = static_cast<int64_t>(nsm) * kRowsPerSm * 2 * kRowsQ * (c.head_dim + 2) * 4;
    const int64_t plans = (std::max<int64_t>(3ll * c.n_seqs + c.n_pages, 4ll * c.n_pages) + 16) * 4;
    return (std::max(part, plans) + 255) / 256 * 256;
}

// Kernel attributes are per device: bit d of `mask` says they are set on device d.
static bool attrs_needed(const std::atomic<unsigned long long> &mask, unsigned long long *bit) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        *bit = 0;
        return true;
    }
    *bit = 1ull << dev;
    return !(mask.load() & *bit);
}

template <int HD>
static cudaError_t rows_launch(Kv8Args &p, int nsm, void *ws, cudaStream_t s) {
    p.q_tile = kRowsQ;
    p.k_tile = kRowsK;
    const long long units = ((static_cast<long long>(p.a.n_rows) * p.gq) / kRowsQ + p.c.n_seqs) * p.c.n_kv_heads;   // at most
    const long long tiles = (p.a.max_len + kRowsK - 1) / kRowsK + (p.a.k ? (p.a.max_rows + kRowsK - 1) / kRowsK : 0);
    // A unit of at most two tiles per warp is not worth splitting: its pieces
    // would cost a second kernel.
    p.whole = tiles <= 2 * kRowsWarps;
    p.workers = p.whole ? static_cast<int>(std::min<long long>(units, 1 << 20)) : nsm * kRowsPerSm;
    p.part = static_cast<float *>(ws);
    p.part_ml = p.part + static_cast<long long>(nsm) * kRowsPerSm * 2 * kRowsQ * HD;
    static std::atomic<unsigned long long> configured{0};
    unsigned long long bit = 0;
    const size_t smem = sizeof(RowsShared<HD>);
    if (attrs_needed(configured, &bit)) {
        cudaError_t e = cudaFuncSetAttribute(k_kv8_rows<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    cudaError_t e = launch_k(k_kv8_rows<HD>, dim3(p.workers), dim3(32 * kRowsWarps), smem, s, p);
    if (e != cudaSuccess || p.whole) return e;
    return launch_k(k_kv8_join<HD>, dim3(static_cast<unsigned>(units)), dim3(kJoinThreads), 0, s, p);
}

cudaError_t kv8_attention_launch(const la_kv8_cache &c, const la_kv8_attn &a, void *ws, int nsm, cudaStream_t s) {
    if (a.n_rows < 1) return cudaSuccess;
    Kv8Args p{};
    p.c = c;
    p.a = a;
    p.gq = a.n_heads / c.n_kv_heads;
    p.scale_log2 = a.scale * kKv8Log2e;
    return c.head_dim == 128 ? rows_launch<128>(p, nsm, ws, s) : rows_launch<64>(p, nsm, ws, s);
}

}  // namespace la
