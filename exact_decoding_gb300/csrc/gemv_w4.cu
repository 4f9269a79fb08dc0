// Products of a few vectors with a matrix of 4-bit weights (la_gemv_w4):
//   y[r][o] = sum over groups j of s[o][j] * sum over k in group j of (q[o][k] - 8) x[r][k]
//
// Bound by the matrix's bytes: every byte is read once and meets all vectors.
// The weights are the A operand of mma.m16n8k16 (16 outputs), the vectors its B
// operand (8 vectors).  A product is a sum over k, so any order of k will do as
// long as both have the same one: lane (g, t) reads a quarter of a group of
// outputs g and g + 8, GROUP / 8 consecutive bytes each, and the same places of
// vector g.  A 32-bit word is 8 weights; a half of 16 bits each takes one of
// nibbles i and i + 4, at the end of a bf16 number that is 128 + q, and 136 less
// is q - 8: both are exact, so the products are, and the sums are fp32.
// A group's sum is multiplied by its scale once.
//
// A block's warps share 16 * wm outputs and 8 / wm parts of k, the blocks of a
// cluster share k further; the parts are added in a fixed order, through shared
// and distributed shared memory.
#include <algorithm>
#include <cstdio>

#include "abi_guard.h"
#include "la_common.cuh"

namespace la {

constexpr int kW4Warps = 8, kW4Rows = 16;

struct W4Args {
    const __nv_bfloat16 *x;
    const uint8_t *w;
    const __nv_bfloat16 *s;
    float *y;
    long long x_stride, y_stride;
    int rows, out, groups;
    int wm;        // warps along the outputs
    int blocks;    // of a cluster, along k
};

// D (16 x 8, fp32) += A (16 x 16, bf16) * B (16 x 8, bf16).
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Nibbles i and i + 4 of w (which is shifted by 4 i) as bf16 numbers q - 8.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w) {
    const uint32_t v = (w & 0x000f000fu) | 0x43004300u;   // 128 + q
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), __floats2bfloat162_rn(136.f, 136.f));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// N words that are read once.
template <int N>
__device__ __forceinline__ void w4_load(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 4)
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    else if constexpr (N == 2)
        asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    else
        w[0] = *reinterpret_cast<const uint32_t *>(p);   // half of a 32-byte sector: the next group is the other
}

// NT: tiles of 8 vectors.
template <int GROUP, int NT>
__global__ void __launch_bounds__(32 * kW4Warps) k_gemv_w4(const __grid_constant__ W4Args p) {
    constexpr int NW = GROUP / 32;             // words of a lane, of each output's group
    constexpr int U = 8 / NW;                  // groups in flight
    constexpr int LD = 20;                     // of the sums in shared memory: lanes write different banks
    __shared__ float sh[kW4Warps][NT * 8 * LD];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int C = p.blocks, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int wm = warp % p.wm, wk = warp / p.wm, parts = kW4Warps / p.wm;
    const int o0 = static_cast<int>(blockIdx.x) / C * (16 * p.wm);
    const int r0 = blockIdx.y * kW4Rows, rows = min(p.rows - r0, kW4Rows);
    const int slice = rank * parts + wk, slices = C * parts;
    const int j0 = static_cast<int>(static_cast<long long>(p.groups) * slice / slices), j1 = static_cast<int>(static_cast<long long>(p.groups) * (slice + 1) / slices);
    pdl_trigger();
    pdl_wait();
    const int oa = min(o0 + 16 * wm + g, p.out - 1), ob = min(o0 + 16 * wm + g + 8, p.out - 1);   // past the last: not written
    const uint8_t *wa = p.w + static_cast<long long>(oa) * p.groups * (GROUP / 2) + t * (GROUP / 8);
    const uint8_t *wb = p.w + static_cast<long long>(ob) * p.groups * (GROUP / 2) + t * (GROUP / 8);
    const __nv_bfloat16 *sa = p.s + static_cast<long long>(oa) * p.groups, *sb = p.s + static_cast<long long>(ob) * p.groups;
    const __nv_bfloat16 *x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = p.x + (r0 + min(8 * n + g, rows - 1)) * p.x_stride + t * (GROUP / 4);   // past the last vector: it again
    float acc[NT][4] = {};
#pragma unroll 1
    for (int j = j0; j < j1; j += U) {
        uint32_t a[U][NW], b[U][NW];
        __nv_bfloat16 fa[U], fb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = min(j + u, j1 - 1);
            w4_load<NW>(wa + static_cast<long long>(i) * (GROUP / 2), a[u]);
            w4_load<NW>(wb + static_cast<long long>(i) * (GROUP / 2), b[u]);
            fa[u] = sa[i];
            fb[u] = sb[i];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u >= j1) break;
            float d[NT][4] = {};
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                uint32_t v[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(x[n] + (j + u) * GROUP + 8 * i);
                    v[n][0] = __byte_perm(q.x, q.z, 0x5410), v[n][1] = __byte_perm(q.x, q.z, 0x7632);
                    v[n][2] = __byte_perm(q.y, q.w, 0x5410), v[n][3] = __byte_perm(q.y, q.w, 0x7632);
                }
                const uint32_t lo[4] = {w4_pair(a[u][i]), w4_pair(b[u][i]), w4_pair(a[u][i] >> 4), w4_pair(b[u][i] >> 4)};
                const uint32_t hi[4] = {w4_pair(a[u][i] >> 8), w4_pair(b[u][i] >> 8), w4_pair(a[u][i] >> 12), w4_pair(b[u][i] >> 12)};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_bf16(d[n], lo, v[n][0], v[n][1]);
                    mma_bf16(d[n], hi, v[n][2], v[n][3]);
                }
            }
            const float ya = __bfloat162float(fa[u]), yb = __bfloat162float(fb[u]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(d[n][0], ya, acc[n][0]);
                acc[n][1] = fmaf(d[n][1], ya, acc[n][1]);
                acc[n][2] = fmaf(d[n][2], yb, acc[n][2]);
                acc[n][3] = fmaf(d[n][3], yb, acc[n][3]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sh[warp][(8 * n + 2 * t + (e & 1)) * LD + g + 8 * (e >> 1)] = acc[n][e];
    __syncthreads();
    // The parts of k of this block, then those of the cluster's blocks
    const int outs = 16 * p.wm;
    if (parts > 1) {
        for (int i = tid; i < outs * NT * 8; i += 32 * kW4Warps) {
            const int n = i / outs, o = i % outs, at = n * LD + (o & 15);
            float v = sh[o >> 4][at];
            for (int k = 1; k < parts; ++k) v += sh[k * p.wm + (o >> 4)][at];
            sh[o >> 4][at] = v;
        }
        __syncthreads();
    }
    if (C > 1) cluster_sync_all();
    const int items = outs * rows;
    for (int i = items * rank / C + tid; i < items * (rank + 1) / C; i += 32 * kW4Warps) {
        const int n = i / outs, o = i % outs;
        const float *at = &sh[o >> 4][n * LD + (o & 15)];
        float v = 0.f;
        if (C > 1) {
            for (int c = 0; c < C; ++c) v += ld_cluster_f32(mapa_shared(smem_u32(at), c));
        } else {
            v = *at;
        }
        if (o0 + o < p.out) p.y[(r0 + n) * p.y_stride + o0 + o] = v;
    }
    if (C > 1) cluster_sync_all();   // nobody leaves while its sums are read
}

namespace {

int w4_bad(const char *what, int code = LA_ERR_INVALID_ARG) {
    char msg[256];
    std::snprintf(msg, sizeof(msg), "la_gemv_w4: %s", what);
    return set_last_error(code, msg);
}

template <int GROUP>
cudaError_t w4_launch(W4Args p, int nsm, cudaStream_t s) {
    auto blocks = [&](int wm) { return (p.out + 16 * wm - 1) / (16 * wm); };
    p.wm = kW4Warps;
    while (p.wm > 1 && blocks(p.wm) * 8 < 2 * nsm) p.wm /= 2;
    p.blocks = 1;
    while (p.blocks < 8 && blocks(p.wm) * p.blocks < 2 * nsm && p.blocks * 2 * (kW4Warps / p.wm) <= p.groups) p.blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks(p.wm) * p.blocks), (p.rows + kW4Rows - 1) / kW4Rows);
    cfg.blockDim = dim3(32 * kW4Warps);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.blocks > 1 ? 2 : 1;
    return p.rows > 8 ? cudaLaunchKernelEx(&cfg, k_gemv_w4<GROUP, 2>, p) : cudaLaunchKernelEx(&cfg, k_gemv_w4<GROUP, 1>, p);
}

int w4_body(const void *x, int64_t x_stride, const void *w, const void *scales, float *y, int64_t y_stride, int32_t rows, int32_t out,
            int32_t k, int32_t group, void *stream) {
    if (group != 32 && group != 64 && group != 128) return w4_bad("group must be 32, 64 or 128", LA_ERR_UNSUPPORTED);
    if (rows < 0 || rows > 256) return w4_bad("rows out of range (0 .. 256)");
    if (out < 1 || out > (1 << 24) || k < group || k > (1 << 24)) return w4_bad("out or k out of range (out 1 .. 2^24, k group .. 2^24)");
    if (k % group) return w4_bad("k must be a multiple of group");
    if (rows == 0) return LA_OK;
    if (!x || !w || !scales || !y) return w4_bad("null argument");
    auto off = [](const void *p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (off(x, 16) || off(w, 16) || off(scales, 2) || off(y, 4)) return w4_bad("x and w must be 16-byte aligned, scales and y to their types");
    if (x_stride < k || x_stride % 8) return w4_bad("x_stride must be a multiple of 8 and at least k");
    if (y_stride < out) return w4_bad("y_stride must be at least out");
    int nsm = 0;
    const int rc = sm_count(&nsm);
    if (rc != LA_OK) return rc;
    W4Args p{static_cast<const __nv_bfloat16 *>(x), static_cast<const uint8_t *>(w), static_cast<const __nv_bfloat16 *>(scales), y, x_stride, y_stride,
             rows, out, k / group, 1, 1};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = group == 128 ? w4_launch<128>(p, nsm, s) : group == 64 ? w4_launch<64>(p, nsm, s) : w4_launch<32>(p, nsm, s);
    return e == cudaSuccess ? LA_OK : w4_bad(cudaGetErrorString(e), LA_ERR_CUDA);
}

}  // namespace
}  // namespace la

extern "C" int la_gemv_w4(const void *x, int64_t x_stride, const void *w, const void *scales, float *y, int64_t y_stride, int32_t rows,
                          int32_t out, int32_t k, int32_t group, void *stream) {
    return la::abi_guard("la_gemv_w4", [&] { return la::w4_body(x, x_stride, w, scales, y, y_stride, rows, out, k, group, stream); });
}
