// Products of a few vectors with a matrix of 4-bit weights (la_gemv_w4):
//   y[r][o] = sum over groups j of s[o][j] * sum over k in group j of (q[o][k] - 8) x[r][k]
//
// Bound by the matrix's bytes: every byte is read once and meets up to 16
// vectors.  What the bytes cost are the instructions that unpack them, so there
// are few: a 32-bit word, 8 weights, is one shift and four times a mask with the
// bits of fp16's 1024 put in (the known way to make small whole numbers floating), so that nibbles i and i + 4 are a pair 1024 + q, or
// 1024 + 16 q where the nibble lies higher; one packed operation each makes it
// q - 8, exactly.  (Without that one, with q as a subnormal number and -8 times the
// sum of x added, products took 0.4 us less in 25 but were off by 3.6e-6 of the result's
// 2-norm, as the tensor cores add with few bits below their largest term; so by
// 9e-8.)  The vectors come as fp16, each group of a vector times
// a power of two that brings its largest value to 2^14 .. 2^15: 11 bits hold bf16's 8, and what is
// too small for them is below 2^-39 of the largest.  A group's sum, in fp32, is multiplied
// by one number, the vector's power times the scale.  That is exact where the largest value
// times the scale is 2^-127 or more, and infinite only where it is above 2^141 (the sum times
// the power alone is infinite for x near 2^127, whatever the scale).
//
// The weights are the A operand of mma.m16n8k16 (16 outputs), the vectors its B
// operand (8 vectors).  A product is a sum over k, so any order of k will do as
// long as both have the same one: lane (g, t) reads a quarter of a group of
// outputs g and g + 8, GROUP / 8 consecutive bytes each, straight into registers,
// some groups ahead (groups of 32: through a ring in shared memory), and the same
// places of vector g.
//
// A block's warps share 16 * MT * wm outputs and 8 / wm parts of k, the blocks of
// a cluster share k further; the parts are added in a fixed order, through
// shared and distributed shared memory.  Each block makes the vectors' operand for its
// part of k in shared memory, which saves a launch; for more than 8 vectors, or a k
// that does not fit, k_w4_operands makes it once for k_w4_tiles.
//
// Measured, groups of 128: 1 vector of 4096 x 4096 5.8 us (8.7 MB, latency), of 8192 x 28672
// 24.9 us (119 MB at 4.8 TB/s; loads alone take 22.8 to 24), 16 vectors 31.0 us (4.0 TB/s),
// 121 vectors, for which k_w4_tiles reads it eight times, 197 us; 5 vectors of 13824 x 5120,
// groups of 64, 13.8 us (2.8 TB/s, latency).
#include <algorithm>
#include <atomic>
#include <cstdio>

#include <cuda_fp16.h>

#include "abi_guard.h"
#include "la_common.cuh"
#include "la_kernels.h"

namespace la {

constexpr int kW4Warps = 8, kW4Rows = 16;
constexpr int kW4Block = 4;          // groups whose scales a quad's lanes load together: a pass of the loop
constexpr int kW4Smem = 100 * 1024;  // most of a block; of three on an SM:
constexpr int kW4SmemOf3 = 60 * 1024;   // more leaves the scales too little of the L1 cache (8 vectors of 28672 x 8192, groups of 64: 53 us with 66 KB, 42 so)
// Blocks of k_gemv_w4 on an SM
constexpr int w4_per_sm(int group, int mt) { return mt == 1 && group < 128 ? 3 : 2; }
// Groups of 32: a lane's part of a group is 4 bytes, and loads of 4 bytes of 8
// outputs each cost the memory system four times what 16 bytes do.  So the bytes
// come 16 at a time into a ring of passes for each warp, and the words from there:
// 16 rows of 64 bytes, 80 apart, so that a warp reads 32 different banks
// (8192 x 28672: 54.2 us with loads of 4 bytes, 42.3 so; four or five stages leave
// room for fewer blocks and take longer at smaller sizes; groups of 64 gain nothing).
constexpr int kW4RingRow = 80, kW4Stages = 3;
constexpr int w4_ring_bytes(int group) { return group == 32 ? kW4Warps * kW4Stages * 16 * kW4RingRow : 0; }

struct W4Args {
    const __nv_bfloat16 *x;
    const uint8_t *w;
    const __nv_bfloat16 *s;
    uint8_t *made;   // operands of k_w4_operands
    float *y;
    long long x_stride, y_stride;
    int rows, out, groups;
    int wm;          // warps along the outputs
    int blocks;      // of a cluster, along k
    int parts;       // of k, over all blocks of a cluster
    int longest;     // groups of the longest part
    int ring;        // the ring's place in shared memory
};

__device__ __forceinline__ float w4_power(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }   // -126 .. 127
__device__ __forceinline__ uint32_t w4_most(uint32_t a, uint32_t b) {   // larger 16-bit halves
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Eight consecutive values of a vector (bf16) as an operand: fp16 pairs (0, 4),
// (1, 5), (2, 6), (3, 7).  LANES lanes have a group together; all lanes of the
// warp call it.  Returns the exponent of the group's power of two.
template <int LANES>
__device__ __forceinline__ int w4_operand(const uint4 &x, uint4 &y) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    constexpr uint32_t kAbs = 0x7fff7fffu;
    uint32_t top = w4_most(w4_most(w[0] & kAbs, w[1] & kAbs), w4_most(w[2] & kAbs, w[3] & kAbs));
    top = max(top & 0xffffu, top >> 16);
    if (__any_sync(0xffffffffu, top >= 0x7f80u)) {   // the largest finite one
        top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = w[i] & 0x7fffu, hi = w[i] >> 16 & 0x7fffu;
            top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = min(14 + 127 - static_cast<int>(top >> 7), 126);   // the largest value, times 2^e, is in 2^14 .. 2^15
    const float f = w4_power(e);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[i] * f, v[i + 4] * f);
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    y = make_uint4(r[0], r[1], r[2], r[3]);
    return e;
}
// The weights of a word as pairs of fp16: nibbles i and i + 4, less 8.
__device__ __forceinline__ uint32_t w4_low(uint32_t x) {   // i = 0, or 2 of a word shifted by 8
    uint32_t r;
    asm("{\n\t.reg .b32 a;\n\tlop3.b32 a, %1, 0x000f000f, 0x64006400, 0xea;\n\tadd.rn.f16x2 %0, a, %2;\n\t}" : "=r"(r) : "r"(x), "r"(0xe408e408u));   // - 1032
    return r;
}
__device__ __forceinline__ uint32_t w4_high(uint32_t x) {   // i = 1, or 3
    uint32_t r;
    asm("{\n\t.reg .b32 a;\n\tlop3.b32 a, %1, 0x00f000f0, 0x64006400, 0xea;\n\tfma.rn.f16x2 %0, a, %2, %3;\n\t}" : "=r"(r) : "r"(x), "r"(0x2c002c00u), "r"(0xd480d480u));   // / 16, - 72
    return r;
}

// D (16 x 8, fp32) = A (16 x 16, fp16) * B (16 x 8, fp16) + C.
__device__ __forceinline__ void mma_f16(float (&d)[4], const float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t w4_two(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t w4_mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t w4_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Words that are read once.
template <int N>
__device__ __forceinline__ void w4_load(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 4)
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    else
        asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
}

// MT tiles of 16 outputs for a warp, up to 8 vectors.
template <int GROUP, int MT>
__global__ void __launch_bounds__(32 * kW4Warps, w4_per_sm(GROUP, MT)) k_gemv_w4(const __grid_constant__ W4Args p) {
    constexpr int NW = GROUP / 32;             // words of a lane, of each output's group
    constexpr int LANES = GROUP / 8;           // lanes that turn a group of a vector
    constexpr int AHEAD = MT == 2 ? 2 : 4;     // groups on their way
    constexpr int LD = 20;                     // of the sums in shared memory: lanes write different banks
    extern __shared__ __align__(128) uint8_t w4_smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int C = p.blocks, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int wm = warp % p.wm, wk = warp / p.wm, parts = kW4Warps / p.wm;
    const int outs = 16 * MT * p.wm, o0 = static_cast<int>(blockIdx.x) / C * outs;
    const int rows = p.rows;
    const int j0 = static_cast<int>(static_cast<unsigned>(p.groups * (rank * parts + wk)) / static_cast<unsigned>(p.parts)),
              j1 = static_cast<int>(static_cast<unsigned>(p.groups * (rank * parts + wk + 1)) / static_cast<unsigned>(p.parts));
    pdl_trigger();
    pdl_wait();

    const uint8_t *w[MT][2];
    const __nv_bfloat16 *fs[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long o = min(o0 + 16 * (MT * wm + m) + g + 8 * h, p.out - 1);   // past the last: not written
            w[m][h] = p.w + (o * p.groups + j0) * (GROUP / 2) + (GROUP == 32 ? 0 : t * (GROUP / 8));
            fs[m][h] = p.s + o * p.groups + j0 + t;
        }
    constexpr bool RING = GROUP == 32;
    constexpr int ROW = kW4RingRow, STAGES = kW4Stages, RUN = kW4Block * GROUP / 2;   // bytes of an output's pass
    static_assert(!RING || MT == 1, "the ring's rows");
    uint32_t a[RING ? 1 : AHEAD][MT][2][NW];
    int left = j1 - j0;        // groups from w on
    auto load = [&](int u, int slot) {   // group u of the pass at w
        if (u < left) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) w4_load(w[m][h] + u * (GROUP / 2), a[slot][m][h]);
        }
    };
    const uint32_t ring = smem_u32(w4_smem) + p.ring + warp * STAGES * 16 * ROW + g * ROW;
    const int run_bytes = (j1 - j0) * (GROUP / 2);
    int to_load = 16 * t, load_slot = 0;   // byte of an output's run, slot of the next pass to load
    auto load_pass = [&]() {
        if constexpr (RING) {
            static_assert(RUN == 64, "16 bytes for each lane of a quad");
            if (to_load < run_bytes) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + load_slot * (16 * ROW) + h * (8 * ROW) + 16 * t), "l"(w[0][h] + to_load) : "memory");
            }
            to_load += RUN;
            load_slot = load_slot + 1 == STAGES ? 0 : load_slot + 1;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Lane t: the scales of groups t, t + 4, ... of the next NF passes, on their way while 512 k or more are multiplied
    // (groups of 32, 8192 x 28672: 53.8 us with NF = 1)
    constexpr int NF = GROUP == 32 ? 4 : 1;
    __nv_bfloat16 fn[MT][2][NF];
    auto load_scales = [&]() {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < NF; ++q)
                    if (t + kW4Block * q < left) fn[m][h][q] = fs[m][h][kW4Block * q];
    };
    if constexpr (RING) {
#pragma unroll 1
        for (int i = 0; i < STAGES - 1; ++i) load_pass();
    } else {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) load(u, u);
    }
    load_scales();

    // This part's warps turn its vectors, 32 words at a time
    uint4 *to = reinterpret_cast<uint4 *>(w4_smem) + wk * p.longest * NW * rows * 4;
    float *tf = reinterpret_cast<float *>(w4_smem + parts * p.longest * GROUP * rows * 2) + wk * p.longest * 8;
    const int per = (j1 - j0) * LANES, words = rows * per;   // 8 values each: of a vector, of all in a row
    constexpr int B = 4;                                     // in flight
#pragma unroll 1
    for (int f0 = wm * 32; f0 < words; f0 += B * 32 * p.wm) {
        uint4 x[B];
        int n[B], i[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int f = f0 + b * 32 * p.wm + lane;
            n[b] = rows == 1 ? 0 : static_cast<int>(static_cast<unsigned>(f) / static_cast<unsigned>(per));
            i[b] = f - n[b] * per;
            x[b] = f < words ? *reinterpret_cast<const uint4 *>(p.x + n[b] * p.x_stride + static_cast<long long>(j0) * GROUP + 8 * i[b]) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int f = f0 + b * 32 * p.wm + lane;
            if (f - lane >= words) break;
            uint4 y;
            const int e = w4_operand<LANES>(x[b], y), j = i[b] / LANES, li = i[b] % LANES;
            if (f < words) {
                to[((j * NW + li % NW) * rows + n[b]) * 4 + li / NW] = y;
                if (li == 0) tf[j * 8 + n[b]] = w4_power(-e);
            }
        }
    }
    __syncthreads();
    const uint4 *bx = to + t;
    const float2 *bf = reinterpret_cast<const float2 *>(tf) + t;
    const int at = min(g, rows - 1) * 4;   // past the last vector: it again
    uint64_t acc[MT][2] = {};   // pairs of sums
    const int n_groups = j1 - j0;
    int slot = 0;
#pragma unroll 1
    for (int j = 0; j < n_groups; j += NF * kW4Block) {
        float f[MT][2][NF];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int q = 0; q < NF; ++q) f[m][h][q] = __bfloat162float(fn[m][h][q]);
                fs[m][h] += NF * kW4Block;
            }
        const int now_all = left;
        left -= NF * kW4Block;
        load_scales();
        left = now_all;
#pragma unroll
        for (int pass = 0; pass < NF; ++pass) {
            const int now = left;
            if (pass && now <= 0) break;
            const uint8_t *from = w4_smem + p.ring + (warp * STAGES + slot) * (16 * ROW) + g * ROW + t * (GROUP / 8);
            if constexpr (RING) {
                asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
                __syncwarp();   // the pass is there, and all lanes are through with the one before
                load_pass();
                slot = slot + 1 == STAGES ? 0 : slot + 1;
            }
#pragma unroll
            for (int u = 0; u < kW4Block; ++u) {
                if (u >= now) break;
                float d[MT][4];
                if constexpr (RING) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) a[0][0][h][0] = *reinterpret_cast<const uint32_t *>(from + h * (8 * ROW) + u * (GROUP / 2));
                }
                const float2 xf = bf[u * 4];
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    const uint4 v = bx[(u * NW + i) * rows * 4 + at];
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint32_t x = a[RING ? 0 : u % AHEAD][m][0][i], y = a[RING ? 0 : u % AHEAD][m][1][i], x8 = x >> 8, y8 = y >> 8;
                        const uint32_t xl = w4_low(x), yl = w4_low(y), xh = w4_high(x), yh = w4_high(y), xl8 = w4_low(x8), yl8 = w4_low(y8), xh8 = w4_high(x8), yh8 = w4_high(y8);
                        float (&to)[4] = d[m];
                        if (i == 0) mma_f16(to, {0.f, 0.f, 0.f, 0.f}, xl, yl, xh, yh, v.x, v.y);
                        else mma_f16(to, to, xl, yl, xh, yh, v.x, v.y);
                        mma_f16(to, to, xl8, yl8, xh8, yh8, v.z, v.w);
                    }
                }
                if constexpr (!RING) load(u + AHEAD, u % AHEAD);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const float fa = __shfl_sync(0xffffffffu, f[m][0][pass], u, 4), fb = __shfl_sync(0xffffffffu, f[m][1][pass], u, 4);
                    const uint64_t xf2 = w4_two(xf.x, xf.y);
                    acc[m][0] = w4_fma2(w4_two(d[m][0], d[m][1]), w4_mul2(xf2, w4_two(fa, fa)), acc[m][0]);
                    acc[m][1] = w4_fma2(w4_two(d[m][2], d[m][3]), w4_mul2(xf2, w4_two(fb, fb)), acc[m][1]);
                }
            }
            left -= kW4Block;
            bx += kW4Block * NW * rows * 4;
            bf += kW4Block * 4;
            if constexpr (!RING) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) w[m][h] += kW4Block * (GROUP / 2);
            }
        }
    }
    // The parts of k of this block, then those of the cluster's blocks
    __syncthreads();
    float *sh = reinterpret_cast<float *>(w4_smem);   // [warp][m][vector][LD]
    auto place = [&](int wp, int o, int n) { return ((wp * MT + o / 16) * 8 + n) * LD + o % 16; };
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sh[place(warp, 16 * m + g + 8 * h, 2 * t)] = __uint_as_float(static_cast<uint32_t>(acc[m][h]));
            sh[place(warp, 16 * m + g + 8 * h, 2 * t + 1)] = __uint_as_float(static_cast<uint32_t>(acc[m][h] >> 32));
        }
    __syncthreads();
    constexpr int OW = 16 * MT;   // outputs of a warp
    const int items = outs * rows, log = 31 - __clz(outs);
    if (parts > 1) {
        for (int i = tid; i < items; i += 32 * kW4Warps) {
            const int n = i >> log, o = i & (outs - 1), to = place(o / OW, o % OW, n);
            float v = sh[to];
            for (int k = 1; k < parts; ++k) v += sh[place(k * p.wm + o / OW, o % OW, n)];
            sh[to] = v;
        }
        __syncthreads();
    }
    if (C > 1) cluster_sync_all();
    for (int i = items * rank / C + tid; i < items * (rank + 1) / C; i += 32 * kW4Warps) {
        const int n = i >> log, o = i & (outs - 1);
        const float *from = &sh[place(o / OW, o % OW, n)];
        float v = 0.f;
        if (C > 1) {
            for (int c = 0; c < C; ++c) v += ld_cluster_f32(mapa_shared(smem_u32(from), c));
        } else {
            v = *from;
        }
        if (o0 + o < p.out) p.y[n * p.y_stride + o0 + o] = v;
    }
    if (C > 1) cluster_sync_all();   // nobody leaves while its sums are read
}

// ------------------------------------------------------------------ many bytes
// k_w4_operands makes the vectors' operands once, in the form that k_w4_tiles
// wants them in shared memory: for each chunk of 128 k 16 rows of fp16 (K-major,
// 128-byte swizzle, two blocks of 64 k) and, per group, the powers of the 16 vectors.
constexpr int kChunkB = 16 * 128 * 2;             // operand
constexpr int kChunkF = 4 * 64;                   // [group][16] powers, for up to 4 groups
constexpr int kChunk = kChunkB + kChunkF;

static __device__ unsigned g_w4_err;              // a bounded wait gave up
// Bounded wait; the loop exists once (code that polls in line costs the roles' code its cache).
__device__ __noinline__ bool w4_wait_on(uint32_t bar, uint32_t parity, unsigned bit) { return mbar_wait(bar, parity, &g_w4_err, bit); }
__device__ __forceinline__ bool w4_wait(uint32_t bar, uint32_t parity, unsigned bit) { return mbar_try_wait(bar, parity) || w4_wait_on(bar, parity, bit); }

template <int GROUP>
__global__ void __launch_bounds__(128) k_w4_operands(const __grid_constant__ W4Args p) {
    constexpr int LANES = GROUP / 8, PER = 128 / GROUP;
    pdl_wait();
    pdl_trigger();   // only now: k_w4_tiles, which starts with it, may read what was written before this call
    const int r0 = blockIdx.z * kW4Rows, n = blockIdx.y;
    const int word = blockIdx.x * 128 + threadIdx.x, chunk = word >> 4;   // 8 k each
    uint4 x = make_uint4(0, 0, 0, 0), y;
    if (r0 + n < p.rows && word * 8 < p.groups * GROUP) x = *reinterpret_cast<const uint4 *>(p.x + (r0 + n) * p.x_stride + static_cast<long long>(word) * 8);
    const int e = w4_operand<LANES>(x, y);   // behind the last group: zeros, as the products want them
    const int chunks = (p.groups + PER - 1) / PER;
    if (chunk >= chunks) return;
    uint8_t *to = p.made + (static_cast<long long>(blockIdx.z) * chunks + chunk) * kChunk;
    const int w = word & 15;
    *reinterpret_cast<uint4 *>(to + (w >> 3) * 2048 + n * 128 + (((w & 7) ^ (n & 7)) << 4)) = y;
    if (w % LANES == 0) reinterpret_cast<float *>(to + kChunkB)[w / LANES * 16 + n] = w4_power(-e);
}

// k_w4_tiles: 128 outputs x 16 vectors on the tcgen05 tensor cores.  Per chunk of 128 k
//   warp 8        brings the weights' bytes (one TMA box of 128 rows x 64 bytes, 64-byte
//                 swizzle) and the chunk's operand (one bulk copy) into a ring
//   warps 0..3    take the even chunks, warps 4..7 the odd ones; each thread an
//                 output: 16 words of its row become 64 columns of fp16 in tensor memory
//   warp 9        issues the products, each group's into 16 columns of its own
//   then the same threads add a group's 16 sums to their own, in registers, with
//   the group's scale and the vectors' powers.
// mma.sync would need a fifth of the instructions more, and its operand's loads
// fill the shared memory's bandwidth at 16 vectors.
// A block's 55 thousand cycles for 16 vectors of 8192 x 28672, groups of 128 (two blocks on an SM): 4
// until the first bytes, 44 in the loop, and 7 until the cluster's last block is through and its sums are
// joined.  A group of warps has 28 chunks, each 1550 cycles: unpacking 460, the product 620 and the sums 235, one
// behind another, the next bytes 135, 100 between them.  256 blocks have 148 SMs, 40 of them one alone.
constexpr int kTileStages = 7, kTileStage = 13 * 1024;   // weights 8 KB, chunk
constexpr int kTileThreads = 320;
constexpr int kTileBars = kTileStages * kTileStage, kTileSmem = kTileBars + 256;

__device__ __forceinline__ void w4_bulk(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void w4_arrive(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); }
__device__ __forceinline__ bool w4_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// D[tmem] (+)= A[tmem] * B[smem]^T, fp16 operands.
__device__ __forceinline__ void w4_umma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
                 "r"(accumulate)
                 : "memory");
}
// NT: tiles of 8 vectors in use.
template <int GROUP, int NT>
__global__ void __launch_bounds__(kTileThreads, 2) k_w4_tiles(const __grid_constant__ W4Args p, const __grid_constant__ CUtensorMap map) {
    constexpr int PER = 128 / GROUP;
    constexpr uint32_t kIdesc = (1u << 4) | (16u >> 3) << 17 | (128u >> 4) << 24;   // fp16 operands, fp32 sums, 128 x 16
    extern __shared__ __align__(1024) uint8_t w4_ring[];
    const uint32_t sm = smem_u32(w4_ring), bars = sm + kTileBars;
    auto full = [&](int s) { return bars + 8 * s; };                     // the ring's copies
    auto empty = [&](int s) { return bars + 8 * (kTileStages + s); };    // products done, and 4 warps through with the powers
    auto a_full = [&](int g) { return bars + 8 * (2 * kTileStages + g); };
    auto d_full = [&](int g) { return bars + 8 * (2 * kTileStages + 2 + g); };
    const uint32_t drain = bars + 8 * (2 * kTileStages + 4);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(w4_ring + kTileBars + 8 * (2 * kTileStages + 5));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = p.blocks, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int o0 = static_cast<int>(blockIdx.x) / C * 128, r0 = blockIdx.y * kW4Rows, rows = min(p.rows - r0, kW4Rows);
    const int chunks = (p.groups + PER - 1) / PER, c0 = static_cast<int>(static_cast<long long>(chunks) * rank / C),
              n_chunks = static_cast<int>(static_cast<long long>(chunks) * (rank + 1) / C) - c0;
    if (tid == 0) {
        for (int s = 0; s < kTileStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 5);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(a_full(g), 4);
            mbar_init(d_full(g), 1);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_trigger();
    bool ok = true;
    float acc[8 * NT] = {};

    if (warp == 8) {
        // ================================================ bytes
        const uint64_t once = policy_evict_first();
        const uint8_t *ops = p.made + (static_cast<long long>(blockIdx.y) * chunks + c0) * kChunk;
        const bool one = w4_elect();
        auto weights = [&](int i, int s) {
            mbar_arrive_expect_tx(full(s), 8192 + kChunk);
            tma_load_2d(sm + s * kTileStage, &map, (c0 + i) * 64, o0, full(s), once);
        };
        // The weights' first stages before the operands are waited for: k_w4_operands
        // lets this kernel start only once all work before it is done.
        if (one)
            for (int i = 0; i < min(n_chunks, kTileStages); ++i) weights(i, i);
        __syncwarp();
        pdl_wait();
        int issued = 0;
        for (; issued < n_chunks; ++issued) {
            const int i = issued, s = i % kTileStages;
            if (i >= kTileStages) {
                ok = __all_sync(0xffffffffu, w4_wait(empty(s), (i / kTileStages - 1) & 1, ERR_TIMEOUT_EMPTY));
                if (!ok) break;
                if (one) weights(i, s);
            }
            if (one) w4_bulk(sm + s * kTileStage + 8192, ops + static_cast<long long>(i) * kChunk, kChunk, full(s));
            __syncwarp();
        }
        // Every copy has landed: where a wait gave up, nobody else has seen that.
        for (int i = max(issued - kTileStages, 0); i < issued; ++i) w4_wait(full(i % kTileStages), i / kTileStages & 1, ERR_TIMEOUT_FULL);
        __syncwarp();
    } else if (warp == 9) {
        // ================================================ products
        for (int i = 0; ok && i < n_chunks; ++i) {
            const int s = i % kTileStages, g = i & 1;
            ok = __all_sync(0xffffffffu, w4_wait(full(s), i / kTileStages & 1, ERR_TIMEOUT_FULL) && w4_wait(a_full(g), i >> 1 & 1, ERR_TIMEOUT_FULL));
            if (!ok) break;
            tc_fence_after();
            if (w4_elect()) {
                const uint32_t a = tmem + 128 * g, d = a + 64;
                const uint64_t b = umma_desc_sw128(sm + s * kTileStage + 8192);
#pragma unroll
                for (int k = 0; k < 8; ++k) w4_umma(d + 16 * (k * PER / 8), a + 8 * k, b + 2 * (k & 3) + 128 * (k >> 2), kIdesc, k * PER % 8 != 0);
                umma_commit(d_full(g));
                umma_commit(empty(s));
            }
            __syncwarp();
        }
        if (!ok) {   // void: wait (bounded) for the products in flight
            if (w4_elect()) umma_commit(drain);
            __syncwarp();
            w4_wait(drain, 0, ERR_TIMEOUT_ACCUM);
        }
        __syncwarp();
    } else {
        // ================================================ operands and sums
        const int g = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t a = tmem + 128 * g + (static_cast<uint32_t>(32 * (warp & 3)) << 16), d = a + 64;
        const __nv_bfloat16 *scale = p.s + static_cast<long long>(min(o0 + row, p.out - 1)) * p.groups;
        const int last = p.groups - 1;
        uint64_t sums[4 * NT];
#pragma unroll
        for (int n = 0; n < 4 * NT; ++n) sums[n] = 0;
        __nv_bfloat16 f[PER];
        auto load_scales = [&](int i) {
#pragma unroll
            for (int u = 0; u < PER; ++u) f[u] = scale[min((c0 + i) * PER + u, last)];
        };
        load_scales(min(g, max(n_chunks - 1, 0)));
        for (int i = g; i < n_chunks; i += 2) {
            const int s = i % kTileStages;
            ok = __all_sync(0xffffffffu, w4_wait(full(s), i / kTileStages & 1, ERR_TIMEOUT_FULL));
            if (!ok) break;
            const uint32_t from = sm + s * kTileStage + row * 64;
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // 8 words, 64 k
                uint32_t w[8], v[32];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[4 * q]), "=r"(w[4 * q + 1]), "=r"(w[4 * q + 2]), "=r"(w[4 * q + 3])
                                 : "r"(from + (((2 * h + q) ^ (row >> 1 & 3)) << 4))
                                 : "memory");
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t x = w[q], x8 = x >> 8;
                    v[4 * q] = w4_low(x);
                    v[4 * q + 1] = w4_high(x);
                    v[4 * q + 2] = w4_low(x8);
                    v[4 * q + 3] = w4_high(x8);
                }
                tmem_st_32x32b_x32(a + 32 * h, v);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) w4_arrive(a_full(g));
            float fs[PER];
#pragma unroll
            for (int u = 0; u < PER; ++u) fs[u] = __bfloat162float(f[u]);
            load_scales(min(i + 2, n_chunks - 1));
            ok = __all_sync(0xffffffffu, w4_wait(d_full(g), i >> 1 & 1, ERR_TIMEOUT_ACCUM));
            if (!ok) break;
            tc_fence_after();
            const uint8_t *table = w4_ring + s * kTileStage + 8192 + kChunkB;
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                if (PER > 1 && (c0 + i) * PER + u > last) break;   // the matrix ends inside the chunk
                uint32_t v[16];
                tmem_ld_32x32b_x16(d + 16 * u, v);
                const uint64_t f2 = w4_two(fs[u], fs[u]);
                uint64_t both[4 * NT];   // powers times scale, while the sums are on their way
#pragma unroll
                for (int n = 0; n < 2 * NT; ++n) {
                    const ulonglong2 e = reinterpret_cast<const ulonglong2 *>(table + u * 64)[n];
                    both[2 * n] = w4_mul2(e.x, f2);
                    both[2 * n + 1] = w4_mul2(e.y, f2);
                }
                tmem_ld_wait();
#pragma unroll
                for (int n = 0; n < 16; ++n) asm volatile("" : "+r"(v[n]));
#pragma unroll
                for (int n = 0; n < 4 * NT; ++n) sums[n] = w4_fma2(w4_two(__uint_as_float(v[2 * n]), __uint_as_float(v[2 * n + 1])), both[n], sums[n]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) w4_arrive(empty(s));
        }
#pragma unroll
        for (int n = 0; n < 4 * NT; ++n) asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[2 * n]), "=f"(acc[2 * n + 1]) : "l"(sums[n]));
    }
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
    // The two halves, then the cluster's blocks, in order
    float *sh = reinterpret_cast<float *>(w4_ring);   // [16 vectors][132]
    constexpr int LD = 132;
    if (warp >= 4 && warp < 8)
#pragma unroll
        for (int n = 0; n < 8 * NT; ++n) sh[n * LD + tid - 128] = acc[n];
    __syncthreads();
    if (warp < 4)
#pragma unroll
        for (int n = 0; n < 8 * NT; ++n) sh[n * LD + tid] = acc[n] + sh[n * LD + tid];
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    const int items = 128 * rows;
    for (int i = items * rank / C + tid; i < items * (rank + 1) / C; i += kTileThreads) {
        const int n = i >> 7, o = i & 127;
        const float *from = &sh[n * LD + o];
        float v = 0.f;
        if (C > 1) {
            for (int c = 0; c < C; ++c) v += ld_cluster_f32(mapa_shared(smem_u32(from), c));
        } else {
            v = *from;
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

// Sets a kernel's shared memory once per device: bit d of `done`.
template <typename K>
cudaError_t w4_allow(K kernel, int bytes, std::atomic<unsigned long long> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
}
template <typename K, typename... Args>
cudaError_t w4_clusters(K kernel, dim3 grid, int threads, int smem, int blocks, cudaStream_t s, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// How a product runs.
struct W4Plan {
    bool large;      // k_w4_operands and k_w4_tiles, which need a workspace
    int mt, wm, blocks;
    int64_t bytes;   // of workspace
};

// k_gemv_w4 up to 8 vectors, k_w4_tiles above.  Device us of 8 vectors, k_gemv_w4 against
// k_w4_tiles, groups of 128: 512 x 512 3.7 and 4.9, 4096 x 4096 6.7 and 8.2, 13824 x 5120 12.5 and 15.2,
// 32000 x 4096 19.4 and 19.2, 8192 x 28672 30.1 and 29.6; groups of 32: 4096 x 4096 9.3 and 9.8, 5120 x 13824
// 20.9 and 24.9, 8192 x 28672 53.7 both.
constexpr int kFewVectors = 8;

W4Plan w4_plan(int rows, int out, int k, int group, int nsm) {
    W4Plan best{};
    const int groups = k / group, chunks = (k + 127) / 128, tiles = (out + 127) / 128, many = (rows + kW4Rows - 1) / kW4Rows;
    // k_gemv_w4: the split of outputs and k that fills most of the SMs in one round
    // (11008 x 4096: 172 blocks 9.2 us, 258 in clusters of 6 8.9 us, 301 in clusters of 7, which
    // take two rounds, 13.7 us), with the most outputs for a block where two do nearly
    // alike (each block turns its vectors; 1 vector, groups of 64: 258 blocks of 256 outputs
    // 10.5 us, 430 of 128 12.2 us); with fewer than 128 only where k is in as many parts
    // as there may be and SMs are idle.
    // Clusters of n blocks leave SMs over where an SM's neighbours do not make a whole
    // one: the blocks that the occupancy query allows at a time, of those of single ones, at least.
    static constexpr double kClusterRoom[8] = {1., 1., .95, .96, .95, .9, .87, .89};
    double most = 0.;
    bool idle = true;
    if (rows <= kFewVectors) {
        const struct {
            int mt, wm;
        } forms[] = {{2, 8}, {1, 8}, {1, 4}, {1, 2}, {1, 1}};
        for (const auto &f : forms) {
            if (f.wm < kW4Warps && !idle) break;
            if (f.mt == 2 && group == 32) continue;   // its ring has the rows of one tile
            const int outs = 16 * f.mt * f.wm, count = (out + outs - 1) / outs, parts = kW4Warps / f.wm, slots = w4_per_sm(group, f.mt) * nsm;
            int blocks = 1;
            while (blocks < 8 && static_cast<int64_t>(count) * (blocks + 1) <= static_cast<int64_t>(slots * kClusterRoom[blocks]) && (blocks + 1) * parts <= groups) ++blocks;
            const int64_t smem = static_cast<int64_t>(parts) * ((groups + blocks * parts - 1) / (blocks * parts)) * (group * rows * 2 + 32);
            const int64_t rounds = (static_cast<int64_t>(count) * blocks + slots - 1) / slots;
            const double fill = static_cast<double>(count) * blocks / (static_cast<double>(rounds) * slots);
            if (smem + w4_ring_bytes(group) > (w4_per_sm(group, f.mt) == 3 ? kW4SmemOf3 : kW4Smem) || parts > groups || fill <= most * 1.12) continue;
            idle = static_cast<int64_t>(count) * blocks * 2 <= slots;
            most = fill;
            best.mt = f.mt, best.wm = f.wm, best.blocks = blocks;
        }
        if (most > 0.) return best;
    }
    best.large = true;
    best.blocks = 1;
    while (best.blocks < 8 && static_cast<int64_t>(tiles) * many * (best.blocks + 1) <= 2 * nsm && best.blocks < chunks) ++best.blocks;
    best.bytes = static_cast<int64_t>(many) * chunks * kChunk;
    return best;
}

template <int GROUP, int NT>
cudaError_t w4_tiles_launch(W4Args p, const W4Plan &plan, const CUtensorMap &map, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    const int chunks = (p.groups * GROUP + 127) / 128, many = (p.rows + kW4Rows - 1) / kW4Rows;
    cudaError_t e = w4_allow(k_w4_tiles<GROUP, NT>, kTileSmem, done);
    if (e == cudaSuccess) e = launch_k(k_w4_operands<GROUP>, dim3((chunks + 7) / 8, std::min(p.rows, kW4Rows), many), dim3(128), 0, s, p);
    if (e != cudaSuccess) return e;
    p.blocks = plan.blocks;
    return w4_clusters(k_w4_tiles<GROUP, NT>, dim3((p.out + 127) / 128 * plan.blocks, many), kTileThreads, kTileSmem, plan.blocks, s, p, map);
}
template <int GROUP, int MT>
cudaError_t w4_few_launch(W4Args p, const W4Plan &plan, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = w4_allow(k_gemv_w4<GROUP, MT>, kW4Smem, done);
    if (e != cudaSuccess) return e;
    p.wm = plan.wm;
    p.blocks = plan.blocks;
    const int parts = kW4Warps / p.wm, outs = 16 * MT * p.wm;
    p.longest = (p.groups + p.blocks * parts - 1) / (p.blocks * parts);
    p.parts = p.blocks * parts;
    p.ring = std::max(parts * p.longest * (GROUP * p.rows * 2 + 32), kW4Warps * MT * 8 * 20 * 4);
    const int smem = p.ring + w4_ring_bytes(GROUP);
    return w4_clusters(k_gemv_w4<GROUP, MT>, dim3((p.out + outs - 1) / outs * p.blocks), 32 * kW4Warps, smem, p.blocks, s, p);
}
template <int GROUP>
cudaError_t w4_launch(const W4Args &p, const W4Plan &plan, const CUtensorMap &map, cudaStream_t s) {
    if (plan.large) return p.rows > 8 ? w4_tiles_launch<GROUP, 2>(p, plan, map, s) : w4_tiles_launch<GROUP, 1>(p, plan, map, s);
    if constexpr (GROUP != 32)
        if (plan.mt == 2) return w4_few_launch<GROUP, 2>(p, plan, s);
    return w4_few_launch<GROUP, 1>(p, plan, s);
}

int w4_sizes(int32_t rows, int32_t out, int32_t k, int32_t group) {
    if (group != 32 && group != 64 && group != 128) return w4_bad("group must be 32, 64 or 128", LA_ERR_UNSUPPORTED);
    if (rows < 0 || rows > 256) return w4_bad("rows out of range (0 .. 256)");
    if (out < 1 || out > (1 << 24) || k < group || k > (1 << 24)) return w4_bad("out or k out of range (out 1 .. 2^24, k group .. 2^24)");
    if (k % group) return w4_bad("k must be a multiple of group");
    return LA_OK;
}

int w4_workspace_body(int32_t rows, int32_t out, int32_t k, int32_t group, int64_t *bytes) {
    int rc = w4_sizes(rows, out, k, group), nsm = 0;
    if (rc != LA_OK) return rc;
    if (!bytes) return w4_bad("null argument");
    if ((rc = sm_count(&nsm)) != LA_OK) return rc;
    *bytes = rows ? w4_plan(rows, out, k, group, nsm).bytes : 0;
    return LA_OK;
}

int w4_body(const void *x, int64_t x_stride, const void *w, const void *scales, float *y, int64_t y_stride, int32_t rows, int32_t out,
            int32_t k, int32_t group, void *workspace, int64_t workspace_bytes, void *stream) {
    int rc = w4_sizes(rows, out, k, group), nsm = 0;
    if (rc != LA_OK || rows == 0) return rc;
    if (!x || !w || !scales || !y) return w4_bad("null argument");
    auto off = [](const void *p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (off(x, 16) || off(w, 16) || off(scales, 2) || off(y, 4)) return w4_bad("x and w must be 16-byte aligned, scales and y to their types");
    if (x_stride < k || x_stride % 8) return w4_bad("x_stride must be a multiple of 8 and at least k");
    if (y_stride < out) return w4_bad("y_stride must be at least out");
    if ((rc = sm_count(&nsm)) != LA_OK) return rc;
    const W4Plan plan = w4_plan(rows, out, k, group, nsm);
    if (plan.bytes > 0 && (!workspace || off(workspace, 16))) return w4_bad("workspace must be 16-byte aligned device memory");
    if (workspace_bytes < plan.bytes) return w4_bad("workspace too small (see la_gemv_w4_workspace)", LA_ERR_CAPACITY);
    CUtensorMap map{};
    if (plan.large && make_tmap_rows64(&map, w, static_cast<uint64_t>(k) / 2, out)) return w4_bad("tensor map of the weights failed", LA_ERR_CUDA);
    W4Args p{};
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.w = static_cast<const uint8_t *>(w);
    p.s = static_cast<const __nv_bfloat16 *>(scales);
    p.made = static_cast<uint8_t *>(workspace);
    p.y = y;
    p.x_stride = x_stride;
    p.y_stride = y_stride;
    p.rows = rows;
    p.out = out;
    p.groups = k / group;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = group == 128 ? w4_launch<128>(p, plan, map, s) : group == 64 ? w4_launch<64>(p, plan, map, s) : w4_launch<32>(p, plan, map, s);
    return e == cudaSuccess ? LA_OK : w4_bad(cudaGetErrorString(e), LA_ERR_CUDA);
}

}  // namespace

// The current device's word of waits that gave up: read to *bits and cleared, on s.
cudaError_t w4_err_take(cudaStream_t s, unsigned *bits) {
    void *word = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&word, g_w4_err);
    if (e == cudaSuccess) e = cudaMemcpyAsync(bits, word, sizeof(unsigned), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(word, 0, sizeof(unsigned), s);
    return e;
}

}  // namespace la

extern "C" {

int la_gemv_w4_workspace(int32_t rows, int32_t out, int32_t k, int32_t group, int64_t *bytes) {
    return la::abi_guard("la_gemv_w4_workspace", [&] { return la::w4_workspace_body(rows, out, k, group, bytes); });
}
int la_gemv_w4(const void *x, int64_t x_stride, const void *w, const void *scales, float *y, int64_t y_stride, int32_t rows, int32_t out,
               int32_t k, int32_t group, void *workspace, int64_t workspace_bytes, void *stream) {
    return la::abi_guard("la_gemv_w4",
                         [&] { return la::w4_body(x, x_stride, w, scales, y, y_stride, rows, out, k, group, workspace, workspace_bytes, stream); });
}

}  // extern "C"
