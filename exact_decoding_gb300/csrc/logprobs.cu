// Log probabilities of given tokens, the distribution's entropy and its most
// probable tokens, in one pass over a row of logits (la_logprobs).
//
//   lse = m + log(1 + r),  m = max z,  r = sum over all but one maximal z of e^(z - m)
//   log p_t = z_t - lse,   H = log(1 + r) - s / (1 + r),  s = sum (z - m) e^(z - m)
//
// The largest term is kept out of the sum, and log1p takes r: where one token has
// nearly all of the probability, log p = -log1p(r) and H keep all their bits, which
// log of a sum of 1 and little more would lose.  Both terms of H are >= 0.
//
// Each thread copies 16 logits after 16 to a place of its own in shared memory, a
// pass ahead, so that only it waits for them, and keeps its part of its warp's running
// (m, r, s), with the terms equal to the maximum counted apart.
// Each warp keeps its best tokens as keys (value, then lowest index), which are all
// different, 32 in its lanes.  A value enters only if it is above a threshold that
// the block's warps share, the largest k-th key that any of them has: old ones are too low,
// never too high, so nobody waits for it.  The first comes from the threads' own
// maxima: if k of them are T or more, the row's k-th best is not below T, and a
// short search finds such a T that few more reach.  Lanes push such keys to shared memory; when 32 have
// gathered the warp sorts them and merges.  The warps' lists are merged at the end.
//
// A row is one block's (of 1 to 8 warps, by its length), or a cluster's: each block
// takes a run of it, and the first joins their sums and keys through distributed
// shared memory.  So there is one launch, no workspace, and results that do not depend
// on any order.
//
// Measured: 2048 rows of 32000 fp32 (262 MB) with 20 alternatives 60.4 us, 4.3 TB/s,
// 64 % of a copy's rate; bound by instructions (71 % of the issue slots; without
// alternatives 41.6 us, 93 %).  76 rows of 32016 bf16 with 20 alternatives 9.4 us, where most
// logits are masked 9.7; one row of 32000 with 5 6.7 us: latency of a pass, the search for the
// threshold and the joins.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <type_traits>

#include "abi_guard.h"
#include "la_common.cuh"

namespace la {

constexpr int kLpPass = 16;       // elements of a thread's pass
constexpr int kLpTop = 32;

template <typename T>
struct LpType;
template <>
struct LpType<float> {
    static constexpr int vec = 4;
};
template <>
struct LpType<__nv_bfloat16> {
    static constexpr int vec = 8;
};

// 2^x, off by 2^-22 of it at most; below 2^-126 it is 0
__device__ __forceinline__ float lp_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct LpSum {
    float m, r, s;   // m = -infinity: nothing yet
};
// The sums of both, each about its own maximum.
__device__ __forceinline__ LpSum lp_join(const LpSum &x, const LpSum &y) {
    const bool xb = x.m >= y.m;
    const LpSum a = xb ? x : y, b = xb ? y : x;
    if (b.m == -INFINITY) return {a.m, a.r + b.r, a.s};   // r is 0, or NaN where a value was
    const float d = b.m - a.m, f = lp_ex2(d * 1.4426950408889634f), n = 1.f + b.r;
    // f = 0 and d = -infinity: a product that is 0
    return {a.m, fmaf(n, f, a.r), f > 0.f ? fmaf(f, fmaf(d, n, b.s), a.s) : a.s};
}

using LpKey = unsigned long long;   // 0: none
__device__ __forceinline__ LpKey lp_key(float z, int i) {
    return static_cast<LpKey>(order_key(z + 0.f)) << 32 | static_cast<uint32_t>(~i);   // -0 is 0
}
__device__ __forceinline__ int lp_index(LpKey k) { return static_cast<int>(~static_cast<uint32_t>(k)); }
__device__ __forceinline__ float lp_value(LpKey k) {
    const uint32_t b = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
// Bitonic steps among a warp's lanes, descending.
__device__ __forceinline__ LpKey lp_swap(LpKey x, int o, bool larger) {
    const LpKey y = __shfl_xor_sync(0xffffffffu, x, o);
    return (x > y) == larger ? x : y;
}
__device__ __forceinline__ LpKey lp_sort(LpKey x, int lane) {
#pragma unroll
    for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
        for (int o = n >> 1; o; o >>= 1) x = lp_swap(x, o, ((lane & o) == 0) == ((lane & n) == 0));
    return x;
}
// The 32 best of two descending lists.
__device__ __forceinline__ LpKey lp_merge(LpKey x, LpKey y, int lane) {
    y = __shfl_sync(0xffffffffu, y, 31 - lane);
    x = x > y ? x : y;
#pragma unroll
    for (int o = 16; o; o >>= 1) x = lp_swap(x, o, (lane & o) == 0);
    return x;
}

struct LpArgs {
    la_logprobs_args a;
    int blocks;   // of a row
};

// The larger, NaN if either is.
__device__ __forceinline__ float lp_max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float lp_max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t lp_two(float a, float b) {
    uint64_t y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float2 lp_halves(uint64_t v) {
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(v));
    return y;
}
__device__ __forceinline__ uint64_t lp_add2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ uint64_t lp_mul2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ uint64_t lp_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}

// Keys that a warp gathers before it merges them, and room for half a pass's.
constexpr int kLpGather = 32, kLpRoom = kLpGather + 16 * kLpPass + 32;
constexpr int kLpStages = 2;   // passes of a thread in shared memory

__device__ __forceinline__ void lp_copy(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

template <typename T, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 32 / WARPS) k_logprobs(const __grid_constant__ LpArgs p) {
    constexpr int THREADS = 32 * WARPS;
    constexpr int VEC = LpType<T>::vec, E = kLpPass, NV = E / VEC;   // 16-byte loads of a pass
    constexpr float kLog2e = 1.4426950408889634f;
    constexpr uint32_t kNone = VEC == 4 ? 0xff800000u : 0xff80ff80u;  // -infinity
    extern __shared__ __align__(16) uint8_t lp_smem[];
    uint4(*sh_ring)[NV][THREADS] = reinterpret_cast<uint4(*)[NV][THREADS]>(lp_smem);
    LpKey(*sh_push)[kLpRoom] = reinterpret_cast<LpKey(*)[kLpRoom]>(lp_smem + kLpStages * NV * THREADS * 16);
    __shared__ LpKey sh_list[WARPS][kLpTop];
    __shared__ uint2 sh_first[WARPS];
    __shared__ LpSum sh_sum[WARPS];
    __shared__ LpSum sh_block;
    __shared__ LpKey sh_t;                       // the largest last key of a full list
    __shared__ int sh_n[WARPS];               // keys that a warp has gathered
    const la_logprobs_args &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = p.blocks, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int row = blockIdx.x / C, top = a.n_top;
    if (lane == 0) sh_n[warp] = 0;
    if (tid == 0) sh_t = 0;
    pdl_trigger();
    pdl_wait();
    const T *z = static_cast<const T *>(a.logits) + row * a.stride;
    // From the first 16-byte boundary on in vectors; the few elements before it and behind the last one singly.
    const int head = min(a.vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / static_cast<int>(sizeof(T)));
    const int vecs = (a.vocab - head) / VEC, tail = head + vecs * VEC, odd = head + a.vocab - tail;
    const int per = (vecs + C - 1) / C, v0 = min(rank * per, vecs), v1 = min(v0 + per, vecs);
    const uint4 *zv = reinterpret_cast<const uint4 *>(z + head);
    // A pass's copies; past the run's end the last vector again, which does not count then
    auto copy = [&](int base, int stage) {
        if (base < v1) {
#pragma unroll
            for (int k = 0; k < NV; ++k) lp_copy(smem_u32(&sh_ring[stage][k][tid]), zv + min(base + k * THREADS + tid, v1 - 1));
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    copy(v0, 0);
    float given = -INFINITY;   // the logit of this thread's given token, read while the row is
    if (rank == 0 && tid < a.n_tokens) {
        const int t = a.tokens[static_cast<long long>(row) * a.n_tokens + tid];
        if (t >= 0 && t < a.vocab) given = to_f32<T>(z[t]);
    }
    // Terms of this thread: r those below its warp's maximum m, ones those equal to it; pairs of sums
    float m = -INFINITY;
    uint64_t r = 0, s = 0;
    int ones = 0;
    auto add = [&](auto &v, float most) {   // all lanes of a warp call it
        constexpr int N = sizeof(v) / sizeof(float);
        const uint32_t key = __reduce_max_sync(0xffffffffu, order_key(most + 0.f));
        most = lp_value(static_cast<LpKey>(key) << 32);
        if (most > m) {
            const float d = m - most, f = lp_ex2(d * kLog2e);   // m = -infinity: f = 0
            const float2 y = lp_halves(r), z = lp_halves(s);
            const float n = y.x + y.y + static_cast<float>(ones), old = z.x + z.y;
            s = lp_two(f > 0.f ? f * fmaf(d, n, old) : 0.f, 0.f);
            r = lp_two(n * f, 0.f);
            ones = 0;
            m = most;
        }
        const float base = m == -INFINITY ? 0.f : -m;
        const bool hit = most == m;         // some of these are equal to m
        const uint64_t base2 = lp_two(base, base), log2e2 = lp_two(kLog2e, kLog2e);
        auto terms = [&](auto apart) {
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                float2 d = lp_halves(lp_add2(lp_two(v[e], e + 1 < N ? v[e + 1 < N ? e + 1 : e] : -INFINITY), base2));
                d.x = lp_max_nan(d.x, -20000.f);   // finite: 0 times d
                d.y = lp_max_nan(d.y, -20000.f);
                const uint64_t d2 = lp_two(d.x, d.y);
                const float2 y = lp_halves(lp_mul2(d2, log2e2));
                float x0 = lp_ex2(y.x), x1 = lp_ex2(y.y);
                if constexpr (decltype(apart)::value) {
                    ones += (d.x == 0.f) + (d.y == 0.f);
                    x0 = d.x == 0.f ? 0.f : x0;
                    x1 = d.y == 0.f ? 0.f : x1;
                }
                const uint64_t x2 = lp_two(x0, x1);
                r = lp_add2(r, x2);
                s = lp_fma2(x2, d2, s);
            }
        };
        if (hit) terms(std::true_type{});   // the whole warp
        else terms(std::false_type{});
    };
    LpKey list = 0;            // the lane's of the warp's best so far
    LpKey limit = 0;           // what may enter is above it
    float least = -3.40282347e38f;   // and its value this or more: an equal one may enter, by its index
    volatile int *gathered = &sh_n[warp];
    volatile LpKey *threshold = &sh_t;
    auto raise = [&](LpKey t) {
        limit = max(limit, t);
        least = lp_value(limit);
    };
    auto push = [&](float x, int i) {
        const LpKey k = lp_key(x, i);
        if (k > limit) sh_push[warp][atomicAdd(&sh_n[warp], 1)] = k;
    };
    auto merge = [&](int n) {   // the warp's keys
#pragma unroll 1
        for (int i = 0; i < n; i += 32) {
            const LpKey x = i + lane < n ? sh_push[warp][i + lane] : 0, last = __shfl_sync(0xffffffffu, list, top - 1);
            if (__any_sync(0xffffffffu, x > last)) list = lp_merge(list, lp_sort(x, lane), lane);
        }
        const LpKey last = __shfl_sync(0xffffffffu, list, top - 1);
        if (lane == 0) {
            *gathered = 0;
            if (last > *threshold) atomicMax(&sh_t, last);
        }
        __syncwarp();
    };
    __syncthreads();

#pragma unroll 1
    for (int base = v0, stage = 0; base < v1; base += THREADS * NV, stage ^= 1) {
        copy(base + THREADS * NV, stage ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        uint4 w[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) w[k] = sh_ring[stage][k][tid];
        if (base + THREADS * NV > v1) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (base + k * THREADS + tid >= v1) w[k] = make_uint4(kNone, kNone, kNone, kNone);
        }
        float v[E];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (VEC == 4) {
                    v[4 * k + i] = __uint_as_float(u[i]);
                } else {
                    v[8 * k + 2 * i] = __uint_as_float(u[i] << 16);
                    v[8 * k + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
                }
            }
        }
        float quad[E / 4], most = -INFINITY;   // largest of four, and of all; a NaN is none
#pragma unroll
        for (int q = 0; q < E / 4; ++q) quad[q] = fmaxf(lp_max3(v[4 * q], v[4 * q + 1], v[4 * q + 2]), v[4 * q + 3]);
        most = lp_max3(lp_max3(most, quad[0], quad[1]), quad[2], quad[3]);
        if (top) {
            if (base == v0) {
                // lo: `top` threads or more reach it (or none is asked to), at first the
                // warps' least k / 8-th; hi: fewer do
                const uint32_t mine = most > -INFINITY ? order_key(most + 0.f) : 0u;
                uint32_t rest = mine, lo = 0, hi = 0;
                for (int i = 0; i < top; i += WARPS) {
                    lo = __reduce_max_sync(0xffffffffu, rest);
                    if (rest == lo) rest = 0;
                    hi = max(hi, lo);
                }
                if (lane == 0) sh_first[warp] = make_uint2(lo, hi);
                __syncthreads();
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    lo = min(lo, sh_first[w].x);
                    hi = max(hi, sh_first[w].y);
                }
                if (lo > 0 && top > 1) {
                    ++hi;
                    for (int i = 0; i < 5 && hi - lo > 1; ++i) {
                        const uint32_t mid = lo + (hi - lo) / 2;
                        if (__syncthreads_count(mine >= mid) >= top) lo = mid;
                        else hi = mid;
                    }
                } else if (top == 1) {
                    lo = hi;
                }
                if (lo) raise((static_cast<LpKey>(lo) << 32) - 1);
            } else {
                const LpKey t = *threshold;
                if (t > limit) raise(t);
            }
            if (__any_sync(0xffffffffu, most >= least)) {
                const int first = head + (base + tid) * VEC;
#pragma unroll
                for (int q = 0; q < E / 4; ++q) {
                    if (quad[q] >= least) {
#pragma unroll
                        for (int e = 4 * q; e < 4 * q + 4; ++e)
                            if (v[e] >= least) push(v[e], first + e / VEC * THREADS * VEC + e % VEC);
                    }
                    if (q & 1) {
                        __syncwarp();
                        const int n = *gathered;
                        if (n >= kLpGather) {
                            merge(n);
                            const LpKey t = *threshold;
                            if (t > limit) raise(t);
                        }
                    }
                }
            }
        }
        add(v, most);
    }
    if (rank == C - 1 && odd > 0) {   // the single elements
        const int i = tid < head ? tid : tail + tid - head;
        float v[1] = {tid < odd ? to_f32<T>(z[i]) : -INFINITY};
        if (top && tid < odd && v[0] > -INFINITY) push(v[0], i);
        __syncwarp();
        add(v, v[0] > -INFINITY ? v[0] : -INFINITY);   // a NaN is none
    }
    if (top) {
        __syncwarp();
        merge(*gathered);
        sh_list[warp][lane] = list;
    }

    // The block's sums and list
    LpSum sum;
    {
        const float2 y = lp_halves(r), z = lp_halves(s);
        ones = __reduce_add_sync(0xffffffffu, ones);
        sum = {m, warp_sum(y.x + y.y) + static_cast<float>(ones > 0 ? ones - 1 : 0), warp_sum(z.x + z.y)};
    }
    if (lane == 0) sh_sum[warp] = sum;
    __syncthreads();
    if (top) {   // the warps' lists, two and two
#pragma unroll 1
        for (int o = WARPS / 2; o; o >>= 1) {
            if (warp < o) sh_list[warp][lane] = list = lp_merge(list, sh_list[warp + o][lane], lane);
            __syncthreads();
        }
    }
    if (warp == 0) {
        sum = sh_sum[0];
        for (int w = 1; w < WARPS; ++w) sum = lp_join(sum, sh_sum[w]);
        if (lane == 0) sh_block = sum;
    }
    if (C > 1) {
        cluster_sync_all();
        if (rank == 0 && warp == 0) {
            LpSum sums[7];   // all on their way at once
            LpKey keys[7];
#pragma unroll
            for (int c = 1; c < 8; ++c) {
                if (c >= C) break;
                const uint32_t at = mapa_shared(smem_u32(&sh_block), c);
                sums[c - 1] = {ld_cluster_f32(at), ld_cluster_f32(at + 4), ld_cluster_f32(at + 8)};
                asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(keys[c - 1]) : "r"(mapa_shared(smem_u32(&sh_list[0][lane]), c)) : "memory");
            }
#pragma unroll
            for (int c = 1; c < 8; ++c) {
                if (c >= C) break;
                sum = lp_join(sum, sums[c - 1]);
                if (top) list = lp_merge(list, keys[c - 1], lane);
            }
            if (lane == 0) sh_block = sum;
        }
        cluster_sync_all();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    const LpSum all = sh_block;
    const float l = log1pf(all.r);
    const bool none = all.m == -INFINITY && !isnan(all.r), bad = isnan(all.r) || all.m == INFINITY;
    auto out = [&](float x) { return bad ? NAN : none || x == -INFINITY ? -INFINITY : (x - all.m) - l; };
    if (a.tokens) {
        for (int i = tid; i < a.n_tokens; i += THREADS) {
            const long long at = static_cast<long long>(row) * a.n_tokens + i;
            if (i >= THREADS) {
                const int t = a.tokens[at];
                given = t >= 0 && t < a.vocab ? to_f32<T>(z[t]) : -INFINITY;
            }
            a.logprob[at] = out(given);
        }
    }
    if (a.entropy && tid == 0) a.entropy[row] = bad ? NAN : none ? 0.f : l - all.s / (1.f + all.r);
    if (warp == 0 && lane < top) {
        const long long at = static_cast<long long>(row) * top + lane;
        a.top_ids[at] = list ? lp_index(list) : -1;
        a.top_logprob[at] = list ? out(lp_value(list)) : bad ? NAN : -INFINITY;
    }
}

namespace {

int lp_bad(const char *what, int code = LA_ERR_INVALID_ARG) {
    char msg[256];
    std::snprintf(msg, sizeof(msg), "la_logprobs: %s", what);
    return set_last_error(code, msg);
}

}  // namespace

// Warps of a block: a warp's pass is 512 logits, and what a row costs beside its
// passes grows with them; with more rows than fit at a time fewer warps for each pay
// sooner.  Device us with 8, 4, 2 and 1 warps (fp32, 20 alternatives): 1838 rows of 120: 30.9,
// 16.1, 12.8, 8.0; 100 of 500: 7.8, 4.9, 4.7, 6.2; 2000 of 2288: 26.1, 17.5, 14.4, 20.3; 100 of 2288: 6.2,
// 5.8, 8.2, 13.8; 300 of 8192: 9.1, 10.5, 15.7; 700 of 32000: 30.1, 35.1, 49.9; 2048 of 32000:
// 63.8, 60.5, 62.0.
static int lp_warps(const la_logprobs_args &a, int nsm) {
    if (a.vocab <= 256) return 1;
    if (a.vocab <= 1024 || (a.vocab <= 2560 && a.rows > 8 * nsm)) return 2;
    return a.vocab <= 4096 || a.rows > 7 * nsm ? 4 : 8;
}

template <typename T, int WARPS>
static cudaError_t logprobs_start(const la_logprobs_args &a, int nsm, cudaStream_t s) {
    constexpr int pass = 32 * WARPS * kLpPass, smem = kLpStages * pass * static_cast<int>(sizeof(T)) + WARPS * kLpRoom * 8;
    LpArgs p{};
    p.a = a;
    // Blocks of a row: while the rows leave SMs idle and each has a pass of its own, or, two
    // on an SM, 3.5 passes (bf16, 20 alternatives, 76 rows of 32016: 1 block 13.3 us, 2 9.4, 4 11.3;
    // 152 of 32000: 1 13.6, 2 11.1, 4 16.2; 100 of 128000: 1 35.0, 2 23.3, 4 21.9).
    p.blocks = 1;
    while (p.blocks < 8 && a.vocab > p.blocks * pass && static_cast<long long>(a.rows) * p.blocks * 2 <= (a.vocab / 7 >= p.blocks * pass ? 2 * nsm : nsm)) p.blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * p.blocks);
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.blocks > 1 ? 2 : 1;
    static std::atomic<unsigned long long> done{0};   // bit d: device d allows that much shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(done.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(k_logprobs<T, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) done.fetch_or(1ull << dev);
    }
    return cudaLaunchKernelEx(&cfg, k_logprobs<T, WARPS>, p);
}

template <typename T>
static cudaError_t logprobs_launch(const la_logprobs_args &a, int nsm, cudaStream_t s) {
    switch (lp_warps(a, nsm)) {
    case 1: return logprobs_start<T, 1>(a, nsm, s);
    case 2: return logprobs_start<T, 2>(a, nsm, s);
    case 4: return logprobs_start<T, 4>(a, nsm, s);
    default: return logprobs_start<T, 8>(a, nsm, s);
    }
}

static int logprobs_body(const la_logprobs_args *args, void *stream) {
    if (!args) return lp_bad("null arguments");
    const la_logprobs_args &a = *args;
    if (a.type != LA_F32 && a.type != LA_BF16) return lp_bad("type must be LA_F32 or LA_BF16", LA_ERR_UNSUPPORTED);
    if (a.rows < 0 || a.rows > (1 << 24)) return lp_bad("rows out of range (0 .. 2^24)");
    if (a.vocab < 1 || a.vocab > (1 << 28)) return lp_bad("vocab out of range (1 .. 2^28)");
    if (a.stride < a.vocab) return lp_bad("stride must be at least vocab");
    if (a.rows == 0) return LA_OK;
    if (a.n_tokens < 0 || (a.n_tokens > 0) != (a.tokens != nullptr) || (a.n_tokens > 0) != (a.logprob != nullptr))
        return lp_bad("n_tokens, tokens and logprob come together");
    if (a.n_top < 0 || a.n_top > kLpTop || a.n_top > a.vocab) return lp_bad("n_top must be 0 .. 32 and at most vocab");
    if ((a.n_top > 0) != (a.top_ids != nullptr) || (a.n_top > 0) != (a.top_logprob != nullptr)) return lp_bad("n_top, top_ids and top_logprob come together");
    if (!a.logits) return lp_bad("null logits");
    if (reinterpret_cast<uintptr_t>(a.logits) % (a.type == LA_F32 ? 4 : 2)) return lp_bad("logits must be aligned to their type");
    int nsm = 0;
    const int rc = sm_count(&nsm);
    if (rc != LA_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a.type == LA_F32 ? logprobs_launch<float>(a, nsm, s) : logprobs_launch<__nv_bfloat16>(a, nsm, s);
    return e == cudaSuccess ? LA_OK : lp_bad(cudaGetErrorString(e), LA_ERR_CUDA);
}

}  // namespace la

extern "C" int la_logprobs(const la_logprobs_args *a, void *stream) {
    return la::abi_guard("la_logprobs", [&] { return la::logprobs_body(a, stream); });
}
