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
// Each thread holds 16 logits at a time and a running (m, r, s).
// The row's best tokens are kept as keys (value, then lowest index) that are
// all different, 32 in the lanes of one warp.  A value enters only if it is above the
// last of them; a thread that holds one pushes it to shared memory, and
// the warp merges what was pushed.  The first threshold comes from the threads'
// own maxima: if k of a warp's 32 lanes hold a key above T, the row's k-th best
// does not lie below T.
//
// A row is one block's, or a cluster's: each block takes a run of it, and the
// first joins their sums and keys through distributed shared memory.  So there
// is one launch, no workspace, and results that do not depend on any order.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "abi_guard.h"
#include "la_common.cuh"

namespace la {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
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
    const float d = b.m - a.m, f = expf(d), n = 1.f + b.r;
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

template <typename T>
__global__ void __launch_bounds__(kLpThreads) k_logprobs(const __grid_constant__ LpArgs p) {
    constexpr int VEC = LpType<T>::vec, E = kLpPass, NV = E / VEC;   // 16-byte loads of a pass
    constexpr float kLog2e = 1.4426950408889634f;
    __shared__ LpKey sh_push[kLpThreads * E];    // a pass can push all that it holds
    __shared__ LpKey sh_list[kLpTop];
    __shared__ LpKey sh_first[kLpWarps];
    __shared__ LpSum sh_sum[kLpWarps];
    __shared__ LpSum sh_block;
    __shared__ LpKey sh_t;                       // last key of the list, once it is full
    __shared__ int sh_n;
    const la_logprobs_args &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = p.blocks, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int row = blockIdx.x / C, top = a.n_top;
    if (tid == 0) {
        sh_n = 0;
        sh_t = 0;
    }
    pdl_trigger();
    pdl_wait();
    const T *z = static_cast<const T *>(a.logits) + row * a.stride;
    // From the first 16-byte boundary on in vectors; the few elements before it and behind the last one singly.
    const int head = min(a.vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / static_cast<int>(sizeof(T)));
    const int vecs = (a.vocab - head) / VEC, tail = head + vecs * VEC, odd = head + a.vocab - tail;
    const int per = (vecs + C - 1) / C, v0 = min(rank * per, vecs), v1 = min(v0 + per, vecs);
    const uint4 *zv = reinterpret_cast<const uint4 *>(z + head);

    float given = -INFINITY;   // the logit of this thread's given token, read while the row is
    if (rank == 0 && tid < a.n_tokens) {
        const int t = a.tokens[static_cast<long long>(row) * a.n_tokens + tid];
        if (t >= 0 && t < a.vocab) given = to_f32<T>(z[t]);
    }
    LpSum sum = {-INFINITY, 0.f, 0.f};
    LpKey list = 0;   // warp 0: the lane's best so far
    // Adds N values (-infinity: none) to the thread's sums.
    auto add = [&](auto &v, float most) {
        constexpr int N = sizeof(v) / sizeof(float);
        if (most > sum.m) {
            const float f = expf(sum.m - most), n = 1.f + sum.r;   // sum.m = -infinity: f = 0
            sum.s = f > 0.f ? f * fmaf(sum.m - most, n, sum.s) : 0.f;
            sum.r = f > 0.f ? n * f : 0.f;
            sum.m = most;
            bool out = false;   // one maximal value stands apart
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const bool it = !out && v[e] == most;
                out |= it;
                if (it) v[e] = -INFINITY;
            }
        }
        const float m = sum.m == -INFINITY ? 0.f : sum.m;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float d = v[e] - m, x = lp_ex2(d * kLog2e);
            sum.r += x;
            sum.s = x == 0.f ? sum.s : fmaf(x, d, sum.s);
        }
    };
    // Warp 0 takes in what has been pushed.
    auto take = [&]() {
        const int n = sh_n;
#pragma unroll 1
        for (int i = 0; i < n; i += 32) {
            const LpKey x = i + lane < n ? sh_push[i + lane] : 0, last = __shfl_sync(0xffffffffu, list, top - 1);
            if (__any_sync(0xffffffffu, x > last)) list = lp_merge(list, lp_sort(x, lane), lane);
        }
        __syncwarp();
        const LpKey last = __shfl_sync(0xffffffffu, list, top - 1);
        if (lane == 0) {
            sh_t = last;
            sh_n = 0;
        }
    };
    __syncthreads();

    bool begun = false;
#pragma unroll 1
    for (int base = v0; base < v1; base += kLpThreads * NV) {
        float v[E];
        float most = -INFINITY;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = base + k * kLpThreads + tid;
            uint4 w;
            if (at < v1) w = __ldcs(zv + at);
            if constexpr (VEC == 4) {
                v[4 * k] = __uint_as_float(w.x), v[4 * k + 1] = __uint_as_float(w.y), v[4 * k + 2] = __uint_as_float(w.z), v[4 * k + 3] = __uint_as_float(w.w);
            } else {
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[8 * k + 2 * i] = __uint_as_float(u[i] << 16);
                    v[8 * k + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
                }
            }
            if (at >= v1) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[VEC * k + i] = -INFINITY;
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) most = fmaxf(most, v[e]);   // a NaN is none
        if (top) {
            auto index = [&](int e) { return head + (base + (e / VEC) * kLpThreads + tid) * VEC + e % VEC; };
            LpKey t = 0;
            if (!begun) {
                // The warp's k-th largest of its lanes' largest keys; the largest of the warps' is the threshold.
                LpKey mine = 0;
#pragma unroll
                for (int e = E - 1; e >= 0; --e)
                    if (v[e] == most && most > -INFINITY) mine = lp_key(most, index(e));
#pragma unroll 1
                for (int i = 0; i < top; ++i) {
                    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(mine >> 32));
                    const bool in = static_cast<uint32_t>(mine >> 32) == hi;
                    const uint32_t lo = __reduce_max_sync(0xffffffffu, in ? static_cast<uint32_t>(mine) : 0u);
                    t = static_cast<LpKey>(hi) << 32 | lo;
                    if (mine == t) mine = 0;
                }
                if (lane == 0) sh_first[warp] = t;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kLpWarps; ++w) t = max(t, sh_first[w]);
                begun = true;
            } else {
                t = sh_t ? sh_t + 1 : 0;
            }
            const float least = t ? lp_value(t) : -INFINITY;
            bool pushed = false;
            if (most >= least && most > -INFINITY) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (v[e] >= least && v[e] > -INFINITY) {
                        const LpKey k = lp_key(v[e], index(e));
                        if (k >= t) {
                            sh_push[atomicAdd(&sh_n, 1)] = k;
                            pushed = true;
                        }
                    }
                }
            }
            if (__syncthreads_or(pushed)) {
                if (warp == 0) take();
                add(v, most);
                __syncthreads();
            } else {
                add(v, most);
            }
        } else {
            add(v, most);
        }
    }
    if (rank == C - 1 && odd > 0) {   // the single elements
        float v[1] = {-INFINITY};
        const int i = tid < head ? tid : tail + tid - head;
        if (tid < odd) v[0] = to_f32<T>(z[i]);
        if (top) {
            __syncthreads();   // sh_t is the last pass's
            const LpKey k = tid < odd && v[0] > -INFINITY ? lp_key(v[0], i) : 0;
            if (k > sh_t) sh_push[atomicAdd(&sh_n, 1)] = k;
            __syncthreads();
            if (warp == 0) take();
        }
        add(v, isnan(v[0]) ? -INFINITY : v[0]);
    }

    // The block's sums and list
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const LpSum y = {__shfl_xor_sync(0xffffffffu, sum.m, o), __shfl_xor_sync(0xffffffffu, sum.r, o), __shfl_xor_sync(0xffffffffu, sum.s, o)};
        sum = lane & o ? lp_join(y, sum) : lp_join(sum, y);
    }
    if (lane == 0) sh_sum[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        sum = sh_sum[0];
        for (int w = 1; w < kLpWarps; ++w) sum = lp_join(sum, sh_sum[w]);
        if (lane == 0) sh_block = sum;
        sh_list[lane] = list;
    }
    if (C > 1) {
        cluster_sync_all();
        if (rank == 0 && warp == 0) {
            for (int c = 1; c < C; ++c) {
                const uint32_t at = mapa_shared(smem_u32(&sh_block), c);
                sum = lp_join(sum, {ld_cluster_f32(at), ld_cluster_f32(at + 4), ld_cluster_f32(at + 8)});
                if (top) {
                    LpKey k;
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(k) : "r"(mapa_shared(smem_u32(&sh_list[lane]), c)) : "memory");
                    list = lp_merge(list, k, lane);
                }
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
        for (int i = tid; i < a.n_tokens; i += kLpThreads) {
            const long long at = static_cast<long long>(row) * a.n_tokens + i;
            if (i >= kLpThreads) {
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

cudaError_t logprobs_launch(const la_logprobs_args &a, int nsm, cudaStream_t s) {
    LpArgs p{};
    p.a = a;
    // Blocks of a row: while the rows leave SMs idle and each has a pass of its own
    const int pass = kLpThreads * kLpPass;
    p.blocks = 1;
    while (p.blocks < 8 && static_cast<long long>(a.rows) * p.blocks * 2 <= 2 * nsm && a.vocab > p.blocks * pass) p.blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * p.blocks);
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.blocks > 1 ? 2 : 1;
    return a.type == LA_F32 ? cudaLaunchKernelEx(&cfg, k_logprobs<float>, p) : cudaLaunchKernelEx(&cfg, k_logprobs<__nv_bfloat16>, p);
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
    const cudaError_t e = logprobs_launch(a, nsm, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LA_OK : lp_bad(cudaGetErrorString(e), LA_ERR_CUDA);
}

}  // namespace la

extern "C" int la_logprobs(const la_logprobs_args *a, void *stream) {
    return la::abi_guard("la_logprobs", [&] { return la::logprobs_body(a, stream); });
}
