// Attention of new rows over the paged 8-bit KV cache (la_kv8_attention).
//
// For a query vector q (one row, one head) and the keys j it sees,
//   z_j = scale * q . K_j,   o = sum_j e^(z_j) V_j / sum_j e^(z_j),
// computed in one pass over the keys with the running maximum of the softmax.
// With a power-of-two scale 2^vx on a page's V (new rows: on a row's or a tile's), the
// kernels keep for each row, z in base 2, two whole numbers r and d and
//   L = sum_j 2^(z_j - r),   w_j = 2^(z_j - r + u), u = vx - d   (fp16),
//   O = sum_j w_j V8_j,      o = O 2^d / L.
// r follows the maximum of z lazily (z_j - r <= kLazy), d follows vx so that u
// stays within kUnitLow .. kUnitHigh: weights are at most 2^15, and those
// below 2^-14 are off by 2^-25 at most, 2^(-24 - kUnitLow) of the largest key's
// weight, whatever scales other pages have.  Were one number (a maximum of
// z + vx) to follow both, a page of large scale would leave no bits of the
// others, even where it has no weight.
//
// The work is the list of (sequence, KV head, tile of query vectors) units,
// each a run of key tiles: the sequence's new rows, then its cached tokens.
// Every worker (CTA) takes an equal share of the flattened key tiles of all
// units, read off the device-side lengths, so ragged batches and single long
// sequences fill the GPU alike.  A unit that one worker does not cover leaves
// partial (O, r, d, L) in the workspace, and k_kv8_join adds them in key order.
//
// Short calls are bound by instruction fetches: code that runs once per call
// comes from L2 a line at a time, about 50 instructions per microsecond.  So
// what runs once is written as small loops, and only the loops over keys are
// unrolled, with one exception: the join of a CTA's warps, whose reads would wait
// for one another (0.4 us of a call).  Divisions by sizes known at run time are
// shifts, and a unit's own loads go out before its copies (117 tokens of 32
// heads: 8.5 us with neither, 7.1 with both).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv8.h"

namespace la {

// Bounded wait.  Its loop exists once, not at every wait: the code of a kernel's
// roles has to stay in the instruction cache (k_kv8_tiles, 256 rows over 16k
// tokens, 8 KV heads: 131.6 us with the loops inline, 125.7 without).
__device__ __noinline__ bool bar_wait_on(uint32_t bar, uint32_t parity, unsigned *err, unsigned bit) { return mbar_wait(bar, parity, err, bit); }
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, unsigned *err, unsigned bit) {
    return mbar_try_wait(bar, parity) || bar_wait_on(bar, parity, err, bit);
}

constexpr float kKv8Log2e = 1.4426950408889634f;
constexpr float kLazy = 8.f;
constexpr float kUnitLow = -5.f, kUnitHigh = 7.f, kUnit = 2.f;   // u, and what it becomes when d changes
// O's reach: |w_j V_j| 2^-d for the keys so far is below 2^(reach - d).  What the
// pages in the window add is kReach above d at most; d stays within kSpan of the
// reach, so that O (2^30 keys) never passes fp32's range.
constexpr float kReach = 25.f, kSpan = 90.f;

struct Kv8Args {
    la_kv8_cache c;
    la_kv8_attn a;
    int gq;            // query heads per KV head
    int page_log2;
    int q_tile;        // query vectors per unit
    int q_log2, k_log2;   // of q_tile and k_tile: a division by a number known at run time takes hundreds of cycles where nothing hides it
    int k_tile, n_tile;   // cached tokens, new rows per key tile (the same, or 0: the new rows are not counted in tiles)
    int unit_cost;     // what a unit costs beside its key tiles, in tiles
    int snap;          // a share that begins within this many tiles of a unit's begin begins with the unit
    int whole;         // 1: worker w runs units w, w + workers, ... whole, and nothing is joined
    int workers;
    int hinted;        // max_rows is the caller's
    float scale_log2;  // scale * log2(e)
    int window, sinks; // of la_kv8_attention_window
    float *part;       // [workers][2][q_tile][head_dim] unnormalised sums
    float *part_ml;    // [workers][2][q_tile][4] r, d and L
    struct Kv8Split *split;   // [workers]
};
// What a worker's range begins with: a unit that earlier workers began, or not.
struct Kv8Split {
    long long t0, t1, total;   // the unit's place in the flattened list, and the list's length
    int inside;                // 1: the range begins inside a unit
    int first, head, qv0, nqv; // the unit: first row of its slot, KV head, query vectors
    int pad;
};

// ------------------------------------------------------------------ work list
struct Kv8Seq {
    int first, rows;         // rows of the slot
    int len;                 // cached tokens
    int qtiles;              // tiles of query vectors
    int ctiles, ntiles;      // key tiles of the cache and of the new rows
    int keep, skip;          // with a window: the cache's first `keep` tiles, then those `skip` behind
    // A unit's length in the flattened list: its key tiles behind unit_cost
    // empty ones, which stand for what a unit costs beside its tiles (its
    // queries, the first copies' latency, the join of the warps).  Where units
    // stay whole the list is one of units.
    int ktiles;
};

// With a window (WIN) a row sees the first `sinks` and the last `window` of its
// list of keys: the cached tokens in order, then the new rows that it sees, in
// order.  Its window begins at place len + n - window of that list, n the new
// rows that it sees: cached tokens before it are seen if they are among the
// first, and tiles between the two that no row of the slot sees are left out of
// the slot's tiles.  So a unit's work is what its rows see, but for tiles at the
// two edges, in which keys are masked.
//
// Windows measured (floor: the window's bytes, or its products): the last 4096 of
// 65413 tokens and 4 first ones, 64 heads over 8 KV heads, 13.5 us (8.4 MB, latency); 64
// sequences of up to 8192, window 1024, 32.9 us (130 MB: 3.9 TB/s); 121 rows of 32
// heads, window 512, 32.2 us; 256 rows over 16k tokens, window 4096, 63.9 us
// (115.7 without).  What a short unit costs beside its tiles bounds them: positions,
// pages and queries are looked up one behind another before the first product.
template <bool WIN>
__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8Args &p, int s) {
    Kv8Seq q;
    q.rows = kv8_rows(p.c, p.a.row_start, p.a.n_rows, s, &q.first);
    q.len = kv8_len(p.c, s);
    q.qtiles = static_cast<int>((static_cast<long long>(q.rows) * p.gq + p.q_tile - 1) >> p.q_log2);
    q.ctiles = (q.len + p.k_tile - 1) >> p.k_log2;
    if constexpr (WIN) {
        const int first = min(max(q.len + (p.a.k && !p.a.vis ? 1 : 0) - p.window, 0), q.len);   // of the slot's earliest window
        q.keep = (min(p.sinks, q.len) + p.k_tile - 1) >> p.k_log2;
        q.skip = max((first == q.len ? q.ctiles : first >> p.k_log2) - q.keep, 0);
        q.ctiles -= q.skip;
    }
    q.ntiles = p.a.k && p.n_tile ? (q.rows + p.n_tile - 1) >> p.k_log2 : 0;
    q.ktiles = p.whole ? 1 : p.unit_cost + q.ctiles + q.ntiles;
    return q;
}

// The cached tile that is number ct of the slot's.
template <bool WIN>
__device__ __forceinline__ int kv8_tile(const Kv8Seq &q, int ct) { return WIN && ct >= q.keep ? ct + q.skip : ct; }

// tiles[s] for s = 0 .. n_seqs; every thread of the CTA calls it.
template <bool WIN>
__device__ __forceinline__ void kv8_plan(const Kv8Args &p, long long *tiles, long long *warp_sum) {
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int per = (p.c.n_seqs + nt - 1) / nt;
    const int s0 = min(tid * per, p.c.n_seqs), s1 = min(s0 + per, p.c.n_seqs);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
        const Kv8Seq q = kv8_seq<WIN>(p, s);
        const long long t = static_cast<long long>(q.qtiles) * p.c.n_kv_heads * q.ktiles;
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
__device__ __forceinline__ long long kv8_div(long long a, long long b) {   // a >= 0, b > 0; 32 bits where they do: 64-bit division is long code
    return (a | b) >> 32 ? a / b : static_cast<long long>(static_cast<unsigned>(a) / static_cast<unsigned>(b));
}
__device__ __forceinline__ long long kv8_share(long long total, int w, int workers) { return kv8_div(total * w, workers); }

// The pieces of work of one worker, in order.
struct Kv8Walk {
    long long at, end;
};
// With snap = unit_cost - 1 a share that begins in a unit's empty tiles begins
// with the unit: a piece without key tiles would cost as much as one with some.
template <bool WIN>
__device__ __forceinline__ Kv8Walk kv8_walk(const Kv8Args &p, const long long *tiles) {
    const long long total = tiles[p.c.n_seqs];
    const int workers = kv8_workers(p, total), b = static_cast<int>(blockIdx.x), w = b + (threadIdx.x & 1);
    if (p.whole) return {b, total};
    if (b >= workers) return {0, 0};
    long long at = kv8_share(total, w, workers);   // even lanes: where the share begins, odd ones: where it ends
    if (p.snap > 0 && w < workers) {
        const int s = kv8_find(tiles, p.c.n_seqs, at), kt = kv8_seq<WIN>(p, s).ktiles;
        const long long in_slot = at - tiles[s];
        const int in_unit = static_cast<int>(in_slot - kv8_div(in_slot, kt) * kt);
        if (in_unit <= p.snap) at -= in_unit;
    }
    return {__shfl_sync(0xffffffffu, at, 0), __shfl_sync(0xffffffffu, at, 1)};
}
struct Kv8Piece {
    int s, head, qv0, nqv;
    int k0, k1;          // key tiles
    bool all, begins;    // the whole unit; its first piece
    Kv8Seq sq;
};
template <bool WIN>
__device__ __forceinline__ bool kv8_next(const Kv8Args &p, const long long *tiles, Kv8Walk &w, Kv8Piece &u) {
    if (w.at >= w.end) return false;
    u.s = kv8_find(tiles, p.c.n_seqs, w.at);
    u.sq = kv8_seq<WIN>(p, u.s);
    const int kt = u.sq.ktiles;
    const long long in_slot = w.at - tiles[u.s];
    const int unit = static_cast<int>(p.whole ? in_slot : kv8_div(in_slot, kt));
    if (p.whole) {
        u.k0 = 0;
        u.k1 = u.sq.ctiles + u.sq.ntiles;
        u.all = u.begins = true;
        w.at += p.workers;
    } else {
        const int v0 = static_cast<int>(in_slot - static_cast<long long>(unit) * kt);
        const int v1 = static_cast<int>(min(static_cast<long long>(kt), v0 + (w.end - w.at)));
        u.k0 = max(v0 - p.unit_cost, 0);
        u.k1 = max(v1 - p.unit_cost, 0);
        u.all = v0 == 0 && v1 == kt;
        u.begins = v0 == 0;
        w.at += v1 - v0;
    }
    u.head = u.sq.qtiles == 1 ? unit : unit / u.sq.qtiles;
    u.qv0 = (unit - u.head * u.sq.qtiles) << p.q_log2;
    u.nqv = min(p.q_tile, u.sq.rows * p.gq - u.qv0);
    return true;
}

// Worker b's entry for k_kv8_join, by one thread: `inside` if its first piece u does not begin its unit.
__device__ __forceinline__ void kv8_note(const Kv8Args &p, const long long *tiles, bool any, const Kv8Piece &u) {
    Kv8Split x{};
    x.total = tiles[p.c.n_seqs];
    x.inside = any && !u.begins;
    if (x.inside) {
        const int kt = u.sq.ktiles;
        const int unit = u.head * u.sq.qtiles + (u.qv0 >> p.q_log2);
        x.t0 = tiles[u.s] + static_cast<long long>(unit) * kt;
        x.t1 = x.t0 + kt;
        x.first = u.sq.first;
        x.head = u.head;
        x.qv0 = u.qv0;
        x.nqv = u.nqv;
    }
    p.split[blockIdx.x] = x;
}

// ------------------------------------------------------------------ window
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
// The n lowest of x's bits that are set.
__device__ __forceinline__ uint32_t low_set(uint32_t x, int n) {
    uint32_t rest = x;
    for (int i = 0; i < n && rest; ++i) rest &= rest - 1;
    return x & ~rest;
}
// New rows that `row` of a slot with `rows` rows, the first at `first`, sees without a window.
__device__ __noinline__ int kv8_seen(const Kv8Args &p, int first, int rows, int row) {
    if (!p.a.k) return 0;
    if (!p.a.vis) return row + 1;
    int n = 0;
    for (int w = 0; w < 8; ++w) n += __popc(p.a.vis[(static_cast<long long>(first) + row) * 8 + w] & low_bits(rows - 32 * w));
    return n;
}
// Of new rows key .. key + 31 (key a multiple of 32) those that `row` sees with the window.
__device__ __noinline__ uint32_t kv8_window_new(const Kv8Args &p, int first, int rows, int len, int row, int key) {
    if (!p.a.vis) return low_bits(row + 1 - key) & (low_bits(p.sinks - len - key) | ~low_bits(row + 1 - p.window - key));
    if (key >= 256) return 0u;
    uint32_t word = 0;
    int before = 0, all = 0;   // of the rows that it sees: those before the word
    for (int w = 0; w < 8; ++w) {
        const uint32_t x = p.a.vis[(static_cast<long long>(first) + row) * 8 + w] & low_bits(rows - 32 * w);
        if (w == key / 32) {
            word = x;
            before = all;
        }
        all += __popc(x);
    }
    return word & (low_set(word, p.sinks - len - before) | ~low_set(word, all - p.window - before));
}
// Of cached tokens key .. key + 31 those that a row sees whose window begins at place `from`.
__device__ __forceinline__ uint32_t kv8_window_old(const Kv8Args &p, int from, int key) { return low_bits(p.sinks - key) | ~low_bits(from - key); }
// Whether some row of a piece may not see some of cached tokens key .. key + n - 1 of its tiles.
__device__ __forceinline__ bool kv8_edge(const Kv8Args &p, const Kv8Seq &q, int last_row, int key, int n) {
    const int seen = !p.a.k ? 0 : p.a.vis ? min(q.rows, 256) : last_row + 1;   // at most
    return key + n > p.sinks && key < q.len + seen - p.window;
}

// ------------------------------------------------------------------ mma
// D (16 x 8, fp32) += A (16 x 16, fp16) * B (16 x 8, fp16).
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
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
// a * b for factors on scores, within fp32's normal numbers: 0 times a masked
// key's -infinity, and infinity times a score of 0, would be NaN.
__device__ __forceinline__ float factor(float a, float b) { return fminf(fmaxf(a * b, 1.17549435e-38f), 3.40282347e38f); }
// Exponent x such that |v| < 2^(x + 15) for the largest finite |v| = amax: v * 2^-x fits fp16.
__device__ __forceinline__ int fit_f16(float amax) { return max(exponent_of(amax) - 14, kKv8MinExp); }

// ------------------------------------------------------------------ few query vectors per KV head
// k_kv8_rows: 16 query vectors per unit (all heads of a KV head's group for
// one row, or some rows).  Bound by the cache's bytes: every byte is read
// once and meets 16 query vectors (64 sequences of up to 8192 tokens, 8 KV
// heads: 548 MB in 94 us).  The warps of a CTA take the unit's tiles
// (one page each) in turn, each with its own running softmax and its own ring
// of page blocks in shared memory, so no barrier is met inside a unit; they
// are joined through shared memory at the unit's end.  A block of K or V of
// one (page, KV head) is one run of page * head_dim bytes: one bulk copy.
//
// From shared memory the bytes go to the B operand of mma.m16n8k16 without a
// transpose: the products are sums over dims (keys), so any order will do as
// long as q (the weights) has the same one.
//   K: column n of product j is key KT/4 (n >> 1) + 2 j + (n & 1) of the piece;
//      lane (n, t) reads HD / 4 consecutive bytes of that key's row.
//   V: lane (n, t) reads its KT / 4 consecutive keys of dim 8 i + n.
// Then the weights of product j's columns 2 t, 2 t + 1 are this lane's keys
// KT/4 t + 2 j, + 1: already the A operand of the second product.
// The new rows, at most a few here, are added key by key in fp32.
constexpr int kRowsQ = 16;
constexpr float kRowsUnit = -9.f;   // d at first: a page of values of order one has a scale of 2^-7, which this fits

template <int HD, int PAGE>
struct Rows {
    static constexpr int block = HD * PAGE;                                     // bytes of one page's K (or V) of a head
    // 8 warps an SM at up to 255 registers.  (12 at 168, two blocks each,
    // spill: 133 us against 118 for 64 sequences of up to 8192 tokens, 8 KV heads.)
    static constexpr int warps = 4;
    static constexpr int slots = block >= 8192 ? 3 : 6;                         // of a warp's ring; K and V alternate
    static constexpr int per_sm = block > 8192 ? 1 : block < 4096 ? 3 : 2;      // CTAs per SM that registers and the ring allow
    static constexpr int ring = block * slots * warps;
    static constexpr int join = warps * kRowsQ * (HD + 4) * 4;                  // over the ring, at the end of a unit
    // q in fp16: lane t's HD / 4 dims and 16 bytes more, so that the lanes
    // (g, t) of a quarter warp read different banks
    static constexpr int q_piece = HD / 2 + 16, q_row = 4 * q_piece;
    static constexpr int q_off = ring > join ? ring : join;
    static constexpr int qf_off = q_off + kRowsQ * q_row;                       // [16] factor on a row's scores
    static constexpr int ml_off = qf_off + kRowsQ * 4;
    static constexpr int reach_off = ml_off + warps * kRowsQ * 16;              // [warp][16] reach of O, relative to r
    static constexpr int bar_off = reach_off + warps * kRowsQ * 4;
    static constexpr int sum_off = bar_off + warps * slots * 8;
    static constexpr int tiles_off = sum_off + warps * 8;                  // (n_seqs + 1) prefix sums follow
    static size_t bytes(int n_seqs) { return tiles_off + (static_cast<size_t>(n_seqs) + 1) * 8; }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Untiled bulk copy global -> shared, completing `bytes` on mbarrier `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
// Larger magnitudes of bf16 pairs: they order like their bits.
__device__ __forceinline__ uint32_t most2(uint32_t m, uint32_t x) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
    return r;
}
// Exponent that fits the larger half of `top` into fp16 (1 stays for what is not finite: it reaches no finite result).
__device__ __forceinline__ int fit_pair(uint32_t top) {
    const uint32_t x = max(top & 0xffffu, top >> 16);
    return x < 0x7f80u ? fit_f16(bf16_bits(x)) : 0;
}
// A bf16 pair times f, as an fp16 pair.
__device__ __forceinline__ uint32_t scaled_f16(uint32_t w, float f) { return pack_f16(bf16_bits(w & 0xffffu) * f, __uint_as_float(w & 0xffff0000u) * f); }

// Online softmax of one piece: scores sc (columns: this lane's keys, `live`
// of them) to the fp16 weights w16, with r, d, the sum l and O's factor.
// reach: of O, for rows g and g + 8 (in shared memory: it is seldom asked for).
// both: rows 8 .. 15 hold query vectors; else their weights are 0.
template <int NJ, int NI>
__device__ __forceinline__ void rows_softmax(float (&sc)[NJ][4], bool both, int live, float kf, const float (&qf)[2], int vx, float (&r)[2], float (&d)[2],
                                             float (&l)[2], float *reach, float (&o)[NI][4], uint32_t (&w16)[NJ][2]) {
    if (live < 2 * NJ) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (2 * j + (e & 1) >= live) sc[j][e] = -INFINITY;   // factors are positive
    }
    // rows g (elements 0, 1 of a product) and g + 8 (2, 3)
    float f[2] = {1.f, 1.f}, nr[2] = {r[0], r[1]}, nd[2] = {d[0], d[1]};
    const float v = static_cast<float>(vx);
    bool change = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h && !both) continue;
        f[h] = factor(kf, qf[h]);
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < NJ; ++j) mx = fmaxf(mx, fmaxf(sc[j][2 * h], sc[j][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float z = mx * f[h];
        const bool grow = r[h] == -INFINITY ? z > -INFINITY : z - r[h] > kLazy;
        const bool shift = z > -INFINITY && (v - d[h] > kUnitHigh || v - d[h] < kUnitLow);
        if (grow) nr[h] = ceilf(z);
        if (shift) nd[h] = fmaxf(v - kUnit, fmaxf(reach[8 * h], d[h] + kReach) - (grow ? nr[h] - r[h] : 0.f) - kSpan);
        change |= grow || shift;
    }
    if (__any_sync(0xffffffffu, change)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool grow = nr[h] != r[h];
            const float far = fmaxf(reach[8 * h], d[h] + kReach) - (grow ? nr[h] - r[h] : 0.f);
            const float fl = grow ? ex2(r[h] - nr[h]) : 1.f, fo = fl * ex2(d[h] - nd[h]);
            __syncwarp();
            reach[8 * h] = far;   // the quad's lanes write the same
            __syncwarp();
            r[h] = nr[h];
            d[h] = nd[h];
            l[h] *= fl;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                o[i][2 * h] *= fo;
                o[i][2 * h + 1] *= fo;
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h && !both) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) w16[j][h] = 0u;
            continue;
        }
        const float u = v - d[h], off = u - (r[h] == -INFINITY ? 0.f : r[h]);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float a = ex2(fmaf(sc[j][2 * h], f[h], off)), b = ex2(fmaf(sc[j][2 * h + 1], f[h], off));
            s0 += a;
            s1 += b;
            w16[j][h] = pack_f16(a, b);
        }
        l[h] += (s0 + s1) * ex2(-u);
    }
}

template <int HD, int PAGE, bool WIN>
__global__ void __launch_bounds__(32 * Rows<HD, PAGE>::warps, Rows<HD, PAGE>::per_sm) k_kv8_rows(const __grid_constant__ Kv8Args p) {
    using Lay = Rows<HD, PAGE>;
    constexpr int NI = HD / 8;                    // 8-dim groups of the output
    constexpr int KT = PAGE < 64 ? PAGE : 64;     // keys per piece
    constexpr int CH = KT / 4, NJ = KT / 8;       // of them, one lane's; products
    constexpr int NS = Lay::slots, NW = Lay::warps;
    extern __shared__ __align__(128) uint8_t smem[];
    float4 *sh_ml = reinterpret_cast<float4 *>(smem + Lay::ml_off);  // [warp][16] r, d, l
    float *sh_o = reinterpret_cast<float *>(smem);                   // [warp][16][HD + 4], over the ring
    float *sh_qf = reinterpret_cast<float *>(smem + Lay::qf_off);
    long long *tiles = reinterpret_cast<long long *>(smem + Lay::tiles_off);
    pdl_trigger();
    const la_kv8_cache &c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * NS * Lay::block, bars = smem_u32(smem + Lay::bar_off) + warp * NS * 8;
    const uint8_t *my_ring = smem + warp * NS * Lay::block;
    float *reach = reinterpret_cast<float *>(smem + Lay::reach_off) + warp * kRowsQ + g;
    if (lane < NS) mbar_init(bars + lane * 8, 1);
    fence_barrier_init();
    pdl_wait();
    kv8_plan<WIN>(p, tiles, reinterpret_cast<long long *>(smem + Lay::sum_off));
    Kv8Walk walk = kv8_walk<WIN>(p, tiles);
    Kv8Piece u;
    int in_slot = 0, out_slot = 0;   // ring positions: the next block to load, the next to read
    uint32_t out_phase = 0;
    bool ok = true;                  // false once a wait gave up: this warp loads nothing more
    bool noted = p.whole;

    for (;;) {
        const bool any = kv8_next<WIN>(p, tiles, walk, u);
        auto note = [&]() {
            if (!noted && tid == 0) kv8_note(p, tiles, any, u);
            noted = true;
        };
        if (!any) {
            note();
            break;
        }
        const Kv8Seq sq = u.sq;
        // This warp's tiles: pages page0 + NW i, i = 0 .. nc - 1.
        const int page0 = u.k0 + warp, s = u.s, head = u.head;
        // The first of its new rows.  Warp 0 has no fewer tiles than another; a window's rows begin with the last warp.
        const int new0 = WIN ? NW - 1 - warp : warp;
        const int nc = ok && page0 < u.k1 ? (u.k1 - page0 + NW - 1) / NW : 0;
        // q first, and the new row that this warp begins with: behind the copies of
        // a full GPU they wait their turn (64 sequences of 1090 tokens, 8 KV heads:
        // 7000 cycles for q alone).
        constexpr int NP = HD / 64;   // 16-byte pieces of a thread's HD / 8 dims
        uint4 q_raw[NP];
        if (tid < 8 * kRowsQ) {
            const int part = tid & 7, qv = u.qv0 + (tid >> 3);
            const bool in = qv - u.qv0 < u.nqv;
            const int row = in ? qv / p.gq : 0;
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.a.q) + (sq.first + row) * p.a.q_stride +
                                                               (head * p.gq + (in ? qv - row * p.gq : 0)) * HD + part * (HD / 8));
#pragma unroll
            for (int i = 0; i < NP; ++i) q_raw[i] = in ? src[i] : make_uint4(0, 0, 0, 0);
        }
        uint4 kw[HD / 32];
        uint32_t vw[NI];
        auto load_new = [&](int j) {
            const uint4 *kj = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.a.k) + (sq.first + j) * p.a.k_stride + head * HD + t * (HD / 4));
            const uint32_t *vj = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.a.v) + (sq.first + j) * p.a.v_stride + head * HD) + t;
#pragma unroll
            for (int i = 0; i < HD / 32; ++i) kw[i] = kj[i];
#pragma unroll
            for (int i = 0; i < NI; ++i) vw[i] = vj[4 * i];
        };
        const int n_new = u.begins && p.a.k ? sq.rows : 0;
        if (new0 < n_new) load_new(new0);
        // Block 2 i is K of tile i, block 2 i + 1 its V.  Page numbers and
        // scales are looked up 32 tiles at a time, lane i for tile 32 n + i
        // (last_*: the 32 tiles before, some of which may still be read).
        int my_page = -1, last_page = -1, issued = 0;
        float my_kf = 0.f, last_kf = 0.f, my_vs = 0.f, last_vs = 0.f;
        auto issue = [&]() {
            const int i = issued >> 1;
            if ((issued & 63) == 0) {
                last_page = my_page;
                last_vs = my_vs;
                last_kf = my_kf;
                my_page = i + lane < nc ? kv8_page(c, s, kv8_tile<WIN>(sq, page0 + NW * (i + lane))) : -1;
                const long long blk = kv8_block(c, p.a.layer, max(my_page, 0), head);
                my_kf = c.k_scale[blk];
                my_vs = c.v_scale[blk];
            }
            const int pg = __shfl_sync(0xffffffffu, my_page, i & 31);
            if (lane == 0) {
                const uint32_t bar = bars + in_slot * 8;
                if (pg >= 0) {
                    mbar_arrive_expect_tx(bar, Lay::block);
                    bulk_load(ring + in_slot * Lay::block,
                              static_cast<const uint8_t *>(issued & 1 ? c.v : c.k) + kv8_block(c, p.a.layer, pg, head) * Lay::block, Lay::block, bar);
                } else {
                    mbar_arrive_expect_tx(bar, 0);   // a page number outside the cache: nothing is loaded, no key counts
                }
            }
            __syncwarp();
            in_slot = in_slot + 1 == NS ? 0 : in_slot + 1;
            ++issued;
        };
#pragma unroll 1
        while (issued < min(NS, 2 * nc)) issue();
        note();   // while the first copies are on their way

        // q as fp16, each vector scaled by a power of two to fit: 8 threads a row.
        if (tid < 8 * kRowsQ) {
            uint4 (&w)[NP] = q_raw;
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < NP; ++i) top = most2(most2(most2(most2(top, w[i].x), w[i].y), w[i].z), w[i].w);
#pragma unroll
            for (int k = 1; k < 8; k <<= 1) top = most2(top, __shfl_xor_sync(0xffffffffu, top, k));
            const int qx = fit_pair(top);
            const float f = power_of(-qx);
            const int r = tid >> 3, part = tid & 7;
            uint4 *dst = reinterpret_cast<uint4 *>(smem + Lay::q_off + r * Lay::q_row + (part >> 1) * Lay::q_piece + (part & 1) * (HD / 4));
#pragma unroll
            for (int i = 0; i < NP; ++i) dst[i] = make_uint4(scaled_f16(w[i].x, f), scaled_f16(w[i].y, f), scaled_f16(w[i].z, f), scaled_f16(w[i].w, f));
            if (part == 0) sh_qf[r] = factor(power_of(qx), p.scale_log2);
        }
        __syncthreads();
        const uint8_t *my_q = smem + Lay::q_off + g * Lay::q_row + t * Lay::q_piece;   // row g; row g + 8 lies 8 rows behind
        const float qf[2] = {sh_qf[g], sh_qf[g + 8]};

        float r[2] = {-INFINITY, -INFINITY}, d[2] = {kRowsUnit, kRowsUnit}, l[2] = {0.f, 0.f};
        float far[2] = {-INFINITY, -INFINITY};   // reach of O, of the new rows
        float o[NI][4];
#pragma unroll
        for (int i = 0; i < NI; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

        int from[2] = {0, 0};   // where the rows' windows begin
        if constexpr (WIN) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h)
            {
                const int row = min(u.qv0 + g + 8 * h, u.qv0 + u.nqv - 1) / p.gq;
                from[h] = sq.len + (p.a.vis ? kv8_seen(p, sq.first, sq.rows, row) : p.a.k ? row + 1 : 0) - p.window;
            }
        }

        // ---- new rows, in the piece that begins the unit: one key at a time
        if (n_new > 0) {
            const int r0 = g < u.nqv ? (u.qv0 + g) / p.gq : -1, r1 = g + 8 < u.nqv ? (u.qv0 + g + 8) / p.gq : -1;
#pragma unroll 1
            for (int j = new0; j < n_new; j += NW) {
                bool see[2];
                if (WIN && !p.a.vis) {
                    const int w0 = p.sinks - sq.len, w1 = p.window;
                    see[0] = j <= r0 && (j < w0 || j > r0 - w1);
                    see[1] = j <= r1 && (j < w0 || j > r1 - w1);
                } else if constexpr (WIN) {
                    see[0] = r0 >= 0 && (kv8_window_new(p, sq.first, sq.rows, sq.len, r0, j & ~31) >> (j & 31) & 1u);
                    see[1] = r1 >= 0 && (kv8_window_new(p, sq.first, sq.rows, sq.len, r1, j & ~31) >> (j & 31) & 1u);
                } else if (p.a.vis) {
                    see[0] = r0 >= 0 && j < 256 && (p.a.vis[(static_cast<long long>(sq.first) + r0) * 8 + j / 32] >> (j % 32) & 1u);
                    see[1] = r1 >= 0 && j < 256 && (p.a.vis[(static_cast<long long>(sq.first) + r1) * 8 + j / 32] >> (j % 32) & 1u);
                } else {
                    see[0] = j <= r0;
                    see[1] = j <= r1;
                }
                float z[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < HD / 32; ++i) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(my_q + 16 * i), b = *reinterpret_cast<const uint4 *>(my_q + 8 * Lay::q_row + 16 * i);
                    const uint32_t x[4] = {kw[i].x, kw[i].y, kw[i].z, kw[i].w}, y[4] = {a.x, a.y, a.z, a.w}, w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float lo = bf16_bits(x[k] & 0xffffu), hi = __uint_as_float(x[k] & 0xffff0000u);
                        const float2 qa = __half22float2(*reinterpret_cast<const __half2 *>(&y[k])), qb = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                        z[0] = fmaf(qa.x, lo, fmaf(qa.y, hi, z[0]));
                        z[1] = fmaf(qb.x, lo, fmaf(qb.y, hi, z[1]));
                    }
                }
                // V's largest magnitude: what it reaches in O may raise d.
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < NI; ++i) top = most2(top, vw[i]);
                top = most2(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = most2(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int ve = exponent_of(bf16_bits(max(top & 0xffffu, top >> 16)));   // 128: a NaN or infinity, which hides its neighbours' size
                float w[2], alpha[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    z[h] += __shfl_xor_sync(0xffffffffu, z[h], 1);
                    z[h] += __shfl_xor_sync(0xffffffffu, z[h], 2);
                    const float x = see[h] ? z[h] * qf[h] : -INFINITY, nr = x > r[h] ? ceilf(x) : r[h], base = nr == -INFINITY ? 0.f : nr;
                    const float fl = ex2(r[h] - base);
                    far[h] = fmaxf(far[h] - (base - r[h]), (x - base) + static_cast<float>(ve == 128 ? 0 : ve + 1));
                    const float nd = fmaxf(d[h], far[h] - kSpan);
                    alpha[h] = fl * ex2(d[h] - nd);
                    r[h] = nr;
                    d[h] = nd;
                    l[h] = l[h] * fl + ex2(x - base);
                    w[h] = ex2((x - base) - nd);
                }
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const float lo = bf16_bits(vw[i] & 0xffffu), hi = __uint_as_float(vw[i] & 0xffff0000u);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // what a row does not see never meets it, not even times 0
                        o[i][2 * h] = fmaf(w[h], see[h] ? lo : 0.f, o[i][2 * h] * alpha[h]);
                        o[i][2 * h + 1] = fmaf(w[h], see[h] ? hi : 0.f, o[i][2 * h + 1] * alpha[h]);
                    }
                }
                if (j + NW < n_new) load_new(j + NW);
            }
            // Every lane of a quad has added the key: l is summed over the quad below.
            if (t != 0) l[0] = l[1] = 0.f;
        }
        reach[0] = far[0];
        reach[8] = far[1];

        // ---- cached tokens
        auto landed = [&]() {   // the next block to read is there
            ok = __all_sync(0xffffffffu, bar_wait(bars + out_slot * 8, out_phase, c.status, LA_KV8_TIMEOUT));
            return ok;
        };
        auto next = [&]() {     // it has been read: its slot takes the next block to load
            __syncwarp();
            if (++out_slot == NS) {
                out_slot = 0;
                out_phase ^= 1;
            }
            if (issued < 2 * nc) issue();
        };
        int read = 0;           // blocks read
#pragma unroll 1
        for (int i = 0; i < nc; ++i) {
            if (!landed()) break;
            const bool old = i >> 5 != (issued - 1) >> 6;   // issue() is in the next 32 tiles already
            const int pg = __shfl_sync(0xffffffffu, old ? last_page : my_page, i & 31);
            const float kf_ = __shfl_sync(0xffffffffu, old ? last_kf : my_kf, i & 31), kf = pg < 0 ? 1.f : kf_;
            const float vs_ = __shfl_sync(0xffffffffu, old ? last_vs : my_vs, i & 31);
            const int vx = pg < 0 ? 0 : exponent_of(vs_);
            const int key0 = kv8_tile<WIN>(sq, page0 + NW * i) * PAGE, left = pg < 0 ? 0 : sq.len - key0;   // keys of this page that count
            const bool edge = WIN && kv8_edge(p, sq, (u.qv0 + u.nqv - 1) / p.gq, key0, PAGE);
            const uint8_t *kblk = my_ring + out_slot * Lay::block, *vblk = nullptr;
#pragma unroll 1
            for (int piece = 0; piece < PAGE / KT; ++piece) {
                float sc[NJ][4];
#pragma unroll
                for (int j = 0; j < NJ; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
                const uint8_t *row = kblk + (piece * KT + CH * (g >> 1) + (g & 1)) * HD + t * (HD / 4);
#pragma unroll 1
                for (int x = 0; x < HD / 64; ++x) {   // steps outside, products inside: their sums do not wait on one another
                    const uint4 qa0 = *reinterpret_cast<const uint4 *>(my_q + 32 * x), qa1 = *reinterpret_cast<const uint4 *>(my_q + 32 * x + 16);
                    const uint4 qb0 = *reinterpret_cast<const uint4 *>(my_q + 8 * Lay::q_row + 32 * x), qb1 = *reinterpret_cast<const uint4 *>(my_q + 8 * Lay::q_row + 32 * x + 16);
                    const uint32_t q[4][4] = {{qa0.x, qb0.x, qa0.y, qb0.y}, {qa0.z, qb0.z, qa0.w, qb0.w}, {qa1.x, qb1.x, qa1.y, qb1.y}, {qa1.z, qb1.z, qa1.w, qb1.w}};
                    uint4 w[NJ];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) w[j] = *reinterpret_cast<const uint4 *>(row + 2 * j * HD + 16 * x);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            uint32_t b0, b1;
                            e4m3x4_f16(k == 0 ? w[j].x : k == 1 ? w[j].y : k == 2 ? w[j].z : w[j].w, b0, b1);
                            mma_f16(sc[j], q[k], b0, b1);
                        }
                }
                if (piece == PAGE / KT - 1) {
                    next();
                    ++read;
                }
                const int live = min(max(left - piece * KT - CH * t, 0), CH);
                if constexpr (WIN) {
                    if (edge) {
                        const int key = key0 + piece * KT + CH * t;   // this lane's first
                        const uint32_t see[2] = {kv8_window_old(p, from[0], key), kv8_window_old(p, from[1], key)};
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!(see[e >> 1] >> (2 * j + (e & 1)) & 1u)) sc[j][e] = -INFINITY;
                    }
                }
                uint32_t w16[NJ][2];
                rows_softmax<NJ, NI>(sc, u.nqv > 8, live, kf, qf, vx, r, d, l, reach, o, w16);
                if (piece == 0) {   // V is the block behind K
                    const int vs = PAGE / KT == 1 ? out_slot : out_slot + 1 == NS ? 0 : out_slot + 1;
                    const uint32_t ph = PAGE / KT == 1 || out_slot + 1 < NS ? out_phase : out_phase ^ 1;
                    ok = __all_sync(0xffffffffu, bar_wait(bars + vs * 8, ph, c.status, LA_KV8_TIMEOUT));
                    if (!ok) break;
                    vblk = my_ring + vs * Lay::block;
                }
                const uint8_t *col = vblk + g * PAGE + piece * KT + CH * t;
                const bool whole = left >= PAGE;
                constexpr int NG = 4;   // output groups in flight together
                [[maybe_unused]] uint32_t odd = 0;   // an edge's bytes that are NaN
#pragma unroll
                for (int n0 = 0; n0 < NI; n0 += NG) {
                    uint32_t w[NG][CH / 4];
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        if constexpr (CH == 16) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(col + 8 * (n0 + n) * PAGE);
                            w[n][0] = x.x, w[n][1] = x.y, w[n][2] = x.z, w[n][3] = x.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2 *>(col + 8 * (n0 + n) * PAGE);
                            w[n][0] = x.x, w[n][1] = x.y;
                        }
                    }
                    if (!whole) {   // bytes behind the last token may be anything
#pragma unroll
                        for (int k = 0; k < CH / 4; ++k) {
                            const int b = live - 4 * k;
                            const uint32_t mask = b >= 4 ? 0xffffffffu : b <= 0 ? 0u : (1u << (8 * b)) - 1u;
#pragma unroll
                            for (int n = 0; n < NG; ++n) w[n][k] &= mask;
                        }
                    }
                    if constexpr (WIN) {
                        if (edge) {   // a NaN counts 0 here: a row that does not see it has a weight of 0
#pragma unroll
                            for (int k = 0; k < CH / 4; ++k)
#pragma unroll
                                for (int n = 0; n < NG; ++n) {
                                    const uint32_t nan = __vcmpeq4(w[n][k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                    odd |= nan;
                                    w[n][k] &= ~nan;
                                }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < CH / 4; ++k) {
                        const uint32_t a[4] = {w16[2 * k][0], w16[2 * k][1], w16[2 * k + 1][0], w16[2 * k + 1][1]};
#pragma unroll
                        for (int n = 0; n < NG; ++n) {
                            uint32_t b0, b1;
                            e4m3x4_f16(w[n][k], b0, b1);
                            mma_f16(o[n0 + n], a, b0, b1);
                        }
                    }
                }
                if constexpr (WIN) {
                    if (edge && __any_sync(0xffffffffu, odd != 0)) {   // and is added for the rows that do
#pragma unroll 1
                        for (int j = 0; j < min(left - piece * KT, KT); ++j) {
                            const int key = key0 + piece * KT + j;
                            const uint8_t *at = vblk + 2 * t * PAGE + piece * KT + j;
#pragma unroll
                            for (int i = 0; i < NI; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if ((at[(8 * i + (e & 1)) * PAGE] & 0x7f) == 0x7f && (key < p.sinks || key >= from[e >> 1])) o[i][e] = NAN;
                        }
                    }
                }
            }
            if (!ok) break;
            next();
            ++read;
        }
        if (!ok) {   // void: wait (bounded) for what is still in flight
            for (; read < issued; ++read) {
                bar_wait(bars + out_slot * 8, out_phase, c.status, LA_KV8_TIMEOUT);
                if (++out_slot == NS) {
                    out_slot = 0;
                    out_phase ^= 1;
                }
            }
        }

        // ---- join the warps at the largest r and d of those that saw a key, in warp order
        __syncthreads();   // the rings are free
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = warp * kRowsQ + g + 8 * h;
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (t == 0) sh_ml[at] = make_float4(r[h], l[h] == 0.f ? -INFINITY : d[h], l[h], 0.f);
            if (g + 8 * h < u.nqv) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    *reinterpret_cast<float2 *>(sh_o + at * (HD + 4) + 8 * i + 2 * t) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
            }
        }
        __syncthreads();
        const int slot = 2 * blockIdx.x + (u.begins ? 1 : 0);
#pragma unroll 1
        for (int i = tid; i < u.nqv * (HD / 4); i += 32 * NW) {
            const int r = i / (HD / 4), d = 4 * (i % (HD / 4));
            float R = -INFINITY, D = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 x = sh_ml[w * kRowsQ + r];
                R = fmaxf(R, x.x);
                D = fmaxf(D, x.y);
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 ml = sh_ml[w * kRowsQ + r];
                if (ml.z == 0.f) continue;   // saw no key
                const float fl = ex2(ml.x - R), f = ex2((ml.x - R) + (ml.y - D));
                const float4 x = *reinterpret_cast<const float4 *>(sh_o + (w * kRowsQ + r) * (HD + 4) + d);
                L += fl * ml.z;
                acc.x += f * x.x;
                acc.y += f * x.y;
                acc.z += f * x.z;
                acc.w += f * x.w;
            }
            if (u.all) {
                const float inv = L == 0.f ? 0.f : ex2(D) / L;
                const int qv = u.qv0 + r;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) + (sq.first + qv / p.gq) * p.a.out_stride +
                                     (head * p.gq + qv % p.gq) * HD + d;
                const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
                *reinterpret_cast<uint2 *>(out) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
            } else {
                *reinterpret_cast<float4 *>(p.part + (static_cast<long long>(slot) * kRowsQ + r) * HD + d) = acc;
                if (d == 0) *reinterpret_cast<float4 *>(p.part_ml + (static_cast<long long>(slot) * kRowsQ + r) * 4) = make_float4(R, D, L, 0.f);
            }
        }
        fence_proxy_async_smem();   // these accesses before the next unit's bulk copies into the same bytes
        __syncthreads();
    }
}

// ------------------------------------------------------------------ up to eight query vectors per KV head, with a window
// k_kv8_few: k_kv8_rows for 8 query vectors, with the operands changed over: keys
// are the rows of the first product (S^T = K Q^T, 16 keys x 8 vectors) and dims those of
// the second (O^T = V^T P^T), so none of a product's rows is empty, and the scores and O
// take half the registers.  That makes room for six warps in a block and 12 on an SM (with
// head_dim 128 and pages of 128 their rings leave room for one block), and for more of
// a unit's tiles at a time: short units are bound by what a tile takes one warp (about
// 2 us, most of it waiting for the instruction before).  Windows of 1024 and 4 first tokens, 64
// sequences, 64 heads over 8 KV heads, pages of 64: 32.9 us, k_kv8_rows 38.6 (4 warps and
// three blocks of ring each 34.0, three CTAs of 4 warps 37.2); 32 of them with pages of 128 27.2 and 35.9; 48
// sequences, head_dim 64, 12 heads over 4, window 700 11.1 and 16.3; one window of 4096 13.5 and
// 14.1.  Without a window k_kv8_rows stays: its sums have another order.
//   S^T: rows g and g + 8 of product b are keys CH (g >> 1) + 4 b + (g & 1) and 2 more of
//        the piece; lane (g, t) reads HD / 4 consecutive bytes of theirs, and has the
//        scores of vectors 2 t and 2 t + 1.
//   P^T: packed pairs turned by movmatrix: lane (g, t) has vector g's weights of keys
//        CH t + 4 b .. + 3, whose bytes of V are those that it reads for dims 16 n + g, + 8.
constexpr int kFewQ = 8;

template <int HD, int PAGE>
struct Few {
    static constexpr int block = HD * PAGE;
    static constexpr int warps = 6;
    static constexpr int slots = block >= 8192 ? 2 : 4;
    static constexpr int per_sm = block > 8192 ? 1 : 2;
    static constexpr int ring = block * slots * warps;
    static constexpr int join = warps * kFewQ * (HD + 4) * 4;
    static constexpr int q_row = HD * 2 + 16;                                   // q in fp16
    static constexpr int q_off = ring > join ? ring : join;
    static constexpr int qf_off = q_off + kFewQ * q_row;
    static constexpr int ml_off = qf_off + kFewQ * 4;
    static constexpr int reach_off = ml_off + warps * kFewQ * 16;
    static constexpr int bar_off = reach_off + warps * kFewQ * 4;
    static constexpr int sum_off = bar_off + warps * slots * 8;
    static constexpr int tiles_off = sum_off + warps * 8;
    static size_t bytes(int n_seqs) { return tiles_off + (static_cast<size_t>(n_seqs) + 1) * 8; }
};

// The 8 x 8 matrix of 16-bit numbers whose rows the warp's lanes hold in pairs, turned.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int HD, int PAGE>
__global__ void __launch_bounds__(32 * Few<HD, PAGE>::warps, Few<HD, PAGE>::per_sm) k_kv8_few(const __grid_constant__ Kv8Args p) {
    using Lay = Few<HD, PAGE>;
    constexpr int ND = HD / 16;                   // 16-dim groups
    constexpr int KT = PAGE < 64 ? PAGE : 64;     // keys per piece
    constexpr int CH = KT / 4, NB = KT / 16;      // of them, one lane's bytes of V; products
    constexpr int NS = Lay::slots, NW = Lay::warps;
    extern __shared__ __align__(128) uint8_t smem[];
    float4 *sh_ml = reinterpret_cast<float4 *>(smem + Lay::ml_off);  // [warp][8] r, d, l
    float *sh_o = reinterpret_cast<float *>(smem);                   // [warp][8][HD + 4], over the ring
    float *sh_qf = reinterpret_cast<float *>(smem + Lay::qf_off);
    long long *tiles = reinterpret_cast<long long *>(smem + Lay::tiles_off);
    pdl_trigger();
    const la_kv8_cache &c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * NS * Lay::block, bars = smem_u32(smem + Lay::bar_off) + warp * NS * 8;
    const uint8_t *my_ring = smem + warp * NS * Lay::block;
    float *reach = reinterpret_cast<float *>(smem + Lay::reach_off) + warp * kFewQ + 2 * t;   // of this lane's two vectors
    if (lane < NS) mbar_init(bars + lane * 8, 1);
    fence_barrier_init();
    pdl_wait();
    kv8_plan<true>(p, tiles, reinterpret_cast<long long *>(smem + Lay::sum_off));
    Kv8Walk walk = kv8_walk<true>(p, tiles);
    Kv8Piece u;
    int in_slot = 0, out_slot = 0;   // ring positions: the next block to load, the next to read
    uint32_t out_phase = 0;
    bool ok = true;                  // false once a wait gave up: this warp loads nothing more
    bool noted = p.whole;

    for (;;) {
        const bool any = kv8_next<true>(p, tiles, walk, u);
        auto note = [&]() {
            if (!noted && tid == 0) kv8_note(p, tiles, any, u);
            noted = true;
        };
        if (!any) {
            note();
            break;
        }
        const Kv8Seq sq = u.sq;
        const int page0 = u.k0 + warp, s = u.s, head = u.head;
        const int new0 = NW - 1 - warp;   // new rows begin with the last warp, which has no more tiles than another
        const int nc = ok && page0 < u.k1 ? (u.k1 - page0 + NW - 1) / NW : 0;
        // q and the first new row before the copies (see k_kv8_rows); 16 threads of the first four warps a vector
        const int q_mine = tid >> 4, q_part = tid & 15;
        uint4 q_raw = make_uint4(0, 0, 0, 0);
        if (q_mine < u.nqv && 8 * q_part < HD) {
            const int qv = u.qv0 + q_mine, its = qv / p.gq;
            q_raw = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.a.q) + (sq.first + its) * p.a.q_stride + (head * p.gq + qv - its * p.gq) * HD + 8 * q_part);
        }
        uint4 kw[HD / 64];          // this lane's HD / 8 dims of a new key
        uint16_t vw[2 * ND];        // and its dims 16 n + g, + 8 of the value
        auto load_new = [&](int j) {
            const uint4 *kj = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.a.k) + (sq.first + j) * p.a.k_stride + head * HD + g * (HD / 8));
            const uint16_t *vj = reinterpret_cast<const uint16_t *>(static_cast<const __nv_bfloat16 *>(p.a.v) + (sq.first + j) * p.a.v_stride + head * HD) + g;
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) kw[i] = kj[i];
#pragma unroll
            for (int i = 0; i < 2 * ND; ++i) vw[i] = vj[8 * i];
        };
        const int n_new = u.begins && p.a.k ? sq.rows : 0;
        if (new0 < n_new) load_new(new0);
        // Block 2 i is K of tile i, block 2 i + 1 its V: as in k_kv8_rows
        int my_page = -1, last_page = -1, issued = 0;
        float my_kf = 0.f, last_kf = 0.f, my_vs = 0.f, last_vs = 0.f;
        auto issue = [&]() {
            const int i = issued >> 1;
            if ((issued & 63) == 0) {
                last_page = my_page;
                last_vs = my_vs;
                last_kf = my_kf;
                my_page = i + lane < nc ? kv8_page(c, s, kv8_tile<true>(sq, page0 + NW * (i + lane))) : -1;
                const long long blk = kv8_block(c, p.a.layer, max(my_page, 0), head);
                my_kf = c.k_scale[blk];
                my_vs = c.v_scale[blk];
            }
            const int pg = __shfl_sync(0xffffffffu, my_page, i & 31);
            if (lane == 0) {
                const uint32_t bar = bars + in_slot * 8;
                if (pg >= 0) {
                    mbar_arrive_expect_tx(bar, Lay::block);
                    bulk_load(ring + in_slot * Lay::block,
                              static_cast<const uint8_t *>(issued & 1 ? c.v : c.k) + kv8_block(c, p.a.layer, pg, head) * Lay::block, Lay::block, bar);
                } else {
                    mbar_arrive_expect_tx(bar, 0);   // a page number outside the cache: nothing is loaded, no key counts
                }
            }
            __syncwarp();
            in_slot = in_slot + 1 == NS ? 0 : in_slot + 1;
            ++issued;
        };
#pragma unroll 1
        while (issued < min(NS, 2 * nc)) issue();
        note();   // while the first copies are on their way

        // q as fp16, each vector scaled by a power of two to fit
        if (q_mine < kFewQ) {   // whole warps
            const uint4 w = q_raw;
            uint32_t top = most2(most2(most2(most2(0u, w.x), w.y), w.z), w.w);
#pragma unroll
            for (int k = 1; k < 16; k <<= 1) top = most2(top, __shfl_xor_sync(0xffffffffu, top, k));
            const int qx = fit_pair(top);
            const float f = power_of(-qx);
            if (8 * q_part < HD)
                *reinterpret_cast<uint4 *>(smem + Lay::q_off + q_mine * Lay::q_row + 16 * q_part) = make_uint4(scaled_f16(w.x, f), scaled_f16(w.y, f), scaled_f16(w.z, f), scaled_f16(w.w, f));
            if (q_part == 0) sh_qf[q_mine] = factor(power_of(qx), p.scale_log2);
        }
        __syncthreads();
        uint32_t q[HD / 8];   // the first product's operand: vector g, dims t HD / 4 on
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) {
            const uint4 x = *reinterpret_cast<const uint4 *>(smem + Lay::q_off + g * Lay::q_row + t * (HD / 2) + 16 * i);
            q[4 * i] = x.x, q[4 * i + 1] = x.y, q[4 * i + 2] = x.z, q[4 * i + 3] = x.w;
        }
        const float qf[2] = {sh_qf[2 * t], sh_qf[2 * t + 1]};

        // Of vectors 2 t and 2 t + 1
        float r[2] = {-INFINITY, -INFINITY}, d[2] = {kRowsUnit, kRowsUnit}, l[2] = {0.f, 0.f};
        float far[2] = {-INFINITY, -INFINITY};   // reach of O, of the new rows
        float o[ND][4];                          // dims 16 n + g (0, 1) and + 8 (2, 3)
#pragma unroll
        for (int i = 0; i < ND; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        int row[2], from[2];                     // their new rows, and where those' windows begin
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int mine = 2 * t + e < u.nqv ? (u.qv0 + 2 * t + e) / p.gq : -1, there = max(mine, 0);
            row[e] = mine;
            from[e] = sq.len + (p.a.vis ? kv8_seen(p, sq.first, sq.rows, there) : p.a.k ? there + 1 : 0) - p.window;
        }

        // ---- new rows, in the piece that begins the unit: one key at a time
        if (n_new > 0) {
#pragma unroll 1
            for (int j = new0; j < n_new; j += NW) {
                bool see[2];
                float z[2] = {0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (p.a.vis) see[e] = row[e] >= 0 && (kv8_window_new(p, sq.first, sq.rows, sq.len, row[e], j & ~31) >> (j & 31) & 1u);
                    else see[e] = j <= row[e] && (j < p.sinks - sq.len || j > row[e] - p.window);
                    const uint8_t *at = smem + Lay::q_off + (2 * t + e) * Lay::q_row + g * (HD / 4);
#pragma unroll
                    for (int i = 0; i < HD / 64; ++i) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(at + 16 * i);
                        const uint32_t x[4] = {kw[i].x, kw[i].y, kw[i].z, kw[i].w}, y[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 qa = __half22float2(*reinterpret_cast<const __half2 *>(&y[k]));
                            z[e] = fmaf(qa.x, bf16_bits(x[k] & 0xffffu), fmaf(qa.y, __uint_as_float(x[k] & 0xffff0000u), z[e]));
                        }
                    }
                }
                uint32_t top = 0;   // V's largest magnitude: what it reaches in O may raise d
#pragma unroll
                for (int i = 0; i < 2 * ND; ++i) top = max(top, vw[i] & 0x7fffu);
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) {
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, k));
                    z[0] += __shfl_xor_sync(0xffffffffu, z[0], k);
                    z[1] += __shfl_xor_sync(0xffffffffu, z[1], k);
                }
                const int ve = exponent_of(bf16_bits(top));   // 128: a NaN or infinity, which hides its neighbours' size
                float w[2], alpha[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = see[e] ? z[e] * qf[e] : -INFINITY, nr = x > r[e] ? ceilf(x) : r[e], base = nr == -INFINITY ? 0.f : nr;
                    const float fl = ex2(r[e] - base);
                    far[e] = fmaxf(far[e] - (base - r[e]), (x - base) + static_cast<float>(ve == 128 ? 0 : ve + 1));
                    const float nd = fmaxf(d[e], far[e] - kSpan);
                    alpha[e] = fl * ex2(d[e] - nd);
                    r[e] = nr;
                    d[e] = nd;
                    l[e] = l[e] * fl + ex2(x - base);
                    w[e] = ex2((x - base) - nd);
                }
#pragma unroll
                for (int i = 0; i < ND; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float v = bf16_bits(vw[2 * i + h]);
#pragma unroll
                        for (int e = 0; e < 2; ++e)   // what a row does not see never meets it, not even times 0
                            o[i][2 * h + e] = fmaf(w[e], see[e] ? v : 0.f, o[i][2 * h + e] * alpha[e]);
                    }
                if (j + NW < n_new) load_new(j + NW);
            }
            // Every lane g has added the key: l is summed over them below.
            if (g != 0) l[0] = l[1] = 0.f;
        }
        reach[0] = far[0];
        reach[1] = far[1];

        // ---- cached tokens
        auto landed = [&]() {   // the next block to read is there
            ok = __all_sync(0xffffffffu, bar_wait(bars + out_slot * 8, out_phase, c.status, LA_KV8_TIMEOUT));
            return ok;
        };
        auto next = [&]() {     // it has been read: its slot takes the next block to load
            __syncwarp();
            if (++out_slot == NS) {
                out_slot = 0;
                out_phase ^= 1;
            }
            if (issued < 2 * nc) issue();
        };
        int read = 0;           // blocks read
#pragma unroll 1
        for (int i = 0; i < nc; ++i) {
            if (!landed()) break;
            const bool old = i >> 5 != (issued - 1) >> 6;   // issue() is in the next 32 tiles already
            const int pg = __shfl_sync(0xffffffffu, old ? last_page : my_page, i & 31);
            const float kf_ = __shfl_sync(0xffffffffu, old ? last_kf : my_kf, i & 31), kf = pg < 0 ? 1.f : kf_;
            const float vs_ = __shfl_sync(0xffffffffu, old ? last_vs : my_vs, i & 31);
            const float v = static_cast<float>(pg < 0 ? 0 : exponent_of(vs_));
            const int key0 = kv8_tile<true>(sq, page0 + NW * i) * PAGE, left = pg < 0 ? 0 : sq.len - key0;   // keys of this page that count
            const bool edge = kv8_edge(p, sq, (u.qv0 + u.nqv - 1) / p.gq, key0, PAGE);
            const uint8_t *kblk = my_ring + out_slot * Lay::block, *vblk = nullptr;
#pragma unroll 1
            for (int piece = 0; piece < PAGE / KT; ++piece) {
                float sc[NB][4];
#pragma unroll
                for (int b = 0; b < NB; ++b) sc[b][0] = sc[b][1] = sc[b][2] = sc[b][3] = 0.f;
                const int mine = CH * (g >> 1) + (g & 1);   // this lane's first key of the piece
                const uint8_t *krow = kblk + (piece * KT + mine) * HD + t * (HD / 4);
#pragma unroll
                for (int x = 0; x < HD / 64; ++x) {   // steps outside, products inside: their sums do not wait on one another
                    uint4 w[NB][2];
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int h = 0; h < 2; ++h) w[b][h] = *reinterpret_cast<const uint4 *>(krow + (4 * b + 2 * h) * HD + 16 * x);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            auto word = [&](const uint4 &y) { return k == 0 ? y.x : k == 1 ? y.y : k == 2 ? y.z : y.w; };
                            uint32_t a[4];
                            e4m3x4_f16(word(w[b][0]), a[0], a[2]);
                            e4m3x4_f16(word(w[b][1]), a[1], a[3]);
                            mma_f16(sc[b], a, q[8 * x + 2 * k], q[8 * x + 2 * k + 1]);
                        }
                }
                if (piece == PAGE / KT - 1) {
                    next();
                    ++read;
                }
                const int live = left - piece * KT;   // keys of the piece that count
                if (live < KT || edge) {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int at = mine + 4 * b + 2 * (e >> 1), key = key0 + piece * KT + at;
                            if (at >= live || (key >= p.sinks && key < from[e & 1])) sc[b][e] = -INFINITY;   // factors are positive
                        }
                }
                // Online softmax, as in k_kv8_rows
                float f[2], nr[2] = {r[0], r[1]}, nd[2] = {d[0], d[1]};
                bool change = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f[e] = factor(kf, qf[e]);
                    float mx = -INFINITY;
#pragma unroll
                    for (int b = 0; b < NB; ++b) mx = fmaxf(mx, fmaxf(sc[b][e], sc[b][2 + e]));
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
                    const float z = mx * f[e];
                    const bool grow = r[e] == -INFINITY ? z > -INFINITY : z - r[e] > kLazy;
                    const bool shift = z > -INFINITY && (v - d[e] > kUnitHigh || v - d[e] < kUnitLow);
                    if (grow) nr[e] = ceilf(z);
                    if (shift) nd[e] = fmaxf(v - kUnit, fmaxf(reach[e], d[e] + kReach) - (grow ? nr[e] - r[e] : 0.f) - kSpan);
                    change |= grow || shift;
                }
                if (__any_sync(0xffffffffu, change)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool grow = nr[e] != r[e];
                        const float to = fmaxf(reach[e], d[e] + kReach) - (grow ? nr[e] - r[e] : 0.f);
                        const float fl = grow ? ex2(r[e] - nr[e]) : 1.f, fo = fl * ex2(d[e] - nd[e]);
                        __syncwarp();
                        reach[e] = to;   // the lanes of a vector write the same
                        __syncwarp();
                        r[e] = nr[e];
                        d[e] = nd[e];
                        l[e] *= fl;
#pragma unroll
                        for (int n = 0; n < ND; ++n) {
                            o[n][e] *= fo;
                            o[n][2 + e] *= fo;
                        }
                    }
                }
                uint32_t w16[NB][2];   // the second product's operand
                float off[2], sum[2] = {0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 2; ++e) off[e] = (v - d[e]) - (r[e] == -INFINITY ? 0.f : r[e]);
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float x = ex2(fmaf(sc[b][2 * h], f[0], off[0])), y = ex2(fmaf(sc[b][2 * h + 1], f[1], off[1]));
                        sum[0] += x;
                        sum[1] += y;
                        w16[b][h] = turned(pack_f16(x, y));
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e) l[e] += sum[e] * ex2(d[e] - v);
                if (piece == 0) {   // V is the block behind K
                    const int vs = PAGE / KT == 1 ? out_slot : out_slot + 1 == NS ? 0 : out_slot + 1;
                    const uint32_t ph = PAGE / KT == 1 || out_slot + 1 < NS ? out_phase : out_phase ^ 1;
                    ok = __all_sync(0xffffffffu, bar_wait(bars + vs * 8, ph, c.status, LA_KV8_TIMEOUT));
                    if (!ok) break;
                    vblk = my_ring + vs * Lay::block;
                }
                const uint8_t *col = vblk + g * PAGE + piece * KT + CH * t;
                const int kept = min(max(live - CH * t, 0), CH);   // of this lane's bytes
                constexpr int NG = 4;   // output groups in flight together
                uint32_t odd = 0;       // an edge's bytes that are NaN
#pragma unroll
                for (int n0 = 0; n0 < ND; n0 += NG) {
                    uint32_t w[NG][2][NB];
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint8_t *at = col + (16 * (n0 + n) + 8 * h) * PAGE;
                            if constexpr (NB == 4) {
                                const uint4 x = *reinterpret_cast<const uint4 *>(at);
                                w[n][h][0] = x.x, w[n][h][1] = x.y, w[n][h][2] = x.z, w[n][h][3] = x.w;
                            } else {
                                const uint2 x = *reinterpret_cast<const uint2 *>(at);
                                w[n][h][0] = x.x, w[n][h][1] = x.y;
                            }
                        }
                    if (live < KT) {   // bytes behind the last token may be anything
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const int k = kept - 4 * b;
                            const uint32_t mask = k >= 4 ? 0xffffffffu : k <= 0 ? 0u : (1u << (8 * k)) - 1u;
#pragma unroll
                            for (int n = 0; n < NG; ++n) w[n][0][b] &= mask, w[n][1][b] &= mask;
                        }
                    }
                    if (edge) {   // a NaN counts 0 here: a row that does not see it has a weight of 0
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int n = 0; n < NG; ++n)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const uint32_t nan = __vcmpeq4(w[n][h][b] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                    odd |= nan;
                                    w[n][h][b] &= ~nan;
                                }
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int n = 0; n < NG; ++n) {
                            uint32_t a[4];
                            e4m3x4_f16(w[n][0][b], a[0], a[2]);
                            e4m3x4_f16(w[n][1][b], a[1], a[3]);
                            mma_f16(o[n0 + n], a, w16[b][0], w16[b][1]);
                        }
                }
                if (edge && __any_sync(0xffffffffu, odd != 0)) {   // and is added for the rows that do
#pragma unroll 1
                    for (int j = 0; j < min(live, KT); ++j) {
                        const int key = key0 + piece * KT + j;
                        const uint8_t *at = vblk + g * PAGE + piece * KT + j;
#pragma unroll
                        for (int n = 0; n < ND; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if ((at[(16 * n + 8 * (e >> 1)) * PAGE] & 0x7f) == 0x7f && (key < p.sinks || key >= from[e & 1])) o[n][e] = NAN;
                    }
                }
            }
            if (!ok) break;
            next();
            ++read;
        }
        if (!ok) {   // void: wait (bounded) for what is still in flight
            for (; read < issued; ++read) {
                bar_wait(bars + out_slot * 8, out_phase, c.status, LA_KV8_TIMEOUT);
                if (++out_slot == NS) {
                    out_slot = 0;
                    out_phase ^= 1;
                }
            }
        }

        // ---- join the warps at the largest r and d of those that saw a key, in warp order
        __syncthreads();   // the rings are free
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int at = warp * kFewQ + 2 * t + e;
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], k);
            if (g == 0) sh_ml[at] = make_float4(r[e], l[e] == 0.f ? -INFINITY : d[e], l[e], 0.f);
#pragma unroll
            for (int n = 0; n < ND; ++n) {
                sh_o[at * (HD + 4) + 16 * n + g] = o[n][e];
                sh_o[at * (HD + 4) + 16 * n + 8 + g] = o[n][2 + e];
            }
        }
        __syncthreads();
        const int slot = 2 * blockIdx.x + (u.begins ? 1 : 0);
#pragma unroll 1
        for (int i = tid; i < u.nqv * (HD / 4); i += 32 * NW) {
            const int qi = i / (HD / 4), dim = 4 * (i % (HD / 4));
            float R = -INFINITY, D = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 x = sh_ml[w * kFewQ + qi];
                R = fmaxf(R, x.x);
                D = fmaxf(D, x.y);
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 ml = sh_ml[w * kFewQ + qi];
                if (ml.z == 0.f) continue;   // saw no key
                const float fl = ex2(ml.x - R), fw = ex2((ml.x - R) + (ml.y - D));
                const float4 x = *reinterpret_cast<const float4 *>(sh_o + (w * kFewQ + qi) * (HD + 4) + dim);
                L += fl * ml.z;
                acc.x += fw * x.x;
                acc.y += fw * x.y;
                acc.z += fw * x.z;
                acc.w += fw * x.w;
            }
            if (u.all) {
                const float inv = L == 0.f ? 0.f : ex2(D) / L;
                const int qv = u.qv0 + qi;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) + (sq.first + qv / p.gq) * p.a.out_stride + (head * p.gq + qv % p.gq) * HD + dim;
                const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
                *reinterpret_cast<uint2 *>(out) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
            } else {
                *reinterpret_cast<float4 *>(p.part + (static_cast<long long>(slot) * kFewQ + qi) * HD + dim) = acc;
                if (dim == 0) *reinterpret_cast<float4 *>(p.part_ml + (static_cast<long long>(slot) * kFewQ + qi) * 4) = make_float4(R, D, L, 0.f);
            }
        }
        fence_proxy_async_smem();   // these accesses before the next unit's bulk copies into the same bytes
        __syncthreads();
    }
}

// ------------------------------------------------------------------ many query vectors per KV head
// k_kv8_tiles: 128 query vectors per unit and 128 keys per tile on the
// tcgen05 tensor cores.  With more than a few query vectors per KV head the
// products and the softmax, not the bytes, bound the attention.
//   warps 8..13  turn a tile's e4m3 bytes of K (or the new rows' bf16) into an
//                fp16 operand in shared memory (128-byte swizzle), [128 keys x
//                HD], then the same for V^T [HD x 128 keys] of the tile before;
//                two buffers each
//   warp 14      brings the bytes into a ring in shared memory, a page's block of
//                K or V by one bulk copy
//   warp 15      issues S = Q K^T of tile i + 1, then O += P V (P from tensor
//                memory) of tile i
//   warps 0..3   softmax of the even tiles, warps 4..7 of the odd ones, each
//                thread a query vector; P replaces S in tensor memory.  Two
//                groups, since one alone waits for tensor memory half of the
//                time: 2.4 us per tile.
// What bounds a tile (1.45 us; its products take 0.55 us) are the instructions of
// these warps, which share four schedulers: anything that waits must not poll
// (the softmax and the products polling: 123.4 us against 118.0 for 256 rows over
// 16k tokens, 8 KV heads), the bytes come by bulk copies (loads to registers by
// seven operand warps: 131.3), and S is read 32 columns at a time (16: 136.0,
// 64: 134.3, both polling).
// The groups have an O each in tensor memory, added at the end, with r and d of
// its own; both follow lazily, so O is rarely read back.  A tile has one d:
// what its page of the largest scale asks for.  Groups of 32 keys of pages that
// are more than 2^kNear below it are left out of the product and added to O in
// fp32 (far_group).  Units are split and joined like those of k_kv8_rows.
constexpr int kTileQ = 128, kTileK = 128;
constexpr int kOpWarps = 6, kLoadWarp = 8 + kOpWarps, kMmaWarp = kLoadWarp + 1;
constexpr int kTileThreads = 32 * (kMmaWarp + 1);   // 16 warps: 4 to a quarter of an SM, 128 registers a thread
// u of the tile's largest scale: with kNear, u of every group in the product is kUnitLow or more.
constexpr int kNear = 6;
constexpr float kTopLow = kUnitLow + kNear, kTop = 4.f;

template <int HD>
struct Tiles {
    static constexpr uint32_t k_block = kTileK * 128;              // [128 keys x 64 dims]
    static constexpr uint32_t v_block = HD * 128;                  // [HD dims x 64 keys]
    static constexpr uint32_t k_bytes = HD / 64 * k_block, v_bytes = 2 * v_block;
    static constexpr uint32_t k_off = 0, v_off = 2 * k_bytes;      // two buffers each
    static constexpr uint32_t q_off = v_off + 2 * v_bytes;         // Q [128 x HD]
    // The cache's bytes as they come: stages of K or V of a tile, in a ring
    static constexpr int raw_slots = HD == 128 ? 3 : 6;
    static constexpr uint32_t raw_off = q_off + k_bytes, raw_bytes = kTileK * HD;
    static constexpr uint32_t head_off = raw_off + raw_slots * raw_bytes;   // [raw_slots] Kv8Meta of the bytes in the ring
    static constexpr uint32_t meta_off = head_off + raw_slots * 64;         // [4] Kv8Meta of the last tiles
    static constexpr uint32_t exp_off = meta_off + 4 * 64;         // [4] Kv8Exps of the last tiles, where those are kMixed
    static constexpr uint32_t red_off = exp_off + 4 * 256;         // [2][2][8] largest and least of the new rows' tile, by warp
    static constexpr uint32_t qf_off = red_off + 128;              // [128] factors on the rows' scores
    static constexpr uint32_t odd_off = qf_off + kTileQ * 4;       // [2 groups]
    static constexpr uint32_t bar_off = odd_off + 16;
    static constexpr uint32_t tiles_off = bar_off + 40 * 8 + (kMmaWarp + 1) * 8;
    static constexpr size_t tiles_end(int n_seqs) { return tiles_off + (static_cast<size_t>(n_seqs) + 1) * 8; }
    // With a window: barriers [4] and flags [4][kOpWarps] of NaN in cached V, by unit.
    static constexpr size_t win_bytes = 4 * 8 + 4 * kOpWarps * 4;
    static constexpr size_t bytes(int n_seqs, bool win) { return tiles_end(n_seqs) + (win ? win_bytes : 0); }
    static_assert(tiles_off + (LA_KV8_MAX_SEQS + 1) * 8 + win_bytes <= 227 * 1024, "shared memory of a block");
};
// TMEM columns: S of even and odd tiles (P over their first halves; behind it,
// once a group is through with a unit, its rows' r, d and sum), then their O.
constexpr uint32_t kColS = 0, kColO = 256, kColAll = 512;

struct Kv8Meta {
    float kf[4];   // per 32 keys: factor of K, exponent of V, keys that count
    int vx[4];
    int live[4];
    int flags;     // kOddV, kMixed, kFar << k
    int top;       // largest vx of the groups that have keys (new rows: 5 more, as their fp16 values are 2^6 times a page's)
    int pad[2];
};
static_assert(sizeof(Kv8Meta) == 64, "layout");
constexpr int kOddV = 1;    // new rows: V holds a NaN or infinity
constexpr int kMixed = 2;   // new rows: each has exponents of its own
constexpr int kFar = 4;     // << k: group k's page has a V scale more than 2^kNear below `top`
// A tile's new rows share one factor of K and one of V (the largest value's)
// where all of their 8-dim pieces that are not zero reach within 2^kSpread of
// it: values keep at least 15 + 24 - kSpread = 23 bits below their piece's
// largest.  Else each row has its own, or a huge row would leave nothing of the
// others, for query vectors too that do not see it.  The code for that is apart:
// in line it cost every call 7 us (121 rows of 32 heads over 2k tokens, 31.6 us; so 32.7).
constexpr int kSpread = 16;
struct Kv8Exps {
    signed char k[kTileK], v[kTileK];   // of fit_f16, -60 .. 113
};
static_assert(sizeof(Kv8Exps) == 256, "layout");

// kind::f16 with fp16 operands, fp32 accumulation.
__device__ constexpr uint32_t idesc_f16(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2_f32(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void mbar_arrive_one(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Waits for this thread's loads from tensor memory; v is what they wrote, which nothing may read before.
template <int N>
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[N]) {
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}

// Four columns of this thread's row of tensor memory.
__device__ __forceinline__ void tmem_st_four(uint32_t at, float a, float b, float c) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %3};" ::"r"(at), "f"(a), "f"(b), "f"(c) : "memory");
}
__device__ __forceinline__ float4 tmem_ld_four(uint32_t at) {
    uint32_t v[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at));
    tmem_ld_wait_for(v);
    return make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]));
}

// 16 e4m3 bytes as 32 bytes of fp16.
__device__ __forceinline__ void e4m3x16_f16(const uint4 &w, uint4 &a, uint4 &b) {
    e4m3x4_f16(w.x, a.x, a.y);
    e4m3x4_f16(w.y, a.z, a.w);
    e4m3x4_f16(w.z, b.x, b.y);
    e4m3x4_f16(w.w, b.z, b.w);
}
__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared(uint32_t at, const uint4 &v) { st_shared_u32x4(at, v.x, v.y, v.z, v.w); }

// ---- new rows that are many binades apart (kMixed): code apart from the roles'
// Largest finite magnitude of 8 bf16 values, as pairs.
__device__ __noinline__ uint32_t finite_top(uint4 x) {
    auto tame = [](uint32_t w) { return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0x7fffu) | ((w >> 16 & 0x7f80u) == 0x7f80u ? 0u : w & 0x7fff0000u); };
    return most2(most2(most2(most2(0u, tame(x.x)), tame(x.y)), tame(x.z)), tame(x.w));
}

// Exponents of a tile's rows, and K's rows turned into fp16 in place.  Thread t
// of the operand warps has the 16-byte pieces t, t + 32 kOpWarps, ..., as when K
// was copied: a row's pieces belong to neighbouring lanes of one warp.
template <int HD>
__device__ __noinline__ void mixed_rows(uint32_t sk, uint32_t k_block, const __nv_bfloat16 *vn, int64_t v_stride, int nkeys, int t, Kv8Exps *ex) {
    constexpr int C8 = HD / 8;
    auto fit_row = [](uint4 x) {
        uint32_t top = finite_top(x);
#pragma unroll
        for (int o = 1; o < C8; o <<= 1) top = most2(top, __shfl_xor_sync(0xffffffffu, top, o));
        return fit_pair(top);
    };
#pragma unroll 1
    for (int i = t; i < kTileK * C8; i += 32 * kOpWarps) {   // whole warps
        const int r = i / C8, c = i % C8;
        const uint32_t at = sk + (c >> 3) * k_block + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        const uint4 x = ld_shared(at), y = r < nkeys ? *reinterpret_cast<const uint4 *>(vn + r * v_stride + 8 * c) : make_uint4(0, 0, 0, 0);
        const int kx = fit_row(x), vx = fit_row(y);
        const float f = power_of(-kx);
        st_shared_u32x4(at, scaled_f16(x.x, f), scaled_f16(x.y, f), scaled_f16(x.z, f), scaled_f16(x.w, f));
        if (c == 0) {
            ex->k[r] = static_cast<signed char>(kx);
            ex->v[r] = static_cast<signed char>(vx);
        }
    }
}

// Such rows' V^T operand: 8 dims of a row at a time.  NaN and infinities count 0, as in the roles' code.
template <int HD>
__device__ __noinline__ void mixed_v(uint32_t sv, uint32_t v_block, const __nv_bfloat16 *vn, int64_t v_stride, int nkeys, int t, const signed char *vx) {
#pragma unroll 1
    for (int j = t; j < kTileK * (HD / 8); j += 32 * kOpWarps) {
        const int r = j % kTileK, d = 8 * (j / kTileK);
        const uint4 x = r < nkeys ? *reinterpret_cast<const uint4 *>(vn + r * v_stride + d) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        const float f = power_of(-vx[r]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float y = bf16_bits(k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xffffu);
            const __half h = __float2half_rn(is_finite(y) ? y * f : 0.f);
            const uint32_t at = sv + (r >> 6) * v_block + (d + k) * 128 + ((((r >> 3) & 7) ^ k) << 4) + (r & 7) * 2;
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(*reinterpret_cast<const uint16_t *>(&h)) : "memory");
        }
    }
}

// Which of new rows key .. key + 31 row `row` of a sequence (-1: none) sees.
template <bool WIN>
__device__ __forceinline__ uint32_t new_rows_seen(const Kv8Args &p, const Kv8Seq &q, int row, int key) {
    const int first = q.first;
    if (row < 0) return 0u;
    if constexpr (WIN) return kv8_window_new(p, first, q.rows, q.len, row, key);
    if (p.a.vis) return key < 256 ? p.a.vis[(static_cast<long long>(first) + row) * 8 + key / 32] : 0u;
    return row >= key + 31 ? 0xffffffffu : row < key ? 0u : (2u << (row - key)) - 1u;
}

// A row's state, and what the softmax seldom asks for.
struct Kv8Row {
    float r, d, l, qf;
    float reach, at;             // of O, relative to r when that was `at`
    float own_r, own_d, own_l;   // behind a tile of own_scores
    // The softmax's other values while begin_tile runs.  Kept in registers over the
    // call they would be spilled in every tile (256 rows over 16k tokens 123 us, so 115).
    int grp, row, units, it, first, end, i, kt, myrow, myhead;
    uint32_t lanes, ts, to;
    bool in, odd;
    int from;   // where the row's window begins
};
// O's reach relative to r, where r has grown from s.r.
__device__ __forceinline__ float reach_now(const Kv8Row &s, float r) { return fmaxf(s.reach - (r - s.at), s.d + kReach - (r - s.r)); }

// O *= f, for this thread's row.
template <int HD>
__device__ __forceinline__ void scale_o(uint32_t to, float f) {
#pragma unroll 1
    for (int q = 0; q < HD / 16; ++q) {
        uint32_t o[16];
        tmem_ld_32x32b_x16(to + 16 * q, o);
        tmem_ld_wait_for(o);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st_32x32b_x16(to + 16 * q, o);
    }
    tmem_st_wait();
}

// A tile of new rows with exponents of their own (kMixed), or which O's reach keeps
// from having the d that it asks for: turns this thread's row of S, at ts, into
// the exponents of its weights, z_j - r + vx_j - d (-infinity for keys that it
// does not see), with r and d as this tile's largest ones have them.  s.own_*
// has r, d and l behind this tile; for the loop over its groups the scores are
// final (r 0, u 0, a factor of 1), and l < 0 says so.
template <int HD, bool WIN>
__device__ __forceinline__ void own_scores(const Kv8Args &p, const Kv8Piece &u, uint32_t ts, uint32_t to, const Kv8Meta &mt, const Kv8Exps &ex, int key0,
                                           int row, bool has_o, Kv8Row &s) {
    const int nkeys = min(u.sq.rows - key0, kTileK);
    const bool mixed = mt.flags & kMixed;
    const float was = s.r;
    float zmax = -INFINITY, xmax = -INFINITY, sum = 0.f, nr = was, nd = s.d;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {   // 16 keys at a time
            uint32_t v[16];
            tmem_ld_32x32b_x16(ts + 16 * k, v);
            tmem_ld_wait_for(v);
            if (pass == 0) {
                const int live = nkeys - 16 * k;
                const uint32_t see = (live <= 0 ? 0u : live >= 16 ? 0xffffu : (1u << live) - 1u) & new_rows_seen<WIN>(p, u.sq, row, key0 + 32 * (k >> 1)) >> 16 * (k & 1);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float z = see >> e & 1u ? __uint_as_float(v[e]) * factor(mixed ? power_of(ex.k[16 * k + e]) : mt.kf[0], s.qf) : -INFINITY;
                    zmax = fmaxf(zmax, z);
                    v[e] = __float_as_uint(z);
                }
            } else if (pass == 1) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float y = __uint_as_float(v[e]) - (nr == -INFINITY ? 0.f : nr), x = y + static_cast<float>(mixed ? ex.v[16 * k + e] : mt.vx[0]);
                    sum += ex2(y);
                    xmax = fmaxf(xmax, x);
                    v[e] = __float_as_uint(x);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) - nd);
            }
            tmem_st_32x32b_x16(ts + 16 * k, v);
        }
        tmem_st_wait();
        if (pass == 0 && zmax > was) nr = ceilf(zmax);
        if (pass == 1 && xmax > -INFINITY) {
            const float reach = was == -INFINITY ? -INFINITY : reach_now(s, nr);
            if (was == -INFINITY || xmax - nd > kUnitHigh || xmax - nd < 0.f) nd = fmaxf(ceilf(xmax) - kTop, reach - kSpan);
            s.reach = fmaxf(reach, xmax + 16.f);   // new rows' fp16 values are below 2^15
            s.at = nr;
        }
    }
    const float fl = nr > was ? ex2(was - nr) : 1.f;
    if (has_o) scale_o<HD>(to, was == -INFINITY ? 0.f : fl * ex2(s.d - nd));
    s.own_r = nr, s.own_d = nd, s.own_l = s.l * fl + sum;
    s.r = 0.f, s.d = static_cast<float>(mt.vx[0]), s.l = -1e30f, s.qf = 1.f / mt.kf[0];
}

// Group k of a cached tile that is left out of the product: its weights' product with
// V in fp32, onto O; S = -infinity.
template <int HD, bool WIN>
__device__ __forceinline__ void far_group(const Kv8Args &p, const Kv8Piece &u, uint32_t ts, uint32_t to, const Kv8Meta &mt, int kt, int k, Kv8Row &s) {
    const int live = mt.live[k], key = kv8_tile<WIN>(u.sq, kt - u.sq.ntiles) * kTileK + 32 * k;   // its page is in the pool: it has keys
    const int page = p.c.table[static_cast<long long>(u.s) * p.c.max_pages + (key >> p.page_log2)];
    const uint8_t *v8 = static_cast<const uint8_t *>(p.c.v) + kv8_block(p.c, p.a.layer, page, u.head) * (p.c.page * HD) + (key & (p.c.page - 1));
    const float f = factor(mt.kf[k], s.qf), ux = static_cast<float>(mt.vx[k]) - s.d;
    [[maybe_unused]] const uint32_t see = WIN ? kv8_window_old(p, s.from, key) : 0u;
    float w[32], top = -INFINITY;
    {
        uint32_t v[32];
        tmem_ld_32x32b_x32(ts + 32 * k, v);
        tmem_ld_wait_for(v);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            w[e] = e < live && (!WIN || (see >> e & 1u)) ? __uint_as_float(v[e]) * f : -INFINITY;
            top = fmaxf(top, w[e]);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0xff800000u;
        tmem_st_32x32b_x16(ts + 32 * k, reinterpret_cast<const uint32_t(&)[16]>(v));
        tmem_st_32x32b_x16(ts + 32 * k + 16, reinterpret_cast<const uint32_t(&)[16]>(v));
    }
    const bool grow = s.r == -INFINITY ? top > -INFINITY : top - s.r > kLazy;
    if (__any_sync(0xffffffffu, grow)) {
        const float nr = grow ? ceilf(top) : s.r, fl = !grow ? 1.f : s.r == -INFINITY ? 0.f : ex2(s.r - nr);
        scale_o<HD>(to, fl);
        s.l *= fl;
        s.reach = reach_now(s, nr);
        s.at = s.r = nr;
    }
    const float at = s.r == -INFINITY ? 0.f : s.r;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        s.l += ex2(w[e] - at);
        w[e] = ex2((w[e] - at) + ux);
    }
#pragma unroll 1
    for (int q = 0; q < HD / 4; ++q) {
        uint32_t o[4];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(to + 4 * q));
        tmem_ld_wait_for(o);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint4 *src = reinterpret_cast<const uint4 *>(v8 + static_cast<long long>(4 * q + e) * p.c.page);
            const uint4 x = src[0], y = src[1];
            const uint32_t b[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            float acc = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int n = live - 4 * i;   // bytes behind the last token may be anything
                uint32_t lo, hi;
                uint32_t bytes = n >= 4 ? b[i] : n <= 0 ? 0u : b[i] & ((1u << (8 * n)) - 1u);
                if constexpr (WIN) bytes &= ((see >> 4 * i & 15u) * 0x00204081u & 0x01010101u) * 255u;   // a byte for each of 4 bits
                e4m3x4_f16(bytes, lo, hi);
                const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), c = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                acc = fmaf(w[4 * i], a.x, fmaf(w[4 * i + 1], a.y, fmaf(w[4 * i + 2], c.x, fmaf(w[4 * i + 3], c.y, acc))));
            }
            o[e] = __float_as_uint(__uint_as_float(o[e]) + acc);
        }
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + 4 * q), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
    }
    tmem_st_wait();
}

// What a tile needs before its weights: d of a tile whose largest scale is
// 2^mt.top, with O following, and the groups and rows that the loop over them cannot take as
// they are.  `row`: this thread's new row, or -1.
template <int HD, bool WIN>
__device__ __noinline__ void begin_tile(const Kv8Args &p, const Kv8Piece &u, uint32_t ts, uint32_t to, const Kv8Meta &mt, const Kv8Exps &ex, int kt, int row,
                                        bool has_o, Kv8Row &s) {
    const bool cached = kt >= u.sq.ntiles;
    const float top = static_cast<float>(mt.top);
    int far = mt.flags / kFar;
    if (!(mt.flags & kMixed)) {
        float nd = s.d, f = 1.f;
        if (top - nd < kTopLow || top - nd > kUnitHigh) {   // not where nothing has been seen: d is the tile's there
            s.reach = reach_now(s, s.r);
            s.at = s.r;
            nd = fmaxf(top - kTop, s.reach - kSpan);
            f = ex2(s.d - nd);
        }
        if (__any_sync(0xffffffffu, f != 1.f)) scale_o<HD>(to, f);   // such a row has an O
        s.d = nd;
        if (__any_sync(0xffffffffu, top - nd < kTopLow)) {   // O's reach keeps d above: no bits would be left of fp16 weights
            if (!cached) {
                own_scores<HD, WIN>(p, u, ts, to, mt, ex, kt * kTileK, row, has_o, s);
                return;
            }
            far = 0;
            for (int k = 0; k < 4; ++k) far |= mt.live[k] > 0 ? 1 << k : 0;
        }
    } else {
        own_scores<HD, WIN>(p, u, ts, to, mt, ex, kt * kTileK, row, has_o, s);
        return;
    }
    if (far && !has_o) {   // O, to add to
        const uint32_t zero[16] = {};
#pragma unroll 1
        for (int q = 0; q < HD / 16; ++q) tmem_st_32x32b_x16(to + 16 * q, zero);
        tmem_st_wait();
    }
#pragma unroll 1
    for (int k = 0; k < 4; ++k)
        if (far >> k & 1) far_group<HD, WIN>(p, u, ts, to, mt, kt, k, s);
}

// The pieces behind the first: one copy of the code for the roles of k_kv8_tiles
// (123.5 us against 126.0 for 256 rows over 16k tokens).  The first piece is found
// before the roles part, which a call like this would delay by 2.3 us.
template <bool WIN>
__device__ __noinline__ bool kv8_next_call(const Kv8Args &p, const long long *tiles, Kv8Walk &w, Kv8Piece &u) { return kv8_next<WIN>(p, tiles, w, u); }

template <int HD, bool WIN>
__global__ void __launch_bounds__(kTileThreads, 1) k_kv8_tiles(const __grid_constant__ Kv8Args p) {
    using Lay = Tiles<HD>;
    extern __shared__ __align__(1024) uint8_t tiles_smem[];   // the operands' swizzle repeats every 1024 bytes
    uint8_t *smem = tiles_smem;
    const uint32_t sm = smem_u32(smem);
    Kv8Meta *meta = reinterpret_cast<Kv8Meta *>(smem + Lay::meta_off);
    Kv8Meta *head = reinterpret_cast<Kv8Meta *>(smem + Lay::head_off);
    Kv8Exps *exps = reinterpret_cast<Kv8Exps *>(smem + Lay::exp_off);
    uint32_t *red = reinterpret_cast<uint32_t *>(smem + Lay::red_off);
    long long *tiles = reinterpret_cast<long long *>(smem + Lay::tiles_off);
    const uint32_t bars = sm + Lay::bar_off;
    auto k_full = [&](int b) { return bars + 8 * b; };             // K's warps
    auto k_empty = [&](int b) { return bars + 8 * (2 + b); };      // commit of S
    auto v_full = [&](int b) { return bars + 8 * (4 + b); };       // V's warps
    auto v_empty = [&](int b) { return bars + 8 * (6 + b); };      // commit of O
    auto s_full = [&](int b) { return bars + 8 * (8 + b); };
    auto p_full = [&](int b) { return bars + 8 * (10 + b); };      // 4 softmax warps
    auto m_full = [&](int t) { return bars + 8 * (12 + t); };      // meta of tile % 4
    auto o_full = [&](int b) { return bars + 8 * (16 + b); };      // commit of O
    auto raw_full = [&](int s) { return bars + 8 * (22 + s); };    // bulk copies
    auto raw_empty = [&](int s) { return bars + 8 * (28 + s); };   // the operand warps
    const uint32_t q_full = bars + 8 * 34, r_full = bars + 8 * 35, drain = bars + 8 * 36, e_full = bars + 8 * 37;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::bar_off + 8 * 38);
    // With a window, by unit % 4: the operand warps are through with the unit's V, and each of them met a NaN at its edges or not.
    const uint32_t win_off = static_cast<uint32_t>(Lay::tiles_end(p.c.n_seqs));
    [[maybe_unused]] auto n_full = [&](int t) { return sm + win_off + 8 * t; };
    [[maybe_unused]] int *nans = reinterpret_cast<int *>(smem + win_off + 32);
    long long *warp_sum = reinterpret_cast<long long *>(smem + Lay::bar_off + 40 * 8);

    const la_kv8_cache &c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(k_full(b), kOpWarps);
            mbar_init(k_empty(b), 1);
            mbar_init(v_full(b), kOpWarps);
            mbar_init(v_empty(b), 1);
            mbar_init(s_full(b), 1);
            mbar_init(p_full(b), 4);
            mbar_init(o_full(b), 1);
        }
        for (int t = 0; t < 4; ++t) mbar_init(m_full(t), 1);
        for (int t = 0; t < Lay::raw_slots; ++t) {
            mbar_init(raw_full(t), 1);
            mbar_init(raw_empty(t), kOpWarps);
        }
        mbar_init(q_full, 8);
        mbar_init(e_full, 8);
        mbar_init(r_full, kOpWarps);
        mbar_init(drain, 1);
        if constexpr (WIN)
            for (int t = 0; t < 4; ++t) mbar_init(n_full(t), kOpWarps);
        fence_barrier_init();
    }
    // Tensor memory is taken once the kernel before has finished, and the one
    // behind may start only when it is taken: neither can wait for the other's.
    pdl_wait();
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), kColAll);
        tmem_relinquish();
    }
    tc_fence_before();
    kv8_plan<WIN>(p, tiles, warp_sum);   // barriers inside
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    Kv8Walk walk = kv8_walk<WIN>(p, tiles);
    Kv8Piece u{};
    const bool begun = kv8_next<WIN>(p, tiles, walk, u);   // the first piece
    int it = 0;          // key tiles so far, the same count in every role: buffer it & 1, its use it >> 1
    bool ok = true;
    unsigned *err = c.status;

    // Table entries of cached tile kt of piece u: lane l < 4 holds that of keys
    // 32 l .. of the tile (-2: none).  They are checked a tile later, so that
    // nothing waits for the load.
    auto entry = [&](int kt) {
        const int key = kv8_tile<WIN>(u.sq, kt - u.sq.ntiles) * kTileK + 32 * (lane & 3);
        return kt < u.k1 && key < u.sq.len ? c.table[static_cast<long long>(u.s) * c.max_pages + (key >> p.page_log2)] : -2;
    };
    auto checked = [&](int e) {
        if (static_cast<unsigned>(e) < static_cast<unsigned>(c.n_pages)) return e;
        if (e != -2) atomicOr(err, LA_KV8_BAD);
        return -1;
    };

    if (warp >= 8 && warp < kLoadWarp) {
        // ================================================ operands
        const int w = __shfl_sync(0xffffffffu, warp - 8, 0);   // the same in all lanes, for the compiler too
        // A tile of K, or of V, is NG groups of 32 16-byte pieces, dealt to the
        // warps in turn, K's from the first and V's from the last on: 8 keys x 64
        // bytes of K, 8 dims x 64 keys of V.  Lane: key (dim) r8, piece cq; where a
        // row has 128 bytes, the odd rows take the other 64, so that the lanes read
        // (and write) different banks.
        constexpr int NG = HD / 4, NR = (NG + kOpWarps - 1) / kOpWarps;
        const int r8 = lane >> 2, cq = lane & 3;
        const uint32_t half = HD == 128 ? r8 & 1 : 0, vhalf = r8 & 1;
        const uint32_t put0 = r8 * 128 + (((2 * cq) ^ r8) << 4), put1 = r8 * 128 + (((2 * cq + 1) ^ r8) << 4);
        auto put_f16 = [&](uint32_t at, const uint4 &bytes) {   // a piece's values, as fp16, to their rows
            uint4 x, y;
            e4m3x16_f16(bytes, x, y);
            st_shared(at + put0, x);
            st_shared(at + put1, y);
        };
        auto v_at = [&](uint32_t h) {   // byte of keys 64 h + 16 cq of dim r8 in V's stage: pages of [HD][page]
            const uint32_t key = 64 * h + 16 * cq;
            return (key >> p.page_log2) * static_cast<uint32_t>(HD << p.page_log2) + (r8 << p.page_log2) + (key & (c.page - 1));
        };
        const uint32_t v_at0 = v_at(vhalf), v_at1 = v_at(vhalf ^ 1);
        int new_tiles = 0, slot = 0;
        uint32_t phase = 0;
        [[maybe_unused]] int units = 0;
        [[maybe_unused]] uint32_t nan_met = 0;
        auto landed = [&]() {   // the next stage of bytes is there
            ok = __all_sync(0xffffffffu, bar_wait(raw_full(slot), phase, err, LA_KV8_TIMEOUT));
            return sm + Lay::raw_off + slot * Lay::raw_bytes;
        };
        auto read = [&]() {     // and has been read
            if (lane == 0) mbar_arrive_one(raw_empty(slot));
            if (++slot == Lay::raw_slots) {
                slot = 0;
                phase ^= 1;
            }
        };
        for (bool any = begun; ok && any; any = kv8_next_call<WIN>(p, tiles, walk, u)) {
            const Kv8Seq sq = u.sq;
            auto k_tile = [&](int kt, int it) {
                const int b = it & 1, use = it >> 1;
                const uint32_t sk = sm + Lay::k_off + b * Lay::k_bytes;
                if (use > 0) ok = __all_sync(0xffffffffu, bar_wait(k_empty(b), (use - 1) & 1, err, LA_KV8_TIMEOUT));
                if (!ok) return;
                if (kt < sq.ntiles) {
                    // New rows: bf16, scaled by a power of two for the whole tile.
                    const int key0 = kt * kTileK, nkeys = min(kTileK, sq.rows - key0);
                    const __nv_bfloat16 *kn = static_cast<const __nv_bfloat16 *>(p.a.k) + (sq.first + key0) * p.a.k_stride + u.head * HD;
                    const __nv_bfloat16 *vn = static_cast<const __nv_bfloat16 *>(p.a.v) + (sq.first + key0) * p.a.v_stride + u.head * HD;
                    constexpr int C8 = HD / 8, NT = 32 * kOpWarps;   // 16-byte pieces of a row
                    const int ot = w * 32 + lane;
                    // K's rows come into its operand buffer as they are (asynchronous
                    // copies, all in flight: one load after another took 12 us) and
                    // are turned into fp16 in place; V's largest magnitude meanwhile.
                    auto kat = [&](int i) { return sk + ((i % C8) >> 3) * Lay::k_block + (i / C8) * 128 + (((i % 8) ^ (i / C8 & 7)) << 4); };
                    uint32_t ak = 0, av = 0, lk = ~0u, lv = ~0u;   // largest; least but zeros, less 1
                    auto least = [](uint32_t l, uint32_t top) { return min(l, max(top & 0xffffu, top >> 16) - 1u); };
#pragma unroll 1
                    for (int i = ot; i < kTileK * C8; i += NT) {
                        const int r = i / C8;
                        const uint32_t n = r < nkeys ? 16 : 0;   // rows past the last: zeros
                        const __nv_bfloat16 *from = kn + (n ? r : 0) * p.a.k_stride + 8 * (i % C8);
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(kat(i)), "l"(from), "r"(n) : "memory");
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll 4
                    for (int i = ot; i < nkeys * C8; i += NT) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(vn + (i / C8) * p.a.v_stride + 8 * (i % C8));
                        const uint32_t top = most2(most2(most2(most2(0u, x.x), x.y), x.z), x.w);
                        av = most2(av, top);
                        lv = least(lv, top);
                    }
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 2
                    for (int i = ot; i < kTileK * C8; i += NT) {   // the pieces that this thread copied
                        const uint4 x = ld_shared(kat(i));
                        const uint32_t top = most2(most2(most2(most2(0u, x.x), x.y), x.z), x.w);
                        ak = most2(ak, top);
                        lk = least(lk, top);
                    }
                    // A NaN or infinity among them: the maxima again, without those.
                    bool odd = max(av & 0xffffu, av >> 16) >= 0x7f80u;
                    if (__any_sync(0xffffffffu, odd || max(ak & 0xffffu, ak >> 16) >= 0x7f80u)) {
                        ak = av = 0;
                        lk = lv = ~0u;
#pragma unroll 1
                        for (int i = ot; i < nkeys * C8; i += NT) {
                            const uint32_t x = finite_top(*reinterpret_cast<const uint4 *>(vn + (i / C8) * p.a.v_stride + 8 * (i % C8))), y = finite_top(ld_shared(kat(i)));
                            av = most2(av, x);
                            lv = least(lv, x);
                            ak = most2(ak, y);
                            lk = least(lk, y);
                        }
                    }
                    ak = max(ak & 0xffffu, ak >> 16);
                    av = max(av & 0xffffu, av >> 16);
                    ak = __reduce_max_sync(0xffffffffu, ak);
                    av = __reduce_max_sync(0xffffffffu, av);
                    lk = min(__reduce_min_sync(0xffffffffu, lk), 0x7fffu);
                    lv = min(__reduce_min_sync(0xffffffffu, lv), 0x7fffu);
                    odd = __any_sync(0xffffffffu, odd);
                    // The warps' maxima: two halves, one for each buffer, so that no
                    // warp writes what another still reads.
                    uint32_t *mine = red + 16 * b;
                    if (lane == 0) {
                        mine[w] = ak | lk << 16;
                        mine[8 + w] = av | lv << 16 | (odd ? 0x80000000u : 0u);
                        mbar_arrive_one(r_full);
                    }
                    __syncwarp();
                    ok = __all_sync(0xffffffffu, bar_wait(r_full, new_tiles & 1, err, LA_KV8_TIMEOUT));
                    if (!ok) return;
                    ++new_tiles;
                    ak = av = 0;
                    lk = lv = 0x7fffu;
                    odd = false;
#pragma unroll
                    for (int k = 0; k < kOpWarps; ++k) {
                        const uint32_t x = mine[k], y = mine[8 + k];
                        ak = max(ak, x & 0xffffu);
                        av = max(av, y & 0xffffu);
                        lk = min(lk, x >> 16);
                        lv = min(lv, y >> 16 & 0x7fffu);
                        odd |= y >> 31 != 0;
                    }
                    int kx = fit_f16(bf16_bits(ak)), vx = fit_f16(bf16_bits(av));
                    // Exponents of bf16 bits; a least of 0x7fff: only zeros
                    const bool mixed = static_cast<int>(ak >> 7) - static_cast<int>((lk + 1) >> 7) > kSpread ||
                                       static_cast<int>(av >> 7) - static_cast<int>((lv + 1) >> 7) > kSpread;
                    if (mixed) {
                        mixed_rows<HD>(sk, Lay::k_block, vn, p.a.v_stride, nkeys, ot, &exps[it & 3]);
                        __syncwarp();
                        if (lane == 0) mbar_arrive_one(r_full);
                        __syncwarp();
                        ok = __all_sync(0xffffffffu, bar_wait(r_full, new_tiles & 1, err, LA_KV8_TIMEOUT));
                        if (!ok) return;
                        ++new_tiles;
                        kx = vx = 0;   // the scores come with all factors (mixed_scores)
                    }
                    if (w == 0) {
                        if (lane < 4) {
                            Kv8Meta &mt = meta[it & 3];
                            mt.kf[lane] = power_of(kx);
                            mt.vx[lane] = vx;
                            mt.live[lane] = min(max(nkeys - 32 * lane, 0), 32);
                            if (lane == 0) {
                                mt.flags = (odd ? kOddV : 0) | (mixed ? kMixed : 0);
                                mt.top = vx + 5;
                            }
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive_one(m_full(it & 3));
                    }
                    const float fk = power_of(-kx);
#pragma unroll 2
                    for (int i = mixed ? kTileK * C8 : ot; i < kTileK * C8; i += NT) {
                        const uint4 x = ld_shared(kat(i));
                        st_shared_u32x4(kat(i), scaled_f16(x.x, fk), scaled_f16(x.y, fk), scaled_f16(x.z, fk), scaled_f16(x.w, fk));
                    }
                } else {
                    const uint32_t raw = landed();
                    if (!ok) return;
                    if (w == 0) {
                        if (lane < 16) reinterpret_cast<uint32_t *>(meta + (it & 3))[lane] = reinterpret_cast<const uint32_t *>(head + slot)[lane];
                        __syncwarp();
                        if (lane == 0) mbar_arrive_one(m_full(it & 3));
                    }
                    uint4 x[NR];
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const int g = w + n * kOpWarps;
                        if (g < NG) x[n] = ld_shared(raw + (HD == 128 ? (g >> 1) * 1024 + r8 * 128 + (((g & 1) ^ half) << 6) : g * 512 + r8 * 64) + 16 * cq);
                    }
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const int g = w + n * kOpWarps;
                        if (g < NG) put_f16(sk + (HD == 128 ? ((g & 1) ^ half) * Lay::k_block + (g >> 1) * 1024 : g * 1024), x[n]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_one(k_full(b));
                if (kt >= sq.ntiles) read();
            };
            auto v_tile = [&](int kt, int it) {
                const int b = it & 1, use = it >> 1;
                const uint32_t sv = sm + Lay::v_off + b * Lay::v_bytes;
                if (use > 0) ok = __all_sync(0xffffffffu, bar_wait(v_empty(b), (use - 1) & 1, err, LA_KV8_TIMEOUT));
                if (!ok) return;
                if (kt < sq.ntiles) {
                    // Two new rows of eight dims at a time, transposed.  A NaN or
                    // infinity counts 0 here and is added at the end for the
                    // rows that see it.
                    ok = __all_sync(0xffffffffu, bar_wait(m_full(it & 3), it >> 2 & 1, err, LA_KV8_TIMEOUT));
                    if (!ok) return;
                    const float fv = power_of(-meta[it & 3].vx[0]);
                    const bool mixed = meta[it & 3].flags & kMixed;
                    const int key0 = kt * kTileK, nkeys = min(kTileK, sq.rows - key0);
                    const __nv_bfloat16 *vn = static_cast<const __nv_bfloat16 *>(p.a.v) + (sq.first + key0) * p.a.v_stride + u.head * HD;
                    constexpr int NT = 32 * kOpWarps, NP = kTileK / 2 * (HD / 8), B = 4;   // pairs of rows, in flight
                    if (mixed) mixed_v<HD>(sv, Lay::v_block, vn, p.a.v_stride, nkeys, w * 32 + lane, exps[it & 3].v);
#pragma unroll 1
                    for (int j0 = mixed ? NP : w * 32 + lane; j0 < NP; j0 += B * NT) {
                        uint4 va[B], vb[B];
#pragma unroll
                        for (int q = 0; q < B; ++q) {
                            const int j = j0 + q * NT, r = 2 * (j % (kTileK / 2)), d = 8 * (j / (kTileK / 2));   // lanes: rows, other banks
                            va[q] = j < NP && r < nkeys ? *reinterpret_cast<const uint4 *>(vn + r * p.a.v_stride + d) : make_uint4(0, 0, 0, 0);
                            vb[q] = j < NP && r + 1 < nkeys ? *reinterpret_cast<const uint4 *>(vn + (r + 1) * p.a.v_stride + d) : make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int q = 0; q < B; ++q) {
                            const int j = j0 + q * NT, r = 2 * (j % (kTileK / 2)), d = 8 * (j / (kTileK / 2));
                            if (j >= NP) break;
                            const uint32_t x[4] = {va[q].x, va[q].y, va[q].z, va[q].w}, y[4] = {vb[q].x, vb[q].y, vb[q].z, vb[q].w};
                            const uint32_t at = sv + (r >> 6) * Lay::v_block + (r & 7) * 2;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                float f0 = bf16_bits(k & 1 ? x[k >> 1] >> 16 : x[k >> 1] & 0xffffu), f1 = bf16_bits(k & 1 ? y[k >> 1] >> 16 : y[k >> 1] & 0xffffu);
                                f0 = is_finite(f0) ? f0 * fv : 0.f;
                                f1 = is_finite(f1) ? f1 * fv : 0.f;
                                const int dim = d + k;
                                asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + dim * 128 + ((((r >> 3) & 7) ^ (dim & 7)) << 4)), "r"(pack_f16(f0, f1)) : "memory");
                            }
                        }
                    }
                } else {
                    const uint32_t raw = landed();
                    if (!ok) return;
                    uint4 x[NR];
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const int g = kOpWarps - 1 - w + n * kOpWarps;
                        if (g < NG) x[n] = ld_shared(raw + (g & 1 ? v_at1 : v_at0) + (g >> 1) * (8 << p.page_log2));
                    }
                    // Bytes behind the last token, and of missing pages, may be anything.
                    const int4 live = *reinterpret_cast<const int4 *>(head[slot].live);
                    if ((live.x & live.y & live.z & live.w) != 32) {
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            const int ch = cq + 4 * (((kOpWarps - 1 - w + n * kOpWarps) & 1) ^ vhalf), keys = head[slot].live[ch >> 1] - 16 * (ch & 1);
                            auto cut = [](uint32_t a, int m) { return m >= 4 ? a : m <= 0 ? 0u : a & ((1u << (8 * m)) - 1u); };
                            x[n] = make_uint4(cut(x[n].x, keys), cut(x[n].y, keys - 4), cut(x[n].z, keys - 8), cut(x[n].w, keys - 12));
                        }
                    }
                    if constexpr (WIN) {
                        // In a tile that has keys which some rows do not see a NaN counts 0, and
                        // is added at the end for the rows that see it.
                        if (kv8_edge(p, sq, (u.qv0 + u.nqv - 1) / p.gq, kv8_tile<WIN>(sq, kt - sq.ntiles) * kTileK, kTileK)) {
#pragma unroll
                            for (int n = 0; n < NR; ++n) {
                                if (kOpWarps - 1 - w + n * kOpWarps >= NG) continue;
                                auto tame = [&](uint32_t &v) {
                                    const uint32_t nan = __vcmpeq4(v & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                    nan_met |= nan;
                                    v &= ~nan;
                                };
                                tame(x[n].x), tame(x[n].y), tame(x[n].z), tame(x[n].w);
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const int g = kOpWarps - 1 - w + n * kOpWarps;
                        if (g < NG) put_f16(sv + ((g & 1) ^ vhalf) * Lay::v_block + (g >> 1) * 1024, x[n]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_one(v_full(b));
                if (kt >= sq.ntiles) read();
            };
            // K a tile ahead of V: S of the next tile is issued before O of this one.
            const int first = it;
#pragma unroll 1
            for (int kt = u.k0 - 1; ok && kt < u.k1; ++kt) {
                if (kt + 1 < u.k1) k_tile(kt + 1, first + kt + 1 - u.k0);
                if (ok && kt >= u.k0) v_tile(kt, first + kt - u.k0);
            }
            it = first + max(u.k1 - u.k0, 0);
            if constexpr (WIN) {
                if (ok && u.k1 > u.k0) {
                    const bool met = __any_sync(0xffffffffu, nan_met != 0);
                    if (lane == 0) {
                        nans[(units & 3) * kOpWarps + w] = met;
                        mbar_arrive_one(n_full(units & 3));
                    }
                    __syncwarp();
                    nan_met = 0;
                    ++units;
                }
            }
        }
    } else if (warp == kLoadWarp) {
        // ================================================ bytes
        // Stages in the order in which they are read: K of a tile, V of the tile before.
        const uint32_t bytes = static_cast<uint32_t>(c.page) * HD;                        // a page's block, of K or V
        const uint32_t starts = c.page == 32 ? 15u : c.page == 64 ? 5u : 1u;              // lanes whose keys begin a page
        int slot = 0;
        uint32_t phase = 0, staged = 0;
        // Lane l < 4: block number of keys 32 l .. of a tile (a block is 2 KB at
        // least, so 32 bits reach all memory), and which lanes have one.
        auto block_of = [&](int page, uint32_t &held) {
            held = __ballot_sync(0xffffffffu, page >= 0) & 15u;
            return static_cast<uint32_t>(kv8_block(c, p.a.layer, max(page, 0), u.head));
        };
        // Tile kt's K or V, with what its readers need to know of its pages.
        auto stage = [&](const void *pool, int kt, uint32_t blk, uint32_t held, float ks, float vs) {
            if (staged >= Lay::raw_slots) ok = __all_sync(0xffffffffu, bar_wait(raw_empty(slot), phase ^ 1, err, LA_KV8_TIMEOUT));
            if (!ok) return;
            const bool have = held >> lane & 1u;
            const int live = have ? min(max(u.sq.len - kv8_tile<WIN>(u.sq, kt - u.sq.ntiles) * kTileK - 32 * lane, 0), 32) : 0, vx = exponent_of(vs);
            const int top = __reduce_max_sync(0xffffffffu, live > 0 ? vx : -127);
            const uint32_t far = __ballot_sync(0xffffffffu, live > 0 && vx < top - kNear);
            if (lane < 4) {
                head[slot].kf[lane] = have ? ks : 1.f;
                head[slot].vx[lane] = have ? vx : 0;
                head[slot].live[lane] = live;
                if (lane == 0) {
                    head[slot].flags = far * kFar;
                    head[slot].top = top;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(raw_full(slot), __popc(held & starts) * bytes);
            __syncwarp();
            if (held & starts & 1u << lane)
                bulk_load(sm + Lay::raw_off + slot * Lay::raw_bytes + (lane >> (p.page_log2 - 5)) * bytes,
                          static_cast<const uint8_t *>(pool) + static_cast<uint64_t>(blk) * bytes, bytes, raw_full(slot));
            __syncwarp();
            ++staged;
            if (++slot == Lay::raw_slots) {
                slot = 0;
                phase ^= 1;
            }
        };
        for (bool any = begun; ok && any; any = kv8_next_call<WIN>(p, tiles, walk, u)) {
            const int c_first = max(u.k0, u.sq.ntiles);   // first cached tile of this piece
            if (c_first >= u.k1) continue;
            uint32_t held = 0, v_held = 0, v_blk = 0, blk = block_of(checked(entry(c_first)), held);
            int after = entry(c_first + 1);
            float ks = c.k_scale[blk], vs = c.v_scale[blk];
#pragma unroll 1
            for (int kt = c_first; ok && kt <= u.k1; ++kt) {
                if (kt < u.k1) stage(c.k, kt, blk, held, ks, vs);
                if (ok && kt > c_first) stage(c.v, kt - 1, v_blk, v_held, 1.f, 1.f);
                v_blk = blk;
                v_held = held;
                blk = block_of(checked(after), held);   // entries and scales are read a tile ahead
                ks = c.k_scale[blk];
                vs = c.v_scale[blk];
                after = entry(kt + 2);
            }
        }
        // The last copies have landed (where a wait gave up, nobody else has seen that).
        for (uint32_t n = min(staged, static_cast<uint32_t>(Lay::raw_slots)); n > 0; --n) {
            slot = slot == 0 ? Lay::raw_slots - 1 : slot - 1;
            if (slot == Lay::raw_slots - 1) phase ^= 1;
            bar_wait(raw_full(slot), phase, err, LA_KV8_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ================================================ products
        // The whole warp runs this loop; one elected lane issues.  (Inside a
        // branch on the lane's number each product took 90 cycles to issue.)
        if (!p.whole && lane == 0) kv8_note(p, tiles, begun, u);
        constexpr uint32_t is = idesc_f16(kTileQ, kTileK), io = idesc_f16(kTileQ, HD);
        auto wait = [&](uint32_t bar, int parity) { return __all_sync(0xffffffffu, bar_wait(bar, parity & 1, err, LA_KV8_TIMEOUT)); };
        int units = 0;
        for (bool any = begun; ok && any; any = kv8_next_call<WIN>(p, tiles, walk, u)) {
            if (u.k0 >= u.k1) continue;
            ok = wait(q_full, units);
            ++units;
            const int first = it, end = it + u.k1 - u.k0;
#pragma unroll 1
            for (; ok && it <= end; ++it) {   // S of tile `it`, then O of the one before
                if (it < end) {
                    const int b = it & 1;
                    ok = wait(k_full(b), it >> 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sk = sm + Lay::k_off + b * Lay::k_bytes;
                    if (elect_one()) {
#pragma unroll
                        for (int db = 0; db < HD / 64; ++db) {
                            const uint64_t d = umma_desc_sw128(sk + db * Lay::k_block), q = umma_desc_sw128(sm + Lay::q_off + db * Lay::k_block);
#pragma unroll
                            for (int k = 0; k < 4; ++k) umma_bf16(tmem + kColS + 128 * b, q + 2 * k, d + 2 * k, is, (db | k) ? 1u : 0u);
                        }
                        umma_commit(s_full(b));
                        umma_commit(k_empty(b));
                    }
                    __syncwarp();
                }
                if (it > first) {
                    const int j = it - 1, b = j & 1;
                    ok = wait(p_full(b), j >> 1) && wait(v_full(b), j >> 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sv = sm + Lay::v_off + b * Lay::v_bytes, pt = tmem + kColS + 128 * b, ot = tmem + kColO + 128 * b;
                    const bool fresh = j < first + 2 && meta[j & 3].flags < kFar;   // O holds nothing yet
                    if (elect_one()) {
#pragma unroll
                        for (int kb = 0; kb < 2; ++kb) {
                            const uint64_t d = umma_desc_sw128(sv + kb * Lay::v_block);
#pragma unroll
                            for (int k = 0; k < 4; ++k) umma_ts(ot, pt + kb * 32 + k * 8, d + 2 * k, io, fresh && !(kb | k) ? 0u : 1u);
                        }
                        umma_commit(v_empty(b));
                        umma_commit(o_full(b));
                    }
                    __syncwarp();
                }
            }
            it = end;
        }
        if (!ok) {   // void: wait (bounded) for the products in flight
            if (elect_one()) umma_commit(drain);
            __syncwarp();
            bar_wait(drain, 0, err, LA_KV8_TIMEOUT);
        }
        __syncwarp();
    } else {
        // ================================================ softmax
        int grp = warp >> 2, row = 32 * (warp & 3) + lane;
        uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        uint32_t ts = tmem + lanes + kColS + 128 * grp, to = tmem + lanes + kColO + 128 * grp;
        float *qfs = reinterpret_cast<float *>(smem + Lay::qf_off);
        int *odds = reinterpret_cast<int *>(smem + Lay::odd_off);
        int units = 0;
        for (bool any = begun; ok && any; any = kv8_next_call<WIN>(p, tiles, walk, u)) {
            Kv8Seq sq = u.sq;
            bool in = row < u.nqv;
            const bool idle = row - lane >= u.nqv;   // none of this warp's rows is in use
            const int qv = u.qv0 + row;
            int myrow = in ? qv / p.gq : 0, myhead = u.head * p.gq + (in ? qv % p.gq : 0), first = it, end = it + max(u.k1 - u.k0, 0);
            float qf = 0.f;
            if (first < end) {
                // q as fp16, each vector scaled by a power of two to fit: 8 lanes a
                // row, 32 rows at a time.  The rows come in by asynchronous copies,
                // all in flight, and are turned in place.
                constexpr int NW = HD / 64;   // 16-byte pieces of a lane's HD / 8 dims
                tc_fence_before();            // the last unit's O is read
                const int part = tid & 7, rows = (u.nqv + 31) / 32 * 32;
                auto qat = [&](int r, int k) {
                    const int ch = part * NW + k;   // 8 dims
                    return sm + Lay::q_off + (ch >> 3) * Lay::k_block + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
                };
#pragma unroll 1
                for (int r = tid >> 3; r < rows; r += 32) {
                    const int v = u.qv0 + r, n = r < u.nqv ? 16 : 0;
                    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.a.q) + (sq.first + (n ? v / p.gq : 0)) * p.a.q_stride +
                                               (u.head * p.gq + (n ? v % p.gq : 0)) * HD + part * (HD / 8);
#pragma unroll
                    for (int k = 0; k < NW; ++k)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(qat(r, k)), "l"(src + 8 * k), "r"(n) : "memory");
                }
                asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
                for (int r = tid >> 3; r < rows; r += 32) {
                    uint4 x[NW];
                    uint32_t top = 0;
#pragma unroll
                    for (int k = 0; k < NW; ++k) {
                        x[k] = ld_shared(qat(r, k));
                        top = most2(most2(most2(most2(top, x[k].x), x[k].y), x[k].z), x[k].w);
                    }
#pragma unroll
                    for (int k = 1; k < 8; k <<= 1) top = most2(top, __shfl_xor_sync(0xffffffffu, top, k));
                    const int qx = fit_pair(top);
                    const float f = power_of(-qx);
#pragma unroll
                    for (int k = 0; k < NW; ++k)
                        st_shared_u32x4(qat(r, k), scaled_f16(x[k].x, f), scaled_f16(x[k].y, f), scaled_f16(x[k].z, f), scaled_f16(x[k].w, f));
                    if (part == 0) qfs[r] = factor(power_of(qx), p.scale_log2);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_one(q_full);
                ok = __all_sync(0xffffffffu, bar_wait(q_full, units & 1, err, LA_KV8_TIMEOUT));
                if (!ok) break;
                qf = idle ? 0.f : qfs[row];
            }
            float r = -INFINITY, d = 0.f, l = 0.f;
            [[maybe_unused]] int from = 0;
            if constexpr (WIN) from = sq.len + kv8_seen(p, sq.first, sq.rows, myrow) - p.window;
            Kv8Row keep;   // in memory: what only the rare paths ask for
            keep.reach = keep.at = -INFINITY;
            bool odd = false;
            for (int kt = u.k0 + ((first ^ grp) & 1); kt < u.k1; kt += 2) {
                int i = first + kt - u.k0, b = grp;   // tile number, of this group's parity
                ok = bar_wait(s_full(b), i >> 1 & 1, err, LA_KV8_TIMEOUT) && bar_wait(m_full(i & 3), i >> 2 & 1, err, LA_KV8_TIMEOUT);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const Kv8Meta *mt = &meta[i & 3];
                odd |= (mt->flags & kOddV) != 0;
                if (!idle) {
                    // What is rare first (begin_tile).  Then 32 keys at a time: the weights'
                    // exponents at r and d as they stand, then the weights, over
                    // columns of S that are read already.  One
                    // copy of this code: unrolled, the roles' code does not fit
                    // the instruction cache (5 us per pair of tiles).
                    bool cached = kt >= sq.ntiles;
                    const float top = static_cast<float>(mt->top);
                    [[maybe_unused]] const int key0 = kv8_tile<WIN>(sq, kt - sq.ntiles) * kTileK;
                    if (r == -INFINITY) d = top - kTop;
                    if (__any_sync(0xffffffffu, top - d < kTopLow || top - d > kUnitHigh) || (mt->flags & ~kOddV)) {
                        if (i >= first + 2) {   // this group's O holds its tile i - 2
                            ok = __all_sync(0xffffffffu, bar_wait(o_full(b), (i - 2) >> 1 & 1, err, LA_KV8_TIMEOUT));
                            if (!ok) break;
                            tc_fence_after();
                        }
                        keep.r = r, keep.d = d, keep.l = l, keep.qf = qf;
                        keep.grp = grp, keep.row = row, keep.units = units, keep.it = it, keep.first = first, keep.end = end, keep.i = i, keep.kt = kt;
                        keep.myrow = myrow, keep.myhead = myhead, keep.lanes = lanes, keep.ts = ts, keep.to = to, keep.in = in, keep.odd = odd;
                        if constexpr (WIN) keep.from = from;
                        begin_tile<HD, WIN>(p, u, ts, to, *mt, exps[i & 3], kt, in ? myrow : -1, i >= first + 2, keep);
                        r = keep.r, d = keep.d, l = keep.l, qf = keep.qf;
                        grp = b = keep.grp, row = keep.row, units = keep.units, it = keep.it, first = keep.first, end = keep.end, i = keep.i, kt = keep.kt;
                        myrow = keep.myrow, myhead = keep.myhead, lanes = keep.lanes, ts = keep.ts, to = keep.to, in = keep.in, odd = keep.odd;
                        sq = u.sq, mt = &meta[i & 3], cached = kt >= sq.ntiles;
                        if constexpr (WIN) from = keep.from;
                    }
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(ts + 32 * k, v);
                        const int live = mt->live[k];
                        const float ux = static_cast<float>(mt->vx[k]) - d;   // u of this group
                        const float f = factor(mt->kf[k], qf), add = ux - (r == -INFINITY ? 0.f : r);
                        tmem_ld_wait_for(v);
                        if (live < 32 || !cached || (WIN && key0 + 32 * k + 32 > p.sinks && key0 + 32 * k < from)) {
                            uint32_t see = live >= 32 ? 0xffffffffu : (1u << live) - 1u;   // keys that this row sees
                            if (!cached) see &= new_rows_seen<WIN>(p, sq, in ? myrow : -1, kt * kTileK + 32 * k);
                            else if constexpr (WIN) see &= kv8_window_old(p, from, key0 + 32 * k);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = see >> e & 1u ? v[e] : 0xff800000u;   // -infinity
                        }
                        float x0 = -INFINITY, x1 = -INFINITY;
                        const uint64_t f2 = pair(f, f), add2 = pair(add, add);
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float2 x = halves(fma2(pair(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), f2, add2));
                            const float2 y = halves(fma2(pair(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), f2, add2));
                            x0 = max3(x0, x.x, x.y);
                            x1 = max3(x1, y.x, y.y);
                            v[e] = __float_as_uint(x.x);
                            v[e + 1] = __float_as_uint(x.y);
                            v[e + 2] = __float_as_uint(y.x);
                            v[e + 3] = __float_as_uint(y.y);
                        }
                        x0 = fmaxf(x0, x1) - ux;   // past r by this much
                        const bool grow = r == -INFINITY ? x0 > -INFINITY : x0 > kLazy;
                        if (__any_sync(0xffffffffu, grow)) {
                            const float by = !grow ? 0.f : ceilf(x0), alpha = !grow ? 1.f : r == -INFINITY ? 0.f : ex2(-by);
                            if (grow) r = r == -INFINITY ? by : r + by;
                            l *= alpha;
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) - by);
                            tmem_st_wait();
                            for (int q = 0; q < k; ++q) {   // this tile's weights so far
                                uint32_t w[16];
                                tmem_ld_32x32b_x16(ts + 16 * q, w);
                                tmem_ld_wait_for(w);
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                                    w[e] = pack_f16(x.x * alpha, x.y * alpha);
                                }
                                tmem_st_32x32b_x16(ts + 16 * q, w);
                            }
                            if (i >= first + 2 || mt->flags >= kFar) {   // this group's O holds its tile i - 2, or far groups of this one
                                if (i >= first + 2) ok = __all_sync(0xffffffffu, bar_wait(o_full(b), (i - 2) >> 1 & 1, err, LA_KV8_TIMEOUT));
                                if (!ok) break;
                                tc_fence_after();
                                for (int q = 0; q < HD / 16; ++q) {
                                    uint32_t o[16];
                                    tmem_ld_32x32b_x16(to + 16 * q, o);
                                    tmem_ld_wait_for(o);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                    tmem_st_32x32b_x16(to + 16 * q, o);
                                }
                            }
                            tmem_st_wait();
                        }
                        uint32_t w[16];
                        uint64_t s0 = 0, s1 = 0;   // pairs of sums
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float x = ex2(__uint_as_float(v[2 * e])), y = ex2(__uint_as_float(v[2 * e + 1]));
                            uint64_t &sum = e & 1 ? s1 : s0;
                            sum = add2_f32(sum, pair(x, y));
                            w[e] = pack_f16(x, y);
                        }
                        const float2 sum = halves(add2_f32(s0, s1));
                        l += (sum.x + sum.y) * ex2(fminf(-ux, 126.f));   // a far group: 0
                        tmem_st_32x32b_x16(ts + 16 * k, w);
                    }
                    if (!ok) break;
                    if (l < 0.f) r = keep.own_r, d = keep.own_d, l = keep.own_l, qf = qfs[row];   // behind own_scores
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_one(p_full(b));
            }
            it = end;
            if (!ok) break;
            float fa = 0.f, fb = 0.f, R = r, D = d, L = l;
            [[maybe_unused]] bool nan_old = false;
            if (first < end) {
                // Both groups' maxima and sums, once all products are done; then
                // each group writes half of the dims.
                tmem_st_four(ts + kTileK / 2, r, d, l);
                tmem_st_wait();
                tc_fence_before();
                if (lane == 0 && (warp & 3) == 0) odds[grp] = odd;
                __syncwarp();
                if (lane == 0) mbar_arrive_one(e_full);
                ok = bar_wait(e_full, units & 1, err, LA_KV8_TIMEOUT) &&
                     bar_wait(o_full((end - 1) & 1), (end - 1) >> 1 & 1, err, LA_KV8_TIMEOUT) &&
                     (end - first < 2 || bar_wait(o_full(end & 1), (end - 2) >> 1 & 1, err, LA_KV8_TIMEOUT));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                ++units;
                const float4 x = tmem_ld_four(tmem + lanes + kColS + kTileK / 2), y = tmem_ld_four(tmem + lanes + kColS + 128 + kTileK / 2);
                odd = (odds[0] | odds[1]) != 0;
                if constexpr (WIN) {
                    ok = __all_sync(0xffffffffu, bar_wait(n_full((units - 1) & 3), (units - 1) >> 2 & 1, err, LA_KV8_TIMEOUT));
                    if (!ok) break;
                    for (int k = 0; k < kOpWarps; ++k) nan_old |= nans[((units - 1) & 3) * kOpWarps + k] != 0;
                }
                // a group that saw no key (a sum of 0) may have an O that was never written
                const bool xs = x.z != 0.f, ys = y.z != 0.f;
                R = fmaxf(x.x, y.x);
                D = !xs ? y.y : !ys ? x.y : fmaxf(x.y, y.y);
                L = (xs ? x.z * ex2(x.x - R) : 0.f) + (ys ? y.z * ex2(y.x - R) : 0.f);
                fa = xs ? ex2((x.x - R) + (x.y - D)) : -1.f;
                fb = ys ? ex2((y.x - R) + (y.y - D)) : -1.f;
            } else {
                fa = fb = -1.f;
            }
            if (idle) continue;
            const float inv = L == 0.f ? 0.f : ex2(D) / L;
            const int slot = 2 * blockIdx.x + (u.begins ? 1 : 0), d0 = grp * (HD / 2);
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) + (sq.first + myrow) * p.a.out_stride + myhead * HD + d0;
            float *part = p.part + (static_cast<long long>(slot) * kTileQ + row) * HD + d0;
#pragma unroll 1
            for (int k = 0; k < HD / 32; ++k) {   // 16 dims at a time
                uint32_t oa[16], ob[16];
                float o[16];
                __syncwarp();
                if (first < end) {
                    tmem_ld_32x32b_x16(tmem + lanes + kColO + d0 + 16 * k, oa);
                    tmem_ld_32x32b_x16(tmem + lanes + kColO + 128 + d0 + 16 * k, ob);
                    tmem_ld_wait_for(oa);
                    tmem_ld_wait_for(ob);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = (fa == -1.f ? 0.f : fa * __uint_as_float(oa[e])) + (fb == -1.f ? 0.f : fb * __uint_as_float(ob[e]));
                if (odd && in) {   // NaN and infinities of the new rows that this row sees
#pragma unroll 1
                    for (int r = u.k0 * kTileK; r < min(sq.rows, min(u.k1, sq.ntiles) * kTileK); ++r) {
                        const bool seen = WIN ? kv8_window_new(p, sq.first, sq.rows, sq.len, myrow, r & ~31) >> (r & 31) & 1u : p.a.vis ? r < 256 && (p.a.vis[(static_cast<long long>(sq.first) + myrow) * 8 + r / 32] >> (r % 32) & 1u) : r <= myrow;
                        if (!seen) continue;
                        const __nv_bfloat16 *vr = static_cast<const __nv_bfloat16 *>(p.a.v) + (sq.first + r) * p.a.v_stride + u.head * HD + d0 + 16 * k;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float x = __bfloat162float(vr[e]);
                            if (!is_finite(x)) o[e] += x;
                        }
                    }
                }
                if constexpr (WIN) {
                    if (nan_old && in) {   // and those of cached tokens at the window's edges
#pragma unroll 1
                        for (int kt = max(u.k0, sq.ntiles); kt < u.k1; ++kt) {
                            const int key0 = kv8_tile<WIN>(sq, kt - sq.ntiles) * kTileK;
                            if (!kv8_edge(p, sq, (u.qv0 + u.nqv - 1) / p.gq, key0, kTileK)) continue;
#pragma unroll 1
                            for (int key = key0; key < min(sq.len, key0 + kTileK); ++key) {
                                if (key >= p.sinks && key < from) continue;
                                const int page = c.table[static_cast<long long>(u.s) * c.max_pages + (key >> p.page_log2)];
                                if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.n_pages)) continue;
                                const uint8_t *vb = static_cast<const uint8_t *>(c.v) + kv8_block(c, p.a.layer, page, u.head) * (c.page * HD) +
                                                    static_cast<long long>(d0 + 16 * k) * c.page + (key & (c.page - 1));
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if ((vb[e * c.page] & 0x7f) == 0x7f) o[e] = NAN;
                            }
                        }
                    }
                }
                if (in && u.all) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t y[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(o[8 * e + 2 * q] * inv, o[8 * e + 2 * q + 1] * inv);
                            y[q] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                        *reinterpret_cast<uint4 *>(out + 16 * k + 8 * e) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                } else if (in) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4 *>(part + 16 * k + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
            if (!u.all && in && grp == 0) *reinterpret_cast<float4 *>(p.part_ml + (static_cast<long long>(slot) * kTileQ + row) * 4) = make_float4(R, D, L, 0.f);
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kColAll);
    }
}

// ------------------------------------------------------------------ join
// A unit that several workers share: worker ranges are contiguous, so the
// unit's pieces are those of consecutive workers, the first in its slot 1
// (the piece begins the unit), the others in their slot 0.  One CTA per border
// between workers; the borders inside a unit share its query vectors.  An item
// (4 dims of a row) is added up in a fixed order, by as many lanes as the pieces
// ask for and the items leave.  BATCH loads are in flight: 4 behind k_kv8_rows (64
// sequences, 8 KV heads: 95.0 us against 97.7 with 8), 8 behind k_kv8_tiles, whose
// units have many rows (121 rows of 32 heads: 31.5 us against 35.0 with 4).
constexpr int kJoinThreads = 512;

template <int HD, int BATCH>
__global__ void __launch_bounds__(kJoinThreads) k_kv8_join(const __grid_constant__ Kv8Args p) {
    pdl_trigger();
    pdl_wait();
    const int border = blockIdx.x + 1;
    const Kv8Split x = p.split[border];
    if (!x.inside) return;
    // First and last worker with a piece: the largest with a share that begins
    // at t0 + snap at most, and before t1.
    const long long total = x.total, workers = kv8_workers(p, total);
    const int w0 = static_cast<int>(kv8_div((x.t0 + p.snap + 1) * workers + total - 1, total)) - 1;
    const int w1 = static_cast<int>(min(kv8_div(x.t1 * workers + total - 1, total), workers)) - 1;
    // The border's share of the unit's items (4 dims of a row), `group` lanes for
    // each: the pieces in turn, BATCH loads in flight, then among the lanes.
    const int items = x.nqv * (HD / 4), share = border - w0 - 1, shares = w1 - w0;
    const int i0 = items * share / shares, n = items * (share + 1) / shares - i0;
    int group = 1;
    while (group < 8 && group * BATCH < shares + 1 && 2 * group * n <= kJoinThreads) group <<= 1;
#pragma unroll 1
    for (int j = threadIdx.x; (j & ~31) < n * group; j += kJoinThreads) {
        const bool on = j < n * group;
        const int i = i0 + (on ? j / group : 0), first = w0 + j % group, r = i / (HD / 4), d = 4 * (i % (HD / 4));
        float4 rdl = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);   // r, d, L so far
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float4 &y, const float4 &v) {   // y.z != 0: a piece that saw a key
            const float R = fmaxf(rdl.x, y.x), D = fmaxf(rdl.y, y.y), e0 = rdl.x - R, e1 = y.x - R;
            const float f0 = ex2(e0 + (rdl.y - D)), f1 = ex2(e1 + (y.y - D));
            acc.x = acc.x * f0 + v.x * f1;
            acc.y = acc.y * f0 + v.y * f1;
            acc.z = acc.z * f0 + v.z * f1;
            acc.w = acc.w * f0 + v.w * f1;
            rdl = make_float4(R, D, rdl.z * ex2(e0) + y.z * ex2(e1), 0.f);
        };
#pragma unroll 1
        for (int w = first; on && w <= w1; w += BATCH * group) {
            float4 ml[BATCH];
            float4 v[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int ww = min(w + b * group, w1);
                const long long rec = static_cast<long long>(2 * ww + (ww == w0 ? 1 : 0)) * p.q_tile + r;
                ml[b] = *reinterpret_cast<const float4 *>(p.part_ml + rec * 4);
                v[b] = *reinterpret_cast<const float4 *>(p.part + rec * HD + d);
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
                if (w + b * group <= w1 && ml[b].z != 0.f) add(ml[b], v[b]);
        }
#pragma unroll 1
        for (int o = 1; o < group; o <<= 1) {
            const float4 y = make_float4(__shfl_xor_sync(0xffffffffu, rdl.x, o), __shfl_xor_sync(0xffffffffu, rdl.y, o), __shfl_xor_sync(0xffffffffu, rdl.z, o), 0.f);
            const float4 v = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, o), __shfl_xor_sync(0xffffffffu, acc.y, o),
                                         __shfl_xor_sync(0xffffffffu, acc.z, o), __shfl_xor_sync(0xffffffffu, acc.w, o));
            if (y.z != 0.f) add(y, v);
        }
        if (!on || j % group != 0) continue;
        const float inv = rdl.z == 0.f ? 0.f : ex2(rdl.y) / rdl.z;
        const int qv = x.qv0 + r;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) + (x.first + qv / p.gq) * p.a.out_stride + (x.head * p.gq + qv % p.gq) * HD + d;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(out) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
}

// ------------------------------------------------------------------ launch
// What a unit costs beside its key tiles, in tiles.  k_kv8_rows: 64 sequences of up
// to 8192 tokens, 8 KV heads: 119.0 us with 4, 99.4 with 10, 95.4 with 13, 95.3
// with 16, 98.8 with 26; 48 of up to 1500, head_dim 64, 4 KV heads: 20.5 with 4,
// 16.4 with 13, 17.4 with 26.  k_kv8_tiles counts 4, and of long units a tenth up to
// 12: with 4, 8 and 12 256 rows, 8 KV heads, take over 16k tokens 114.4, 113.1 and
// 110.2 us, over 8k 76.9, 74.2 and 79.5; 121 rows of 32 heads over 4k 33.5, 36.4 and
// 36.5 (with so few tiles for each CTA a wide count only moves the borders).
constexpr int kRowsUnitCost = 14, kTilesUnitCost = 4;
constexpr int kRowsPerSm = 4;   // most CTAs of k_kv8_rows per SM

int64_t kv8_workspace_bytes(const la_kv8_cache &c, int nsm) {
    const int64_t part = static_cast<int64_t>(nsm) * std::max(kRowsPerSm * kRowsQ, kTileQ) * 2 * (c.head_dim + 4) * 4;
    const int64_t splits = static_cast<int64_t>(nsm) * kRowsPerSm * sizeof(Kv8Split);
    const int64_t plans = (std::max<int64_t>(6ll * c.n_seqs + c.n_pages, 4ll * c.n_pages) + 16) * 4;
    return (std::max(part + splits, plans) + 255) / 256 * 256;
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

// Units of the call, at most, if max_rows holds.  Where it is given, a sequence
// with that many rows leaves the others n_rows - max_rows: slots without rows
// do not count (one row of 32 heads in one of 2048 slots: 2995 us when they did,
// as units by the ten thousand kept the real ones whole).
static long long unit_bound(const Kv8Args &p) {
    const long long qt = p.q_tile, slots = std::min<long long>(p.c.n_seqs, p.hinted ? 1 + p.a.n_rows - p.a.max_rows : p.a.n_rows);
    const long long all = (static_cast<long long>(p.a.n_rows) * p.gq + (qt - 1) * slots) / qt;
    return std::min(all, (static_cast<long long>(p.a.max_rows) * p.gq + qt - 1) / qt * slots) * p.c.n_kv_heads;
}

// Units are split where that saves more than `cost` tiles' time: a split costs the
// join's kernel and the pieces' way through memory.  Units of more than `most` tiles
// always: where the lengths differ, whole ones leave SMs idle at the end.
static bool keep_whole(const Kv8Args &p, long long units, long long tiles, int cost, int most) {
    const long long rounds = (units + p.workers - 1) / p.workers;
    return tiles <= most && rounds * tiles - units * (tiles + p.unit_cost) / p.workers <= cost;
}

// FEW: k_kv8_few, of 8 query vectors a unit, else k_kv8_rows, of 16.
template <int HD, int PAGE, bool WIN, bool FEW>
static cudaError_t rows_launch(Kv8Args &p, int nsm, void *ws, cudaStream_t s) {
    using Lay = std::conditional_t<FEW, Few<HD, PAGE>, Rows<HD, PAGE>>;
    const auto kernel = [] {
        if constexpr (FEW) return k_kv8_few<HD, PAGE>;
        else return k_kv8_rows<HD, PAGE, WIN>;
    }();
    static_assert(Lay::per_sm <= kRowsPerSm, "workspace");
    p.q_tile = FEW ? kFewQ : kRowsQ;
    p.q_log2 = FEW ? 3 : 4;
    p.k_tile = PAGE;
    p.k_log2 = p.page_log2;
    static_assert(kRowsQ == 1 << 4 && kFewQ == 1 << 3, "shift");
    p.n_tile = 0;
    p.unit_cost = kRowsUnitCost;
    p.snap = p.unit_cost - 1;
    // Whole against split: one row of 64 heads over 8 KV heads, pages of 64, 13
    // tiles 13.1 us against 11.3, 19 tiles 14.8 against 11.5; 16 such sequences 19
    // tiles 17.7 against 19.7, 32 tiles 24.4 against 22.5; 48 sequences, head_dim
    // 64, 4 KV heads, pages of 32, 16 tiles 10.7 against 13.5, 47 tiles 19.6
    // against 16.4.
    // k_kv8_few counts tokens, as its six warps take pages of any size at about the same rate:
    // units of up to 2304 stay whole where that costs less than 896 tokens' time.
    // Whole against split, windows of 512, 1024 and 2048: one row of 64 heads over 8 KV heads, pages
    // of 64 8.9, 11.3, 16.4 against 11.1, 11.4, 11.6, pages of 128 9.2, 11.7, 15.7 against 12.0, 12.1,
    // 12.5; of 32 heads over 4, pages of 32 9.3, 13.1, 20.8 against 10.5, 11.2, 11.5; 16 sequences, pages of
    // 64 10.8, 13.6, 20.3 against 14.8, 16.6, 19.6; 64 of them 22.0, 33.0, 51.6 against 26.9, 37.3,
    // 55.7; 48, head_dim 64, 4 KV heads, pages of 32 9.2, 12.8, 19.2 against 14.5, 17.0, 20.5.  A window
    // of 4096, different lengths: 64 sequences 76.2 against 77.8, 32 with pages of 128 53.6 against
    // 51.0.  A unit_cost of 8 or 22 does neither better nor worse than 14.
    constexpr int kCost = FEW ? 896 / PAGE : 8, kMost = FEW ? 2304 / PAGE : 32;
    const long long tiles = (p.a.max_len + PAGE - 1) / PAGE;
    p.workers = nsm * Lay::per_sm;
    if (keep_whole(p, unit_bound(p), tiles, kCost, kMost)) p.whole = 1, p.workers = static_cast<int>(std::min<long long>(unit_bound(p), 1 << 20));
    p.part = static_cast<float *>(ws);
    p.part_ml = p.part + static_cast<long long>(nsm) * kRowsPerSm * 2 * kRowsQ * HD;
    p.split = reinterpret_cast<Kv8Split *>(p.part_ml + static_cast<long long>(nsm) * kRowsPerSm * 2 * kRowsQ * 4);
    static std::atomic<unsigned long long> configured{0};
    unsigned long long bit = 0;
    if (attrs_needed(configured, &bit)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(Lay::bytes(LA_KV8_MAX_SEQS)));
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    cudaError_t e = launch_k(kernel, dim3(p.workers), dim3(32 * Lay::warps), Lay::bytes(p.c.n_seqs), s, p);
    if (e != cudaSuccess || p.whole) return e;
    if (p.workers < 2) return cudaSuccess;
    return launch_k(k_kv8_join<HD, 4>, dim3(p.workers - 1), dim3(kJoinThreads), 0, s, p);
}

template <int HD, bool WIN>
static cudaError_t tiles_launch(Kv8Args &p, int nsm, void *ws, cudaStream_t s) {
    using Lay = Tiles<HD>;
    p.q_tile = kTileQ;
    p.k_tile = p.n_tile = kTileK;
    p.q_log2 = p.k_log2 = 7;
    static_assert(kTileQ == 1 << 7 && kTileK == 1 << 7, "shift");
    p.snap = 0;   // finding the unit costs more than an empty piece (121 rows over 2k tokens, 32 heads: 34.4 us against 33.1)
    // Whole against split: 121 rows of 32 heads, 6 tiles 24.2 us against 25.4, 9
    // tiles 29.9 against 25.4; four such sequences, which fill the SMs whole, 12
    // tiles 35.7 against 57, 25 tiles 58.5 against 73, and 33 tiles of 8 sequences
    // with 160 query vectors for each of 8 KV heads 62.8 against 73.8.
    const long long tiles = (p.a.max_len + kTileK - 1) / kTileK + (p.a.k ? (p.a.max_rows + kTileK - 1) / kTileK : 0);
    p.unit_cost = static_cast<int>(std::min<long long>(std::max<long long>(tiles / 10, kTilesUnitCost), 3 * kTilesUnitCost));
    p.workers = nsm;
    if (keep_whole(p, unit_bound(p), tiles, 5, 64)) p.whole = 1, p.workers = static_cast<int>(std::min<long long>(unit_bound(p), 1 << 20));
    p.part = static_cast<float *>(ws);
    p.part_ml = p.part + static_cast<long long>(nsm) * 2 * kTileQ * HD;
    p.split = reinterpret_cast<Kv8Split *>(p.part_ml + static_cast<long long>(nsm) * 2 * kTileQ * 4);
    static std::atomic<unsigned long long> configured{0};
    unsigned long long bit = 0;
    if (attrs_needed(configured, &bit)) {
        cudaError_t e = cudaFuncSetAttribute(k_kv8_tiles<HD, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(Lay::bytes(LA_KV8_MAX_SEQS, WIN)));
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    cudaError_t e = launch_k(k_kv8_tiles<HD, WIN>, dim3(p.workers), dim3(kTileThreads), Lay::bytes(p.c.n_seqs, WIN), s, p);
    if (e != cudaSuccess || p.whole || p.workers < 2) return e;
    return launch_k(k_kv8_join<HD, 8>, dim3(p.workers - 1), dim3(kJoinThreads), 0, s, p);
}

// Query vectors per sequence and KV head up to which k_kv8_rows is used (k_kv8_rows
// against k_kv8_tiles: 8 sequences of 4000 tokens, 8 KV heads, 16 vectors 22.7 us
// against 36.9, 32 vectors 31.8 against 38.3, 48 vectors 41.1 against 40.9, 64
// vectors 50.6 against 42.1; one of 2000 tokens, 32 KV heads, 64 vectors 32.7
// against 24.0).
constexpr int kFewVectors = 32;

template <int HD, bool WIN>
static cudaError_t attention_launch_hd(Kv8Args &p, int nsm, void *ws, cudaStream_t s) {
    if (static_cast<long long>(p.a.max_rows) * p.gq > kFewVectors) return tiles_launch<HD, WIN>(p, nsm, ws, s);
    if constexpr (WIN) {
        if (static_cast<long long>(p.a.max_rows) * p.gq <= kFewQ) {
            if (p.c.page == 32) return rows_launch<HD, 32, WIN, true>(p, nsm, ws, s);
            if (p.c.page == 64) return rows_launch<HD, 64, WIN, true>(p, nsm, ws, s);
            return rows_launch<HD, 128, WIN, true>(p, nsm, ws, s);
        }
    }
    if (p.c.page == 32) return rows_launch<HD, 32, WIN, false>(p, nsm, ws, s);
    if (p.c.page == 64) return rows_launch<HD, 64, WIN, false>(p, nsm, ws, s);
    return rows_launch<HD, 128, WIN, false>(p, nsm, ws, s);
}

cudaError_t kv8_attention_launch(const la_kv8_cache &c, const la_kv8_attn &a, int window, int sinks, void *ws, int nsm, cudaStream_t s,
                                 int64_t *launched) {
    if (a.n_rows < 1) return cudaSuccess;
    Kv8Args p{};
    p.c = c;
    p.a = a;
    const int room = c.max_pages * c.page;
    p.hinted = !a.row_start || (a.max_rows > 0 && a.max_rows <= a.n_rows);
    if (!a.row_start) p.a.max_rows = 1;
    else if (!p.hinted) p.a.max_rows = a.n_rows;
    if (a.max_len <= 0 || a.max_len > room) p.a.max_len = room;
    p.gq = a.n_heads / c.n_kv_heads;
    p.page_log2 = c.page == 32 ? 5 : c.page == 64 ? 6 : 7;
    p.scale_log2 = a.scale * kKv8Log2e;
    // What a slot's rows see together, at most; a window as long as every list is none.
    const bool win = window > 0 && window < static_cast<int64_t>(room) + a.n_rows;
    if (win) {
        p.window = window;
        p.sinks = sinks;
        p.a.max_len = static_cast<int>(std::min<int64_t>(p.a.max_len, static_cast<int64_t>(window) + sinks + p.a.max_rows + 128));
    }
    const cudaError_t e = c.head_dim == 128 ? (win ? attention_launch_hd<128, true>(p, nsm, ws, s) : attention_launch_hd<128, false>(p, nsm, ws, s))
                                            : (win ? attention_launch_hd<64, true>(p, nsm, ws, s) : attention_launch_hd<64, false>(p, nsm, ws, s));
    if (launched) *launched += p.whole ? 1 : 2;
    return e;
}

}  // namespace la
