// mx_attn_tc.cu -- attention over the paged cache on the tensor cores
// (tcgen05), heads of 64 or 128, sm_103a.
//
//   S = Q K^T,  P = 2^(scale log2(e) S - m),  O = P V,  out = O / sum P
//
// One persistent CTA per SM.  A row tile is 128 rows of (token, query head)
// that share a cache head, a key tile 128 keys.  Two groups of four warps each
// own one accumulator pair (S, O) in tensor memory; a thread owns a row, so
// the softmax needs no shuffles.  What the two groups work on goes by the
// item at hand:
//   rows  (more than one row tile of new tokens): two row tiles over the same
//         keys, each key tile read once for 256 rows;
//   keys  (few tokens, e.g. one per sequence): the same row tile over
//         alternate key tiles, merged at the end; the context streams through
//         shared memory once.
// While one group computes its softmax the tensor cores work for the other.
// P is written over its S in tensor memory as bf16 and is operand A of the
// second product from there; V is its operand B as it lies in the cache
// (keys x dimensions, i.e. N-major).
//
// The maximum that P is taken against is only raised when a row's scores
// outgrow it by 2^8 (the sums stay far inside fp32 and are exact ratios
// either way): O then is rescaled in tensor memory by the row's own threads.
//
// Work is cut by cost, not by item: the (sequence, cache head, row tiles)
// items laid end to end, each as long as the keys it sees, are divided into
// equal stretches, one per CTA, so that any mix of prompts and single tokens
// loads every SM the same.  An item cut across CTAs leaves partial (m, l, O)
// rows in the workspace and the last CTA to arrive adds them in order.  Few
// and short items are not cut (AT_WHOLE_KEYS).
//
// P is rounded to bf16 because the tensor cores take their operands so: each
// weight is off by up to 2^-8 of itself, as the values of a bf16 cache are already, and
// the sum that divides them is of the unrounded weights.  64 heads on 8 of 128:
//   prompt of 4096 on 8192     590 us  1.40 PFLOP/s, 73 % of the measured rate
//                                      (581 to 597; 548 where few calls run)
//   64 tokens on 0.5-8 K       181 us  6.3 TB/s, 95 % of the measured copy
//   16 x 2-6 tokens on 1-16 K  105 us  5.8 TB/s
//   one token on 131 keys        9 us  a chain of latencies
//   MXFP8, 5 tokens on 24-66 K 211 us  the decode to bf16
// A prompt is bound by the softmax between two MMAs of a group (tensor cores
// busy 54 % of the time, as the MMAs' own rate goes), single tokens by HBM.
//
//   warps 0-3, 4-7  softmax groups and epilogue
//   warp 9          MMA issuer
//   warp 10         TMA producer (queries, keys, values); not on the SM's first
//                   quarter, whose softmax warps have the rows when there are few
//                   (verification 122 -> 113 us against warp 8)
//   warps 11-18     MXFP8 cache only: decoders.  The codes and scales of a tile
//                   land in a ring of their own and are decoded exactly to the
//                   bf16 tiles that the MMAs read, as in the prefill GEMM.
//                   (The other warps only fill up the warpgroups.)
//
// Every wait is bounded as in the GEMMs; a CTA whose wait gives up makes its
// outputs NaN and sets MX_DEVERR_TIMEOUT.
#include "mx_attn.cuh"
#include "mx_decode_bf16.cuh"
#include "mx_tc.cuh"

namespace mx {

constexpr int AT_ROWS = 128;  // rows of a tile
constexpr int AT_KEYS = 128;  // keys of a tile
// What an item costs beside its keys, and more than its tiles' rounding: its
// queries, epilogue and the cuts (4, 2, 6 tiles, 64 heads on 8 x 128 bf16, us:
// 16 x 1-200 tokens on 0.1-4 K 126, 168, 127; 64 tokens on 50-2000 62, 72, 62,
// in MXFP8 87, 90, 90; 124, 62 and 89 now).
constexpr int AT_SPLIT_KEYS = 4 * AT_KEYS;
// Up to so many tokens' queries are copied one by one, of more the whole row tile
// (32 sequences on 1024: 2 tokens each 35.0 us, 34.9 as a tile, but a call of so few
// tokens need not encode the tile's copy; 8 tokens each 35.9 as a tile, 36.8 one by one).
constexpr int AT_Q_COPIES = 4;
// Whether an item of n tokens takes whole row tiles of queries, of s1 tokens each:
// always where it needs two of them, which is from two tokens on in wide groups.  The
// host encodes the copies by the call's tokens, which no item outnumbers.
__host__ __device__ constexpr bool at_whole_tiles(int n, int s1) { return n > AT_Q_COPIES || n > s1; }
// Items of up to so many keys are not cut when there is a CTA for each; more when
// they have two row tiles, whose parts cost more to add up.  Uncut against cut,
// 64 on 8 heads x 128 bf16, us: one token on 512 keys 9.4, 12.9; on 1024 13.6,
// 13.3; on 1500 20.0, 13.4; 16 sequences of 50 to 1000 keys 18.0, 23.5; prompts:
// 512 on 512 17.0, 31.8; 2 x 128 on 1500 28.5, 43.5; 32 on 2000 32.3, 35.2
// (MXFP8 44.3, 40.3).
constexpr int AT_WHOLE_KEYS = 8 * AT_KEYS, AT_WHOLE_KEYS_2 = 16 * AT_KEYS;
// Shortest stretch of a CTA that only divides an item (one token on 1500 keys
// 13.8 us; with 4 tiles 15.5, with 6 17.9; on 8192 19.7, 17.8, 19.6).
constexpr int AT_MIN_KEYS = 3 * AT_KEYS;
constexpr int AT_RING = 3;                  // pieces the producer may run ahead by
// log2 by which scores may outgrow the maximum before it is raised (0: the
// prompt of 4096 on 8192 takes 782 us instead of 560)
constexpr float AT_RAISE = 8.0f;
constexpr unsigned long long AT_WAIT_NS = 2000000000ull;

template <int D, int KVF>
struct AtGeo {
    static constexpr bool MX8 = KVF == KV_MXFP8;
    static constexpr int THREADS = MX8 ? 640 : 384;
    // registers: what the launch gives each thread (168, 96), shared out again
    // between the softmax warps and the others (on each of the SM's quarters two,
    // and one or three)
    static constexpr int R_SOFTMAX = MX8 ? 144 : 208, R_OTHER = MX8 ? 64 : 88;
    static_assert(2 * R_SOFTMAX + (MX8 ? 3 : 1) * R_OTHER <= (MX8 ? 5 * 96 : 3 * 168), "register split");
    static constexpr int SLABS = D / 64;                    // 128-byte swizzled slabs of 64 dimensions
    static constexpr int SLAB = 128 * 128;                  // bytes of a slab: 128 rows x 128 bytes
    static constexpr int TILE = SLABS * SLAB;               // bytes of a row tile or a bf16 key tile
    static constexpr int SLOTS = MX8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 11);  // bf16 key/value tiles
    // MXFP8: ring of packed tiles, codes [128][D] then scales [128][D / 32]
    static constexpr int CODES = 128 * D, SCALES = 128 * (D / 32);
    static constexpr int C_SLOTS = MX8 ? (D == 128 ? 3 : 8) : 1;
    static constexpr int DECODERS = 8;                      // warps
    static constexpr int UNITS = D / 8;                // warp-sized parts of a tile's decode
    static constexpr int OFF_KV = 2 * TILE;                 // after two row tiles
    static constexpr int OFF_C = OFF_KV + SLOTS * TILE;
    static constexpr int OFF_SC = OFF_C + (MX8 ? C_SLOTS * CODES : 0);
    static constexpr int OFF_BAR = OFF_SC + (MX8 ? C_SLOTS * SCALES : 0);
    static constexpr int CTRL = 3072;                       // control block
    static constexpr int SMEM = OFF_BAR + CTRL;
    static_assert(2 * SLOTS + (MX8 ? 2 * C_SLOTS : 0) <= 28, "barriers");
    // tensor memory columns
    static constexpr int S_COL = 0, O_COL = 256;
    static_assert(SMEM <= 232448, "shared memory");
};

struct AtParams {
    AttnArgs a;
    int *counters;      // 2 per CTA, zero between calls
    float *partials;    // see partial_base
    int part_rows;      // rows a partial has room for
    int page_rows;      // rows of a TMA copy: min(page_size, 128)
    unsigned long long wait_ns;
    int out32;          // out is 32-byte aligned
    int stall;          // test hook: load no queries
};

// ------------------------------------------------------------ work

// What a sequence's items cost: an item is (cache head, pair of row tiles).
struct Seq {
    int q0, n, len;   // first token row, new tokens, context
    int pairs;        // items per cache head
};

__device__ __forceinline__ long long sum_range(long long a, long long s, long long lo, long long hi)
{
    // sum of a + i s for lo <= i < hi
    const long long n = hi - lo;
    return n <= 0 ? 0 : n * a + s * ((lo + hi - 1) * n / 2);
}

// Sum over i < p of max(a + i s, 0).
__device__ __forceinline__ long long sum_pos(long long a, long long s, long long p)
{
    if (a >= 0) return sum_range(a, s, 0, p);
    const uint32_t x = (uint32_t)min(-a, 0xFFFFFFFFll), z = x / (uint32_t)s + (x % (uint32_t)s != 0);
    return sum_range(a, s, z, p);
}

struct Cost {
    int s2;             // tokens of a pair of row tiles
    int causal, window;
    int heads;          // cache heads
    int flat;           // every item costs AT_SPLIT_KEYS: one CTA each

    // Keys before which items p, p + 1, ... of a head start (each item's own
    // keys and AT_SPLIT_KEYS): items see [lo(p), hi(p)).
    __device__ __noinline__ long long before(const Seq q, int p) const  // (one copy, for the instruction cache)
    {
        if (flat) return (long long)p * AT_SPLIT_KEYS;
        const long long base = (long long)q.len - q.n;
        long long h = (long long)p * q.len, l = 0;
        if (causal) {
            h = sum_pos(base + s2, s2, p);
            if (p == q.pairs) h -= max(0ll, base + (long long)p * s2 - q.len);
        }
        if (window > 0) l = sum_pos(base - window + 1, s2, p);
        return h - l + (long long)p * AT_SPLIT_KEYS;
    }
    __device__ __forceinline__ void range(const Seq &q, int p, int &lo, int &hi) const
    {
        const long long base = (long long)q.len - q.n;
        hi = causal ? (int)max(0ll, min((long long)q.len, base + (p + 1ll) * s2)) : q.len;
        lo = window > 0 ? (int)max(0ll, base + (long long)p * s2 - window + 1) : 0;
        if (lo > hi) lo = hi;
    }
    __device__ __forceinline__ long long total(const Seq &q) const
    {
        return q.pairs > 0 ? before(q, q.pairs) * heads : 0;
    }
};

__device__ __forceinline__ Seq load_seq(const AttnArgs &a, int b, int s1)
{
    Seq q;
    const int e0 = min(max(__ldg(a.q_start + b), 0), a.T), e1 = min(max(__ldg(a.q_start + b + 1), e0), a.T);
    q.q0 = e0;
    q.n = e1 - e0;
    q.len = max(__ldg(a.kv_len + b), 0);
    q.pairs = (q.n + 2 * s1 - 1) / (2 * s1);
    return q;
}

// The first sequence from b on that has new tokens (B: none), by the whole warp, 32 at
// a time: a batch may have many unused slots (one token in 4096 slots: 797 us one
// by one, 39 so).
__device__ __forceinline__ int next_with_tokens(const AttnArgs &a, int b)
{
    for (; b < a.B; b += 32) {
        const int i = b + (threadIdx.x & 31);
        const unsigned some = __ballot_sync(0xFFFFFFFFu, i < a.B && __ldg(a.q_start + i + 1) > __ldg(a.q_start + i));
        if (some != 0) return b + __ffs(some) - 1;
    }
    return a.B;
}

// A CTA's stretch of the work, found once per launch.
struct Stretch {
    long long total, start, end;  // cost
    long long at;                 // cost before the first item
    int b, kvh, p;                // the first item (b = B: none)
    int ctas;
    int flat;  // as the cost's
};

// One piece: key tiles [k0, k1) of an item.
struct Piece {
    int b, kvh;
    int q0, ntok;       // first token row of the item and its tokens
    int first;          // position in the context of its first token
    int len;            // context
    int lo, hi;         // keys any of its rows may see
    int tile0;          // key tile lo lies in
    int k0, k1, tiles;  // this piece's tiles, relative to tile0, and the item's
    int rows;           // two row tiles (else alternate key tiles)
    int c0, c1;         // CTAs the item is cut across
    int end;            // no piece: the stretch is done
};

// Walks a CTA's pieces.
struct Walk {
    const AttnArgs &a;
    const Stretch &st;
    Cost cost;
    int s1;  // tokens of a row tile
    Seq q;
    int b, kvh, p;
    long long at;  // cost before the item

    __device__ __forceinline__ Walk(const AttnArgs &args, const Stretch &stretch, const Cost &c)
        : a(args), st(stretch), cost(c), s1(c.s2 / 2), b(stretch.b), kvh(stretch.kvh), p(stretch.p), at(stretch.at)
    {
        if (b < a.B) q = load_seq(a, b, s1);
    }
    // The CTA whose stretch holds cost x: the last c with total c / ctas <= x,
    // guessed in fp32 and set right exactly.
    __device__ __forceinline__ int cta_of(long long x) const
    {
        const long long lim = (x + 1) * st.ctas - 1;
        int c = (int)((float)x * (float)st.ctas / (float)st.total);
        while (st.total * c > lim) --c;
        while (st.total * (c + 1) <= lim) ++c;
        return c;
    }
    __device__ __forceinline__ bool next(Piece &o)
    {
        for (;;) {
            if (at >= st.end) return false;
            if (kvh >= cost.heads) {  // the sequence is done
                b = next_with_tokens(a, b + 1);
                kvh = 0;
                if (b < a.B) q = load_seq(a, b, s1);
            }
            if (b >= a.B) return false;
            cost.range(q, p, o.lo, o.hi);
            o.tile0 = o.lo / AT_KEYS;
            o.tiles = o.hi > o.lo ? (o.hi - 1) / AT_KEYS + 1 - o.tile0 : 0;  // (hi: up to 2^31 - 1)
            // tile k begins at cost at + 128 k and is its CTA's whose stretch holds that
            o.k0 = st.start <= at ? 0 : (int)min((st.start - at + AT_KEYS - 1) / AT_KEYS, (long long)o.tiles);
            o.k1 = st.flat ? o.tiles : (int)min((st.end - at + AT_KEYS - 1) / AT_KEYS, (long long)o.tiles);
            o.b = b;
            o.kvh = kvh;
            o.q0 = q.q0 + p * cost.s2;
            o.ntok = min(q.n - p * cost.s2, cost.s2);
            o.first = q.len - q.n + p * cost.s2;
            o.len = q.len;
            o.rows = o.ntok > s1;
            o.c0 = o.c1 = 0;
            if (o.k1 - o.k0 != o.tiles) {
                o.c0 = cta_of(at);
                o.c1 = cta_of(at + (o.tiles - 1ll) * AT_KEYS);
            }
            const bool mine = o.tiles > 0 ? o.k0 < o.k1 : st.start <= at;
            at += (st.flat ? 0 : (long long)(o.hi - o.lo)) + AT_SPLIT_KEYS;
            if (++p >= q.pairs) {
                p = 0;
                ++kvh;
            }
            if (mine) return true;
        }
    }
};

// A CTA's stretch, by one warp (the producer's, which walks it; nobody else waits for
// more than its first piece): the costs of all sequences, 32 at a time, then
// the item that holds the stretch's start.
__device__ __forceinline__ long long warp_sum_before(long long v, long long *total)
{
    const int lane = threadIdx.x & 31;
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += x;
    }
    *total = __shfl_sync(0xFFFFFFFFu, inc, 31);
    return inc - v;
}

__device__ __forceinline__ void plan(const AttnArgs &a, Cost &cost, Stretch &st)
{
    const int lane = threadIdx.x & 31, s1 = cost.s2 / 2;
    int items = 0, over = 0;  // items of this lane's sequences; is one longer than is left whole?
    auto cost_at = [&](int b) {
        if (b >= a.B) return 0ll;
        const Seq q = load_seq(a, b, s1);
        items += min(q.pairs * cost.heads, 1024);
        const long long most = cost.window > 0 ? min((long long)q.len, (long long)cost.window + cost.s2) : q.len;
        over |= q.pairs > 0 && most > (q.n > s1 ? AT_WHOLE_KEYS_2 : AT_WHOLE_KEYS);
        return cost.total(q);
    };
    cost.flat = 0;
    long long c0 = cost_at(lane);  // of the first 32, kept
    long long total, first_total;
    long long before0 = warp_sum_before(c0, &first_total);
    total = first_total;
    if (a.B > 32) {
        long long rest = 0;
#pragma unroll 4
        for (int b = 32 + lane; b < a.B; b += 32) rest += cost_at(b);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xFFFFFFFFu, rest, o);
        total += rest;
    }
    // Few and short items: a CTA for each, uncut.  Else, a CTA for every item or
    // every AT_MIN_KEYS keys, whichever are more, as many to an item as to the
    // next if they are alike.  A stretch is longer than
    // a tile, so no CTA between an item's first and last is left without one.
    const int grid = gridDim.x;
    items = (int)__reduce_add_sync(0xFFFFFFFFu, (unsigned)min(items, 1 << 24));
    int ctas = grid;
    if (!__any_sync(0xFFFFFFFFu, over) && items <= grid) {
        cost.flat = 1;
        ctas = max(items, 1);
        total = (long long)items * AT_SPLIT_KEYS;
        c0 = cost_at(lane);
        before0 = warp_sum_before(c0, &first_total);
    } else if (total < (long long)grid * AT_MIN_KEYS) {
        ctas = max(1, min(grid, max(items, (int)total / AT_MIN_KEYS)));
        if (items > 0 && items < ctas) ctas -= ctas % items;
    }
    st.flat = cost.flat;
    const int c = blockIdx.x;
    st.total = total;
    st.ctas = ctas;
    st.start = st.end = total;
    st.b = a.B;
    if (c >= ctas) return;
    if (total < (1ll << 23)) {  // the usual case: 32-bit division
        st.start = (uint32_t)total * (uint32_t)c / (uint32_t)ctas;
        st.end = (uint32_t)total * (uint32_t)(c + 1) / (uint32_t)ctas;
    } else {
        st.start = total * c / ctas;
        st.end = total * (c + 1) / ctas;
    }
    if (st.start >= st.end) return;
    // the sequence that holds the start
    long long at = before0, mine = c0, sum = first_total, base = 0;
    int b0 = 0;
    while (base + sum <= st.start && b0 < a.B) {
        base += sum;
        b0 += 32;
        mine = cost_at(b0 + lane);
        at = base + warp_sum_before(mine, &sum);
    }
    const unsigned holds = __ballot_sync(0xFFFFFFFFu, at <= st.start && st.start < at + mine);
    if (holds == 0) return;  // (only if the lengths change meanwhile)
    const int src = __ffs(holds) - 1;
    at = __shfl_sync(0xFFFFFFFFu, at, src);
    mine = __shfl_sync(0xFFFFFFFFu, mine, src);
    st.b = b0 + src;
    // its cache head and item
    const Seq q = load_seq(a, st.b, s1);
    const long long head = cost.before(q, q.pairs);  // mine = heads * head
    int kvh = min((int)((float)(st.start - at) / (float)head), cost.heads - 1);
    while (kvh * head > st.start - at) --kvh;
    while ((kvh + 1) * head <= st.start - at) ++kvh;
    at += kvh * head;
    int lo = 0, n = q.pairs;  // the last p with at + before(p) <= start, 32 candidates a round
    while (n > 1) {
        const int step = (n + 31) >> 5, i = lane * step;
        const unsigned le = __ballot_sync(0xFFFFFFFFu, i < n && at + cost.before(q, lo + i) <= st.start);
        const int k = 31 - __clz(le);
        lo += k * step;
        n = min(step, n - k * step);
    }
    st.kvh = kvh;
    st.p = lo;
    st.at = at + cost.before(q, lo);
}

// ------------------------------------------------------------ tensor ops

// What the waits of a CTA watch beside their barrier.
struct Watch {
    int gave_up;  // a wait ran out
    int busy;     // warps that compute rows again (rows_again): over a long context longer than
                  // the limit, which counts from when they are done
};

// mbar_wait without a call: ptxas (13.0) cannot allocate the softmax warps'
// registers past the launch's count across the call of its slow path.
__device__ __forceinline__ bool at_wait(uint64_t *bar, uint32_t parity, volatile Watch *watch,
                                        unsigned long long limit_ns, bool respect_abort = true)
{
    unsigned long long t0 = 0;
#pragma unroll 1
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
        if (__builtin_expect((i & 63u) == 0u, 0)) {
            if (respect_abort && watch->gave_up) return false;
            const unsigned long long t = globaltimer();
            if (t0 == 0 || watch->busy) {
                t0 = t;
            } else if (t - t0 > limit_ns) {
                watch->gave_up = 1;
                return false;
            }
        }
    }
    return true;
}

// A wait of the whole warp, polled by all of it: polled by one lane in a branch
// of its own a prompt took 764 us instead of 585.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile Watch *watch,
                                          unsigned long long limit_ns)
{
    return __all_sync(0xFFFFFFFFu, at_wait(bar, parity, watch, limit_ns)) != 0;
}

// The same for the producer, the MMA issuer and the decoders, whose loops have the
// slow path in a call: the roles share an instruction cache (mixed batch 288 -> 249 us,
// prompt 608 -> 586).  (A lane that has seen the phase complete sees it again: the
// next one does not come before this warp goes on.)
__device__ __noinline__ bool at_wait_call(uint64_t *bar, uint32_t parity, volatile Watch *watch,
                                          unsigned long long limit_ns)
{
    return at_wait(bar, parity, watch, limit_ns);
}

__device__ __forceinline__ bool role_wait(uint64_t *bar, uint32_t parity, volatile Watch *watch,
                                          unsigned long long limit_ns)
{
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xFFFFFFFFu, ok)) ok = __all_sync(0xFFFFFFFFu, at_wait_call(bar, parity, watch, limit_ns)) != 0;
    return ok;
}

__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
                 : "memory");
}

// Operand A in tensor memory.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(at), "l"(bd), "r"(idesc), "r"(acc)
                 : "memory");
}

__device__ __forceinline__ void umma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// bf16 operands, fp32 accumulator, M = 128; B K-major or N-major.
template <int N>
__device__ __forceinline__ constexpr uint32_t at_idesc(bool b_n_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((128u >> 4) << 24);
}

// Shared-memory matrix descriptors, 128-byte swizzle, the 8-row groups 1024
// bytes apart.  Q and K are K-major (sw128_desc); V is operand B as it lies,
// N-major: rows of 64 dimensions (128 bytes), 8 keys every 1024 bytes, the
// next 64 dimensions `lead` bytes further.  The low word holds the address and
// the leading offset, so that a step through a tile is an addition to it.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead)
{
    return ((saddr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}

__device__ __forceinline__ uint64_t desc64(uint32_t lo)
{
    constexpr uint32_t hi = (1024 >> 4) | (1u << 14) | (2u << 29);  // stride, descriptor version, 128-byte swizzle
    return ((uint64_t)hi << 32) | lo;
}

// One lane of the warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "elect.sync _|p, 0xFFFFFFFF;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

#define MX_R32(r, o)                                                                                                  \
    "=r"(r[o + 0]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]),  \
        "=r"(r[o + 7]), "=r"(r[o + 8]), "=r"(r[o + 9]), "=r"(r[o + 10]), "=r"(r[o + 11]), "=r"(r[o + 12]),            \
        "=r"(r[o + 13]), "=r"(r[o + 14]), "=r"(r[o + 15]), "=r"(r[o + 16]), "=r"(r[o + 17]), "=r"(r[o + 18]),         \
        "=r"(r[o + 19]), "=r"(r[o + 20]), "=r"(r[o + 21]), "=r"(r[o + 22]), "=r"(r[o + 23]), "=r"(r[o + 24]),         \
        "=r"(r[o + 25]), "=r"(r[o + 26]), "=r"(r[o + 27]), "=r"(r[o + 28]), "=r"(r[o + 29]), "=r"(r[o + 30]),         \
        "=r"(r[o + 31])

// 32 columns of the thread's lane into r[o..], without waiting.
template <int NR>
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[NR], const int o)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : MX_R32(r, o)
                 : "r"(taddr));
}
#undef MX_R32

// 16 columns.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}

// Keeps uses of r[o..o+31] behind the wait that precedes it.
template <int NR>
__device__ __forceinline__ void pin32(uint32_t (&r)[NR], const int o)
{
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+r"(r[o + i]), "+r"(r[o + i + 1]), "+r"(r[o + i + 2]), "+r"(r[o + i + 3]),
                          "+r"(r[o + i + 4]), "+r"(r[o + i + 5]), "+r"(r[o + i + 6]), "+r"(r[o + i + 7]));
}

__device__ __forceinline__ void pin16(uint32_t (&r)[16])
{
#pragma unroll
    for (int i = 0; i < 16; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                          "+r"(r[i + 6]), "+r"(r[i + 7]));
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
                 "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                 "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two fp32 in one 64-bit register.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void group_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// A barrier of the threads that also tells whether all came with `ok`.
__device__ __forceinline__ bool vote(int id, int threads, bool ok)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.b32 p, %1, 0;\n\t"
                 "barrier.cta.red.and.pred q, %2, %3, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)ok), "r"(id), "r"(threads)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                            uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// 32 MXFP8 elements (codes w, block scale e) to bf16: chunks 4 half .. of the
// row's 128 bytes in a slab (chunk c at c ^ sw).  Through fp32, exactly, for every code
// and scale: the conversions and products run on the floating-point pipes,
// which are free here, where moving bits into place keeps the integer pipe busy
// (a tile of 128 x 128 by eight warps: 673 cycles against 906 to 1064 for three ways of bit placement).
__device__ __forceinline__ void decode32(const uint32_t (&w)[8], uint32_t e, uint8_t *row, int half, int sw)
{
    const float s = e8m0_to_f32(e);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h0, h1;
            e4m3x4_to_f16x2(w[2 * c + i], h0, h1);
            o[2 * i] = scaled_bf16x2(h0, s);
            o[2 * i + 1] = scaled_bf16x2(h1, s);
        }
        store_chunk(row, 4 * half + c, sw, o[0], o[1], o[2], o[3]);
    }
}

// ------------------------------------------------------------ kernel

// Shared control block, after the tiles.
struct AtCtrl {
    uint64_t slot_bars[28];          // full and empty barriers of the bf16 slots, then of the packed ones (MXFP8)
    uint64_t q_full, q_empty;
    uint64_t s_full[2], o_full[2];
    uint64_t p_full[2][2];           // by group, and half of the key tile
    uint64_t done;
    uint64_t r_full[AT_RING], r_free[AT_RING];
    Piece ring[AT_RING];             // pieces, from the producer to the other roles
    Stretch stretch;
    uint32_t tmem;
    Watch watch;
    int missing[8];                  // by piece number: a page of it is missing
    int last[2];                     // by group: its part of a cut item was the last to come
    Piece pending[2];                // by group: a part that is written but not counted yet
    unsigned again[2][4];            // by group: rows to compute again
    float m[2][AT_ROWS], l[2][AT_ROWS];
};
static_assert(sizeof(AtCtrl) <= AtGeo<128, KV_BF16>::CTRL, "control block");

__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// A position in a ring of N slots and the phase of its barriers there.
template <int N>
struct Slot {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++i == N) {
            i = 0;
            phase ^= 1;
        }
    }
};

// Load number of V tile t within a piece of n key tiles.  The keys' tiles
// run `ahead` tiles ahead: K 0 .. ahead-1, then V t, K t + ahead in turn.
__device__ __forceinline__ int k_load(int t, int ahead) { return t < ahead ? t : 2 * t - ahead + 1; }
__device__ __forceinline__ int v_load(int t, int n, int ahead) { return t + min(n, ahead + t); }

// Where the partial of (CTA, which of its two, group) lies: m and l of the
// rows, then O in units of four dimensions, rows fastest.
template <int D>
__device__ __forceinline__ float *partial_base(const AtParams &p, int cta, int which, int group)
{
    return p.partials + (size_t)((cta * 2 + which) * 2 + group) * p.part_rows * (D + 2);
}

// Calls use(key of the 32, offsets of its place) ... for keys [lo, hi) of a cache head,
// by the whole warp: each lane finds the place of one of 32 keys, then all take
// them in turn, AHEAD at a time so that their loads are in flight together.
// first(at, sat): a lane's own key, before.
template <int AHEAD, typename First, typename Use>
__device__ __forceinline__ void for_keys(const mx_paged_kv &kv, int b, int kvh, int lo, int hi, First first, Use use)
{
    const int lane = threadIdx.x & 31;
    const int32_t *table = kv.block_table + (size_t)b * kv.table_stride;
    for (long long k0 = lo; k0 < hi; k0 += 32) {
        const int key = (int)min(k0 + lane, hi - 1ll), n = (int)min(32ll, hi - k0);
        const int pi = key / kv.page_size, slot = key - pi * kv.page_size;
        const int page = max(page_of(kv, table, pi), 0);
        const long long at = page * kv.page_stride + kvh * kv.head_stride + slot * kv.token_stride;
        const long long sat = page * kv.scale_page_stride + kvh * kv.scale_head_stride + slot * kv.scale_token_stride;
        first(lane < n, at, sat);
#pragma unroll 1
        for (int j = 0; j < n; j += AHEAD) {
            long long ats[AHEAD], sats[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                ats[i] = __shfl_sync(0xFFFFFFFFu, at, (j + i) & 31);
                sats[i] = __shfl_sync(0xFFFFFFFFu, sat, (j + i) & 31);
            }
            use(j, n - j, ats, sats);
        }
    }
}

constexpr int AGAIN_AHEAD = 4;  // (8: the softmax warps of the MXFP8 kernel spill)

// What is not finite among the values of keys [lo, hi), in this lane's dimensions
// 2 lane + 64 i and the one after: for each of them three bits, NaN, +infinity
// and -infinity.
template <int D, int KVF>
__device__ __noinline__ uint32_t kinds_of_values(const mx_paged_kv &kv, int b, int kvh, int lo, int hi)
{
    const int d = 2 * (threadIdx.x & 31);
    uint32_t kinds = 0;
    for_keys<AGAIN_AHEAD>(
        kv, b, kvh, lo, hi, [](bool, long long, long long) {},
        [&](int, int left, const long long(&at)[AGAIN_AHEAD], const long long(&sat)[AGAIN_AHEAD]) {
            RawPair<KVF> r[AGAIN_AHEAD][D / 64];
#pragma unroll
            for (int k = 0; k < AGAIN_AHEAD; ++k)
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                    r[k][i].load(kv, at[k < left ? k : 0], sat[k < left ? k : 0], d + 64 * i);
#pragma unroll
            for (int k = 0; k < AGAIN_AHEAD; ++k)
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const float2 v = r[k][i].get();
                    if (v.x * 0.0f != 0.0f) kinds |= (v.x != v.x ? 1u : v.x > 0.0f ? 2u : 4u) << (6 * i);
                    if (v.y * 0.0f != 0.0f) kinds |= (v.y != v.y ? 1u : v.y > 0.0f ? 2u : 4u) << (6 * i + 3);
                }
        });
    return kinds;
}

// One row from its own keys [lo, hi) alone, each weight divided by the sum before it is
// used, dimensions [d0, d1); by the whole warp.
template <int D, int KVF>
__device__ __noinline__ void row_again(const AttnArgs &a, int b, int t, int h, int lo, int hi, int d0, int d1,
                                       float inv_total, float m_used)
{
    const int d = 2 * (threadIdx.x & 31);
    const mx_paged_kv &kv = a.kv;
    const uint16_t *q = a.q + (long long)t * a.q_token_stride + (long long)h * a.q_head_stride;
    float o[D / 32] = {}, p = 0.0f;
    for_keys<AGAIN_AHEAD>(
        kv, b, h / a.g, lo, hi,
        [&](bool mine, long long at, long long sat) {
            p = mine ? exp2f(key_dot<KVF>(kv, q, at, sat) * a.scale_log2 - m_used) * inv_total : 0.0f;
        },
        [&](int j, int left, const long long(&at)[AGAIN_AHEAD], const long long(&sat)[AGAIN_AHEAD]) {
            RawPair<KVF> r[AGAIN_AHEAD][D / 64];
#pragma unroll
            for (int k = 0; k < AGAIN_AHEAD; ++k)
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                    r[k][i].load(kv, at[k < left ? k : 0], sat[k < left ? k : 0], d + 64 * i);
#pragma unroll
            for (int k = 0; k < AGAIN_AHEAD; ++k) {
                const float pk = __shfl_sync(0xFFFFFFFFu, p, (j + k) & 31);
                if (k < left)
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        const float2 v = r[k][i].get();
                        o[2 * i] = fmaf(pk, v.x, o[2 * i]);
                        o[2 * i + 1] = fmaf(pk, v.y, o[2 * i + 1]);
                    }
            }
        });
    uint16_t *out = a.out + ((size_t)t * a.Hq + h) * D;
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
        if (d + 64 * i >= d0 && d + 64 * i < d1)
            *reinterpret_cast<uint32_t *>(out + d + 64 * i) = f32x2_to_bf16x2(o[2 * i], o[2 * i + 1]);
}

// Rows (the lanes in the mask, each with its own arguments) whose outputs are not
// finite: a product with a weight of zero is NaN when the value is NaN or
// infinite, and such a value may lie where the row may not see it; and values
// near the type's largest can overflow a sum whose weights are divided only at
// its end.  What the values that all these rows see account for stands: a NaN
// where one of them is NaN or both infinities are among them, an infinity where it
// is among them (with a weight of zero it had become NaN).  Other rows are computed
// again one by one.
template <int D, int KVF>
__device__ __noinline__ void rows_again(const AttnArgs &a, unsigned rows, int b, int t, int h, int lo, int hi, int d0,
                                        int d1, float inv_total, float m_used, int *busy)
{
    const int lane = threadIdx.x & 31;
    const bool mine = rows >> lane & 1;
    if (lane == 0) atomicAdd(busy, 1);
    __syncwarp();
    const int all_lo = __reduce_max_sync(0xFFFFFFFFu, mine ? lo : 0);
    const int all_hi = __reduce_min_sync(0xFFFFFFFFu, mine ? hi : 0x7FFFFFFF);
    const int kvh = __shfl_sync(0xFFFFFFFFu, h, __ffs(rows) - 1) / a.g;
    const uint32_t kinds = kinds_of_values<D, KVF>(a.kv, b, kvh, all_lo, all_hi);
    for (; rows != 0; rows &= rows - 1) {
        const int src = __ffs(rows) - 1;
        const int row_t = __shfl_sync(0xFFFFFFFFu, t, src), row_h = __shfl_sync(0xFFFFFFFFu, h, src);
        const volatile uint32_t *out = reinterpret_cast<const uint32_t *>(a.out + ((size_t)row_t * a.Hq + row_h) * D);
        bool stands = true;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const int d = 2 * lane + 64 * i;
            if (d < d0 || d >= d1) continue;
            const uint32_t w = out[d / 2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = e ? bf16_hi(w) : bf16_lo(w);
                const uint32_t k = kinds >> (6 * i + 3 * e) & 7u;
                if (x != x) stands = stands && ((k & 1u) || (k & 6u) == 6u);
                else if (x * 0.0f != 0.0f) stands = stands && (k & (x > 0.0f ? 2u : 4u));
            }
        }
        const int row_lo = __shfl_sync(0xFFFFFFFFu, lo, src), row_hi = __shfl_sync(0xFFFFFFFFu, hi, src);
        const float row_inv = __shfl_sync(0xFFFFFFFFu, inv_total, src), row_m = __shfl_sync(0xFFFFFFFFu, m_used, src);
        if (!__all_sync(0xFFFFFFFFu, stands))
            row_again<D, KVF>(a, b, row_t, row_h, row_lo, row_hi, d0, d1, row_inv, row_m);
    }
    if (lane == 0) atomicSub(busy, 1);
}

// Is a page missing that holds any of a sequence's keys [lo, hi)?  (Rare: a loop over
// the table's entries in each row's own thread.)
__device__ __noinline__ bool any_missing(const AttnArgs &a, int b, int lo, int hi)
{
    const int32_t *table = a.kv.block_table + (size_t)b * a.kv.table_stride;
    if (lo >= hi) return false;
    for (int i = lo / a.kv.page_size, end = (hi - 1) / a.kv.page_size; i <= end; ++i)
        if (page_of(a.kv, table, i) < 0) return true;
    return false;
}

// Two sums against maxima m0 and m1 become one against the larger: the first
// times f0 plus the second times f1.
struct Merge {
    float m, f0, f1;
    __device__ __forceinline__ Merge(float m0, float m1)
    {
        m = fmaxf(m0, m1);
        const bool none = m == -INFINITY;
        f0 = none ? 0.0f : exp2_approx(m0 - m);
        f1 = none ? 0.0f : exp2_approx(m1 - m);
    }
    __device__ __forceinline__ float add(float x0, float x1) const { return fmaf(x1, f1, x0 * f0); }
};

// Are all parts of a cut item but this group's in?  Then its count is ready
// for the next call again.
__device__ __forceinline__ bool all_others_in(const AtParams &p, const Piece &pc, int w, int row, volatile int *last)
{
    if (row == 0) {
        int *count = p.counters + 2 * pc.c0 + w;
        int v;
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
        last[w] = v == pc.c1 - pc.c0;
        if (last[w]) *count = 0;
        __threadfence();
    }
    group_sync(2 + w, 128);
    const bool in = last[w] != 0;
    group_sync(2 + w, 128);
    return in;
}

// A group's part of a cut item is written: counts it; true if it was the last.
__device__ __forceinline__ bool last_of(const AtParams &p, const Piece &pc, int w, int row, volatile int *last)
{
    __threadfence();
    group_sync(2 + w, 128);
    if (row == 0) {
        int *count = p.counters + 2 * pc.c0 + w;
        const int pieces = pc.c1 - pc.c0 + 1, arrived = atomicAdd(count, 1) + 1;
        if (arrived == pieces) *count = 0;  // ready for the next call
        last[w] = arrived == pieces;
        __threadfence();
    }
    group_sync(2 + w, 128);
    return last[w] != 0;
}

// Counts a group's part of a cut item; the last to come adds all parts up, in
// their order, and writes the outputs: a thread takes sixteen dimensions of a row
// (loads of four at a time left 512 tokens of prompt waiting 30 us), neighbouring
// threads neighbouring rows.
template <int D, int KVF>
__device__ __noinline__ void arrive_cut(const AtParams &p, const Piece &piece, int w, int tid, volatile int *last,
                                        unsigned *again, Watch *watch)
{
    const Piece pc = piece;
    if (tid < 4) again[tid] = 0u;
    if (!last_of(p, pc, w, tid, last)) return;
    const AttnArgs &a = p.a;
    const int s1 = AT_ROWS / a.g;
    const int t0 = pc.rows ? w * s1 : 0, R = min(pc.ntok - t0, s1) * a.g;
    const int d0 = pc.rows ? 0 : w * (D / 2), W = pc.rows ? D : D / 2, parts = pc.c1 - pc.c0 + 1;
    __threadfence();
    constexpr int U = 4;  // quads a thread takes at once
    for (int e = tid; e < R * (W / (4 * U)); e += 128) {
        const int quad = e / R * U, row = e % R;
        const int t = pc.q0 + t0 + row / a.g, head = pc.kvh * a.g + row % a.g;
        float m = -INFINITY, total = 0.0f;
        float4 o[U];
#pragma unroll
        for (int k = 0; k < U; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
        for (int i = 0; i < parts; ++i) {
            const float *pi = partial_base<D>(p, pc.c0 + i, i == 0 ? 1 : 0, w);
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(pi) + row);
            const float4 *ri = reinterpret_cast<const float4 *>(pi + 2 * p.part_rows) + (size_t)quad * p.part_rows + row;
            float4 r[U];
#pragma unroll
            for (int k = 0; k < U; ++k) r[k] = __ldcg(ri + (size_t)k * p.part_rows);
            const Merge mg(m, ml.x);
            m = mg.m;
            total = mg.add(total, ml.y);
#pragma unroll
            for (int k = 0; k < U; ++k)
                o[k] = make_float4(mg.add(o[k].x, r[k].x), mg.add(o[k].y, r[k].y), mg.add(o[k].z, r[k].z),
                                   mg.add(o[k].w, r[k].w));
        }
        const float sink = a.sinks ? __ldg(a.sinks + head) * 1.4426950408889634f : -INFINITY;
        const float ref = fmaxf(m, sink), base2 = ref == -INFINITY ? 0.0f : ref;
        const float f = m == -INFINITY ? 0.0f : exp2_approx(m - base2);
        float den = total * f;
        if (a.sinks) den += exp2_approx(sink - base2);
        const float inv = den == 0.0f ? 0.0f : f / den;
        const size_t out_row = (size_t)t * a.Hq + head;
        if (a.lse && quad == 0 && (pc.rows || w == 0)) a.lse[out_row] = (base2 + log2f(den)) * 0.6931471805599453f;
        uint32_t *out = reinterpret_cast<uint32_t *>(a.out + out_row * D + d0 + 4 * quad);
        float check = 0.0f;
        uint32_t b[2 * U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const float x = fmaf(o[k].x, inv, 0.0f), y = fmaf(o[k].y, inv, 0.0f), z = fmaf(o[k].z, inv, 0.0f),
                        u = fmaf(o[k].w, inv, 0.0f);
            b[2 * k] = f32x2_to_bf16x2(x, y);
            b[2 * k + 1] = f32x2_to_bf16x2(z, u);
            check += x * 0.0f + y * 0.0f + z * 0.0f + u * 0.0f;
        }
#pragma unroll
        for (int k = 0; k < U; k += 2)
            reinterpret_cast<uint4 *>(out)[k / 2] = make_uint4(b[2 * k], b[2 * k + 1], b[2 * k + 2], b[2 * k + 3]);
        if (check != 0.0f && inv == inv) atomicOr(again + row / 32, 1u << (row % 32));
    }
    group_sync(2 + w, 128);
    const unsigned rows = again[tid / 32];
    if (rows == 0) return;
    const int tok = t0 + tid / a.g, head = pc.kvh * a.g + tid % a.g, pos = pc.first + tok;
    const int hi = a.causal ? min(pos + 1, pc.len) : pc.len;
    const int lo = a.window > 0 ? (int)max((long long)pos - a.window + 1, 0ll) : 0;
    float den = 0.0f, base2 = 0.0f;
    if (rows >> tid % 32 & 1) {
        float m = -INFINITY, total = 0.0f;
        for (int i = 0; i < parts; ++i) {
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(partial_base<D>(p, pc.c0 + i, i == 0 ? 1 : 0, w)) + tid);
            const Merge mg(m, ml.x);
            m = mg.m;
            total = mg.add(total, ml.y);
        }
        const float sink = a.sinks ? __ldg(a.sinks + head) * 1.4426950408889634f : -INFINITY;
        const float ref = fmaxf(m, sink);
        base2 = ref == -INFINITY ? 0.0f : ref;
        den = m == -INFINITY ? 0.0f : total * exp2_approx(m - base2);
        if (a.sinks) den += exp2_approx(sink - base2);
    }
    __syncwarp();
    rows_again<D, KVF>(a, rows, pc.b, pc.q0 + tok, head, lo, hi, d0, d0 + W, 1.0f / den, base2, &watch->busy);
}

// A CTA whose wait gave up: the outputs of its pieces from number `done` on
// become NaN, its parts of cut items too.
template <int D, int KVF>
__device__ __noinline__ void poison(const AtParams &p, const Cost &cost, int done, int w, int row,
                                    AtCtrl &c)
{
    const AttnArgs &a = p.a;
    const float nan = __uint_as_float(0x7FC00000u);
    const int s1 = cost.s2 / 2;
    if (row == 0) set_device_error(a.err, DEVERR_TIMEOUT);
    Walk walk(a, c.stretch, cost);
    Piece pc;
    for (int i = 0; walk.next(pc); ++i) {
        if (i < done) continue;
        const int tok = (pc.rows ? w * s1 : 0) + row / a.g, head = pc.kvh * a.g + row % a.g;
        const bool valid = row < s1 * a.g && tok < pc.ntok;
        if (pc.c0 != pc.c1) {
            float *part = partial_base<D>(p, blockIdx.x, (int)blockIdx.x == pc.c0 ? 1 : 0, w);
            if (valid) part[2 * row] = part[2 * row + 1] = nan;
            arrive_cut<D, KVF>(p, pc, w, row, c.last, c.again[w], &c.watch);
        } else if (valid) {
            const size_t r = (size_t)(pc.q0 + tok) * a.Hq + head;
            if (a.lse) a.lse[r] = nan;
            for (int d = pc.rows ? 0 : w * (D / 2); d < (pc.rows ? D : (w + 1) * (D / 2)); ++d)
                a.out[r * D + d] = 0x7FC0u;
        }
    }
}

template <int D, int KVF>
__global__ void __launch_bounds__(AtGeo<D, KVF>::THREADS, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_q1,
                   const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ AtParams prm)
{
    using G = AtGeo<D, KVF>;
    extern __shared__ __align__(1024) uint8_t smem[];  // 1024: the swizzle's period
    AtCtrl &c = *reinterpret_cast<AtCtrl *>(smem + G::OFF_BAR);
    const AttnArgs &a = prm.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile Watch *watch = &c.watch;
    uint64_t *full = c.slot_bars, *empty = full + G::SLOTS, *c_full = empty + G::SLOTS, *c_empty = c_full + G::C_SLOTS;
    Cost cost;
    const int s1 = AT_ROWS / a.g;
    cost.s2 = 2 * s1;
    cost.causal = a.causal;
    cost.window = a.window;
    cost.heads = a.kv.Hkv;
    cost.flat = 0;

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int s = 0; s < G::SLOTS; ++s) {
            mbar_init(&full[s], G::MX8 ? G::DECODERS : 1);
            mbar_init(&empty[s], 1);
        }
        if (G::MX8)
            for (int s = 0; s < G::C_SLOTS; ++s) {
                mbar_init(&c_full[s], 1);
                mbar_init(&c_empty[s], G::DECODERS);
            }
        mbar_init(&c.q_full, 1);
        mbar_init(&c.q_empty, 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(&c.s_full[w], 1);
            mbar_init(&c.p_full[w][0], 4);
            mbar_init(&c.p_full[w][1], 4);
            mbar_init(&c.o_full[w], 1);
        }
        mbar_init(&c.done, 1);
        for (int i = 0; i < AT_RING; ++i) {
            mbar_init(&c.r_full[i], 1);
            mbar_init(&c.r_free[i], 1 + 8 + (G::MX8 ? G::DECODERS : 0));  // MMA issuer, softmax and decoder warps
        }
        c.watch.gave_up = 0;
        c.watch.busy = 0;
        for (int i = 0; i < 8; ++i) c.missing[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&c.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    if (warp != 10) pdl_wait();
    Piece pc;
    // the i-th piece from the ring, by a whole warp
    auto take = [&](int i) {
        const bool ok = warp_wait(&c.r_full[i % AT_RING], (i / AT_RING) & 1, watch, prm.wait_ns);
        if (ok) pc = c.ring[i % AT_RING];
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&c.r_free[i % AT_RING]);
        return ok;
    };

    // (setmaxnreg stands inside the roles' branches: the register allocation
    // goes by what reaches a point)
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::R_SOFTMAX));
        // ---------------- softmax groups
        const int w = warp >> 2;            // group
        const int row = threadIdx.x & 127;  // row of the tile; also the tensor-memory lane
        const uint32_t lane_base = tmem + ((uint32_t)(row & ~31) << 16);
        const uint32_t s_addr = lane_base + G::S_COL + 128 * w;
        const float sl2 = a.scale_log2;
        bool pending = false;  // c.pending[w] waits to be counted
        int base = 0, piece = 0, steps = 0;  // steps: softmax steps of this group so far
        bool alive = true;
        // warp-uniform, as the tensor-memory instructions that follow a wait must be
        auto wait = [&](uint64_t *bar, int phase) {
            return warp_wait(bar, phase & 1, watch, prm.wait_ns);
        };
        for (int np = 0;; ++np) {
            alive = take(np);
            if (pending) {
                // the last piece's part: its stores are on their way while the next
                // piece's queries and first scores are
                group_sync(2 + w, 128);
                arrive_cut<D, KVF>(prm, c.pending[w], w, row, c.last, c.again[w], &c.watch);
                pending = false;
            }
            if (!alive || pc.end) {  // an empty piece, to the vote below
                pc.k0 = pc.k1 = pc.ntok = 0;
                pc.rows = 1;
                pc.c0 = pc.c1 = 0;
            }
            const int n = pc.k1 - pc.k0, ahead = pc.rows ? 1 : 2;
            const int tok = (pc.rows ? w * s1 : 0) + row / a.g, head = pc.kvh * a.g + row % a.g;
            const bool valid = row < s1 * a.g && tok < pc.ntok;
            const int pos = pc.first + tok;
            int rlo = 0, rhi = 0x7FFFFFFF;  // (a lane without a row needs no mask)
            if (valid) {
                rhi = a.causal ? min(pos + 1, pc.len) : pc.len;
                rlo = a.window > 0 ? (int)max((long long)pos - a.window + 1, 0ll) : 0;
                if (rhi < rlo) rhi = rlo;
            }
            // warps with rows, the first ones of the group; the others go to the
            // vote, and the first warp arrives for them
            const int R = min(pc.ntok - (pc.rows ? w * s1 : 0), s1) * a.g, warps_on = (R + 31) / 32;
            const bool warp_on = (warp & 3) < warps_on;
            const uint32_t arrivals = (warp & 3) == 0 ? 5 - warps_on : 1;
            const int n_mine = pc.rows ? n : (n + 1 - w) / 2;  // this group's steps
            float m = -INFINITY, l = 0.0f;  // m: log2 units, what P was taken against
            int mine = 0;                   // steps of this piece
            for (int t = pc.rows ? 0 : w; t < n && alive && warp_on; t += ahead) {
                alive = wait(&c.s_full[w], steps);
                if (!alive) break;
                const int key0 = (pc.tile0 + pc.k0 + t) * AT_KEYS;
                // rows of V that no row sees, or that were not loaded: their
                // weights are zero, their values must be finite
                if ((key0 < pc.lo || key0 > pc.hi - AT_KEYS) && (w == 0 || !pc.rows)) {
                    const int vi = base + v_load(t, n, ahead);
                    alive = wait(&full[vi % G::SLOTS], vi / G::SLOTS);
                    if (!alive) break;
                    // (eight lanes to a 128-byte row, so that a store covers all banks)
                    uint8_t *v = smem + G::OFF_KV + (vi % G::SLOTS) * G::TILE + (lane & 7) * 16;
                    for (int r = (row >> 5) * 4 + (lane >> 3); r < AT_KEYS; r += 4 * warps_on)
                        if (key0 + r < pc.lo || key0 + r >= pc.hi)
#pragma unroll
                            for (int i = 0; i < G::SLABS; ++i)
                                *reinterpret_cast<uint4 *>(v + i * G::SLAB + r * 128) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                tc_fence_after();
                if (__builtin_expect(__any_sync(0xFFFFFFFFu, key0 < rlo || key0 > rhi - AT_KEYS), 0)) {
                    // scores that the row may not see, in place: a small loop, for the instruction cache
                    const int klo = rlo - key0, khi = rhi - key0;
#pragma unroll 1
                    for (int i = 0; i < AT_KEYS; i += 16) {
                        uint32_t x[16];
                        tmem_ld16_async(s_addr + i, x);
                        tmem_wait_ld();
                        pin16(x);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (i + j < klo || i + j >= khi) x[j] = 0xFF800000u;
                        tmem_st16(s_addr + i, x);
                    }
                    tmem_wait_st();
                }
                // half h of the scores (32 pairs)
                auto load_half = [&](int h, uint32_t(&s)[64]) {
                    tmem_ld32_async(s_addr + 64 * h, s, 0);
                    tmem_ld32_async(s_addr + 64 * h + 32, s, 32);
                };
                auto pin_half = [&](uint32_t(&s)[64]) {
                    pin32(s, 0);
                    pin32(s, 32);
                };
                auto max_half = [&](const uint32_t(&s)[64]) {
                    float x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = max3(__uint_as_float(s[3 * j]), __uint_as_float(s[3 * j + 1]), __uint_as_float(s[3 * j + 2]));
#pragma unroll
                    for (int i = 12; i < 60; i += 8)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[j] = max3(x[j], __uint_as_float(s[i + 2 * j]), __uint_as_float(s[i + 2 * j + 1]));
                    return fmaxf(max3(x[0], x[1], __uint_as_float(s[60])),
                                 max3(max3(x[2], x[3], __uint_as_float(s[61])), __uint_as_float(s[62]), __uint_as_float(s[63])));
                };
                // weights 2^(s scale - m) as bf16 pairs, and their sum
                const uint64_t sl22 = pack2(sl2, sl2);
                auto weights = [&](const uint32_t(&s)[64], uint32_t(&pk)[32]) {
                    const float neg = m == -INFINITY ? 0.0f : -m;
                    const uint64_t neg2 = pack2(neg, neg);
                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const uint64_t e2 = fma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sl22, neg2);
                        float e0, e1;
                        unpack2(e2, e0, e1);
                        e0 = exp2_approx(e0);
                        e1 = exp2_approx(e1);
                        sum[i & 1] = add2(sum[i & 1], pack2(e0, e1));
                        pk[i] = f32x2_to_bf16x2(e0, e1);
                    }
                    float s0, s1_, s2, s3;
                    unpack2(sum[0], s0, s1_);
                    unpack2(sum[1], s2, s3);
                    return (s0 + s1_) + (s2 + s3);
                };
                // raise the maximum: at the first tile that has one, and when it is
                // outgrown; true if any of the warp's rows did
                auto raise_to = [&](float top) {
                    const bool raise = valid && (top > m + AT_RAISE || (m == -INFINITY && top > -INFINITY));
                    if (__builtin_expect(!__any_sync(0xFFFFFFFFu, raise), 1)) return false;
                    const float m_new = raise ? top : m;
                    const float f = m == -INFINITY ? 0.0f : exp2_approx(m - m_new);
                    m = m_new;
                    l *= f;
                    if (mine > 0) {
                        // the O so far belongs to the old maximum
                        alive = wait(&c.o_full[w], steps - 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int i = 0; i < D && alive; i += 16) {
                            uint32_t o[16];
                            tmem_ld16_async(lane_base + G::O_COL + 128 * w + i, o);
                            tmem_wait_ld();
                            pin16(o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st16(lane_base + G::O_COL + 128 * w + i, o);
                        }
                    }
                    return true;
                };
                // a half's weights over its own scores
                auto publish = [&](int h, const uint32_t(&pk)[32]) {
                    tmem_st32(s_addr + 64 * h, pk);
                    tmem_wait_st();
                    tc_fence_before();
                };
                // the product with the first half of V may start
                auto half_done = [&]() {
                    __syncwarp();
                    if (lane == 0) mbar_arrive_n(&c.p_full[w][0], arrivals);
                };
                if constexpr (G::MX8) {
                    // one half at a time, its scores read twice: fewer registers and
                    // half the code (327 against 367 us for the mixed batch; the bf16
                    // kernel, with registers for both halves, loses 1-4 %)
                    uint32_t s0[64], pk[32];
                    float top = -INFINITY;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        load_half(h, s0);
                        tmem_wait_ld();
                        pin_half(s0);
                        top = fmaxf(top, max_half(s0));
                    }
                    raise_to(top * sl2);
                    if (!alive) break;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        load_half(h, s0);
                        tmem_wait_ld();
                        pin_half(s0);
                        l += weights(s0, pk);
                        publish(h, pk);
                        if (h == 0) half_done();
                    }
                } else {
                    // the first half's weights against the maximum so far, while the
                    // tile's maximum is found; again in the rare case that it is raised,
                    // and only then at the piece's first tile, which sets it
                    uint32_t s0[64], s1[64], pk[32];
                    load_half(0, s0);
                    load_half(1, s1);
                    tmem_wait_ld();
                    pin_half(s0);
                    pin_half(s1);
                    const float top = fmaxf(max_half(s0), max_half(s1)) * sl2;
                    float sum = 0.0f;
                    if (mine > 0) sum = weights(s0, pk);
                    if (__builtin_expect(raise_to(top) || mine == 0, 0)) {
                        if (!alive) break;
                        load_half(0, s0);
                        tmem_wait_ld();
                        pin_half(s0);
                        sum = weights(s0, pk);
                    }
                    publish(0, pk);
                    half_done();
                    sum += weights(s1, pk);
                    publish(1, pk);
                    l += sum;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_n(&c.p_full[w][1], arrivals);
                ++steps;
                ++mine;
            }
            if (!warp_on) steps += n_mine;
            // the last product must be in before O is read
            if (mine > 0 && alive) alive = wait(&c.o_full[w], steps - 1);
            if (!pc.rows) {
                c.m[w][row] = m;
                c.l[w][row] = l;
            }
            tc_fence_before();
            // both groups go on only together: one that gave up does not come to their barriers any more
            const bool go_on = vote(1, 256, alive);
            if (!go_on) poison<D, KVF>(prm, cost, np, w, row, c);
            if (!go_on || pc.end) break;
            tc_fence_after();
            bool bad = n > 0 && c.missing[piece & 7] != 0;
            if (bad) {
                // the row's own keys among this piece's, or the tiles' other rows alone?
                if (row == 0) set_device_error(a.err, DEVERR_BAD_PAGE);
                const int k0 = (pc.tile0 + pc.k0) * AT_KEYS, k1 = min((pc.tile0 + pc.k1 - 1) * AT_KEYS, 0x7FFFFFFF - AT_KEYS) + AT_KEYS;
                bad = valid && any_missing(a, pc.b, max(rlo, k0), min(rhi, k1));
                __syncwarp();
            }
            // rows: the group's own rows, all dimensions.  keys: both groups'
            // sums of the same rows; group w takes half of the dimensions.
            int d0 = 0, d1 = D;
            float f_own = 1.0f, f_other = 0.0f;
            if (!pc.rows) {
                const float m2 = c.m[w ^ 1][row], l2 = c.l[w ^ 1][row];
                const float top = fmaxf(m, m2);
                if (top > -INFINITY) {
                    f_own = m == -INFINITY ? 0.0f : exp2_approx(m - top);
                    f_other = m2 == -INFINITY ? 0.0f : exp2_approx(m2 - top);
                }
                // in the same order in both groups
                l = w == 0 ? fmaf(l, f_own, l2 * f_other) : fmaf(l2, f_other, l * f_own);
                m = top;
                d0 = w * (D / 2);
                d1 = d0 + D / 2;
            }
            const bool cut = pc.c0 != pc.c1;
            // The first CTA of a cut item reaches its part last, as the end of its
            // stretch; the others' is the start of theirs.  Where the one other
            // part is in, the first CTA adds it to its own from registers;
            // otherwise parts go through memory and are counted before the next piece.
            const bool first = (int)blockIdx.x == pc.c0;
            const bool two = cut && first && pc.c1 == pc.c0 + 1 && all_others_in(prm, pc, w, row, c.last);
            const bool finish_here = !cut || two;
            float *part = nullptr;  // this group's part, or the one to add
            if (cut) part = partial_base<D>(prm, two ? pc.c1 : (int)blockIdx.x, first && !two ? 1 : 0, w);
            float4 *part_o = reinterpret_cast<float4 *>(part + 2 * prm.part_rows) + row;
            float m_all = m, total = l;  // over all of the item's pieces
            Merge mg(m, -INFINITY);
            if (two && valid) {
                const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part) + row);
                mg = Merge(m, ml.x);
                total = mg.add(l, ml.y);
                m_all = mg.m;
            } else if (cut && valid) {
                part[2 * row] = bad ? __uint_as_float(0x7FC00000u) : m;
                part[2 * row + 1] = bad ? __uint_as_float(0x7FC00000u) : l;
            }
            float sink = -INFINITY;
            if (a.sinks && valid) sink = __ldg(a.sinks + head) * 1.4426950408889634f;
            const float ref = fmaxf(m_all, sink);
            const float base2 = ref == -INFINITY ? 0.0f : ref;
            const float f = m_all == -INFINITY ? 0.0f : exp2_approx(m_all - base2);
            float den = total * f;
            if (a.sinks) den += exp2_approx(sink - base2);
            float inv = den == 0.0f ? 0.0f : f / den;
            if (bad) inv = den = __uint_as_float(0x7FC00000u);
            const size_t out_row = (size_t)(pc.q0 + tok) * a.Hq + head;
            if (finish_here && valid && a.lse && (pc.rows || w == 0))
                a.lse[out_row] = (base2 + log2f(den)) * 0.6931471805599453f;
            uint64_t check = 0ull;
            if (warp_on) {
                constexpr int EC = 16;  // dimensions at a time: little code, which comes from beyond the instruction cache
                const bool own = n > 1 || (n == 1 && (pc.rows || w == 0)), oth = !pc.rows && (n > 1 || (n == 1 && w == 1));
#pragma unroll 1
                for (int d = d0; d < d1; d += EC) {
                    uint32_t u[EC], v[EC];
                    __syncwarp();  // lanes without a row come back from below
                    tmem_ld16_async(lane_base + G::O_COL + 128 * w + d, u);
                    tmem_ld16_async(lane_base + G::O_COL + 128 * (w ^ 1) + d, v);
                    tmem_wait_ld();
                    pin16(u);
                    pin16(v);
                    float o[EC];  // the row's sums against m
#pragma unroll
                    for (int i = 0; i < EC; ++i) {
                        // (a group that had no tile of this piece has anything in its O; in rows the other O is not the row's)
                        o[i] = own ? __uint_as_float(u[i]) * f_own : 0.0f;
                        if (oth) o[i] += __uint_as_float(v[i]) * f_other;
                    }
                    if (!valid) continue;
                    float4 *po = part_o + (size_t)((d - d0) / 4) * prm.part_rows;
                    if (two) {
                        float4 r[EC / 4];  // in flight together
#pragma unroll
                        for (int j = 0; j < EC / 4; ++j) r[j] = __ldcg(po + (size_t)j * prm.part_rows);
#pragma unroll
                        for (int j = 0; j < EC / 4; ++j) {
                            o[4 * j] = mg.add(o[4 * j], r[j].x);
                            o[4 * j + 1] = mg.add(o[4 * j + 1], r[j].y);
                            o[4 * j + 2] = mg.add(o[4 * j + 2], r[j].z);
                            o[4 * j + 3] = mg.add(o[4 * j + 3], r[j].w);
                        }
                    } else if (cut) {
#pragma unroll
                        for (int j = 0; j < EC / 4; ++j)
                            po[(size_t)j * prm.part_rows] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                        continue;
                    }
                    uint16_t *dst = a.out + out_row * D + d;
                    const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
                    for (int q = 0; q < EC / 16; ++q) {
                        uint32_t r[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint64_t x2 = fma2(pack2(o[16 * q + 2 * j], o[16 * q + 2 * j + 1]), inv2, 0ull);
                            check = fma2(x2, 0ull, check);  // NaN once a value is not finite
                            float x, y;
                            unpack2(x2, x, y);
                            r[j] = f32x2_to_bf16x2(x, y);
                        }
                        if (prm.out32) {
                            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 16 * q), "r"(r[0]),
                                         "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                                         : "memory");
                        } else {
                            uint4 *d4 = reinterpret_cast<uint4 *>(dst + 16 * q);
                            d4[0] = make_uint4(r[0], r[1], r[2], r[3]);
                            d4[1] = make_uint4(r[4], r[5], r[6], r[7]);
                        }
                    }
                }
            }
            if (finish_here && warp_on) {
                float c0, c1;
                unpack2(check, c0, c1);
                const unsigned again = __ballot_sync(0xFFFFFFFFu, valid && inv == inv && c0 + c1 != 0.0f);
                if (__builtin_expect(again != 0, 0))
                    rows_again<D, KVF>(a, again, pc.b, pc.q0 + tok, head, rlo, rhi, d0, d1, 1.0f / den, base2, &c.watch.busy);
            }
            if (cut && !finish_here) {
                if (row == 0) c.pending[w] = pc;
                pending = true;
            }
            if (!pc.rows) {
                // the other group's O is read; it may be overwritten after this
                tc_fence_before();
                group_sync(1, 256);
            }
            tc_fence_before();
            base += 2 * max(n, 0);
            if (n > 0) ++piece;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::R_OTHER));
        if (warp == 10) {
            // ---------------- producer: walks the stretch for everybody.  Lengths
            // and the block table are read before the wait for the preceding kernel.
            plan(a, cost, c.stretch);
            __syncwarp();
            Walk walk(a, c.stretch, cost);
            bool waited = false;
            const int ppt = AT_KEYS / prm.page_rows;  // TMA copies per tile and slab
            int load = 0, piece = 0;
            Slot<G::MX8 ? G::C_SLOTS : G::SLOTS> slot;
            bool fresh = true;  // the ring's first round: nothing to wait for
            const bool elected = elect_one();
            bool go = true;
            for (int np = 0; go; ++np) {
                const bool some = walk.next(pc);
                pc.end = !some;
                int ok = 1;
                if (lane == 0) {
                    if (np >= AT_RING) ok = at_wait(&c.r_free[np % AT_RING], ((np / AT_RING) - 1) & 1, watch, prm.wait_ns);
                    if (ok) {
                        c.ring[np % AT_RING] = pc;
                        mbar_arrive(&c.r_full[np % AT_RING]);
                    }
                }
                if (!some || !__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
                if (pc.k0 >= pc.k1) continue;
                const int32_t *table = a.kv.block_table + (size_t)pc.b * a.kv.table_stride;
                const int ahead = pc.rows ? 1 : 2, n = pc.k1 - pc.k0;
                if (lane == 0) c.missing[piece & 7] = 0;
                // page ids: lane i holds copy i of a window of 32 copies; the keys'
                // window, the one before it (the values lag by up to two tiles)
                // and the one after it (on its way)
                const int per_win = 32 / ppt;  // tiles per window
                auto id_index = [&](int wn) {  // in the table's row; -1: not seen, no copy; -2: past the row
                    const long long key = (long long)(pc.tile0 + wn * per_win) * AT_KEYS + lane * prm.page_rows;
                    if (key >= pc.hi || key + prm.page_rows <= pc.lo) return -1;
                    const int i = (int)key / a.kv.page_size;
                    return i < a.kv.table_pages ? i : -2;
                };
                auto id_of = [&](int index, int entry) {  // -2: missing
                    return index < 0 ? index : (unsigned)entry < (unsigned)a.kv.num_pages ? entry : -2;
                };
                auto entry = [&](int index) { return index >= 0 ? __ldg(table + index) : 0; };
                int win = pc.k0 / per_win, id_before = -1;
                const int i0 = id_index(win), i1 = id_index(win + 1);
                const int e0 = entry(i0), e1 = entry(i1);  // both on their way
                // queries
                if (!waited) {
                    pdl_wait();
                    waited = true;
                }
                if (lane == 0 && piece > 0) ok = at_wait(&c.q_empty, (piece - 1) & 1, watch, prm.wait_ns);
                if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
                if (lane == 0 && !prm.stall) {
                    const uint32_t dst = smem_u32(smem);
                    if (pc.rows) {
                        mbar_arrive_expect_tx(&c.q_full, 2 * G::SLABS * (uint32_t)(s1 * a.g) * 128u);
    #pragma unroll
                        for (int r = 0; r < 2; ++r)
    #pragma unroll
                            for (int s = 0; s < G::SLABS; ++s)
                                tma_load_3d(dst + r * G::TILE + s * G::SLAB, &map_q, 64 * s, pc.kvh * a.g,
                                            pc.q0 + r * s1, &c.q_full);
                    } else if (at_whole_tiles(pc.ntok, s1)) {
                        // whole row tile: the rows past the item's tokens are not used
                        mbar_arrive_expect_tx(&c.q_full, G::SLABS * (uint32_t)(s1 * a.g) * 128u);
    #pragma unroll
                        for (int s = 0; s < G::SLABS; ++s)
                            tma_load_3d(dst + s * G::SLAB, &map_q, 64 * s, pc.kvh * a.g, pc.q0, &c.q_full);
                    } else {
                        mbar_arrive_expect_tx(&c.q_full, G::SLABS * (uint32_t)(pc.ntok * a.g) * 128u);
                        for (int t = 0; t < pc.ntok; ++t)
    #pragma unroll
                            for (int s = 0; s < G::SLABS; ++s)
                                tma_load_3d(dst + s * G::SLAB + (uint32_t)(t * a.g) * 128u, &map_q1, 64 * s,
                                            pc.kvh * a.g, pc.q0 + t, &c.q_full);
                    }
                }
                int id_here = id_of(i0, e0), id_after = id_of(i1, e1);
                // One tile into the ring.  The copies are issued by one elected lane
                // from warp-uniform values (a lane per copy took about 150 cycles
                // for each: pages of 16 tokens ran at 3.9 TB/s instead of 6).
                auto load_tile = [&](bool is_k, int t) {
                    const int kt = pc.k0 + t, wn = kt / per_win;
                    if (wn > win) {
                        win = wn;
                        id_before = id_here;
                        id_here = id_after;
                        const int i = id_index(win + 1);
                        id_after = id_of(i, entry(i));
                    }
                    const int ids = wn == win ? id_here : id_before, first = (kt - wn * per_win) * ppt;
                    const bool here = lane >= first && lane < first + ppt;
                    const int copies = __popc(__ballot_sync(0xFFFFFFFFu, here && ids >= 0));
                    if (__any_sync(0xFFFFFFFFu, here && ids == -2) && lane == 0) c.missing[piece & 7] = 1;
                    uint64_t *bar = (G::MX8 ? c_full : full) + slot.i;
                    if (!fresh && !role_wait((G::MX8 ? c_empty : empty) + slot.i, slot.phase ^ 1, watch, prm.wait_ns))
                        return false;
                    if (elected)
                        mbar_arrive_expect_tx(bar, (uint32_t)(copies * prm.page_rows) *
                                                       (G::MX8 ? (uint32_t)(D + D / 32) : 128u * G::SLABS));
                    const CUtensorMap *map = is_k ? &map_k : &map_v;
                    int row = (int)((unsigned)((pc.tile0 + kt) * AT_KEYS) % (unsigned)a.kv.page_size);  // 0 in pages of up to a tile
                    for (int j = 0; j < ppt; ++j) {
                        const int page = __shfl_sync(0xFFFFFFFFu, ids, first + j);
                        if (page < 0 || !elected) continue;
                        const uint32_t r0 = (uint32_t)(j * prm.page_rows);
                        if constexpr (G::MX8) {
                            tma_load_4d(smem_u32(smem + G::OFF_C + slot.i * G::CODES) + r0 * D, map, 0, row, pc.kvh, page, bar);
                            const uint8_t *sc = static_cast<const uint8_t *>(is_k ? a.kv.k_scales : a.kv.v_scales) +
                                                page * a.kv.scale_page_stride + pc.kvh * a.kv.scale_head_stride +
                                                (long long)row * (D / 32);
                            bulk_load(smem_u32(smem + G::OFF_SC + slot.i * G::SCALES) + r0 * (D / 32), sc,
                                      (uint32_t)prm.page_rows * (D / 32), bar);
                        } else {
#pragma unroll
                            for (int sl = 0; sl < G::SLABS; ++sl)
                                tma_load_4d(smem_u32(smem + G::OFF_KV + slot.i * G::TILE + sl * G::SLAB) + r0 * 128u, map,
                                            64 * sl, row, pc.kvh, page, bar);
                        }
                    }
                    ++load;
                    slot.next();
                    if (slot.i == 0) fresh = false;
                    return true;
                };
                // (one call: the roles' loops share an instruction cache)
                for (int kt = 0, vt = 0; vt < n && go;) {
                    const bool is_k = kt < min(n, vt + ahead);
                    go = load_tile(is_k, is_k ? kt : vt);
                    if (is_k) ++kt;
                    else ++vt;
                }
                ++piece;
            }
            if (watch->gave_up) {
                // copies in flight must land before the CTA may exit
                __syncwarp();
                if (lane == 0) {
                    constexpr int RING = G::MX8 ? G::C_SLOTS : G::SLOTS;
                    for (int i = max(load - RING, 0); i < load; ++i)
                        at_wait(G::MX8 ? &c_full[i % RING] : &full[i % RING], (i / RING) & 1, watch, AT_WAIT_NS, false);
                    if (!prm.stall && piece > 0) at_wait(&c.q_full, (piece - 1) & 1, watch, AT_WAIT_NS, false);
                    if (!prm.stall) at_wait(&c.q_full, piece & 1, watch, 1000000ull, false);
                }
            }
        } else if (warp == 9) {
            // ---------------- MMA issuer: the whole warp waits, so that what the
            // instructions take is warp-uniform, and one elected lane issues.
            // (One lane in a branch of its own took about 100 cycles per MMA
            // to bring the descriptors into uniform registers, more than the
            // 32 to 64 cycles that an MMA of this size runs.)
            // What this warp does between two MMAs is on the critical path of
            // both groups: positions in the ring are counted, not divided, and
            // everything that is ready together is issued together.
            const uint32_t q_lo = desc_lo(smem_u32(smem), 16);
            const uint32_t kv_addr = smem_u32(smem + G::OFF_KV);
            const bool elected = elect_one();
            constexpr uint32_t idesc_s = at_idesc<AT_KEYS>(false), idesc_o = at_idesc<D>(true);
            Slot<G::SLOTS> cur;          // next tile of the ring, in the order of the loads
            int piece = 0;
            uint32_t p_phase[2] = {0, 0};  // of each group's p_full
            bool go = true;
            auto wait = [&](uint64_t *bar, uint32_t phase) {
                return role_wait(bar, phase, watch, prm.wait_ns);
            };
            auto commit = [&](uint64_t *bar) {
                if (elected) umma_commit(bar);
            };
            // (elected lane) S of group w from row tile `qtile` and the keys in slot i
            auto s_mma = [&](int w, int qtile, int i) {
                const uint32_t kb = desc_lo(kv_addr + (uint32_t)i * G::TILE, 16);
                const uint32_t qb = q_lo + (uint32_t)qtile * (G::TILE >> 4);
                const uint32_t d = tmem + G::S_COL + 128 * w;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((uint32_t)(kk / 4) * G::SLAB + (kk % 4) * 32) >> 4;
                    umma_ss(d, desc64(qb + off), desc64(kb + off), idesc_s, kk > 0);
                }
                umma_commit(&c.s_full[w]);
            };
            // (elected lane) group w's O plus its weights of half a tile times the values in slot i
            auto o_mma = [&](int w, int i, int half, bool first) {
                const uint32_t vb = desc_lo(kv_addr + (uint32_t)i * G::TILE, G::SLAB);
                const uint32_t d = tmem + G::O_COL + 128 * w, at = tmem + G::S_COL + 128 * w + 64 * half;
#pragma unroll
                for (int kk = 0; kk < AT_KEYS / 32; ++kk)
                    umma_ts(d, at + 8 * kk, desc64(vb + (kk + half * (AT_KEYS / 32)) * (2048 >> 4)), idesc_o, !(first && kk == 0));
            };
            for (int i = 0; go && take(i) && !pc.end; ++i) {
                if (pc.k0 >= pc.k1) continue;
                const int n = pc.k1 - pc.k0, ahead = pc.rows ? 1 : 2;
                // the first scores of each group
                go = wait(&c.q_full, piece & 1) && wait(&full[cur.i], cur.phase);
                if (!go) break;
                if (elected) {
                    s_mma(0, 0, cur.i);
                    if (pc.rows) s_mma(1, 1, cur.i);
                    umma_commit(&empty[cur.i]);
                }
                cur.next();
                if (!pc.rows && n > 1) {
                    go = wait(&full[cur.i], cur.phase);
                    if (!go) break;
                    if (elected) {
                        s_mma(1, 0, cur.i);
                        umma_commit(&empty[cur.i]);
                    }
                    cur.next();
                }
                if (n <= ahead) commit(&c.q_empty);
                for (int t = 0; t < n && go; ++t) {
                    const bool more = t + ahead < n, last = t + ahead == n - 1;
                    const Slot<G::SLOTS> v = cur;  // V t
                    cur.next();
                    const Slot<G::SLOTS> k = cur;  // K t + ahead
                    if (more) cur.next();
                    // both tiles first, so that nothing is waited for between the
                    // weights and the next scores
                    go = wait(&full[v.i], v.phase) && (!more || wait(&full[k.i], k.phase));
                    if (!go) break;
                    const int w_end = pc.rows ? 2 : (t & 1) + 1;
                    for (int w = pc.rows ? 0 : (t & 1); w < w_end; ++w) {
                        go = wait(&c.p_full[w][0], p_phase[w]);
                        if (!go) break;
                        tc_fence_after();
                        if (elected) o_mma(w, v.i, 0, pc.rows ? t == 0 : t < 2);
                        go = wait(&c.p_full[w][1], p_phase[w]);
                        if (!go) break;
                        p_phase[w] ^= 1;
                        tc_fence_after();
                        if (elected) {
                            o_mma(w, v.i, 1, false);
                            umma_commit(&c.o_full[w]);
                            const bool rel = w == w_end - 1;
                            if (rel) umma_commit(&empty[v.i]);
                            if (more) {
                                s_mma(w, pc.rows ? w : 0, k.i);
                                if (rel) {
                                    umma_commit(&empty[k.i]);
                                    if (last) umma_commit(&c.q_empty);  // the last scores are on their way
                                }
                            }
                        }
                    }
                }
                ++piece;
            }
            commit(&c.done);
        } else if (G::MX8 && warp >= 11 && warp < 11 + G::DECODERS) {
            if constexpr (G::MX8) {
                // ---------------- decoders: each takes UNITS / 8 parts of every tile.  A
                // unit is 8 (D = 128) or 16 rows: a lane decodes 32 elements of one
                // row, neighbouring lanes the two halves of a slab's row, so that the
                // 16-byte stores of each 8 lanes cover all banks.
                constexpr int ND = G::DECODERS;
                const int half = lane & 1, slab = D == 128 ? lane >> 4 : 0;
                const int row0 = D == 128 ? (lane >> 1) & 7 : lane >> 1, rows = D == 128 ? 8 : 16;  // of a unit
                const int block = 2 * slab + half;
                // the two 16-byte reads in a row-dependent order, for the banks
                const int f = D == 128 ? row0 & 1 : (row0 >> 1) & 1;
                const int first = warp - 11;  // this warp's first unit of a tile
                Slot<G::C_SLOTS> sc;
                Slot<G::SLOTS> sd;
                bool fresh = true;  // the decoded ring's first round: nothing to wait for
                bool go = true;
                for (int np = 0; go && take(np) && !pc.end; ++np) {
                    for (int left = 2 * (pc.k1 - pc.k0); left > 0; --left) {
                        go = role_wait(&c_full[sc.i], sc.phase, watch, prm.wait_ns);
                        if (!go) break;
                        const uint8_t *codes = smem + G::OFF_C + sc.i * G::CODES + block * 32;
                        const uint8_t *scales = smem + G::OFF_SC + sc.i * G::SCALES + block;
                        uint8_t *tile = smem + G::OFF_KV + sd.i * G::TILE + slab * G::SLAB;
                        if (!fresh) {
                            go = role_wait(&empty[sd.i], sd.phase ^ 1, watch, prm.wait_ns);
                            if (!go) break;
                        }
#pragma unroll 1
                        for (int u = first; u < G::UNITS; u += ND) {
                            const int row = u * rows + row0;
                            const uint4 x = *reinterpret_cast<const uint4 *>(codes + row * D + 16 * f);
                            const uint4 y = *reinterpret_cast<const uint4 *>(codes + row * D + 16 * (f ^ 1));
                            const uint32_t e = scales[row * (D / 32)];
                            const uint4 a0 = f ? y : x, a1 = f ? x : y;
                            const uint32_t wds[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
                            decode32(wds, e, tile + row * 128, half, row & 7);
                        }
                        fence_proxy_async_smem();  // the tile is read by MMAs, the packed slot refilled by TMA
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&full[sd.i]);
                            mbar_arrive(&c_empty[sc.i]);
                        }
                        sc.next();
                        sd.next();
                        if (sd.i == 0) fresh = false;
                    }
                }
            }
        }
    }
    __syncthreads();
    if (warp == 9) {
        if (lane == 0) at_wait(&c.done, 0, watch, AT_WAIT_NS, false);
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ------------------------------------------------------------ host

constexpr int AT_MAX_CTAS = 160;

static int part_rows(int T, int g)
{
    const int s1 = AT_ROWS / g;
    return ((T < s1 ? T : s1) * g + 7) / 8 * 8;
}

size_t attn_tc_workspace_bytes(int T, int Hq, int Hkv, int D)
{
    return ((size_t)AT_MAX_CTAS * 4 * part_rows(T, Hq / Hkv) * (D + 2) * sizeof(float) + 255) / 256 * 256;
}

bool attn_tc_ok(const AttnArgs &a)
{
    const int ps = a.kv.page_size;
    if (a.kv.D != 64 && a.kv.D != 128) return false;
    // whole copies of at least 16 rows per key tile; a maximum that is raised needs a positive scale
    if (ps % AT_KEYS != 0 && (ps < 16 || AT_KEYS % ps != 0)) return false;
    if (!(a.scale_log2 > 0.0f && a.scale_log2 < INFINITY)) return false;
    if (a.kv.kv_fmt == KV_BF16) return true;
    // a page's scales of one head come in one bulk copy
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.kv.k_scales) | reinterpret_cast<uintptr_t>(a.kv.v_scales);
    return a.kv.scale_token_stride == a.kv.D / 32 && a.kv.scale_head_stride % 16 == 0 &&
           a.kv.scale_page_stride % 16 == 0 && at % 16 == 0;
}

template <int D, int KVF>
static cudaError_t run_attn_tc(const DeviceState &ds, cudaStream_t st, const AttnArgs &a)
{
    using G = AtGeo<D, KVF>;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    if (G::SMEM > ds.max_smem_optin || ds.ws_counters < 2 * AT_MAX_CTAS) return cudaErrorInvalidValue;
    AtParams p;
    p.a = a;
    p.counters = ds.ws_count;
    p.partials = static_cast<float *>(a.workspace);
    p.part_rows = part_rows(a.T, a.g);
    p.page_rows = a.kv.page_size < AT_KEYS ? a.kv.page_size : AT_KEYS;
    p.out32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
    p.stall = qmm_stall(&p.wait_ns);
    const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
    const int s1 = AT_ROWS / a.g;
    CUtensorMap maps[4];
    // whole row tiles of queries (not needed by calls of few tokens), single tokens
    const bool whole_tiles = at_whole_tiles(a.T, s1);
    for (int i = whole_tiles ? 0 : 1; i < 2; ++i) {
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
        const cuuint64_t strides[2] = {(cuuint64_t)a.q_head_stride * 2, (cuuint64_t)a.q_token_stride * 2};
        const cuuint32_t box[3] = {64u, (cuuint32_t)a.g, i == 0 ? (cuuint32_t)s1 : 1u};
        if (enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(a.q), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    if (!whole_tiles) maps[0] = maps[1];
    for (int i = 0; i < 2; ++i) {
        const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.kv.page_size, (cuuint64_t)a.kv.Hkv,
                                    (cuuint64_t)a.kv.num_pages};
        const cuuint64_t e = G::MX8 ? 1 : 2;  // bytes of an element
        const cuuint64_t strides[3] = {(cuuint64_t)a.kv.token_stride * e, (cuuint64_t)a.kv.head_stride * e,
                                       (cuuint64_t)a.kv.page_stride * e};
        const cuuint32_t box[4] = {G::MX8 ? (cuuint32_t)D : 64u, (cuuint32_t)p.page_rows, 1u, 1u};
        if (enc(&maps[2 + i], G::MX8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                i == 0 ? a.kv.k : a.kv.v, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                G::MX8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    static int configured_dev[64] = {0};
    if (ds.device < 64 && !configured_dev[ds.device]) {
        cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D, KVF>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             G::SMEM);
        if (e != cudaSuccess) return e;
        configured_dev[ds.device] = 1;
    }
    const int ctas = ds.num_sms < AT_MAX_CTAS ? ds.num_sms : AT_MAX_CTAS;
    return launch_k(attn_tc_kernel<D, KVF>, dim3(ctas), dim3(G::THREADS), G::SMEM, st, maps[0], maps[1], maps[2],
                    maps[3], p);
}

cudaError_t launch_attn_tc(const DeviceState &ds, cudaStream_t st, const AttnArgs &a)
{
    if (a.kv.kv_fmt == KV_MXFP8)
        return a.kv.D == 128 ? run_attn_tc<128, KV_MXFP8>(ds, st, a) : run_attn_tc<64, KV_MXFP8>(ds, st, a);
    return a.kv.D == 128 ? run_attn_tc<128, KV_BF16>(ds, st, a) : run_attn_tc<64, KV_BF16>(ds, st, a);
}

}  // namespace mx
