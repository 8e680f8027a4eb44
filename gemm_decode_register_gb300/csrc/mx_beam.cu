// mx_beam.cu -- the beams' selection over the vocabulary: the k best
// continuations of each batch entry's beams, sm_103a.
//
//   key(r, v) = score[r] + x[r][v] - lse_r,  lse_r = log sum_v e^x[r][v],
// over the tokens v that row r's mask allows; the k largest of a batch
// entry's W rows (bound: HBM, one pass over the logits).
//
// One launch.  The rows, laid end to end in steps of four
// 16-byte vectors per thread, are cut into equal stretches, one for each
// block that fits on the GPU; a block walks its own with the next two steps'
// copies to shared memory in flight (cp.async; each thread reads back its own),
// over row ends too.  Within a row the order of the keys is that
// of the logits, so a row's part of a stretch (a piece) needs no more of its row
// than itself:
//   - the largest element of each vector (packed maxima) and thread.  In the
//     first step each warp finds the r-th largest of its lanes' by r warp-wide
//     maxima; with r times the warps at least k, the smallest of these is a
//     bound that k elements reach, and not many more do;
//   - vectors that reach the bound go to a queue in shared memory.  When it
//     fills, and after 2, 8, 32, .. steps, a few threads take their elements
//     apart and the bound rises in the same way by what is found so far: so
//     each such stretch adds a few times k elements.  (A bisection to the k-th best cost
//     3 us each time, this 0.3.)  Rows whose later steps keep bringing better
//     elements get a bound from the step at hand too;
//   - exponentials are summed over the thread's own reference, a maximum that
//     is raised only when it falls behind by more than 10.
// At the end each element found counts those before it: its rank.
// The last block to finish a piece of a batch entry (a counter) joins its
// pieces: the rows' sums, the same bound from the heads of the pieces' lists (in fp32,
// with what its rounding may be off on either side), and the ranks of
// those that reach it by keys of 48 bits: near ties between beams are decided
// by bits that fp32 scores of -20 do not have.  Nothing depends on the order in
// which blocks finish.
// Where more elements reach a bound than the shared memory holds, both go
// slower ways to the same result: a piece through bisections over all of it, up to 64
// passes.  Ties do that, and in a piece logits that rise with the token: the
// bound of a step is the least of its warps', of which the first sees little of what
// is best, and the next step's vectors all reach it.  (Us for logits in any order, rising, and
// whole numbers: 4 beams over 32000, k = 8, 8, 38, 9; 128 over 128000, k = 16,
// 25, 534, 27; 1024 over 152000, k = 32, 95, 5200, 103, k = 128 207, 5700, 2900.)
#include <cfloat>
#include <cmath>
#include <cstddef>

#include "../../include/mx.h"
#include "mx_common.cuh"
#include "mx_serve.h"

namespace mx {

constexpr int BEAM_THREADS = 256;
constexpr int BEAM_WARPS = BEAM_THREADS / 32;
constexpr int BEAM_U = 4;                      // vectors of a thread and step
constexpr int BEAM_STEP = BEAM_THREADS * BEAM_U;  // vectors of a step
constexpr int BEAM_RING = 3;                      // steps in shared memory
constexpr int BEAM_BLOCKS = 3;                    // blocks of an SM
// Vectors that reach a piece's bound, and elements that do.  Between two rises of
// the bound some 4 k vectors come, more where bf16 logits are equal; too small
// a queue sends pieces the slow way (256: one seed's 1024 beams 104 us, another's 775).
constexpr int BEAM_QUEUE = 1024;
constexpr int BEAM_FOUND = 768;
constexpr int BEAM_JOIN = 1024;   // and a batch entry's
constexpr int BEAM_ENTRIES = 4096;  // of the lists, in the join's shared memory

struct BeamArgs {
    const void *logits;
    long long row_stride;
    const float *scores;
    const uint32_t *mask;
    long long mask_stride;
    int B, W, V, k, eos;
    int steps, span, pieces;  // steps of a row and of a stretch; most pieces of a row
    float *score, *next_score;
    int32_t *parent, *token, *next_parent, *next_token;
    float2 *sums;              // [rows][pieces] reference and sum
    unsigned long long *best;  // [rows][pieces][kpad] (logit, token) in order, 0 past the last
    int kpad;                  // k rounded up to 4
    int *count;                // [B] pieces that are done, zero between calls
};

// Whole numbers in the order of the values: -inf is 0x007FFFFF, +inf the
// largest but NaNs.  -0 and +0 must be made equal before.
__device__ __forceinline__ uint32_t ordered(float f)
{
    const uint32_t b = __float_as_uint(f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o)
{
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// The first stretch with a step of a row, and how many there are.  (All rows'
// steps are little more than 2^24: a row of 2^20 logits has 257, there are less than 2^16 rows.)
__device__ __forceinline__ int first_stretch(const BeamArgs &a, int row) { return (int)((unsigned)(row * a.steps) / (unsigned)a.span); }
__device__ __forceinline__ int pieces_of(const BeamArgs &a, int row)
{
    return (int)((unsigned)((row + 1) * a.steps - 1) / (unsigned)a.span) - first_stretch(a, row) + 1;
}

constexpr uint32_t ORD_NEG_INF = 0x007FFFFFu;

// (logit, token) as one whole number: larger logits first, the two zeros
// alike, then lower tokens.
__device__ __forceinline__ unsigned long long logit_token(float f, int v)
{
    return ((unsigned long long)ordered(f + 0.0f) << 32) | (0xFFFFFFFFu - (uint32_t)v);
}

// One element type's vectors.
template <typename E>
struct Elem;
template <>
struct Elem<uint16_t> {
    static constexpr int VEC = 8;
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    // Largest element; NaNs do not count.
    static __device__ __forceinline__ float top(const uint4 &v)
    {
        const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
        return fmaxf(bf16_lo(m), bf16_hi(m));
    }
    // Element number i of a row of vectors.
    static __device__ __forceinline__ float one(const uint4 *v, int i) { return bf16_to_f32(reinterpret_cast<const uint16_t *>(v)[i]); }
    // Elements whose bit is not set become -inf.
    static __device__ __forceinline__ void keep(uint4 &v, uint32_t bits)
    {
        uint32_t *w = &v.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t m = ((bits >> (2 * j) & 1u) * 0xFFFFu) | ((bits >> (2 * j + 1) & 1u) * 0xFFFF0000u);
            w[j] = (w[j] & m) | (0xFF80FF80u & ~m);
        }
    }
    static __device__ __forceinline__ float get(const uint4 &v, int j)
    {
        const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
        return (j & 1) ? bf16_hi(w) : bf16_lo(w);
    }
};
template <>
struct Elem<float> {
    static constexpr int VEC = 4;
    static __device__ __forceinline__ float top(const uint4 &v)
    {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ float one(const uint4 *v, int i) { return reinterpret_cast<const float *>(v)[i]; }
    static __device__ __forceinline__ void keep(uint4 &v, uint32_t bits)
    {
        uint32_t *w = &v.x;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (!(bits >> j & 1u)) w[j] = 0xFF800000u;
    }
    static __device__ __forceinline__ float get(const uint4 &v, int j)
    {
        return __uint_as_float(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w);
    }
};

// The r-th largest of the lanes' values, equal ones counted one by one; `next`
// gives what a lane holds after it lost its largest.
template <typename F>
__device__ __forceinline__ uint32_t warp_nth(uint32_t mine, int r, F next)
{
    const int lane = threadIdx.x & 31;
    for (;;) {
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, mine);
        if (--r == 0 || m == 0u) return m;
        if (lane == __ffs((int)__ballot_sync(0xFFFFFFFFu, mine == m)) - 1) mine = next();
    }
}

// The block's sum of the threads' numbers; scratch: BEAM_WARPS ints.
__device__ __forceinline__ int block_sum(int v, int *scratch)
{
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < BEAM_WARPS; ++w) s += scratch[w];
    return s;
}

// How many of n numbers are larger than c, and how many equal it; v on a
// 16-byte boundary.  (Four at a time without a branch: one by one with the order of
// equal ones beside it, 100 took 4 us.)
__device__ __forceinline__ int rank_of(const unsigned long long *v, int n, unsigned long long c, int &equal)
{
    int rank = 0, eq = 0, j = 0;
#pragma unroll 2
    for (; j + 4 <= n; j += 4) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(v + j), y = *reinterpret_cast<const ulonglong2 *>(v + j + 2);
        rank += (x.x > c) + (x.y > c) + (y.x > c) + (y.y > c);
        eq += (x.x == c) + (x.y == c) + (y.x == c) + (y.y == c);
    }
    for (; j < n; ++j) {
        rank += v[j] > c;
        eq += v[j] == c;
    }
    equal = eq;
    return rank;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A vector at the edge of a row: its elements lo .. hi - 1, -inf for the others.
// (A loop that shifts them in: rows have two such vectors at most, and the
// common path should not pay registers for them.)
__device__ __noinline__ uint4 edge_vector(const uint16_t *p, int lo, int hi)
{
    uint4 v;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = j >= lo && j < hi ? p[j] : 0xFF80u;
        v.x = __funnelshift_r(v.x, v.y, 16);
        v.y = __funnelshift_r(v.y, v.z, 16);
        v.z = __funnelshift_r(v.z, v.w, 16);
        v.w = v.w >> 16 | b << 16;
    }
    return v;
}
__device__ __noinline__ uint4 edge_vector(const float *p, int lo, int hi)
{
    uint4 v;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        v.x = v.y;
        v.y = v.z;
        v.z = v.w;
        v.w = j >= lo && j < hi ? __float_as_uint(p[j]) : 0xFF800000u;
    }
    return v;
}

// ---- join of one batch entry's pieces

// The total order: key, then beam, then (logit, token).
__device__ __forceinline__ bool before(unsigned long long ka, int ra, unsigned long long la, unsigned long long kb, int rb,
                                       unsigned long long lb)
{
    return ka != kb ? ka > kb : ra != rb ? ra < rb : la > lb;
}

// A number as the sum of two floats, the second what the first's rounding
// left: 48 bits at a few additions (fp64 has a sixteenth warp instruction per
// cycle here: the keys of one batch entry took 11 us).
struct Pair {
    float h, l;
};
// a + b, exactly.
__device__ __forceinline__ Pair two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}

// m + log t, t > 0.  t is a power of two times a number near 1, whose logarithm
// is small and so is its rounding; the power's logarithm is a pair.
__device__ __forceinline__ Pair log_sum(float m, float t)
{
    int e = (int)(__float_as_uint(t) >> 23) - 127;  // (t is 1 or more, but for rounding)
    float f = __uint_as_float((__float_as_uint(t) & 0x007FFFFFu) | 0x3F800000u);
    if (f > 1.4142135f) {
        f *= 0.5f;
        ++e;
    }
    // ln 2 in two parts (as Cody and Waite do), the first of 15 bits: its multiples are exact
    const float eh = (float)e * 0.693145751953125f, el = fmaf((float)e, 1.4286068e-6f, logf(f));
    const Pair p = two_sum(m, eh);
    const Pair q = two_sum(p.h, el);
    return two_sum(q.h, q.l + p.l);
}

struct JoinSmem {
    unsigned long long entry[BEAM_ENTRIES];  // the lists' first `staged`, list after list
    unsigned long long key[BEAM_JOIN], lt[BEAM_JOIN];
    uint8_t beam[BEAM_JOIN], beam_of[BEAM_ENTRIES / 4];  // a candidate's, a list's
    float score[BEAM_MAX_W];
    Pair lse[BEAM_MAX_W];  // NaN: the beam has no candidates
    float2 part[BEAM_MAX_W];
    uint32_t warp_bound[BEAM_WARPS];
    float out_score[BEAM_MAX_K];
    int out_parent[BEAM_MAX_K], out_token[BEAM_MAX_K], n_found, n_kept;
};

// Within `off` of a candidate's key, in fp32; NaN: no candidate.
__device__ __forceinline__ float key_about(const JoinSmem &sm, int row, unsigned long long l, float &off)
{
    const float c = sm.score[row], s = sm.lse[row].h, x = unordered((uint32_t)(l >> 32));
    off = (fabsf(c) + fabsf(x) + fabsf(s)) * 2.3841858e-7f;  // three roundings of a quarter of that, and one spare
    return l != 0ull ? c + (x - s) : NAN;
}
// The key as a whole number in its order: both floats of the pair.
__device__ __forceinline__ unsigned long long key_exact(const JoinSmem &sm, int row, unsigned long long l)
{
    const Pair d = two_sum(unordered((uint32_t)(l >> 32)), -sm.lse[row].h);
    const Pair k = two_sum(sm.score[row], d.h);
    const Pair f = two_sum(k.h, k.l + (d.l - sm.lse[row].l));
    return (unsigned long long)ordered(f.h + 0.0f) << 32 | ordered(f.l + 0.0f);
}

// More candidates than fit reach the bound (long ties between beams): one after
// the other, each the best of what follows the last.
__device__ __noinline__ void join_one_by_one(const BeamArgs &a, JoinSmem &sm, const unsigned long long *best, int b)
{
    const int tid = threadIdx.x, lists = a.W * a.pieces;
    unsigned long long pk = 0xFFFFFFFFFFFFFFFFull, pl = 0;
    int pr = -1;
    for (int i = 0; i < a.k; ++i) {
        unsigned long long mk = 0ull, ml = 0ull;
        int mr = 0x7FFFFFFF;
        for (int l = tid; l < lists; l += BEAM_THREADS) {
            const int row = l / a.pieces;
            if (!(sm.lse[row].h == sm.lse[row].h) || l - row * a.pieces >= pieces_of(a, b * a.W + row)) continue;
            for (int e = 0; e < a.k; ++e) {
                const unsigned long long h = __ldcg(best + (size_t)l * a.kpad + e);
                if (h == 0ull) break;
                const unsigned long long c = key_exact(sm, row, h);
                if (pr >= 0 && !before(pk, pr, pl, c, row, h)) continue;
                if (before(c, row, h, mk, mr, ml)) {
                    mk = c;
                    mr = row;
                    ml = h;
                }
                break;  // (the list's next are later in the order)
            }
        }
        __syncthreads();
        sm.key[tid] = mk;
        sm.lt[tid] = ml;
        sm.beam[tid] = (uint8_t)(mr & 255);
        __syncthreads();
        for (int j = 0; j < BEAM_THREADS; ++j)
            if (before(sm.key[j], sm.beam[j], sm.lt[j], mk, mr, ml)) {
                mk = sm.key[j];
                mr = sm.beam[j];
                ml = sm.lt[j];
            }
        pk = mk;
        pr = mr;
        pl = ml;
        if (tid == 0) {
            sm.out_score[i] = unordered((uint32_t)(mk >> 32));
            sm.out_parent[i] = b * a.W + mr;
            sm.out_token[i] = (int)(0xFFFFFFFFu - (uint32_t)ml);
        }
    }
}

// (Loops are left rolled: this code runs once per block, and what it takes is the
// fetching of its instructions more than their execution.)
__device__ __forceinline__ void beam_join(const BeamArgs &a, JoinSmem &sm, int b)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int lists = a.W * a.pieces;
    const unsigned long long *best = a.best + (size_t)b * lists * a.kpad;
    // as many of each list as fit, in groups of four (there are at most some 700 lists)
    const int depth = min(a.kpad / 4, max(1, BEAM_ENTRIES / 4 / lists)), staged = 4 * depth;

    const float own_score = tid < a.W ? __ldcg(a.scores + (size_t)b * a.W + tid) : 0.0f;
    // a warp per row: its sums, its lists
#pragma unroll 1
    for (int w = warp; w < a.W; w += BEAM_WARPS) {
        const size_t first = ((size_t)b * a.W + w) * a.pieces;
        const int pieces = pieces_of(a, b * a.W + w);
        float m = -INFINITY, t = 0.0f;
        // (a row has up to 257 pieces)
#pragma unroll 1
        for (int c0 = 0; c0 < a.pieces; c0 += 32) {
            const int c = c0 + lane;
            const float2 v = c < pieces ? __ldcg(a.sums + first + c) : make_float2(-INFINITY, 0.0f);
            const int entries = min(32, a.pieces - c0) * depth * 2;  // in pairs
#pragma unroll 4
            for (int i = lane; i < entries; i += 32) {
                const int l = i / (2 * depth), p = i - l * (2 * depth);  // list, pair
                ulonglong2 e = make_ulonglong2(0ull, 0ull);
                if (c0 + l < pieces) e = __ldcg(reinterpret_cast<const ulonglong2 *>(a.best + (first + c0 + l) * a.kpad) + p);
                reinterpret_cast<ulonglong2 *>(sm.entry)[(w * a.pieces + c0 + l) * (2 * depth) + p] = e;
            }
            if (c < a.pieces) sm.beam_of[w * a.pieces + c] = (uint8_t)w;
            const float nm = fmaxf(m, v.x);
            // (equal maxima, infinite ones too: no scaling; NaN sums stay)
            t = (m == nm ? t : t * __expf(m - nm)) + (v.x == nm ? v.y : v.y * __expf(v.x - nm));
            m = nm;
        }
        float top = m;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        t = m == top ? t : t * __expf(m - top);
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        if (lane == 0) sm.part[w] = make_float2(top, t);
    }
    if (tid == 0) sm.n_found = sm.n_kept = 0;
    __syncthreads();
    if (tid < a.W) {
        const float2 p = sm.part[tid];
        // NaN sums: a NaN or +inf among the logits; nothing allowed: no maximum
        const bool ok = p.y > 0.0f && fabsf(p.x) < INFINITY && fabsf(own_score) < INFINITY;
        sm.score[tid] = own_score;
        sm.lse[tid] = ok ? log_sum(p.x, p.y) : Pair{NAN, NAN};
    }
    __syncthreads();

    // A bound that k candidates reach, from one group of a list for each lane:
    // groups in the order of their depth, dealt out so that each warp sees all
    // beams and depths.
    const int groups = lists * depth, warps = min(BEAM_WARPS, (groups + 31) / 32);
    const int mine = lane * warps + (warp + lane + (lane >> 2)) % warps;
    uint32_t bound = 0xFFFFFFFFu;
    if (warp < warps) {
        uint32_t low[4] = {0u, 0u, 0u, 0u};
        // (of several groups of a lane, the one with the best head)
#pragma unroll 1
        for (int q = mine; q < groups; q += 32 * warps) {
            const int l = q % lists, row = sm.beam_of[l];
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float off;
                const float f = key_about(sm, row, sm.entry[l * staged + 4 * (q / lists) + i], off);
                v[i] = f > -INFINITY ? ordered((f - off) + 0.0f) : 0u;
            }
            if (v[0] > low[0]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) low[i] = v[i];
            }
        }
        // (rounded down in fp32, the entries still descend)
        bound = warp_nth(low[0], (a.k + warps - 1) / warps, [&] {
            low[0] = low[1];
            low[1] = low[2];
            low[2] = low[3];
            low[3] = 0u;
            return low[0];
        });
    }
    if (lane == 0) sm.warp_bound[warp] = bound;
    __syncthreads();
    bound = __reduce_min_sync(0xFFFFFFFFu, sm.warp_bound[lane % BEAM_WARPS]);
    float least = bound == 0u ? -FLT_MAX : unordered(bound);

    // what may reach it, of the staged entries, and of those behind them where a
    // list's last staged one does (lists descend)
    auto offer = [&](int row, unsigned long long l) {
        float off;
        const float f = key_about(sm, row, l, off);
        if (!(f + off >= least && f > -INFINITY)) return false;
        const int at = atomicAdd(&sm.n_found, 1);
        if (at < BEAM_JOIN) {
            sm.lt[at] = l;
            sm.beam[at] = (uint8_t)row;
        }
        return true;
    };
    // the bound again, from what was stored (each thread's best of up to four)
    auto raise = [&](int stored) {
        uint32_t low = 0u;
#pragma unroll 1
        for (int i = lane * BEAM_WARPS + warp; i < stored; i += BEAM_THREADS) {
            float off;
            const float f = key_about(sm, sm.beam[i], sm.lt[i], off);
            low = max(low, ordered((f - off) + 0.0f));
        }
        low = warp_nth(low, (a.k + BEAM_WARPS - 1) / BEAM_WARPS, [] { return 0u; });
        if (lane == 0) sm.warp_bound[warp] = low;
        __syncthreads();
        low = __reduce_min_sync(0xFFFFFFFFu, sm.warp_bound[lane % BEAM_WARPS]);
        return low == 0u ? -FLT_MAX : unordered(low);
    };
    int n;
#pragma unroll 1
    for (int turn = 0;; ++turn) {
#pragma unroll 1
        for (int e = tid; e < lists * staged; e += BEAM_THREADS) offer(sm.beam_of[e / staged], sm.entry[e]);
        if (staged < a.kpad)
#pragma unroll 1
            for (int l = tid; l < lists; l += BEAM_THREADS) {
                const int row = sm.beam_of[l];
                float off;
                const float f = key_about(sm, row, sm.entry[l * staged + staged - 1], off);
                if (!(f + off >= least)) continue;
#pragma unroll 1
                for (int e = staged; e < a.k && offer(row, __ldcg(best + (size_t)l * a.kpad + e)); ++e) {
                }
            }
        __syncthreads();
        n = sm.n_found;
        if (n <= 2 * a.k) break;
        // many: a better bound (ranks cost the square of their number); more than fit: again with that
        const float better = raise(min(n, BEAM_JOIN));
        const bool again = n > BEAM_JOIN && better > least && turn < 8;
        least = fmaxf(least, better);
        if (!again) break;
        if (tid == 0) sm.n_found = 0;
        __syncthreads();
    }
    if (n <= BEAM_JOIN) {
        unsigned long long *order = sm.entry;
#pragma unroll 1
        for (int i = tid; i < n; i += BEAM_THREADS) {
            const unsigned long long l = sm.lt[i];
            const int row = sm.beam[i];
            float off;
            const float f = key_about(sm, row, l, off);
            if (f + off < least) continue;
            const int at = atomicAdd(&sm.n_kept, 1);
            sm.key[at] = key_exact(sm, row, l);
            // the order of equal keys, in 58 bits: beam (6), logit (32), token (20)
            order[at] = (unsigned long long)(BEAM_MAX_W - 1 - row) << 52 | (l >> 32) << 20 | ((uint32_t)l & (BEAM_MAX_V - 1));
        }
        __syncthreads();
        n = sm.n_kept;
#pragma unroll 1
        for (int i = tid; i < n; i += BEAM_THREADS) {
            const unsigned long long ki = sm.key[i], li = order[i];
            int equal;
            int rank = rank_of(sm.key, n, ki, equal);
            if (equal > 1)  // (bf16 logits often are)
#pragma unroll 4
                for (int j = 0; j < n; ++j) rank += (sm.key[j] == ki) & (order[j] > li);
            if (rank < a.k) {
                sm.out_score[rank] = unordered((uint32_t)(ki >> 32));
                sm.out_parent[rank] = b * a.W + BEAM_MAX_W - 1 - (int)(li >> 52);
                sm.out_token[rank] = BEAM_MAX_V - 1 - (int)((uint32_t)li & (BEAM_MAX_V - 1));
            }
        }
        for (int i = n + tid; i < a.k; i += BEAM_THREADS) {
            sm.out_score[i] = -INFINITY;
            sm.out_parent[i] = -1;
            sm.out_token[i] = 0;
        }
    } else {
        join_one_by_one(a, sm, best, b);
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < a.k; i += BEAM_THREADS) {
        const size_t at = (size_t)b * a.k + i;
        a.score[at] = sm.out_score[i];
        a.parent[at] = sm.out_parent[i];
        a.token[at] = sm.out_token[i];
    }
    // the first W that do not end go on
    if (warp == 0 && a.next_token != nullptr) {
        int at = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < a.k && at < a.W; i0 += 32) {
            const int i = i0 + lane;
            const bool on = i < a.k && sm.out_parent[i] >= 0 && sm.out_token[i] != a.eos;
            const unsigned g = __ballot_sync(0xFFFFFFFFu, on);
            const int o = at + __popc(g & ((1u << lane) - 1u));
            if (on && o < a.W) {
                const size_t q = (size_t)b * a.W + o;
                a.next_score[q] = sm.out_score[i];
                a.next_parent[q] = sm.out_parent[i];
                a.next_token[q] = sm.out_token[i];
            }
            at += __popc(g);
        }
#pragma unroll 1
        for (int o = at + lane; o < a.W; o += 32) {
            const size_t q = (size_t)b * a.W + o;
            a.next_score[q] = -INFINITY;
            a.next_parent[q] = -1;
            a.next_token[q] = 0;
        }
    }
}

// ---- pieces

// Mask bits of the VEC elements from element e on (may be negative or past
// V: those bits do not count, their elements are -inf already).
template <int VEC>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t *row, int e, int words)
{
    if (e < 0) return mask_bits<VEC>(row, 0, words) << (-e);
    const int w = e >> 5;
    uint32_t lo = w < words ? __ldg(row + w) : 0u;
    const int s = e & 31;
    if (s + VEC > 32) {
        const uint32_t hi = w + 1 < words ? __ldg(row + w + 1) : 0u;
        return __funnelshift_r(lo, hi, s);
    }
    return lo >> s;
}

struct ChunkSmem {
    uint4 ring[BEAM_RING][BEAM_STEP];
    uint4 queue[BEAM_QUEUE];
    int queue_at[BEAM_QUEUE];  // the vector's first token
    unsigned long long found[BEAM_FOUND];
};
static_assert(sizeof(JoinSmem) <= sizeof(ChunkSmem), "the join's shared memory lies over the stretch's");
static_assert(offsetof(ChunkSmem, found) % 16 == 0 && offsetof(JoinSmem, key) % 16 == 0, "rank_of");
static_assert(BEAM_MAX_W == 64 && BEAM_MAX_V == 1 << 20, "the order of equal keys");
static_assert(BEAM_BLOCKS * (sizeof(ChunkSmem) + 1024 + 256) <= 228 * 1024, "blocks of an SM");

// 16 bytes to shared memory.
__device__ __forceinline__ void copy_async16(uint4 *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Too many elements of a piece reach its bound: the k largest
// (logit, token) of tokens t0 .. t1 - 1 into found, by bisection over the
// whole piece, read once per round.  Nothing outside [lo, ..) is among them.
template <typename E, bool MASK>
__device__ __noinline__ void piece_exact(const E *x, const uint32_t *mask, int t0, int t1, int V, int k, unsigned long long lo,
                                         unsigned long long *found, int *n_found, int *scratch)
{
    using L = Elem<E>;
    constexpr int VEC = L::VEC;
    auto each = [&](auto f) {
#pragma unroll 1
        for (int e = t0 + (int)threadIdx.x * VEC; e < t1; e += BEAM_THREADS * VEC) {
            uint4 v;
            if (e >= 0 && e + VEC <= V) v = __ldcg(reinterpret_cast<const uint4 *>(x + e));
            else v = edge_vector(x + e, e < 0 ? -e : 0, min(VEC, V - e));
            if constexpr (MASK) L::keep(v, mask_bits<VEC>(mask, e, (V + 31) >> 5));
#pragma unroll
            for (int j = 0; j < VEC; ++j) f(logit_token(L::get(v, j), e + j));
        }
    };
    unsigned long long hi = 0xFFFFFFFFFFFFFFFFull;
    while (lo < hi) {
        const unsigned long long mid = lo + (hi - lo) / 2 + 1;
        int c = 0;
        each([&](unsigned long long v) { c += v >= mid; });
        c = block_sum(c, scratch);
        if (c >= k) lo = mid;
        else hi = mid - 1;
        if (c == k) break;
    }
    __syncthreads();
    if (threadIdx.x == 0) *n_found = 0;
    __syncthreads();
    // (k at most, unless another stream writes the logits meanwhile)
    each([&](unsigned long long v) {
        if (v < lo) return;
        const int at = atomicAdd(n_found, 1);
        if (at < BEAM_FOUND) found[at] = v;
    });
}

template <typename E, bool MASK>
__global__ void __launch_bounds__(BEAM_THREADS, BEAM_BLOCKS) beam_kernel(const __grid_constant__ BeamArgs a)
{
    using L = Elem<E>;
    constexpr int VEC = L::VEC, U = BEAM_U;
    extern __shared__ __align__(16) uint8_t smem[];
    ChunkSmem &sm = *reinterpret_cast<ChunkSmem *>(smem);
    uint4 *queue = sm.queue;
    int *queue_at = sm.queue_at;
    unsigned long long *found = sm.found;
    __shared__ float warp_ref[BEAM_WARPS], warp_sum[BEAM_WARPS];
    __shared__ uint32_t warp_bound[BEAM_WARPS];
    __shared__ int n_queue[2], n_found, joins, scratch[BEAM_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    if (tid == 0) n_queue[0] = n_queue[1] = n_found = 0;
    int turn = 0;
    pdl_trigger();
    pdl_wait();
    const int words = (a.V + 31) >> 5;
    // a row, and the first token of its step 0: vectors are counted from the
    // 16-byte boundary at or before the row, and one that the row only partly
    // covers is read element by element
    struct Row {
        const E *x;
        int token0;
    };
    auto row_at = [&](int row) {
        const E *x = static_cast<const E *>(a.logits) + (size_t)row * a.row_stride;
        return Row{x, -(int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(E))};
    };
    // the step whose first token is e0: to the ring, and from there (or, of its
    // vectors that the row covers in part, element by element)
    auto fetch = [&](int slot, const E *x, int e0) {
        uint4 *d = &sm.ring[slot][tid];
        const uint4 *p = reinterpret_cast<const uint4 *>(x + e0) + tid;
        if (e0 >= 0 && e0 + BEAM_STEP * VEC <= a.V) {
#pragma unroll
            for (int u = 0; u < U; ++u) copy_async16(d + u * BEAM_THREADS, p + u * BEAM_THREADS);
        } else {
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                const int e = e0 + (u * BEAM_THREADS + tid) * VEC;
                if (e >= 0 && e + VEC <= a.V) copy_async16(d + u * BEAM_THREADS, p + u * BEAM_THREADS);
            }
        }
    };
    auto take = [&](uint4 (&v)[U], int slot, const E *x, int e0) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = sm.ring[slot][u * BEAM_THREADS + tid];
        if (e0 < 0 || e0 + BEAM_STEP * VEC > a.V) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = e0 + (u * BEAM_THREADS + tid) * VEC;
                if (e < 0 || e + VEC > a.V) v[u] = edge_vector(x + e, e < 0 ? -e : 0, min(VEC, a.V - e));
            }
        }
    };
    auto load_bits = [&](uint32_t (&bits)[U], int row, int e0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            bits[u] = mask_bits<VEC>(a.mask + (size_t)row * a.mask_stride, e0 + (u * BEAM_THREADS + tid) * VEC, words);
    };

    float bound = -FLT_MAX;  // (-inf is no candidate)
    bool lost = false;       // more reach it than there is room for
    // raises it to what k of the threads' values reach, of which the first
    // `have` threads have one: r lanes of each of their warps.  Two barriers.
    auto raise = [&](float v, int have) {
        const int warps = max(1, min(BEAM_WARPS, (have + 31) / 32)), r = (a.k + warps - 1) / warps;
        uint32_t n = 0xFFFFFFFFu;  // (no values, no say)
        if (warp < warps) n = r > 32 ? 0u : warp_nth(ordered(v + 0.0f), r, [] { return 0u; });
        if (lane == 0) warp_bound[warp] = n;
        __syncthreads();
        n = __reduce_min_sync(0xFFFFFFFFu, warp_bound[lane % BEAM_WARPS]);
        if (n > ORD_NEG_INF) bound = fmaxf(bound, unordered(n));
        __syncthreads();
    };
    // the bound from what is found so far, dealt out over the warps (each
    // thread's largest of three); what no longer reaches it is dropped.  n: how
    // much is found, as everyone has read it before a barrier of `raise`.
    auto sift = [&](int n) {
        constexpr int F = BEAM_FOUND / BEAM_THREADS;
        unsigned long long mine[F];
        uint32_t v = 0u;
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int at = (i * 32 + lane) * BEAM_WARPS + warp;
            mine[i] = at < n ? found[at] : 0ull;
            v = max(v, (uint32_t)(mine[i] >> 32));
        }
        raise(v > ORD_NEG_INF ? unordered(v) : -INFINITY, BEAM_THREADS);
        if (tid == 0) n_found = 0;
        __syncthreads();
        const unsigned long long lo = (unsigned long long)ordered(bound + 0.0f) << 32;
#pragma unroll
        for (int i = 0; i < F; ++i)
            if (mine[i] >= lo) found[atomicAdd(&n_found, 1)] = mine[i];
        __syncthreads();
    };

    // The queue's elements that reach the bound are found, a thread for each
    // vector, and sifted; later pushes go to the other counter.  (The code of
    // loops that run a few times is left rolled: it is fetched more than run.)
    auto drain = [&] {
        const int n = min(n_queue[turn], BEAM_QUEUE);
        lost |= n_queue[turn] > BEAM_QUEUE;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += BEAM_THREADS) {
            const int i = i0 + tid;
            unsigned hits = 0u;
            if (i < n) {
                const uint4 v = queue[i];
#pragma unroll
                for (int j = 0; j < VEC; ++j) hits |= (L::get(v, j) >= bound ? 1u : 0u) << j;
            }
            int o = __popc(hits);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int before = __shfl_up_sync(0xFFFFFFFFu, o, d);
                if (lane >= d) o += before;
            }
            int base = 0;
            if (lane == 31 && o > 0) base = atomicAdd(&n_found, o);
            o += __shfl_sync(0xFFFFFFFFu, base, 31) - __popc(hits);
            for (; hits; hits &= hits - 1, ++o) {
                const int j = __ffs((int)hits) - 1;
                if (o < BEAM_FOUND) found[o] = logit_token(L::one(queue, i * VEC + j), queue_at[i] + j);
            }
            __syncthreads();
            const int f = n_found;
            lost |= f > BEAM_FOUND;
            if (lost) break;
            // (Fewer are ranked sooner than sifted: 128 beams over 128000 tokens 26.4 us if every
            // number is sifted, 25.9 so, 27.1 if only what is above BEAM_THREADS is; 1024, k = 32, 96.8, 96.7
            // and 102.4.  k = 128 would rather have the last: 202 us for 214.)
            if (f > BEAM_THREADS / 4) sift(f);
            else __syncthreads();               // (everyone has read the count)
        }
        if (tid == 0) n_queue[turn] = 0;
        turn ^= 1;
    };

    const long long end = min((long long)(blockIdx.x + 1) * a.span, (long long)a.B * a.W * a.steps);
    long long at = (long long)blockIdx.x * a.span;
    int row = (int)(at / a.steps), step = (int)(at - (long long)row * a.steps), first = step;
    Row here = row_at(row);
    int token0 = here.token0 + step * BEAM_STEP * VEC;
    // the step that is fetched next, and its number (of the stretch)
    Row ahead = here;
    int arow = row, astep = step, ahead_n = 0;
    const int steps = (int)(end - at);
    auto fetch_next = [&] {
        if (ahead_n < steps) {
            fetch(ahead_n % BEAM_RING, ahead.x, ahead.token0 + astep * BEAM_STEP * VEC);
            if (++astep == a.steps && ahead_n + 1 < steps) {
                astep = 0;
                ahead = row_at(++arow);
            }
        }
        ++ahead_n;
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < BEAM_RING - 1; ++i) fetch_next();
    uint4 cur[U];
    uint32_t bits[U];
    float ref = -INFINITY;
    float2 sum2 = make_float2(0.0f, 0.0f);
    bool hot = true;
    for (int i = 0; i < steps; ++i) {
        const bool row_ends = step + 1 == a.steps, last = row_ends || i + 1 == steps;  // of the piece
        fetch_next();
        if constexpr (MASK) load_bits(bits, row, token0);
        copy_wait<BEAM_RING - 1>();
        take(cur, i % BEAM_RING, here.x, token0);
        if constexpr (MASK) {
#pragma unroll
            for (int u = 0; u < U; ++u) L::keep(cur[u], bits[u]);
        }
        float top[U], m = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            top[u] = L::top(cur[u]);
            m = fmaxf(m, top[u]);
        }
        if (hot) raise(m, (a.V - token0 + VEC - 1) / VEC);
        bool filling = false;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (top[u] >= bound) {
                const int i = atomicAdd(&n_queue[turn], 1);
                filling |= i >= BEAM_QUEUE / 2;
                if (i < BEAM_QUEUE) {
                    queue[i] = cur[u];
                    queue_at[i] = token0 + (u * BEAM_THREADS + tid) * VEC;
                }
            }
        if (m > ref + 10.0f) {  // (the first time too)
            const float s = ref > -INFINITY ? __expf(ref - m) : 1.0f;
            sum2.x *= s;
            sum2.y *= s;
            ref = m;
        }
        // (x - reference before the factor: its rounding stays relative to the
        // difference, whatever the size of x)
        const float off = ref > -INFINITY ? -ref : 0.0f;
        const float2 shift = make_float2(off, off), log2e = make_float2(1.4426950408889634f, 1.4426950408889634f);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {
                const float2 d = mul2(add2(make_float2(L::get(cur[u], j), L::get(cur[u], j + 1)), shift), log2e);
                sum2 = add2(sum2, make_float2(exp2_fast(d.x), exp2_fast(d.y)));
            }
        if (last) {
            // the warp's sum, over its largest reference
            float wr = ref, ws = sum2.x + sum2.y;
#pragma unroll
            for (int o = 16; o; o >>= 1) wr = fmaxf(wr, __shfl_xor_sync(0xFFFFFFFFu, wr, o));
            ws = ref == wr ? ws : ws * __expf(ref - wr);
#pragma unroll
            for (int o = 16; o; o >>= 1) ws += __shfl_xor_sync(0xFFFFFFFFu, ws, o);
            if (lane == 0) {
                warp_ref[warp] = wr;
                warp_sum[warp] = ws;
            }
        }
        hot = __syncthreads_or(filling);  // (n_queue itself may have grown by another's next step)
        const int done = step - first + 1;
        // (2, 8, 32, .. steps.  1, 2, 4, .. take longer: 1024 beams over 152000 tokens, k = 32, 102 us
        // for 97, k = 128 212 for 206; 128 over 128000, k = 128, 72 for 66)
        if (last || hot || ((done & (done - 1)) == 0 && (done & 0x2AAAAAAA) != 0)) drain();
        if (last) {
            // ---- the piece ends
            const size_t list = (size_t)row * a.pieces + (blockIdx.x - first_stretch(a, row));
            if (warp == 0) {
                const float wr = warp_ref[lane % BEAM_WARPS];
                float top = wr, s = lane < BEAM_WARPS ? warp_sum[lane] : 0.0f;
#pragma unroll
                for (int o = 4; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                s = wr == top ? s : s * __expf(wr - top);
#pragma unroll
                for (int o = 4; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
                if (lane == 0) a.sums[list] = make_float2(top, s);
            }
            if (lost)
                piece_exact<E, MASK>(here.x, MASK ? a.mask + (size_t)row * a.mask_stride : nullptr,
                                     here.token0 + first * BEAM_STEP * VEC, min(a.V, here.token0 + (step + 1) * BEAM_STEP * VEC),
                                     a.V, a.k, (unsigned long long)ordered(bound + 0.0f) << 32, found, &n_found, scratch);
            __syncthreads();
            const int n = min(n_found, BEAM_FOUND);
            unsigned long long *best = a.best + list * a.kpad;
            for (int i = tid; i < n; i += BEAM_THREADS) {
                const unsigned long long c = found[i];
                int equal;
                const int rank = rank_of(found, n, c, equal);
                if (rank < a.k) best[rank] = c;
            }
            for (int i = min(n, a.k) + tid; i < a.kpad; i += BEAM_THREADS) best[i] = 0ull;
            __syncthreads();
            if (tid == 0) n_found = 0;  // (the next piece begins with two barriers)
            first = 0;
            bound = -FLT_MAX;
            ref = -INFINITY;
            sum2 = make_float2(0.0f, 0.0f);
            hot = true;
            lost = false;
        }
        token0 += BEAM_STEP * VEC;
        ++step;
        if (row_ends && i + 1 < steps) {
            here = row_at(++row);
            token0 = here.token0;
            step = 0;
        }
    }
    copy_wait<0>();

    // ---- this block's pieces are done: batch entries that are complete are joined
    const int row0 = (int)((long long)blockIdx.x * a.span / a.steps), row1 = (int)((end - 1) / a.steps);
    for (int b = row0 / a.W; b <= row1 / a.W; ++b) {
        __syncthreads();
        if (warp == 0) {
            const int done = min(row1, (b + 1) * a.W - 1) - max(row0, b * a.W) + 1;
            int total = 0;
            for (int w = lane; w < a.W; w += 32) total += pieces_of(a, b * a.W + w);
            total = __reduce_add_sync(0xFFFFFFFFu, total);
            if (lane == 0) {
                // (of what the block wrote before the barrier, and of what is read after the next)
                int before;
                asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(before) : "l"(a.count + b), "r"(done) : "memory");
                joins = before + done == total;
                if (joins) a.count[b] = 0;
            }
        }
        __syncthreads();
        if (joins) beam_join(a, *reinterpret_cast<JoinSmem *>(smem), b);
    }
}

// ------------------------------------------------------------ host

// Steps of a row, of a stretch, and the most pieces of a row.  As many
// stretches as blocks fit on the GPU.
constexpr long long BEAM_SMS = 152;
struct BeamSplit {
    int steps, span, pieces, stretches;
};
static BeamSplit beam_split(int rows, int V, int vec)
{
    BeamSplit s;
    // (a row may begin inside its first vector)
    s.steps = ((V + vec - 1 + vec - 1) / vec + BEAM_STEP - 1) / BEAM_STEP;
    const long long total = (long long)rows * s.steps, blocks = BEAM_SMS * BEAM_BLOCKS;
    s.span = (int)((total + blocks - 1) / blocks);
    s.pieces = (s.steps + s.span - 1) / s.span + (s.steps % s.span != 0 ? 1 : 0);
    s.stretches = (int)((total + s.span - 1) / s.span);
    return s;
}

static size_t beam_lists(int B, int W, int V, int vec)
{
    return (size_t)B * W * beam_split(B * W, V, vec).pieces;
}

size_t beam_workspace_bytes(int B, int W, int V, int k)
{
    const size_t l4 = beam_lists(B, W, V, 4), l8 = beam_lists(B, W, V, 8);  // fp32, bf16
    return ((l4 > l8 ? l4 : l8) * (((size_t)k + 3) / 4 * 4 + 1) * 8 + 255) / 256 * 256;
}

template <typename E>
static cudaError_t run_beam(const DeviceState &ds, cudaStream_t st, const BeamArgs &a, int stretches)
{
    const dim3 grid((unsigned)stretches);
    static unsigned char plain[64], masked[64];
    auto kernel = a.mask ? beam_kernel<E, true> : beam_kernel<E, false>;
    const cudaError_t e = allow_smem(ds, kernel, (int)sizeof(ChunkSmem), a.mask ? masked : plain);
    return e != cudaSuccess ? e : launch_k(kernel, grid, dim3(BEAM_THREADS), sizeof(ChunkSmem), st, a);
}

cudaError_t launch_beam_select(const DeviceState &ds, cudaStream_t st, const BeamCall &c, void *workspace)
{
    const int vec = c.dtype == MX_F32 ? 4 : 8;
    const BeamSplit split = beam_split(c.B * c.W, c.V, vec);
    BeamArgs a;
    a.logits = c.logits;
    a.row_stride = c.row_stride;
    a.scores = c.scores;
    a.mask = c.mask;
    a.mask_stride = c.mask_stride;
    a.B = c.B;
    a.W = c.W;
    a.V = c.V;
    a.k = c.k;
    a.eos = c.eos;
    a.steps = split.steps;
    a.span = split.span;
    a.pieces = split.pieces;
    a.score = c.score;
    a.parent = c.parent;
    a.token = c.token;
    a.next_score = c.next_score;
    a.next_parent = c.next_parent;
    a.next_token = c.next_token;
    const size_t lists = (size_t)c.B * c.W * a.pieces;
    a.kpad = (c.k + 3) / 4 * 4;
    a.count = ds.ws_count;
    a.best = static_cast<unsigned long long *>(workspace);
    a.sums = reinterpret_cast<float2 *>(a.best + lists * a.kpad);
    return c.dtype == MX_F32 ? run_beam<float>(ds, st, a, split.stretches) : run_beam<uint16_t>(ds, st, a, split.stretches);
}

}  // namespace mx
