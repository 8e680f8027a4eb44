// mx_beam.cu -- the beams' selection over the vocabulary: the k best
// continuations of each batch entry's beams, sm_103a.
//
//   key(r, v) = score[r] + x[r][v] - lse_r,  lse_r = log sum_v e^x[r][v],
// over the tokens v that row r's mask allows; the k largest of a batch
// entry's W rows (bound: HBM, one pass over the logits).
//
// One launch.  The rows, laid end to end in steps of four
// 16-byte vectors per thread, are cut into equal stretches, one for each
// block that fits on the GPU; a block walks its own with the next step's loads
// in flight, over row ends too.  Within a row the order of the keys is that
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
// Where ties let more elements reach a bound than the shared memory holds,
// both go slower ways to the same result.
#include <cfloat>
#include <cmath>

#include "../../include/mx.h"
#include "mx_common.cuh"
#include "mx_serve.h"

namespace mx {

constexpr int BEAM_THREADS = 256;
constexpr int BEAM_WARPS = BEAM_THREADS / 32;
constexpr int BEAM_U = 4;                      // vectors of a thread and step
constexpr int BEAM_STEP = BEAM_THREADS * BEAM_U;  // vectors of a step
constexpr int BEAM_QUEUE = 512;   // vectors that reach a piece's bound
constexpr int BEAM_FOUND = 1024;  // elements that do (a piece's, a batch entry's)

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
// The first stretch with a step of a row, and how many there are.
__device__ __forceinline__ int first_stretch(const BeamArgs &a, int row) { return (int)((long long)row * a.steps / a.span); }
__device__ __forceinline__ int pieces_of(const BeamArgs &a, int row)
{
    return (int)(((long long)(row + 1) * a.steps - 1) / a.span) - first_stretch(a, row) + 1;
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
    float score[BEAM_MAX_W];
    Pair lse[BEAM_MAX_W];  // NaN: the beam has no candidates
    float2 part[BEAM_MAX_W];
    unsigned long long key[BEAM_FOUND], lt[BEAM_FOUND];
    uint8_t beam[BEAM_FOUND];
    uint32_t warp_bound[BEAM_WARPS];
    float out_score[BEAM_MAX_K];
    int out_parent[BEAM_MAX_K], out_token[BEAM_MAX_K], n_found;
};

__device__ __forceinline__ void beam_join(const BeamArgs &a, JoinSmem &sm, int b)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int lists = a.W * a.pieces;
    const unsigned long long *best = a.best + (size_t)b * lists * a.kpad;
    float *score = sm.score, *out_score = sm.out_score;
    Pair *lse = sm.lse;
    unsigned long long *key = sm.key, *lt = sm.lt;
    uint8_t *beam = sm.beam;
    int *out_parent = sm.out_parent, *out_token = sm.out_token;

    // Four entries of a list are a group; groups in the order of their depth,
    // then of the list.  The first R groups of each thread stay in registers.
    // (lane, warp) -> group: each warp sees all beams and depths.
    constexpr int R = 3;
    const int groups = lists * (a.kpad / 4), warps = min(BEAM_WARPS, (groups + 31) / 32);
    const int mine = warp < warps ? lane * warps + (warp + lane + (lane >> 2)) % warps : groups;
    struct Group {
        unsigned long long v[4];
        int row;
    };
    auto fetch = [&](int g) {
        Group q;
        const int l = g % lists, d = g / lists;
        q.row = l / a.pieces;
        if (l - q.row * a.pieces >= pieces_of(a, b * a.W + q.row)) {
            q.v[0] = q.v[1] = q.v[2] = q.v[3] = 0ull;
            return q;
        }
        const ulonglong2 *p = reinterpret_cast<const ulonglong2 *>(best + (size_t)l * a.kpad + 4 * d);
        const ulonglong2 x = __ldcg(p), y = __ldcg(p + 1);
        q.v[0] = x.x;
        q.v[1] = x.y;
        q.v[2] = y.x;
        q.v[3] = y.y;
        return q;
    };
    Group q[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int g = mine + i * 32 * warps;
        if (g < groups) q[i] = fetch(g);
        else q[i] = Group{{0ull, 0ull, 0ull, 0ull}, 0};
    }
    const float own_score = tid < a.W ? __ldcg(a.scores + (size_t)b * a.W + tid) : 0.0f;
    // the rows' sums
    for (int w = warp; w < a.W; w += BEAM_WARPS) {
        const float2 *p = a.sums + ((size_t)b * a.W + w) * a.pieces;
        const int pieces = pieces_of(a, b * a.W + w);
        float m = -INFINITY, t = 0.0f;
        for (int c = lane; c < pieces; c += 32) {
            const float2 v = __ldcg(p + c);
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
    if (tid == 0) sm.n_found = 0;
    __syncthreads();
    if (tid < a.W) {
        const float2 p = sm.part[tid];
        // NaN sums: a NaN or +inf among the logits; nothing allowed: no maximum
        const bool ok = p.y > 0.0f && fabsf(p.x) < INFINITY && fabsf(own_score) < INFINITY;
        score[tid] = own_score;
        lse[tid] = ok ? log_sum(p.x, p.y) : Pair{NAN, NAN};
    }
    __syncthreads();

    // Within `off` of a candidate's key, in fp32; NaN: no candidate.
    auto about = [&](int row, unsigned long long l, float &off) {
        const float c = score[row], s = lse[row].h, x = unordered((uint32_t)(l >> 32));
        off = (fabsf(c) + fabsf(x) + fabsf(s)) * 2.3841858e-7f;  // three roundings of a quarter of that, and one spare
        return l != 0ull ? c + (x - s) : NAN;
    };
    // The key as a whole number in its order: both floats of the pair.
    auto exact = [&](int row, unsigned long long l) {
        const Pair d = two_sum(unordered((uint32_t)(l >> 32)), -lse[row].h);
        const Pair k = two_sum(score[row], d.h);
        const Pair f = two_sum(k.h, k.l + (d.l - lse[row].l));
        return (unsigned long long)ordered(f.h + 0.0f) << 32 | ordered(f.l + 0.0f);
    };
    // A bound that k candidates reach, from the thread's first group.
    uint32_t bound = 0xFFFFFFFFu;
    if (warp < warps) {
        uint32_t low[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float off;
            const float f = about(q[0].row, q[0].v[i], off);
            low[i] = f > -INFINITY ? ordered((f - off) + 0.0f) : 0u;
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
    const float least = bound == 0u ? -FLT_MAX : unordered(bound);

    // what may reach it
    auto gather = [&](const Group &p) {
        bool any = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float off;
            const float f = about(p.row, p.v[j], off);
            if (f + off >= least && f > -INFINITY) {
                const int at = atomicAdd(&sm.n_found, 1);
                if (at < BEAM_FOUND) {
                    lt[at] = p.v[j];
                    beam[at] = (uint8_t)p.row;
                }
                any = true;
            }
        }
        return any;
    };
#pragma unroll
    for (int i = 0; i < R; ++i) gather(q[i]);
    // more groups than registers: until as many in a row as there are lists
    // have nothing (lists descend)
    for (int g0 = R * 32 * warps, idle = 0; g0 < groups && idle < lists; g0 += BEAM_THREADS) {
        const bool any = g0 + tid < groups && gather(fetch(g0 + tid));
        idle = __syncthreads_or(any) ? 0 : idle + BEAM_THREADS;
    }
    __syncthreads();
    const int n = sm.n_found;
    if (n <= BEAM_FOUND) {
        for (int i = tid; i < n; i += BEAM_THREADS) key[i] = exact(beam[i], lt[i]);
        __syncthreads();
        for (int i = tid; i < n; i += BEAM_THREADS) {
            const unsigned long long ki = key[i], li = lt[i];
            const int ri = beam[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) {
                const unsigned long long kj = key[j];
                rank += kj > ki || (kj == ki && before(kj, beam[j], lt[j], ki, ri, li));
            }
            if (rank < a.k) {
                out_score[rank] = unordered((uint32_t)(ki >> 32));
                out_parent[rank] = b * a.W + ri;
                out_token[rank] = (int)(0xFFFFFFFFu - (uint32_t)li);
            }
        }
        for (int i = n + tid; i < a.k; i += BEAM_THREADS) {
            out_score[i] = -INFINITY;
            out_parent[i] = -1;
            out_token[i] = 0;
        }
    } else {
        // more than fit (long ties between beams): one after the other, each
        // the best of what follows the last
        unsigned long long pk = 0xFFFFFFFFFFFFFFFFull, pl = 0;
        int pr = -1;
        for (int i = 0; i < a.k; ++i) {
            unsigned long long mk = 0ull, ml = 0ull;
            int mr = 0x7FFFFFFF;
            for (int l = tid; l < lists; l += BEAM_THREADS) {
                const int row = l / a.pieces;
                if (!(lse[row].h == lse[row].h) || l - row * a.pieces >= pieces_of(a, b * a.W + row)) continue;
                for (int e = 0; e < a.k; ++e) {
                    const unsigned long long h = __ldcg(best + (size_t)l * a.kpad + e);
                    if (h == 0ull) break;
                    const unsigned long long c = exact(row, h);
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
            key[tid] = mk;
            lt[tid] = ml;
            beam[tid] = (uint8_t)(mr & 255);
            __syncthreads();
            for (int j = 0; j < BEAM_THREADS; ++j)
                if (before(key[j], beam[j], lt[j], mk, mr, ml)) {
                    mk = key[j];
                    mr = beam[j];
                    ml = lt[j];
                }
            pk = mk;
            pr = mr;
            pl = ml;
            if (tid == 0) {
                out_score[i] = unordered((uint32_t)(mk >> 32));
                out_parent[i] = b * a.W + mr;
                out_token[i] = (int)(0xFFFFFFFFu - (uint32_t)ml);
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < a.k; i += BEAM_THREADS) {
        const size_t at = (size_t)b * a.k + i;
        a.score[at] = out_score[i];
        a.parent[at] = out_parent[i];
        a.token[at] = out_token[i];
    }
    // the first W that do not end go on
    if (warp == 0 && a.next_token != nullptr) {
        int at = 0;
        for (int i0 = 0; i0 < a.k && at < a.W; i0 += 32) {
            const int i = i0 + lane;
            const bool on = i < a.k && out_parent[i] >= 0 && out_token[i] != a.eos;
            const unsigned g = __ballot_sync(0xFFFFFFFFu, on);
            const int o = at + __popc(g & ((1u << lane) - 1u));
            if (on && o < a.W) {
                const size_t q = (size_t)b * a.W + o;
                a.next_score[q] = out_score[i];
                a.next_parent[q] = out_parent[i];
                a.next_token[q] = out_token[i];
            }
            at += __popc(g);
        }
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
    uint4 queue[BEAM_QUEUE];
    int queue_at[BEAM_QUEUE];  // the vector's first token
    unsigned long long found[BEAM_FOUND];
};

template <typename E, bool MASK>
__global__ void __launch_bounds__(BEAM_THREADS, MASK ? 2 : 4) beam_kernel(const __grid_constant__ BeamArgs a)
{
    using L = Elem<E>;
    constexpr int VEC = L::VEC, U = BEAM_U;
    __shared__ __align__(16) uint8_t smem[sizeof(ChunkSmem) > sizeof(JoinSmem) ? sizeof(ChunkSmem) : sizeof(JoinSmem)];
    uint4 *queue = reinterpret_cast<ChunkSmem *>(smem)->queue;
    int *queue_at = reinterpret_cast<ChunkSmem *>(smem)->queue_at;
    unsigned long long *found = reinterpret_cast<ChunkSmem *>(smem)->found;
    __shared__ float warp_ref[BEAM_WARPS], warp_sum[BEAM_WARPS];
    __shared__ uint32_t warp_bound[BEAM_WARPS];
    __shared__ int n_queue, n_found, joins, scratch[BEAM_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    if (tid == 0) n_queue = n_found = 0;
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
    auto load = [&](uint4 (&v)[U], const Row &r, int e0) {  // the step whose first token is e0
        if (e0 >= 0 && e0 + BEAM_STEP * VEC <= a.V) {
            const uint4 *p = reinterpret_cast<const uint4 *>(r.x + e0) + tid;
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = __ldcs(p + u * BEAM_THREADS);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = e0 + (u * BEAM_THREADS + tid) * VEC;
                if (e >= 0 && e + VEC <= a.V) v[u] = __ldcs(reinterpret_cast<const uint4 *>(r.x + e));
                else v[u] = edge_vector(r.x + e, e < 0 ? -e : 0, min(VEC, a.V - e));
            }
        }
    };
    auto load_bits = [&](uint32_t (&bits)[U], int row, int e0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            bits[u] = mask_bits<VEC>(a.mask + (size_t)row * a.mask_stride, e0 + (u * BEAM_THREADS + tid) * VEC, words);
    };

    float bound = -FLT_MAX;  // (-inf is no candidate)
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
    // the queue's elements that reach the bound are found, a thread for each; the
    // queue is empty after it
    auto drain = [&] {
        const int n = min(n_queue, BEAM_QUEUE) * VEC;
        for (int i0 = 0; i0 < n; i0 += BEAM_THREADS) {
            const int i = i0 + tid;
            const float f = i < n ? L::one(queue, i) : -INFINITY;
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, f >= bound);
            if (hit == 0u) continue;
            int o = 0;
            if (lane == 0) o = atomicAdd(&n_found, __popc(hit));
            o = __shfl_sync(0xFFFFFFFFu, o, 0) + __popc(hit & ((1u << lane) - 1u));
            if (f >= bound && o < BEAM_FOUND) found[o] = logit_token(f, queue_at[i / VEC] + i % VEC);
        }
        __syncthreads();
        if (tid == 0) n_queue = 0;
    };
    // the bound from what is found so far, dealt out over the warps: each
    // thread's largest of up to four
    auto raise_by_found = [&] {
        const int n = n_found;
        uint32_t v = 0u;
        for (int i = lane * BEAM_WARPS + warp; i < n; i += BEAM_THREADS) v = max(v, (uint32_t)(found[i] >> 32));
        raise(v > ORD_NEG_INF ? unordered(v) : -INFINITY, BEAM_THREADS);
    };

    const long long end = min((long long)(blockIdx.x + 1) * a.span, (long long)a.B * a.W * a.steps);
    long long at = (long long)blockIdx.x * a.span;
    int row = (int)(at / a.steps), step = (int)(at - (long long)row * a.steps), first = step;
    Row r = row_at(row);
    int token0 = r.token0 + step * BEAM_STEP * VEC;
    uint4 cur[U], nxt[U];
    uint32_t bits[U], nbits[U];
    load(cur, r, token0);
    if constexpr (MASK) load_bits(bits, row, token0);
    float ref = -INFINITY;
    float2 sum2 = make_float2(0.0f, 0.0f);
    bool hot = true, lost = false;
    for (; at < end; ++at) {
        const bool row_ends = step + 1 == a.steps, last = row_ends || at + 1 == end;  // of the piece
        const Row here = r;
        int ntoken0 = token0 + BEAM_STEP * VEC;
        if (at + 1 < end) {
            if (row_ends) {
                r = row_at(row + 1);
                ntoken0 = r.token0;
            }
            load(nxt, r, ntoken0);
            if constexpr (MASK) load_bits(nbits, row + row_ends, ntoken0);
        }
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
                const int i = atomicAdd(&n_queue, 1);
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
        if (!last) {
            hot = __syncthreads_or(filling);  // (n_queue itself may have grown by another's next step)
            const int done = step - first + 1;
            // (2, 8, 32, .. steps; for many candidates every power of two)
            if (hot || ((done & (done - 1)) == 0 && (done & (a.k > 48 ? ~1 : 0x2AAAAAAA)) != 0)) {
                lost |= n_queue > BEAM_QUEUE;
                __syncthreads();
                drain();
                lost |= n_found > BEAM_FOUND;
                __syncthreads();
                if (!lost) raise_by_found();
            }
        } else {
            // ---- the piece ends: its sums, over the largest reference
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
            __syncthreads();
            const size_t list = (size_t)row * a.pieces + (blockIdx.x - first_stretch(a, row));
            if (warp == 0) {
                const float wr8 = warp_ref[lane % BEAM_WARPS];
                float top = wr8, s = lane < BEAM_WARPS ? warp_sum[lane] : 0.0f;
#pragma unroll
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                s = wr8 == top ? s : s * __expf(wr8 - top);
#pragma unroll
                for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
                if (lane == 0) a.sums[list] = make_float2(top, s);
            }
            lost |= n_queue > BEAM_QUEUE;
            __syncthreads();
            drain();
            lost |= n_found > BEAM_FOUND;
            __syncthreads();
            if (!lost) {
                const int n = n_found;
                if (n > BEAM_THREADS / 2) {  // (fewer are ranked sooner than sifted)
                    raise_by_found();
                    // what no longer reaches the bound is dropped
                    constexpr int F = BEAM_FOUND / BEAM_THREADS;
                    unsigned long long mine[F];
#pragma unroll
                    for (int i = 0; i < F; ++i) mine[i] = i * BEAM_THREADS + tid < n ? found[i * BEAM_THREADS + tid] : 0ull;
                    if (tid == 0) n_found = 0;
                    __syncthreads();
                    const unsigned long long lo = (unsigned long long)ordered(bound + 0.0f) << 32;
#pragma unroll
                    for (int i = 0; i < F; ++i)
                        if (mine[i] >= lo) found[atomicAdd(&n_found, 1)] = mine[i];
                }
            } else {
                // too many reach the bound (ties, most often): the k-th largest of
                // (logit, token) by bisection over the whole piece, read once per round
                auto each = [&](auto f) {
                    for (int s = first; s <= step; ++s) {
                        const int e0 = here.token0 + s * BEAM_STEP * VEC;
                        load(cur, here, e0);
                        if constexpr (MASK) {
                            load_bits(bits, row, e0);
#pragma unroll
                            for (int u = 0; u < U; ++u) L::keep(cur[u], bits[u]);
                        }
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int j = 0; j < VEC; ++j)
                                f(logit_token(L::get(cur[u], j), e0 + (u * BEAM_THREADS + tid) * VEC + j));
                    }
                };
                unsigned long long lo = (unsigned long long)ordered(bound + 0.0f) << 32, hi = 0xFFFFFFFFFFFFFFFFull;
                while (lo < hi) {
                    const unsigned long long mid = lo + (hi - lo) / 2 + 1;
                    int c = 0;
                    each([&](unsigned long long v) { c += v >= mid; });
                    c = block_sum(c, scratch);
                    if (c >= a.k) lo = mid;
                    else hi = mid - 1;
                    if (c == a.k) break;
                }
                __syncthreads();
                if (tid == 0) n_found = 0;
                __syncthreads();
                each([&](unsigned long long v) {
                    if (v >= lo) found[atomicAdd(&n_found, 1)] = v;
                });
            }
            __syncthreads();
            const int n = n_found;
            unsigned long long *best = a.best + list * a.kpad;
            for (int i = tid; i < n; i += BEAM_THREADS) {
                const unsigned long long c = found[i];
                int rank = 0;
                for (int j = 0; j < n; ++j) rank += found[j] > c;
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
        row += row_ends;
        step = row_ends ? 0 : step + 1;
        token0 = ntoken0;
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = nxt[u];
        if constexpr (MASK) {
#pragma unroll
            for (int u = 0; u < U; ++u) bits[u] = nbits[u];
        }
    }

    // ---- this block's pieces are done: batch entries that are complete are joined
    __threadfence();
    const int row0 = (int)((long long)blockIdx.x * a.span / a.steps), row1 = (int)((end - 1) / a.steps);
    for (int b = row0 / a.W; b <= row1 / a.W; ++b) {
        __syncthreads();
        if (tid == 0) {
            const int done = min(row1, (b + 1) * a.W - 1) - max(row0, b * a.W) + 1;
            int total = 0;
            for (int w = 0; w < a.W; ++w) total += pieces_of(a, b * a.W + w);
            joins = atomicAdd(a.count + b, done) + done == total;
            if (joins) a.count[b] = 0;
            __threadfence();
        }
        __syncthreads();
        if (joins) beam_join(a, *reinterpret_cast<JoinSmem *>(smem), b);
    }
}

// ------------------------------------------------------------ host

// Steps of a row, of a stretch, and the most pieces of a row.  As many
// stretches as blocks fit on the GPU (those with a mask hold more registers).
constexpr long long BEAM_SMS = 152;
struct BeamSplit {
    int steps, span, pieces, stretches;
};
static BeamSplit beam_split(int rows, int V, int vec, bool mask)
{
    BeamSplit s;
    // (a row may begin inside its first vector)
    s.steps = ((V + vec - 1 + vec - 1) / vec + BEAM_STEP - 1) / BEAM_STEP;
    const long long total = (long long)rows * s.steps, blocks = BEAM_SMS * (mask ? 2 : 4);
    s.span = (int)((total + blocks - 1) / blocks);
    s.pieces = (s.steps + s.span - 1) / s.span + (s.steps % s.span != 0 || s.span == 0 ? 1 : 0);
    s.stretches = (int)((total + s.span - 1) / s.span);
    return s;
}

static size_t beam_lists(int B, int W, int V, int vec)
{
    const size_t p = beam_split(B * W, V, vec, false).pieces, m = beam_split(B * W, V, vec, true).pieces;
    return (size_t)B * W * (p > m ? p : m);
}

size_t beam_workspace_bytes(int B, int W, int V, int k)
{
    const size_t l4 = beam_lists(B, W, V, 4), l8 = beam_lists(B, W, V, 8);  // fp32, bf16
    return ((l4 > l8 ? l4 : l8) * (((size_t)k + 3) / 4 * 4 + 1) * 8 + 255) / 256 * 256;
}

template <typename E>
static cudaError_t run_beam(cudaStream_t st, const BeamArgs &a, int stretches)
{
    const dim3 grid((unsigned)stretches);
    return a.mask ? launch_k(beam_kernel<E, true>, grid, dim3(BEAM_THREADS), 0, st, a)
                  : launch_k(beam_kernel<E, false>, grid, dim3(BEAM_THREADS), 0, st, a);
}

cudaError_t launch_beam_select(const DeviceState &ds, cudaStream_t st, const BeamCall &c, void *workspace)
{
    const int vec = c.dtype == MX_F32 ? 4 : 8;
    const BeamSplit split = beam_split(c.B * c.W, c.V, vec, c.mask != nullptr);
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
    return c.dtype == MX_F32 ? run_beam<float>(st, a, split.stretches) : run_beam<uint16_t>(st, a, split.stretches);
}

}  // namespace mx
