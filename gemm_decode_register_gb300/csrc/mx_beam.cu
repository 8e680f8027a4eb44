// mx_beam.cu -- the beams' selection over the vocabulary: the k best
// continuations of each batch entry's beams, sm_103a.
//
//   key(r, v) = score[r] + x[r][v] - lse_r,  lse_r = log sum_v e^x[r][v],
// over the tokens v that row r's mask allows; the k largest of a batch
// entry's W rows (bound: HBM, one pass over the logits).
//
// Two launches.  beam_chunk_kernel: a block takes a chunk of one row, up to
// eight 16-byte vectors per thread, held in registers.  Within a row the
// order of the keys is that of the logits, so a chunk needs no more of its row
// than itself:
//   - the largest element of each vector (packed maxima) and thread; each warp
//     finds the r-th largest of its lanes' by r warp-wide maxima.  With r warps
//     times k at least k, the smallest of these is a bound that k elements of
//     the block reach, and not many more do;
//   - the vectors that reach it go to a queue in shared memory, a few threads
//     take their elements apart, and each one that reaches the bound counts
//     those before it: its rank;
//   - the sum of exponentials over the block's maximum.
// beam_join_kernel: a block takes a batch entry: the rows' sums, the same
// bound from the heads of the chunks' lists (in fp32, with what its rounding may
// be off on either side), and the ranks of those that reach it by keys in 64
// bits: near ties between beams are decided by bits that fp32 scores of -20
// do not have.  It is launched while the chunks run and waits for them.
// Where ties let more elements reach a bound than the shared memory holds,
// both kernels go slower ways to the same result (one that orders equal logits by their
// places).
#include <cfloat>
#include <cmath>

#include "../../include/mx.h"
#include "mx_common.cuh"
#include "mx_serve.h"

namespace mx {

constexpr int BEAM_THREADS = 256;
constexpr int BEAM_WARPS = BEAM_THREADS / 32;
constexpr int BEAM_QUEUE = 512;   // vectors that reach a chunk's bound
constexpr int BEAM_FOUND = 1024;  // elements that do (a chunk's, a batch entry's)

struct BeamArgs {
    const void *logits;
    long long row_stride;
    const float *scores;
    const uint32_t *mask;
    long long mask_stride;
    int B, W, V, k, eos, chunks;
    float *score, *next_score;
    int32_t *parent, *token, *next_parent, *next_token;
    float2 *sums;              // [rows][chunks] maximum and sum
    unsigned long long *best;  // [rows][chunks][kpad] (logit, token) in order, 0 past the last
    int kpad;                  // k rounded up to 4
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
__device__ __forceinline__ unsigned long long ordered64(double d)
{
    const long long b = __double_as_longlong(d);
    return (unsigned long long)b ^ ((unsigned long long)(b >> 63) | 0x8000000000000000ull);
}

constexpr uint32_t ORD_NEG_INF = 0x007FFFFFu;

// One element type's vectors, and (logit, place in the chunk) as one number:
// bf16 in 32 bits (a chunk has at most 2^16 places), fp32 in 64.
template <typename E>
struct Elem;
template <>
struct Elem<uint16_t> {
    static constexpr int VEC = 8;
    using Key = uint32_t;
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
        return ((j & 1) ? bf16_hi(w) : bf16_lo(w)) + 0.0f;
    }
    static __device__ __forceinline__ Key key(float f, int place)
    {
        return (ordered(f) & 0xFFFF0000u) | (0xFFFFu - (uint32_t)place);
    }
    static constexpr Key NONE = (ORD_NEG_INF & 0xFFFF0000u) | 0xFFFFu, LAST = 0xFFFFFFFFu;  // keys up to NONE are no candidates
    // (a negative bf16's ordered number ends in ones)
    static __device__ __forceinline__ uint32_t value(Key k) { return (k >> 31) ? k & 0xFFFF0000u : k | 0xFFFFu; }
    static __device__ __forceinline__ int place(Key k) { return (int)(0xFFFFu - (k & 0xFFFFu)); }
};
template <>
struct Elem<float> {
    static constexpr int VEC = 4;
    using Key = unsigned long long;
    static __device__ __forceinline__ float top(const uint4 &v)
    {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ void keep(uint4 &v, uint32_t bits)
    {
        uint32_t *w = &v.x;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (!(bits >> j & 1u)) w[j] = 0xFF800000u;
    }
    static __device__ __forceinline__ float get(const uint4 &v, int j)
    {
        return __uint_as_float(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w) + 0.0f;
    }
    static __device__ __forceinline__ Key key(float f, int place)
    {
        return ((Key)ordered(f) << 32) | (0xFFFFFFFFu - (uint32_t)place);
    }
    static constexpr Key NONE = ((Key)ORD_NEG_INF << 32) | 0xFFFFFFFFu, LAST = 0xFFFFFFFFFFFFFFFFull;
    static __device__ __forceinline__ uint32_t value(Key k) { return (uint32_t)(k >> 32); }
    static __device__ __forceinline__ int place(Key k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }
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

// ---- chunks

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

template <typename E, int U, bool MASK>
__global__ void __launch_bounds__(BEAM_THREADS, U == 8 && !MASK ? 4 : 3) beam_chunk_kernel(const __grid_constant__ BeamArgs a)
{
    using L = Elem<E>;
    using Key = typename L::Key;
    constexpr int VEC = L::VEC;
    __shared__ uint4 queue[BEAM_QUEUE];
    __shared__ uint16_t queue_at[BEAM_QUEUE];
    __shared__ Key found[BEAM_FOUND];
    __shared__ float warp_top[BEAM_WARPS], warp_sum[BEAM_WARPS];
    __shared__ uint32_t warp_bound[BEAM_WARPS];
    __shared__ int n_queue, n_found, scratch[BEAM_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int chunk = blockIdx.x, row = blockIdx.y;

    pdl_trigger();
    pdl_wait();
    const E *x = static_cast<const E *>(a.logits) + (size_t)row * a.row_stride;
    // vectors of the row counted from the 16-byte boundary at or before it;
    // one that the row only partly covers is read element by element
    const int lead = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(E));
    const int first = chunk * BEAM_THREADS * U;
    uint4 raw[U];
    auto load = [&] {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = (first + u * BEAM_THREADS + tid) * VEC - lead;
            if (e >= 0 && e + VEC <= a.V) raw[u] = __ldcs(reinterpret_cast<const uint4 *>(x + e));
            else raw[u] = edge_vector(x + e, e < 0 ? -e : 0, min(VEC, a.V - e));
        }
        if constexpr (MASK) {
            const uint32_t *m = a.mask + (size_t)row * a.mask_stride;
            const int words = (a.V + 31) >> 5;
            uint32_t bits[U];
#pragma unroll
            for (int u = 0; u < U; ++u) bits[u] = mask_bits<VEC>(m, (first + u * BEAM_THREADS + tid) * VEC - lead, words);
#pragma unroll
            for (int u = 0; u < U; ++u) L::keep(raw[u], bits[u]);
        }
    };
    load();
    if (tid == 0) n_queue = n_found = 0;

    // largest elements; the warp's part of the bound: r of its lanes reach it,
    // and the warps that have elements make r times their number k or more
    float top[U], m = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        top[u] = L::top(raw[u]);
        m = fmaxf(m, top[u]);
    }
    {
        const int vecs = min(BEAM_THREADS, (lead + a.V + VEC - 1) / VEC - first);
        const int warps = max(1, (vecs + 31) / 32), r = (a.k + warps - 1) / warps;
        const uint32_t mine = ordered(m + 0.0f);
        const float wm = unordered(__reduce_max_sync(0xFFFFFFFFu, mine));
        uint32_t bound = r > 32 ? 0u : warp_nth(mine, r, [] { return 0u; });
        if (warp >= warps) bound = 0xFFFFFFFFu;  // (no elements, no say)
        if (lane == 0) {
            warp_top[warp] = wm;
            warp_bound[warp] = bound;
        }
    }
    __syncthreads();
    float all = warp_top[0];
    uint32_t least = warp_bound[0];
#pragma unroll
    for (int w = 1; w < BEAM_WARPS; ++w) {
        all = fmaxf(all, warp_top[w]);
        least = min(least, warp_bound[w]);
    }
    const float bound = least > ORD_NEG_INF ? unordered(least) : -FLT_MAX;  // (-inf is no candidate)

    // the vectors that reach the bound; the sum over the block's maximum
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (top[u] >= bound) {
            const int i = atomicAdd(&n_queue, 1);
            if (i < BEAM_QUEUE) {
                queue[i] = raw[u];
                queue_at[i] = (uint16_t)(u * BEAM_THREADS + tid);
            }
        }
    const float over = all > -INFINITY ? all : 0.0f;
    // (x - maximum before the factor: its rounding stays relative to the difference)
    const float2 shift = make_float2(-over, -over), log2e = make_float2(1.4426950408889634f, 1.4426950408889634f);
    float2 sum2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
            const float2 d = mul2(add2(make_float2(L::get(raw[u], j), L::get(raw[u], j + 1)), shift), log2e);
            sum2[(j / 2) & 1] = add2(sum2[(j / 2) & 1], make_float2(exp2_fast(d.x), exp2_fast(d.y)));
        }
    float sum = (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) warp_sum[warp] = sum;
    __syncthreads();
    const size_t list = (size_t)row * a.chunks + chunk;
    if (tid == 0) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < BEAM_WARPS; ++w) s += warp_sum[w];
        a.sums[list] = make_float2(all, s);
    }
    const int vectors = n_queue;
    if (vectors <= BEAM_QUEUE)
        for (int i = tid; i < vectors; i += BEAM_THREADS) {
            const uint4 v = queue[i];
            const int place = (int)queue_at[i] * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float f = L::get(v, j);
                if (f >= bound) {
                    const int at = atomicAdd(&n_found, 1);
                    if (at < BEAM_FOUND) found[at] = L::key(f + 0.0f, place + j);
                }
            }
        }
    __syncthreads();
    int n = n_found;
    if (vectors > BEAM_QUEUE || n > BEAM_FOUND) {
        // too many reach it (ties, most often): the k-th largest key, places
        // and all, by bisection over every element (loaded again, so that the
        // registers are free till here)
        load();
        Key lo = L::NONE + 1, hi = L::LAST;
        while (lo < hi) {
            const Key mid = lo + (hi - lo) / 2 + 1;
            int c = 0;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < VEC; ++j) c += L::key(L::get(raw[u], j) + 0.0f, (u * BEAM_THREADS + tid) * VEC + j) >= mid;
            c = block_sum(c, scratch);
            if (c >= a.k) lo = mid;
            else hi = mid - 1;
            if (c == a.k) break;
        }
        if (tid == 0) n_found = 0;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const Key c = L::key(L::get(raw[u], j) + 0.0f, (u * BEAM_THREADS + tid) * VEC + j);
                if (c >= lo) found[atomicAdd(&n_found, 1)] = c;
            }
        __syncthreads();
        n = n_found;
    }
    unsigned long long *best = a.best + list * a.kpad;
    for (int i = tid; i < n; i += BEAM_THREADS) {
        const Key c = found[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += found[j] > c;
        if (rank < a.k) {
            const int v = first * VEC + L::place(c) - lead;
            best[rank] = ((unsigned long long)L::value(c) << 32) | (0xFFFFFFFFu - (uint32_t)v);
        }
    }
    for (int i = min(n, a.k) + tid; i < a.kpad; i += BEAM_THREADS) best[i] = 0ull;
}

// ---- join of one batch entry's chunks

// The total order: key (64 bits), then beam, then (logit, token).
__device__ __forceinline__ bool before(unsigned long long ka, int ra, unsigned long long la, unsigned long long kb, int rb,
                                       unsigned long long lb)
{
    return ka != kb ? ka > kb : ra != rb ? ra < rb : la > lb;
}

__device__ __forceinline__ double key_value(unsigned long long k)
{
    return __longlong_as_double((long long)(k ^ ((k >> 63) ? 0x8000000000000000ull : 0xFFFFFFFFFFFFFFFFull)));
}

__global__ void __launch_bounds__(BEAM_THREADS) beam_join_kernel(const __grid_constant__ BeamArgs a)
{
    __shared__ double score[BEAM_MAX_W], lse[BEAM_MAX_W];  // lse NaN: the beam has no candidates
    __shared__ float2 part[BEAM_MAX_W];
    __shared__ unsigned long long key[BEAM_FOUND], lt[BEAM_FOUND];
    __shared__ int beam[BEAM_FOUND];
    __shared__ uint32_t warp_bound[BEAM_WARPS];
    __shared__ float out_score[BEAM_MAX_K];
    __shared__ int out_parent[BEAM_MAX_K], out_token[BEAM_MAX_K], n_found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x, b = blockIdx.x;
    const int lists = a.W * a.chunks;
    pdl_trigger();
    pdl_wait();
    const unsigned long long *best = a.best + (size_t)b * lists * a.kpad;

    // heads of the thread's (first) list.  Neighbouring lists go to different
    // warps, so that each warp sees every beam.
    const int warps = min(BEAM_WARPS, (lists + 31) / 32);
    const int mine = lane * warps + warp;
    ulonglong2 head[2] = {make_ulonglong2(0ull, 0ull), make_ulonglong2(0ull, 0ull)};
    if (warp < warps && mine < lists) {
        const ulonglong2 *p = reinterpret_cast<const ulonglong2 *>(best + (size_t)mine * a.kpad);
        head[0] = __ldcg(p);
        head[1] = __ldcg(p + 1);
    }
    // the rows' sums
    for (int w = warp; w < a.W; w += BEAM_WARPS) {
        const float2 *p = a.sums + ((size_t)b * a.W + w) * a.chunks;
        float m = -INFINITY, t = 0.0f;
        for (int c = lane; c < a.chunks; c += 32) {
            const float2 v = __ldcg(p + c);
            const float nm = fmaxf(m, v.x);
            // (equal maxima, infinite ones too: no scaling; NaN sums stay)
            t = (m == nm ? t : t * expf(m - nm)) + (v.x == nm ? v.y : v.y * expf(v.x - nm));
            m = nm;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float om = __shfl_xor_sync(0xFFFFFFFFu, m, o), ot = __shfl_xor_sync(0xFFFFFFFFu, t, o);
            const float nm = fmaxf(m, om);
            t = (m == nm ? t : t * expf(m - nm)) + (om == nm ? ot : ot * expf(om - nm));
            m = nm;
        }
        if (lane == 0) part[w] = make_float2(m, t);
    }
    if (tid == 0) n_found = 0;
    __syncthreads();
    if (tid < a.W) {
        const float c = __ldcg(a.scores + (size_t)b * a.W + tid);
        const float2 p = part[tid];
        // NaN sums: a NaN or +inf among the logits; nothing allowed: no maximum
        const bool ok = p.y > 0.0f && fabsf(p.x) < INFINITY && fabsf(c) < INFINITY;
        score[tid] = (double)c;
        lse[tid] = ok ? (double)p.x + log((double)p.y) : (double)NAN;
    }
    __syncthreads();

    // A candidate's key lies within off of fp32 arithmetic: below, above.
    auto about = [&](int row, unsigned long long l, float &off) {
        const float c = (float)score[row], s = (float)lse[row], x = unordered((uint32_t)(l >> 32));
        off = (fabsf(c) + fabsf(x) + fabsf(s)) * 2.3841858e-7f;  // three roundings of a quarter of that, and one spare
        return c + (x - s);
    };
    auto exact = [&](int row, unsigned long long l) {
        return ordered64(score[row] + ((double)unordered((uint32_t)(l >> 32)) - lse[row]));
    };
    // A bound that k candidates reach, from the first four of a list per lane.
    uint32_t bound = 0u;
    if (warp < warps) {
        uint32_t low[4] = {0u, 0u, 0u, 0u};
        const int row = mine / a.chunks;
        if (mine < lists && lse[row] == lse[row]) {
            const unsigned long long h[4] = {head[0].x, head[0].y, head[1].x, head[1].y};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (h[i] != 0ull) {
                    float off;
                    const float f = about(row, h[i], off);
                    low[i] = ordered((f - off) + 0.0f);
                }
        }
        // (rounded down in fp32, the heads still descend)
        const int r = (a.k + warps - 1) / warps;
        bound = warp_nth(low[0], r, [&] {
            low[0] = low[1];
            low[1] = low[2];
            low[2] = low[3];
            low[3] = 0u;
            return low[0];
        });
        if (lane == 0) warp_bound[warp] = bound;
    }
    __syncthreads();
    bound = warp_bound[0];
    for (int w = 1; w < warps; ++w) bound = min(bound, warp_bound[w]);
    const float least = bound == 0u ? -INFINITY : unordered(bound);

    // what may reach it (its key, then)
    for (int l = mine; warp < warps && l < lists; l += 32 * warps) {
        const int row = l / a.chunks;
        if (!(lse[row] == lse[row])) continue;
        bool more = true;
        for (int i = 0; more && i < a.kpad; i += 4) {
            const ulonglong2 *p = reinterpret_cast<const ulonglong2 *>(best + (size_t)l * a.kpad + i);
            const ulonglong2 v0 = l == mine && i == 0 ? head[0] : __ldcg(p), v1 = l == mine && i == 0 ? head[1] : __ldcg(p + 1);
            const unsigned long long h[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float off = 0.0f;
                const float f = h[j] != 0ull ? about(row, h[j], off) : 0.0f;
                more = more && h[j] != 0ull && f + off >= least;
                if (!more) break;
                const int at = atomicAdd(&n_found, 1);
                if (at < BEAM_FOUND) {
                    key[at] = exact(row, h[j]);
                    lt[at] = h[j];
                    beam[at] = row;
                }
            }
        }
    }
    __syncthreads();
    const int n = n_found;
    if (n <= BEAM_FOUND) {
        for (int i = tid; i < n; i += BEAM_THREADS) {
            const unsigned long long ki = key[i], li = lt[i];
            const int ri = beam[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) {
                const unsigned long long kj = key[j];
                rank += kj > ki || (kj == ki && before(kj, beam[j], lt[j], ki, ri, li));
            }
            if (rank < a.k) {
                out_score[rank] = (float)key_value(ki);
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
                const int row = l / a.chunks;
                if (!(lse[row] == lse[row])) continue;
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
            beam[tid] = mr;
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
                out_score[i] = (float)key_value(mk);
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

// ------------------------------------------------------------ host

static int beam_chunks(int V, int vec, int unroll)
{
    // a row may begin inside its first vector
    return (V + vec - 1 + BEAM_THREADS * unroll * vec - 1) / (BEAM_THREADS * unroll * vec);
}

// Vectors per thread: eight, as long as the chunks still make two blocks per
// SM; else two, so that a few rows reach more of the GPU.
constexpr int BEAM_FEW = 304;
static int beam_unroll(int rows, int V, int vec) { return (long long)rows * beam_chunks(V, vec, 8) >= BEAM_FEW ? 8 : 2; }

static size_t beam_lists(int B, int W, int V, int vec) { return (size_t)B * W * beam_chunks(V, vec, beam_unroll(B * W, V, vec)); }

size_t beam_workspace_bytes(int B, int W, int V, int k)
{
    const size_t l4 = beam_lists(B, W, V, 4), l8 = beam_lists(B, W, V, 8);  // fp32, bf16
    return ((l4 > l8 ? l4 : l8) * (((size_t)k + 3) / 4 * 4 + 2) * 8 + 255) / 256 * 256;
}

template <typename E, int U>
static cudaError_t run_beam(cudaStream_t st, const BeamArgs &a)
{
    const dim3 grid(a.chunks, a.B * a.W);
    const cudaError_t e = a.mask ? launch_k(beam_chunk_kernel<E, U, true>, grid, dim3(BEAM_THREADS), 0, st, a)
                                 : launch_k(beam_chunk_kernel<E, U, false>, grid, dim3(BEAM_THREADS), 0, st, a);
    return e != cudaSuccess ? e : launch_k(beam_join_kernel, dim3(a.B), dim3(BEAM_THREADS), 0, st, a);
}

cudaError_t launch_beam_select(const DeviceState &, cudaStream_t st, const BeamCall &c, void *workspace)
{
    const int vec = c.dtype == MX_F32 ? 4 : 8;
    const int unroll = beam_unroll(c.B * c.W, c.V, vec);
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
    a.chunks = beam_chunks(c.V, vec, unroll);
    a.score = c.score;
    a.parent = c.parent;
    a.token = c.token;
    a.next_score = c.next_score;
    a.next_parent = c.next_parent;
    a.next_token = c.next_token;
    const size_t lists = (size_t)c.B * c.W * a.chunks;
    a.kpad = (c.k + 3) / 4 * 4;
    a.best = static_cast<unsigned long long *>(workspace);
    a.sums = reinterpret_cast<float2 *>(a.best + lists * a.kpad);
    if (c.dtype == MX_F32) return unroll == 8 ? run_beam<float, 8>(st, a) : run_beam<float, 2>(st, a);
    return unroll == 8 ? run_beam<uint16_t, 8>(st, a) : run_beam<uint16_t, 2>(st, a);
}

}  // namespace mx
