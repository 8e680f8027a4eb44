// mx_beam.cu -- the beams' selection over the vocabulary: the k best
// continuations of each batch entry's beams, sm_103a.
//
//   key(r, v) = score[r] + x[r][v] - lse_r,  lse_r = log sum_v e^x[r][v],
// over the tokens v that row r's mask allows; the k largest of a batch
// entry's W rows (bound: HBM, one pass over the logits).
//
// One launch.  A block takes a chunk of one row, up to BEAM_UNROLL 16-byte
// vectors per thread, held in registers: the running maximum and sum of
// exponentials (fp32) and the chunk's k largest logits.  Within a row the
// order of the keys is that of the logits, so a chunk needs no more of its
// row than itself:
//   - each thread's largest (logit, token) as one whole number; a bisection
//     over the block's 256 of them finds a bound that k to 2k of them reach;
//   - only those threads look at their elements again and put the ones that
//     reach the bound into shared memory, where each counts the ones before
//     it: its rank.
// The last block of a batch entry to finish (a counter) joins: the rows'
// sums, then keys in 64 bits (near ties between beams are decided by bits
// that fp32 scores of -20 do not have), and the same selection over the
// chunks' lists.  Nothing depends on the order in which blocks finish.
#include <cmath>

#include "../../include/mx.h"
#include "mx_common.cuh"
#include "mx_serve.h"

namespace mx {

constexpr int BEAM_THREADS = 256;
constexpr int BEAM_JOIN_CAP = 1024;  // candidates ranked at once in the join

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
    unsigned long long *best;  // [rows][chunks][k] (logit, token), 0 past the last
    int *count;                // [B] blocks that finished, zero between calls
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
    static __device__ __forceinline__ float get(const uint4 &v, int j)
    {
        const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
        return ((j & 1) ? bf16_hi(w) : bf16_lo(w)) + 0.0f;
    }
    static __device__ __forceinline__ uint4 edge(const uint16_t *p, int lo, int hi)
    {
        uint32_t w[4] = {0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};  // -inf
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j >= lo && j < hi) {
                const uint32_t b = p[j];
                w[j / 2] = (j & 1) ? (w[j / 2] & 0xFFFFu) | (b << 16) : (w[j / 2] & 0xFFFF0000u) | b;
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ Key key(float f, int place)
    {
        return (ordered(f) & 0xFFFF0000u) | (0xFFFFu - (uint32_t)place);
    }
    static constexpr Key NONE = (ORD_NEG_INF & 0xFFFF0000u) | 0xFFFFu;  // keys up to this are no candidates
    // (a negative bf16's ordered number ends in ones)
    static __device__ __forceinline__ uint32_t value(Key k) { return (k >> 31) ? k & 0xFFFF0000u : k | 0xFFFFu; }
    static __device__ __forceinline__ int place(Key k) { return (int)(0xFFFFu - (k & 0xFFFFu)); }
};
template <>
struct Elem<float> {
    static constexpr int VEC = 4;
    using Key = unsigned long long;
    static __device__ __forceinline__ float get(const uint4 &v, int j)
    {
        return __uint_as_float(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w) + 0.0f;
    }
    static __device__ __forceinline__ uint4 edge(const float *p, int lo, int hi)
    {
        uint32_t w[4] = {0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j >= lo && j < hi) w[j] = __float_as_uint(p[j]);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ Key key(float f, int place)
    {
        return ((Key)ordered(f) << 32) | (0xFFFFFFFFu - (uint32_t)place);
    }
    static constexpr Key NONE = ((Key)ORD_NEG_INF << 32) | 0xFFFFFFFFu;
    static __device__ __forceinline__ uint32_t value(Key k) { return (uint32_t)(k >> 32); }
    static __device__ __forceinline__ int place(Key k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }
};

// Elements of the set that reach the bound at most: the threads that do times
// what a thread holds.
template <typename E, int U>
__host__ __device__ constexpr int beam_cap(int k)
{
    return (2 * k < BEAM_THREADS ? 2 * k : BEAM_THREADS) * U * Elem<E>::VEC;
}

// A bound in [lo, hi] that at least n and, where that can be, at most `most`
// of the block's keys reach; lo if fewer than n reach that.  No key is above hi.
template <typename Key>
__device__ __forceinline__ Key block_bound(Key mine, Key lo, Key hi, int n, int most)
{
    if (__syncthreads_count(mine >= lo) <= most) return lo;
    while (lo < hi) {
        const Key mid = lo + (hi - lo) / 2 + 1;
        const int c = __syncthreads_count(mine >= mid);
        if (c >= n) {
            lo = mid;
            if (c <= most) break;
        } else {
            hi = mid - 1;
        }
    }
    return lo;
}

// ---- join of one batch entry's chunks

// The join's total order: key (64 bits), then beam, then (logit, token).
__device__ __forceinline__ bool before(unsigned long long ka, int ra, unsigned long long la, unsigned long long kb, int rb,
                                       unsigned long long lb)
{
    return ka != kb ? ka > kb : ra != rb ? ra < rb : la > lb;
}

// Shared memory of the join, laid over the selection's.
struct JoinSmem {
    double score[64], lse[64];  // lse NaN: the beam has no candidates
    unsigned long long key[BEAM_JOIN_CAP], lt[BEAM_JOIN_CAP];
    int row[BEAM_JOIN_CAP];
    float out_score[128];
    int out_parent[128], out_token[128];
    int n;
};

// A candidate's key as an ordered number; 0: not one.
__device__ __forceinline__ unsigned long long cand_key(const JoinSmem &s, int row, unsigned long long lt)
{
    if (lt == 0ull || !(s.lse[row] == s.lse[row])) return 0ull;
    return ordered64(s.score[row] + ((double)unordered((uint32_t)(lt >> 32)) - s.lse[row]));
}

__device__ __forceinline__ double key_value(unsigned long long k)
{
    return __longlong_as_double((long long)(k ^ ((k >> 63) ? 0x8000000000000000ull : 0xFFFFFFFFFFFFFFFFull)));
}

__device__ void beam_join(const BeamArgs &a, JoinSmem &s, int b)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lists = a.W * a.chunks;
    const unsigned long long *best = a.best + (size_t)b * lists * a.k;
    // the rows' sums; a row without log-probabilities is marked NaN
    for (int w = warp; w < a.W; w += BEAM_THREADS / 32) {
        const float2 *p = a.sums + ((size_t)b * a.W + w) * a.chunks;
        float m = -INFINITY;
        bool bad = false;
        for (int c = lane; c < a.chunks; c += 32) {
            const float2 v = __ldcg(p + c);
            bad |= !(v.y < INFINITY);  // NaN, or a NaN or infinity among the logits
            m = fmaxf(m, v.x);
        }
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        bad = __any_sync(0xFFFFFFFFu, bad) || !(m > -INFINITY && m < INFINITY);
        double t = 0.0;
        if (!bad)
            for (int c = lane; c < a.chunks; c += 32) {
                const float2 v = __ldcg(p + c);
                if (v.x > -INFINITY) t += (double)v.y * exp((double)v.x - (double)m);
            }
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        const float c = __ldcg(a.scores + (size_t)b * a.W + w);
        if (lane == 0) {
            s.score[w] = (double)c;
            s.lse[w] = bad || !(fabsf(c) < INFINITY) ? (double)NAN : (double)m + log(t);
        }
    }
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    // A bound that k candidates reach: where q lists' elements number d reach
    // it, q (d + 1) do.  Beams alike call for small d, one beam ahead of the
    // others for large: the largest bound of several d counts (upper halves
    // of the keys are enough for it).
    uint32_t bound = 1u;
    if (lists <= BEAM_THREADS) {
        const int l = threadIdx.x, row = l / a.chunks;
        for (int d = (a.k + lists - 1) / lists - 1; d < a.k; d = 4 * d + 3) {
            const uint32_t mine = l < lists ? (uint32_t)(cand_key(s, row, __ldcg(best + (size_t)l * a.k + d)) >> 32) : 0u;
            const int q = (a.k + d) / (d + 1);
            const uint32_t c = block_bound(mine, 1u, 0xFFFFFFFEu, q, q);
            bound = c > bound ? c : bound;
        }
    } else {
        // more lists than threads: each thread's largest stands for its lists
        uint32_t mine = 0u;
        for (int l = threadIdx.x; l < lists; l += BEAM_THREADS) {
            const uint32_t c = (uint32_t)(cand_key(s, l / a.chunks, __ldcg(best + (size_t)l * a.k)) >> 32);
            mine = c > mine ? c : mine;
        }
        bound = block_bound(mine, 1u, 0xFFFFFFFEu, a.k, a.k);
    }
    for (int l = threadIdx.x; l < lists; l += BEAM_THREADS) {
        const int row = l / a.chunks;
        for (int i = 0; i < a.k; ++i) {
            const unsigned long long lt = __ldcg(best + (size_t)l * a.k + i);
            const unsigned long long c = cand_key(s, row, lt);
            if ((uint32_t)(c >> 32) < bound) break;
            const int at = atomicAdd(&s.n, 1);
            if (at < BEAM_JOIN_CAP) {
                s.key[at] = c;
                s.lt[at] = lt;
                s.row[at] = row;
            }
        }
    }
    __syncthreads();
    const int n = s.n;
    if (n <= BEAM_JOIN_CAP) {
        for (int i = threadIdx.x; i < n; i += BEAM_THREADS) {
            const unsigned long long ki = s.key[i], li = s.lt[i];
            const int ri = s.row[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += before(s.key[j], s.row[j], s.lt[j], ki, ri, li);
            if (rank < a.k) {
                s.out_score[rank] = (float)key_value(ki);
                s.out_parent[rank] = b * a.W + ri;
                s.out_token[rank] = (int)(0xFFFFFFFFu - (uint32_t)li);
            }
        }
        for (int i = n + threadIdx.x; i < a.k; i += BEAM_THREADS) {
            s.out_score[i] = -INFINITY;
            s.out_parent[i] = -1;
            s.out_token[i] = 0;
        }
    } else {
        // more candidates reach the bound than fit (long ties between beams):
        // one after the other, each the best of what follows the last
        unsigned long long pk = 0xFFFFFFFFFFFFFFFFull, pl = 0;
        int pr = -1;
        for (int i = 0; i < a.k; ++i) {
            unsigned long long mk = 0ull, ml = 0ull;
            int mr = 0x7FFFFFFF;
            for (int l = threadIdx.x; l < lists; l += BEAM_THREADS) {
                const int row = l / a.chunks;
                for (int e = 0; e < a.k; ++e) {
                    const unsigned long long lt = __ldcg(best + (size_t)l * a.k + e);
                    const unsigned long long c = cand_key(s, row, lt);
                    if ((uint32_t)(c >> 32) < bound) break;
                    if ((pr < 0 || before(pk, pr, pl, c, row, lt)) && before(c, row, lt, mk, mr, ml)) {
                        mk = c;
                        mr = row;
                        ml = lt;
                    }
                }
            }
            __syncthreads();
            s.key[threadIdx.x] = mk;
            s.lt[threadIdx.x] = ml;
            s.row[threadIdx.x] = mr;
            __syncthreads();
            for (int j = 0; j < BEAM_THREADS; ++j)
                if (before(s.key[j], s.row[j], s.lt[j], mk, mr, ml)) {
                    mk = s.key[j];
                    mr = s.row[j];
                    ml = s.lt[j];
                }
            pk = mk;
            pr = mr;
            pl = ml;
            if (threadIdx.x == 0) {
                s.out_score[i] = (float)key_value(mk);
                s.out_parent[i] = b * a.W + mr;
                s.out_token[i] = (int)(0xFFFFFFFFu - (uint32_t)ml);
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.k; i += BEAM_THREADS) {
        const size_t at = (size_t)b * a.k + i;
        a.score[at] = s.out_score[i];
        a.parent[at] = s.out_parent[i];
        a.token[at] = s.out_token[i];
    }
    // the first W that do not end go on
    if (warp == 0 && a.next_token != nullptr) {
        int at = 0;
        for (int i0 = 0; i0 < a.k && at < a.W; i0 += 32) {
            const int i = i0 + lane;
            const bool on = i < a.k && s.out_parent[i] >= 0 && s.out_token[i] != a.eos;
            const unsigned m = __ballot_sync(0xFFFFFFFFu, on);
            const int o = at + __popc(m & ((1u << lane) - 1u));
            if (on && o < a.W) {
                const size_t q = (size_t)b * a.W + o;
                a.next_score[q] = s.out_score[i];
                a.next_parent[q] = s.out_parent[i];
                a.next_token[q] = s.out_token[i];
            }
            at += __popc(m);
        }
        for (int o = at + lane; o < a.W; o += 32) {
            const size_t q = (size_t)b * a.W + o;
            a.next_score[q] = -INFINITY;
            a.next_parent[q] = -1;
            a.next_token[q] = 0;
        }
    }
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
__global__ void __launch_bounds__(BEAM_THREADS) beam_kernel(BeamArgs a)
{
    using L = Elem<E>;
    using Key = typename L::Key;
    constexpr int VEC = L::VEC;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 warp_sum[BEAM_THREADS / 32];
    __shared__ Key warp_top[BEAM_THREADS / 32], warp_low[BEAM_THREADS / 32];
    __shared__ int n_found, last;
    Key *found = reinterpret_cast<Key *>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunk = blockIdx.x, row = blockIdx.y, b = row / a.W;

    pdl_trigger();
    pdl_wait();
    const E *x = static_cast<const E *>(a.logits) + (size_t)row * a.row_stride;
    // vectors of the row counted from the 16-byte boundary at or before it;
    // one that the row only partly covers is read element by element
    const int lead = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(E));
    const int first = chunk * BEAM_THREADS * U;
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int e = (first + u * BEAM_THREADS + (int)threadIdx.x) * VEC - lead;
        if (e >= 0 && e + VEC <= a.V) raw[u] = __ldcs(reinterpret_cast<const uint4 *>(x + e));
        else raw[u] = L::edge(x + e, e < 0 ? -e : 0, min(VEC, a.V - e));
    }
    uint32_t allow[U];
    if constexpr (MASK) {
        const uint32_t *m = a.mask + (size_t)row * a.mask_stride;
        const int words = (a.V + 31) >> 5;
#pragma unroll
        for (int u = 0; u < U; ++u)
            allow[u] = mask_bits<VEC>(m, (first + u * BEAM_THREADS + (int)threadIdx.x) * VEC - lead, words);
    }
    if (threadIdx.x == 0) n_found = 0;

    // the thread's largest element, then its sum over that
    auto at = [&](int u, int j) {
        const float f = L::get(raw[u], j);
        if constexpr (MASK) return (allow[u] >> j) & 1u ? f : -INFINITY;
        return f;
    };
    float m = -INFINITY;
    int where = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float f = at(u, j);
            if (f > m) {
                m = f;
                where = u * BEAM_THREADS * VEC + j;
            }
        }
    const int mine0 = (int)threadIdx.x * VEC;  // place of the thread's element (0, 0)
    const Key mine = L::key(m, mine0 + where);
    const float mm = m > -INFINITY ? m : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum += __expf(at(u, j) - mm);

    // the block's: maximum and sum, largest key
    {
        float wm = m, ws = sum;
        Key wk = mine, wl = mine;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float om = __shfl_xor_sync(0xFFFFFFFFu, wm, o), os = __shfl_xor_sync(0xFFFFFFFFu, ws, o);
            const Key ok = __shfl_xor_sync(0xFFFFFFFFu, wk, o), ol = __shfl_xor_sync(0xFFFFFFFFu, wl, o);
            const float nm = fmaxf(wm, om);
            // (equal maxima, infinite ones too: no scaling)
            ws = (wm == nm ? ws : ws * __expf(wm - nm)) + (om == nm ? os : os * __expf(om - nm));
            wm = nm;
            wk = ok > wk ? ok : wk;
            wl = ol < wl ? ol : wl;
        }
        if (lane == 0) {
            warp_sum[warp] = make_float2(wm, ws);
            warp_top[warp] = wk;
            warp_low[warp] = wl;
        }
    }
    __syncthreads();
    Key top = warp_top[0], low = warp_low[0];
#pragma unroll
    for (int w = 1; w < BEAM_THREADS / 32; ++w) {
        top = warp_top[w] > top ? warp_top[w] : top;
        low = warp_low[w] < low ? warp_low[w] : low;
    }
    if (low <= L::NONE) low = L::NONE + 1;  // (a thread without candidates)
    if (top < low) top = low;
    const size_t list = (size_t)row * a.chunks + chunk;
    if (threadIdx.x == 0) {
        float bm = warp_sum[0].x, bs = warp_sum[0].y;
        for (int w = 1; w < BEAM_THREADS / 32; ++w) {
            const float om = warp_sum[w].x, os = warp_sum[w].y, nm = fmaxf(bm, om);
            bs = (bm == nm ? bs : bs * __expf(bm - nm)) + (om == nm ? os : os * __expf(om - nm));
            bm = nm;
        }
        a.sums[list] = make_float2(bm, bs);
    }
    const Key bound = block_bound(mine, low, top, a.k, 2 * a.k);
    if (mine >= bound) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const Key c = L::key(at(u, j), mine0 + u * BEAM_THREADS * VEC + j);
                if (c >= bound) found[atomicAdd(&n_found, 1)] = c;
            }
    }
    __syncthreads();
    const int n = n_found;
    unsigned long long *best = a.best + list * a.k;
    for (int i = threadIdx.x; i < n; i += BEAM_THREADS) {
        const Key c = found[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += found[j] > c;
        if (rank < a.k) {
            const int v = first * VEC + L::place(c) - lead;
            best[rank] = ((unsigned long long)L::value(c) << 32) | (0xFFFFFFFFu - (uint32_t)v);
        }
    }
    for (int i = n + threadIdx.x; i < a.k; i += BEAM_THREADS) best[i] = 0ull;

    // the last block of the batch entry joins
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int total = a.W * a.chunks;
        last = atomicAdd(a.count + b, 1) == total - 1;
        if (last) a.count[b] = 0;
        __threadfence();
    }
    __syncthreads();
    if (last) beam_join(a, *reinterpret_cast<JoinSmem *>(smem), b);
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
    return ((l4 > l8 ? l4 : l8) * ((size_t)k + 1) * 8 + 255) / 256 * 256;
}

template <typename E, int U>
static cudaError_t run_beam(cudaStream_t st, const BeamArgs &a)
{
    const int cap = beam_cap<E, U>(a.k) * (int)sizeof(typename Elem<E>::Key);
    const int smem = cap > (int)sizeof(JoinSmem) ? cap : (int)sizeof(JoinSmem);
    const dim3 grid(a.chunks, a.B * a.W);
    auto go = [&](auto kernel) {
        if (smem > 40 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        return launch_k(kernel, grid, dim3(BEAM_THREADS), smem, st, a);
    };
    return a.mask ? go(beam_kernel<E, U, true>) : go(beam_kernel<E, U, false>);
}

cudaError_t launch_beam_select(const DeviceState &ds, cudaStream_t st, const BeamCall &c, void *workspace)
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
    a.sums = static_cast<float2 *>(workspace);
    a.best = static_cast<unsigned long long *>(workspace) + lists;
    a.count = ds.ws_count;
    if (c.dtype == MX_F32) return unroll == 8 ? run_beam<float, 8>(st, a) : run_beam<float, 2>(st, a);
    return unroll == 8 ? run_beam<uint16_t, 8>(st, a) : run_beam<uint16_t, 2>(st, a);
}

}  // namespace mx
