// mx_rope.cu -- rotary positions, and the append of new keys and values to
// the paged cache with the rotation on the way.
//
// Rotation of a pair (a, b) of a head by the angle p f_i of its token's
// position: (a c - b s, b c + a s).  The cosines and sines come from a table
// (fp32, rounded once from fp64): at position 131072 an angle formed in fp32
// is off by up to 2^-7, as much as a bf16 result's own rounding.  The inverse
// (s -> -s) is the transpose, i.e. the gradient.
//
// Both kernels move each element once and are bound by HBM for prompts, by
// the launch and the chain of dependent loads (sequence, length, page, table
// row) for single tokens: 4 tokens x 72 heads x 128 turn in 2.4 us, and are
// appended in 2.4 us.
#include "mx_attn.cuh"

namespace mx {

// ------------------------------------------------------------ table

__global__ void rope_table_kernel(const double *__restrict__ inv_freq, double factor, float2 *__restrict__ table,
                                  long long pos0, long long n, int half)
{
    pdl_trigger();
    pdl_wait();
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n * half;
         i += (long long)gridDim.x * blockDim.x) {
        const long long p = i / half;
        double s, c;
        sincos((double)(pos0 + p) * inv_freq[i - p * half], &s, &c);
        table[i] = make_float2((float)(c * factor), (float)(s * factor));
    }
}

cudaError_t launch_rope_table(const DeviceState &ds, cudaStream_t st, const double *inv_freq, double factor,
                              float *table, int64_t pos0, int n, int half)
{
    const long long blocks = ((long long)n * half + 255) / 256, cap = (long long)ds.num_sms * 8;
    return launch_k(rope_table_kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, st, inv_freq,
                    factor, reinterpret_cast<float2 *>(table), (long long)pos0, (long long)n, half);
}

// ------------------------------------------------------------ vectors

// N elements of the type per 16-byte access; Raw holds them as they lie (half
// the registers of their fp32 values for bf16) until they are used.
template <typename T>
struct Vec;

template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4 &r, float (&v)[N])
    {
        v[0] = __uint_as_float(r.x);
        v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z);
        v[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[N])
    {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    static __device__ __forceinline__ float one(const float *p) { return *p; }
    static __device__ __forceinline__ void set_one(float *p, float v) { *p = v; }
};

template <>
struct Vec<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4 &r, float (&v)[N])
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[N])
    {
        return make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                          f32x2_to_bf16x2(v[6], v[7]));
    }
    static __device__ __forceinline__ float one(const uint16_t *p) { return bf16_to_f32(*p); }
    static __device__ __forceinline__ void set_one(uint16_t *p, float v)
    {
        *p = (uint16_t)(f32x2_to_bf16x2(v, 0.0f) & 0xFFFFu);
    }
};

// One pair; every product and sum rounded by itself.
__device__ __forceinline__ void turn(float &a, float &b, float c, float s)
{
    const float ra = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = ra;
}

// ------------------------------------------------------------ rope

// N cosines and sines from pair i of a table row on.
template <int N>
__device__ __forceinline__ void load_angles(const float2 *row, int i, float (&c)[N], float (&s)[N])
{
    if constexpr (N % 2 == 0) {  // (vector paths: i a multiple of 2, rows 16-byte aligned)
        const float4 *p = reinterpret_cast<const float4 *>(row + i);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            const float4 v = __ldg(p + j);
            c[2 * j] = v.x;
            s[2 * j] = v.y;
            c[2 * j + 1] = v.z;
            s[2 * j + 1] = v.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float2 v = __ldg(row + i + j);
            c[j] = v.x;
            s[j] = v.y;
        }
    }
}

struct RopeArgs {
    const int32_t *positions;
    const float *table;
    int table_len, T, H, D, rot;
    long long xt, xh, yt, yh;
    int inverse;
    int turning;  // work units of a head that turn; then those that are copied
    int units;    // work units per head: two vectors each
    int chunks;   // threads that share a token's heads
    int *err;
};

constexpr int ROPE_HEADS = 4;  // heads a thread takes, with the same cosines and sines

// A unit is two vectors of NV elements (16 bytes, or one element where the
// call is not aligned): of a head's turning part the two vectors that turn with
// each other (half layout) or two neighbouring ones (interleaved), of the rest
// neighbouring ones; the second may be missing.  A thread takes one unit of ROPE_HEADS
// heads (chunk, chunk + chunks, ...) of a token, so its cosines and sines are
// loaded once and its loads are all in flight together; consecutive threads
// take consecutive units, then consecutive heads.  HBM bounds it: 4096 x 64
// heads x 128 bf16 in 24.6 us, 82 % of a plain copy's rate, 5003 x 64 x 64
// fp32 in 25.4 us, 97 %.
template <typename T, int NV, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(const T *x, T *y, RopeArgs a)
{
    pdl_trigger();
    pdl_wait();
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    const int per_token = a.units * a.chunks;
    const int t = (int)(i / per_token);
    if (t >= a.T) return;
    const int r = (int)(i - (long long)t * per_token);
    const int chunk = r / a.units, u = r - chunk * a.units;
    const int half = a.rot / 2;
    const bool turns = u < a.turning;
    int d0, d1;  // the unit's vectors; d1 = -1: none
    if (turns && !INTER) {
        d0 = NV * u;
        d1 = d0 + half;
    } else {
        d0 = turns ? 2 * NV * u : a.rot + 2 * NV * (u - a.turning);
        d1 = d0 + NV < (turns ? a.rot : a.D) ? d0 + NV : -1;
    }
    uint4 r0[ROPE_HEADS], r1[ROPE_HEADS];  // NV = 1: one element in .x
    const T *xp = x + t * a.xt;
#pragma unroll
    for (int k = 0; k < ROPE_HEADS; ++k) {
        const int h = chunk + k * a.chunks;
        if (h >= a.H) break;
        const T *p = xp + h * a.xh;
        if constexpr (NV > 1) {
            r0[k] = *reinterpret_cast<const uint4 *>(p + d0);
            if (d1 >= 0) r1[k] = *reinterpret_cast<const uint4 *>(p + d1);
        } else {
            r0[k].x = __float_as_uint(Vec<T>::one(p + d0));
            if (d1 >= 0) r1[k].x = __float_as_uint(Vec<T>::one(p + d1));
        }
    }
    const int pos = a.positions[t];
    const bool ok = a.rot == 0 || (unsigned)pos < (unsigned)a.table_len;  // (no rotation: a copy)
    if (!ok && r == 0) set_device_error(a.err, DEVERR_BAD_POSITION);
    float c[NV], s[NV];  // of the pairs of both vectors
    if (turns) {
        const float2 *row = reinterpret_cast<const float2 *>(a.table) + (size_t)(ok ? pos : 0) * half;
        if (!INTER || NV == 1) {
            load_angles<NV>(row, INTER ? d0 / 2 : d0, c, s);
        } else if constexpr (NV > 1) {
            float ca[NV / 2], sa[NV / 2], cb[NV / 2] = {}, sb[NV / 2] = {};
            load_angles<NV / 2>(row, d0 / 2, ca, sa);
            if (d1 >= 0) load_angles<NV / 2>(row, d1 / 2, cb, sb);
#pragma unroll
            for (int j = 0; j < NV / 2; ++j) {
                c[j] = ca[j];
                s[j] = sa[j];
                c[NV / 2 + j] = cb[j];
                s[NV / 2 + j] = sb[j];
            }
        }
        if (a.inverse)
#pragma unroll
            for (int j = 0; j < NV; ++j) s[j] = -s[j];
    }
    T *yp = y + t * a.yt;
#pragma unroll
    for (int k = 0; k < ROPE_HEADS; ++k) {
        const int h = chunk + k * a.chunks;
        if (h >= a.H) break;
        T *p = yp + h * a.yh;
        const float nan = __uint_as_float(0x7FC00000u);
        if constexpr (NV > 1) {
            if (turns || !ok) {
                float v0[NV], v1[NV];
                Vec<T>::get(r0[k], v0);
                Vec<T>::get(r1[k], v1);
#pragma unroll
                for (int j = 0; j < (INTER ? NV / 2 : NV); ++j) {
                    if constexpr (INTER) {
                        turn(v0[2 * j], v0[2 * j + 1], c[j], s[j]);
                        turn(v1[2 * j], v1[2 * j + 1], c[NV / 2 + j], s[NV / 2 + j]);
                    } else {
                        turn(v0[j], v1[j], c[j], s[j]);
                    }
                }
                if (!ok)
#pragma unroll
                    for (int j = 0; j < NV; ++j) v0[j] = v1[j] = nan;
                r0[k] = Vec<T>::put(v0);
                r1[k] = Vec<T>::put(v1);
            }
            *reinterpret_cast<uint4 *>(p + d0) = r0[k];
            if (d1 >= 0) *reinterpret_cast<uint4 *>(p + d1) = r1[k];
        } else {
            float v0 = __uint_as_float(r0[k].x), v1 = d1 >= 0 ? __uint_as_float(r1[k].x) : 0.0f;
            if (turns) turn(v0, v1, c[0], s[0]);
            Vec<T>::set_one(p + d0, ok ? v0 : nan);
            if (d1 >= 0) Vec<T>::set_one(p + d1, ok ? v1 : nan);
        }
    }
}

template <typename T>
static cudaError_t run_rope(cudaStream_t st, const void *x, void *y, RopeArgs a, bool inter)
{
    constexpr int N = Vec<T>::N;
    // 16-byte accesses need every vector of every head aligned, and whole vectors on both sides of `rot`
    // (of rot / 2 where the halves are the pairs).  4096 x 64 heads x 128 bf16: 23.2 us, and 56.0 us
    // by single elements (the same call, one element off).
    const uintptr_t addr = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y);
    const bool vec = (addr & 15u) == 0 && (a.xt | a.xh | a.yt | a.yh) % N == 0 && a.D % N == 0 &&
                     (inter ? a.rot : a.rot / 2) % N == 0 && a.rot % N == 0;
    const int nv = vec ? N : 1;
    a.turning = inter ? (a.rot + 2 * nv - 1) / (2 * nv) : a.rot / 2 / nv;
    a.units = a.turning + (a.D - a.rot + 2 * nv - 1) / (2 * nv);
    if ((long long)a.units * ((a.H + ROPE_HEADS - 1) / ROPE_HEADS) > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    a.chunks = (a.H + ROPE_HEADS - 1) / ROPE_HEADS;
    const long long blocks = ((long long)a.T * a.units * a.chunks + 255) / 256;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(256);
    const T *xs = static_cast<const T *>(x);
    T *ys = static_cast<T *>(y);
    if (vec && inter) return launch_k(rope_kernel<T, N, true>, grid, block, 0, st, xs, ys, a);
    if (vec) return launch_k(rope_kernel<T, N, false>, grid, block, 0, st, xs, ys, a);
    if (inter) return launch_k(rope_kernel<T, 1, true>, grid, block, 0, st, xs, ys, a);
    return launch_k(rope_kernel<T, 1, false>, grid, block, 0, st, xs, ys, a);
}

cudaError_t launch_rope(const DeviceState &ds, cudaStream_t st, const void *x, void *y, int dtype,
                        const int32_t *positions, const float *table, int table_len, int T, int H, int D, int rot,
                        int64_t xt, int64_t xh, int64_t yt, int64_t yh, int flags)
{
    RopeArgs a;
    a.positions = positions;
    a.table = table;
    a.table_len = table_len;
    a.T = T;
    a.H = H;
    a.D = D;
    a.rot = rot;
    a.xt = xt;
    a.xh = xh;
    a.yt = yt;
    a.yh = yh;
    a.inverse = (flags & MX_ROPE_INVERSE) != 0;
    a.err = ds.err;
    const bool inter = (flags & MX_ROPE_INTERLEAVED) != 0;
    return dtype == MX_F32 ? run_rope<float>(st, x, y, a, inter) : run_rope<uint16_t>(st, x, y, a, inter);
}

// ------------------------------------------------------------ append

struct AppendArgs {
    mx_paged_kv kv;
    const int32_t *q_start, *kv_len;
    const float *table;
    int table_len, rot;
    uint16_t *q;
    int T, B, Hq, heads;  // heads: Hq + 2 Hkv
    int slots;            // heads a block of kv_append_kernel covers in a round
    long long row_stride;
    int *err;
};

constexpr int APPEND_THREADS = 256;
constexpr int APPEND_VECTORS = 2;  // vectors of eight elements a thread of the any-layout kernel takes

// Blocks per SM of kv_append_kernel, by its registers: three for bf16 rows (45
// -> 37 us at 4096 x 80 heads x 128 into MXFP8), two for fp32 rows, which
// would spill (49 against 57 us; one token per block).
template <typename T>
constexpr int append_resident()
{
    return sizeof(T) == 2 ? 3 : 2;
}

// Eight elements of a row as they lie, and as fp32.
template <typename T>
struct Raw8 {
    uint4 r[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        if constexpr (sizeof(T) == 2) {
            Vec<uint16_t>::get(r[0], v);
        } else {
            float a[4], b[4];
            Vec<float>::get(r[0], a);
            Vec<float>::get(r[1], b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8])
{
    Raw8<T> r;
    r.load(p);
    r.get(v);
}

// Where a token's keys and values go, found by the whole warp.
struct Place {
    bool some, pos_ok;  // the row belongs to a sequence; its position is in the table
    long long pos;
    int page, slot;     // page < 0: none
};

__device__ __forceinline__ Place place_of(const AppendArgs &a, int t, bool report)
{
    Place p;
    const int b = sequence_of(a.q_start, a.B, t);
    p.some = b >= 0;
    p.pos_ok = false;
    p.page = -1;
    p.slot = 0;
    p.pos = 0;
    if (!p.some) return p;
    const int first = __ldg(a.q_start + b), end = __ldg(a.q_start + b + 1);
    p.pos = (long long)__ldg(a.kv_len + b) - (end - first) + (t - first);
    p.pos_ok = p.pos >= 0 && (a.rot == 0 || p.pos < a.table_len);
    if (p.pos_ok) {
        const int pi = (int)p.pos / a.kv.page_size;
        p.slot = (int)p.pos - pi * a.kv.page_size;
        p.page = page_of(a.kv, a.kv.block_table + (size_t)b * a.kv.table_stride, pi);
    }
    if (p.page < 0 && report) set_device_error(a.err, p.pos_ok ? DEVERR_BAD_PAGE : DEVERR_BAD_POSITION);
    return p;
}

// Eight elements (from d on) of head h of the keys or the values to the cache.
// MXFP8: four neighbouring lanes hold a block.
template <int KVF>
__device__ __forceinline__ void cache8(const AppendArgs &a, const Place &at, bool is_v, int h, int d, const float (&v)[8])
{
    const long long o = at.page * a.kv.page_stride + h * a.kv.head_stride + at.slot * a.kv.token_stride + d;
    if constexpr (KVF == KV_BF16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(is_v ? a.kv.v : a.kv.k) + o) = Vec<uint16_t>::put(v);
    } else {
        // the block's largest magnitude as bits: a NaN or an infinity is 0x7F800000 or above
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        const unsigned four = 0xFu << (threadIdx.x & 28);
        m = max(m, __shfl_xor_sync(four, m, 1));
        m = max(m, __shfl_xor_sync(four, m, 2));
        uint32_t sb = 0xFFu;
        uint2 c = make_uint2(0u, 0u);
        if (m < 0x7F800000u) {
            const int e = max((int)(m >> 23) - 127 - 8, -127);
            const float mul = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, exact products
            sb = (uint32_t)(e + 127);
            c.x = e4m3x4_plus_zero(f32x4_to_e4m3x4(v[0] * mul, v[1] * mul, v[2] * mul, v[3] * mul));
            c.y = e4m3x4_plus_zero(f32x4_to_e4m3x4(v[4] * mul, v[5] * mul, v[6] * mul, v[7] * mul));
        }
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_v ? a.kv.v : a.kv.k) + o) = c;
        if ((d & 31) == 0)
            static_cast<uint8_t *>(is_v ? a.kv.v_scales
                                        : a.kv.k_scales)[at.page * a.kv.scale_page_stride + h * a.kv.scale_head_stride +
                                                         at.slot * a.kv.scale_token_stride + d / 32] = (uint8_t)sb;
    }
}

constexpr int APPEND_HEADS = 3;  // heads a thread takes at a time

// A block takes a token (or part of its heads), with MANY one token after the
// other; a thread takes unit u, two vectors of eight elements, of heads slot, slot + slots, ...; in the half layout the
// two vectors of a turning unit turn with each other, so nothing is read
// twice and the cosines and sines are loaded once for all heads.  Needs whole units, and
// for MXFP8 blocks of 32 that lie in four neighbouring lanes (append_units_ok).
// The row's loads are issued before the search for the token's place, a chain of
// four or five loads; with MANY each warp searches for one of the block's next
// tokens, so the chain is gone through once for as many.
// Bound by HBM: 4096 x 80 heads x 128 bf16 into MXFP8 33.2 us (73 % of a plain copy's
// rate; 37.2 with a block for each token), 8192 tokens 61.5 us (79 %; 68.4), of
// fp32 rows 80.7 us (91 %; 92.6).  Up to as many tokens as blocks are resident the loop only
// costs (one token 2.8 us, 3.2 with it).
template <typename T, int KVF, bool INTER, bool MANY>
__global__ void __launch_bounds__(APPEND_THREADS, append_resident<T>()) kv_append_kernel(const T *__restrict__ rows, AppendArgs a)
{
    pdl_trigger();
    __shared__ Place places[APPEND_THREADS / 32];
    const int D = a.kv.D, units = D / 16, slots = a.slots, warps = blockDim.x / 32;
    const int slot = threadIdx.x / units, u = threadIdx.x - slot * units;
    const int turning = a.Hq + a.kv.Hkv, half = a.rot / 2, hu = a.rot / 16;
    // the unit's vectors in heads that turn (half layout: partners) and in the others
    const bool partners = !INTER && u < hu;
    const int dt0 = INTER ? 8 * u : (partners ? 8 * u : a.rot + 8 * (u - hu));
    const int dt1 = INTER ? dt0 + D / 2 : (partners ? dt0 + half : dt0 + (D - a.rot) / 2);
    const int dv0 = 8 * u, dv1 = dv0 + D / 2;
    pdl_wait();
    float c0[8], s0[8], c1[4], s1[4];
    const int step = slots * gridDim.y;  // heads a round of all blocks of the token covers
    int i = 0;
    int t = blockIdx.x;
    do {
        const T *row = rows + t * a.row_stride;
        Place at;
        for (int h0 = slot < slots ? blockIdx.y * slots + slot : a.heads, round = 0;; h0 += APPEND_HEADS * step, ++round) {
            const bool some = h0 < a.heads;
            Raw8<T> r0[APPEND_HEADS], r1[APPEND_HEADS];
            if (some)
#pragma unroll
                for (int k = 0; k < APPEND_HEADS; ++k) {
                    const int h = h0 + k * step;
                    if (h >= a.heads) break;
                    r0[k].load(row + (long long)h * D + (h < turning ? dt0 : dv0));
                    r1[k].load(row + (long long)h * D + (h < turning ? dt1 : dv1));
                }
            if (round == 0) {
                if constexpr (!MANY) {
                    at = place_of(a, t, threadIdx.x == 0 && blockIdx.y == 0);
                } else if (i % warps == 0) {  // a warp for each of the block's next tokens
                    __syncthreads();
                    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
                    const long long mine = t + (long long)warp * gridDim.x;
                    if (mine < a.T) {
                        const Place p = place_of(a, (int)mine, lane == 0 && blockIdx.y == 0);
                        if (lane == 0) places[warp] = p;
                    }
                    __syncthreads();
                }
                if constexpr (MANY) at = places[i % warps];
                if (!at.some) break;
                const float2 *cs = reinterpret_cast<const float2 *>(a.table) + (at.pos_ok ? at.pos : 0) * half;
                if (partners) load_angles<8>(cs, dt0, c0, s0);
                if constexpr (INTER) {
                    float ca[4], sa[4];
                    if (dt0 < a.rot) load_angles<4>(cs, dt0 / 2, ca, sa);
                    if (dt1 < a.rot) load_angles<4>(cs, dt1 / 2, c1, s1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        c0[j] = ca[j];
                        s0[j] = sa[j];
                    }
                }
            }
            if (!some) break;
#pragma unroll
            for (int k = 0; k < APPEND_HEADS; ++k) {
                const int h = h0 + k * step;
                if (h >= a.heads) break;
                float v0[8], v1[8];
                r0[k].get(v0);
                r1[k].get(v1);
                if (h < turning) {
                    if (partners) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) turn(v0[j], v1[j], c0[j], s0[j]);
                    }
                    if constexpr (INTER) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (dt0 < a.rot) turn(v0[2 * j], v0[2 * j + 1], c0[j], s0[j]);
                            if (dt1 < a.rot) turn(v1[2 * j], v1[2 * j + 1], c1[j], s1[j]);
                        }
                    }
                }
                if (h < a.Hq) {
                    if (at.page < 0)
#pragma unroll
                        for (int j = 0; j < 8; ++j) v0[j] = v1[j] = __uint_as_float(0x7FC00000u);
                    uint16_t *q = a.q + ((size_t)t * a.Hq + h) * D;
                    *reinterpret_cast<uint4 *>(q + dt0) = Vec<uint16_t>::put(v0);
                    *reinterpret_cast<uint4 *>(q + dt1) = Vec<uint16_t>::put(v1);
                } else if (at.page >= 0) {
                    const bool is_v = h >= turning;
                    cache8<KVF>(a, at, is_v, h - (is_v ? turning : a.Hq), is_v ? dv0 : dt0, v0);
                    cache8<KVF>(a, at, is_v, h - (is_v ? turning : a.Hq), is_v ? dv1 : dt1, v1);
                }
            }
        }
        // (by the distance left: t + gridDim.x could pass 32 bits)
    } while (MANY && a.T - t > (int)gridDim.x && (t += gridDim.x, ++i, true));
}

// Whether kv_append_kernel's units fit: whole vectors on both sides of rot (of
// rot / 2 in the half layout), units that divide a block of threads, and blocks of MXFP8
// in four neighbouring lanes.  4096 x 80 heads x 128 into bf16 30 us, MXFP8 34 us; by
// kv_append_any_kernel (rot = 120) 95 and 98 us.
static bool append_units_ok(const AppendArgs &a, bool inter)
{
    const int D = a.kv.D, unit = a.kv.kv_fmt == KV_MXFP8 ? 64 : 16;
    return D % unit == 0 && a.rot % (inter ? 8 : unit) == 0 && (!inter || D / 2 % 8 == 0) && APPEND_THREADS % (D / 16) == 0;
}

// The elements that eight consecutive ones turn with, half layout: `half`
// elements up or down.  Vector load where half is a multiple of 8 (so the
// eight lie on one side), element by element otherwise.
template <typename T>
__device__ __forceinline__ void load_partners(const T *head, int d, int rot, float (&v)[8])
{
    const int half = rot / 2;
    if (half % 8 == 0) {
        if (d < rot) load8(head + (d < half ? d + half : d - half), v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = d + j < half ? Vec<T>::one(head + d + j + half)
                            : (d + j < rot ? Vec<T>::one(head + d + j - half) : 0.0f);
}

// The same for any head size and layout: block (t, y) takes vectors
// y * 512 .. of token t's row; a thread's eight elements are one 16-byte store
// to q or to a bf16 page, or 8 code bytes.  In the half layout each vector also
// loads its partners (its neighbours' own loads, found in L1).
template <typename T, int KVF, bool INTER>
__global__ void __launch_bounds__(APPEND_THREADS) kv_append_any_kernel(const T *__restrict__ rows, AppendArgs a)
{
    pdl_trigger();
    const int t = blockIdx.x;
    const int per_head = a.kv.D / 8, total = a.heads * per_head;
    pdl_wait();
    const int turning = a.Hq + a.kv.Hkv;  // heads that turn
    const Place at = place_of(a, t, threadIdx.x == 0 && blockIdx.y == 0);
    if (!at.some) return;
    const int half = a.rot / 2;
    const float2 *cs = reinterpret_cast<const float2 *>(a.table) + (at.pos_ok ? at.pos : 0) * half;
    for (int k = 0; k < APPEND_VECTORS; ++k) {
        const int u = (blockIdx.y * APPEND_VECTORS + k) * APPEND_THREADS + threadIdx.x;
        if (u >= total) break;
        const int head = u / per_head, d = (u - head * per_head) * 8;
        const T *p = rows + t * a.row_stride + (long long)head * a.kv.D;
        float v[8], w[8];
        load8(p + d, v);
        if (head < turning && d < a.rot && at.pos_ok) {
            if constexpr (INTER) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (d + 2 * j < a.rot) {
                        const float2 c = __ldg(cs + d / 2 + j);
                        turn(v[2 * j], v[2 * j + 1], c.x, c.y);
                    }
            } else {
                load_partners(p, d, a.rot, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = d + j;
                    if (i < half) {
                        const float2 c = __ldg(cs + i);
                        v[j] = __fsub_rn(__fmul_rn(v[j], c.x), __fmul_rn(w[j], c.y));
                    } else if (i < a.rot) {
                        const float2 c = __ldg(cs + i - half);
                        v[j] = __fadd_rn(__fmul_rn(v[j], c.x), __fmul_rn(w[j], c.y));
                    }
                }
            }
        }
        if (head < a.Hq) {
            if (at.page < 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(0x7FC00000u);
            *reinterpret_cast<uint4 *>(a.q + ((size_t)t * a.Hq + head) * a.kv.D + d) = Vec<uint16_t>::put(v);
        } else if (at.page >= 0) {
            const bool is_v = head >= turning;
            cache8<KVF>(a, at, is_v, head - (is_v ? turning : a.Hq), d, v);
        }
    }
}

template <typename T, int KVF>
static cudaError_t run_append(cudaStream_t st, int sms, const void *rows, AppendArgs a, bool inter)
{
    const T *r = static_cast<const T *>(rows);
    if (append_units_ok(a, inter)) {
        // a block as large as a token's heads need; a block for each round of heads
        // where all of them are resident, so that no load waits for another (80 heads
        // into MXFP8: one token 2.8 us, 3.2 with one block, 128 tokens 3.9 against 4.2;
        // 512 tokens, not resident, 10.2 against 6.9)
        const int units = a.kv.D / 16, most = APPEND_THREADS / units;
        a.slots = a.heads < most ? a.heads : most;
        const dim3 block((unsigned)(a.slots * units + 31) / 32 * 32);
        const int resident = sms * (append_resident<T>() * APPEND_THREADS / (int)block.x);
        const int rounds = (a.heads + a.slots - 1) / a.slots;
        const bool few = (long long)a.T * rounds <= resident;
        const dim3 grid((unsigned)(a.T < resident ? a.T : resident), few ? (unsigned)rounds : 1u);
        if (a.T <= resident)
            return inter ? launch_k(kv_append_kernel<T, KVF, true, false>, grid, block, 0, st, r, a)
                         : launch_k(kv_append_kernel<T, KVF, false, false>, grid, block, 0, st, r, a);
        return inter ? launch_k(kv_append_kernel<T, KVF, true, true>, grid, block, 0, st, r, a)
                     : launch_k(kv_append_kernel<T, KVF, false, true>, grid, block, 0, st, r, a);
    }
    const int total = a.heads * (a.kv.D / 8), per_block = APPEND_THREADS * APPEND_VECTORS;
    const dim3 grid((unsigned)a.T, (unsigned)((total + per_block - 1) / per_block));
    if (inter) return launch_k(kv_append_any_kernel<T, KVF, true>, grid, dim3(APPEND_THREADS), 0, st, r, a);
    return launch_k(kv_append_any_kernel<T, KVF, false>, grid, dim3(APPEND_THREADS), 0, st, r, a);
}

cudaError_t launch_kv_append(const DeviceState &ds, cudaStream_t st, const mx_paged_kv &kv, const void *rows,
                             int dtype, int64_t row_stride, const int32_t *q_start, const int32_t *kv_len,
                             const float *table, int table_len, int rot, uint16_t *q, int T, int B, int Hq, int flags)
{
    AppendArgs a;
    a.kv = kv;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.table = table;
    a.table_len = table_len;
    a.rot = rot;
    a.q = q;
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.heads = Hq + 2 * kv.Hkv;
    a.row_stride = row_stride;
    a.err = ds.err;
    const bool inter = (flags & MX_ROPE_INTERLEAVED) != 0;
    if (kv.kv_fmt == KV_MXFP8)
        return dtype == MX_F32 ? run_append<float, KV_MXFP8>(st, ds.num_sms, rows, a, inter)
                               : run_append<uint16_t, KV_MXFP8>(st, ds.num_sms, rows, a, inter);
    return dtype == MX_F32 ? run_append<float, KV_BF16>(st, ds.num_sms, rows, a, inter)
                           : run_append<uint16_t, KV_BF16>(st, ds.num_sms, rows, a, inter);
}

}  // namespace mx
