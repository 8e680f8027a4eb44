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
// the chain of dependent loads (sequence, length, page, table row) and the
// launch for single tokens.
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

// 16 bytes of the type as fp32 and back (rounded once).
template <typename T>
struct Vec;

template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float *p, float (&v)[N])
    {
        const float4 r = *reinterpret_cast<const float4 *>(p);
        v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[N])
    {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float v) { *p = v; }
};

template <>
struct Vec<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const uint16_t *p, float (&v)[N])
    {
        const uint4 r = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    static __device__ __forceinline__ void store(uint16_t *p, const float (&v)[N])
    {
        *reinterpret_cast<uint4 *>(p) = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                                                   f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
    }
    static __device__ __forceinline__ float get(const uint16_t *p) { return bf16_to_f32(*p); }
    static __device__ __forceinline__ void put(uint16_t *p, float v)
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

struct RopeArgs {
    const int32_t *positions;
    const float *table;
    int table_len, T, H, D, rot;
    long long xt, xh, yt, yh;
    int inverse;
    int units;   // work units per head: pairs of vectors that turn, then single vectors that are copied
    int chunks;  // threads that share a token's heads
    int *err;
};

constexpr int ROPE_HEADS = 4;  // heads a thread takes, with the same cosines and sines

// A thread takes one unit of ROPE_HEADS heads (chunk, chunk + chunks, ...)
// of a token, so its cosines and sines are loaded once and its loads are all
// in flight together; consecutive threads take consecutive units, then
// consecutive heads.  NV elements per access: a 16-byte vector, or 1.
template <typename T, int NV, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(const T *x, T *y, RopeArgs a)
{
    pdl_trigger();
    pdl_wait();
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    const long long per_token = (long long)a.units * a.chunks;
    const int t = (int)(i / per_token);
    if (t >= a.T) return;
    const int r = (int)(i - t * per_token);
    const int chunk = r / a.units, u = r - chunk * a.units;
    const int half = a.rot / 2;
    // offsets of the unit's first and second vector; -1: none
    const int turning = INTER ? (a.rot + 2 * NV - 1) / (2 * NV) : half / NV;
    int d0, d1;
    if (u < turning) {
        d0 = INTER ? 2 * NV * u : NV * u;
        d1 = INTER ? (NV == 1 || d0 + NV < a.rot ? d0 + NV : -1) : d0 + half;
    } else {
        d0 = a.rot + NV * (u - turning);
        d1 = -1;
    }
    const int pos = a.positions[t];
    const bool ok = (unsigned)pos < (unsigned)a.table_len;
    if (!ok && r == 0) set_device_error(a.err, DEVERR_BAD_POSITION);
    float c[NV], s[NV];
    if (u < turning) {
        const float2 *cs = reinterpret_cast<const float2 *>(a.table) + (size_t)(ok ? pos : 0) * half + (INTER ? d0 / 2 : d0);
        const int pairs = INTER && d1 < 0 ? NV / 2 : NV;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const float2 v = j < pairs ? __ldg(cs + j) : make_float2(1.0f, 0.0f);
            c[j] = v.x;
            s[j] = a.inverse ? -v.y : v.y;
        }
    }
    float v0[ROPE_HEADS][NV], v1[ROPE_HEADS][NV];
#pragma unroll
    for (int k = 0; k < ROPE_HEADS; ++k) {
        const int h = chunk + k * a.chunks;
        if (h >= a.H) break;
        const T *p = x + t * a.xt + h * a.xh;
        if constexpr (NV > 1) {
            Vec<T>::load(p + d0, v0[k]);
            if (d1 >= 0) Vec<T>::load(p + d1, v1[k]);
        } else {
            v0[k][0] = Vec<T>::get(p + d0);
            if (d1 >= 0) v1[k][0] = Vec<T>::get(p + d1);
        }
    }
#pragma unroll
    for (int k = 0; k < ROPE_HEADS; ++k) {
        const int h = chunk + k * a.chunks;
        if (h >= a.H) break;
        if (u < turning) {
            if constexpr (INTER && NV > 1) {
#pragma unroll
                for (int j = 0; j < NV / 2; ++j) turn(v0[k][2 * j], v0[k][2 * j + 1], c[j], s[j]);
                if (d1 >= 0)
#pragma unroll
                    for (int j = 0; j < NV / 2; ++j)
                        turn(v1[k][2 * j], v1[k][2 * j + 1], c[NV / 2 + j], s[NV / 2 + j]);
            } else {
#pragma unroll
                for (int j = 0; j < NV; ++j) turn(v0[k][j], v1[k][j], c[j], s[j]);
            }
        }
        if (!ok) {
#pragma unroll
            for (int j = 0; j < NV; ++j) v0[k][j] = v1[k][j] = __uint_as_float(0x7FC00000u);
        }
        T *p = y + t * a.yt + h * a.yh;
        if constexpr (NV > 1) {
            Vec<T>::store(p + d0, v0[k]);
            if (d1 >= 0) Vec<T>::store(p + d1, v1[k]);
        } else {
            Vec<T>::put(p + d0, v0[k][0]);
            if (d1 >= 0) Vec<T>::put(p + d1, v1[k][0]);
        }
    }
}

template <typename T>
static cudaError_t run_rope(cudaStream_t st, const void *x, void *y, RopeArgs a, bool inter)
{
    constexpr int N = Vec<T>::N;
    // 16-byte accesses need every vector of every head aligned, and whole vectors on both sides of `rot`
    // (of rot / 2 where the halves are the pairs)
    const uintptr_t addr = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y);
    const bool vec = (addr & 15u) == 0 && (a.xt | a.xh | a.yt | a.yh) % N == 0 && a.D % N == 0 &&
                     (inter ? a.rot : a.rot / 2) % N == 0 && a.rot % N == 0;
    const int nv = vec ? N : 1;
    a.units = (inter ? (a.rot + 2 * nv - 1) / (2 * nv) : a.rot / 2 / nv) + (a.D - a.rot) / nv;
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
    long long row_stride;
    int *err;
};

constexpr int APPEND_THREADS = 256;
constexpr int APPEND_UNITS = 2;  // units of 8 elements a thread takes

// Eight elements of a row from element d of a head.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8])
{
    if constexpr (sizeof(T) == 2) {
        Vec<uint16_t>::load(p, v);
    } else {
        const float4 r0 = *reinterpret_cast<const float4 *>(p), r1 = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = r0.x; v[1] = r0.y; v[2] = r0.z; v[3] = r0.w;
        v[4] = r1.x; v[5] = r1.y; v[6] = r1.z; v[7] = r1.w;
    }
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
        v[j] = d + j < half ? Vec<T>::get(head + d + j + half)
                            : (d + j < rot ? Vec<T>::get(head + d + j - half) : 0.0f);
}

// Block (t, y) takes units y * 512 .. of token t's row: a unit is eight
// consecutive elements of one head, so that a unit's results are one 16-byte
// store to q or to a bf16 page, or 8 code bytes of an MXFP8 page, whose
// blocks of 32 are then four neighbouring lanes.  In the half layout each
// unit also loads its partners (its neighbours' own loads, found in L1).  The
// row's loads are issued before the search for the token's place.
template <typename T, int KVF, bool INTER>
__global__ void __launch_bounds__(APPEND_THREADS) kv_append_kernel(const T *__restrict__ rows, AppendArgs a)
{
    pdl_trigger();
    const int t = blockIdx.x;
    const int per_head = a.kv.D / 8, total = a.heads * per_head;
    int head[APPEND_UNITS], d[APPEND_UNITS];
#pragma unroll
    for (int k = 0; k < APPEND_UNITS; ++k) {
        const int u = (blockIdx.y * APPEND_UNITS + k) * APPEND_THREADS + threadIdx.x;
        head[k] = u < total ? u / per_head : -1;
        d[k] = (u - head[k] * per_head) * 8;
    }
    pdl_wait();
    const int turning = a.Hq + a.kv.Hkv;  // heads that turn
    float v[APPEND_UNITS][8], w[APPEND_UNITS][8];
#pragma unroll
    for (int k = 0; k < APPEND_UNITS; ++k) {
        if (head[k] < 0) continue;
        const T *p = rows + t * a.row_stride + (long long)head[k] * a.kv.D;
        load8(p + d[k], v[k]);
        if (!INTER && head[k] < turning) load_partners(p, d[k], a.rot, w[k]);
    }
    const int b = sequence_of(a.q_start, a.B, t);
    if (b < 0) return;  // a row of no sequence
    const int first = __ldg(a.q_start + b), end = __ldg(a.q_start + b + 1);
    const long long pos = (long long)__ldg(a.kv_len + b) - (end - first) + (t - first);
    const bool pos_ok = pos >= 0 && (a.rot == 0 || pos < a.table_len);
    int page = -1, slot = 0;
    if (pos_ok) {
        const int pi = (int)(pos / a.kv.page_size);
        slot = (int)(pos - (long long)pi * a.kv.page_size);
        page = page_of(a.kv, a.kv.block_table + (size_t)b * a.kv.table_stride, pi);
    }
    if (page < 0 && threadIdx.x == 0 && blockIdx.y == 0)
        set_device_error(a.err, pos_ok ? DEVERR_BAD_PAGE : DEVERR_BAD_POSITION);
    const int half = a.rot / 2;
    const float2 *cs = reinterpret_cast<const float2 *>(a.table) + (pos_ok ? pos : 0) * half;
#pragma unroll
    for (int k = 0; k < APPEND_UNITS; ++k) {
        if (head[k] < 0) continue;
        if (head[k] < turning && d[k] < a.rot && pos_ok) {
            if constexpr (INTER) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (d[k] + 2 * j < a.rot) {
                        const float2 c = __ldg(cs + d[k] / 2 + j);
                        turn(v[k][2 * j], v[k][2 * j + 1], c.x, c.y);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = d[k] + j;
                    if (i < half) {
                        const float2 c = __ldg(cs + i);
                        v[k][j] = __fsub_rn(__fmul_rn(v[k][j], c.x), __fmul_rn(w[k][j], c.y));
                    } else if (i < a.rot) {
                        const float2 c = __ldg(cs + i - half);
                        v[k][j] = __fadd_rn(__fmul_rn(v[k][j], c.x), __fmul_rn(w[k][j], c.y));
                    }
                }
            }
        }
        if (head[k] < a.Hq) {
            if (page < 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[k][j] = __uint_as_float(0x7FC00000u);
            Vec<uint16_t>::store(a.q + ((size_t)t * a.Hq + head[k]) * a.kv.D + d[k], v[k]);
            continue;
        }
        if (page < 0) continue;
        const bool is_v = head[k] >= turning;
        const int h = head[k] - (is_v ? turning : a.Hq);
        const long long at = page * a.kv.page_stride + h * a.kv.head_stride + slot * a.kv.token_stride + d[k];
        if constexpr (KVF == KV_BF16) {
            Vec<uint16_t>::store(static_cast<uint16_t *>(is_v ? a.kv.v : a.kv.k) + at, v[k]);
        } else {
            // the block's largest magnitude as bits: a NaN or an infinity is 0x7F800000 or above
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[k][j]) & 0x7FFFFFFFu);
            const unsigned four = 0xFu << (threadIdx.x & 28);
            m = max(m, __shfl_xor_sync(four, m, 1));
            m = max(m, __shfl_xor_sync(four, m, 2));
            uint32_t sb = 0xFFu;
            uint2 c = make_uint2(0u, 0u);
            if (m < 0x7F800000u) {
                const int e = max((int)(m >> 23) - 127 - 8, -127);
                const float mul = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, exact products
                sb = (uint32_t)(e + 127);
                c.x = e4m3x4_plus_zero(f32x4_to_e4m3x4(v[k][0] * mul, v[k][1] * mul, v[k][2] * mul, v[k][3] * mul));
                c.y = e4m3x4_plus_zero(f32x4_to_e4m3x4(v[k][4] * mul, v[k][5] * mul, v[k][6] * mul, v[k][7] * mul));
            }
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_v ? a.kv.v : a.kv.k) + at) = c;
            if ((d[k] & 31) == 0)
                static_cast<uint8_t *>(is_v ? a.kv.v_scales : a.kv.k_scales)[page * a.kv.scale_page_stride +
                                                                             h * a.kv.scale_head_stride +
                                                                             slot * a.kv.scale_token_stride +
                                                                             d[k] / 32] = (uint8_t)sb;
        }
    }
}

template <typename T, int KVF>
static cudaError_t run_append(cudaStream_t st, const void *rows, const AppendArgs &a, bool inter)
{
    const int total = a.heads * (a.kv.D / 8), per_block = APPEND_THREADS * APPEND_UNITS;
    const dim3 grid((unsigned)a.T, (unsigned)((total + per_block - 1) / per_block));
    const T *r = static_cast<const T *>(rows);
    if (inter) return launch_k(kv_append_kernel<T, KVF, true>, grid, dim3(APPEND_THREADS), 0, st, r, a);
    return launch_k(kv_append_kernel<T, KVF, false>, grid, dim3(APPEND_THREADS), 0, st, r, a);
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
        return dtype == MX_F32 ? run_append<float, KV_MXFP8>(st, rows, a, inter)
                               : run_append<uint16_t, KV_MXFP8>(st, rows, a, inter);
    return dtype == MX_F32 ? run_append<float, KV_BF16>(st, rows, a, inter)
                           : run_append<uint16_t, KV_BF16>(st, rows, a, inter);
}

}  // namespace mx
