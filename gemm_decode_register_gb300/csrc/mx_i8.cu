// mx_i8.cu -- products of 8-bit integers with a scale for each token and each
// output channel, sm_103a:
//   y[m][n] = (sum_k xq[m][k] wq[n][k]) * sx[m] * sw[n].
//
// Quantisation (bound: latency; for many tokens a block's loads, barrier and stores
// take turns: 4096 rows of 8192 bf16 take 37 us, where HBM would allow 15; of 28672 100, of
// 53): a block per token, its row, or as much as fits, held in registers between
// the maximum and the rounding.
//
// Few tokens (bound: HBM, the weights once): mma.sync m16n8k32 on 8-bit
// integers, 32-bit sums, exact.  A warp's 16 weight rows come straight from
// global memory, 16 bytes per lane; the order of k within 64 elements is the
// lanes' own (lane t of four holds elements 16t .. 16t+15 of both operands),
// which a sum does not mind, so nothing is rearranged or decoded.  The warps
// of a CTA share out a row tile's K between them, the tile's sums meet in
// shared memory, and the next tile's loads are in flight meanwhile.  1.05 GB of
// weights take 154-158 us for up to eight tokens, the measured copy's rate; 84 MB 16,
// of 12.5, since 640 row tiles make five rounds of 152 SMs.  (Equal stretches
// of K for each CTA, with the shared tiles' sums through global memory, took longer: 24
// against 20 us, 167 against 156; so do pairs of CTAs where single ones have the room, 25
// against 19; quantising the tokens here too saves a launch, and 0.5 to 2 us are lost.)
//
// Many tokens: mx_qmm.cu's tensor-core GEMM.  sm_103a has no 8-bit integer
// form of tcgen05.mma, and integers up to 2048 are exact in f16: tokens are
// written as f16 integers by the quantisation, weights decoded to f16 in
// shared memory, products summed in fp32 (exact while sums stay below 2^24).
#include <cmath>

#include "mx_common.cuh"
#include "mx_serve.h"
#include "mx_tc.cuh"

namespace mx {

// ------------------------------------------------------------ quantisation

constexpr int QI8_KEEP = 4;  // 8-element groups per thread kept in registers

// Eight elements as fp32.
__device__ __forceinline__ void load8(const uint16_t *p, float (&v)[8])
{
    const uint4 r = __ldcg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const float4 a = __ldcg(reinterpret_cast<const float4 *>(p)), b = __ldcg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Adding it rounds a number of less than 2^22 to the nearest even integer, which the
// sum's low bits then are (by 1024 threads each, 4096 rows of 16384 took 120 us by
// conversions, 105 by this).
constexpr float INT_AT = 12582912.0f;  // 1.5 * 2^23

// x / s to the nearest integers, r = 1 / s.  x r is within 3 * 2^-24 of the
// quotient (relative; 127 * that is 2.3e-5), so it has the same nearest integer unless
// a tie is that near; then, and where r or the product is no number, the quotients
// themselves decide.
__device__ __forceinline__ void codes_of(const float (&x)[8], float s, float r, float (&c)[8])
{
    bool near = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = __fmul_rn(x[j], r);
        c[j] = __fsub_rn(__fadd_rn(t, INT_AT), INT_AT);
        near |= !(fabsf(t - c[j]) < 0.4999f);
    }
    if (near)
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = rintf(fminf(fmaxf(__fdiv_rn(x[j], s), -127.0f), 127.0f));
}

// The larger of m and the magnitudes, as bits: these are in the order of the
// values, infinities above them and a NaN above those.
__device__ __forceinline__ uint32_t most_of(uint32_t m, const float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    return m;
}

__device__ __forceinline__ void store8(int8_t *p, const float (&c)[8])
{
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = __float_as_uint(__fadd_rn(c[j], INT_AT));
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040), __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}
// f16 integers (bits), exact.
__device__ __forceinline__ void store8(uint16_t *p, const float (&c)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32x2_to_f16x2(c[2 * i], c[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// One token per block: s = max |x| / 127, q = x / s to the nearest even
// integer.  s = 0 (a row of zeros, or of values that small): q = 0.  A NaN or
// an infinity in the row: s = NaN, q = 0.  early: whether dependents may start
// at once; not when the codes may be the next call's weights, which its kernel
// reads before it waits.
template <typename In, typename Out, int THREADS>
__global__ void __launch_bounds__(THREADS) i8_quantize_kernel(const In *__restrict__ x, Out *__restrict__ q,
                                                              float *__restrict__ scales, int K, bool early)
{
    __shared__ uint32_t wmax[THREADS / 32];
    if (early) pdl_trigger();
    pdl_wait();
    const size_t row = blockIdx.x;
    const In *xr = x + row * K;
    Out *qr = q + row * K;
    const int groups = K / 8;
    float keep[QI8_KEEP][8];
    uint32_t m = 0u;
#pragma unroll
    for (int u = 0; u < QI8_KEEP; ++u) {
        const int i = u * THREADS + (int)threadIdx.x;
        if (i >= groups) break;
        load8(xr + 8 * i, keep[u]);
        m = most_of(m, keep[u]);
    }
    for (int i = QI8_KEEP * THREADS + (int)threadIdx.x; i < groups; i += THREADS) {
        float v[8];
        load8(xr + 8 * i, v);
        m = most_of(m, v);
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0u;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) m = max(m, wmax[w]);
    const float s = m >= 0x7F800000u ? NAN : __fdiv_rn(__uint_as_float(m), 127.0f);
    if (threadIdx.x == 0) scales[row] = s;
    const float r = __frcp_rn(s);
    const auto write = [&](int i, const float (&v)[8]) {
        float c[8] = {};
        if (s > 0.0f) codes_of(v, s, r, c);
        store8(qr + 8 * i, c);
    };
#pragma unroll
    for (int u = 0; u < QI8_KEEP; ++u) {
        const int i = u * THREADS + (int)threadIdx.x;
        if (i >= groups) break;
        write(i, keep[u]);
    }
    for (int i = QI8_KEEP * THREADS + (int)threadIdx.x; i < groups; i += THREADS) {
        float v[8];
        load8(xr + 8 * i, v);
        write(i, v);
    }
    if (!early) __threadfence();
}

// 8-bit integers as f16 integers, 16 at a time.
__global__ void __launch_bounds__(256) i8_widen_kernel(const int8_t *__restrict__ q, uint16_t *__restrict__ h, size_t n16)
{
    pdl_trigger();
    pdl_wait();
    for (size_t i = blockIdx.x * (size_t)256 + threadIdx.x; i < n16; i += (size_t)gridDim.x * 256) {
        const uint4 r = __ldcg(reinterpret_cast<const uint4 *>(q) + i);
        uint32_t o[8];
        i8x4_to_f16x2(r.x, o[0], o[1]);
        i8x4_to_f16x2(r.y, o[2], o[3]);
        i8x4_to_f16x2(r.z, o[4], o[5]);
        i8x4_to_f16x2(r.w, o[6], o[7]);
        uint4 *d = reinterpret_cast<uint4 *>(h) + 2 * i;
        d[0] = make_uint4(o[0], o[1], o[2], o[3]);
        d[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// ------------------------------------------------------------ few tokens

constexpr int MV_WARPS = 16;
constexpr int MV_THREADS = 32 * MV_WARPS;
constexpr int MV_GROUP = 4;  // 64-element steps of K whose loads are in flight together

struct I8MvArgs {
    const int8_t *x;  // [M][K]
    const float *sx;
    const int8_t *w;
    const float *sw;
    void *y;
    int N, K;
    int tokens;  // of this pass, at most 8 NB
    int parts;   // warps that share a row tile's K: 1, 2, 4, 8 or 16
    int span;    // elements of K of a CTA: all, or the half of a pair's (a multiple of 64)
    int xpitch;  // bytes of a staged token, an odd multiple of 64
};

__device__ __forceinline__ uint4 ld_stream_v4(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// D += A(16x32, s8, row) * B(32x8, s8, col), exact in 32 bits.
__device__ __forceinline__ void mma_s8_16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NB: groups of 8 tokens (places past the last token repeat it).  Y: float or uint16_t (bf16).
// mma.sync does about 130 T 8-bit operations a second here (and no more of f16), what eight
// tokens ask of the weights' stream: 8 through 128000 x 8192 take 154 us, 16 258.
//
// PAIR: where a CTA's shared memory has no room for the tokens, a cluster of two shares
// each row tile, either half of K its own; the halves' sums meet through each
// other's shared memory, and a pass more over the weights is saved (eight tokens
// through 8192 x 28672 48 us after their quantisation, 93 in two passes).
template <int NB, typename Y, bool PAIR>
__global__ void __launch_bounds__(MV_THREADS, 1) i8_mv_kernel(const __grid_constant__ I8MvArgs a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *xs = smem;                                                        // [tokens][xpitch]
    int4 *red = reinterpret_cast<int4 *>(smem + (size_t)a.tokens * a.xpitch);  // [2][warps][NB][32]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int steps = a.span / 64;                 // of a row
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    const int k0 = rank * a.span, ks = min(a.K - k0, a.span);  // this CTA's stretch of K
    const int stride = PAIR ? gridDim.x / 2 : gridDim.x, start = PAIR ? blockIdx.x / 2 : blockIdx.x;
    const int per_cta = MV_WARPS / a.parts;        // row tiles at a time
    const int part = warp % a.parts, sub = warp / a.parts;
    const int tiles = (a.N + 15) / 16;
    const int groups = (steps + a.parts * MV_GROUP - 1) / (a.parts * MV_GROUP);
    const int rounds = (tiles + per_cta - 1) / per_cta;

    // Two buffers of loads, each refilled as soon as it is used, so that two
    // groups are in flight while a warp waits (with one, eight tokens through
    // 128000 x 8192 took 186 us instead of 156).  The loads run ahead over tile ends.
    uint4 even[MV_GROUP][2], odd[MV_GROUP][2];
    int load_round = start, load_q = 0;
    // step number i of group q: part + parts * (q * MV_GROUP + i)
    auto load = [&](uint4 (&v)[MV_GROUP][2]) {
        const int tile = load_round * per_cta + sub;
        const int n0 = 16 * tile + g, n1 = n0 + 8;
        const int8_t *w = a.w + k0 + 16 * t;
#pragma unroll
        for (int i = 0; i < MV_GROUP; ++i) {
            const int k = 64 * (part + a.parts * (load_q * MV_GROUP + i));
            const bool in = load_round < rounds && k + 16 * t < ks;
            v[i][0] = in && n0 < a.N ? ld_stream_v4(w + (size_t)n0 * a.K + k) : make_uint4(0u, 0u, 0u, 0u);
            v[i][1] = in && n1 < a.N ? ld_stream_v4(w + (size_t)n1 * a.K + k) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (++load_q == groups) {
            load_q = 0;
            load_round += stride;
        }
    };
    pdl_trigger();
    load(even);  // weights: before the tokens are there
    load(odd);
    pdl_wait();
    const int vecs = a.xpitch / 16;
    for (int i = threadIdx.x; i < a.tokens * vecs; i += MV_THREADS) {
        const int m = i / vecs, c = i - m * vecs;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (16 * c < ks) v = __ldcg(reinterpret_cast<const uint4 *>(a.x + (size_t)m * a.K + k0) + c);
        *reinterpret_cast<uint4 *>(xs + (size_t)m * a.xpitch + 16 * c) = v;
    }
    __syncthreads();

    int flip = 0, round = start, q = 0;
    int acc[NB][4] = {};
    auto step = [&](uint4 (&v)[MV_GROUP][2]) {
#pragma unroll
        for (int i = 0; i < MV_GROUP; ++i) {
            const int k = min(64 * (part + a.parts * (q * MV_GROUP + i)), 64 * (steps - 1));  // (past the row: weights of zero)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint4 x = *reinterpret_cast<const uint4 *>(xs + (size_t)min(8 * b + g, a.tokens - 1) * a.xpitch + k + 16 * t);
                mma_s8_16832(acc[b], v[i][0].x, v[i][1].x, v[i][0].y, v[i][1].y, x.x, x.y);
                mma_s8_16832(acc[b], v[i][0].z, v[i][1].z, v[i][0].w, v[i][1].w, x.z, x.w);
            }
        }
        load(v);
        if (++q < groups) return;
        q = 0;
        // the parts' sums meet; outputs in rows of 16 channels
        int4 *r = red + (size_t)flip * MV_WARPS * NB * 32;
        flip ^= 1;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            r[(warp * NB + b) * 32 + lane] = make_int4(acc[b][0], acc[b][1], acc[b][2], acc[b][3]);
            acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0;
        }
        if constexpr (PAIR) cluster_sync_all();
        else __syncthreads();
        const int *ri = reinterpret_cast<const int *>(r);
        for (int o = threadIdx.x + rank * MV_THREADS; o < per_cta * NB * 128; o += (PAIR ? 2 : 1) * MV_THREADS) {
            const int row = o % 16, c = o / 16 % 8, b = o / 128 % NB, s = o / (128 * NB);
            const int m = 8 * b + c, n = 16 * (round * per_cta + s) + row;
            if (m >= a.tokens || n >= a.N) continue;
            const int at = 4 * (4 * (row % 8) + c / 2) + 2 * (row / 8) + c % 2;
            int sum = 0;
            for (int p = 0; p < a.parts; ++p) {
                const int *v = ri + ((s * a.parts + p) * NB + b) * 128 + at;
                sum += *v;
                if constexpr (PAIR) sum += ld_cluster_s32(map_to_cta(smem_u32(v), rank ^ 1));
            }
            const float y = __fmul_rn(__fmul_rn((float)sum, __ldcg(a.sx + m)), __ldg(a.sw + n));
            if constexpr (sizeof(Y) == 4) static_cast<float *>(a.y)[(size_t)m * a.N + n] = y;
            else static_cast<uint16_t *>(a.y)[(size_t)m * a.N + n] = (uint16_t)f32x2_to_bf16x2(y, 0.0f);
        }
        round += stride;
    };
    while (round < rounds) {
        step(even);
        if (round >= rounds) break;
        step(odd);
    }
    if constexpr (PAIR) cluster_sync_all();  // (the other CTA may still read this one's sums)
}

// ------------------------------------------------------------ host

// Elements of K that a CTA takes: all, or half where a pair shares them.
static int mv_span(int K, bool pair) { return ((pair ? (K + 1) / 2 : K) + 63) / 64 * 64; }

static int mv_pitch(int span) { return span % 128 == 0 ? span + 64 : span; }  // two tokens' 64 bytes then fall into different banks

static int mv_smem(int tokens, int span) { return tokens * mv_pitch(span) + 2 * MV_WARPS * ((tokens + 7) / 8) * 512; }

constexpr int MV_NB = 2;  // most groups of 8 tokens of a pass

// Most tokens a pass can stage beside the sums' space.
static int mv_pass_tokens(const DeviceState &ds, int span)
{
    for (int m = 8 * MV_NB; m > 0; --m)
        if (mv_smem(m, span) <= ds.max_smem_optin) return m;
    return 0;
}

struct I8Passes {
    int tokens;  // of a pass; 0: not by passes
    bool pair;
};

template <int NB, typename Y, bool PAIR>
static cudaError_t run_mv(const DeviceState &ds, cudaStream_t st, const I8MvArgs &a)
{
    static unsigned char done[64];
    const cudaError_t e = allow_smem(ds, i8_mv_kernel<NB, Y, PAIR>, ds.max_smem_optin, done);
    if (e != cudaSuccess) return e;
    const int rounds = ((a.N + 15) / 16 + MV_WARPS / a.parts - 1) / (MV_WARPS / a.parts), most = ds.num_sms / (PAIR ? 2 : 1);
    const int ctas = (rounds < most ? rounds : most) * (PAIR ? 2 : 1);
    return launch_cluster_k(i8_mv_kernel<NB, Y, PAIR>, PAIR ? 2 : 1, dim3(ctas), dim3(MV_THREADS), mv_smem(a.tokens, a.span), st, a);
}

template <typename Y>
static cudaError_t run_mv_pass(const DeviceState &ds, cudaStream_t st, const I8MvArgs &a, bool pair)
{
    if (pair) return a.tokens <= 8 ? run_mv<1, Y, true>(ds, st, a) : run_mv<2, Y, true>(ds, st, a);
    return a.tokens <= 8 ? run_mv<1, Y, false>(ds, st, a) : run_mv<2, Y, false>(ds, st, a);
}

static cudaError_t launch_i8_mv(const DeviceState &ds, cudaStream_t st, const int8_t *x, const float *sx, const int8_t *w,
                                const float *sw, void *y, int ydtype, int M, int N, int K, I8Passes by)
{
    const size_t ye = ydtype == MX_F32 ? 4 : 2;
    I8MvArgs a;
    a.span = mv_span(K, by.pair);
    a.xpitch = mv_pitch(a.span);
    const int steps = a.span / 64;
    a.parts = 1;  // (each warp has two groups of loads of a tile or more)
    while (a.parts < MV_WARPS && steps >= 2 * a.parts * MV_GROUP) a.parts *= 2;
    for (int m = 0; m < M; m += by.tokens) {
        a.x = x + (size_t)m * K;
        a.sx = sx + m;
        a.w = w;
        a.sw = sw;
        a.y = static_cast<char *>(y) + (size_t)m * N * ye;
        a.N = N;
        a.K = K;
        a.tokens = M - m < by.tokens ? M - m : by.tokens;
        const cudaError_t e = ydtype == MX_F32 ? run_mv_pass<float>(ds, st, a, by.pair) : run_mv_pass<uint16_t>(ds, st, a, by.pair);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename In, typename Out, int THREADS>
static cudaError_t run_quantize_with(cudaStream_t st, const void *x, void *q, float *scales, int M, int K, bool early)
{
    return launch_k(i8_quantize_kernel<In, Out, THREADS>, dim3(M), dim3(THREADS), 0, st, static_cast<const In *>(x),
                    static_cast<Out *>(q), scales, K, early);
}

// Threads of a row, us by 256 / by 1024, of which an SM holds one block.
//   No more rows than SMs: what counts is a row's latency.  8 of 1024 values 1.9 /
// 2.5, of 4096 2.6 / 2.6, of 28672 8.6 / 5.0; 152 of 8192 5.3 / 4.2, of 16384 8.4 / 5.8.
//   More: blocks that overlap (bf16: 153 of 16384 8.4 / 7.9, 256 9.3 / 9.3, 512 11.7 / 16.0;
// 4096 of 4096 22 / 63, of 8192 37 / 74, of 16384 61 / 105, of 28672 101 / 155), also where 256
// threads read twice what registers do not hold; up to rows of 128 KB, of
// which four on every SM are still in L2 then (4096 of 32768 bf16 107 / 162, fp32 140 / 154, of
// 49152 fp32 250 / 240, of 98304 535 / 439; 2048 of 65536 bf16 115 / 140, fp32 184 / 159).
template <typename In, typename Out>
static cudaError_t run_quantize(const DeviceState &ds, cudaStream_t st, const void *x, void *q, float *scales, int M, int K,
                                bool early)
{
    return K > 2048 && (M <= ds.num_sms || K * (long long)sizeof(In) > 128 * 1024)
               ? run_quantize_with<In, Out, 1024>(st, x, q, scales, M, K, early)
               : run_quantize_with<In, Out, 256>(st, x, q, scales, M, K, early);
}

cudaError_t launch_i8_quantize(const DeviceState &ds, cudaStream_t st, const void *x, int dtype, int8_t *q, float *scales,
                               int M, int K, bool early)
{
    return dtype == MX_F32 ? run_quantize<float, int8_t>(ds, st, x, q, scales, M, K, early)
                           : run_quantize<uint16_t, int8_t>(ds, st, x, q, scales, M, K, early);
}

size_t i8_mm_workspace_bytes(int M, int K)
{
    // codes (8-bit for the streaming kernel, f16 for the GEMM), then scales
    const size_t codes = ((size_t)M * K * 2 + 255) / 256 * 256;
    return codes + ((size_t)M * 4 + 255) / 256 * 256;
}

// Passes of the streaming kernel, by single CTAs or pairs, or the GEMM: whichever
// takes least by these estimates (us, measured on GB300).  A pass streams the
// weights, at 6.6 MB per us for up to 8 tokens and 4.0 for up to 16, and takes
// about 5 beside, a pair's 1 more.  The GEMM: see qmm_i8_estimate.
static I8Passes i8_passes(const DeviceState &ds, int M, int N, int K)
{
    I8Passes best = {0, false};
    double least = qmm_i8_estimate(ds, M, N, K);
    for (const bool pair : {false, true}) {
        const int most = mv_pass_tokens(ds, mv_span(K, pair));
        if (most == 0) continue;
        const int passes = (M + most - 1) / most, tokens = (M + passes - 1) / passes;  // (equal passes)
        // (crowded: loads in flight want room in what shared memory leaves of L1)
        const bool crowded = mv_smem(tokens, mv_span(K, pair)) > 200 * 1024;
        const double rate = tokens <= 8 ? (crowded ? 4.4e6 : 6.6e6) : (crowded ? 3.4e6 : 4.0e6);
        const double us = passes * ((double)N * K / rate + (pair ? 6.0 : 5.0));
        if (us > least || (pair && us == least)) continue;
        least = us;
        best = {tokens, pair};
    }
    return best;
}

cudaError_t launch_i8_mm(const DeviceState &ds, cudaStream_t st, const I8Call &c, void *workspace)
{
    const size_t codes = ((size_t)c.M * c.K * 2 + 255) / 256 * 256;
    float *own_sx = reinterpret_cast<float *>(static_cast<char *>(workspace) + codes);
    const float *sx = c.xdtype == MX_I8 ? c.sx : own_sx;
    cudaError_t e;
    const I8Passes by = i8_passes(ds, c.M, c.N, c.K);
    if (by.tokens) {
        const int8_t *x = static_cast<const int8_t *>(c.x);
        if (c.xdtype != MX_I8) {
            e = launch_i8_quantize(ds, st, c.x, c.xdtype, static_cast<int8_t *>(workspace), own_sx, c.M, c.K, true);
            if (e != cudaSuccess) return e;
            x = static_cast<const int8_t *>(workspace);
        }
        return launch_i8_mv(ds, st, x, sx, c.w, c.sw, c.y, c.ydtype, c.M, c.N, c.K, by);
    }
    uint16_t *h = static_cast<uint16_t *>(workspace);
    if (c.xdtype == MX_I8) {
        const size_t n16 = (size_t)c.M * c.K / 16, blocks = (n16 + 255) / 256, most = 8 * (size_t)ds.num_sms;
        e = launch_k(i8_widen_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, st,
                     static_cast<const int8_t *>(c.x), h, n16);
    } else {
        e = c.xdtype == MX_F32 ? run_quantize<float, uint16_t>(ds, st, c.x, h, own_sx, c.M, c.K, true)
                               : run_quantize<uint16_t, uint16_t>(ds, st, c.x, h, own_sx, c.M, c.K, true);
    }
    if (e != cudaSuccess) return e;
    return launch_qmm_i8(ds, st, reinterpret_cast<const uint8_t *>(c.w), c.sw, h, sx, c.y, c.ydtype == MX_F32, c.M, c.N, c.K);
}

}  // namespace mx
