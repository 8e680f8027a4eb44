// mx_attn.cu -- attention of new tokens over the paged cache, direct loads:
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),
//   s_j = q . k_j * scale * log2(e),  m = the largest s_j so far,
//
// in one pass over the keys; when m grows by d the sums so far shrink by
// 2^-d.  One CTA takes one query head of one token, its warps take the
// context's groups of 32 keys in turn.
#include "mx_attn.cuh"

namespace mx {

constexpr int DIRECT_WARPS = 4;
constexpr int MAX_D = 256;

// Running softmax of one row: the sums belong to the maximum m (log2 units);
// lane l holds dimensions 2 l + 64 i and the one after.
struct RowState {
    float m = -INFINITY, l = 0.0f;
    float o[MAX_D / 32] = {};
};

// One key's product with the row q (fp32, shared memory).
template <int KVF>
__device__ __forceinline__ float key_dot(const mx_paged_kv &kv, const float *q, long long at, long long sat)
{
    float acc = 0.0f;
    if constexpr (KVF == KV_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(kv.k) + at;
        for (int d = 0; d < kv.D; d += 8) {
            const uint4 r = *reinterpret_cast<const uint4 *>(p + d);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc = fmaf(q[d + 2 * i], bf16_lo(w[i]), acc);
                acc = fmaf(q[d + 2 * i + 1], bf16_hi(w[i]), acc);
            }
        }
    } else {
        const uint8_t *p = static_cast<const uint8_t *>(kv.k) + at;
        const uint8_t *sc = static_cast<const uint8_t *>(kv.k_scales) + sat;
        for (int d = 0; d < kv.D; d += 32) {
            float part = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; j += 16) {
                const uint4 r = *reinterpret_cast<const uint4 *>(p + d + j);
                const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t h0, h1;
                    e4m3x4_to_f16x2(w[i], h0, h1);
                    const float *qq = q + d + j + 4 * i;
                    part = fmaf(qq[0], f16_lo_to_f32(h0), part);
                    part = fmaf(qq[1], f16_hi_to_f32(h0), part);
                    part = fmaf(qq[2], f16_lo_to_f32(h1), part);
                    part = fmaf(qq[3], f16_hi_to_f32(h1), part);
                }
            }
            acc = fmaf(part, e8m0_to_f32(sc[d / 32]), acc);
        }
    }
    return acc;
}

// Adds keys first, first + 32 step, ... (32 at a time) below hi to the row;
// keys below lo are skipped.  false if a page is missing.
template <int KVF>
__device__ bool row_keys(const mx_paged_kv &kv, const int32_t *table, int kvh, const float *q, float scale_log2,
                         int lo, int hi, int first, int step, RowState &r)
{
    const int lane = threadIdx.x & 31;
    bool all = true;
    for (long long k0 = first; k0 < hi; k0 += 32ll * step) {
        const long long key = k0 + lane;
        bool seen = key >= lo && key < hi;
        long long at = 0, sat = 0;
        float s = -INFINITY;
        if (seen) {
            const int pi = (int)key / kv.page_size, slot = (int)key - pi * kv.page_size;
            const int page = page_of(kv, table, pi);
            if (page < 0) {
                seen = all = false;
            } else {
                at = page * kv.page_stride + kvh * kv.head_stride + slot * kv.token_stride;
                sat = page * kv.scale_page_stride + kvh * kv.scale_head_stride + slot * kv.scale_token_stride;
                s = key_dot<KVF>(kv, q, at, sat) * scale_log2;
            }
        }
        const unsigned mask = __ballot_sync(0xFFFFFFFFu, seen);
        float top = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const float m = fmaxf(r.m, top);
        // nothing seen yet, or only scores of -infinity: their weights are zero, unless one is NaN
        const float base = m == -INFINITY ? 0.0f : m;
        const float p = seen ? exp2f(s - base) : 0.0f;
        const float shrink = exp2f(r.m - base);
        r.m = m;
        float sum = p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        r.l = fmaf(r.l, shrink, sum);
#pragma unroll
        for (int i = 0; i < MAX_D / 32; ++i) r.o[i] *= shrink;
        for (unsigned left = mask; left != 0; left &= left - 1) {
            const int src = __ffs(left) - 1;
            const float pj = __shfl_sync(0xFFFFFFFFu, p, src);
            const long long vat = __shfl_sync(0xFFFFFFFFu, at, src);
            const long long vsat = __shfl_sync(0xFFFFFFFFu, sat, src);
#pragma unroll
            for (int i = 0; i < MAX_D / 64; ++i) {
                const int d = 2 * lane + 64 * i;
                if (d >= kv.D) break;
                if constexpr (KVF == KV_BF16) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(kv.v) + vat + d);
                    r.o[2 * i] = fmaf(pj, bf16_lo(w), r.o[2 * i]);
                    r.o[2 * i + 1] = fmaf(pj, bf16_hi(w), r.o[2 * i + 1]);
                } else {
                    const uint32_t w = *reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(kv.v) + vat + d);
                    const float sc = e8m0_to_f32(static_cast<const uint8_t *>(kv.v_scales)[vsat + d / 32]);
                    const uint32_t h2 = e4m3x2_to_f16x2(w);
                    r.o[2 * i] = fmaf(pj, f16_lo_to_f32(h2) * sc, r.o[2 * i]);
                    r.o[2 * i + 1] = fmaf(pj, f16_hi_to_f32(h2) * sc, r.o[2 * i + 1]);
                }
            }
        }
    }
    return all;
}

template <int KVF>
__global__ void __launch_bounds__(DIRECT_WARPS * 32) attn_direct_kernel(AttnArgs a)
{
    __shared__ float q[MAX_D];
    __shared__ float part_m[DIRECT_WARPS], part_l[DIRECT_WARPS], part_o[DIRECT_WARPS][MAX_D];
    __shared__ int missing;
    pdl_trigger();
    const int t = blockIdx.x / a.Hq, h = blockIdx.x - t * a.Hq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = sequence_of(a.q_start, a.B, t);
    if (b < 0) return;
    const int end = __ldg(a.q_start + b + 1), len = __ldg(a.kv_len + b);
    const long long pos = (long long)len - end + t;
    const int hi = a.causal ? (int)(pos + 1 < len ? pos + 1 : len) : len;
    const int lo = a.window > 0 && pos - a.window + 1 > 0 ? (int)(pos - a.window + 1) : 0;
    if (threadIdx.x == 0) missing = 0;
    pdl_wait();
    for (int d = threadIdx.x; d < a.kv.D; d += blockDim.x)
        q[d] = bf16_to_f32(a.q[t * a.q_token_stride + h * a.q_head_stride + d]);
    __syncthreads();
    RowState r;
    const bool all = row_keys<KVF>(a.kv, a.kv.block_table + (size_t)b * a.kv.table_stride, h / a.g, q, a.scale_log2,
                                   lo, hi, (lo & ~31) + 32 * warp, DIRECT_WARPS, r);
    if (!all) missing = 1;
    if (lane == 0) {
        part_m[warp] = r.m;
        part_l[warp] = r.l;
    }
#pragma unroll
    for (int i = 0; i < MAX_D / 32; ++i) part_o[warp][2 * lane + 64 * (i / 2) + i % 2] = r.o[i];
    __syncthreads();
    const float sink = a.sinks ? __ldg(a.sinks + h) * 1.4426950408889634f : -INFINITY;
    float m = sink;
#pragma unroll
    for (int w = 0; w < DIRECT_WARPS; ++w) m = fmaxf(m, part_m[w]);
    const float base = m == -INFINITY ? 0.0f : m;
    float f[DIRECT_WARPS], l = a.sinks ? exp2f(sink - base) : 0.0f;
#pragma unroll
    for (int w = 0; w < DIRECT_WARPS; ++w) {
        f[w] = exp2f(part_m[w] - base);
        l = fmaf(part_l[w], f[w], l);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const bool bad = missing != 0;
    if (bad && threadIdx.x == 0) set_device_error(a.err, DEVERR_BAD_PAGE);
    const size_t row = (size_t)t * a.Hq + h;
    for (int d = threadIdx.x; d < a.kv.D; d += blockDim.x) {
        float o = 0.0f;
#pragma unroll
        for (int w = 0; w < DIRECT_WARPS; ++w) o = fmaf(part_o[w][d], f[w], o);
        o = bad ? __uint_as_float(0x7FC00000u) : o * inv;
        a.out[row * a.kv.D + d] = (uint16_t)(f32x2_to_bf16x2(o, 0.0f) & 0xFFFFu);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[row] = bad ? __uint_as_float(0x7FC00000u) : (base + log2f(l)) * 0.6931471805599453f;
}

size_t attn_workspace_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_paged_attn(const DeviceState &ds, cudaStream_t st, const AttnArgs &a)
{
    const long long blocks = (long long)a.T * a.Hq;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(DIRECT_WARPS * 32);
    if (a.kv.kv_fmt == KV_MXFP8) return launch_k(attn_direct_kernel<KV_MXFP8>, grid, block, 0, st, a);
    return launch_k(attn_direct_kernel<KV_BF16>, grid, block, 0, st, a);
}

}  // namespace mx
