// mx_attn.cu -- attention of new tokens over the paged cache, direct loads:
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),
//   s_j = q . k_j * scale * log2(e),  m = the largest s_j so far,
//
// in one pass over the keys; when m grows by d the sums so far shrink by
// 2^-d.  One CTA takes one query head of one token, its warps take the
// context's groups of 32 keys in turn.
//
// For what the tensor-core kernel cannot take (attn_tc_ok: other head sizes,
// pages that its copies cannot tile, scales of zero or less).  Bound by its loads:
// every query head reads the cache again, and by single keys.  64 heads on 8 x
// 128 bf16, pages of 48 against pages of 64 on the tensor cores: one token on 16
// keys 10.3 us, 8.5; 16 tokens on 2048 559 us, 33; a prompt of 512 on 1024
// 3168 us, 23.  The weights stay fp32.
#include "mx_attn.cuh"

namespace mx {

constexpr int DIRECT_WARPS = 4;

// (eight blocks per SM: the second pass's registers would leave seven, 3464 us for the
// prompt above)
template <int KVF>
__global__ void __launch_bounds__(DIRECT_WARPS * 32, 8) attn_direct_kernel(AttnArgs a)
{
    __shared__ float q[MAX_D];
    __shared__ float part_m[DIRECT_WARPS], part_l[DIRECT_WARPS], part_o[DIRECT_WARPS][MAX_D];
    __shared__ int missing;
    pdl_trigger();
    const int t = blockIdx.x / a.Hq, h = blockIdx.x - t * a.Hq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = sequence_of(a.q_start, a.B, t);
    if (b < 0) {
        // all rows may belong to no sequence: the grid must not end before the kernel before it has
        pdl_wait();
        return;
    }
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
                                   lo, hi, (lo & ~31ll) + 32 * warp, DIRECT_WARPS, r);
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
    float check = 0.0f;
    for (int d = threadIdx.x; d < a.kv.D; d += blockDim.x) {
        float o = 0.0f;
#pragma unroll
        for (int w = 0; w < DIRECT_WARPS; ++w) o = fmaf(part_o[w][d], f[w], o);
        check += o * 0.0f;
        o = bad ? __uint_as_float(0x7FC00000u) : o * inv;
        a.out[row * a.kv.D + d] = (uint16_t)(f32x2_to_bf16x2(o, 0.0f) & 0xFFFFu);
    }
    // Values near the type's largest can overflow sums that are divided only at the
    // end: a second pass with the weights divided first, in the rare case that one is not finite.
    if (__syncthreads_or(!bad && inv == inv && check != 0.0f)) {
        RowState again;
        again.m = base;
        row_keys<KVF, true>(a.kv, a.kv.block_table + (size_t)b * a.kv.table_stride, h / a.g, q, a.scale_log2, lo, hi,
                            (lo & ~31ll) + 32 * warp, DIRECT_WARPS, again, inv);
#pragma unroll
        for (int i = 0; i < MAX_D / 32; ++i) part_o[warp][2 * lane + 64 * (i / 2) + i % 2] = again.o[i];
        __syncthreads();
        for (int d = threadIdx.x; d < a.kv.D; d += blockDim.x) {
            float o = 0.0f;
#pragma unroll
            for (int w = 0; w < DIRECT_WARPS; ++w) o += part_o[w][d];
            a.out[row * a.kv.D + d] = (uint16_t)(f32x2_to_bf16x2(o, 0.0f) & 0xFFFFu);
        }
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[row] = bad ? __uint_as_float(0x7FC00000u) : (base + log2f(l)) * 0.6931471805599453f;
}

size_t attn_workspace_bytes(int T, int, int Hq, int Hkv, int D) { return attn_tc_workspace_bytes(T, Hq, Hkv, D); }

cudaError_t launch_paged_attn(const DeviceState &ds, cudaStream_t st, const AttnArgs &a)
{
    if (attn_tc_ok(a)) return launch_attn_tc(ds, st, a);
    const long long blocks = (long long)a.T * a.Hq;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(DIRECT_WARPS * 32);
    if (a.kv.kv_fmt == KV_MXFP8) return launch_k(attn_direct_kernel<KV_MXFP8>, grid, block, 0, st, a);
    return launch_k(attn_direct_kernel<KV_BF16>, grid, block, 0, st, a);
}

}  // namespace mx
