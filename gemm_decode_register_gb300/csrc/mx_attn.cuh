// mx_attn.cuh -- shared by the attention-side kernels (rotary positions,
// append to the paged cache, attention over it): the cache's layout on the
// device, the search for a token's sequence, and the launchers.
#pragma once

#include "../../include/mx.h"
#include "mx_common.cuh"
#include "mx_internal.h"

namespace mx {

enum : int { KV_BF16 = MX_KV_BF16, KV_MXFP8 = MX_KV_MXFP8 };

// The sequence that new token t belongs to, found by the whole warp: the last
// b with q_start[b] <= t, 32 candidates per round of one load per lane (two
// rounds up to 1024 sequences).  -1 if t belongs to none.
__device__ __forceinline__ int sequence_of(const int32_t *q_start, int B, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;
    for (;;) {
        const int step = (n + 31) >> 5;
        const int i = lane * step;
        const unsigned le = __ballot_sync(0xFFFFFFFFu, i < n && __ldg(q_start + lo + i) <= t);
        if (le == 0) return -1;
        const int c = 31 - __clz(le);
        lo += c * step;
        n = min(step, n - c * step);
        if (step == 1) break;
    }
    return t < __ldg(q_start + lo + 1) ? lo : -1;
}

// Page of position `pos` (>= 0) of a sequence, -1 if it has none.
__device__ __forceinline__ int page_of(const mx_paged_kv &kv, const int32_t *row, int page_index)
{
    if (page_index >= kv.table_pages) return -1;
    const int p = __ldg(row + page_index);
    return (unsigned)p < (unsigned)kv.num_pages ? p : -1;
}

constexpr int MAX_D = 256;  // largest head

// Running softmax of one row: the sums belong to the maximum m (log2 units);
// lane l holds dimensions 2 l + 64 i and the one after.
struct RowState {
    float m = -INFINITY, l = 0.0f;
    float o[MAX_D / 32] = {};
};

// A query's elements: fp32 (shared memory) or bf16.
__device__ __forceinline__ float q_at(const float *q, int d) { return q[d]; }
__device__ __forceinline__ float q_at(const uint16_t *q, int d) { return bf16_to_f32(q[d]); }

// One key's product with the row q.
template <int KVF, typename Q>
__device__ __forceinline__ float key_dot(const mx_paged_kv &kv, const Q *q, long long at, long long sat)
{
    float acc = 0.0f;
    if constexpr (KVF == KV_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(kv.k) + at;
        for (int d = 0; d < kv.D; d += 8) {
            const uint4 r = *reinterpret_cast<const uint4 *>(p + d);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc = fmaf(q_at(q, d + 2 * i), bf16_lo(w[i]), acc);
                acc = fmaf(q_at(q, d + 2 * i + 1), bf16_hi(w[i]), acc);
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
                    const Q *qq = q + d + j + 4 * i;
                    part = fmaf(q_at(qq, 0), f16_lo_to_f32(h0), part);
                    part = fmaf(q_at(qq, 1), f16_hi_to_f32(h0), part);
                    part = fmaf(q_at(qq, 2), f16_lo_to_f32(h1), part);
                    part = fmaf(q_at(qq, 3), f16_hi_to_f32(h1), part);
                }
            }
            acc = fmaf(part, e8m0_to_f32(sc[d / 32]), acc);
        }
    }
    return acc;
}

// Two neighbouring elements of a value as they lie in the cache, and as fp32.
template <int KVF>
struct RawPair {
    uint32_t w, e;
    __device__ __forceinline__ void load(const mx_paged_kv &kv, long long at, long long sat, int d)
    {
        if constexpr (KVF == KV_BF16) {
            w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(kv.v) + at + d);
        } else {
            w = *reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(kv.v) + at + d);
            e = static_cast<const uint8_t *>(kv.v_scales)[sat + d / 32];
        }
    }
    __device__ __forceinline__ float2 get() const
    {
        if constexpr (KVF == KV_BF16) return make_float2(bf16_lo(w), bf16_hi(w));
        const float sc = e8m0_to_f32(e);
        const uint32_t h2 = e4m3x2_to_f16x2(w);
        return make_float2(f16_lo_to_f32(h2) * sc, f16_hi_to_f32(h2) * sc);
    }
};

// o += p v of one key; lane l holds dimensions 2 l + 64 i and the one after.
template <int KVF>
__device__ __forceinline__ void add_value(const mx_paged_kv &kv, long long at, long long sat, float p,
                                          float (&o)[MAX_D / 32])
{
#pragma unroll
    for (int i = 0; i < MAX_D / 64; ++i) {
        const int d = 2 * (threadIdx.x & 31) + 64 * i;
        if (d >= kv.D) break;
        RawPair<KVF> r;
        r.load(kv, at, sat, d);
        const float2 v = r.get();
        o[2 * i] = fmaf(p, v.x, o[2 * i]);
        o[2 * i + 1] = fmaf(p, v.y, o[2 * i + 1]);
    }
}

// Adds keys first, first + 32 step, ... (32 at a time) below hi to the row;
// keys below lo are skipped.  false if a page is missing.  FIXED: against the
// row's final maximum r.m, each weight times 1 / sum (`inv`) before it is used; only r.o is added to.
template <int KVF, bool FIXED = false>
__device__ bool row_keys(const mx_paged_kv &kv, const int32_t *table, int kvh, const float *q, float scale_log2,
                         int lo, int hi, long long first, int step, RowState &r, float inv = 1.0f)
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
        float p;
        if constexpr (FIXED) {
            p = seen ? exp2f(s - r.m) * inv : 0.0f;
        } else {
            float top = s;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const float m = fmaxf(r.m, top);
            // nothing seen yet, or only scores of -infinity: their weights are zero, unless one is NaN
            const float base = m == -INFINITY ? 0.0f : m;
            p = seen ? exp2f(s - base) : 0.0f;
            const float shrink = exp2f(r.m - base);
            r.m = m;
            float sum = p;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            r.l = fmaf(r.l, shrink, sum);
#pragma unroll
            for (int i = 0; i < MAX_D / 32; ++i) r.o[i] *= shrink;
        }
        for (unsigned left = mask; left != 0; left &= left - 1) {
            const int src = __ffs(left) - 1;
            const float pj = __shfl_sync(0xFFFFFFFFu, p, src);
            const long long vat = __shfl_sync(0xFFFFFFFFu, at, src);
            const long long vsat = __shfl_sync(0xFFFFFFFFu, sat, src);
            add_value<KVF>(kv, vat, vsat, pj, r.o);
        }
    }
    return all;
}

// mx_rope.cu
cudaError_t launch_rope_table(const DeviceState &ds, cudaStream_t st, const double *inv_freq, double factor,
                              float *table, int64_t pos0, int n, int half);
cudaError_t launch_rope(const DeviceState &ds, cudaStream_t st, const void *x, void *y, int dtype,
                        const int32_t *positions, const float *table, int table_len, int T, int H, int D, int rot,
                        int64_t xt, int64_t xh, int64_t yt, int64_t yh, int flags);
cudaError_t launch_kv_append(const DeviceState &ds, cudaStream_t st, const mx_paged_kv &kv, const void *rows,
                             int dtype, int64_t row_stride, const int32_t *q_start, const int32_t *kv_len,
                             const float *table, int table_len, int rot, uint16_t *q, int T, int B, int Hq, int flags);

// A call of mx_paged_attn on the device.
struct AttnArgs {
    mx_paged_kv kv;
    const uint16_t *q;
    int64_t q_token_stride, q_head_stride;
    const int32_t *q_start, *kv_len;
    float scale_log2;  // scale * log2(e): the softmax runs on powers of two
    int causal, window;
    const float *sinks;
    uint16_t *out;
    float *lse;
    int T, B, Hq, g;  // g: query heads per cache head
    void *workspace;
    int *err;
};

size_t attn_workspace_bytes(int T, int B, int Hq, int Hkv, int D);
cudaError_t launch_paged_attn(const DeviceState &ds, cudaStream_t st, const AttnArgs &a);

// mx_attn_tc.cu: the tensor-core kernel, and whether it takes a call.
size_t attn_tc_workspace_bytes(int T, int Hq, int Hkv, int D);
bool attn_tc_ok(const AttnArgs &a);
cudaError_t launch_attn_tc(const DeviceState &ds, cudaStream_t st, const AttnArgs &a);

}  // namespace mx
