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
    if (page_index >= kv.table_stride) return -1;
    const int p = __ldg(row + page_index);
    return (unsigned)p < (unsigned)kv.num_pages ? p : -1;
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

}  // namespace mx
