// mx_serve.h -- host-side declarations of the decode loop's calls (beam
// selection, page pool, 8-bit integer products).  Not part of the ABI.
#pragma once

#include "../../include/mx.h"
#include "mx_internal.h"

namespace mx {

// Limits checked on the host.
constexpr int BEAM_MAX_W = 64;       // beams of a batch entry
constexpr int BEAM_MAX_K = 128;      // candidates of a batch entry
constexpr int BEAM_MAX_V = 1 << 20;  // vocabulary
constexpr int BEAM_MAX_B = WS_COUNTERS;
constexpr int BEAM_MAX_ROWS = 65535;  // B * W (all rows' steps are counted in an int)

struct BeamCall {
    const void *logits;
    int dtype;
    int64_t row_stride;
    const float *scores;
    const uint32_t *mask;
    int64_t mask_stride;
    int B, W, V, k, eos;
    float *score, *next_score;
    int32_t *parent, *token, *next_parent, *next_token;
};
size_t beam_workspace_bytes(int B, int W, int V, int k);
cudaError_t launch_beam_select(const DeviceState &ds, cudaStream_t st, const BeamCall &c, void *workspace);

// The page pool.
constexpr int POOL_MAX_SLOTS = 4096;      // sequences of a table
constexpr int POOL_MAX_PAGES = 1 << 24;   // pages
constexpr int COPY_MAX_LAYERS = 256;      // caches of one copy call

struct RemapCall {
    mx_page_pool pool;
    int page_size;
    const int32_t *table_in, *kv_len_in;
    int32_t *table_out, *kv_len_out;
    int in_stride, in_pages, S_in, out_stride, out_pages, S_out;
    const int32_t *parent, *keep, *add;
    int add_all;
    int32_t *copies;
};
size_t pool_work_bytes(int num_pages);
cudaError_t launch_kv_remap(const DeviceState &ds, cudaStream_t st, const RemapCall &c);
cudaError_t launch_kv_compact(const DeviceState &ds, cudaStream_t st, const mx_page_pool &pool, int page_size,
                              int32_t *table, int stride, int pages, const int32_t *kv_len, int S, int32_t *copies);
cudaError_t launch_kv_copy_pages(const DeviceState &ds, cudaStream_t st, const mx_paged_kv *kv, int layers,
                                 const int32_t *copies, int max_copies);

// 8-bit integer products.
constexpr int I8_MAX_K = 131056;  // 2^14 K stays below 2^31

struct I8Call {
    const void *x;
    int xdtype;
    const float *sx;  // MX_I8 only
    const int8_t *w;
    const float *sw;
    void *y;
    int ydtype, M, N, K;
};
size_t i8_mm_workspace_bytes(int M, int K);
cudaError_t launch_i8_quantize(const DeviceState &ds, cudaStream_t st, const void *x, int dtype, int8_t *q, float *scales,
                               int M, int K, bool early);
cudaError_t launch_i8_mm(const DeviceState &ds, cudaStream_t st, const I8Call &c, void *workspace);
// mx_qmm.cu: X f16 integers, y = (X W^T) xscale wscale; its time in us, by
// measurements on GB300 (for each 64 elements of K of a round of tiles, one tile
// per pair of SMs)
double qmm_i8_estimate(const DeviceState &ds, int M, int N, int K);
cudaError_t launch_qmm_i8(const DeviceState &ds, cudaStream_t st, const uint8_t *w, const float *wscale,
                          const uint16_t *X, const float *xscale, void *Y, bool yf32, int M, int N, int K);

}  // namespace mx
