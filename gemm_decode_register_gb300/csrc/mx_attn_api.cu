// mx_attn_api.cu -- the C ABI of the attention-side calls (rotary positions,
// append to the paged cache, attention over it): argument validation.
#include "mx_attn.cuh"

using namespace mx;

namespace {

constexpr int MAX_HEADS = 4096;      // query or cache heads
constexpr int MAX_HEAD_DIM = 256;    // of the cache
constexpr int MAX_SEQUENCES = 1 << 20;
constexpr int MAX_GROUP = 128;       // query heads per cache head

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The cache descriptor by itself.
int check_kv(const mx_paged_kv *kv)
{
    if (!kv || !kv->k || !kv->v || !kv->block_table) return MX_EINVAL;
    if (kv->kv_fmt != MX_KV_BF16 && kv->kv_fmt != MX_KV_MXFP8) return MX_EUNSUPPORTED;
    const bool mx8 = kv->kv_fmt == MX_KV_MXFP8;
    if (kv->num_pages <= 0 || kv->page_size <= 0 || kv->Hkv <= 0 || kv->D <= 0 || kv->table_stride <= 0 ||
        kv->table_pages < 0 || kv->table_pages > kv->table_stride)
        return MX_EINVAL;
    if (kv->page_stride <= 0 || kv->head_stride <= 0 || kv->token_stride <= 0) return MX_EINVAL;
    if (mx8 && (!kv->k_scales || !kv->v_scales || kv->scale_page_stride <= 0 || kv->scale_head_stride <= 0 ||
                kv->scale_token_stride <= 0))
        return MX_EINVAL;
    if (kv->D > MAX_HEAD_DIM || kv->D % (mx8 ? 32 : 8) != 0 || kv->Hkv > MAX_HEADS) return MX_EUNSUPPORTED;
    const int64_t unit = mx8 ? 16 : 8;  // 16 bytes
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || kv->page_stride % unit || kv->head_stride % unit ||
        kv->token_stride % unit || !aligned(kv->block_table, 4))
        return MX_EALIGN;
    return MX_OK;
}

// The descriptor as the kernels take it.
mx_paged_kv filled_in(const mx_paged_kv &kv)
{
    mx_paged_kv d = kv;
    if (d.table_pages == 0) d.table_pages = d.table_stride;
    return d;
}

int check_batch(const int32_t *q_start, const int32_t *kv_len, int T, int B)
{
    if (!q_start || !kv_len || T <= 0 || B <= 0) return MX_EINVAL;
    if (B > MAX_SEQUENCES) return MX_EUNSUPPORTED;
    return aligned(q_start, 4) && aligned(kv_len, 4) ? MX_OK : MX_EALIGN;
}

int finish(cudaError_t e)
{
    if (e == cudaErrorInvalidValue) return MX_EUNSUPPORTED;
    return e == cudaSuccess ? MX_OK : MX_ECUDA;
}

}  // namespace

extern "C" int mx_rope_table(const double *inv_freq, double factor, float *table, int64_t pos0, int n, int half)
{
    if (!inv_freq || !table || pos0 < 0 || n <= 0 || half <= 0) return MX_EINVAL;
    if (!aligned(inv_freq, 8) || !aligned(table, 16)) return MX_EALIGN;
    DeviceState *ds = device_state();
    if (!ds) return MX_ECUDA;
    return finish(launch_rope_table(*ds, current_stream(), inv_freq, factor, table, pos0, n, half));
}

extern "C" int mx_rope(const void *x, void *y, int dtype, const int32_t *positions, const float *table, int table_len,
                       int T, int H, int D, int rot, int64_t x_token_stride, int64_t x_head_stride,
                       int64_t y_token_stride, int64_t y_head_stride, int flags)
{
    if (dtype != MX_BF16 && dtype != MX_F32) return MX_EUNSUPPORTED;
    if (!x || !y || !positions || (rot > 0 && (!table || table_len == 0))) return MX_EINVAL;
    if (T <= 0 || H <= 0 || D <= 0 || rot < 0 || rot > D || rot % 2 != 0 || table_len < 0) return MX_EINVAL;
    if (flags & ~(MX_ROPE_INTERLEAVED | MX_ROPE_INVERSE)) return MX_EINVAL;
    if (x_token_stride < 0 || x_head_stride < 0 || y_token_stride <= 0 || y_head_stride <= 0) return MX_EINVAL;
    const uintptr_t e = dtype == MX_F32 ? 4 : 2;
    if (!aligned(x, e) || !aligned(y, e) || !aligned(positions, 4) || !aligned(table, 16)) return MX_EALIGN;
    DeviceState *ds = device_state();
    if (!ds) return MX_ECUDA;
    return finish(launch_rope(*ds, current_stream(), x, y, dtype, positions, table, table_len, T, H, D, rot,
                              x_token_stride, x_head_stride, y_token_stride, y_head_stride, flags));
}

extern "C" int mx_kv_append(const mx_paged_kv *kv, const void *rows, int dtype, int64_t row_stride,
                            const int32_t *q_start, const int32_t *kv_len, const float *table, int table_len, int rot,
                            void *q, int T, int B, int Hq, int flags)
{
    int s = check_kv(kv);
    if (s == MX_OK) s = check_batch(q_start, kv_len, T, B);
    if (s != MX_OK) return s;
    if (dtype != MX_BF16 && dtype != MX_F32) return MX_EUNSUPPORTED;
    if (!rows || Hq < 0 || (Hq > 0 && !q) || rot < 0 || rot > kv->D || rot % 2 != 0 || table_len < 0 ||
        (rot > 0 && (!table || table_len == 0)) || (flags & ~MX_ROPE_INTERLEAVED))
        return MX_EINVAL;
    if (Hq > MAX_HEADS) return MX_EUNSUPPORTED;
    if (row_stride < (int64_t)(Hq + 2 * kv->Hkv) * kv->D) return MX_EINVAL;
    if (!aligned(rows, 16) || row_stride % (dtype == MX_F32 ? 4 : 8) != 0 || (Hq > 0 && !aligned(q, 16)) ||
        !aligned(table, 16))
        return MX_EALIGN;
    DeviceState *ds = device_state();
    if (!ds) return MX_ECUDA;
    return finish(launch_kv_append(*ds, current_stream(), filled_in(*kv), rows, dtype, row_stride, q_start, kv_len, table,
                                   table_len, rot, static_cast<uint16_t *>(q), T, B, Hq, flags));
}

static bool attn_sizes_ok(int T, int B, int Hq, int Hkv, int D)
{
    return T > 0 && B > 0 && Hq > 0 && Hkv > 0 && D > 0 && Hq % Hkv == 0 && Hq <= MAX_HEADS &&
           Hq / Hkv <= MAX_GROUP && D <= MAX_HEAD_DIM && B <= MAX_SEQUENCES;
}

extern "C" size_t mx_paged_attn_workspace_size(int T, int B, int Hq, int Hkv, int D)
{
    return attn_sizes_ok(T, B, Hq, Hkv, D) ? attn_workspace_bytes(T, B, Hq, Hkv, D) : 0;
}

extern "C" int mx_paged_attn(const mx_paged_kv *kv, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                             const int32_t *q_start, const int32_t *kv_len, float scale, int flags, int window,
                             const float *sinks, void *out, float *lse, int T, int B, int Hq, void *workspace,
                             size_t workspace_bytes)
{
    int s = check_kv(kv);
    if (s == MX_OK) s = check_batch(q_start, kv_len, T, B);
    if (s != MX_OK) return s;
    if (!q || !out || Hq <= 0 || Hq % kv->Hkv != 0 || window < 0 || (flags & ~MX_ATTN_CAUSAL) ||
        !(scale == scale) || q_token_stride <= 0 || q_head_stride <= 0)
        return MX_EINVAL;
    if (!attn_sizes_ok(T, B, Hq, kv->Hkv, kv->D)) return MX_EUNSUPPORTED;
    const size_t need = attn_workspace_bytes(T, B, Hq, kv->Hkv, kv->D);
    if (workspace ? workspace_bytes < need : workspace_bytes != 0 || need > WS_FLOATS * sizeof(float)) return MX_EINVAL;
    if (!aligned(q, 16) || q_token_stride % 8 || q_head_stride % 8 || !aligned(out, 16) || !aligned(workspace, 256) ||
        !aligned(lse, 4) || !aligned(sinks, 4))
        return MX_EALIGN;
    DeviceState *ds = device_state();
    if (!ds) return MX_ECUDA;
    AttnArgs a;
    a.kv = filled_in(*kv);
    a.q = static_cast<const uint16_t *>(q);
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.causal = (flags & MX_ATTN_CAUSAL) != 0;
    a.window = window;
    a.sinks = sinks;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.g = Hq / kv->Hkv;
    a.workspace = workspace;
    a.err = ds->err;
    DeviceState v = *ds;  // the slot's counters, for items cut across CTAs, and its sums' space
    if (!attach_stream_workspace(v, current_stream())) return MX_ECUDA;
    if (!workspace) a.workspace = v.ws;
    return finish(launch_paged_attn(v, current_stream(), a));
}
