// mx_serve_api.cu -- the C ABI of the decode loop's calls (beam selection, page
// pool, page copies) and of the 8-bit integer products: argument validation.
#include "mx_serve.h"

using namespace mx;

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int finish(cudaError_t e)
{
    if (e == cudaErrorInvalidValue) return MX_EUNSUPPORTED;
    return e == cudaSuccess ? MX_OK : MX_ECUDA;
}

bool beam_sizes_ok(int B, int W, int V, int k)
{
    return B > 0 && W > 0 && V > 0 && k > 0 && B <= BEAM_MAX_B && W <= BEAM_MAX_W && V <= BEAM_MAX_V && k <= BEAM_MAX_K &&
           (long long)B * W <= BEAM_MAX_ROWS;
}

int check_pool(const mx_page_pool *p)
{
    if (!p || !p->count || !p->refs || !p->free_pages || !p->work || p->num_pages <= 0) return MX_EINVAL;
    if (p->num_pages > POOL_MAX_PAGES) return MX_EUNSUPPORTED;
    if (!aligned(p->count, 4) || !aligned(p->refs, 4) || !aligned(p->free_pages, 4) || !aligned(p->work, 256)) return MX_EALIGN;
    return MX_OK;
}

int check_table(const int32_t *table, int stride, int pages, const int32_t *kv_len, int S)
{
    if (!table || !kv_len || S <= 0 || pages <= 0 || (S > 1 && stride < pages)) return MX_EINVAL;
    if (S > POOL_MAX_SLOTS) return MX_EUNSUPPORTED;
    return aligned(table, 4) && aligned(kv_len, 4) ? MX_OK : MX_EALIGN;
}

// [a, a + n) and [b, b + m) in bytes.
bool overlap(const void *a, size_t n, const void *b, size_t m)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + m && y < x + n;
}

size_t table_bytes(int stride, int pages, int S) { return 4 * ((size_t)(S - 1) * (size_t)(S > 1 ? stride : 0) + (size_t)pages); }

// A cache as the copies use it (mx_kv_append and mx_paged_attn check the rest).
int check_cache(const mx_paged_kv &kv)
{
    if (!kv.k || !kv.v) return MX_EINVAL;
    if (kv.kv_fmt != MX_KV_BF16 && kv.kv_fmt != MX_KV_MXFP8) return MX_EUNSUPPORTED;
    const bool mx8 = kv.kv_fmt == MX_KV_MXFP8;
    if (kv.num_pages <= 0 || kv.page_size <= 0 || kv.Hkv <= 0 || kv.D <= 0) return MX_EINVAL;
    if (kv.page_stride <= 0 || kv.head_stride <= 0 || kv.token_stride <= 0) return MX_EINVAL;
    if (mx8 && (!kv.k_scales || !kv.v_scales || kv.scale_page_stride <= 0 || kv.scale_head_stride <= 0 ||
                kv.scale_token_stride <= 0))
        return MX_EINVAL;
    if (kv.D > 256 || kv.D % (mx8 ? 32 : 8) != 0 || kv.Hkv > 4096 || (long long)kv.Hkv * kv.page_size > (1ll << 24))
        return MX_EUNSUPPORTED;
    const int64_t unit = mx8 ? 16 : 8;  // 16 bytes
    if (!aligned(kv.k, 16) || !aligned(kv.v, 16) || kv.page_stride % unit || kv.head_stride % unit || kv.token_stride % unit)
        return MX_EALIGN;
    return MX_OK;
}

bool same_shape(const mx_paged_kv &a, const mx_paged_kv &b)
{
    return a.kv_fmt == b.kv_fmt && a.num_pages == b.num_pages && a.page_size == b.page_size && a.Hkv == b.Hkv && a.D == b.D &&
           a.page_stride == b.page_stride && a.head_stride == b.head_stride && a.token_stride == b.token_stride &&
           a.scale_page_stride == b.scale_page_stride && a.scale_head_stride == b.scale_head_stride &&
           a.scale_token_stride == b.scale_token_stride;
}

}  // namespace

extern "C" size_t mx_beam_select_workspace_size(int B, int W, int V, int k)
{
    return beam_sizes_ok(B, W, V, k) ? beam_workspace_bytes(B, W, V, k) : 0;
}

extern "C" int mx_beam_select(const void *logits, int dtype, int64_t row_stride, const float *scores, const uint32_t *mask,
                              int64_t mask_stride, int B, int W, int V, int k, int eos, float *cand_score,
                              int32_t *cand_parent, int32_t *cand_token, float *next_score, int32_t *next_parent,
                              int32_t *next_token, void *workspace, size_t workspace_bytes)
{
    if (dtype != MX_BF16 && dtype != MX_F32) return MX_EUNSUPPORTED;
    if (!logits || !scores || !cand_score || !cand_parent || !cand_token || B <= 0 || W <= 0 || V <= 0 || k <= 0)
        return MX_EINVAL;
    if ((next_score != nullptr) != (next_parent != nullptr) || (next_score != nullptr) != (next_token != nullptr))
        return MX_EINVAL;
    if (!beam_sizes_ok(B, W, V, k)) return MX_EUNSUPPORTED;
    if (((long long)B * W > 1 && row_stride < V) || (mask && (long long)B * W > 1 && mask_stride < (V + 31) / 32))
        return MX_EINVAL;
    const size_t need = beam_workspace_bytes(B, W, V, k);
    if (workspace ? workspace_bytes < need : workspace_bytes != 0 || need > WS_FLOATS * sizeof(float)) return MX_EINVAL;
    if (!aligned(logits, dtype == MX_F32 ? 4 : 2) || !aligned(scores, 4) || !aligned(mask, 4) || !aligned(cand_score, 4) ||
        !aligned(cand_parent, 4) || !aligned(cand_token, 4) || !aligned(next_score, 4) || !aligned(next_parent, 4) ||
        !aligned(next_token, 4) || !aligned(workspace, 256))
        return MX_EALIGN;
    DeviceState *ds = device_state();
    if (!ds) return MX_ECUDA;
    DeviceState v = *ds;  // the slot's counters, and its space for the pieces' lists
    if (!attach_stream_workspace(v, current_stream())) return MX_ECUDA;
    BeamCall c;
    c.logits = logits;
    c.dtype = dtype;
    c.row_stride = row_stride;
    c.scores = scores;
    c.mask = mask;
    c.mask_stride = mask_stride;
    c.B = B;
    c.W = W;
    c.V = V;
    c.k = k;
    c.eos = eos < 0 ? -1 : eos;
    c.score = cand_score;
    c.parent = cand_parent;
    c.token = cand_token;
    c.next_score = next_score;
    c.next_parent = next_parent;
    c.next_token = next_token;
    return finish(launch_beam_select(v, current_stream(), c, workspace ? workspace : v.ws));
}

extern "C" size_t mx_page_pool_work_size(int num_pages)
{
    return num_pages > 0 && num_pages <= POOL_MAX_PAGES ? pool_work_bytes(num_pages) : 0;
}

extern "C" int mx_kv_remap(const mx_page_pool *pool, int page_size, const int32_t *table_in, int in_stride, int in_pages,
                           const int32_t *kv_len_in, int S_in, int32_t *table_out, int out_stride, int out_pages,
                           int32_t *kv_len_out, int S_out, const int32_t *parent, const int32_t *keep, const int32_t *add,
                           int add_all, int32_t *copies)
{
    int s = check_pool(pool);
    if (s == MX_OK) s = check_table(table_in, in_stride, in_pages, kv_len_in, S_in);
    if (s == MX_OK) s = check_table(table_out, out_stride, out_pages, kv_len_out, S_out);
    if (s != MX_OK) return s;
    if (page_size <= 0 || !parent || !copies || add_all < 0) return MX_EINVAL;
    if (overlap(table_in, table_bytes(in_stride, in_pages, S_in), table_out, table_bytes(out_stride, out_pages, S_out)) ||
        overlap(kv_len_in, 4 * (size_t)S_in, kv_len_out, 4 * (size_t)S_out))
        return MX_EINVAL;
    if (!aligned(parent, 4) || !aligned(keep, 4) || !aligned(add, 4) || !aligned(copies, 16)) return MX_EALIGN;
    DeviceState *ds = device_state();
    if (!ds) return MX_ECUDA;
    RemapCall c;
    c.pool = *pool;
    c.page_size = page_size;
    c.table_in = table_in;
    c.kv_len_in = kv_len_in;
    c.table_out = table_out;
    c.kv_len_out = kv_len_out;
    c.in_stride = in_stride;
    c.in_pages = in_pages;
    c.S_in = S_in;
    c.out_stride = out_stride;
    c.out_pages = out_pages;
    c.S_out = S_out;
    c.parent = parent;
    c.keep = keep;
    c.add = add;
    c.add_all = add_all;
    c.copies = copies;
    return finish(launch_kv_remap(*ds, current_stream(), c));
}

extern "C" int mx_kv_compact(const mx_page_pool *pool, int page_size, int32_t *table, int stride, int pages,
                             const int32_t *kv_len, int S, int32_t *copies)
{
    int s = check_pool(pool);
    if (s == MX_OK) s = check_table(table, stride, pages, kv_len, S);
    if (s != MX_OK) return s;
    if (page_size <= 0 || !copies) return MX_EINVAL;
    if (!aligned(copies, 16)) return MX_EALIGN;
    DeviceState *ds = device_state();
    if (!ds) return MX_ECUDA;
    return finish(launch_kv_compact(*ds, current_stream(), *pool, page_size, table, stride, pages, kv_len, S, copies));
}

extern "C" int mx_kv_copy_pages(const mx_paged_kv *kv, int layers, const int32_t *copies, int max_copies)
{
    if (!kv || !copies || layers <= 0 || max_copies <= 0) return MX_EINVAL;
    if (layers > COPY_MAX_LAYERS || max_copies > POOL_MAX_PAGES) return MX_EUNSUPPORTED;
    for (int l = 0; l < layers; ++l) {
        const int s = check_cache(kv[l]);
        if (s != MX_OK) return s;
        if (l > 0 && !same_shape(kv[0], kv[l])) return MX_EINVAL;
    }
    if (!aligned(copies, 16)) return MX_EALIGN;
    DeviceState *ds = device_state();
    if (!ds) return MX_ECUDA;
    return finish(launch_kv_copy_pages(*ds, current_stream(), kv, layers, copies, max_copies));
}

extern "C" int mx_i8_quantize(const void *x, int dtype, int8_t *q, float *scales, int M, int K)
{
    if (dtype != MX_BF16 && dtype != MX_F32) return MX_EUNSUPPORTED;
    if (!x || !q || !scales || M <= 0 || K <= 0 || K % 16 != 0) return MX_EINVAL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 4)) return MX_EALIGN;
    DeviceState *ds = device_state();
    if (!ds) return MX_ECUDA;
    return finish(launch_i8_quantize(*ds, current_stream(), x, dtype, q, scales, M, K, false));
}

extern "C" size_t mx_i8_mm_workspace_size(int M, int K)
{
    return M > 0 && K > 0 && K % 16 == 0 && K <= I8_MAX_K ? i8_mm_workspace_bytes(M, K) : 0;
}

extern "C" int mx_i8_mm(const void *x, int xdtype, const float *x_scales, const int8_t *w, const float *w_scales, void *y,
                        int ydtype, int M, int N, int K, void *workspace, size_t workspace_bytes)
{
    if ((xdtype != MX_BF16 && xdtype != MX_F32 && xdtype != MX_I8) || (ydtype != MX_BF16 && ydtype != MX_F32))
        return MX_EUNSUPPORTED;
    if (!x || !w || !w_scales || !y || (xdtype == MX_I8) != (x_scales != nullptr) || M <= 0 || N <= 0 || K <= 0 || K % 16 != 0)
        return MX_EINVAL;
    if (K > I8_MAX_K) return MX_EUNSUPPORTED;
    const size_t need = i8_mm_workspace_bytes(M, K);
    if (workspace ? workspace_bytes < need : workspace_bytes != 0 || need > WS_FLOATS * sizeof(float)) return MX_EINVAL;
    if (!aligned(x, 16) || !aligned(x_scales, 4) || !aligned(w, 16) || !aligned(w_scales, 4) || !aligned(y, 16) ||
        !aligned(workspace, 256))
        return MX_EALIGN;
    DeviceState *ds = device_state();
    if (!ds) return MX_ECUDA;
    DeviceState v = *ds;
    if (!workspace && !attach_stream_workspace(v, current_stream())) return MX_ECUDA;
    I8Call c;
    c.x = x;
    c.xdtype = xdtype;
    c.sx = x_scales;
    c.w = w;
    c.sw = w_scales;
    c.y = y;
    c.ydtype = ydtype;
    c.M = M;
    c.N = N;
    c.K = K;
    return finish(launch_i8_mm(v, current_stream(), c, workspace ? workspace : v.ws));
}
