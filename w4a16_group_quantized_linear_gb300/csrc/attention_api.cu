// C ABI of the attention operators: argument validation. The entry points and
// their contracts are documented in include/w4a16.h.
#include <cmath>

#include "cache8.cuh"

namespace w4a16 {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool bad_stride(int64_t s) { return s < 0 || s % 8 != 0; }

w4a16_status check_device(const DeviceInfo** dev) {
    *dev = device_info();
    if (!*dev) return W4A16_ERR_CUDA;
    return (*dev)->cc_major == 10 && (*dev)->cc_minor == 3 ? W4A16_OK : W4A16_ERR_UNSUPPORTED;
}

w4a16_status check_dtype(int32_t dtype) {
    return dtype == W4A16_DTYPE_F16 || dtype == W4A16_DTYPE_BF16 ? W4A16_OK : W4A16_ERR_UNSUPPORTED;
}

w4a16_status check_rotary(const w4a16_rotary& r, int32_t head_dim, bool need_positions) {
    if (r.rotary_dim <= 0 || r.rotary_dim > head_dim || r.rows < 0 || r.axes < 1) return W4A16_ERR_INVALID_ARG;
    if (r.rotary_dim % 16 != 0 || r.rotary_dim > 256 || r.axes > 4) return W4A16_ERR_UNSUPPORTED;
    if (!r.table || (!r.positions && (need_positions || r.axes != 1))) return W4A16_ERR_INVALID_ARG;
    if (!aligned16(r.table)) return W4A16_ERR_MISALIGNED;
    if (r.pair_axes)
        for (int i = 0; i < r.rotary_dim / 2; ++i)
            if (r.pair_axes[i] >= r.axes) return W4A16_ERR_INVALID_ARG;
    return W4A16_OK;
}

// Everything of a cache, its scales (8 bits) and its batch that the host can see.
w4a16_status check_cache(const w4a16_paged_cache* c, int64_t T, const w4a16_cache_scales* scales = nullptr) {
    if (!c || T < 0 || c->batch < 0 || c->pages < 0 || c->max_pages < 0 || c->kv_heads < 1 || c->page_size < 1)
        return W4A16_ERR_INVALID_ARG;
    w4a16_status s = check_dtype(c->dtype);
    if (s != W4A16_OK) return s;
    if ((c->head_dim != 64 && c->head_dim != 128) || c->page_size % 16 != 0 ||
        (int64_t)c->max_pages * c->page_size > (int64_t)1 << 30 || c->pages > 0x7fffffffLL || T > 0x7fffffffLL)
        return W4A16_ERR_UNSUPPORTED;
    if (bad_stride(c->page_stride) || bad_stride(c->slot_stride) || bad_stride(c->head_stride) ||
        c->page_table_stride < 0)
        return W4A16_ERR_INVALID_ARG;
    if (scales) {
        if (scales->format != W4A16_CACHE_INT8 && scales->format != W4A16_CACHE_E4M3) return W4A16_ERR_UNSUPPORTED;
        if (c->page_stride % 16 != 0 || c->slot_stride % 16 != 0 || c->head_stride % 16 != 0 ||
            scales->page_stride < 0 || scales->page_stride % 4 != 0 || scales->head_stride < 0 ||
            scales->head_stride % 4 != 0)
            return W4A16_ERR_INVALID_ARG;
    }
    if (T == 0) return W4A16_OK;
    if (scales) {
        if (!scales->k || !scales->v) return W4A16_ERR_INVALID_ARG;
        if (!aligned16(scales->k) || !aligned16(scales->v)) return W4A16_ERR_MISALIGNED;
    }
    if (c->batch == 0 || c->pages == 0 || !c->k || !c->v || !c->page_table || !c->q_offsets || !c->kv_lens)
        return W4A16_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v)) return W4A16_ERR_MISALIGNED;
    return W4A16_OK;
}

CacheArgs cache_args(const w4a16_paged_cache& c, int64_t T, unsigned int* err) {
    CacheArgs a{};
    a.k = c.k;
    a.v = c.v;
    a.pages = c.pages;
    a.page_stride = c.page_stride;
    a.slot_stride = c.slot_stride;
    a.head_stride = c.head_stride;
    a.table = c.page_table;
    a.table_stride = c.page_table_stride;
    a.page_size = c.page_size;
    a.max_pages = c.max_pages;
    a.by_page = fast_div(c.page_size);
    a.q_offsets = c.q_offsets;
    a.kv_lens = c.kv_lens;
    a.batch = c.batch;
    a.kv_heads = c.kv_heads;
    a.head_dim = c.head_dim;
    a.T = T;
    a.err = err;
    return a;
}

int format_of(const w4a16_cache_scales* s) { return s ? s->format : 0; }

ScaleArgs scale_args(const w4a16_cache_scales* s) {
    return s ? ScaleArgs{s->k, s->v, s->page_stride, s->head_stride} : ScaleArgs{};
}

w4a16_status check_norm(const float* weight, float eps) {
    if (!std::isfinite(eps) || !(eps >= 0.0f)) return W4A16_ERR_INVALID_ARG;
    return aligned16(weight) ? W4A16_OK : W4A16_ERR_MISALIGNED;
}

// w4a16_rope, and w4a16_rope_norm where `normed`
w4a16_status rope(int32_t dtype, const uint16_t* x, int64_t x_row_stride, int64_t x_head_stride, uint16_t* out,
                  int64_t out_row_stride, int64_t out_head_stride, int64_t T, int32_t heads, int32_t head_dim,
                  bool normed, const float* weight, float eps, const w4a16_rotary* rotary, void* stream) {
    w4a16_status s = check_dtype(dtype);
    if (s != W4A16_OK) return s;
    if (T < 0 || heads < 0 || head_dim < 1 || !rotary || bad_stride(x_row_stride) || bad_stride(x_head_stride) ||
        bad_stride(out_row_stride) || bad_stride(out_head_stride))
        return W4A16_ERR_INVALID_ARG;
    if (head_dim % 16 != 0 || head_dim > 1024 || T > 0x7fffffffLL) return W4A16_ERR_UNSUPPORTED;
    if (normed && head_dim > 512) return W4A16_ERR_UNSUPPORTED;
    if (T == 0 || heads == 0) return W4A16_OK;
    s = check_rotary(*rotary, head_dim, true);
    if (s != W4A16_OK) return s;
    if (!x || !out || (normed && !weight)) return W4A16_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(out)) return W4A16_ERR_MISALIGNED;
    if (normed && (s = check_norm(weight, eps)) != W4A16_OK) return s;
    const DeviceInfo* dev;
    s = check_device(&dev);
    if (s != W4A16_OK) return s;
    if (normed)
        return rope_norm_launch(*dev, dtype, x, x_row_stride, x_head_stride, out, out_row_stride, out_head_stride, T,
                                heads, head_dim, weight, eps, rotary, (cudaStream_t)stream);
    return rope_launch(*dev, dtype, x, x_row_stride, x_head_stride, out, out_row_stride, out_head_stride, T, heads,
                       head_dim, rotary, (cudaStream_t)stream);
}

// w4a16_kv_append, and w4a16_kv_append_ex with scales or norms
w4a16_status append(const w4a16_paged_cache* cache, const w4a16_cache_scales* scales, int64_t T, const uint16_t* k,
                    int64_t k_row_stride, int64_t k_head_stride, const uint16_t* v, int64_t v_row_stride,
                    int64_t v_head_stride, const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride,
                    int32_t heads, uint16_t* q_out, const w4a16_head_norms* norms, const w4a16_rotary* rotary,
                    void* stream) {
    w4a16_status s = check_cache(cache, T, scales);
    if (s != W4A16_OK) return s;
    if (heads < 0 || bad_stride(k_row_stride) || bad_stride(k_head_stride) || bad_stride(v_row_stride) ||
        bad_stride(v_head_stride) || bad_stride(q_row_stride) || bad_stride(q_head_stride))
        return W4A16_ERR_INVALID_ARG;
    if (T == 0) return W4A16_OK;
    if (rotary) {
        s = check_rotary(*rotary, cache->head_dim, false);
        if (s != W4A16_OK) return s;
    }
    if (norms && ((s = check_norm(norms->q, norms->eps)) != W4A16_OK ||
                  (s = check_norm(norms->k, norms->eps)) != W4A16_OK))
        return s;
    if (!k || !v || (q && heads > 0 && !q_out)) return W4A16_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out)) return W4A16_ERR_MISALIGNED;
    const DeviceInfo* dev;
    s = check_device(&dev);
    if (s != W4A16_OK) return s;
    if (scales || (norms && (norms->q || norms->k)))
        return append_ex_launch(*dev, cache->dtype, format_of(scales), cache_args(*cache, T, dev->error_word),
                                scale_args(scales), q, q_row_stride, q_head_stride, heads, q_out, k, k_row_stride,
                                k_head_stride, v, v_row_stride, v_head_stride, norms, rotary, (cudaStream_t)stream);
    return append_launch(*dev, cache->dtype, cache_args(*cache, T, dev->error_word), q, q_row_stride, q_head_stride,
                         heads, q_out, k, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride, rotary,
                         (cudaStream_t)stream);
}

// w4a16_paged_attention, and w4a16_paged_attention_ex with scales
w4a16_status attend(const w4a16_paged_cache* cache, const w4a16_cache_scales* scales, int64_t T, const uint16_t* q,
                    int64_t q_row_stride, int64_t q_head_stride, int32_t heads, int64_t max_q_len, uint32_t flags,
                    int32_t window, float scale, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                    void* stream) {
    w4a16_status s = check_cache(cache, T, scales);
    if (s != W4A16_OK) return s;
    const float scale_log2 = scale * 1.4426950408889634f;
    if (heads < 1 || heads % cache->kv_heads != 0 || max_q_len < 0 || (flags & ~W4A16_CAUSAL) || window < 0 ||
        (window > 0 && !(flags & W4A16_CAUSAL)) || !std::isfinite(scale_log2) || !(scale > 0.0f) ||
        bad_stride(q_row_stride) || bad_stride(q_head_stride))
        return W4A16_ERR_INVALID_ARG;
    if (T == 0) return W4A16_OK;
    if (!q || !out || max_q_len == 0) return W4A16_ERR_INVALID_ARG;
    if (T * (heads / cache->kv_heads) > 0x7ffffc00LL) return W4A16_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(out) || ((uintptr_t)lse & 3u)) return W4A16_ERR_MISALIGNED;
    const DeviceInfo* dev;
    s = check_device(&dev);
    if (s != W4A16_OK) return s;
    AttentionArgs a{};
    a.c = cache_args(*cache, T, dev->error_word);
    a.q = q;
    a.q_row_stride = q_row_stride;
    a.q_head_stride = q_head_stride;
    a.out = out;
    a.lse = lse;
    a.heads = heads;
    a.ratio = heads / cache->kv_heads;
    a.by_ratio = fast_div(a.ratio);
    a.causal = (flags & W4A16_CAUSAL) ? 1 : 0;
    a.window = window;
    a.scale_log2 = scale_log2;
    a.max_q_len = max_q_len < T ? max_q_len : T;
    if (scales)
        return attention8_launch(*dev, cache->dtype, scales->format, a, scale_args(scales), workspace, workspace_bytes,
                                 (cudaStream_t)stream);
    return attention_launch(*dev, cache->dtype, a, workspace, workspace_bytes, (cudaStream_t)stream);
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

w4a16_status w4a16_rope(int32_t dtype, const uint16_t* x, int64_t x_row_stride, int64_t x_head_stride, uint16_t* out,
                        int64_t out_row_stride, int64_t out_head_stride, int64_t T, int32_t heads, int32_t head_dim,
                        const w4a16_rotary* rotary, void* stream) {
    return rope(dtype, x, x_row_stride, x_head_stride, out, out_row_stride, out_head_stride, T, heads, head_dim, false,
                nullptr, 0.0f, rotary, stream);
}

w4a16_status w4a16_rope_norm(int32_t dtype, const uint16_t* x, int64_t x_row_stride, int64_t x_head_stride,
                             uint16_t* out, int64_t out_row_stride, int64_t out_head_stride, int64_t T, int32_t heads,
                             int32_t head_dim, const float* weight, float eps, const w4a16_rotary* rotary,
                             void* stream) {
    return rope(dtype, x, x_row_stride, x_head_stride, out, out_row_stride, out_head_stride, T, heads, head_dim, true,
                weight, eps, rotary, stream);
}

w4a16_status w4a16_kv_append(const w4a16_paged_cache* cache, int64_t T, const uint16_t* k, int64_t k_row_stride,
                             int64_t k_head_stride, const uint16_t* v, int64_t v_row_stride, int64_t v_head_stride,
                             const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int32_t heads,
                             uint16_t* q_out, const w4a16_rotary* rotary, void* stream) {
    return append(cache, nullptr, T, k, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride, q, q_row_stride,
                  q_head_stride, heads, q_out, nullptr, rotary, stream);
}

w4a16_status w4a16_kv_append_ex(const w4a16_paged_cache* cache, const w4a16_cache_scales* scales, int64_t T,
                                const uint16_t* k, int64_t k_row_stride, int64_t k_head_stride, const uint16_t* v,
                                int64_t v_row_stride, int64_t v_head_stride, const uint16_t* q, int64_t q_row_stride,
                                int64_t q_head_stride, int32_t heads, uint16_t* q_out, const w4a16_head_norms* norms,
                                const w4a16_rotary* rotary, void* stream) {
    return append(cache, scales, T, k, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride, q, q_row_stride,
                  q_head_stride, heads, q_out, norms, rotary, stream);
}

w4a16_status w4a16_kv_read(const w4a16_paged_cache* cache, const w4a16_cache_scales* scales, int64_t T, uint16_t* k,
                           uint16_t* v, void* stream) {
    w4a16_status s = check_cache(cache, T, scales);
    if (s != W4A16_OK || T == 0) return s;
    if (!k || !v) return W4A16_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return W4A16_ERR_MISALIGNED;
    const DeviceInfo* dev;
    s = check_device(&dev);
    if (s != W4A16_OK) return s;
    return read_launch(*dev, cache->dtype, format_of(scales), cache_args(*cache, T, dev->error_word),
                       scale_args(scales), k, v, (cudaStream_t)stream);
}

size_t w4a16_paged_attention_workspace_bytes(int64_t T, int32_t batch, int32_t heads, int32_t kv_heads,
                                             int32_t head_dim, int64_t max_q_len) {
    if (T <= 0 || batch <= 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0 || max_q_len <= 0 ||
        (head_dim != 64 && head_dim != 128))
        return 0;
    const DeviceInfo* dev = device_info();
    if (!dev) return 0;
    return attention_workspace_bytes(*dev, T, batch, heads, kv_heads, head_dim, max_q_len);
}

w4a16_status w4a16_paged_attention(const w4a16_paged_cache* cache, int64_t T, const uint16_t* q,
                                   int64_t q_row_stride, int64_t q_head_stride, int32_t heads, int64_t max_q_len,
                                   uint32_t flags, int32_t window, float scale, uint16_t* out, float* lse,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    return attend(cache, nullptr, T, q, q_row_stride, q_head_stride, heads, max_q_len, flags, window, scale, out, lse,
                  workspace, workspace_bytes, stream);
}

w4a16_status w4a16_paged_attention_ex(const w4a16_paged_cache* cache, const w4a16_cache_scales* scales, int64_t T,
                                      const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int32_t heads,
                                      int64_t max_q_len, uint32_t flags, int32_t window, float scale, uint16_t* out,
                                      float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    return attend(cache, scales, T, q, q_row_stride, q_head_stride, heads, max_q_len, flags, window, scale, out, lse,
                  workspace, workspace_bytes, stream);
}

}  // extern "C"
