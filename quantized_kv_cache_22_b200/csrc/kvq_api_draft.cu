// kvq_api_draft.cu -- the extern "C" boundary of the calls around drafted tokens: rotary
// append, read-back, tree attention and path commit.  Arguments are checked on the host
// before anything is launched; nothing is allocated and no state is kept.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kvq_internal.h"
#include "../../include/kvq.h"

using namespace kvq;

namespace {

bool valid_dtype(int32_t d) { return d == KVQ_F16 || d == KVQ_F32 || d == KVQ_BF16; }

CacheRows cache_rows(const kvq_config *c, const int32_t *table)
{
    CacheRows r{};
    r.batch = c->batch;
    r.cap = c->capacity;
    if (c->mode == KVQ_MODE_H) {
        r.heads = 1;
        return r;
    }
    r.heads = c->n_kv_heads;
    r.window = c->window;
    r.n_anchor = c->n_anchor;
    if (c->page_tokens) {
        r.block_table = table;
        r.max_pages = c->capacity / kPageTokens;
        r.n_pages = c->n_pages;
    }
    return r;
}

CacheTensor cache_tensor(void *codes, void *scales, int bits, int group)
{
    return CacheTensor{static_cast<uint8_t *>(codes), static_cast<__half *>(scales), bits, bits == 16 ? 32 : group};
}

// Resolve a kvq_rows (strides in elements of dtype): KVQ_OK, INVALID_ARG or ALIGN.
int rows_view(const kvq_rows *r, int64_t row, int32_t n, int32_t dtype, RowsView *out)
{
    if (!r->data || r->batch_stride < 0 || r->token_stride < 0) return KVQ_ERR_INVALID_ARG;
    out->data = r->data;
    out->token_stride = r->token_stride ? r->token_stride : row;
    out->batch_stride = r->batch_stride ? r->batch_stride : out->token_stride * n;
    const int64_t unit = dtype == KVQ_F32 ? 4 : 8;   // elements of 16 bytes
    if (!aligned16(r->data) || out->token_stride % unit || out->batch_stride % unit) return KVQ_ERR_ALIGN;
    return KVQ_OK;
}

int check_rope(const kvq_rope_config *r)
{
    if (!r) return KVQ_ERR_INVALID_ARG;
    if (r->rot_dim < 8 || r->rot_dim > 128 || r->rot_dim % 8 != 0) return KVQ_ERR_UNSUPPORTED;
    if (r->layout != KVQ_ROPE_HALF && r->layout != KVQ_ROPE_INTERLEAVED) return KVQ_ERR_INVALID_ARG;
    return KVQ_OK;
}

int check_scaling(const kvq_rope_config *r)
{
    if (r->scaling < KVQ_ROPE_PLAIN || r->scaling > KVQ_ROPE_BANDS) return KVQ_ERR_INVALID_ARG;
    if (!std::isfinite(r->base) || r->base <= 1.0 || !std::isfinite(r->gain) || r->gain < 0.0)
        return KVQ_ERR_INVALID_ARG;
    if (r->scaling != KVQ_ROPE_PLAIN && (!std::isfinite(r->factor) || r->factor < 1.0)) return KVQ_ERR_INVALID_ARG;
    if (r->scaling == KVQ_ROPE_YARN || r->scaling == KVQ_ROPE_BANDS)
        if (r->orig_len < 1 || !std::isfinite(r->high) || !(r->low > 0.0) || !(r->high > r->low))
            return KVQ_ERR_INVALID_ARG;
    return KVQ_OK;
}

// Frequencies of the pairs and the factor on cos and sin (see kvq_rope_scaling in kvq.h).
void rope_frequencies(const kvq_rope_config *r, double *freq, double *gain)
{
    const int rot = r->rot_dim, pairs = rot / 2;
    const double two_pi = 6.283185307179586476925286766559;
    double base = r->base;
    if (r->scaling == KVQ_ROPE_NTK) base *= std::pow(r->factor, (double)rot / (rot - 2));
    double lo = 0.0, hi = 0.0;
    if (r->scaling == KVQ_ROPE_YARN) {
        // the pair that turns n times in orig_len: orig_len base^(-2i / rot) / 2 pi = n
        lo = std::floor(rot * std::log(r->orig_len / (r->high * two_pi)) / (2.0 * std::log(base)));
        hi = std::ceil(rot * std::log(r->orig_len / (r->low * two_pi)) / (2.0 * std::log(base)));
        // (where even pair 0 turns less than `low` times, the ramp ends before it)
        lo = hi < 0.0 ? -1.0 : std::max(lo, 0.0);
        hi = hi < 0.0 ? 0.0 : std::min(hi, (double)(rot - 1));
    }
    for (int i = 0; i < pairs; i++) {
        const double f = std::pow(base, -2.0 * i / rot);
        double stretch = 0.0;   // share of the stretched frequency
        if (r->scaling == KVQ_ROPE_LINEAR) stretch = 1.0;
        if (r->scaling == KVQ_ROPE_YARN)
            stretch = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
        if (r->scaling == KVQ_ROPE_BANDS)
            stretch = 1.0 - std::min(1.0, std::max(0.0, (r->orig_len * f / two_pi - r->low) / (r->high - r->low)));
        freq[i] = stretch == 0.0 ? f : f / r->factor * stretch + f * (1.0 - stretch);
    }
    *gain = r->gain != 0.0 ? r->gain : (r->scaling == KVQ_ROPE_YARN ? 0.1 * std::log(r->factor) + 1.0 : 1.0);
}

// CTAs of a tree launch: one per SM unless the caller says otherwise.
int tree_ctas(int32_t num_ctas, int32_t *ctas)
{
    int sms = 0, smem = 0;
    if (num_ctas == 0) {
        const int rc = current_device_props(&sms, &smem);
        if (rc) return rc;
    }
    *ctas = num_ctas ? num_ctas : sms;
    return KVQ_OK;
}

uint64_t tree_seg_bytes(const kvq_config *cfg, int32_t n_tree, int G)
{
    const uint64_t n = (uint64_t)cfg->batch * cfg->n_kv_heads * tree_row_tiles(n_tree, G) * sizeof(int4);
    return (n + 255) / 256 * 256;
}

// What every KV-mode call here needs of its configuration and layer.
int check_draft(const kvq_config *cfg, const kvq_layer *layer)
{
    int rc = check_cfg(cfg);
    if (rc) return rc;
    if (cfg->mode != KVQ_MODE_KV || !layer) return KVQ_ERR_INVALID_ARG;
    return check_kv_layer(cfg, layer);
}

// kvq_tree_attn with its wait limit, and the segments that each CTA's producer copies.
int tree_attn(const kvq_config *cfg, const kvq_layer *layer, const void *q, int32_t q_dtype, int32_t n_tree,
              const int32_t *d_len, int32_t max_len_host, const int32_t *d_n_tree, const uint64_t *d_mask,
              float softmax_scale, void *out, int32_t out_dtype, void *workspace, uint64_t workspace_bytes,
              int32_t num_ctas, uint64_t timeout_ns, int32_t serve, kvq_stream_t stream)
{
    int rc = check_draft(cfg, layer);
    if (rc) return rc;
    if (!q || !d_len || !out || !workspace || num_ctas < 0 || max_len_host < 0 || n_tree < 1 ||
        n_tree > KVQ_TREE_MAX || !valid_dtype(q_dtype) || !valid_dtype(out_dtype) || !std::isfinite(softmax_scale))
        return KVQ_ERR_INVALID_ARG;
    if ((int64_t)max_len_host + n_tree > cfg->capacity) return KVQ_ERR_CAPACITY;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(d_mask) & 7u))
        return KVQ_ERR_ALIGN;
    uint64_t need = 0;
    rc = kvq_tree_workspace_bytes(cfg, n_tree, num_ctas, &need);
    if (rc) return rc;
    if (workspace_bytes < need) return KVQ_ERR_WORKSPACE;
    TreeParams p{};
    p.rows = cache_rows(cfg, layer->block_table);
    p.k = cache_tensor(layer->k_codes, layer->k_scales, cfg->k_bits, cfg->k_group);
    p.v = cache_tensor(layer->v_codes, layer->v_scales, cfg->v_bits, cfg->v_group);
    p.q = q;
    p.out = out;
    p.d_len = d_len;
    p.d_n_tree = d_n_tree;
    p.d_mask = d_mask;
    p.q_dtype = q_dtype;
    p.out_dtype = out_dtype;
    p.fmt = cfg->kv_format;
    p.n_tree = n_tree;
    p.n_q_heads = cfg->n_q_heads;
    p.G = cfg->n_q_heads / cfg->n_kv_heads;
    p.dh = cfg->head_dim;
    const float scale = softmax_scale != 0.f ? softmax_scale : 1.f / std::sqrt((float)cfg->head_dim);
    p.tau_log2e = scale * 1.4426950408889634f;
    p.timeout_ns = timeout_ns;
    p.serve = serve;
    p.row_tiles = tree_row_tiles(n_tree, p.G);
    p.slot_rows = tree_slot_rows(n_tree, p.G);
    p.status = static_cast<int *>(workspace);
    uint8_t *ws = static_cast<uint8_t *>(workspace) + kWorkspaceHeaderFloats * 4;
    p.seg = reinterpret_cast<int4 *>(ws);
    p.slots = reinterpret_cast<float *>(ws + tree_seg_bytes(cfg, n_tree, p.G));
    int sms = 0, max_smem = 0;
    rc = current_device_props(&sms, &max_smem);
    if (rc) return rc;
    if (!plan_tree(p, max_smem, &p.l)) return KVQ_ERR_UNSUPPORTED;
    rc = tree_ctas(num_ctas, &p.l.num_ctas);
    if (rc) return rc;
    cudaError_t e = launch_tree(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVQ_OK : fail("tree attention launch", e);
}

}  // namespace

extern "C" {

int kvq_rope_table(const kvq_rope_config *rope, int32_t first_pos, int32_t n_pos, float *table, kvq_stream_t stream)
{
    int rc = check_rope(rope);
    if (!rc) rc = check_scaling(rope);
    if (rc) return rc;
    if (first_pos < 0 || n_pos < 0 || (int64_t)first_pos + n_pos > 0x7fffffff) return KVQ_ERR_INVALID_ARG;
    if (n_pos == 0) return KVQ_OK;
    if (!table) return KVQ_ERR_INVALID_ARG;
    if (!aligned16(table)) return KVQ_ERR_ALIGN;
    RopeTableParams p{};
    rope_frequencies(rope, p.freq, &p.gain);
    p.table = reinterpret_cast<float2 *>(table);
    p.first_pos = first_pos;
    p.n_pos = n_pos;
    p.pairs = rope->rot_dim / 2;
    cudaError_t e = launch_rope_table(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVQ_OK : fail("rope table launch", e);
}

int kvq_rope_append(const kvq_config *cfg, const kvq_layer *layer, const kvq_rope_config *rope, const float *table,
                    int32_t table_len, const kvq_rows *q, const kvq_rows *k, const kvq_rows *v, const kvq_rows *q_out,
                    int32_t dtype, const int32_t *d_pos, int32_t max_pos_host, int32_t n_new, const int32_t *d_count,
                    const int32_t *d_rope_pos, kvq_stream_t stream)
{
    int rc = check_draft(cfg, layer);
    if (!rc) rc = check_rope(rope);
    if (rc) return rc;
    if (rope->rot_dim > cfg->head_dim) return KVQ_ERR_UNSUPPORTED;
    if (!table || table_len < 1 || !k || !v || !d_pos || (q == nullptr) != (q_out == nullptr) || n_new < 0 ||
        max_pos_host < 0 || !valid_dtype(dtype))
        return KVQ_ERR_INVALID_ARG;
    if (!aligned16(table)) return KVQ_ERR_ALIGN;
    if (cfg->window == 0 && (int64_t)max_pos_host + n_new > cfg->capacity) return KVQ_ERR_CAPACITY;
    if (!d_rope_pos && (int64_t)max_pos_host + n_new > table_len) return KVQ_ERR_CAPACITY;
    if (n_new == 0) return KVQ_OK;
    RopeAppendParams p{};
    const int64_t kv_row = (int64_t)cfg->n_kv_heads * cfg->head_dim, q_row = (int64_t)cfg->n_q_heads * cfg->head_dim;
    rc = rows_view(k, kv_row, n_new, dtype, &p.k_in);
    if (!rc) rc = rows_view(v, kv_row, n_new, dtype, &p.v_in);
    if (!rc && q) rc = rows_view(q, q_row, n_new, dtype, &p.q_in);
    if (!rc && q) rc = rows_view(q_out, q_row, n_new, dtype, &p.q_out);
    if (rc) return rc;
    p.rows = cache_rows(cfg, layer->block_table);
    p.k = cache_tensor(layer->k_codes, layer->k_scales, cfg->k_bits, cfg->k_group);
    p.v = cache_tensor(layer->v_codes, layer->v_scales, cfg->v_bits, cfg->v_group);
    p.table = reinterpret_cast<const float2 *>(table);
    p.d_pos = d_pos;
    p.d_count = d_count;
    p.d_rope_pos = d_rope_pos;
    p.table_len = table_len;
    p.rot = rope->rot_dim;
    p.interleaved = rope->layout == KVQ_ROPE_INTERLEAVED;
    p.dtype = dtype;
    p.fmt = cfg->kv_format;
    p.n_new = n_new;
    p.n_q_heads = cfg->n_q_heads;
    p.dh = cfg->head_dim;
    cudaError_t e = launch_rope_append(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVQ_OK : fail("rope append launch", e);
}

int kvq_read(const kvq_config *cfg, const kvq_layer *layer, const kvq_rows *k_out, const kvq_rows *v_out,
             int32_t out_dtype, const int32_t *d_pos, int32_t max_pos_host, int32_t n, const int32_t *d_count,
             kvq_stream_t stream)
{
    int rc = check_cfg(cfg);
    if (rc) return rc;
    if (!layer || !d_pos || n < 0 || max_pos_host < 0 || !valid_dtype(out_dtype)) return KVQ_ERR_INVALID_ARG;
    ReadParams p{};
    if (cfg->mode == KVQ_MODE_KV) {
        if (!k_out && !v_out) return KVQ_ERR_INVALID_ARG;
        rc = check_kv_layer(cfg, layer);
        if (rc) return rc;
        p.dim = cfg->head_dim;
        p.fmt = cfg->kv_format;
        p.t[0] = cache_tensor(layer->k_codes, layer->k_scales, cfg->k_bits, cfg->k_group);
        p.t[1] = cache_tensor(layer->v_codes, layer->v_scales, cfg->v_bits, cfg->v_group);
    } else {
        if (!k_out || v_out || !layer->k_codes || (cfg->h_bits != 16 && !layer->k_scales)) return KVQ_ERR_INVALID_ARG;
        if (!aligned16(layer->k_codes) || (layer->k_scales && !aligned16(layer->k_scales))) return KVQ_ERR_ALIGN;
        p.dim = cfg->d_model;
        p.fmt = KVQ_FMT_INT;
        p.t[0] = cache_tensor(layer->k_codes, layer->k_scales, cfg->h_bits,
                              cfg->h_bits == 16 ? 32 : cfg->d_model / cfg->h_groups);
    }
    if (cfg->window == 0 && (int64_t)max_pos_host + n > cfg->capacity) return KVQ_ERR_CAPACITY;
    if (n == 0) return KVQ_OK;
    p.rows = cache_rows(cfg, layer->block_table);
    const int64_t row = (int64_t)p.rows.heads * p.dim;
    if (k_out) rc = rows_view(k_out, row, n, out_dtype, &p.out[0]);
    if (!rc && v_out) rc = rows_view(v_out, row, n, out_dtype, &p.out[1]);
    if (rc) return rc;
    p.d_pos = d_pos;
    p.d_count = d_count;
    p.n = n;
    p.out_dtype = out_dtype;
    cudaError_t e = launch_read(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVQ_OK : fail("read launch", e);
}

int kvq_tree_workspace_bytes(const kvq_config *cfg, int32_t n_tree, int32_t num_ctas, uint64_t *bytes)
{
    int rc = check_cfg(cfg);
    if (rc) return rc;
    if (cfg->mode != KVQ_MODE_KV || !bytes || num_ctas < 0 || n_tree < 1 || n_tree > KVQ_TREE_MAX)
        return KVQ_ERR_INVALID_ARG;
    if (cfg->window != 0 || cfg->n_q_heads / cfg->n_kv_heads > 8) return KVQ_ERR_UNSUPPORTED;
    rc = tree_ctas(num_ctas, &num_ctas);
    if (rc) return rc;
    const int G = cfg->n_q_heads / cfg->n_kv_heads;
    *bytes = (uint64_t)kWorkspaceHeaderFloats * 4 + tree_seg_bytes(cfg, n_tree, G) +
             2ull * num_ctas * tree_slot_floats(tree_slot_rows(n_tree, G), cfg->head_dim) * 4;
    return KVQ_OK;
}

int kvq_tree_attn(const kvq_config *cfg, const kvq_layer *layer, const void *q, int32_t q_dtype, int32_t n_tree,
                  const int32_t *d_len, int32_t max_len_host, const int32_t *d_n_tree, const uint64_t *d_mask,
                  float softmax_scale, void *out, int32_t out_dtype, void *workspace, uint64_t workspace_bytes,
                  int32_t num_ctas, kvq_stream_t stream)
{
    return tree_attn(cfg, layer, q, q_dtype, n_tree, d_len, max_len_host, d_n_tree, d_mask, softmax_scale, out, out_dtype,
                     workspace, workspace_bytes, num_ctas, kTimeoutNs, INT32_MAX, stream);
}

int kvq_selftest_tree_timeout(const kvq_config *cfg, const kvq_layer *layer, const void *q, int32_t q_dtype,
                              int32_t n_tree, const int32_t *d_len, int32_t max_len_host, void *out, int32_t out_dtype,
                              void *workspace, uint64_t workspace_bytes, int32_t num_ctas, int32_t n_segments,
                              uint64_t timeout_ns, kvq_stream_t stream)
{
    if (n_segments < 0 || timeout_ns == 0 || timeout_ns > 2000000000ull) return KVQ_ERR_INVALID_ARG;
    return tree_attn(cfg, layer, q, q_dtype, n_tree, d_len, max_len_host, nullptr, nullptr, 0.f, out, out_dtype, workspace,
                     workspace_bytes, num_ctas, timeout_ns, n_segments, stream);
}

int kvq_tree_commit(const kvq_config *cfg, const kvq_layer *layers, int32_t n_layers, const int32_t *d_len,
                    int32_t max_len_host, int32_t n_tree, const int32_t *d_path, int32_t path_stride,
                    const int32_t *d_n_path, int32_t *d_len_out, kvq_stream_t stream)
{
    int rc = check_cfg(cfg);
    if (rc) return rc;
    if (cfg->mode != KVQ_MODE_KV || !layers || n_layers < 1 || !d_len || !d_path || !d_n_path || max_len_host < 0 ||
        n_tree < 1 || n_tree > KVQ_TREE_MAX || path_stride < 1 || path_stride > n_tree || d_len_out == d_len)
        return KVQ_ERR_INVALID_ARG;
    if (cfg->window != 0) return KVQ_ERR_UNSUPPORTED;
    if ((int64_t)max_len_host + n_tree > cfg->capacity) return KVQ_ERR_CAPACITY;
    // Two layers of the same rows: two warps' moves would race.  Layers may have one page pool, with a
    // block table each.
    const bool ks = scale_row_vals(cfg, cfg->k_bits, cfg->k_group) != 0, vs = scale_row_vals(cfg, cfg->v_bits, cfg->v_group) != 0;
    auto same_rows = [&](const kvq_layer &a, const kvq_layer &b) {
        if (cfg->page_tokens && a.block_table != b.block_table) return false;
        return a.k_codes == b.k_codes || a.v_codes == b.v_codes || (ks && a.k_scales == b.k_scales) ||
               (vs && a.v_scales == b.v_scales);
    };
    for (int32_t i = 0; i < n_layers; i++) {
        rc = check_kv_layer(cfg, &layers[i]);
        if (rc) return rc;
        for (int32_t j = 0; j < i; j++)
            if (same_rows(layers[j], layers[i])) return KVQ_ERR_INVALID_ARG;
    }
    CommitParams p{};
    p.rows = cache_rows(cfg, nullptr);
    p.row_bytes[0] = cfg->head_dim * cfg->k_bits / 8;
    p.row_bytes[1] = cfg->head_dim * cfg->v_bits / 8;
    p.scale_bytes[0] = scale_row_vals(cfg, cfg->k_bits, cfg->k_group) * 2;
    p.scale_bytes[1] = scale_row_vals(cfg, cfg->v_bits, cfg->v_group) * 2;
    p.n_tree = n_tree;
    p.path_stride = path_stride;
    p.d_len = d_len;
    p.d_path = d_path;
    p.d_n_path = d_n_path;
    p.d_len_out = d_len_out;
    for (int32_t i0 = 0; i0 < n_layers; i0 += kCommitLayers) {
        p.n_layers = std::min(kCommitLayers, n_layers - i0);
        for (int32_t i = 0; i < p.n_layers; i++) {
            const kvq_layer &l = layers[i0 + i];
            p.table[i] = cfg->page_tokens ? l.block_table : nullptr;
            p.codes[0][i] = static_cast<uint8_t *>(l.k_codes);
            p.codes[1][i] = static_cast<uint8_t *>(l.v_codes);
            p.scales[0][i] = static_cast<__half *>(l.k_scales);
            p.scales[1][i] = static_cast<__half *>(l.v_scales);
        }
        cudaError_t e = launch_commit(p, reinterpret_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return fail("commit launch", e);
    }
    return KVQ_OK;
}

}  // extern "C"
