// attn_api.cuh -- C ABI of the attention layer's operators: argument checks
// and launches.  Included by wlq_api.cu after its host helpers.
#pragma once

namespace {

wlq_status check_rope(int head_dim, const int32_t* positions, int axes, const float* inv_freq, int rotary_dim,
                      const int32_t* sections, double eps, wlq::RopeArgs* out) {
    std::memset(out, 0, sizeof *out);
    if (!(eps >= 0.0) || std::isinf(eps)) return fail(WLQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
    out->eps = eps;
    out->axes = 1;
    if (!positions) return WLQ_OK;
    if (axes < 1 || axes > wlq::ROPE_MAX_AXES) return fail(WLQ_ERR_SHAPE, "positions need 1..4 axes");
    if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16)
        return fail(WLQ_ERR_SHAPE, "rotary_dim must be a multiple of 16, at most head_dim");
    if (!inv_freq || !sections) return fail(WLQ_ERR_INVALID_ARG, "positions need inv_freq and sections");
    if ((reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(inv_freq) & 3u))
        return fail(WLQ_ERR_ALIGN, "positions and inv_freq must be 4-byte aligned");
    int64_t sum = 0;
    for (int i = 0; i < axes; ++i) {
        if (sections[i] < 0) return fail(WLQ_ERR_SHAPE, "a section is negative");
        sum += sections[i];
        out->sec_end[i] = static_cast<int>(std::min<int64_t>(sum, rotary_dim));
    }
    if (sum != rotary_dim / 2) return fail(WLQ_ERR_SHAPE, "sections must add up to rotary_dim / 2");
    out->pos = positions;
    out->inv_freq = inv_freq;
    out->axes = axes;
    out->pairs = rotary_dim / 2;
    return WLQ_OK;
}

bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

wlq_status check_head_dim(int head_dim) {
    if (head_dim != 64 && head_dim != 128) return fail(WLQ_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    return WLQ_OK;
}

// Rows of `heads` heads at x + t * stride (may be null with 0 heads).
wlq_status check_rows(const char* what, const void* x, int64_t stride, int heads, int head_dim) {
    if (heads < 0 || heads > 65536) return fail(WLQ_ERR_SHAPE, "%s: number of heads", what);
    if (heads == 0) return WLQ_OK;
    if (!x) return fail(WLQ_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!aligned16(x) || stride % 8) return fail(WLQ_ERR_ALIGN, "%s must be 16-byte aligned with a token stride of whole 16 bytes", what);
    if (stride < static_cast<int64_t>(heads) * head_dim) return fail(WLQ_ERR_SHAPE, "%s: token stride below heads * head_dim", what);
    return WLQ_OK;
}

// CTAs per token: one, or more where few tokens leave the SMs idle.
unsigned head_splits(int64_t tokens, int bites, int sms) {
    const int64_t most = cdiv(bites, wlq::KV_THREADS / 32);
    const int64_t want = std::max<int64_t>(1, 4ll * sms / std::max<int64_t>(tokens, 1));
    return static_cast<unsigned>(std::max<int64_t>(1, std::min(most, want)));
}

wlq_status check_batch(const int32_t* cu, const int32_t* kv_lens, int batch, int max_q, const int32_t* table,
                       int64_t table_width, int64_t tokens, wlq::KvBatch* out) {
    if (batch < 0 || max_q < 0 || tokens < 0 || table_width < 0)
        return fail(WLQ_ERR_INVALID_ARG, "batch, max_q, tokens and table_width must be >= 0");
    if (tokens >= (int64_t(1) << 31) || static_cast<int64_t>(batch) * max_q >= (int64_t(1) << 31))
        return fail(WLQ_ERR_SHAPE, "tokens and batch * max_q must stay below 2^31");
    if (batch > 0 && (!cu || !kv_lens)) return fail(WLQ_ERR_INVALID_ARG, "cu_seqlens or kv_lens: null pointer");
    if (batch > 0 && table_width > 0 && !table) return fail(WLQ_ERR_INVALID_ARG, "block_table: null pointer");
    if (!aligned4(cu) || !aligned4(kv_lens) || !aligned4(table))
        return fail(WLQ_ERR_ALIGN, "cu_seqlens, kv_lens and block_table must be 4-byte aligned");
    *out = wlq::KvBatch{cu, kv_lens, table, table_width, batch, max_q, tokens};
    return WLQ_OK;
}

wlq_status check_pool(const void* kc, const void* ks, const void* vc, const void* vs, int64_t num_pages, int page_size,
                      int group, int heads, int head_dim, wlq::Kv4Pool* out) {
    if (heads < 1 || heads > 65536) return fail(WLQ_ERR_SHAPE, "the cache needs 1..65536 heads");
    if (!(group == 32 || group == 64 || group == 128) || group > head_dim)
        return fail(WLQ_ERR_UNSUPPORTED, "group must be 32, 64 or 128, at most head_dim");
    int shift = 0;
    while ((1 << shift) < page_size && shift < 9) ++shift;
    if (shift < 4 || shift > 8 || (1 << shift) != page_size)
        return fail(WLQ_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
    if (num_pages < 0 || num_pages >= (int64_t(1) << 31)) return fail(WLQ_ERR_SHAPE, "num_pages");
    if (num_pages > 0 && (!kc || !ks || !vc || !vs)) return fail(WLQ_ERR_INVALID_ARG, "cache: null pointer");
    if (!aligned16(kc) || !aligned16(vc) || !aligned16(ks) || !aligned16(vs))
        return fail(WLQ_ERR_ALIGN, "cache arrays must be 16-byte aligned");
    out->k = static_cast<uint8_t*>(const_cast<void*>(kc));
    out->ks = static_cast<__half*>(const_cast<void*>(ks));
    out->v = static_cast<uint8_t*>(const_cast<void*>(vc));
    out->vs = static_cast<__half*>(const_cast<void*>(vs));
    out->pages = num_pages;
    out->page_shift = shift;
    out->heads = heads;
    out->lg_group = group == 32 ? 5 : group == 64 ? 6 : 7;
    return WLQ_OK;
}

// How a call of the decode kernel is cut: row tiles of 8 nt rows, and the
// splits of a sequence's cached tokens over CTAs.
constexpr int kPlanSms = 148;  // the SMs of a B200: plans, and with them workspace sizes, need no device

struct DecPlan {
    int nt = 1, row_tiles = 1, splits = 1;
    size_t off_ml = 0, ws = 0;
};

DecPlan dec_plan(int64_t tokens, int batch, int max_q, int64_t max_kv, int q_heads, int kv_heads, int head_dim, int window,
                 int sms) {
    DecPlan p;
    const int64_t rows = static_cast<int64_t>(max_q) * (q_heads / kv_heads);
    p.nt = rows > 8 ? 2 : 1;
    p.row_tiles = static_cast<int>(cdiv(rows, 8 * p.nt));
    int64_t seen = std::max<int64_t>(max_kv, 1);
    if (window > 0) seen = std::min<int64_t>(seen, static_cast<int64_t>(window) + max_q);
    const int64_t units = cdiv(seen, wlq::DEC_UNIT);
    const int64_t base = static_cast<int64_t>(batch) * kv_heads * p.row_tiles;
    // enough CTAs for four on each SM, but at least two units for each warp of a split
    const int64_t want = cdiv(4ll * sms, base), most = std::max<int64_t>(1, units / (2 * wlq::DEC_WARPS));
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, most, 128})));
    if (p.splits > 1) {
        const size_t parts = static_cast<size_t>(tokens) * q_heads * p.splits;
        p.off_ml = align256(parts * head_dim * sizeof(float));
        p.ws = p.off_ml + align256(parts * sizeof(float2));
    }
    return p;
}

template <int D>
wlq_status launch_decode(const wlq::AttnArgs& a, const DecPlan& p, cudaStream_t s) {
    const int64_t grid = static_cast<int64_t>(a.B.batch) * a.P.heads * p.row_tiles * p.splits;
    if (grid >= (int64_t(1) << 31)) return fail(WLQ_ERR_SHAPE, "too many queries in one call");
    const unsigned gx = static_cast<unsigned>(grid);
    cudaError_t e = p.nt == 1 ? launch_k(wlq::kv4_decode_kernel<D, 1>, gx, wlq::DEC_WARPS * 32, 0, s, a)
                              : launch_k(wlq::kv4_decode_kernel<D, 2>, gx, wlq::DEC_WARPS * 32, 0, s, a);
    if (e == cudaSuccess && p.splits > 1) {
        const int64_t units = cdiv(static_cast<int64_t>(a.B.batch) * a.B.max_q * a.q_heads, 8);
        if (units >= (int64_t(1) << 31)) return fail(WLQ_ERR_SHAPE, "too many queries in one call");
        e = launch_k(wlq::kv4_combine_kernel<D>, static_cast<unsigned>(units), 256, 0, s, a);
    }
    return e == cudaSuccess ? WLQ_OK : cuda_fail(e, "kv4_attention launch");
}

wlq_status check_heads(int q_heads, int kv_heads) {
    if (q_heads < 1 || kv_heads < 1 || q_heads > 65536 || q_heads % kv_heads)
        return fail(WLQ_ERR_SHAPE, "q_heads must be a positive multiple of kv_heads");
    return WLQ_OK;
}

}  // namespace

extern "C" {

wlq_status wlq_qk_norm_rope(const void* q, int64_t q_stride, int q_heads, const void* k, int64_t k_stride, int k_heads,
                            int64_t tokens, int head_dim, const void* q_weight, const void* k_weight, double eps,
                            const int32_t* positions, int axes, const float* inv_freq, int rotary_dim,
                            const int32_t* sections, int interleaved, void* q_out, int64_t q_out_stride, void* k_out,
                            int64_t k_out_stride, void* stream) {
    wlq_status st;
    if (tokens < 0 || tokens >= (int64_t(1) << 31)) return fail(WLQ_ERR_SHAPE, "tokens must be 0 .. 2^31 - 1");
    if ((st = check_head_dim(head_dim)) != WLQ_OK) return st;
    wlq::RopeArgs a;
    if ((st = check_rope(head_dim, positions, axes, inv_freq, rotary_dim, sections, eps, &a)) != WLQ_OK) return st;
    if (tokens == 0 || (q_heads == 0 && k_heads == 0)) return WLQ_OK;
    if ((st = check_rows("q", q, q_stride, q_heads, head_dim)) != WLQ_OK) return st;
    if ((st = check_rows("k", k, k_stride, k_heads, head_dim)) != WLQ_OK) return st;
    if ((st = check_rows("q_out", q_out, q_out_stride, q_heads, head_dim)) != WLQ_OK) return st;
    if ((st = check_rows("k_out", k_out, k_out_stride, k_heads, head_dim)) != WLQ_OK) return st;
    if (!aligned2(q_weight) || !aligned2(k_weight)) return fail(WLQ_ERR_ALIGN, "weights must be 2-byte aligned");
    if ((q_heads && q == q_out && q_stride != q_out_stride) || (k_heads && k == k_out && k_stride != k_out_stride))
        return fail(WLQ_ERR_INVALID_ARG, "in place needs the same token stride");
    int dev;
    DeviceInfo* d;
    if ((st = current_device(&dev, &d)) != WLQ_OK) return st;
    const wlq::HeadRows Q{static_cast<const uint16_t*>(q), q_stride, q_heads, static_cast<const uint16_t*>(q_weight),
                          static_cast<uint16_t*>(q_out), q_out_stride};
    const wlq::HeadRows K{static_cast<const uint16_t*>(k), k_stride, k_heads, static_cast<const uint16_t*>(k_weight),
                          static_cast<uint16_t*>(k_out), k_out_stride};
    const int rpw = 32 / (head_dim / 8);
    const int bites = static_cast<int>(cdiv(q_heads, rpw) + cdiv(k_heads, rpw));
    const dim3 grid(static_cast<unsigned>(tokens), head_splits(tokens, bites, d->sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (head_dim == 128)
        e = interleaved ? launch_k(wlq::qk_norm_rope_kernel<128, true>, grid, wlq::KV_THREADS, 0, s, Q, K, a, tokens)
                        : launch_k(wlq::qk_norm_rope_kernel<128, false>, grid, wlq::KV_THREADS, 0, s, Q, K, a, tokens);
    else
        e = interleaved ? launch_k(wlq::qk_norm_rope_kernel<64, true>, grid, wlq::KV_THREADS, 0, s, Q, K, a, tokens)
                        : launch_k(wlq::qk_norm_rope_kernel<64, false>, grid, wlq::KV_THREADS, 0, s, Q, K, a, tokens);
    return e == cudaSuccess ? WLQ_OK : cuda_fail(e, "qk_norm_rope launch");
}

wlq_status wlq_kv4_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t tokens, int heads,
                          int head_dim, const void* k_weight, double eps, const int32_t* positions, int axes,
                          const float* inv_freq, int rotary_dim, const int32_t* sections, int interleaved,
                          const int32_t* cu_seqlens, const int32_t* kv_lens, int batch, int max_q,
                          const int32_t* block_table, int64_t table_width, void* k_codes, void* k_scales, void* v_codes,
                          void* v_scales, int64_t num_pages, int page_size, int group, void* stream) {
    wlq_status st;
    if ((st = check_head_dim(head_dim)) != WLQ_OK) return st;
    wlq::RopeArgs a;
    if ((st = check_rope(head_dim, positions, axes, inv_freq, rotary_dim, sections, eps, &a)) != WLQ_OK) return st;
    wlq::KvBatch B;
    if ((st = check_batch(cu_seqlens, kv_lens, batch, max_q, block_table, table_width, tokens, &B)) != WLQ_OK) return st;
    wlq::Kv4Pool P;
    if ((st = check_pool(k_codes, k_scales, v_codes, v_scales, num_pages, page_size, group, heads, head_dim, &P)) != WLQ_OK)
        return st;
    if (batch == 0 || max_q == 0 || tokens == 0) return WLQ_OK;
    if ((st = check_rows("k", k, k_stride, heads, head_dim)) != WLQ_OK) return st;
    if ((st = check_rows("v", v, v_stride, heads, head_dim)) != WLQ_OK) return st;
    if (!aligned2(k_weight)) return fail(WLQ_ERR_ALIGN, "weights must be 2-byte aligned");
    int dev;
    DeviceInfo* d;
    if ((st = current_device(&dev, &d)) != WLQ_OK) return st;
    const wlq::HeadRows K{static_cast<const uint16_t*>(k), k_stride, heads, static_cast<const uint16_t*>(k_weight), nullptr, 0};
    const wlq::HeadRows V{static_cast<const uint16_t*>(v), v_stride, heads, nullptr, nullptr, 0};
    const int bites = static_cast<int>(2 * cdiv(heads, 32 / (head_dim / 8)));
    const int64_t units = static_cast<int64_t>(batch) * max_q;
    const dim3 grid(static_cast<unsigned>(units), head_splits(std::min(units, tokens), bites, d->sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (head_dim == 128)
        e = interleaved ? launch_k(wlq::kv4_append_kernel<128, true>, grid, wlq::KV_THREADS, 0, s, K, V, a, B, P)
                        : launch_k(wlq::kv4_append_kernel<128, false>, grid, wlq::KV_THREADS, 0, s, K, V, a, B, P);
    else
        e = interleaved ? launch_k(wlq::kv4_append_kernel<64, true>, grid, wlq::KV_THREADS, 0, s, K, V, a, B, P)
                        : launch_k(wlq::kv4_append_kernel<64, false>, grid, wlq::KV_THREADS, 0, s, K, V, a, B, P);
    return e == cudaSuccess ? WLQ_OK : cuda_fail(e, "kv4_append launch");
}

wlq_status wlq_kv4_read(const int32_t* cu_seqlens, const int32_t* kv_lens, int batch, int max_q,
                        const int32_t* block_table, int64_t table_width, const void* k_codes, const void* k_scales,
                        const void* v_codes, const void* v_scales, int64_t num_pages, int page_size, int group,
                        int64_t tokens, int heads, int head_dim, void* k_out, void* v_out, void* stream) {
    wlq_status st;
    if ((st = check_head_dim(head_dim)) != WLQ_OK) return st;
    wlq::KvBatch B;
    if ((st = check_batch(cu_seqlens, kv_lens, batch, max_q, block_table, table_width, tokens, &B)) != WLQ_OK) return st;
    wlq::Kv4Pool P;
    if ((st = check_pool(k_codes, k_scales, v_codes, v_scales, num_pages, page_size, group, heads, head_dim, &P)) != WLQ_OK)
        return st;
    if (batch == 0 || max_q == 0 || tokens == 0) return WLQ_OK;
    if (!k_out || !v_out) return fail(WLQ_ERR_INVALID_ARG, "k_out or v_out: null pointer");
    if (!aligned16(k_out) || !aligned16(v_out)) return fail(WLQ_ERR_ALIGN, "k_out and v_out must be 16-byte aligned");
    int dev;
    DeviceInfo* d;
    if ((st = current_device(&dev, &d)) != WLQ_OK) return st;
    const int bites = static_cast<int>(2 * cdiv(heads, 32 / (head_dim / 8)));
    const int64_t units = static_cast<int64_t>(batch) * max_q;
    const dim3 grid(static_cast<unsigned>(units), head_splits(std::min(units, tokens), bites, d->sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint16_t *ko = static_cast<uint16_t*>(k_out), *vo = static_cast<uint16_t*>(v_out);
    const cudaError_t e = head_dim == 128 ? launch_k(wlq::kv4_read_kernel<128>, grid, wlq::KV_THREADS, 0, s, ko, vo, B, P)
                                          : launch_k(wlq::kv4_read_kernel<64>, grid, wlq::KV_THREADS, 0, s, ko, vo, B, P);
    return e == cudaSuccess ? WLQ_OK : cuda_fail(e, "kv4_read launch");
}

size_t wlq_kv4_attention_workspace(int64_t tokens, int batch, int max_q, int64_t max_kv, int q_heads, int kv_heads,
                                   int head_dim) {
    if (tokens <= 0 || batch <= 0 || max_q <= 0 || max_kv < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads ||
        (head_dim != 64 && head_dim != 128))
        return 0;
    return dec_plan(tokens, batch, max_q, max_kv, q_heads, kv_heads, head_dim, 0, kPlanSms).ws;
}

wlq_status wlq_kv4_attention(const void* q, int64_t q_stride, int64_t tokens, int q_heads, int kv_heads, int head_dim,
                             const int32_t* cu_seqlens, const int32_t* kv_lens, int batch, int max_q, int64_t max_kv,
                             const int32_t* block_table, int64_t table_width, const void* k_codes, const void* k_scales,
                             const void* v_codes, const void* v_scales, int64_t num_pages, int page_size, int group,
                             float scale, int causal, int window, void* out, float* lse, void* workspace,
                             size_t ws_bytes, void* stream) {
    wlq_status st;
    if ((st = check_head_dim(head_dim)) != WLQ_OK || (st = check_heads(q_heads, kv_heads)) != WLQ_OK) return st;
    wlq::AttnArgs a;
    std::memset(&a, 0, sizeof a);
    if ((st = check_batch(cu_seqlens, kv_lens, batch, max_q, block_table, table_width, tokens, &a.B)) != WLQ_OK) return st;
    if ((st = check_pool(k_codes, k_scales, v_codes, v_scales, num_pages, page_size, group, kv_heads, head_dim, &a.P)) != WLQ_OK)
        return st;
    if (max_kv < 0) return fail(WLQ_ERR_INVALID_ARG, "max_kv must be >= 0");
    if (!std::isfinite(scale)) return fail(WLQ_ERR_INVALID_ARG, "scale must be finite");
    if (window < 0 || (window > 0 && !causal)) return fail(WLQ_ERR_INVALID_ARG, "a window needs causal and must be >= 0");
    if (static_cast<int64_t>(max_q) * (q_heads / kv_heads) >= (int64_t(1) << 31))
        return fail(WLQ_ERR_SHAPE, "max_q * q_heads / kv_heads must stay below 2^31");
    if (batch == 0 || max_q == 0 || tokens == 0) return WLQ_OK;
    if ((st = check_rows("q", q, q_stride, q_heads, head_dim)) != WLQ_OK) return st;
    if (!out) return fail(WLQ_ERR_INVALID_ARG, "out: null pointer");
    if (!aligned16(out) || !aligned4(lse)) return fail(WLQ_ERR_ALIGN, "out must be 16-byte aligned, lse 4-byte");
    const DecPlan p = dec_plan(tokens, batch, max_q, max_kv, q_heads, kv_heads, head_dim, window, kPlanSms);
    if (p.ws > 0) {
        if (!workspace || ws_bytes < p.ws) return fail(WLQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", p.ws, workspace ? ws_bytes : size_t(0));
        if (!aligned16(workspace)) return fail(WLQ_ERR_ALIGN, "workspace must be 16-byte aligned");
    }
    int dev;
    DeviceInfo* d;
    if ((st = current_device(&dev, &d)) != WLQ_OK) return st;
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.q_heads = q_heads;
    a.share = q_heads / kv_heads;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.causal = causal != 0;
    a.window = window;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.splits = p.splits;
    a.row_tiles = p.row_tiles;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.off_ml);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return head_dim == 128 ? launch_decode<128>(a, p, s) : launch_decode<64>(a, p, s);
}

}  // extern "C"
