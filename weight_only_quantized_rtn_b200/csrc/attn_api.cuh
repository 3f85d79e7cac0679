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

// The cache kernels' grid: a CTA takes a piece of `tpc` tokens of a sequence --
// several where there are enough of them, so that looking up their places (three
// loads that depend on each other) is paid once.
struct KvGrid {
    dim3 grid;
    int tpc, pieces;
};
KvGrid kv_grid(int batch, int max_q, int64_t tokens, int bites, int tpc, int sms) {
    KvGrid g;
    g.tpc = std::min<int64_t>(tokens, static_cast<int64_t>(batch) * max_q) >= 16ll * sms && max_q >= tpc ? tpc : 1;
    g.pieces = static_cast<int>(cdiv(max_q, g.tpc));
    const int64_t units = static_cast<int64_t>(batch) * g.pieces;
    g.grid = dim3(static_cast<unsigned>(units), head_splits(std::min(units, tokens), bites, sms));
    return g;
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

// How a call is cut: the kernel, its row tiles (8 nt rows; 256 of the chunk
// kernel), and the splits of a sequence's cached tokens over CTAs.
constexpr int kPlanSms = 148;  // the SMs of a B200: plans, and with them workspace sizes, need no device

struct DecPlan {
    bool chunk = false, cluster = false;
    int nt = 1, row_tiles = 1, splits = 1;
    int64_t whole = 0, tiles = 0;  // chunk: row tiles in one piece, all row tiles
    size_t off_ml = 0, ws = 0;
};

DecPlan dec_plan(int64_t tokens, int batch, int max_q, int64_t max_kv, int q_heads, int kv_heads, int head_dim, bool causal,
                 int window, int sms) {
    DecPlan p;
    const int64_t rows = static_cast<int64_t>(max_q) * (q_heads / kv_heads);
    // Up to 32 rows the few-row kernel, which reads the cache once for each 16 (8 sequences of 8192, 1 of 32768, 32 of
    // 1500 tokens, 8 cache heads, D = 128, groups of 64: 71, 41, 59 us against 77, 47, 62 by the chunk kernel; 48 rows: 104,
    // 53, 86 against 77, 48, 63).
    p.chunk = rows > 32;
    p.nt = rows > 8 ? 2 : 1;
    p.row_tiles = static_cast<int>(cdiv(rows, p.chunk ? 2 * wlq::CH_ROWS : 8 * p.nt));
    int64_t seen = std::min(std::max<int64_t>(max_kv, 1), int64_t(1) << 31);  // a bound beyond what a length can be is none
    if (window > 0) seen = std::min<int64_t>(seen, static_cast<int64_t>(window) + max_q);
    const int64_t base = static_cast<int64_t>(batch) * kv_heads * p.row_tiles;
    const int64_t units = cdiv(seen, p.chunk ? wlq::CH_KEYS : wlq::DEC_UNIT);
    if (p.chunk) {
        // One CTA an SM: whole rounds of row tiles stay in one piece, those of the last round are split over its SMs, with
        // at least four steps a part (1560 queries over 7800 tokens, D = 128: 154 tiles 194 us against 282, 196 tiles 225
        // against 302, 448 tiles 472 against 581; over 3120: 154 tiles 101 against 127).  Up to 98 of them in three
        // parts, two rounds, where the third saved is worth the parts' traffic (76 left: 288 against 300 us for 61 steps,
        // but 151 against 138 for 25).  Causal prompts end with their shortest tiles: those stay whole.
        p.tiles = base;
        p.whole = base / sms * sms;
        const int64_t tail = base - p.whole;
        const bool uneven = causal && static_cast<int64_t>(max_q) * 2 > max_kv;
        if (tail > 0 && tail * 2 <= sms && (p.whole == 0 || !uneven))
            p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({sms / tail, units / 4, 32})));
        else if (tail > 0 && tail * 3 <= sms * 2 && units >= 48 && !uneven)
            p.splits = 3;
        if (p.splits == 1) p.whole = base;
    } else {
        // Many sequences: about three rounds of four CTAs an SM, so that ragged ones even out, with at least four
        // units for each warp of a part.  Few: one round (37 parts a head against 111 took 85 us against 100 for two
        // sequences of up to 131072 tokens), with two units for each warp.
        const int64_t want = base >= sms ? std::min<int64_t>(cdiv(12ll * sms, base), units / (4 * wlq::DEC_WARPS))
                                         : std::min<int64_t>(4ll * sms / base, units / (2 * wlq::DEC_WARPS));
        p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, 128)));
        // Short parts are joined by their cluster: no workspace, no second launch (1 sequence of 1560 tokens: 15 us with
        // the host's side against 19).  Long ones run apart: as clusters of four, 64 ragged sequences of up to 8191
        // tokens took 113 us against 109.  (Fewer units, as under a window, never turn a joined plan into one that needs
        // a workspace: a part starts from 8 or 16 units.)
        p.cluster = p.splits > 1 && p.splits <= 8 && units <= 32ll * p.splits;
    }
    if (p.splits > 1 && !p.cluster) {
        const size_t rows_kept = p.chunk ? static_cast<size_t>(p.tiles - p.whole) * (2 * wlq::CH_ROWS) : static_cast<size_t>(tokens) * q_heads;
        const size_t parts = rows_kept * p.splits;
        p.off_ml = align256(parts * head_dim * sizeof(float));
        p.ws = p.off_ml + align256(parts * sizeof(float2));
    }
    return p;
}

template <int D, int NT, int G>
cudaError_t launch_dec(unsigned grid, cudaStream_t s, const wlq::AttnArgs& a, DeviceInfo* d) {
    constexpr size_t smem = wlq::dec_smem_bytes<D, NT, G>();
    constexpr int kid = 64 + (D == 128 ? 6 : 0) + (NT == 2 ? 3 : 0) + (G == 4 ? 2 : G == 2 ? 1 : 0);  // 64..75
    if (!d->smem_set[kid]) {
        const cudaError_t e = cudaFuncSetAttribute(wlq::kv4_decode_kernel<D, NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        d->smem_set[kid] = true;
    }
    if (!a.cluster) return launch_k(wlq::kv4_decode_kernel<D, NT, G>, grid, wlq::DEC_WARPS * 32, smem, s, a);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(wlq::DEC_WARPS * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, wlq::kv4_decode_kernel<D, NT, G>, a);
}

template <int D>
wlq_status launch_attention(const wlq::AttnArgs& a, const DecPlan& p, DeviceInfo* d, cudaStream_t s) {
    const int64_t grid = p.chunk ? p.whole + (p.tiles - p.whole) * p.splits
                                 : static_cast<int64_t>(a.B.batch) * a.P.heads * p.row_tiles * p.splits;
    if (grid >= (int64_t(1) << 31)) return fail(WLQ_ERR_SHAPE, "too many queries in one call");
    const unsigned gx = static_cast<unsigned>(grid);
    cudaError_t e;
    if (p.chunk) {
        const int kid = D == 128 ? 55 : 54;
        if (!d->smem_set[kid]) {
            e = cudaFuncSetAttribute(wlq::kv4_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(wlq::ch_smem_bytes<D>()));
            if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
            d->smem_set[kid] = true;
        }
        e = launch_k(wlq::kv4_chunk_kernel<D>, gx, wlq::CH_THREADS, wlq::ch_smem_bytes<D>(), s, a, kDefaultTimeoutNs);
    } else if (D >> a.P.lg_group == 4) {
        e = p.nt == 1 ? launch_dec<D, 1, 4 * D / 128>(gx, s, a, d) : launch_dec<D, 2, 4 * D / 128>(gx, s, a, d);
    } else if (D >> a.P.lg_group == 2) {
        e = p.nt == 1 ? launch_dec<D, 1, 2>(gx, s, a, d) : launch_dec<D, 2, 2>(gx, s, a, d);
    } else {
        e = p.nt == 1 ? launch_dec<D, 1, 1>(gx, s, a, d) : launch_dec<D, 2, 1>(gx, s, a, d);
    }
    if (e == cudaSuccess && p.splits > 1 && p.chunk) {
        e = launch_k(wlq::kv4_chunk_combine_kernel<D>, static_cast<unsigned>((p.tiles - p.whole) * (2 * wlq::CH_ROWS / 8)), 256, 0, s, a);
    } else if (e == cudaSuccess && p.splits > 1 && !p.cluster) {
        const int64_t units = static_cast<int64_t>(a.B.batch) * a.B.max_q * a.q_heads;
        if (units >= (int64_t(1) << 31)) return fail(WLQ_ERR_SHAPE, "too many queries in one call");
        e = launch_k(wlq::kv4_combine_kernel<D>, static_cast<unsigned>(units), 128, 0, s, a);
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
    const KvGrid g = kv_grid(batch, max_q, tokens, static_cast<int>(2 * cdiv(heads, 32 / (head_dim / 8))), 2, d->sms);
    const dim3 grid = g.grid;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (head_dim == 128)
        e = interleaved ? launch_k(wlq::kv4_append_kernel<128, true>, grid, wlq::KV_THREADS, 0, s, K, V, a, B, P, g.tpc, g.pieces)
                        : launch_k(wlq::kv4_append_kernel<128, false>, grid, wlq::KV_THREADS, 0, s, K, V, a, B, P, g.tpc, g.pieces);
    else
        e = interleaved ? launch_k(wlq::kv4_append_kernel<64, true>, grid, wlq::KV_THREADS, 0, s, K, V, a, B, P, g.tpc, g.pieces)
                        : launch_k(wlq::kv4_append_kernel<64, false>, grid, wlq::KV_THREADS, 0, s, K, V, a, B, P, g.tpc, g.pieces);
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
    const KvGrid g = kv_grid(batch, max_q, tokens, static_cast<int>(cdiv(heads, 32 / (head_dim / 8))), wlq::KV_TPC, d->sms);
    const dim3 grid = g.grid;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint16_t *ko = static_cast<uint16_t*>(k_out), *vo = static_cast<uint16_t*>(v_out);
    const cudaError_t e = head_dim == 128 ? launch_k(wlq::kv4_read_kernel<128>, grid, wlq::KV_THREADS, 0, s, ko, vo, B, P, g.tpc, g.pieces)
                                          : launch_k(wlq::kv4_read_kernel<64>, grid, wlq::KV_THREADS, 0, s, ko, vo, B, P, g.tpc, g.pieces);
    return e == cudaSuccess ? WLQ_OK : cuda_fail(e, "kv4_read launch");
}

size_t wlq_kv4_attention_workspace(int64_t tokens, int batch, int max_q, int64_t max_kv, int q_heads, int kv_heads,
                                   int head_dim) {
    if (tokens <= 0 || batch <= 0 || max_q <= 0 || max_kv < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads ||
        (head_dim != 64 && head_dim != 128))
        return 0;
    return dec_plan(tokens, batch, max_q, max_kv, q_heads, kv_heads, head_dim, false, 0, kPlanSms).ws;
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
    if (!(std::fabs(scale) <= 2e38f)) return fail(WLQ_ERR_INVALID_ARG, "scale must be finite, at most 2e38 in magnitude");  // times log2(e): fp32
    if (window < 0 || (window > 0 && !causal)) return fail(WLQ_ERR_INVALID_ARG, "a window needs causal and must be >= 0");
    if (static_cast<int64_t>(max_q) * (q_heads / kv_heads) >= (int64_t(1) << 31))
        return fail(WLQ_ERR_SHAPE, "max_q * q_heads / kv_heads must stay below 2^31");
    if (batch == 0 || max_q == 0 || tokens == 0) return WLQ_OK;
    if ((st = check_rows("q", q, q_stride, q_heads, head_dim)) != WLQ_OK) return st;
    if (!out) return fail(WLQ_ERR_INVALID_ARG, "out: null pointer");
    if (!aligned16(out) || !aligned4(lse)) return fail(WLQ_ERR_ALIGN, "out must be 16-byte aligned, lse 4-byte");
    const DecPlan p = dec_plan(tokens, batch, max_q, max_kv, q_heads, kv_heads, head_dim, causal != 0, window, kPlanSms);
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
    a.cluster = p.cluster ? 1 : 0;
    a.whole = static_cast<int>(p.whole);
    a.row_tiles = p.row_tiles;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.off_ml);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return head_dim == 128 ? launch_attention<128>(a, p, d, s) : launch_attention<64>(a, p, d, s);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// W8A8 Linear
namespace {

struct I8Plan {
    bool pair = false;
    int bn = 16, NT = 0, MT = 0, S = 1, stages = 0;
    uint32_t b_bytes = 0, stage_bytes = 0;
    size_t smem = 0;
};

I8Plan i8_plan(int64_t M, int64_t N, int64_t K) {
    I8Plan p;
    const int64_t KB = cdiv(K, 128);
    // CTA pairs from half as many 256 x 256 tiles as there are pairs (48 tiles, 768 x 4096 x 4096: 13.5 us against 16.1 by
    // single CTAs; 32 tiles, 512 x 4096 x 4096: 10.6 against 10.1)
    const int64_t pairs = kPlanSms / 2, nt2 = cdiv(N, 256), mt256 = cdiv(M, 256);
    if (nt2 * mt256 * 2 >= pairs) {
        // even token tiles: the count (a few from the least possible) whose rounds of tiles take the fewest columns
        int64_t best = -1;
        for (int64_t t = mt256; t <= mt256 + 3; ++t) {
            const int64_t bn = cdiv(cdiv(M, t), 32) * 32, tiles = nt2 * cdiv(M, bn);
            const int64_t cost = cdiv(tiles, pairs) * (bn + 16);  // 16: what a tile costs beside its columns
            if (best < 0 || cost < best) {
                best = cost;
                p.bn = static_cast<int>(bn);
            }
        }
        p.pair = true;
        p.NT = static_cast<int>(nt2);
        p.b_bytes = static_cast<uint32_t>(p.bn / 2) * 128u;
    } else {
        // Token tiles of 64 to 128: halved while that still leaves SMs without one (256 x 4096 x 4096: four of 64 take
        // 8.8 us, two of 128 with K split in two 12.5).
        int64_t t = cdiv(M, 128);
        while (cdiv(N, 128) * t * 2 <= kPlanSms && cdiv(M, t) >= 128) t *= 2;
        p.bn = static_cast<int>(cdiv(cdiv(M, t), 16) * 16);
        p.NT = static_cast<int>(cdiv(N, 128));
        const int64_t tiles = p.NT * t;
        // K split over a cluster while SMs are idle; no more than 15 clusters of eight fit at once (96 x 2048 x 4096 with
        // 16 of them: 12.6 us, a second round)
        while (p.S * 2 <= 8 && tiles * p.S * 2 <= (p.S * 2 == 8 ? 120 : kPlanSms) && KB >= p.S * 2) p.S *= 2;
        p.b_bytes = static_cast<uint32_t>(p.bn) * 128u;
    }
    p.MT = static_cast<int>(cdiv(M, p.bn));
    p.stage_bytes = wlq::I8_A_BYTES + p.b_bytes;
    p.stages = wlq::I8_MAX_STAGES;
    while (wlq::i8_smem_bytes(p.stages, p.stage_bytes) > kSmemLimit) --p.stages;
    p.smem = wlq::i8_smem_bytes(p.stages, p.stage_bytes);
    return p;
}

template <bool PAIR>
wlq_status launch_i8(const I8Plan& p, const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& ty,
                     const wlq::I8Args& a, DeviceInfo* d, cudaStream_t s) {
    auto kern = wlq::int8_gemm_kernel<PAIR>;
    const int kid = PAIR ? 53 : 52;
    if (!d->smem_set[kid]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemLimit));
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        d->smem_set[kid] = true;
    }
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const int csize = PAIR ? 2 : p.S;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(csize);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    // split tiles: one cluster each; else persistent CTAs (pairs)
    const int clusters = (!PAIR && p.S > 1) ? a.tiles : std::min(a.tiles, d->sms / csize);
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * csize), 1, 1);
    cfg.blockDim = dim3(wlq::I8_THREADS, 1, 1);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tw, tx, ty, a);
    return e == cudaSuccess ? WLQ_OK : cuda_fail(e, "int8 gemm launch");
}

wlq_status check_int8(const void* x, int64_t M, const void* wq, const float* ws, int64_t N, int64_t K, const void* bias,
                      const void* y, int y_dtype, bool* noop) {
    *noop = false;
    if (M < 0 || N < 0) return fail(WLQ_ERR_INVALID_ARG, "M and N must be >= 0");
    if (K <= 0 || K % 16) return fail(WLQ_ERR_SHAPE, "the int8 Linear needs K a positive multiple of 16");
    if (K > 131056) return fail(WLQ_ERR_SHAPE, "K above 131056: a 32-bit sum could overflow");
    if (M > (int64_t(1) << 30) || N > (int64_t(1) << 30)) return fail(WLQ_ERR_SHAPE, "M or N too large");
    if (y_dtype != WLQ_OUT_BF16 && y_dtype != WLQ_OUT_F32) return fail(WLQ_ERR_INVALID_ARG, "bad y_dtype");
    if (M == 0 || N == 0) {
        *noop = true;
        return WLQ_OK;
    }
    if (cdiv(N, 128) * cdiv(M, 16) >= (int64_t(1) << 31)) return fail(WLQ_ERR_SHAPE, "M x N too large");
    if (!x || !wq || !ws || !y) return fail(WLQ_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(x) || !aligned16(wq) || !aligned4(ws) || !aligned2(bias) || !aligned4(y))
        return fail(WLQ_ERR_ALIGN, "x and wq must be 16-byte aligned, ws and y 4-byte, bias 2-byte");
    return WLQ_OK;
}

wlq_status int8_linear_impl(const void* xq, const float* xs, int64_t M, const void* wq, const float* ws, int64_t N, int64_t K,
                            const void* bias, void* y, int y_dtype, DeviceInfo* d, cudaStream_t s) {
    const I8Plan p = i8_plan(M, N, K);
    CUtensorMap tw, tx, ty;
    std::memset(&ty, 0, sizeof ty);
    wlq_status st;
    if ((st = make_map_u8(&tw, wq, N, K, 128)) != WLQ_OK) return st;
    if ((st = make_map_u8(&tx, xq, M, K, p.pair ? p.bn / 2 : p.bn)) != WLQ_OK) return st;
    wlq::I8Args a;
    std::memset(&a, 0, sizeof a);
    a.xs = xs;
    a.ws = ws;
    a.bias = static_cast<const uint16_t*>(bias);
    a.y = y;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.NT = p.NT;
    a.KB = static_cast<int>(cdiv(K, 128));
    a.tiles = p.NT * p.MT;
    a.bn = p.bn;
    a.S = p.S;
    a.stages = p.stages;
    a.b_bytes = p.b_bytes;
    a.stage_bytes = p.stage_bytes;
    a.acc2 = p.pair ? 256u : 128u;
    a.tmem_cols = 2 * a.acc2;
    a.y_f32 = (y_dtype == WLQ_OUT_F32) ? 1 : 0;
    const size_t esize = a.y_f32 ? 4 : 2;
    if (p.S == 1 && p.bn % 32 == 0 && aligned16(y) && (static_cast<size_t>(N) * esize) % 16 == 0) {
        EncodeTiledFn fn = encode_fn();
        if (!fn) return fail(WLQ_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * esize};
        const cuuint32_t box[2] = {32, 32};
        const cuuint32_t estr[2] = {1, 1};
        const CUresult cr = fn(&ty, a.y_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, y, dims, strides, box,
                               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (cr != CUDA_SUCCESS) return fail(WLQ_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(cr));
        a.tma_store = 1;
    }
    a.timeout_ns = kDefaultTimeoutNs;
    return p.pair ? launch_i8<true>(p, tw, tx, ty, a, d, s) : launch_i8<false>(p, tw, tx, ty, a, d, s);
}

wlq_status launch_quantize_tokens(const void* x, int64_t M, int64_t K, int8_t* codes, float* scales, DeviceInfo* d, cudaStream_t s) {
    const int per = static_cast<int>(cdiv(K / 8, 256));
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(M, static_cast<int64_t>(d->sms) * 8));
    const uint16_t* xb = static_cast<const uint16_t*>(x);
    const int m = static_cast<int>(M), k = static_cast<int>(K);
    cudaError_t e;
    if (per <= 1) e = launch_k(wlq::quantize_tokens_kernel<1>, grid, 256, 0, s, xb, m, k, codes, scales);
    else if (per <= 2) e = launch_k(wlq::quantize_tokens_kernel<2>, grid, 256, 0, s, xb, m, k, codes, scales);
    else if (per <= 4) e = launch_k(wlq::quantize_tokens_kernel<4>, grid, 256, 0, s, xb, m, k, codes, scales);
    else if (per <= 8) e = launch_k(wlq::quantize_tokens_kernel<8>, grid, 256, 0, s, xb, m, k, codes, scales);
    else if (per <= 16) e = launch_k(wlq::quantize_tokens_kernel<16>, grid, 256, 0, s, xb, m, k, codes, scales);
    else e = launch_k(wlq::quantize_tokens_kernel<0>, grid, 256, 0, s, xb, m, k, codes, scales);
    return e == cudaSuccess ? WLQ_OK : cuda_fail(e, "quantize_tokens launch");
}

}  // namespace

extern "C" {

wlq_status wlq_int8_linear(const void* xq, const float* xs, int64_t M, const void* wq, const float* ws, int64_t N,
                           int64_t K, const void* bias, void* y, int y_dtype, void* stream) {
    bool noop = false;
    wlq_status st = check_int8(xq, M, wq, ws, N, K, bias, y, y_dtype, &noop);
    if (st != WLQ_OK || noop) return st;
    if (!xs) return fail(WLQ_ERR_INVALID_ARG, "null pointer");
    if (!aligned4(xs)) return fail(WLQ_ERR_ALIGN, "xs must be 4-byte aligned");
    int dev;
    DeviceInfo* d;
    if ((st = current_device(&dev, &d)) != WLQ_OK) return st;
    return int8_linear_impl(xq, xs, M, wq, ws, N, K, bias, y, y_dtype, d, static_cast<cudaStream_t>(stream));
}

size_t wlq_w8a8_workspace(int64_t M, int64_t K) {
    if (M <= 0 || K <= 0 || K % 16) return 0;
    return align256(static_cast<size_t>(M) * static_cast<size_t>(K)) + align256(static_cast<size_t>(M) * 4);
}

wlq_status wlq_w8a8_linear(const void* x, int64_t M, const void* wq, const float* ws, int64_t N, int64_t K,
                           const void* bias, void* y, int y_dtype, void* workspace, size_t ws_bytes, void* stream) {
    bool noop = false;
    wlq_status st = check_int8(x, M, wq, ws, N, K, bias, y, y_dtype, &noop);
    if (st != WLQ_OK || noop) return st;
    const size_t need = wlq_w8a8_workspace(M, K);
    if (!workspace || ws_bytes < need)
        return fail(WLQ_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? ws_bytes : size_t(0));
    if (!aligned16(workspace)) return fail(WLQ_ERR_ALIGN, "workspace must be 16-byte aligned");
    int dev;
    DeviceInfo* d;
    if ((st = current_device(&dev, &d)) != WLQ_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int8_t* codes = static_cast<int8_t*>(workspace);
    float* scales = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256(static_cast<size_t>(M) * static_cast<size_t>(K)));
    if ((st = launch_quantize_tokens(x, M, K, codes, scales, d, s)) != WLQ_OK) return st;
    return int8_linear_impl(codes, scales, M, wq, ws, N, K, bias, y, y_dtype, d, s);
}

}  // extern "C"
