// kv4_decode.cuh -- attention of few queries over the paged 4-bit cache: the
// form for single tokens (and for any call the chunk kernel does not take).
//
// The queries of one cache head that a CTA works on (tokens x the query heads
// that share it, 8 NT rows) stay in registers; the cache streams past once.
// Everything is transposed, so that the cache is the 16-row operand of
// mma.sync m16n8k16 and no row of it is wasted:
//   S^T [16 tokens x 8 rows] = K [16 x D] Q^T,   O^T [16 inputs x 8 rows] += V^T [16 x 16 tokens] P^T.
// A lane reads K as one run of D / 4 codes of two tokens, V as runs of D / 8
// codes of four tokens: the inner dimensions of both products are renumbered
// to what a lane's run holds, so codes go from global memory to MMA operands
// without shared memory.  P^T moves from accumulator to operand layout by one
// movmatrix per 8 x 8 block.
//
// A pair of codes becomes two fp16 by one mask-or (1024 + u, or 1024 + 16 u)
// and one exact subtraction or fma, then one product with the scale: fp16 of
// code * scale, one rounding (2^-11).  Weights exp(x - m) are fp16 (2^-11);
// scores, m, l and the outputs are fp32.
// m follows the running maximum lazily: it is moved only when a score exceeds
// it by more than 8 (in powers of two), so weights stay below 2^8 and most
// steps need one vote instead of a reduction and a rescaling.
//
// Bound: HBM (each cached byte once).  One warp holds a unit of 32 tokens in
// flight while it works on the one before; 4 warps share a CTA's part of the
// sequence, and long sequences are split over CTAs whose partial (m, l, O)
// kv4_combine_kernel joins in split order.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "kvcache.cuh"
#include "ptx.cuh"

namespace wlq {

constexpr int DEC_WARPS = 4;
constexpr int DEC_UNIT = 32;           // tokens of one warp step
constexpr float ATT_LAZY = 8.0f;       // how far a score may pass the running maximum (log2)

struct AttnArgs {
    const uint16_t* q;
    int64_t q_stride;
    int q_heads, share;  // share = q_heads / cache heads
    KvBatch B;
    Kv4Pool P;
    float scale_log2;  // scale * log2(e)
    int causal, window;
    uint16_t* out;
    float* lse;
    float* part_o;   // [tokens * q_heads][splits][D]
    float2* part_ml;  // [tokens * q_heads][splits]: (m, l)
    int splits, row_tiles;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// Four pairs of nibbles of w (nibble i of each half, i = 0..3) as fp16 code * s.
__device__ __forceinline__ void nibbles_f16(uint32_t w, __half2 s, uint32_t (&o)[4]) {
    const __half2 k1032 = bits_h2(0x64086408u), k16 = bits_h2(0x2C002C00u), k72 = bits_h2(0xD480D480u);  // 1032, 1/16, -72
    const uint32_t v = w >> 8;
    o[0] = h2_bits(__hmul2(__hsub2(bits_h2((w & 0x000F000Fu) | 0x64006400u), k1032), s));
    o[1] = h2_bits(__hmul2(__hfma2(bits_h2((w & 0x00F000F0u) | 0x64006400u), k16, k72), s));
    o[2] = h2_bits(__hmul2(__hsub2(bits_h2((v & 0x000F000Fu) | 0x64006400u), k1032), s));
    o[3] = h2_bits(__hmul2(__hfma2(bits_h2((v & 0x00F000F0u) | 0x64006400u), k16, k72), s));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The cached tokens a query at position p of a sequence of kv sees: [lo, hi).
__device__ __forceinline__ void seen_range(const AttnArgs& a, int p, int kv, int& lo, int& hi) {
    lo = 0;
    hi = kv;
    if (a.causal) {
        hi = min(kv, p + 1);
        if (a.window > 0) lo = max(0, p - a.window + 1);
    }
}

// 2^e that puts the largest |q| of a row into [2^14, 2^15) (1 for zero or
// non-finite rows): every bf16 value down to 2^-31 of it is then exact in fp16.
__device__ __forceinline__ int row_exponent(uint32_t absmax_bits16) {
    const int ex = static_cast<int>(absmax_bits16 >> 7);  // biased exponent
    return (absmax_bits16 == 0 || ex == 255) ? 0 : 14 + 127 - max(ex, 1);
}
__device__ __forceinline__ float pow2f(int e) {  // 2^e for e in [-252, 252]: two exact factors
    const int h = e / 2;
    return __uint_as_float(static_cast<uint32_t>(127 + h) << 23) * __uint_as_float(static_cast<uint32_t>(127 + e - h) << 23);
}

template <int D>
struct DecUnit {  // one unit's codes and scales of a lane
    static constexpr int KW = D / 32;  // words of a K run
    static constexpr int VW = D / 64;  // words of a V run
    uint32_t k[4][KW];  // rows g, g + 8 of the two 16-token tiles
    uint32_t v[8][VW];  // tokens 2t, 2t+1, 2t+8, 2t+9 of each tile
    __half ks[4], vs[8];
    bool ok[2];  // the tile's page is in range
};

template <int D>
__device__ __forceinline__ void dec_pages(const AttnArgs& a, int b, int unit, int end, int (&pg)[2]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int tok = unit * DEC_UNIT + 16 * t;
        pg[t] = -1;
        if (tok < end) {  // a tile with a token of the range
            const int64_t e = tok >> a.P.page_shift;
            if (e < a.B.table_stride) pg[t] = a.B.table[b * a.B.table_stride + e];
            if (!kv_page_ok(pg[t], a.P.pages)) {
                raise_error(ERRBIT_INDEX);
                pg[t] = -1;
            }
        }
    }
}

template <int D>
__device__ __forceinline__ void dec_load(const AttnArgs& a, int h, int unit, const int (&pg)[2], int lane, DecUnit<D>& u) {
    const int g = lane >> 2, t = lane & 3;
    const int lg = a.P.lg_group, gpr = D >> lg;  // groups of a row
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        u.ok[m] = pg[m] >= 0;
        const int place = (unit * DEC_UNIT + 16 * m) & ((1 << a.P.page_shift) - 1);
        const int64_t row = ((static_cast<int64_t>(max(pg[m], 0)) * a.P.heads + h) << a.P.page_shift) + place;
        if (u.ok[m]) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint8_t* p = a.P.k + (row + g + 8 * r) * (D / 2) + t * (D / 8);
                if constexpr (D == 128) {
                    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
                    u.k[2 * m + r][0] = x.x; u.k[2 * m + r][1] = x.y; u.k[2 * m + r][2] = x.z; u.k[2 * m + r][3] = x.w;
                } else {
                    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
                    u.k[2 * m + r][0] = x.x; u.k[2 * m + r][1] = x.y;
                }
                u.ks[2 * m + r] = a.P.ks[(row + g + 8 * r) * gpr + ((t * (D / 4)) >> lg)];
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t vr = row + 2 * t + (r & 1) + 8 * (r >> 1);
                const uint8_t* p = a.P.v + vr * (D / 2) + g * (D / 16);
                if constexpr (D == 128) {
                    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
                    u.v[4 * m + r][0] = x.x; u.v[4 * m + r][1] = x.y;
                } else {
                    u.v[4 * m + r][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
                }
                u.vs[4 * m + r] = a.P.vs[vr * gpr + ((g * (D / 8)) >> lg)];
            }
        } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int w = 0; w < D / 32; ++w) u.k[2 * m + r][w] = 0x88888888u;
                u.ks[2 * m + r] = __float2half_rn(0.0f);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
                for (int w = 0; w < D / 64; ++w) u.v[4 * m + r][w] = 0x88888888u;
                u.vs[4 * m + r] = __float2half_rn(0.0f);
            }
        }
    }
}

// Cached rows that were never written may hold any bits: a NaN or infinite
// scale there would survive a weight of zero, so unseen tokens' V scales are
// zeroed with their weights.
template <int D, int NT>
__global__ void __launch_bounds__(DEC_WARPS * 32) kv4_decode_kernel(const AttnArgs a) {
    constexpr int KS = D / 16;  // 16-input steps of the scores, 16-input tiles of the outputs
    __shared__ float sm_o[DEC_WARPS][8 * NT][D + 4];
    __shared__ float2 sm_ml[DEC_WARPS][8 * NT];
    grid_dependency_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    int idx = blockIdx.x;
    const int split = idx % a.splits;
    idx /= a.splits;
    const int rt = idx % a.row_tiles;
    idx /= a.row_tiles;
    const int h = idx % a.P.heads, b = idx / a.P.heads;
    const int64_t r0 = a.B.cu[b], r1 = a.B.cu[b + 1];
    const int kv = a.B.kv_len[b];
    const KvRange seq = kv_sequence(r0, r1, kv, a.B.max_q, a.B.tokens);
    if (seq != KV_OK) {
        if (seq == KV_BAD && threadIdx.x == 0) raise_error(ERRBIT_INDEX);
        return;
    }
    const int n = static_cast<int>(r1 - r0), rows = n * a.share, row0 = rt * 8 * NT;
    if (row0 >= rows) return;
    const int row_last = min(rows, row0 + 8 * NT) - 1;
    // what any row of the tile sees, what all of them see
    int lo, hi, lo_all, hi_all;
    seen_range(a, kv - n + row0 / a.share, kv, lo, hi_all);
    seen_range(a, kv - n + row_last / a.share, kv, lo_all, hi);
    const int u0 = lo / DEC_UNIT, u1 = (hi + DEC_UNIT - 1) / DEC_UNIT, units = max(0, u1 - u0);
    const int ub = u0 + static_cast<int>(static_cast<int64_t>(units) * split / a.splits);
    const int ue = u0 + static_cast<int>(static_cast<int64_t>(units) * (split + 1) / a.splits);

    // queries: row 8 nt + g, inputs t D/4 + 4 j .. + 3 for step j
    uint32_t qf[NT][KS][2];
    float cs[NT][2];  // score factor of this lane's accumulator columns (rows 8 nt + 2 t, + 1)
    int clo[NT][2], chi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = row0 + 8 * nt + g;
        uint2 raw[KS];
        uint32_t m2 = 0;
#pragma unroll
        for (int j = 0; j < KS; ++j) raw[j] = make_uint2(0u, 0u);
        if (row < rows) {
            const uint16_t* p = a.q + (r0 + row / a.share) * a.q_stride + static_cast<int64_t>(h * a.share + row % a.share) * D + t * (D / 4);
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                raw[j] = *reinterpret_cast<const uint2*>(p + 4 * j);
                m2 = __vmaxu2(m2, __vmaxu2(raw[j].x & 0x7FFF7FFFu, raw[j].y & 0x7FFF7FFFu));
            }
        }
        uint32_t mx = max(m2 & 0xFFFFu, m2 >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = row_exponent(mx);
        const float f = pow2f(e);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            qf[nt][j][0] = h2_bits(__floats2half2_rn(__uint_as_float(raw[j].x << 16) * f, __uint_as_float(raw[j].x & 0xFFFF0000u) * f));
            qf[nt][j][1] = h2_bits(__floats2half2_rn(__uint_as_float(raw[j].y << 16) * f, __uint_as_float(raw[j].y & 0xFFFF0000u) * f));
        }
        const float c = a.scale_log2 * pow2f(-e);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            cs[nt][k] = __shfl_sync(0xffffffffu, c, (2 * t + k) * 4);
            const int cr = min(row0 + 8 * nt + 2 * t + k, row_last);
            seen_range(a, kv - n + cr / a.share, kv, clo[nt][k], chi[nt][k]);
        }
    }
    float m[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            m[nt][k] = -INFINITY;
            l[nt][k] = 0.0f;
        }
#pragma unroll
        for (int d = 0; d < KS; ++d)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nt][d][k] = 0.0f;
    }

    DecUnit<D> cur, nxt;
    int pg[2], pn[2];
    int u = ub + warp;
    if (u < ue) {
        dec_pages<D>(a, b, u, hi, pg);
        dec_load<D>(a, h, u, pg, lane, cur);
        if (u + DEC_WARPS < ue) dec_pages<D>(a, b, u + DEC_WARPS, hi, pn);
    }
    for (; u < ue; u += DEC_WARPS) {
        if (u + DEC_WARPS < ue) {
            dec_load<D>(a, h, u + DEC_WARPS, pn, lane, nxt);
            if (u + 2 * DEC_WARPS < ue) dec_pages<D>(a, b, u + 2 * DEC_WARPS, hi, pn);
        }
        const int tok0 = u * DEC_UNIT;
        const bool inside = tok0 >= lo_all && tok0 + DEC_UNIT <= hi_all && cur.ok[0] && cur.ok[1];
        float s[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[mt][nt][k] = 0.0f;
            const __half2 sa = __half2half2(cur.ks[2 * mt]), sb = __half2half2(cur.ks[2 * mt + 1]);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                uint32_t fa[4], fb[4];
                nibbles_f16(cur.k[2 * mt][w], sa, fa);
                nibbles_f16(cur.k[2 * mt + 1][w], sb, fb);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma16816_f16(s[mt][nt], fa[0], fb[0], fa[1], fb[1], qf[nt][2 * w][0], qf[nt][2 * w][1]);
                    mma16816_f16(s[mt][nt], fa[2], fb[2], fa[3], fb[3], qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
                }
            }
        }
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float top = -INFINITY;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float x = s[mt][nt][2 * r + k] * cs[nt][k];
                        if (!inside) {
                            const int tok = tok0 + 16 * mt + 8 * r + g;
                            if (tok < clo[nt][k] || tok >= chi[nt][k] || !cur.ok[mt]) x = -INFINITY;
                        }
                        s[mt][nt][2 * r + k] = x;
                        top = fmaxf(top, x);
                    }
                move |= top > m[nt][k] + ATT_LAZY;
            }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float top = fmaxf(fmaxf(s[0][nt][k], s[0][nt][2 + k]), fmaxf(s[1][nt][k], s[1][nt][2 + k]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    const float mn = fmaxf(m[nt][k], top);
                    const float f = mn == -INFINITY ? 1.0f : ex2(m[nt][k] - mn);
                    m[nt][k] = mn;
                    l[nt][k] *= f;
#pragma unroll
                    for (int d = 0; d < KS; ++d) {
                        o[nt][d][k] *= f;
                        o[nt][d][2 + k] *= f;
                    }
                }
        }
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float p[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float base = m[nt][k] == -INFINITY ? 0.0f : m[nt][k];  // nothing seen yet: x is -inf too
                        p[k] = ex2(s[mt][nt][2 * r + k] - base);
                        l[nt][k] += p[k];
                    }
                    pf[mt][nt][r] = movmatrix(h2_bits(__floats2half2_rn(p[0], p[1])));
                }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            if (!inside) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tok = tok0 + 16 * mt + 2 * t + (r & 1) + 8 * (r >> 1);
                    if (tok >= kv) cur.vs[4 * mt + r] = __float2half_rn(0.0f);
                }
            }
            const __half2 sab = __halves2half2(cur.vs[4 * mt], cur.vs[4 * mt + 1]);
            const __half2 scd = __halves2half2(cur.vs[4 * mt + 2], cur.vs[4 * mt + 3]);
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
                uint32_t ae[4], ao[4], ce[4], co[4];  // even / odd inputs of token pairs (2t, 2t+1), (2t+8, 2t+9)
                const uint32_t va = cur.v[4 * mt][w], vb = cur.v[4 * mt + 1][w], vc = cur.v[4 * mt + 2][w], vd = cur.v[4 * mt + 3][w];
                nibbles_f16(__byte_perm(va, vb, 0x5410), sab, ae);
                nibbles_f16(__byte_perm(va, vb, 0x7632), sab, ao);
                nibbles_f16(__byte_perm(vc, vd, 0x5410), scd, ce);
                nibbles_f16(__byte_perm(vc, vd, 0x7632), scd, co);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816_f16(o[nt][4 * w + i], ae[i], ao[i], ce[i], co[i], pf[mt][nt][0], pf[mt][nt][1]);
            }
        }
        cur = nxt;
    }

    // the warps' parts, then the CTA's
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], off);
            const int r = 8 * nt + 2 * t + k;
            if (g == 0) sm_ml[warp][r] = make_float2(m[nt][k], l[nt][k]);
#pragma unroll
            for (int d = 0; d < KS; ++d) {  // tile d: word d / 4, nibble d % 4 of the run of row g
                const int at = g * (D / 8) + 8 * (d / 4) + 2 * (d % 4);
                *reinterpret_cast<float2*>(&sm_o[warp][r][at]) = make_float2(o[nt][d][k], o[nt][d][2 + k]);
            }
        }
    __syncthreads();
    for (int r = warp; r < 8 * NT && row0 + r < rows; r += DEC_WARPS) {
        float M = -INFINITY, L = 0.0f, w[DEC_WARPS];
#pragma unroll
        for (int i = 0; i < DEC_WARPS; ++i) M = fmaxf(M, sm_ml[i][r].x);
#pragma unroll
        for (int i = 0; i < DEC_WARPS; ++i) {
            w[i] = M == -INFINITY ? 0.0f : ex2(sm_ml[i][r].x - M);
            L += w[i] * sm_ml[i][r].y;
        }
        const int64_t head_row = (r0 + (row0 + r) / a.share) * a.q_heads + h * a.share + (row0 + r) % a.share;
        const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);  // a NaN stays one
#pragma unroll
        for (int d = 2 * lane; d < D; d += 64) {
            float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < DEC_WARPS; ++i) {
                const float2 x = *reinterpret_cast<const float2*>(&sm_o[i][r][d]);
                v.x += w[i] * x.x;
                v.y += w[i] * x.y;
            }
            if (a.splits == 1) {
                const __nv_bfloat162 y = __floats2bfloat162_rn(v.x * inv, v.y * inv);
                *reinterpret_cast<__nv_bfloat162*>(a.out + head_row * D + d) = y;
            } else {
                *reinterpret_cast<float2*>(a.part_o + (head_row * a.splits + split) * D + d) = v;
            }
        }
        if (lane == 0) {
            if (a.splits > 1) a.part_ml[head_row * a.splits + split] = make_float2(M, L);
            else if (a.lse) a.lse[head_row] = L > 0.0f ? (M + __log2f(L)) * 0.6931471805599453f : (L == 0.0f ? -INFINITY : L);
        }
    }
}

// Joins the splits' parts in order: one warp per query and head; grid (units of
// 8 warps) over batch * max_q * q_heads.
template <int D>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const AttnArgs a) {
    grid_dependency_sync();
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int head = static_cast<int>(unit % a.q_heads);
    const int64_t bi = unit / a.q_heads;
    const int b = static_cast<int>(bi / a.B.max_q), i = static_cast<int>(bi % a.B.max_q);
    if (b >= a.B.batch) return;
    const int64_t r0 = a.B.cu[b], r1 = a.B.cu[b + 1];
    if (kv_sequence(r0, r1, a.B.kv_len[b], a.B.max_q, a.B.tokens) != KV_OK || i >= r1 - r0) return;
    const int64_t head_row = (r0 + i) * a.q_heads + head;
    const float2* ml = a.part_ml + head_row * a.splits;
    float M = -INFINITY;
    for (int s = lane; s < a.splits; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    constexpr int V = D / 32;
    float acc[V] = {}, L = 0.0f;
    const float* po = a.part_o + head_row * a.splits * D + lane * V;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const float2 x = ml[s];
        const float w = M == -INFINITY ? 0.0f : ex2(x.x - M);
        L += w * x.y;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += w * po[static_cast<int64_t>(s) * D + k];
    }
    const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
    uint16_t* out = a.out + head_row * D + lane * V;
#pragma unroll
    for (int k = 0; k < V; k += 2)
        *reinterpret_cast<__nv_bfloat162*>(out + k) = __floats2bfloat162_rn(acc[k] * inv, acc[k + 1] * inv);
    if (a.lse && lane == 0) a.lse[head_row] = L > 0.0f ? (M + __log2f(L)) * 0.6931471805599453f : (L == 0.0f ? -INFINITY : L);
}

}  // namespace wlq
