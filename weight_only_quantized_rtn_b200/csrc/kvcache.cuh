// kvcache.cuh -- the steps between an attention layer's projections and its
// attention ("Joy-face_change_optimized" model card: fused ops row, QK-norm +
// 3D RoPE; section 1, the KV-dtype setting, cached keys and values quantized
// with scales per token and head):
//
//   qk_norm_rope_kernel  norms of queries and keys for each head, rotated by
//                        their positions (up to four axes), one pass
//   kv4_append_kernel    the same for keys, then keys and values rounded to
//                        4 bits and written into a paged cache
//   kv4_read_kernel      cached rows back as bf16
//
// Norm and rotation of one row x (a head's D values of one token):
//   r = 1 / sqrt(mean x^2 + eps),  n_d = x_d w_d r,
//   a pair (a, b) of rotated inputs becomes (a c - b s, a s + b c) with
//   c, s = cos, sin of position(axis of the pair) * inv_freq(pair).
// It is evaluated in fp32, within
//   E = 9 * 2^-24 r (|a| + |b|)
// of the real value: c and s are fp64 values rounded once (2^-25 each), r is
// within 5 * 2^-24 (squares exact, at most 7 additions of one-signed terms,
// halved by the root; then the roundings of mean + eps and of the root), x w
// is exact (8 + 8 bits), and there are three more roundings; then it is
// rounded to bf16.  Rows whose squares come near fp32's lower end are lifted
// by a power of two first.
//
// The cache's codes are those of the REAL keys rounded to fp32 and from there
// to bf16 (as a cast from a wider type rounds): a key on the other side of a
// border would change its code by a whole step, so the append has to round as
// any exact evaluation does.  A value that can get
// a code other than 0 (its magnitude is at least a 14th of its group's
// largest) and has a bf16 midpoint within E, about one in three thousand, is
// evaluated again in fp64 and rounded from there.  Doing so for every value
// of every row cost 25 us of 71 for 6240 tokens of 64 heads; the queries and
// keys that stay bf16 do without.
//
// Bound: HBM.  A row is read and written once; 16 (D = 128) or 8 (D = 64)
// lanes hold it, 8 adjacent values each (one 16-byte load), so the norm is a
// shuffle reduction and the half-split partner one shuffle.  A CTA works out
// its token's angles once, in fp64, and walks the token's heads with cos and
// sin in registers.  Measured for 6240 tokens: norm + rotation of 64 heads 45 us
// (205 MB: 0.69 of the copy rate; issue 69 % active, half of the warps that fit
// resident), append of 32 heads 77 us (129 MB; issue 74 % active: norm, rotation
// and the exact rounding of the keys), read back 28 us (129 MB).
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "ptx.cuh"
#include "kvslot.h"
#include "quantize_ext.cuh"

namespace wlq {

constexpr int ROPE_MAX_AXES = 4;
constexpr int ROPE_MAX_PAIRS = 64;
constexpr int KV_THREADS = 128;
// 4-bit cache rows hold values up to this magnitude: with a scale of
// fp16(a / 7) every code times its scale stays finite in fp16.
constexpr float KV4_MAX_ABS = 65280.0f;  // the largest bf16 below 2^16

struct RopeArgs {
    const int32_t* pos;     // [tokens, axes] or null: no rotation
    const float* inv_freq;  // [rot / 2]
    int axes;
    int pairs;                   // rot / 2
    int sec_end[ROPE_MAX_AXES];  // pairs [sec_end[a - 1], sec_end[a]) turn by axis a
    double eps;
};

// One projection's rows: token t, head h at x + t * stride + h * D.
struct HeadRows {
    const uint16_t* x;
    int64_t stride;
    int heads;
    const uint16_t* w;  // [D] norm weight, or null: no norm
    uint16_t* out;      // token t, head h at out + t * out_stride + h * D
    int64_t out_stride;
};

// A paged 4-bit cache: codes [page][head][token][D / 2], scales
// [page][head][token][D / group] fp16.  A word holds 8 codes + 8: input t of
// the word at nibble t / 2 (even t) or 4 + t / 2 (odd t), as in the packed
// int4 weights.
struct Kv4Pool {
    uint8_t* k;
    __half* ks;
    uint8_t* v;
    __half* vs;
    int64_t pages;
    int page_shift;  // log2 of the tokens of a page
    int heads;
    int lg_group;
};

// Sequences of a call: sequence b has tokens cu[b] .. cu[b + 1] of this call,
// the last ones of its kv_len[b] cached tokens, on pages table[b][...].
struct KvBatch {
    const int32_t* cu;
    const int32_t* kv_len;
    const int32_t* table;
    int64_t table_stride;
    int batch;
    int max_q;
    int64_t tokens;  // rows of the token-indexed tensors
};

__device__ __forceinline__ void unpack8(uint4 u, float2 (&f)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t bf16_rn_bits(float y) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

// cos and sin of the token's angles for each pair, fp64 and rounded to fp32.
struct TokenTurns {
    float2 f[ROPE_MAX_PAIRS];
    double2 d[ROPE_MAX_PAIRS];
};
__device__ __forceinline__ void token_turns(const RopeArgs& a, int64_t token, TokenTurns& T, int first = threadIdx.x, int step = KV_THREADS) {
    for (int i = first; i < a.pairs; i += step) {
        int ax = 0;
#pragma unroll
        for (int k = 0; k < ROPE_MAX_AXES - 1; ++k)
            if (k + 1 < a.axes && i >= a.sec_end[k]) ax = k + 1;
        // the angle has up to 32 + 24 bits: the product and what its rounding left off; 1 / (2 pi) as a sum
        // of two doubles.  The turns are then right to about 2^-53 at any position.
        const double pos = static_cast<double>(a.pos[token * a.axes + ax]), freq = static_cast<double>(a.inv_freq[i]);
        const double angle = pos * freq, off = fma(pos, freq, -angle);
        const double t = angle * 0.15915494309189535;
        const double rest = fma(angle, -9.839338337591243e-18, fma(angle, 0.15915494309189535, -t)) + off * 0.15915494309189535;
        double c, s;
        sincospi(2.0 * ((t - rint(t)) + rest), &s, &c);
        T.d[i] = make_double2(c, s);
        T.f[i] = make_float2(static_cast<float>(c), static_cast<float>(s));
    }
}

// Lane l (of the row's D / 8) holds inputs 8 l .. 8 l + 7.
template <int D, bool INTER>
struct RopeLane {
    float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
    int src;    // half-split: the lane with the partners
    int first;  // the lane's first pair, or -1: not rotated
    bool lo;    // half-split: this lane has the pairs' first inputs
    __device__ __forceinline__ void load(const RopeArgs& a, const TokenTurns& T, bool rope, int lane) {
        constexpr int LPR = D / 8, NP = INTER ? 4 : 8;
        const int l = lane & (LPR - 1), base = lane & ~(LPR - 1), h8 = a.pairs >> 3;
        if constexpr (INTER) {
            src = lane;
            lo = false;
            first = rope && 4 * l < a.pairs ? 4 * l : -1;  // pairs is a multiple of 8
        } else {
            lo = l < h8;
            const bool rot = rope && l < 2 * h8;
            src = base + (!rot ? l : lo ? l + h8 : l - h8);
            first = rot ? 8 * (lo ? l : l - h8) : -1;
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            c[i] = 1.0f;
            s[i] = 0.0f;
            if (first >= 0) {
                const float2 v = T.f[first + i];
                c[i] = v.x;
                s[i] = lo ? -v.y : v.y;  // the first of the pair: a c - b s
            }
        }
    }
};

// A row's evaluation (8 values a lane): the products x w, the partners, the
// results in fp32.
// Rows whose mean square and eps leave little of fp32's range below them are
// evaluated as x 2^100 and eps 2^200, which norm to the same values.
constexpr float NORM_LOW = 7.888609052210118e-31f, NORM_UP = 1.2676506002282294e30f;  // 2^-100, 2^100
struct RowEval {
    float2 x[4], p[4], y[4];
    float r;
};
template <int D, bool INTER>
__device__ __forceinline__ uint4 norm_rope_row(uint4 raw, const float2 (&w)[4], bool norm, const RopeArgs& a, const RopeLane<D, INTER>& R,
                                               RowEval& v) {
    constexpr int LPR = D / 8, RM = INTER ? 3 : 7;
    unpack8(raw, v.x);
    v.r = 1.0f;
    if (norm) {
        const float2 q = add_f32x2(add_f32x2(mul_f32x2(v.x[0], v.x[0]), mul_f32x2(v.x[1], v.x[1])),
                                   add_f32x2(mul_f32x2(v.x[2], v.x[2]), mul_f32x2(v.x[3], v.x[3])));
        float ss = q.x + q.y;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        float ms = fmaf(ss, 1.0f / D, static_cast<float>(a.eps));
        if (__any_sync(0xffffffffu, ms < NORM_LOW)) {
            const bool low = ms < NORM_LOW;
            const float up = low ? NORM_UP : 1.0f;
            ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v.x[i] = mul_f32x2(v.x[i], make_float2(up, up));
                ss = fmaf(v.x[i].x, v.x[i].x, fmaf(v.x[i].y, v.x[i].y, ss));
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (low) ms = fmaf(ss, 1.0f / D, static_cast<float>(a.eps * NORM_UP * NORM_UP));
        }
        v.r = __frsqrt_rn(ms);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v.x[i] = mul_f32x2(v.x[i], w[i]);  // exact: 8 x 8 bits
    uint4 out;
    uint32_t* o = reinterpret_cast<uint32_t*>(&out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (INTER) v.p[i] = make_float2(-v.x[i].y, v.x[i].x);  // signs fold into the products
        else v.p[i] = make_float2(__shfl_sync(0xffffffffu, v.x[i].x, R.src), __shfl_sync(0xffffffffu, v.x[i].y, R.src));
        const float c0 = R.c[INTER ? i : (2 * i) & RM], c1 = INTER ? c0 : R.c[(2 * i + 1) & RM];
        const float s0 = R.s[INTER ? i : (2 * i) & RM], s1 = INTER ? s0 : R.s[(2 * i + 1) & RM];
        v.y[i] = make_float2(fmaf(v.x[i].x, c0, v.p[i].x * s0) * v.r, fmaf(v.x[i].y, c1, v.p[i].y * s1) * v.r);
        const __nv_bfloat162 b = __floats2bfloat162_rn(v.y[i].x, v.y[i].y);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return out;
}

// Whether a bf16 midpoint lies within e of y: minus the midpoint above y's
// upper half is those bits with 0x8000 below and the sign turned.
__device__ __forceinline__ bool near_midpoint(float y, float e) {
    return fabsf(y + __uint_as_float((__float_as_uint(y) & 0xFFFF0000u) ^ 0x80008000u)) <= e;
}

// Rounds again, from fp64, the values of at least `least` in magnitude that a
// bf16 midpoint lies close to.  The whole warp; true where any was.
template <int D, bool INTER>
__device__ __forceinline__ bool settle_row(uint4 raw, bool norm, const RopeArgs& a, const RopeLane<D, INTER>& R, const TokenTurns& T,
                                           const RowEval& v, float least, uint4& out) {
    constexpr int LPR = D / 8;
    const float k = v.r * 5.364418029785156e-7f;  // 9 * 2^-24 r
    bool near = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        near |= near_midpoint(v.y[i].x, (fabsf(v.x[i].x) + fabsf(v.p[i].x)) * k) && fabsf(v.y[i].x) >= least;
        near |= near_midpoint(v.y[i].y, (fabsf(v.x[i].y) + fabsf(v.p[i].y)) * k) && fabsf(v.y[i].y) >= least;
    }
    if (!__any_sync(0xffffffffu, near)) return false;
    double r64 = 1.0;
    if (norm) {
        double ss = 0.0;
        float2 f[4];
        unpack8(raw, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ss = fma(static_cast<double>(f[i].x), static_cast<double>(f[i].x), ss);
            ss = fma(static_cast<double>(f[i].y), static_cast<double>(f[i].y), ss);
        }
#pragma unroll
        for (int j = LPR / 2; j > 0; j >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, j);
        // two Newton steps from the fp32 root: 2^-22 -> 2^-43 -> fp64's own rounding
        r64 = static_cast<double>(v.r);
        double h = 0.5 * (ss / D + a.eps);
        if (h * r64 * r64 < 0.25) h *= static_cast<double>(NORM_UP) * NORM_UP;  // a lifted row (1/2 otherwise)
        r64 = r64 * fma(-h * r64, r64, 1.5);
        r64 = r64 * fma(-h * r64, r64, 1.5);
    }
    if (near) {
        uint32_t* o = reinterpret_cast<uint32_t*>(&out);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float xi = (i & 1) ? v.x[i / 2].y : v.x[i / 2].x, pi = (i & 1) ? v.p[i / 2].y : v.p[i / 2].x;
            const float yi = (i & 1) ? v.y[i / 2].y : v.y[i / 2].x;
            if (!near_midpoint(yi, (fabsf(xi) + fabsf(pi)) * k)) continue;
            double c = 1.0, s = 0.0;
            if (R.first >= 0) {
                const double2 t = T.d[R.first + (INTER ? i / 2 : i)];
                c = t.x;
                s = R.lo ? -t.y : t.y;
            }
            const uint32_t b = bf16_rn_bits(static_cast<float>((static_cast<double>(xi) * c + static_cast<double>(pi) * s) * r64));
            o[i / 2] = (i & 1) ? ((o[i / 2] & 0xFFFFu) | (b << 16)) : ((o[i / 2] & 0xFFFF0000u) | b);
        }
    }
    __syncwarp();
    return true;
}

__device__ __forceinline__ void load_weight8(const uint16_t* w, int l, float2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = w ? make_float2(__uint_as_float(static_cast<uint32_t>(__ldg(w + 8 * l + 2 * i)) << 16),
                               __uint_as_float(static_cast<uint32_t>(__ldg(w + 8 * l + 2 * i + 1)) << 16))
                 : make_float2(1.0f, 1.0f);
}

// The rows of one side that this warp takes: bites of RPW heads, every `step`-th
// from `b`; two bites are in flight.
template <int D, bool INTER>
__device__ __forceinline__ void norm_rope_side(const HeadRows& S, int64_t token, int b, int step, bool rope, const RopeArgs& a,
                                               const RopeLane<D, INTER>& R, int lane) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const int l = lane & (LPR - 1);
    const bool plain = !rope && !S.w;  // neither: a copy
    int h = b * RPW + lane / LPR;
    if (b * RPW >= S.heads) return;
    float2 w[4];
    load_weight8(S.w, l, w);
    const uint16_t* x = S.x + token * S.stride + static_cast<int64_t>(h) * D + 8 * l;
    uint16_t* o = S.out + token * S.out_stride + static_cast<int64_t>(h) * D + 8 * l;
    const int hs = step * RPW, left = (S.heads - b * RPW + hs - 1) / hs;  // bites of this warp
    uint4 r0 = h < S.heads ? *reinterpret_cast<const uint4*>(x) : make_uint4(0u, 0u, 0u, 0u);
    for (int i = 0; i < left; ++i) {
        x += hs * D;
        uint4 r1 = make_uint4(0u, 0u, 0u, 0u);
        if (h + hs < S.heads) r1 = *reinterpret_cast<const uint4*>(x);
        RowEval v;
        const uint4 y = plain ? r0 : norm_rope_row<D, INTER>(r0, w, S.w != nullptr, a, R, v);
        if (h < S.heads) *reinterpret_cast<uint4*>(o) = y;
        o += hs * D;
        h += hs;
        r0 = r1;
    }
}

// grid (tokens, splits of the token's rows).
template <int D, bool INTER>
__global__ void __launch_bounds__(KV_THREADS) qk_norm_rope_kernel(const HeadRows q, const HeadRows k, const RopeArgs a,
                                                                  int64_t tokens) {
    constexpr int RPW = 32 / (D / 8);
    __shared__ TokenTurns turns;
    grid_dependency_sync();
    const int64_t token = blockIdx.x;
    const bool rope = a.pos != nullptr;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (rope) token_turns(a, token, turns);
    __syncthreads();
    RopeLane<D, INTER> R;
    R.load(a, turns, rope, lane);
    const int step = gridDim.y * (KV_THREADS / 32), first = blockIdx.y * (KV_THREADS / 32) + warp;
    norm_rope_side<D, INTER>(q, token, first, step, rope, a, R, lane);
    // the keys' bites go on where the queries' ended
    const int bites_q = (q.heads + RPW - 1) / RPW, skip = bites_q % step;
    norm_rope_side<D, INTER>(k, token, first >= skip ? first - skip : first + step - skip, step, rope, a, R, lane);
}

// The cached position of token i of sequence b: its page and place, or -1
// (an offset or page out of range: recorded, nothing is read or written).
struct KvSlot {
    int64_t page;
    int place;
    int64_t row;  // in the token-indexed tensors
};
__device__ __forceinline__ bool kv_slot(const KvBatch& B, const Kv4Pool& P, int b, int i, KvSlot& s) {
    const int64_t r0 = B.cu[b], r1 = B.cu[b + 1], kv_len = B.kv_len[b];
    const KvRange seq = kv_sequence(r0, r1, kv_len, B.max_q, B.tokens);
    if (seq == KV_OK && i >= r1 - r0) return false;
    int64_t entry;
    bool ok = seq == KV_OK && kv_entry(kv_len - (r1 - r0) + i, B.table_stride, P.page_shift, &entry, &s.place) == KV_OK;
    if (ok) {
        s.page = B.table[b * B.table_stride + entry];
        s.row = r0 + i;
        ok = kv_page_ok(s.page, P.pages);
    }
    if (!ok && seq != KV_NONE) raise_error(ERRBIT_INDEX);
    return ok;
}

// Element index of (slot, head) in units of rows of D codes.
__device__ __forceinline__ int64_t kv_row(const Kv4Pool& P, const KvSlot& s, int h) {
    return ((s.page * P.heads + h) << P.page_shift) + s.place;
}

// The scale fp16(a / 7) of a group, a the largest magnitude of bf16 values: the
// fp32 quotient, rounded to nearest (one Newton step on a / 7 with the exact
// remainder), rounds to the fp16 value nearest to the real quotient.  A
// midpoint m of two fp16 values has at most 12 bits; if 7 m is not a, which has
// 8, the two differ by 2^-15 of their size at least, far more than the fp32
// rounding; if it is, the quotient is exact.
__device__ __forceinline__ float kv4_scale(float a) {
    const float q = a * 0.14285714924335480f;
    return __half2float(__float2half_rn(fmaf(fmaf(-7.0f, q, a), 0.14285714924335480f, q)));
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 8 bf16 values of a group with scale s > 0 as a word of the cache.
// code = the integer nearest to x / s, ties to even, exactly: x has 8
// significant bits and s at most 11, so x / s is a half-integer or at least
// 2^-12 away from one.  x * inv (2^-20 off at most) is first rounded to a
// multiple of 2^-14 -- a half-integer if and only if the quotient is one -- by
// the fma's addition of 1.5 * 2^9, then to an integer, ties to even, by the
// step to 1.5 * 2^23 + 8, which leaves code + 8 in the low bits.
// |x / s| is below 7.5 unless s is an fp16 subnormal (its rounding may be
// half of it): then the sums are clamped.
__device__ __forceinline__ uint32_t kv4_quantize(const float2 (&x)[4], float s) {
    const float inv = rcp_approx(s);
    const float2 inv2 = make_float2(inv, inv), m1 = make_float2(768.0f, 768.0f), m2 = make_float2(12582920.0f - 768.0f, 12582920.0f - 768.0f);
    float2 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = add_f32x2(fma_f32x2(x[i], inv2, m1), m2);
    if (s < 6.103515625e-5f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = make_float2(fminf(fmaxf(u[i].x, 12582913.0f), 12582927.0f), fminf(fmaxf(u[i].y, 12582913.0f), 12582927.0f));
    }
    // inputs 0, 4, 1, 5 at the bytes' low nibbles, 2, 6, 3, 7 at the high ones
    const uint32_t lo = __byte_perm(__byte_perm(__float_as_uint(u[0].x), __float_as_uint(u[2].x), 0x0040),
                                    __byte_perm(__float_as_uint(u[0].y), __float_as_uint(u[2].y), 0x0040), 0x5410);
    const uint32_t hi = __byte_perm(__byte_perm(__float_as_uint(u[1].x), __float_as_uint(u[3].x), 0x0040),
                                    __byte_perm(__float_as_uint(u[1].y), __float_as_uint(u[3].y), 0x0040), 0x5410);
    return lo | (hi << 4);
}

// grid (batch * the sequences' pieces of `tpc` tokens, splits of a token's 2 H
// rows): the places of a piece's tokens are looked up side by side, then each
// token's key rows and value rows are taken a warp-sized bite at a time.
constexpr int KV_TPC = 4;  // tokens of a CTA at most

template <int D, bool INTER>
__global__ void __launch_bounds__(KV_THREADS) kv4_append_kernel(const HeadRows k, const HeadRows v, const RopeArgs a,
                                                                const KvBatch B, const Kv4Pool P, int tpc, int pieces) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    __shared__ TokenTurns turns[KV_TPC];
    __shared__ KvSlot slots[KV_TPC];
    grid_dependency_sync();
    const int b = blockIdx.x / pieces, i0 = (blockIdx.x - b * pieces) * tpc;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (LPR - 1), sub = lane / LPR;
    const bool rope = a.pos != nullptr;
    if (threadIdx.x < tpc && !(i0 + static_cast<int>(threadIdx.x) < B.max_q && kv_slot(B, P, b, i0 + threadIdx.x, slots[threadIdx.x])))
        slots[threadIdx.x].page = -1;
    float2 w[4];
    load_weight8(k.w, l, w);
    __syncthreads();
    if (rope) {
        for (int t = 0; t < tpc; ++t)  // the threads go on where the token before ended
            if (slots[t].page >= 0) token_turns(a, slots[t].row, turns[t], (threadIdx.x + KV_THREADS - t * a.pairs % KV_THREADS) % KV_THREADS);
        __syncthreads();
    }
    const int bites_k = (P.heads + RPW - 1) / RPW;
    const int lg8 = P.lg_group - 3;  // log2 of the lanes of a group
    const int step = gridDim.y * (KV_THREADS / 32), first = blockIdx.y * (KV_THREADS / 32) + warp;
    bool bad = false;
    for (int tok = 0; tok < tpc; ++tok) {
        const KvSlot slot = slots[tok];
        if (slot.page < 0) continue;
        auto fetch = [&](int t) {
            const bool isk = t < bites_k;
            const HeadRows& S = isk ? k : v;
            const int h = (isk ? t : t - bites_k) * RPW + sub;
            return t < 2 * bites_k && h < P.heads ? *reinterpret_cast<const uint4*>(S.x + slot.row * S.stride + static_cast<int64_t>(h) * D + 8 * l)
                                                  : make_uint4(0u, 0u, 0u, 0u);
        };
        uint4 next = fetch(first);
        RopeLane<D, INTER> R;
        R.load(a, turns[tok], rope, lane);
        for (int t = first; t < 2 * bites_k; t += step) {
            uint4 raw = next;
            next = fetch(t + step);
            const bool isk = t < bites_k;
            const int h = (isk ? t : t - bites_k) * RPW + sub;
            const bool in = h < P.heads;
            auto group_max = [&](uint4 u) {  // the group's largest magnitude, as bf16 bits
                const uint32_t m2 = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
                uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
                for (int o = (1 << lg8) >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                return m;
            };
            uint32_t m;
            if (isk && (rope || k.w)) {  // the same for the whole warp
                RowEval e;
                const uint4 in_row = raw;
                raw = norm_rope_row<D, INTER>(in_row, w, k.w != nullptr, a, R, e);
                m = group_max(raw);
                if (settle_row<D, INTER>(in_row, k.w != nullptr, a, R, turns[tok], e, __uint_as_float(m << 16) * 0.0625f, raw)) m = group_max(raw);
            } else {
                m = group_max(raw);
            }
            const float amax = __uint_as_float(m << 16);
            const bool gbad = !(amax <= KV4_MAX_ABS);  // too large, an infinity or a NaN
            const float s = gbad ? 0.0f : kv4_scale(amax);
            bad |= gbad && in;
            uint32_t word = 0x88888888u;
            if (s > 0.0f) {
                float2 f[4];
                unpack8(raw, f);
                word = kv4_quantize(f, s);
            }
            if (in) {
                const int64_t row = kv_row(P, slot, h);
                reinterpret_cast<uint32_t*>(isk ? P.k : P.v)[row * LPR + l] = word;
                if ((l & ((1 << lg8) - 1)) == 0)
                    (isk ? P.ks : P.vs)[row * (LPR >> lg8) + (l >> lg8)] = __float2half_rn(s);
            }
        }
    }
    if (bad) raise_error(ERRBIT_NONFINITE);
}

// Eight bf16 values code * scale (one rounding) of a word: codes as fp32 by
// 2^23 + u - (2^23 + 8).
__device__ __forceinline__ uint4 kv4_values(uint32_t word, float s) {
    uint4 out;
    uint32_t* o = reinterpret_cast<uint32_t*>(&out);
    const float2 off = make_float2(-8388616.0f, -8388616.0f), s2 = make_float2(s, s);
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // inputs 2 j (nibble j) and 2 j + 1 (nibble 4 + j)
        const uint32_t v = word >> (4 * j);
        const float2 u = make_float2(__uint_as_float((v & 15u) | 0x4B000000u), __uint_as_float((v >> 16 & 15u) | 0x4B000000u));
        const float2 y = mul_f32x2(add_f32x2(u, off), s2);
        const __nv_bfloat162 p = __floats2bfloat162_rn(y.x, y.y);
        o[j] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return out;
}

template <int D>
__global__ void __launch_bounds__(KV_THREADS) kv4_read_kernel(uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out,
                                                              const KvBatch B, const Kv4Pool P, int tpc, int pieces) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    __shared__ KvSlot slots[KV_TPC];
    grid_dependency_sync();
    const int b = blockIdx.x / pieces, i0 = (blockIdx.x - b * pieces) * tpc;
    if (threadIdx.x < tpc && !(i0 + static_cast<int>(threadIdx.x) < B.max_q && kv_slot(B, P, b, i0 + threadIdx.x, slots[threadIdx.x])))
        slots[threadIdx.x].page = -1;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (LPR - 1), sub = lane / LPR;
    const int step = gridDim.y * (KV_THREADS / 32), bites = (P.heads + RPW - 1) / RPW;
    const int lg8 = P.lg_group - 3;
    for (int tok = 0; tok < tpc; ++tok) {
        const KvSlot slot = slots[tok];
        if (slot.page < 0) continue;
#pragma unroll 2
        for (int t = blockIdx.y * (KV_THREADS / 32) + warp; t < bites; t += step) {  // a bite of key rows and of value rows
            const int h = t * RPW + sub;
            if (h >= P.heads) continue;
            const int64_t row = kv_row(P, slot, h);
            const uint32_t wk = reinterpret_cast<const uint32_t*>(P.k)[row * LPR + l], wv = reinterpret_cast<const uint32_t*>(P.v)[row * LPR + l];
            const float s_k = __half2float(P.ks[row * (LPR >> lg8) + (l >> lg8)]), s_v = __half2float(P.vs[row * (LPR >> lg8) + (l >> lg8)]);
            const int64_t at = (slot.row * P.heads + h) * D + 8 * l;
            *reinterpret_cast<uint4*>(k_out + at) = kv4_values(wk, s_k);
            *reinterpret_cast<uint4*>(v_out + at) = kv4_values(wv, s_v);
        }
    }
}

}  // namespace wlq
