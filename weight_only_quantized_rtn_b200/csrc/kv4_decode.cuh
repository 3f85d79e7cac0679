// kv4_decode.cuh -- attention of few queries over the paged 4-bit cache: the
// form for single tokens (and for any call the chunk kernel does not take).
//
// The queries of one cache head that a CTA works on (tokens x the query heads
// that share it, 8 NT rows) stay in registers; the cache streams past once.
// Everything is transposed, so that the cache is the 16-row operand of
// mma.sync m16n8k16 and no row of it is wasted:
//   S^T [16 tokens x 8 rows] = K [16 x D] Q^T,   O^T [16 inputs x 8 rows] += V^T [16 x 16 tokens] P^T.
//
// The products take the CODES, as exact fp16; no scale is applied to them:
//  - K: 16 bytes of a row are 32 inputs of one group (groups are 32 and more),
//    so the scores of each group are accumulated apart and scaled in fp32;
//  - V: an MMA's 16 outputs lie in one such block too, so the scale goes into
//    the weights: P' = 2^(x - M) vs, one fp16 rounding (2^-11).  The reference
//    M is the running maximum m of the scores plus E - 6, E the exponent of the
//    largest V scale so far, so P' stays below 2^15; l is summed with the same
//    M and cancels it.  That holds while a warp meets only scales within 2^7 of
//    each other: a product that is an fp16 subnormal is then off by at most
//    2^-25 of the largest product of its row and group.
//  - From the first scale further off on, the warp's rows and groups have
//    factors of their own: P' = 2^(x - m) vs f, where f keeps the largest product
//    of THIS row and group between 2^6 and 2^15.  Otherwise one token or group
//    with large values, seen or not, would cost all others their bits.  The
//    factors lie in shared memory; with them alone (no common reference) 64
//    ragged sequences took 120 us against 111, two long ones 88 against 74.
// ldmatrix hands a lane word t of 16 bytes of row g (K), and with .trans the
// 16-bit pieces of two tokens side by side (V): four inputs of a token pair,
// one mask-or and one exact fp16 operation from the MMA's operand.  P^T moves
// from accumulator to operand layout by one movmatrix per 8 x 8 block.
// The maximum is moved lazily: only when a score exceeds it by more than 8 (in
// powers of two), or E grows; most steps need one vote instead of a reduction
// and a rescaling.
//
// A warp keeps two units of 32 tokens in a ring of its own in shared memory
// (cp.async, 16-byte pieces permuted so that ldmatrix meets no bank twice); 4
// warps share a CTA's part of the sequence, and long sequences are split over
// CTAs whose partial (M, l, O) are joined in split order: up to eight short
// parts by their cluster through distributed shared memory, others by
// kv4_combine_kernel.
//
// Bound: none at its limit.  A warp issues 765 instructions for 32 tokens of
// D = 128 (745 before the scales were watched), as many as there are issue
// slots at HBM's rate (748), and with 15 of the 16 warps that fit an SM
// resident issue is 65 % active, the integer pipe, which takes the codes apart,
// 53 %.  Measured: 64 sequences of up to 8191 tokens, 368 MB, 109 us (3.4 TB/s,
// 0.51 of the copy rate); two of up to 131072, 262 MB, 73 us.  Where scales lie
// too far apart for the common reference 126 and 84 us.  Scales on the codes
// and register prefetch took 207 and 136 us.  Feeding K's stored nibbles without
// their exact subtraction (the offsets' sum taken off the scores) left the
// integer work as it is and was no faster.  Registers spilled a thread, of
// D = 128: 8 to 24 bytes for up to 8 rows in groups of 64 and 32, 68 to 256
// bytes for 16 rows.
#pragma once
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "kvcache.cuh"
#include "ptx.cuh"

namespace wlq {

constexpr int DEC_WARPS = 4;
constexpr int DEC_UNIT = 32;           // tokens of one warp step
constexpr float ATT_LAZY = 8.0f;       // how far a score may pass the running maximum (log2)
constexpr int DEC_ROOM = 6;            // P' = weight * V scale * 2^6 against the references: at most 2^(8 + 1 + 6), an fp16 number
constexpr float DEC_TOP = 32768.0f;    // how large P' may get with factors of its own
constexpr float DEC_FMAX = 7.922816251426434e28f;  // 2^96, the largest factor: times a weight (2^8) and a scale (2^13.2) still an fp32 number

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
    float* part_o;   // [tokens * q_heads][splits][D]; many rows: [rows of the split tiles][splits][D]
    float2* part_ml;  // the same without D: (m, l)
    int splits, row_tiles;
    int whole;    // many rows: the row tiles that are not split
    int cluster;  // the splits are the CTAs of a cluster, which joins their parts itself
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// (w & mask) | 0x64006400 in one instruction (as C it becomes two, each with an immediate).
__device__ __forceinline__ __half2 magic_pair(uint32_t w, uint32_t mask) {
    uint32_t o;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(o) : "r"(w), "r"(mask), "r"(0x64006400u));
    return bits_h2(o);
}
// Four pairs of nibbles of w (nibble i of each half, i = 0..3) as fp16 code * s.
__device__ __forceinline__ void nibbles_f16(uint32_t w, __half2 s, uint32_t (&o)[4]) {
    const __half2 k1032 = bits_h2(0x64086408u), k16 = bits_h2(0x2C002C00u), k72 = bits_h2(0xD480D480u);  // 1032, 1/16, -72
    const uint32_t v = w >> 8;
    o[0] = h2_bits(__hmul2(__hsub2(magic_pair(w, 0x000F000Fu), k1032), s));
    o[1] = h2_bits(__hmul2(__hfma2(magic_pair(w, 0x00F000F0u), k16, k72), s));
    o[2] = h2_bits(__hmul2(__hsub2(magic_pair(v, 0x000F000Fu), k1032), s));
    o[3] = h2_bits(__hmul2(__hfma2(magic_pair(v, 0x00F000F0u), k16, k72), s));
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
// At most 2^126, which stays an fp32 number and takes bf16's smallest value,
// 2^-133, to 2^-7.
__device__ __forceinline__ int row_exponent(uint32_t absmax_bits16) {
    const int ex = static_cast<int>(absmax_bits16 >> 7);  // biased exponent
    return (absmax_bits16 == 0 || ex == 255) ? 0 : min(14 + 127 - ex, 126);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }  // -126 <= e <= 127

// 16 bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// Four pairs of nibbles of w (nibble i of each half) as fp16 codes, exact.
__device__ __forceinline__ void nibbles_codes(uint32_t w, uint32_t (&o)[4]) {
    const __half2 k1032 = bits_h2(0x64086408u), k16 = bits_h2(0x2C002C00u), k72 = bits_h2(0xD480D480u);  // 1032, 1/16, -72
    const uint32_t v = w >> 8;
    o[0] = h2_bits(__hsub2(magic_pair(w, 0x000F000Fu), k1032));
    o[1] = h2_bits(__hfma2(magic_pair(w, 0x00F000F0u), k16, k72));
    o[2] = h2_bits(__hsub2(magic_pair(v, 0x000F000Fu), k1032));
    o[3] = h2_bits(__hfma2(magic_pair(v, 0x00F000F0u), k16, k72));
}

constexpr int DEC_STAGES = 2;  // three: 111 us against 109 for 64 ragged sequences, 78 against 73 for two long ones
template <int D, int G>  // G groups a row
struct DecRing {
    static constexpr int ROW = D / 2;                  // bytes of a row's codes
    static constexpr int CODES = DEC_UNIT * ROW;       // of a unit's codes of K or V
    static constexpr int SCALES = DEC_UNIT * G * 2;
    static constexpr int STAGE = 2 * CODES + 2 * SCALES;  // K codes, V codes, K scales, V scales
    static constexpr int BYTES = DEC_WARPS * DEC_STAGES * STAGE;
    // Place of 16-byte piece c of row r: eight rows' same piece lie in eight different bank groups.
    static __device__ __forceinline__ uint32_t at(int r, int c) {
        if constexpr (D == 128) return r * ROW + ((c ^ ((r >> 1) & 3)) << 4);
        else return r * ROW + ((c ^ ((r >> 2) & 1)) << 4);
    }
};
template <int D, int NT>
__host__ __device__ constexpr size_t dec_out_bytes() { return static_cast<size_t>(DEC_WARPS) * 8 * NT * (D + 4) * 4 + DEC_WARPS * 8 * NT * 8; }
// The rings, after them the parts; behind both the warps' factors, [nt][group][8 rows].
template <int D, int NT, int G>
__host__ __device__ constexpr size_t dec_factors_at() {
    return DecRing<D, G>::BYTES > dec_out_bytes<D, NT>() ? DecRing<D, G>::BYTES : dec_out_bytes<D, NT>();
}
template <int D, int NT, int G>
__host__ __device__ constexpr size_t dec_smem_bytes() { return dec_factors_at<D, NT, G>() + DEC_WARPS * NT * G * 8 * sizeof(float); }

// Pages of a unit's two 16-token tiles (0xFFFFFFFF: no token of the range, or out of range).
__device__ __forceinline__ void dec_pages(const AttnArgs& a, const int32_t* table, int unit, int ue, int end, uint32_t (&pg)[2]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int tok = unit * DEC_UNIT + 16 * t, e = tok >> a.P.page_shift;
        pg[t] = 0xFFFFFFFFu;
        if (unit < ue && tok < end && e < a.B.table_stride) pg[t] = static_cast<uint32_t>(__ldg(table + e));
    }
}

// What a lane needs to fetch units: its pieces of the pool's first page of this
// head, and how far a page and a token are.
template <int D, int G>
struct DecFetch {
    using R = DecRing<D, G>;
    static constexpr int CPR = D / 32;    // pieces of a row
    static constexpr int RPI = 32 / CPR;  // rows of one instruction
    const uint8_t *k, *v, *sc;
    uint32_t page_codes, page_scales, npages, pmask;
    uint32_t dst, dst_sc;  // places in a stage
    int sc_tile;           // whose scales this lane fetches (-1: none)
    __device__ __forceinline__ DecFetch(const AttnArgs& a, int h, int lane) {
        const int r0 = lane / CPR, c = lane % CPR;
        const int64_t head = static_cast<int64_t>(h) << a.P.page_shift;
        k = a.P.k + (head + r0) * R::ROW + c * 16;
        v = a.P.v + (head + r0) * R::ROW + c * 16;
        page_codes = static_cast<uint32_t>(a.P.heads << a.P.page_shift) * R::ROW;  // at most 2^30
        page_scales = static_cast<uint32_t>(a.P.heads << a.P.page_shift) * (2 * G);
        npages = static_cast<uint32_t>(a.P.pages);
        pmask = (1u << a.P.page_shift) - 1;
        dst = R::at(r0, c);  // eight rows further the piece's place is the same
        const int which = lane / (4 * G), idx = lane % (4 * G), off = idx % (2 * G);
        sc_tile = lane < 8 * G ? idx / (2 * G) : -1;
        sc = reinterpret_cast<const uint8_t*>(which ? a.P.vs : a.P.ks) + head * (2 * G) + off * 16;
        dst_sc = 2 * R::CODES + which * R::SCALES + idx * 16;
    }
    // A unit's codes and scales on their way into a stage.
    __device__ __forceinline__ void operator()(int unit, const uint32_t (&pg)[2], uint32_t stage) const {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (pg[t] < npages) {
                const uint32_t place = static_cast<uint32_t>(unit * DEC_UNIT + 16 * t) & pmask;
                const uint64_t at = static_cast<uint64_t>(pg[t]) * page_codes + place * R::ROW;
                const uint8_t *kp = k + at, *vp = v + at;
                const uint32_t d = stage + dst + 16 * t * R::ROW;
#pragma unroll
                for (int i = 0; i < 16 / RPI; ++i) {
                    cp_async16(d + i * RPI * R::ROW, kp + i * RPI * R::ROW);
                    cp_async16(d + R::CODES + i * RPI * R::ROW, vp + i * RPI * R::ROW);
                }
                if (sc_tile == t) cp_async16(stage + dst_sc, sc + static_cast<uint64_t>(pg[t]) * page_scales + place * (2 * G));
            }
        }
    }
};

// G fp16 scales of one token, two a word (G == 1: one in both halves).
template <int G>
__device__ __forceinline__ void load_scales(const uint8_t* p, uint32_t (&s)[(G + 1) / 2]) {
    if constexpr (G == 1) {
        s[0] = *reinterpret_cast<const uint16_t*>(p) * 0x10001u;
    } else if constexpr (G == 2) {
        s[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        s[0] = u.x;
        s[1] = u.y;
    }
}
__device__ __forceinline__ float scale_of(const uint32_t* s, int i) {
    return __half2float((i & 1) ? __high2half(bits_h2(s[i / 2])) : __low2half(bits_h2(s[i / 2])));
}

template <int D, int NT, int G>
__global__ void __launch_bounds__(DEC_WARPS * 32, NT == 1 ? 4 : 3) kv4_decode_kernel(const AttnArgs a) {
    using R = DecRing<D, G>;
    constexpr int W = D / 32;           // 32-input blocks of a row
    constexpr int BPG = W / G;          // blocks of a group
    extern __shared__ __align__(128) uint8_t dec_smem[];
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
    const int cover = kv_covered(kv, a.B.table_stride, a.P.page_shift);
    if (cover < kv && threadIdx.x == 0) raise_error(ERRBIT_INDEX);
    const int n = static_cast<int>(r1 - r0), rows = n * a.share, row0 = rt * 8 * NT;
    if (row0 >= rows) return;
    const int row_last = min(rows, row0 + 8 * NT) - 1;
    // what any row of the tile sees, what all of them see
    int lo, hi, lo_all, hi_all;
    seen_range(a, kv - n + row0 / a.share, kv, lo, hi_all);
    seen_range(a, kv - n + row_last / a.share, kv, lo_all, hi);
    hi = min(hi, cover);
    const int u0 = lo / DEC_UNIT, u1 = hi > 0 ? (hi - 1) / DEC_UNIT + 1 : 0, units = max(0, u1 - u0);
    const int ub = u0 + static_cast<int>(static_cast<int64_t>(units) * split / a.splits);
    const int ue = u0 + static_cast<int>(static_cast<int64_t>(units) * (split + 1) / a.splits);

    // the first units on their way
    const uint32_t ring = smem_u32(dec_smem) + warp * DEC_STAGES * R::STAGE;
    const int32_t* table = a.B.table + b * a.B.table_stride;
    const DecFetch<D, G> fetch(a, h, lane);
    uint32_t pg[DEC_STAGES][2];  // pages of the units in flight, in order
#pragma unroll
    for (int i = 0; i < DEC_STAGES; ++i) dec_pages(a, table, ub + warp + i * DEC_WARPS, ue, hi, pg[i]);
    // the first tile may lie behind the window: its page may have been given back
    if (ub + warp == u0 && lo >= u0 * DEC_UNIT + 16) pg[0][0] = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < DEC_STAGES - 1; ++i) {
        fetch(ub + warp + i * DEC_WARPS, pg[i], ring + i * R::STAGE);
        cp_async_commit();
    }

    // queries: row 8 nt + g; in 32-input block w, lane t has inputs 8 t .. 8 t + 7 of the block
    uint32_t qf[NT][2 * W][2];
    float cs[NT][2];  // score factor of this lane's accumulator columns (rows 8 nt + 2 t, + 1)
    int clo[NT][2], chi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = row0 + 8 * nt + g;
        uint4 raw[W];
        uint32_t m2 = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) raw[w] = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows) {
            const uint16_t* p = a.q + (r0 + row / a.share) * a.q_stride + static_cast<int64_t>(h * a.share + row % a.share) * D + 8 * t;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                raw[w] = *reinterpret_cast<const uint4*>(p + 32 * w);
                m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(raw[w].x & 0x7FFF7FFFu, raw[w].y & 0x7FFF7FFFu),
                                           __vmaxu2(raw[w].z & 0x7FFF7FFFu, raw[w].w & 0x7FFF7FFFu)));
            }
        }
        uint32_t mx = max(m2 & 0xFFFFu, m2 >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = row_exponent(mx);
        const float f = pow2f(e);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint32_t x[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                qf[nt][2 * w + k / 2][k & 1] = h2_bits(__floats2half2_rn(__uint_as_float(x[k] << 16) * f, __uint_as_float(x[k] & 0xFFFF0000u) * f));
        }
        const float c = a.scale_log2 * pow2f(-e);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            cs[nt][k] = __shfl_sync(0xffffffffu, c, (2 * t + k) * 4);
            const int cr = min(row0 + 8 * nt + 2 * t + k, row_last);
            seen_range(a, kv - n + cr / a.share, kv, clo[nt][k], chi[nt][k]);
        }
    }
    // m: running maximum of the scores; ev: E - 6, E the exponent of the largest V scale so far; M = m + ev
    float m[NT][2], l[NT][2], o[NT][2 * W][4], ev = -24.0f - DEC_ROOM;
    __half2 vtop = bits_h2(0u);             // (twice) 2^E's upper end: a larger scale moves E
    __half2 vlow = bits_h2(0u);             // 2^(E - 6): a smaller scale asks for factors
    __half2 vleast = bits_h2(0x7C007C00u);  // the smallest scales this lane has met
    float* factors = reinterpret_cast<float*>(dec_smem + dec_factors_at<D, NT, G>()) + warp * NT * G * 8 + 2 * t;  // of this lane's rows
    auto factor = [&](int nt, int i) -> float2& { return *reinterpret_cast<float2*>(factors + (nt * G + i) * 8); };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            m[nt][k] = -INFINITY;
            l[nt][k] = 0.0f;
        }
#pragma unroll
        for (int d = 0; d < 2 * W; ++d)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nt][d][k] = 0.0f;
    }

    // ldmatrix rows of this lane.  K, D = 128: matrices are the blocks 0..3 of 8 rows; D = 64: blocks 0, 1 of
    // rows 0..7, then of rows 8..15.  V: blocks (2 i, tokens 0..7), (2 i, 8..15), (2 i + 1, ...), ...
    const int mat = lane >> 3, mr = lane & 7;
    int stage = 0, u = ub + warp;
    bool apart = false;  // the rows and groups have factors of their own
    auto walk = [&](auto apart_tag) {  // the units, until one asks for factors
        constexpr bool APART = decltype(apart_tag)::value;
        bool fetched = APART;  // that unit's copies are there and the next one's on their way
        for (; u < ue; u += DEC_WARPS) {
            // the unit DEC_STAGES - 1 ahead, into the stage read last
            if (!fetched) {
                const int ahead = u + (DEC_STAGES - 1) * DEC_WARPS, st = stage == 0 ? DEC_STAGES - 1 : stage - 1;
                if (ahead < ue) fetch(ahead, pg[DEC_STAGES - 1], ring + st * R::STAGE);
                cp_async_commit();
            }
            fetched = false;
            cp_async_wait<DEC_STAGES - 1>();
            __syncwarp();
            const uint32_t sk = ring + stage * R::STAGE, sv = sk + R::CODES;
            const uint8_t* sc = dec_smem + (sk - smem_u32(dec_smem)) + 2 * R::CODES;
            const int tok0 = u * DEC_UNIT;
            const bool in0 = pg[0][0] < fetch.npages, in1 = pg[0][1] < fetch.npages;
            const bool inside = tok0 >= lo_all && tok0 <= hi_all - DEC_UNIT && in0 && in1;  // (tok0 + 32 may leave 32 bits)
            if (!inside) {  // a page that some row sees a token of (the first row sees the earliest) must be there
                const int first = __shfl_sync(0xffffffffu, clo[0][0], 0);
                if (((!in0 && tok0 + 16 > first && tok0 < hi) || (!in1 && tok0 + 16 < hi)) && lane == 0) raise_error(ERRBIT_INDEX);
            }
            float x[2][NT][4];
            uint32_t vs[2][2][(G + 1) / 2];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                float acc[NT][G][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < G; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[nt][i][k] = 0.0f;
                uint32_t kr[2][W];  // words t of the row's blocks, rows g and g + 8
                if constexpr (D == 128) {
                    uint32_t q0[4], q1[4];
                    ldsm_x4(sk + R::at(16 * mt + mr, mat), q0);
                    ldsm_x4(sk + R::at(16 * mt + 8 + mr, mat), q1);
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        kr[0][w] = q0[w];
                        kr[1][w] = q1[w];
                    }
                } else {
                    uint32_t q[4];
                    ldsm_x4(sk + R::at(16 * mt + 8 * (mat >> 1) + mr, mat & 1), q);
                    kr[0][0] = q[0]; kr[0][1] = q[1]; kr[1][0] = q[2]; kr[1][1] = q[3];
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint32_t fa[4], fb[4];
                    nibbles_codes(kr[0][w], fa);
                    nibbles_codes(kr[1][w], fb);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816_f16(acc[nt][w / BPG], fa[0], fb[0], fa[1], fb[1], qf[nt][2 * w][0], qf[nt][2 * w][1]);
                        mma16816_f16(acc[nt][w / BPG], fa[2], fb[2], fa[3], fb[3], qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
                    }
                }
                uint32_t ks[2][(G + 1) / 2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    load_scales<G>(sc + (16 * mt + 8 * r + g) * G * 2, ks[r]);
                    load_scales<G>(sc + R::SCALES + (16 * mt + 8 * r + g) * G * 2, vs[mt][r]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float s = acc[nt][0][k] * scale_of(ks[k >> 1], 0);
#pragma unroll
                        for (int i = 1; i < G; ++i) s = fmaf(acc[nt][i][k], scale_of(ks[k >> 1], i), s);
                        x[mt][nt][k] = s * cs[nt][k & 1];
                    }
            }
            __half2 least = bits_h2(0x7C007C00u);  // the unit's smallest scales
            if (!inside) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int tok = tok0 + 16 * mt + 8 * (k >> 1) + g;
                            if (tok < clo[nt][k & 1] || tok >= chi[nt][k & 1] || !(mt ? in1 : in0)) x[mt][nt][k] = -INFINITY;
                        }
                // places no token was written to may hold anything
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const bool none = tok0 + 16 * mt + 8 * r + g >= kv || !(mt ? in1 : in0);
#pragma unroll
                        for (int i = 0; i < (G + 1) / 2; ++i) {
                            if (none) vs[mt][r][i] = 0;
                            else least = __hmin2(least, bits_h2(vs[mt][r][i]));
                        }
                    }
            }
            bool move = false;
            __half2 vm2 = bits_h2(0u);
            if constexpr (!APART) {
#pragma unroll
                for (int i = 0; i < (G + 1) / 2; ++i)
                    vm2 = __hmax2(vm2, __hmax2(__hmax2(bits_h2(vs[0][0][i]), bits_h2(vs[0][1][i])), __hmax2(bits_h2(vs[1][0][i]), bits_h2(vs[1][1][i]))));
                __half2 vn2 = bits_h2(0x7C007C00u);
#pragma unroll
                for (int i = 0; i < (G + 1) / 2; ++i)
                    vn2 = __hmin2(vn2, __hmin2(__hmin2(bits_h2(vs[0][0][i]), bits_h2(vs[0][1][i])), __hmin2(bits_h2(vs[1][0][i]), bits_h2(vs[1][1][i]))));
                vleast = __hmin2(vleast, inside ? vn2 : least);
                move = !__hble2(vm2, vtop) || !__hbge2(vleast, vlow);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    move |= fmaxf(fmaxf(x[0][nt][k], x[0][nt][2 + k]), fmaxf(x[1][nt][k], x[1][nt][2 + k])) > m[nt][k] + ATT_LAZY;
            if (__any_sync(0xffffffffu, move)) {
                // a new reference: the largest scores, the exponent of the largest V scale
                float step = 0.0f;
                if constexpr (!APART) {
                    const uint32_t vmax = __reduce_max_sync(0xffffffffu, max(h2_bits(vm2) & 0xFFFFu, h2_bits(vm2) >> 16));
                    int e = static_cast<int>(ev);
                    if (vmax > (h2_bits(vtop) & 0xFFFFu)) {
                        const uint32_t top = vmax | 0x03FFu;  // up to the next power of two (subnormals: 2^-14)
                        e = max(static_cast<int>(top >> 10), 1) - 15 - DEC_ROOM;
                        vtop = bits_h2(top * 0x10001u);
                        vlow = __float2half2_rn(pow2f(e));
                    }
                    if (__any_sync(0xffffffffu, !__hbge2(vleast, vlow))) {
                        apart = true;
                        return;
                    }
                    step = static_cast<float>(e) - ev;
                    ev = static_cast<float>(e);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float top = fmaxf(fmaxf(x[0][nt][k], x[0][nt][2 + k]), fmaxf(x[1][nt][k], x[1][nt][2 + k]));
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                        const float mn = fmaxf(m[nt][k], top);
                        const float fall = mn == -INFINITY ? 1.0f : ex2(m[nt][k] - mn - step);
                        m[nt][k] = mn;
                        l[nt][k] *= fall;
                        if constexpr (!APART) {
#pragma unroll
                            for (int d = 0; d < 2 * W; ++d) {
                                o[nt][d][k] *= fall;
                                o[nt][d][2 + k] *= fall;
                            }
                        } else {  // what o holds stays, its factors grow as the weights fall
#pragma unroll
                            for (int i = 0; i < G; ++i) {
                                float& f = k ? factor(nt, i).y : factor(nt, i).x;
                                const float was = f, grown = was / fall;  // from -inf: infinite, and o is 0
                                const float keep = grown <= DEC_FMAX ? 1.0f : DEC_FMAX * (fall / was);
#pragma unroll
                                for (int d = 2 * BPG * i; d < 2 * BPG * (i + 1); ++d) {
                                    o[nt][d][k] *= keep;
                                    o[nt][d][2 + k] *= keep;
                                }
                                __syncwarp();  // the row's eight lanes have read it; all write the same
                                f = fminf(grown, DEC_FMAX);
                            }
                        }
                    }
                __syncwarp();
            }
            // weights, then by groups: P' = weight * V scale as the operand of both token halves
            uint32_t pf[2][NT][G][2];
            if constexpr (!APART) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float M[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) M[k] = m[nt][k] == -INFINITY ? 0.0f : m[nt][k] + ev;  // nothing seen yet: x is -inf too
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float p0 = ex2(x[mt][nt][2 * r] - M[0]), p1 = ex2(x[mt][nt][2 * r + 1] - M[1]);
                            l[nt][0] += p0;
                            l[nt][1] += p1;
#pragma unroll
                            for (int i = 0; i < G; ++i) {
                                const float v = scale_of(vs[mt][r], i);
                                pf[mt][nt][i][r] = movmatrix(h2_bits(__floats2half2_rn(p0 * v, p1 * v)));
                            }
                        }
                }
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {  // the scores become weights
                            const float mk = m[nt][k & 1];
                            x[mt][nt][k] = ex2(x[mt][nt][k] - (mk == -INFINITY ? 0.0f : mk));
                            l[nt][k & 1] += x[mt][nt][k];
                        }
#pragma unroll
                    for (int i = 0; i < G; ++i) {
                        float2 f = factor(nt, i), top = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float v = scale_of(vs[mt][r], i);
                                top.x = fmaxf(top.x, x[mt][nt][2 * r] * v * f.x);
                                top.y = fmaxf(top.y, x[mt][nt][2 * r + 1] * v * f.y);
                            }
                        if (__any_sync(0xffffffffu, fmaxf(top.x, top.y) > DEC_TOP)) {
                            // smaller factors where a product is too large: the largest one to 2^6
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1)
                                top = make_float2(fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, off)), fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, off)));
                            const uint32_t six = (254u + DEC_ROOM) << 23;  // less top's biased exponent: 2^(6 - exponent)
                            const float s0 = top.x > DEC_TOP ? __uint_as_float(six - (__float_as_uint(top.x) & 0x7F800000u)) : 1.0f;
                            const float s1 = top.y > DEC_TOP ? __uint_as_float(six - (__float_as_uint(top.y) & 0x7F800000u)) : 1.0f;
                            f = make_float2(f.x * s0, f.y * s1);
#pragma unroll
                            for (int d = 2 * BPG * i; d < 2 * BPG * (i + 1); ++d) {
                                o[nt][d][0] *= s0;
                                o[nt][d][1] *= s1;
                                o[nt][d][2] *= s0;
                                o[nt][d][3] *= s1;
                            }
                            __syncwarp();
                            factor(nt, i) = f;
                        }
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float v = scale_of(vs[mt][r], i);
                                pf[mt][nt][i][r] = movmatrix(h2_bits(__floats2half2_rn(x[mt][nt][2 * r] * v * f.x, x[mt][nt][2 * r + 1] * v * f.y)));
                            }
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int w2 = 0; w2 < W / 2; ++w2) {
                    uint32_t vr[4];  // block 2 w2: tokens 0..7, 8..15; block 2 w2 + 1
                    ldsm_x4_trans(sv + R::at(16 * mt + 8 * (mat & 1) + mr, 2 * w2 + (mat >> 1)), vr);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int w = 2 * w2 + j;
                        uint32_t fa[4], fb[4];
                        nibbles_codes(vr[2 * j], fa);
                        nibbles_codes(vr[2 * j + 1], fb);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816_f16(o[nt][2 * w], fa[0], fa[1], fb[0], fb[1], pf[mt][nt][w / BPG][0], pf[mt][nt][w / BPG][1]);
                            mma16816_f16(o[nt][2 * w + 1], fa[2], fa[3], fb[2], fb[3], pf[mt][nt][w / BPG][0], pf[mt][nt][w / BPG][1]);
                        }
                    }
                }
            __syncwarp();  // the stage may be written again
            stage = stage == DEC_STAGES - 1 ? 0 : stage + 1;
#pragma unroll
            for (int i = 0; i + 1 < DEC_STAGES; ++i) {
                pg[i][0] = pg[i + 1][0];
                pg[i][1] = pg[i + 1][1];
            }
            dec_pages(a, table, u + DEC_STAGES * DEC_WARPS, ue, hi, pg[DEC_STAGES - 1]);
        }
    };
    walk(std::false_type{});
    if (apart) {
        // from the common reference to factors, which start 2^64 above it (o stays below 2^15 2^31 2^64) and come down to
        // what each row and group needs; then the rest, from that unit on
        const float up = pow2f(64), f = pow2f(64 - static_cast<int>(ev)), inv = pow2f(static_cast<int>(ev));
        ev = 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt][0] *= inv;
            l[nt][1] *= inv;
#pragma unroll
            for (int i = 0; i < G; ++i) factor(nt, i) = make_float2(f, f);
#pragma unroll
            for (int d = 0; d < 2 * W; ++d)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[nt][d][k] *= up;
        }
        __syncwarp();
        walk(std::true_type{});
    }

    // the warps' parts, then the CTA's (over the rings)
    cp_async_wait<0>();
    if (apart) {  // the factors off again
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const float2 f = factor(nt, i);
                const float inv[2] = {1.0f / f.x, 1.0f / f.y};
#pragma unroll
                for (int d = 2 * BPG * i; d < 2 * BPG * (i + 1); ++d)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[nt][d][k] *= inv[k & 1];
            }
    }
    __syncthreads();
    float* sm_o = reinterpret_cast<float*>(dec_smem);                                       // [warps][8 NT][D + 4]
    float2* sm_ml = reinterpret_cast<float2*>(dec_smem + static_cast<size_t>(DEC_WARPS) * 8 * NT * (D + 4) * 4);  // [warps][8 NT]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], off);
            const int r = 8 * nt + 2 * t + k;
            if (g == 0) sm_ml[warp * 8 * NT + r] = make_float2(m[nt][k] + ev, l[nt][k]);
#pragma unroll
            for (int d = 0; d < 2 * W; ++d) {  // block d / 2: nibbles 2 (d & 1) and 2 (d & 1) + 1 of 16-bit piece g
                const int at = 32 * (d / 2) + 8 * (g >> 1) + 4 * (d & 1) + (g & 1);
                float* dst = sm_o + (warp * 8 * NT + r) * (D + 4) + at;
                dst[0] = o[nt][d][k];
                dst[2] = o[nt][d][2 + k];
            }
        }
    __syncthreads();
    const bool join = a.cluster != 0;
    auto finish = [&](int r, int d, float2 v, float M, float L) {  // inputs d, d + 1 of row r's result
        const int64_t head_row = (r0 + (row0 + r) / a.share) * a.q_heads + h * a.share + (row0 + r) % a.share;
        const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);  // a NaN stays one
        *reinterpret_cast<__nv_bfloat162*>(a.out + head_row * D + d) = __floats2bfloat162_rn(v.x * inv, v.y * inv);
        if (d == 0 && a.lse) a.lse[head_row] = L > 0.0f ? (M + __log2f(L)) * 0.6931471805599453f : (L == 0.0f ? -INFINITY : L);
    };
    for (int r = warp; r < 8 * NT && row0 + r < rows; r += DEC_WARPS) {
        float M = -INFINITY, L = 0.0f, w[DEC_WARPS];
#pragma unroll
        for (int i = 0; i < DEC_WARPS; ++i) M = fmaxf(M, sm_ml[i * 8 * NT + r].x);
#pragma unroll
        for (int i = 0; i < DEC_WARPS; ++i) {
            w[i] = M == -INFINITY ? 0.0f : ex2(sm_ml[i * 8 * NT + r].x - M);
            L += w[i] * sm_ml[i * 8 * NT + r].y;
        }
        const int64_t part = ((r0 + (row0 + r) / a.share) * a.q_heads + h * a.share + (row0 + r) % a.share) * a.splits + split;
#pragma unroll
        for (int d = 2 * lane; d < D; d += 64) {
            float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < DEC_WARPS; ++i) {
                const float2 y = *reinterpret_cast<const float2*>(sm_o + (i * 8 * NT + r) * (D + 4) + d);
                v.x += w[i] * y.x;
                v.y += w[i] * y.y;
            }
            if (a.splits == 1) finish(r, d, v, M, L);
            else if (join) *reinterpret_cast<float2*>(sm_o + r * (D + 4) + d) = v;  // over warp 0's part, which this lane has read
            else *reinterpret_cast<float2*>(a.part_o + part * D + d) = v;
        }
        __syncwarp();
        if (lane == 0 && a.splits > 1) (join ? sm_ml[r] : a.part_ml[part]) = make_float2(M, L);
    }
    if (join) {
        // the cluster's parts, in order: a warp for each row
        cluster_sync_all();
        const uint32_t o_at = smem_u32(sm_o), ml_at = smem_u32(sm_ml);
        for (int r = split * DEC_WARPS + warp; r < 8 * NT && row0 + r < rows; r += a.splits * DEC_WARPS) {
            float M = -INFINITY, L = 0.0f;
            for (int i = 0; i < a.splits; ++i) M = fmaxf(M, ld_dsmem_f32(mapa_shared(ml_at + r * 8, i)));
            float2 v[D / 64];
#pragma unroll
            for (int k = 0; k < D / 64; ++k) v[k] = make_float2(0.0f, 0.0f);
            for (int i = 0; i < a.splits; ++i) {
                const uint32_t ml = mapa_shared(ml_at + r * 8, i), o = mapa_shared(o_at + r * (D + 4) * 4, i);
                const float w = M == -INFINITY ? 0.0f : ex2(ld_dsmem_f32(ml) - M);
                L += w * ld_dsmem_f32(ml + 4);
#pragma unroll
                for (int k = 0; k < D / 64; ++k) {
                    v[k].x += w * ld_dsmem_f32(o + (2 * lane + 64 * k) * 4);
                    v[k].y += w * ld_dsmem_f32(o + (2 * lane + 64 * k) * 4 + 4);
                }
            }
#pragma unroll
            for (int k = 0; k < D / 64; ++k) finish(r, 2 * lane + 64 * k, v[k], M, L);
        }
        cluster_sync_all();  // no CTA leaves while its part is being read
    }
}

// Joins the splits' parts: a CTA of four warps per query and head (grid over
// batch * max_q * q_heads), each warp a quarter of the splits in order, then
// the four sums in order.
template <int D>
__global__ void __launch_bounds__(128) kv4_combine_kernel(const AttnArgs a) {
    constexpr int V = D / 32;
    __shared__ float sm[4][D + 1];
    grid_dependency_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = blockIdx.x % a.q_heads, bi = blockIdx.x / a.q_heads;
    const int b = bi / a.B.max_q, i = bi % a.B.max_q;
    const int64_t r0 = a.B.cu[b], r1 = a.B.cu[b + 1];
    if (kv_sequence(r0, r1, a.B.kv_len[b], a.B.max_q, a.B.tokens) != KV_OK || i >= r1 - r0) return;  // the whole CTA
    const int64_t head_row = (r0 + i) * a.q_heads + head;
    const float2* ml = a.part_ml + head_row * a.splits;
    float M = -INFINITY;
    for (int s = lane; s < a.splits; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float acc[V] = {}, L = 0.0f;
    const float* po = a.part_o + head_row * a.splits * D + lane * V;
#pragma unroll 8
    for (int s = warp; s < a.splits; s += 4) {
        const float2 x = ml[s];
        const float w = M == -INFINITY ? 0.0f : ex2(x.x - M);
        L += w * x.y;
        if constexpr (V == 4) {
            const float4 o = *reinterpret_cast<const float4*>(po + static_cast<int64_t>(s) * D);
            acc[0] += w * o.x; acc[1] += w * o.y; acc[2] += w * o.z; acc[3] += w * o.w;
        } else {
            const float2 o = *reinterpret_cast<const float2*>(po + static_cast<int64_t>(s) * D);
            acc[0] += w * o.x; acc[1] += w * o.y;
        }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) sm[warp][lane * V + k] = acc[k];
    if (lane == 0) sm[warp][D] = L;
    __syncthreads();
    L = (sm[0][D] + sm[1][D]) + (sm[2][D] + sm[3][D]);
    const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
    for (int d = 2 * static_cast<int>(threadIdx.x); d < D; d += 256) {
        const float x = (sm[0][d] + sm[1][d]) + (sm[2][d] + sm[3][d]), y = (sm[0][d + 1] + sm[1][d + 1]) + (sm[2][d + 1] + sm[3][d + 1]);
        *reinterpret_cast<__nv_bfloat162*>(a.out + head_row * D + d) = __floats2bfloat162_rn(x * inv, y * inv);
    }
    if (a.lse && threadIdx.x == 0) a.lse[head_row] = L > 0.0f ? (M + __log2f(L)) * 0.6931471805599453f : (L == 0.0f ? -INFINITY : L);
}

}  // namespace wlq
