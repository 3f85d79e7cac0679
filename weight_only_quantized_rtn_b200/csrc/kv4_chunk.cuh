// kv4_chunk.cuh -- attention of many queries (prompts, chunks of video tokens)
// over the paged 4-bit cache, on the tcgen05 tensor cores.
//
// A CTA takes 256 rows (tokens x the query heads that share a cache head) as
// two tiles of 128 and walks the cached tokens in tiles of 128:
//   S_t = Q_t K^T   (shared memory x shared memory, fp32 in tensor memory)
//   P_t = exp2(S_t c - m)   as fp16 over S_t's own tensor-memory columns
//   O_t += P_t V    (tensor memory x shared memory), in two halves of 64 tokens
// Roles: two warpgroups of softmax (a thread owns a row: no shuffles), one that
// dequantises keys and one values, one warp that issues MMAs.  While one tile's weights are
// computed the tensor cores work on the other, and on the first half of these
// weights while the second is computed: the issue order is PV_0(j),
// QK_0(j+1), PV_1(j), QK_1(j+1), and since they execute in that order S_t(j+1)
// may overwrite the columns PV_t(j) has read.
//
// K and V tiles are written by the dequantisation warps as fp16 code * scale
// (one rounding) in one layout: rows of 64 inputs (128 bytes, 128-byte
// swizzle), which is the K-major operand of the scores and the MN-major operand
// of the outputs.  (Exact codes would want their scales on the scores, one more
// multiplication each in the warps that set the pace, and on the weights; the
// rounding and that of the weights leave 0.00172 of the result's 2-norm where
// bf16's own output rounding leaves 0.00166.)  A lane takes 16 bytes of codes (32 inputs, one scale); the
// order in which it stores its four 16-byte results alternates with the
// row half, so a quarter warp's stores cover all banks.
//
// A thread holds 64 scores of its row in registers: maximum, weights and their
// sum are taken from there.  The running maximum is lazy, as in kv4_decode.cuh:
// O_t is rescaled only when a half step's maximum passes it by more than 8
// (log2).
//
// Bound: the exponentials (16 a clock and SM) and the tensor cores, which take
// the same time for D = 128: 4 x 512 clocks of MMAs and 2 x 1024 of
// exponentials for 256 rows x 128 tokens.  Measured: 1560 queries over 7800
// tokens, 32 heads, 288 us (691 TFLOP/s; 298 before the 76 of its 224 row tiles
// that a second round of 148 CTAs took were split; 4300 clocks a step, tensor
// pipe 34 % active, exponentials 40 %).  One warpgroup for keys and values took 424 us,
// weights handed over whole 352; 64-column score buffers used in turn, so that
// no softmax waits for PV and QK, 317 to 326 against 309 then: the softmax
// warps set the pace.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "kv4_decode.cuh"
#include "kvcache.cuh"
#include "nvfp4.cuh"
#include "ptx.cuh"

namespace wlq {

constexpr int CH_ROWS = 128;  // rows of a tile
constexpr int CH_KEYS = 128;  // cached tokens of a step
// Two softmax warpgroups, one that dequantises keys, one values, one whose first warp issues MMAs.
constexpr int CH_THREADS = 640;
constexpr int CH_STAGES = 2;
// Registers a thread of each role, moved after the start: 2 x 120 + 2 x 96 + 48 = 5 x 96, what the block was launched with.
constexpr int CH_REGS_SOFTMAX = 120, CH_REGS_DEQUANT = 96, CH_REGS_MMA = 48;
static_assert(2 * CH_REGS_SOFTMAX + 2 * CH_REGS_DEQUANT + CH_REGS_MMA == 5 * 96, "register shares");
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <int D>
__host__ __device__ constexpr uint32_t ch_tile_bytes() { return 128u * D * 2u; }
template <int D>
__host__ __device__ constexpr size_t ch_smem_bytes() { return 1024 + (2 + 2 * CH_STAGES) * ch_tile_bytes<D>() + 256; }

// Low words of shared-memory descriptors (128-byte swizzle, version 1); the
// high word is the same for all of them: eight rows are 1024 bytes apart.
// K-major: the leading offset is unused.  MN-major: rows of 64 MN values (128
// bytes), the next 64 MN values `chunk` bytes away (leading offset).
constexpr uint32_t CH_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo_k(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t saddr, uint32_t chunk) { return ((saddr & 0x3FFFFu) >> 4) | ((chunk >> 4) << 16); }

// mma_ss / mma_ts issued by a converged warp (ptx.cuh, elect_one), descriptors
// given by their low words.
__device__ __forceinline__ void mma_ss_lo(uint32_t on, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(CH_DESC_HI), "r"(on)
        : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t on, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(CH_DESC_HI), "r"(on)
        : "memory");
}
// Cached-token steps [jb, je) of a row tile within the CTA's split.
struct ChRange {
    int jb, je;
    __device__ __forceinline__ bool at(int j) const { return j >= jb && j < je; }
};

// The CTA's row tile and its part of the cached tokens: late row tiles (the longest, where causal) first, a.whole of
// them in one piece, then the others in a.splits parts.
struct ChTile {
    int h, b, rt, split, parts;
    int64_t part;  // first row of the tile's parts
    __device__ __forceinline__ ChTile(const AttnArgs& a, int idx) : split(0), parts(1), part(0) {
        if (idx >= a.whole) {
            const int i = idx - a.whole;
            parts = a.splits;
            split = i % parts;
            idx = a.whole + i / parts;
            part = static_cast<int64_t>(i / parts) * (2 * CH_ROWS);
        }
        h = idx % a.P.heads;
        idx /= a.P.heads;
        b = idx % a.B.batch;
        rt = a.row_tiles - 1 - idx / a.B.batch;
    }
};

// Joins the parts of the split row tiles, in order: a warp for each row.
template <int D>
__global__ void __launch_bounds__(256) kv4_chunk_combine_kernel(const AttnArgs a) {
    constexpr int V = D / 32;
    grid_dependency_sync();
    const int lane = threadIdx.x & 31, r = (blockIdx.x * 8 + (threadIdx.x >> 5)) % (2 * CH_ROWS);
    const ChTile at(a, a.whole + static_cast<int>(blockIdx.x / (2 * CH_ROWS / 8)) * a.splits);
    const int64_t r0 = a.B.cu[at.b], r1 = a.B.cu[at.b + 1];
    if (kv_sequence(r0, r1, a.B.kv_len[at.b], a.B.max_q, a.B.tokens) != KV_OK) return;
    const int row = at.rt * 2 * CH_ROWS + r;
    if (row >= static_cast<int>(r1 - r0) * a.share) return;
    const int64_t head_row = (r0 + row / a.share) * a.q_heads + at.h * a.share + row % a.share, first = (at.part + r) * a.splits;
    const float2* ml = a.part_ml + first;
    const float* po = a.part_o + first * D + lane * V;
    float M = -INFINITY, L = 0.0f, acc[V] = {};
    for (int s = 0; s < a.splits; ++s) M = fmaxf(M, ml[s].x);
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const float2 x = ml[s];
        const float w = M == -INFINITY ? 0.0f : ex2(x.x - M);
        L += w * x.y;
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const float2 o = *reinterpret_cast<const float2*>(po + static_cast<int64_t>(s) * D + k);
            acc[k] += w * o.x;
            acc[k + 1] += w * o.y;
        }
    }
    const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
#pragma unroll
    for (int k = 0; k < V; k += 2)
        *reinterpret_cast<__nv_bfloat162*>(a.out + head_row * D + lane * V + k) = __floats2bfloat162_rn(acc[k] * inv, acc[k + 1] * inv);
    if (a.lse && lane == 0) a.lse[head_row] = L > 0.0f ? (M + __log2f(L)) * 0.6931471805599453f : (L == 0.0f ? -INFINITY : L);
}

template <int D>
__global__ void __launch_bounds__(CH_THREADS, 1) kv4_chunk_kernel(const AttnArgs a, uint64_t timeout_ns) {
    constexpr uint32_t TILE = ch_tile_bytes<D>();
    constexpr uint32_t HALF = 128u * 128u;  // one 64-input column block of a tile
    extern __shared__ uint8_t ch_smem_raw[];
    uint8_t* base = ch_smem_raw + ((1024u - (smem_u32(ch_smem_raw) & 1023u)) & 1023u);
    uint8_t* sq = base;
    uint8_t* sk = base + 2 * TILE;
    uint8_t* sv = sk + CH_STAGES * TILE;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sv + CH_STAGES * TILE);
    uint64_t* kfull = bars;                  // [2]
    uint64_t* kempty = bars + 2;             // [2]
    uint64_t* vfull = bars + 4;              // [2]
    uint64_t* vempty = bars + 6;             // [2]
    uint64_t* sfull = bars + 8;              // [2] scores of tile t are in tensor memory
    uint64_t* pfull = bars + 10;             // [2][2] a half step's weights of tile t are (a barrier for each half: the
                                             // second may be there before the MMA warp has looked for the first)
    uint64_t* pvdone = bars + 14;            // [2][2] O_t has a half step's weights
    uint64_t* qfull = bars + 18;
    uint64_t* drain = bars + 19;
    uint32_t* pbad = reinterpret_cast<uint32_t*>(bars + 20);  // [4 steps][4 warps] a bit for each 16 tokens whose page is out of range
    uint32_t* tmem_slot = pbad + 16;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_sync();
    const ChTile at(a, blockIdx.x);
    const int h = at.h, b = at.b, rt = at.rt;
    const int64_t r0 = a.B.cu[b], r1 = a.B.cu[b + 1];
    const int kv = a.B.kv_len[b];
    const KvRange seq = kv_sequence(r0, r1, kv, a.B.max_q, a.B.tokens);
    if (seq != KV_OK) {
        if (seq == KV_BAD && threadIdx.x == 0) raise_error(ERRBIT_INDEX);
        return;
    }
    const int cover = kv_covered(kv, a.B.table_stride, a.P.page_shift);
    if (cover < kv && threadIdx.x == 0) raise_error(ERRBIT_INDEX);
    const int n = static_cast<int>(r1 - r0), rows = n * a.share, row0 = rt * 2 * CH_ROWS;
    if (row0 >= rows) return;

    ChRange R[2];
    int j0, j1, first_seen;
    {
        int lo, hi, unused;
        seen_range(a, kv - n + row0 / a.share, kv, lo, unused);
        first_seen = lo;
        seen_range(a, kv - n + (min(rows, row0 + 2 * CH_ROWS) - 1) / a.share, kv, unused, hi);
        hi = min(hi, cover);
        const int u0 = lo / CH_KEYS, u1 = hi > 0 ? (hi - 1) / CH_KEYS + 1 : 0, units = max(0, u1 - u0);
        j0 = u0 + static_cast<int>(static_cast<int64_t>(units) * at.split / at.parts);
        j1 = u0 + static_cast<int>(static_cast<int64_t>(units) * (at.split + 1) / at.parts);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int f = row0 + t * CH_ROWS, l = min(rows, f + CH_ROWS) - 1;
            R[t].jb = R[t].je = j1;
            if (f < rows) {
                seen_range(a, kv - n + f / a.share, kv, lo, unused);
                seen_range(a, kv - n + l / a.share, kv, unused, hi);
                R[t].jb = max(j0, lo / CH_KEYS);
                hi = min(hi, cover);
                R[t].je = max(R[t].jb, min(j1, hi > 0 ? (hi - 1) / CH_KEYS + 1 : 0));
            }
        }
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kfull[i], 4);
            mbar_init(&kempty[i], 1);
            mbar_init(&vfull[i], 4);
            mbar_init(&vempty[i], 1);
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[2 * i], 4);
            mbar_init(&pfull[2 * i + 1], 4);
            mbar_init(&pvdone[2 * i], 1);
            mbar_init(&pvdone[2 * i + 1], 1);
        }
        mbar_init(qfull, 8);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 16) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        regs_inc<CH_REGS_SOFTMAX>();
        const int t = warp >> 2, q4 = warp & 3;
        const int row = row0 + t * CH_ROWS + q4 * 32 + lane;
        const bool live = row < rows;
        const int crow = min(row, rows - 1);
        const int64_t token = r0 + crow / a.share;
        const int head = h * a.share + crow % a.share;
        float c;  // scores to powers of two
        {
            // the row's queries: fp16 of q 2^e, into the tile's swizzled rows
            const uint4* p = reinterpret_cast<const uint4*>(a.q + token * a.q_stride + static_cast<int64_t>(head) * D);
            uint4 raw[D / 8];
            uint32_t m2 = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                raw[i] = live ? p[i] : make_uint4(0u, 0u, 0u, 0u);
                m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(raw[i].x & 0x7FFF7FFFu, raw[i].y & 0x7FFF7FFFu),
                                           __vmaxu2(raw[i].z & 0x7FFF7FFFu, raw[i].w & 0x7FFF7FFFu)));
            }
            const int e = row_exponent(max(m2 & 0xFFFFu, m2 >> 16));
            // a negative scale turns the queries round; a factor of zero makes them zero (and stays
            // positive: unseen scores are -inf before it is applied)
            float f = a.scale_log2 < 0.0f ? -pow2f(e) : pow2f(e);
            c = fabsf(a.scale_log2) * pow2f(-e);
            if (c == 0.0f) {
                f = 0.0f;
                c = 1.0f;
            }
            const int r = q4 * 32 + lane;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] = h2_bits(__floats2half2_rn(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f));
                uint8_t* dst = sq + t * TILE + (i / 8) * HALF + r * 128 + (((i & 7) ^ (r & 7)) << 4);
                *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull);
        }
        int lo, hi;
        seen_range(a, kv - n + crow / a.share, kv, lo, hi);
        const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
        const uint32_t s_t = tmem + lane_base + t * 128, o_t = tmem + lane_base + 256 + t * 128;
        float m = -INFINITY, l = 0.0f;
        int done = 0;  // steps of this tile so far
        bool ok = true;
        const ChRange Rt = t ? R[1] : R[0];
        for (int j = Rt.jb; j < Rt.je; ++j, ++done) {
            if (!warp_wait(&sfull[t], done & 1, timeout_ns, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const int k0 = j * CH_KEYS;
            // the step's slot is written again four steps later, when this tile's weights have been used
            const uint4 bad4 = *reinterpret_cast<const uint4*>(pbad + (j & 3) * 4);
            const uint32_t bad = bad4.x | bad4.y | bad4.z | bad4.w;
            const bool inside = __all_sync(0xffffffffu, k0 >= lo && k0 <= hi - CH_KEYS && bad == 0);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                uint32_t v[4][16];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) tmem_ld16(s_t + 64 * half + 16 * ch, v[ch]);
                tmem_wait_ld();
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) reg_pin(v[ch]);
                if (!inside) {
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        // keys of this piece from `first` to `last` are seen
                        const int at = k0 + 64 * half + 16 * ch;
                        const int first = lo - at, last = (bad >> (4 * half + ch) & 1u) ? 0 : hi - at;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < first || i >= last) v[ch][i] = 0xFF800000u;
                    }
                }
                float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        top4[(i / 2) & 3] = fmaxf(top4[(i / 2) & 3], fmaxf(__uint_as_float(v[ch][i]), __uint_as_float(v[ch][i + 1])));
                const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * c;  // c > 0
                const bool move = top > m + ATT_LAZY;  // also from -inf
                if (__any_sync(0xffffffffu, move)) {
                    const float f = move ? ex2(m - top) : 1.0f;  // 0 from -inf
                    if (move) m = top;
                    l *= f;
                    if (done + half > 0) {  // O_t has what came before: the last step's second half, or this one's first
                        if (!warp_wait(&pvdone[2 * t + (half ^ 1)], (done + half - 1) & 1, timeout_ns, abort_flag)) { ok = false; break; }
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < D; d += 16) {
                            uint32_t o[16];
                            tmem_ld16(o_t + d, o);
                            tmem_wait_ld_pin(o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(o_t + d, o);
                        }
                        tmem_wait_st();
                    }
                }
                const float nm = m == -INFINITY ? 0.0f : -m;  // nothing seen yet: every score is -inf
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float p0 = ex2(fmaf(__uint_as_float(v[2 * ch + i / 8][(2 * i) & 15]), c, nm));
                        const float p1 = ex2(fmaf(__uint_as_float(v[2 * ch + i / 8][(2 * i + 1) & 15]), c, nm));
                        sum[0] += p0;
                        sum[1] += p1;
                        pk[i] = h2_bits(__floats2half2_rn(p0, p1));
                    }
                    tmem_st16(s_t + 32 * half + 16 * ch, pk);  // over scores that have been read
                }
                l += sum[0] + sum[1];
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[2 * t + half]);
            }
            if (!ok) break;
        }
        // the row's result
        if (ok && done > 0) ok = warp_wait(&pvdone[2 * t + 1], (done - 1) & 1, timeout_ns, abort_flag);
        if (ok) {
            tc_fence_after();
            const int64_t head_row = token * a.q_heads + head;
            const int64_t part = (at.part + row - row0) * at.parts + at.split;
            const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
            for (int d = 0; d < D; d += 16) {
                uint32_t v[16];
                if (done > 0) {
                    tmem_ld16(o_t + d, v);
                    tmem_wait_ld_pin(v);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = 0;
                }
                if (live && at.parts == 1) {
                    uint32_t o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
                        o[i] = *reinterpret_cast<const uint32_t*>(&y);
                    }
                    uint4* dst = reinterpret_cast<uint4*>(a.out + head_row * D + d);
                    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
                    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
                } else if (live) {
                    uint4* dst = reinterpret_cast<uint4*>(a.part_o + part * D + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dst[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
                __syncwarp();
            }
            if (live) {
                if (at.parts > 1) a.part_ml[part] = make_float2(m, l);
                else if (a.lse) a.lse[head_row] = l > 0.0f ? (m + __log2f(l)) * 0.6931471805599453f : (l == 0.0f ? -INFINITY : l);
            }
            tc_fence_before();
        }
    } else if (warp < 16) {
        // ----------------------------------------------------- dequantisation
        regs_dec<CH_REGS_DEQUANT>();
        const bool isv = warp >= 12;
        constexpr int CPT = D / 32;     // 16-byte pieces of a token's codes
        constexpr int TOK = 128 / CPT;  // tokens the 128 threads take at once
        constexpr int REP = 128 / TOK;  // pieces a thread has of a tile
        const int i = threadIdx.x & 127, piece = i % CPT, tk = i / CPT;
        const int lg = a.P.lg_group, gpr = D >> lg, grp = (piece * 32) >> lg;
        const int shift = a.P.page_shift, pmask = (1 << shift) - 1;
        const uint4* codes = reinterpret_cast<const uint4*>(isv ? a.P.v : a.P.k) + piece;
        const __half* scales = (isv ? a.P.vs : a.P.ks) + grp;
        const int32_t* table = a.B.table + b * a.B.table_stride;
        uint8_t* tiles = isv ? sv : sk;
        uint64_t* full = isv ? vfull : kfull;
        uint64_t* empty = isv ? vempty : kempty;
        int32_t page[REP];  // of the step that is loaded next, as the table has them (-1: none)
        uint4 w[REP];
        __half sc[REP];
        uint32_t bad = 0;  // 16-token pieces with a token whose page is out of range
        auto pages = [&](int j) {
#pragma unroll
            for (int r = 0; r < REP; ++r) {
                const int tok = j * CH_KEYS + tk + r * TOK;
                page[r] = -1;
                if (j < j1 && tok < kv && (tok >> shift) < a.B.table_stride) page[r] = __ldg(table + (tok >> shift));
            }
        };
        // codes and scales of step j (zeros where there is no token)
        auto load = [&](int j) {
            bad = 0;
#pragma unroll
            for (int r = 0; r < REP; ++r) {
                const int tok = j * CH_KEYS + tk + r * TOK;
                const bool is = j < j1 && tok < kv, in = is && kv_page_ok(page[r], a.P.pages);
                if (is && !in) bad |= 1u << ((tk + r * TOK) >> 4);
                w[r] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
                sc[r] = __float2half_rn(0.0f);
                if (in) {
                    const int64_t row = ((static_cast<int64_t>(page[r]) * a.P.heads + h) << shift) + (tok & pmask);
                    w[r] = __ldg(codes + row * CPT);
                    sc[r] = __ldg(scales + row * gpr);
                }
            }
        };
        pages(j0);
        // the first step may begin behind the window, where pages may have been given back: its 16-token pieces before that
        // of the first token seen are taken as no tokens
        const int behind = (first_seen - j0 * CH_KEYS) & ~15;
#pragma unroll
        for (int r = 0; r < REP; ++r)
            if (tk + r * TOK < behind) page[r] = -1;
        load(j0);
        if (behind > 0) bad &= ~0u << (behind >> 4);
        pages(j0 + 1);
        for (int j = j0, it = 0; j < j1; ++j, ++it) {
            const int st = it & 1, ph = (it >> 1) & 1;
            if (!warp_wait(&empty[st], ph ^ 1, timeout_ns, abort_flag)) break;
            uint8_t* tile = tiles + st * TILE + (piece / 2) * HALF;
#pragma unroll
            for (int r = 0; r < REP; ++r) {
                const int tok = tk + r * TOK;
                const uint32_t x[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
                const __half2 s2 = __half2half2(sc[r]);
                const bool odd = CPT == 4 && (piece & 2);  // the other column block: another store order
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t o[4];
                    nibbles_f16(odd ? x[k ^ 2] : x[k], s2, o);
                    const int unit = (piece & 1) * 4 + (odd ? (k ^ 2) : k);
                    *reinterpret_cast<uint4*>(tile + tok * 128 + ((unit ^ (tok & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (!isv) {
                bad = __reduce_or_sync(0xffffffffu, bad);
                if (lane == 0) {
                    pbad[(j & 3) * 4 + warp - 8] = bad;
                    if (bad) raise_error(ERRBIT_INDEX);
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
            load(j + 1);
            pages(j + 2);
        }
    } else {
        // ---------------------------------------------------------------- MMAs
        regs_dec<CH_REGS_MMA>();
        if (warp == 16) {
            constexpr uint32_t id_s = idesc_f16(0, 128, CH_KEYS);
            constexpr uint32_t id_o = idesc_f16(0, 128, D) | (1u << 16);  // B is MN-major
            const uint32_t on = elect_one();
            const uint32_t q_lo = desc_lo_k(smem_u32(sq)), k_lo = desc_lo_k(smem_u32(sk)), v_lo = desc_lo_mn(smem_u32(sv), HALF);
            uint32_t cnt[2] = {0, 0};  // half steps of weights of each tile so far
            bool ok = warp_wait(qfull, 0, timeout_ns, abort_flag);
            auto scores = [&](int t, int it) {  // S_t = Q_t K^T
                const uint32_t qa = q_lo + t * (TILE >> 4), ka = k_lo + (it & 1) * (TILE >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k / 4) * (HALF >> 4) + 2 * (k % 4);
                    mma_ss_lo(on, tmem + t * 128, qa + off, ka + off, id_s, k);
                }
                mma_commit_on(on, &sfull[t]);
            };
            auto outputs = [&](int t, int it, int half) {  // O_t += P_t V over 64 tokens
                const uint32_t va = v_lo + (it & 1) * (TILE >> 4) + half * 4 * 128, pa = tmem + t * 128 + half * 32;
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ts_lo(on, tmem + 256 + t * 128, pa + 8 * k, va + 128 * k, id_o, cnt[t] + k);
                mma_commit_on(on, &pvdone[2 * t + half]);
                ++cnt[t];
            };
            if (ok && j0 < j1) {
                ok = warp_wait(&kfull[0], 0, timeout_ns, abort_flag);
                if (ok) {
                    tc_fence_after();
                    for (int t = 0; t < 2; ++t)
                        if (R[t].at(j0)) scores(t, 0);
                    mma_commit_on(on, &kempty[0]);
                }
            }
            for (int j = j0, it = 0; ok && j < j1; ++j, ++it) {
                const int st = it & 1;
                if (!(ok = warp_wait(&vfull[st], (it >> 1) & 1, timeout_ns, abort_flag))) break;
                const bool more = j + 1 < j1;
                bool knext = false;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (R[t].at(j)) {
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            if (!(ok = warp_wait(&pfull[2 * t + half], (cnt[t] >> 1) & 1, timeout_ns, abort_flag))) break;
                            tc_fence_after();
                            outputs(t, it, half);
                        }
                        if (!ok) break;
                    }
                    if (t == 1) mma_commit_on(on, &vempty[st]);
                    if (more) {
                        if (!knext) {
                            if (!(ok = warp_wait(&kfull[st ^ 1], ((it + 1) >> 1) & 1, timeout_ns, abort_flag))) break;
                            tc_fence_after();
                            knext = true;
                        }
                        if (R[t].at(j + 1)) scores(t, it + 1);
                        if (t == 1) mma_commit_on(on, &kempty[st ^ 1]);
                    }
                }
            }
            // every MMA issued has completed before tensor memory is freed
            mma_commit_on(on, drain);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < timeout_ns) {
            }
        }
        __syncwarp();
    }
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace wlq
