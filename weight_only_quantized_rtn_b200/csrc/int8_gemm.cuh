// int8_gemm.cuh -- the Linear in 8-bit integers with a scale for each token
// and each output channel (W8A8, the integer form of the pages' int8 Linear):
//   y[m, n] = xs[m] ws[n] sum_k xq[m, k] wq[n, k] + b[n]
//
// quantize_tokens_kernel: bf16 rows to int8 codes and fp32 scales, the row in
// registers (same arithmetic as quantize_ex: bit-identical results).
//
// int8_gemm_kernel: tcgen05.mma kind::i8 (int8 x int8, exact 32-bit sums in
// tensor memory).  The MMA's M is output channels (lane = channel), its N is
// tokens, both operands K-major in shared memory with the 128-byte swizzle.
// A stage holds 128 inputs: four K = 32 MMAs.
//  - PAIR (many tiles): two CTAs share each MMA (256 channels x bn tokens);
//    each loads its 128 channels and half of the tokens, all loads of a stage
//    complete on the first CTA's barrier, whose thread issues the MMAs.  Per
//    SM and stage that is 32 KB for 512 clocks of MMAs; a single CTA with the
//    same tile would need 48 KB.  bn is chosen so that the token tiles are
//    even and the last round of tiles is as full as can be; over the shapes
//    timed (1560 x 16384 x 4096: 75.0 to 75.5 us for every bn from 128 to 256)
//    it hardly matters.
//  - single CTAs otherwise, 128 channels x bn tokens, K split over the S CTAs
//    of a cluster when there are few tiles: the integer partial sums are added
//    through distributed shared memory, in any order the same.
// The accumulator is double-buffered, so a tile's epilogue runs under the next
// tile's MMAs: 32 tokens x 32 channels at a time are scaled in fp32, staged
// and stored (TMA when y's rows are whole 16-byte units).
// Copies and MMAs are issued by converged warps with one elected lane: from one
// lane's divergent code the same tiles took 134 us instead of 87 (1560 x 16384
// x 4096).
//
// Bound: the tensor pipe and the power cap for many tokens (back to back 6240 x
// 4096 x 16384: 273 us, 3.07 POP/s, single launches 264; 1560 x 16384 x 4096:
// 75 us, 2.79 POP/s, twice the sustained bf16 rate, the tensor pipe 72 % active
// and 8.65 of its 9 rounds of tiles filled; the weights pass once for each of
// its ten token tiles and leave L2 on the way: 141 MB read from DRAM where the
// operands have 73), the weights' bytes and the launch for few (16 x 4096 x 4096:
// 6.9 us back to back).  quantize_tokens_kernel: HBM (6240 x 16384: 60 us for
// 306 MB).
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "nvfp4.cuh"
#include "ptx.cuh"
#include "quantize_ext.cuh"

namespace wlq {

constexpr int I8_THREADS = 192;
constexpr int I8_MAX_STAGES = 12;
constexpr uint32_t I8_A_BYTES = 128u * 128u;
constexpr uint32_t I8_EPI_STAGE = 4096 + 1024;  // per epilogue warp: 32 tokens x 32 channels (two bf16 halves or one fp32), a tile's xs

__host__ __device__ constexpr size_t i8_smem_bytes(int stages, uint32_t stage_bytes) {
    return 1024 + static_cast<size_t>(stages) * stage_bytes + 512 + 4 * I8_EPI_STAGE;
}

struct I8Args {
    const float* xs;
    const float* ws;
    const uint16_t* bias;
    void* y;
    int M, N;
    int NT, KB;     // channel tiles (128, or 256 for pairs), 128-input blocks
    int tiles, bn;  // bn: tokens of a tile
    int S;          // K splits (cluster size) of the single-CTA form
    int stages;
    uint32_t b_bytes, stage_bytes, tmem_cols, acc2;  // acc2: column of the second accumulator
    int y_f32, tma_store;
    uint64_t timeout_ns;
};

__host__ __device__ constexpr uint32_t idesc_i8(uint32_t m, uint32_t n) {
    return (2u << 4)           // accumulator s32
           | (1u << 7)         // A s8
           | (1u << 10)        // B s8
           | ((n >> 3) << 17) | ((m >> 4) << 24);
}
constexpr uint32_t I8_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);  // descriptors' high word, as smem_desc_sw128
// Issued by a converged warp (elect_one), descriptors given by their low words.
template <bool PAIR>
__device__ __forceinline__ void mma_i8(uint32_t on, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
            "mov.b64 a, {%1, %5};\n\t"
            "mov.b64 b, {%2, %5};\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %6, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::i8 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(I8_DESC_HI), "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
            "mov.b64 a, {%1, %5};\n\t"
            "mov.b64 b, {%2, %5};\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %6, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::i8 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(I8_DESC_HI), "r"(on)
            : "memory");
}
// A tile into this CTA's shared memory, completing on a barrier of the pair's
// first CTA (its shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster, int32_t c0, int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ int4 ld_dsmem_s32x4(uint32_t cluster_addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

template <bool PAIR>
__global__ void __launch_bounds__(I8_THREADS, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_y, const I8Args a) {
    extern __shared__ uint8_t i8_smem_raw[];
    uint8_t* base = i8_smem_raw + ((1024u - (smem_u32(i8_smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(base + static_cast<size_t>(a.stages) * a.stage_bytes);
    uint64_t* empty = full + I8_MAX_STAGES;
    uint64_t* accfull = empty + I8_MAX_STAGES;  // [2]
    uint64_t* accempty = accfull + 2;           // [2]
    uint64_t* drain = accempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint8_t* epi_stage = reinterpret_cast<uint8_t*>(full) + 512;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], PAIR ? 8 : 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async();
        prefetch_tensormap(&tm_w);
        prefetch_tensormap(&tm_x);
        if (a.tma_store) prefetch_tensormap(&tm_y);
    }
    if (warp == 1) {
        if constexpr (PAIR) tmem_alloc_pair(tmem_slot, a.tmem_cols);
        else tmem_alloc(tmem_slot, a.tmem_cols);
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR || a.S > 1) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_sync();

    const int first_tile = (PAIR || a.S > 1) ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
    const int tile_step = (PAIR || a.S > 1) ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
    // this CTA's K blocks
    const int kb0 = PAIR ? 0 : static_cast<int>(static_cast<int64_t>(a.KB) * rank / a.S);
    const int kb1 = PAIR ? a.KB : static_cast<int>(static_cast<int64_t>(a.KB) * (rank + 1) / a.S);

    if (warp == 0) {
        // a converged warp, one lane of which issues the copies
        const uint32_t on = elect_one();
        uint32_t it = 0, st = 0, ph = 0;
        bool ok = true;
        const uint32_t full0 = PAIR ? mapa_shared(smem_u32(full), 0) : smem_u32(full);
        for (int tile = first_tile; tile < a.tiles && ok; tile += tile_step) {
            const int nt = tile % a.NT, mt = tile / a.NT;
            const int wrow = PAIR ? nt * 256 + static_cast<int>(rank) * 128 : nt * 128;
            const int xrow = PAIR ? mt * a.bn + static_cast<int>(rank) * (a.bn / 2) : mt * a.bn;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                if (!warp_wait(&empty[st], ph ^ 1, a.timeout_ns, abort_flag)) { ok = false; break; }
                uint8_t* sb = base + static_cast<size_t>(st) * a.stage_bytes;
                if (on) {
                    if constexpr (PAIR) {
                        if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * a.stage_bytes);
                        tma_load_2d_pair(sb, &tm_w, full0 + st * 8, kb * 128, wrow);
                        tma_load_2d_pair(sb + I8_A_BYTES, &tm_x, full0 + st * 8, kb * 128, xrow);
                    } else {
                        mbar_arrive_expect_tx(&full[st], a.stage_bytes);
                        tma_load_2d(sb, &tm_w, &full[st], kb * 128, wrow);
                        tma_load_2d(sb + I8_A_BYTES, &tm_x, &full[st], kb * 128, xrow);
                    }
                }
                __syncwarp();
                if (++st == static_cast<uint32_t>(a.stages)) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (lane == 0) {
            // copies still in flight land before the CTA leaves (bounded).  In a pair the first CTA's
            // barrier covers both; the second waits for its stages to be consumed instead.
            const uint32_t n = it < static_cast<uint32_t>(a.stages) ? it : static_cast<uint32_t>(a.stages);
            for (uint32_t i = it - n; i < it; ++i) {
                const uint64_t t0 = globaltimer_ns();
                uint64_t* bar = (PAIR && rank != 0) ? &empty[i % a.stages] : &full[i % a.stages];
                while (!mbar_try_wait(bar, (i / a.stages) & 1) && globaltimer_ns() - t0 < a.timeout_ns) {
                }
            }
        }
    } else if (warp == 1) {
        if (!PAIR || rank == 0) {
            const uint32_t idesc = idesc_i8(PAIR ? 256 : 128, static_cast<uint32_t>(a.bn));
            const uint32_t on = elect_one();
            const uint32_t lo0 = ((smem_u32(base) & 0x3FFFFu) >> 4) | (1u << 16);
            uint32_t st = 0, ph = 0, tc = 0;
            for (int tile = first_tile; tile < a.tiles; tile += tile_step, ++tc) {
                const uint32_t buf = tc & 1;
                if (!warp_wait(&accempty[buf], ((tc >> 1) & 1) ^ 1, a.timeout_ns, abort_flag)) break;
                tc_fence_after();
                const uint32_t acc = tmem + buf * a.acc2;
                bool ok = true;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!warp_wait(&full[st], ph, a.timeout_ns, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t da = lo0 + st * (a.stage_bytes >> 4), db = da + (I8_A_BYTES >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_i8<PAIR>(on, acc, da + 2 * k, db + 2 * k, idesc, static_cast<uint32_t>(kb - kb0) + k);
                    if constexpr (PAIR) mma_commit_pair_both_on(on, &empty[st]);
                    else mma_commit_on(on, &empty[st]);
                    if (++st == static_cast<uint32_t>(a.stages)) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                if (!ok) break;
                if constexpr (PAIR) mma_commit_pair_both_on(on, &accfull[buf]);
                else mma_commit_on(on, &accfull[buf]);
            }
            // every MMA issued has completed before tensor memory is freed.  Signalled in this CTA only: the
            // pair's second CTA does not wait for it, and an arrival may not reach a CTA that has left.
            if constexpr (PAIR) mma_commit_pair_on(on, drain);
            else mma_commit_on(on, drain);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < a.timeout_ns) {
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3;  // TMEM lane quarter this warp may read
        uint8_t* stg = epi_stage + static_cast<size_t>(warp - 2) * I8_EPI_STAGE;
        uint32_t tc = 0, chunk = 0;
        for (int tile = first_tile; tile < a.tiles; tile += tile_step, ++tc) {
            const int nt = tile % a.NT, mt = tile / a.NT;
            const uint32_t buf = tc & 1;
            if (!warp_wait(&accfull[buf], (tc >> 1) & 1, a.timeout_ns, abort_flag)) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * a.acc2 + (static_cast<uint32_t>(q * 32) << 16);
            const int n0 = nt * (PAIR ? 256 : 128) + (PAIR ? static_cast<int>(rank) * 128 : 0) + q * 32, n = n0 + lane;
            const int m0 = mt * a.bn, m_end = min(a.bn, a.M - m0);
            if (!PAIR && a.S > 1) {
                // partial sums, token-major, into the idle ring: [bn][128]
                int* part = reinterpret_cast<int*>(base);
                for (int c0 = 0; c0 < m_end; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld16(acc + c0, v);
                    tmem_wait_ld_pin(v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[(c0 + i) * 128 + q * 32 + lane] = static_cast<int>(v[i]);
                }
                continue;
            }
            const float wsc = n < a.N ? __ldg(a.ws + n) : 0.0f;
            const float bv = (a.bias && n < a.N) ? bf16_bits_to_f32(a.bias[n]) : 0.0f;
            float* xs_s = reinterpret_cast<float*>(stg + 4096);  // this tile's token scales
            __syncwarp();
            for (int i = lane; i < a.bn; i += 32) xs_s[i] = __ldg(a.xs + min(m0 + i, a.M - 1));
            __syncwarp();
            for (int c0 = 0; c0 < m_end; c0 += 32) {
                uint32_t v[2][16];
                tmem_ld16(acc + c0, v[0]);
                if (c0 + 16 < a.bn) tmem_ld16(acc + c0 + 16, v[1]);
                tmem_wait_ld();
                reg_pin(v[0]);
                reg_pin(v[1]);
                float f[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 x4 = *reinterpret_cast<const float4*>(xs_s + c0 + i);
                    const float xs4[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        f[i + k] = fmaf(static_cast<float>(static_cast<int>(v[(i + k) / 16][(i + k) & 15])) * xs4[k], wsc, bv);
                }
                if (a.tma_store) {
                    if (n0 < a.N) {  // the same for the whole warp
                        const bool half = !a.y_f32;  // bf16: two alternating 2 KB halves
                        uint8_t* dst = stg + ((half && (chunk & 1)) ? 2048 : 0);
                        if (lane == 0) {
                            if (half) bulk_wait_read<1>();
                            else bulk_wait_read<0>();
                        }
                        __syncwarp();
                        if (half) {
                            uint16_t* d = reinterpret_cast<uint16_t*>(dst);
#pragma unroll
                            for (int i = 0; i < 32; ++i) d[i * 32 + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
                        } else {
                            float* d = reinterpret_cast<float*>(dst);
#pragma unroll
                            for (int i = 0; i < 32; ++i) d[i * 32 + lane] = f[i];
                        }
                        fence_proxy_async();
                        __syncwarp();
                        // tokens past M are clipped by the store (bn is a multiple of 32 here)
                        if (lane == 0) tma_store_2d(&tm_y, dst, n0, m0 + c0);
                        ++chunk;
                    }
                } else if (n < a.N) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int m = m0 + c0 + i;
                        if (c0 + i < m_end) {
                            if (a.y_f32) static_cast<float*>(a.y)[static_cast<int64_t>(m) * a.N + n] = f[i];
                            else static_cast<uint16_t*>(a.y)[static_cast<int64_t>(m) * a.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR && rank != 0) mbar_arrive_peer(mapa_shared(smem_u32(&accempty[buf]), 0));
                else mbar_arrive(&accempty[buf]);
            }
        }
        if (a.tma_store && lane == 0) bulk_wait_read<0>();
    }

    if (!PAIR && a.S > 1) {
        // one tile per cluster: CTA `rank` adds the parts of its share of the tokens
        tc_fence_before();
        __syncwarp();
        cluster_sync_all();
        const int tile = first_tile, nt = tile % a.NT, mt = tile / a.NT;
        const int m0 = mt * a.bn, m_end = min(a.bn, a.M - m0);
        const int c_lo = m_end * static_cast<int>(rank) / a.S, c_hi = m_end * static_cast<int>(rank + 1) / a.S;
        const uint32_t part = smem_u32(base);
        for (int i = static_cast<int>(threadIdx.x); i < (c_hi - c_lo) * 32; i += I8_THREADS) {
            const int c = c_lo + i / 32, n = nt * 128 + (i % 32) * 4;  // four channels of one token
            int4 s = make_int4(0, 0, 0, 0);
            for (int r = 0; r < a.S; ++r) {
                const int4 v = ld_dsmem_s32x4(mapa_shared(part + static_cast<uint32_t>(c * 128 + (i % 32) * 4) * 4u, static_cast<uint32_t>(r)));
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            const int sv[4] = {s.x, s.y, s.z, s.w};
            const float xsc = __ldg(a.xs + m0 + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (n + k >= a.N) break;
                const float bv = a.bias ? bf16_bits_to_f32(a.bias[n + k]) : 0.0f;
                const float f = fmaf(static_cast<float>(sv[k]) * xsc, __ldg(a.ws + n + k), bv);
                const int64_t at = static_cast<int64_t>(m0 + c) * a.N + n + k;
                if (a.y_f32) static_cast<float*>(a.y)[at] = f;
                else static_cast<uint16_t*>(a.y)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(f));
            }
        }
    }
    // TMEM is freed, and a CTA of a cluster leaves, when everyone is done with it
    tc_fence_before();
    __syncthreads();
    if (PAIR || a.S > 1) cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, a.tmem_cols);
        else tmem_dealloc(tmem, a.tmem_cols);
    }
}

// One CTA per token: the row's 16-byte chunks in registers (PER a thread),
// absolute maximum, scale fp32(max / 127), exact codes.  With PER = 0 (rows of
// more than 32768 inputs) the row is read twice.
template <int PER>
__global__ void __launch_bounds__(256) quantize_tokens_kernel(const uint16_t* __restrict__ x, int M, int K, int8_t* __restrict__ codes,
                                                              float* __restrict__ scales) {
    __shared__ uint32_t sm[8];
    grid_dependency_sync();
    const int K8 = K / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int m = blockIdx.x; m < M; m += gridDim.x) {
        const uint4* row = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(m) * K);
        uint2* out = reinterpret_cast<uint2*>(codes + static_cast<int64_t>(m) * K);
        constexpr int R = PER > 0 ? PER : 1;
        uint4 raw[R];
        uint32_t m2 = 0;
        auto top = [&](uint4 r) {
            m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu), __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu)));
        };
        if constexpr (PER > 0) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int i = threadIdx.x + j * 256;
                raw[j] = i < K8 ? row[i] : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int j = 0; j < R; ++j) top(raw[j]);
        } else {
            for (int i = threadIdx.x; i < K8; i += 256) top(row[i]);
        }
        uint32_t mx = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) sm[warp] = mx;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = max(mx, sm[i]);
        __syncthreads();
        const bool bad = mx >= 0x7F80u;
        const float s = bad ? 0.0f : __fdiv_rn(__uint_as_float(mx << 16), 127.0f);
        const bool normal = s >= 1.17549435e-38f;
        const float inv = normal ? __frcp_rn(s) : 0.0f;
        if (threadIdx.x == 0) {
            scales[m] = s;
            if (bad) raise_error(ERRBIT_NONFINITE);
        }
        auto put = [&](int i, uint4 r) {
            float f[8];
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f[2 * k] = __uint_as_float(w[k] << 16);
                f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
            const float4 lo = make_float4(f[0], f[1], f[2], f[3]), hi = make_float4(f[4], f[5], f[6], f[7]);
            uint2 c = make_uint2(0u, 0u);
            if (normal) {
                c = make_uint2(rtn4_f32(lo, s, inv, 0.5f * s), rtn4_f32(hi, s, inv, 0.5f * s));
            } else if (s > 0.0f) {
                GroupScale gs;
                gs.s = s;
                gs.normal = false;
                gs.inv = 0.0f;
                gs.inv64 = 1.0 / static_cast<double>(s);
                bool unused = false;
                c = make_uint2(pack_codes4(lo, gs, 127, unused), pack_codes4(hi, gs, 127, unused));
            }
            out[i] = c;
        };
        if constexpr (PER > 0) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int i = threadIdx.x + j * 256;
                if (i < K8) put(i, raw[j]);
            }
        } else {
            for (int i = threadIdx.x; i < K8; i += 256) put(i, row[i]);
        }
    }
}

}  // namespace wlq
