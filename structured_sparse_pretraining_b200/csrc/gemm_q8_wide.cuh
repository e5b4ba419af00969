// gemm_q8_wide.cuh -- the int8 2:4 product at many tokens, on pairs of SMs
// with two row blocks per CTA (see gemm_q8.cuh for the product and the codes,
// gemm_wide.cuh for why two blocks share the token operand).
//
// Pair tile: 512 output channels x 224 tokens.  A k-tile is 256 dense
// positions: per CTA two blocks of 128 rows x 128 kept int8 (32 KB), 112 token
// rows x 256 int8 (28 KB) and the codes (8 KB), for 2 x 4 sparse MMAs of
// M256 N224 K64.  Codes go from the stage straight into TMEM (tcgen05.cp); the
// code columns of stage s are written again only after the stage was refilled,
// that is after the MMAs that read them.
//
// TMEM: 2 x 224 columns of integers and 48 of codes leave no room for
// the adapter's fp32 accumulator.  So with an adapter the epilogue turns the
// integers into scaled fp32 in place (float(acc) xscale wscale), the rank-r
// bf16 MMAs then accumulate onto that, and the result is read and rounded
// once.
//
// Roles (384 threads): warp 0 operand producer, warp 1 TMEM owner and (pair
// leader) MMA issuer, warps 2..5 epilogue of block 0, warps 6..9 of block 1,
// warps 10 and 11 the codes of block 0 and 1 where TMA cannot address them
// (the peer's warp 1 then tells the leader of them: q8_relay_codes).
// An epilogue warp takes its 32 channels x 224 tokens into registers as bf16
// pairs, releases the accumulator, and only then transposes and stores, beside
// the next tile's MMAs.  Row blocks past the end start at M - 128 instead and
// store only their own rows, so that every code read is a legal one.
//
// Bound by the tensor pipe and, over milliseconds, by the power limit: 8192
// tokens on 9216 -> 36864 with rank 96 take 1168 us cool and 1344 under the
// limit (4.8 and 4.1e15 operations a second, the pruned half counted).  Scales
// read from global memory in the epilogue cost 9500 clocks a tile, from shared
// memory 3100, which the next tile's first stages hide in part.
#pragma once
#include <cstdint>
#include "gemm_q8.cuh"

namespace slope {

struct Q8WideCfg {
    static constexpr int BN = 224, BNH = 112;
    static constexpr int NBLK = 2, TILE_M = 512;
    static constexpr int A_BYTES = 16384;
    static constexpr int B_PANEL = BNH * 128;
    static constexpr int E_BYTES = 4096;
    static constexpr int STAGE_BYTES = NBLK * A_BYTES + 2 * B_PANEL + NBLK * E_BYTES;
    static constexpr int NS = 3;
    static constexpr int STAGING_BYTES = 8 * 2048;  // a 32 x 32 bf16 transpose tile per epilogue warp
    static constexpr int E_COL = NBLK * BN;         // 8 columns per block and stage
    static constexpr int TMEM_COLS = 512;
    static constexpr int SMEM_BYTES = NS * STAGE_BYTES + STAGING_BYTES + 256 + 1024;
    static_assert(E_COL + 8 * NBLK * NS <= TMEM_COLS, "TMEM budget");
    static_assert(256 >= 8 * (3 * NS + 1 + 3 * NBLK) + 8, "barrier area");
    static_assert(STAGE_BYTES % 1024 == 0 && B_PANEL % 1024 == 0, "swizzle-atom alignment");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

struct Q8WideParams {
    int M, T, K, r;
    int m_tiles, n_tiles, raster_g, num_work;
    const uint16_t *meta;  // [M x K/16]
    const float *xscale, *wscale;
    uint16_t *Y;
};

// A code tile (rows m0 .. m0 + 127 of the layer, k-tile kt) into `e` where TMA
// cannot address it (see q8_load_codes), as asynchronous copies of one warp.
// Here two of them in flight beat loads ahead into registers, whose fence
// leaves one, and the accumulators' 168 registers leave no room for more warps
// (2458 tokens, 27200 -> 5824: 263 us; codes by TMA, 27264: 181).
__device__ __forceinline__ void q8_copy_codes(uint8_t *e, const uint16_t *meta, int M, int K, int m0, int kt, int lane) {
    const int words = K >> 4;  // a multiple of 4
    const int c = lane & 3;  // four lanes to a row, so that a copy touches 8 sectors and not 32
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int row = 8 * i + (lane >> 2), x = (row >> 2) & 1;
        const int64_t at = (int64_t)(m0 + row) * words + kt * 16 + 4 * c;
        uint8_t *dst = e + row * 32 + 16 * ((c >> 1) ^ x) + 8 * (c & 1);
        const bool in = kt * 16 + 4 * c < words && in_bounds(at, 4, (int64_t)M * words);
        cp_async8(dst, in ? meta + at : meta, in ? 8u : 0u);
    }
}

// META_TMA: codes by TMA, else by warps 10 and 11.
template <bool META_TMA>
__global__ void __launch_bounds__(384, 1)
    q8_wide_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmE, const __grid_constant__ CUtensorMap tmR,
                   const __grid_constant__ CUtensorMap tmXL, const __grid_constant__ Q8WideParams p) {
    using C = Q8WideCfg;
    constexpr int NS = C::NS, BN = C::BN, BNH = C::BNH, NBLK = C::NBLK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *staging = smem + NS * C::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + C::STAGING_BYTES);  // leader: both CTAs' bytes
    uint64_t *empty = full + NS;         // each CTA: stage s may be refilled
    uint64_t *acc_full = empty + NS;        // each CTA: the integer sums are complete
    uint64_t *conv = acc_full + 1;          // per block: leader: both CTAs' sums are scaled fp32 (8 arrivals)
    uint64_t *adp_full = conv + NBLK;       // per block: each CTA: the adapter is added
    uint64_t *acc_empty = adp_full + NBLK;  // per block: leader: both CTAs drained it (8 arrivals)
    uint64_t *codes = acc_empty + NBLK;     // peer: its codes of stage s are written (not by TMA; an arrival per block)
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(codes + NS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
    const int kts = (p.K + 255) >> 8, adp_kts = (p.r + 63) >> 6;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], META_TMA ? 1 : 1 + NBLK + 1);
            mbar_init(&empty[s], 1);
            mbar_init(&codes[s], NBLK);
        }
        mbar_init(acc_full, 1);
        for (int b = 0; b < NBLK; ++b) {
            mbar_init(&conv[b], 8);
            mbar_init(&adp_full[b], 1);
            mbar_init(&acc_empty[b], 8);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        if (META_TMA) tma_prefetch_desc(&tmE);
        if (p.r > 0) {
            tma_prefetch_desc(&tmR);
            tma_prefetch_desc(&tmXL);
        }
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, C::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers are initialised before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    grid_dep_wait();
    grid_dep_launch();

    if (warp == 0) {
        // ------------------------------------------------------------ operand producer (both CTAs)
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (int w = pair; w < p.num_work; w += num_pairs) {
                int mt, nt;
                grouped_tile(w, p.m_tiles, p.n_tiles, p.raster_g, mt, nt);
                int m0[NBLK];
#pragma unroll
                for (int blk = 0; blk < NBLK; ++blk) m0[blk] = min(mt * C::TILE_M + 256 * blk + 128 * (int)rank, p.M - 128);
                const int n0 = nt * BN + BNH * (int)rank;
                for (int kt = 0; kt < kts + adp_kts; ++kt) {
                    if (!mbar_wait(&empty[s], ph ^ 1, abort_flag)) goto done;
                    uint8_t *a = smem + s * C::STAGE_BYTES;
                    uint8_t *b = a + NBLK * C::A_BYTES;
                    uint8_t *e = b + 2 * C::B_PANEL;
                    const uint32_t lead_full = cluster_addr(&full[s], 0);
                    if (kt < kts) {
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (C::STAGE_BYTES - (META_TMA ? 0 : NBLK * C::E_BYTES)));
#pragma unroll
                        for (int blk = 0; blk < NBLK; ++blk) {
                            tma_load_2d_pair(a + blk * C::A_BYTES, &tmA, lead_full, kt * 128, m0[blk]);
                            if (META_TMA) tma_load_2d_pair(e + blk * C::E_BYTES, &tmE, lead_full, kt * 16, m0[blk]);
                        }
                        tma_load_2d_pair(b, &tmB, lead_full, kt * 256, n0);
                        tma_load_2d_pair(b + C::B_PANEL, &tmB, lead_full, kt * 256 + 128, n0);
                    } else {  // adapter: R^T (MN-major, two panels of 64 channels per block) and XL, 64 of the rank
                        const int j0 = (kt - kts) * 64;
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (NBLK * C::A_BYTES + C::B_PANEL));
#pragma unroll
                        for (int blk = 0; blk < NBLK; ++blk) {
                            tma_load_2d_pair(a + blk * C::A_BYTES, &tmR, lead_full, m0[blk], j0);
                            tma_load_2d_pair(a + blk * C::A_BYTES + 8192, &tmR, lead_full, m0[blk] + 64, j0);
                        }
                        tma_load_2d_pair(b, &tmXL, lead_full, j0, n0);
                    }
                    if (++s == NS) { s = 0; ph ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (leader's whole warp, one lane elected)
        if (rank == 0) {
            constexpr uint32_t IDESC_SP = instr_desc_sp_i8(256, BN);
            constexpr uint32_t IDESC_AD = instr_desc(256, BN, 1, 0, 0);
            const uint32_t base = smem_addr(smem);
            const uint64_t a_desc0 = smem_desc(base, 16, 1024, SWZ_128B);
            const uint64_t b_desc0 = smem_desc(base + NBLK * C::A_BYTES, 16, 1024, SWZ_128B);
            const uint64_t e_desc0 = smem_desc(base + NBLK * C::A_BYTES + 2 * C::B_PANEL, 16, 256, SWZ_32B);
            const uint64_t a2_desc0 = smem_desc(base, 8192, 1024, SWZ_128B);
            int s = 0;
            uint32_t ph = 0;
            int it = 0;
            auto adapter = [&](int st, int blk, int kt) {
                const uint64_t off = (uint64_t)((st * C::STAGE_BYTES) >> 4);
                const int nk = min(4, (p.r - kt * 64 + 15) >> 4);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c < nk)
                        elect_mma_bf16<true>(tmem_base + blk * BN, a2_desc0 + off + (uint64_t)(((blk * C::A_BYTES) >> 4) + 128 * c),
                                             b_desc0 + off + (uint64_t)(2 * c), IDESC_AD, 1u);
            };
            for (int w = pair; w < p.num_work; w += num_pairs, ++it) {
                // (Running the first or last one to three k-tiles block by block, so that one block's drain overlaps
                // the other's MMAs, was measured within 1% of this at 9216 -> 36864 and 1024 -> 4096.)
                for (int blk = 0; blk < NBLK; ++blk)
                    if (!mbar_wait_warp(&acc_empty[blk], (it & 1) ^ 1, abort_flag)) goto done;
                tc_fence_after();
                for (int kt = 0; kt < kts; ++kt) {
                    if (!(META_TMA ? mbar_wait_warp(&full[s], ph, abort_flag) : mbar_wait_codes(&full[s], ph, abort_flag))) goto done;
                    tc_fence_after();
                    const uint64_t off = (uint64_t)((s * C::STAGE_BYTES) >> 4);
                    const uint32_t ecol = tmem_base + C::E_COL + 8 * NBLK * s;
#pragma unroll
                    for (int blk = 0; blk < NBLK; ++blk)
                        elect_cp_128x256b<true>(ecol + 8 * blk, e_desc0 + off + (uint64_t)((blk * C::E_BYTES) >> 4));
                    const int nk = min(4, (p.K - kt * 256) >> 6);
#pragma unroll
                    for (int blk = 0; blk < NBLK; ++blk)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (c < nk)
                                elect_mma_sp_i8<true>(tmem_base + blk * BN,
                                                      a_desc0 + off + (uint64_t)(((blk * C::A_BYTES) >> 4) + 2 * c),
                                                      b_desc0 + off + (uint64_t)(((c >> 1) * C::B_PANEL + (c & 1) * 64) >> 4),
                                                      ecol + 8 * blk + 2 * c, IDESC_SP, (kt > 0 || c > 0) ? 1u : 0u);
                    elect_commit<true>(&empty[s]);
                    if (++s == NS) { s = 0; ph ^= 1; }
                }
                elect_commit<true>(acc_full);
                if (adp_kts == 0) continue;
                // block by block while the ring holds the whole adapter, else stage by stage
                const int group = adp_kts <= NS ? adp_kts : 1;
                for (int kt = 0; kt < adp_kts; kt += group) {
                    const int s0 = s;
#pragma unroll
                    for (int blk = 0; blk < NBLK; ++blk) {
                        if (kt == 0) {
                            if (!mbar_wait_warp(&conv[blk], it & 1, abort_flag)) goto done;
                            tc_fence_after();
                        }
                        int st = s0;
                        for (int i = 0; i < group; ++i) {
                            if (blk == 0) {
                                if (!mbar_wait_warp(&full[s], ph, abort_flag)) goto done;
                                tc_fence_after();
                                if (++s == NS) { s = 0; ph ^= 1; }
                            }
                            adapter(st, blk, kt + i);
                            if (blk == NBLK - 1) elect_commit<true>(&empty[st]);
                            if (++st == NS) st = 0;
                        }
                        if (kt + group == adp_kts) elect_commit<true>(&adp_full[blk]);
                    }
                }
            }
        } else if (!META_TMA) {
            if (!q8_relay_codes<NS>(codes, full, lane, pair, num_pairs, p.num_work, kts + adp_kts, abort_flag)) goto done;
        }
    } else if (warp < 10) {
        // ------------------------------------------------------------ epilogue (both CTAs)
        const int q = warp & 3, blk = (warp - 2) >> 2;
        uint8_t *tile = staging + (warp - 2) * 2048;  // [32 tokens][32 channels] bf16
        const int seg = lane & 3, rsub = lane >> 2, odd = lane & 1;
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + blk * BN;
        constexpr int NCH = BN / 32;
        int it = 0;
        for (int w = pair; w < p.num_work; w += num_pairs, ++it) {
            int mt, nt;
            grouped_tile(w, p.m_tiles, p.n_tiles, p.raster_g, mt, nt);
            const int own = mt * C::TILE_M + 256 * blk + 128 * (int)rank;  // the rows this block stores start here
            const int m0 = min(own, p.M - 128) + 32 * q;                   // this warp's first channel
            const int n0 = nt * BN;
            const float ws = in_bounds(m0 + lane, 1, p.M) ? __ldg(p.wscale + m0 + lane) : 0.0f;
            // the tile's token scales (0 past the end), through this warp's transpose tile: read from global
            // memory chunk by chunk they cost most of the drain, beside 1 KB of L1 left by shared memory
            float *xs = reinterpret_cast<float *>(tile);
#pragma unroll
            for (int cc = 0; cc < NCH; ++cc) {
                const int t = n0 + 32 * cc + lane;
                xs[32 * cc + lane] = t < p.T && in_bounds(t, 1, p.T) ? __ldg(p.xscale + t) : 0.0f;
            }
            __syncwarp();
            // 16 columns of integer sums to scaled fp32 (the scales one by one, as their product may leave the range)
            auto scaled = [&](uint32_t (&v)[16], int h) {
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(xs + 16 * h + j);
                    v[j] = __float_as_uint((float)(int)v[j] * ws * x.x);
                    v[j + 1] = __float_as_uint((float)(int)v[j + 1] * ws * x.y);
                    v[j + 2] = __float_as_uint((float)(int)v[j + 2] * ws * x.z);
                    v[j + 3] = __float_as_uint((float)(int)v[j + 3] * ws * x.w);
                }
            };
            if (!mbar_wait_warp(acc_full, it & 1, abort_flag)) break;
            tc_fence_after();
            uint32_t v[2][16];  // the next 16 columns are on their way while these are worked on
            if (adp_kts > 0) {
                tmem_ld_32x32_n(taddr, v[0]);
#pragma unroll
                for (int h = 0; h < 2 * NCH; ++h) {
                    tmem_ld_wait();
                    if (h + 1 < 2 * NCH) tmem_ld_32x32_n(taddr + 16 * (h + 1), v[(h + 1) & 1]);
                    scaled(v[h & 1], h);
                    tmem_st_32x32_n(taddr + 16 * h, v[h & 1]);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(&conv[blk]);
                    else mbar_arrive_cluster(cluster_addr(&conv[blk], 0));
                }
                if (!mbar_wait_warp(&adp_full[blk], it & 1, abort_flag)) break;
                tc_fence_after();
            }
            uint32_t out[NCH][16];  // bf16 pairs of neighbouring tokens, this lane's channel
            tmem_ld_32x32_n(taddr, v[0]);
#pragma unroll
            for (int h = 0; h < 2 * NCH; ++h) {
                tmem_ld_wait();
                if (h + 1 < 2 * NCH) tmem_ld_32x32_n(taddr + 16 * (h + 1), v[(h + 1) & 1]);
                if (adp_kts == 0) scaled(v[h & 1], h);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    out[h >> 1][8 * (h & 1) + j] = pack_bf16x2(bits_to_f32(v[h & 1][2 * j]), bits_to_f32(v[h & 1][2 * j + 1]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) mbar_arrive(&acc_empty[blk]);
                else mbar_arrive_cluster(cluster_addr(&acc_empty[blk], 0));
            }
            __syncwarp();  // the scales have been read: the tile is free
            const bool m_ok = m0 + 8 * seg >= own && own < p.M;  // rows of the clamped overlap belong to the block before
#pragma unroll
            for (int cc = 0; cc < NCH; ++cc) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    // neighbouring lanes swap a token so that each holds two channels of one
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, out[cc][j], 1);
                    const uint32_t pr = odd ? __byte_perm(other, out[cc][j], 0x7632) : __byte_perm(out[cc][j], other, 0x5410);
                    *reinterpret_cast<uint32_t *>(tile + ((2 * j + odd) * 32 + (lane & ~1)) * 2) = pr;
                }
                __syncwarp();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int t = n0 + 32 * cc + 8 * g + rsub;
                    const uint4 val = *reinterpret_cast<const uint4 *>(tile + ((8 * g + rsub) * 32 + seg * 8) * 2);
                    const int64_t at = (int64_t)t * p.M + m0 + seg * 8;
                    if (m_ok && t < p.T && in_bounds(at, 8, (int64_t)p.T * p.M)) *reinterpret_cast<uint4 *>(p.Y + at) = val;
                }
                __syncwarp();  // every lane has read the tile before the next chunk overwrites it
            }
        }
    } else if (!META_TMA) {
        // ------------------------------------------------------------ code loaders (both CTAs)
        // LAG stages of copies stay in flight: a stage is published once those of the next are issued, or sooner while
        // the next stage is not free yet (2458 tokens, 27200 -> 5824: 263 us, 294 if it always waits for that)
        const int blk = warp - 10;
        constexpr int LAG = 1;
        int s = 0, issued = 0, published = 0;
        uint32_t ph = 0;
        auto publish = [&]() {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(rank == 0 ? &full[published % NS] : &codes[published % NS]);
            ++published;
        };
        for (int w = pair; w < p.num_work; w += num_pairs) {
            int mt, nt;
            grouped_tile(w, p.m_tiles, p.n_tiles, p.raster_g, mt, nt);
            const int m0 = min(mt * C::TILE_M + 256 * blk + 128 * (int)rank, p.M - 128);
            for (int kt = 0; kt < kts + adp_kts; ++kt) {
                if (published < issued && !__all_sync(0xffffffffu, mbar_test(&empty[s], ph ^ 1))) {
                    cp_async_wait<0>();
                    publish();
                }
                if (!mbar_wait_warp(&empty[s], ph ^ 1, abort_flag)) {
                    cp_async_wait<0>();
                    goto done;
                }
                if (kt < kts)
                    q8_copy_codes(smem + s * C::STAGE_BYTES + NBLK * C::A_BYTES + 2 * C::B_PANEL + blk * C::E_BYTES, p.meta, p.M, p.K,
                                  m0, kt, lane);
                cp_async_commit();
                if (++issued - published > LAG) {
                    cp_async_wait<LAG>();
                    publish();
                }
                if (++s == NS) { s = 0; ph ^= 1; }
            }
        }
        cp_async_wait<0>();
        while (published < issued) publish();
    }
done:
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while its peer may still signal it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace slope
