// gemm_q8_pair.cuh -- the int8 2:4 product at a few hundred tokens, where the
// weights' streaming and the tensor work are of one size: pair tiles of 256
// channels x 256 tokens (see gemm_q8.cuh for the product and the codes).
//
// Why a third tensor-core form.  128 x 128 tiles read every token row once per
// 128 channels: at 256 tokens that is 3.2 bytes from L2 for each byte of
// weights, and the SMs' ingest (about 72 B a clock) bounds the product at
// three times the weights' own time.  512 x 224 tiles need few bytes, but a
// layer has too few of them at this size to fill the SM pairs.  Here a pair
// shares 256 token rows (128 in each CTA) against 256 channels (128 in each):
// 52 KB per CTA and k-tile, of which 20 KB are weights and codes, four stages
// deep: 49 us at 256 tokens on 9216 -> 27648, against 75 and 65 us of the two
// (floor 27.7, the weights at the measured copy rate; 108 tiles are 1.46 rounds
// of the 74 pairs, and a k-tile takes about 1100 clocks for 512 of MMA).
// (Two pairs sharing a tile's sum over K, to even out the tiles per pair, were
// measured slower: 70 against 53 us at 128 tokens.  Their partials are 64 KB a
// tile and CTA, and distributed shared memory took them at about 10 B a clock.)
//
// TMEM: 256 columns of integers, 32 of codes.  The adapter as in
// gemm_q8_wide.cuh: the epilogue scales the integers to fp32 in place, the
// rank-r MMAs accumulate onto that.
//
// Roles (384 threads): warp 0 operand producer, warp 1 TMEM owner and (pair
// leader) MMA issuer, warps 2..9 epilogue (a quarter of the rows, half of the
// columns each), warps 10 and 11 the codes where TMA cannot address them (the
// peer's warp 1 then tells the leader of them: q8_relay_codes).
#pragma once
#include <cstdint>
#include "gemm_q8.cuh"

namespace slope {

struct Q8PairCfg {
    static constexpr int BN = 256, BNH = 128;
    static constexpr int A_BYTES = 16384;
    static constexpr int B_PANEL = BNH * 128;
    static constexpr int E_BYTES = 4096;
    static constexpr int STAGE_BYTES = A_BYTES + 2 * B_PANEL + E_BYTES;
    static constexpr int NS = 4;
    static constexpr int STAGING_BYTES = 8 * 2048;         // a 32 x 32 bf16 transpose tile per epilogue warp
    static constexpr int E_COL = BN;                       // 8 columns per stage
    static constexpr int TMEM_COLS = 512;
    static constexpr int SMEM_BYTES = NS * STAGE_BYTES + STAGING_BYTES + 256 + 1024;
    static_assert(E_COL + 8 * NS <= TMEM_COLS, "TMEM budget");
    static_assert(256 >= 8 * (3 * NS + 4) + 8, "barrier area");
    static_assert(STAGE_BYTES % 1024 == 0 && B_PANEL % 1024 == 0, "swizzle-atom alignment");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

struct Q8PairParams {
    int M, T, K, r;
    int n_tiles, num_work;
    const uint16_t *meta;
    const float *xscale, *wscale;
    uint16_t *Y;
};

// META_TMA: codes by TMA, else by warps 10 and 11.
template <bool META_TMA>
__global__ void __launch_bounds__(384, 1)
    q8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmE, const __grid_constant__ CUtensorMap tmR,
                   const __grid_constant__ CUtensorMap tmXL, const __grid_constant__ Q8PairParams p) {
    using C = Q8PairCfg;
    constexpr int NS = C::NS, BN = C::BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *staging = smem + NS * C::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + C::STAGING_BYTES);  // leader: both CTAs' bytes
    uint64_t *empty = full + NS;          // each CTA: stage s may be refilled
    uint64_t *acc_full = empty + NS;      // each CTA: the integer sums are complete
    uint64_t *conv = acc_full + 1;        // leader: both CTAs' sums are scaled fp32 (16 arrivals)
    uint64_t *adp_full = conv + 1;        // each CTA: the adapter is added
    uint64_t *acc_empty = adp_full + 1;   // leader: both CTAs drained the accumulator (16 arrivals)
    uint64_t *codes = acc_empty + 1;      // peer: its codes of stage s are written (not by TMA)
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(codes + NS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
    const int kts = (p.K + 255) >> 8, adp_kts = (p.r + 63) >> 6;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], META_TMA ? 1 : 3);
            mbar_init(&empty[s], 1);
            mbar_init(&codes[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(conv, 16);
        mbar_init(adp_full, 1);
        mbar_init(acc_empty, 16);
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
        // ------------------------------------------------------------ operand producer
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (int w = pair; w < p.num_work; w += num_pairs) {
                const int nt = w % p.n_tiles, mt = w / p.n_tiles;  // tiles of the same channels run together
                const int m0 = min(mt * 256 + 128 * (int)rank, p.M - 128), n0 = nt * BN;
                for (int kt = 0; kt < kts + adp_kts; ++kt) {
                    if (!mbar_wait(&empty[s], ph ^ 1, abort_flag)) goto done;
                    uint8_t *a = smem + s * C::STAGE_BYTES;
                    uint8_t *b = a + C::A_BYTES;
                    const uint32_t lead_full = cluster_addr(&full[s], 0);
                    if (kt < kts) {
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (C::STAGE_BYTES - (META_TMA ? 0 : C::E_BYTES)));
                        tma_load_2d_pair(a, &tmA, lead_full, kt * 128, m0);
                        if (META_TMA) tma_load_2d_pair(b + 2 * C::B_PANEL, &tmE, lead_full, kt * 16, m0);
                        tma_load_2d_pair(b, &tmB, lead_full, kt * 256, n0 + 128 * (int)rank);
                        tma_load_2d_pair(b + C::B_PANEL, &tmB, lead_full, kt * 256 + 128, n0 + 128 * (int)rank);
                    } else {  // adapter: R^T (MN-major, two panels of 64 channels) and XL, 64 of the rank
                        const int j0 = (kt - kts) * 64;
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (C::A_BYTES + C::B_PANEL));
                        tma_load_2d_pair(a, &tmR, lead_full, m0, j0);
                        tma_load_2d_pair(a + 8192, &tmR, lead_full, m0 + 64, j0);
                        tma_load_2d_pair(b, &tmXL, lead_full, j0, n0 + 128 * (int)rank);
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
            const uint64_t b_desc0 = smem_desc(base + C::A_BYTES, 16, 1024, SWZ_128B);
            const uint64_t e_desc0 = smem_desc(base + C::A_BYTES + 2 * C::B_PANEL, 16, 256, SWZ_32B);
            const uint64_t a2_desc0 = smem_desc(base, 8192, 1024, SWZ_128B);
            int s = 0, it = 0;
            uint32_t ph = 0;
            for (int w = pair; w < p.num_work; w += num_pairs, ++it) {
                if (!mbar_wait_warp(acc_empty, (it & 1) ^ 1, abort_flag)) goto done;
                tc_fence_after();
                for (int kt = 0; kt < kts; ++kt) {
                    if (!(META_TMA ? mbar_wait_warp(&full[s], ph, abort_flag) : mbar_wait_codes(&full[s], ph, abort_flag))) goto done;
                    tc_fence_after();
                    const uint64_t off = (uint64_t)((s * C::STAGE_BYTES) >> 4);
                    const uint32_t ecol = tmem_base + C::E_COL + 8 * s;
                    elect_cp_128x256b<true>(ecol, e_desc0 + off);
                    const int nk = min(4, (p.K - kt * 256) >> 6);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c < nk)
                            elect_mma_sp_i8<true>(tmem_base, a_desc0 + off + (uint64_t)(2 * c),
                                                  b_desc0 + off + (uint64_t)(((c >> 1) * C::B_PANEL + (c & 1) * 64) >> 4),
                                                  ecol + 2 * c, IDESC_SP, (kt > 0 || c > 0) ? 1u : 0u);
                    elect_commit<true>(&empty[s]);
                    if (++s == NS) { s = 0; ph ^= 1; }
                }
                elect_commit<true>(acc_full);
                if (adp_kts == 0) continue;
                if (!mbar_wait_warp(conv, it & 1, abort_flag)) goto done;
                tc_fence_after();
                for (int kt = 0; kt < adp_kts; ++kt) {
                    if (!mbar_wait_warp(&full[s], ph, abort_flag)) goto done;
                    tc_fence_after();
                    const uint64_t off = (uint64_t)((s * C::STAGE_BYTES) >> 4);
                    const int nk = min(4, (p.r - kt * 64 + 15) >> 4);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c < nk)
                            elect_mma_bf16<true>(tmem_base, a2_desc0 + off + (uint64_t)(128 * c),
                                                 b_desc0 + off + (uint64_t)(2 * c), IDESC_AD, 1u);
                    elect_commit<true>(&empty[s]);
                    if (++s == NS) { s = 0; ph ^= 1; }
                }
                elect_commit<true>(adp_full);
            }
        } else if (!META_TMA) {
            if (!q8_relay_codes<NS>(codes, full, lane, pair, num_pairs, p.num_work, kts + adp_kts, abort_flag)) goto done;
        }
    } else if (warp < 10) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, hh = (warp - 2) >> 2;
        uint8_t *tile = staging + (warp - 2) * 2048;  // [32 tokens][32 channels] bf16
        const int seg = lane & 3, rsub = lane >> 2, odd = lane & 1;
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
        constexpr int NCH = BN / 64;  // this warp's chunks of 32 columns, from col(cc) on
        auto col = [&](int cc) { return 128 * hh + 32 * cc; };
        int it = 0;
        for (int w = pair; w < p.num_work; w += num_pairs, ++it) {
            const int nt = w % p.n_tiles, mt = w / p.n_tiles;
            const int own = mt * 256 + 128 * (int)rank;        // the rows this CTA stores start here
            const int m0 = min(own, p.M - 128) + 32 * q;  // this warp's first channel
            const int n0 = nt * BN;
            const float ws = in_bounds(m0 + lane, 1, p.M) ? __ldg(p.wscale + m0 + lane) : 0.0f;
            // the scales of this warp's tokens (0 past the end), through its transpose tile
            float *xs = reinterpret_cast<float *>(tile);
#pragma unroll
            for (int cc = 0; cc < NCH; ++cc) {
                const int t = n0 + col(cc) + lane;
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
            uint32_t out[NCH][16];  // bf16 pairs of neighbouring tokens, this lane's channel
            auto packed = [&](const uint32_t (&v)[16], int h) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    out[h >> 1][8 * (h & 1) + j] = pack_bf16x2(bits_to_f32(v[2 * j]), bits_to_f32(v[2 * j + 1]));
            };
            if (!mbar_wait_warp(acc_full, it & 1, abort_flag)) break;
            tc_fence_after();
            uint32_t v[2][16];  // the next 16 columns are on their way while these are worked on
            tmem_ld_32x32_n(taddr + col(0), v[0]);
#pragma unroll
            for (int h = 0; h < 2 * NCH; ++h) {
                tmem_ld_wait();
                if (h + 1 < 2 * NCH) tmem_ld_32x32_n(taddr + col(0) + 16 * (h + 1), v[(h + 1) & 1]);
                scaled(v[h & 1], h);
                if (adp_kts > 0) tmem_st_32x32_n(taddr + col(0) + 16 * h, v[h & 1]);
                else packed(v[h & 1], h);
            }
            if (adp_kts > 0) {
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(conv);
                    else mbar_arrive_cluster(cluster_addr(conv, 0));
                }
                if (!mbar_wait_warp(adp_full, it & 1, abort_flag)) break;
                tc_fence_after();
                tmem_ld_32x32_n(taddr + col(0), v[0]);
#pragma unroll
                for (int h = 0; h < 2 * NCH; ++h) {
                    tmem_ld_wait();
                    if (h + 1 < 2 * NCH) tmem_ld_32x32_n(taddr + col(0) + 16 * (h + 1), v[(h + 1) & 1]);
                    packed(v[h & 1], h);
                }
            }
            tc_fence_before();
            __syncwarp();  // the scales have been read too: the tile is free
            if (lane == 0) {
                if (rank == 0) mbar_arrive(acc_empty);
                else mbar_arrive_cluster(cluster_addr(acc_empty, 0));
            }
            const bool m_ok = m0 + 8 * seg >= own && own < p.M;  // rows of the clamped overlap belong to the tile before
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
                    const int t = n0 + col(cc) + 8 * g + rsub;
                    const uint4 val = *reinterpret_cast<const uint4 *>(tile + ((8 * g + rsub) * 32 + seg * 8) * 2);
                    const int64_t at = (int64_t)t * p.M + m0 + seg * 8;
                    if (m_ok && t < p.T && in_bounds(at, 8, (int64_t)p.T * p.M)) *reinterpret_cast<uint4 *>(p.Y + at) = val;
                }
                __syncwarp();  // every lane has read the tile before the next chunk overwrites it
            }
        }
    } else if (!META_TMA) {
        // ------------------------------------------------------------ code loaders (both CTAs)
        if (!q8_load_codes<2, NS>(
                p.meta, p.M, p.K, warp - 10, lane, pair, num_pairs, p.num_work, 0, kts, adp_kts,
                [&](int w) { return min(w / p.n_tiles * 256 + 128 * (int)rank, p.M - 128); },
                [&](int st) { return smem + st * C::STAGE_BYTES + C::A_BYTES + 2 * C::B_PANEL; },
                [&](int st, uint32_t phase) { return mbar_wait_warp(&empty[st], phase, abort_flag); },
                [&](int st) { mbar_arrive(rank == 0 ? &full[st] : &codes[st]); }))
            goto done;
    }
done:
    __syncwarp();
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
