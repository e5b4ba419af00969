// gemm_q8.cuh -- the int8 2:4 product on tensor cores at few tokens, where the
// streaming of the weights bounds it: 128 x BN tiles.
//
//   Y[t][o] = xscale[t] wscale[o] (Xq . Wq^T)[t][o] + (XL . R)[t][o]
//
// tcgen05.mma.sp kind::i8: the kept int8 values of 128 output channels
// (K-major, 128 stored = 256 dense positions a k-tile), BN int8 token rows,
// exact sums in 32-bit integers in TMEM.  The codes need no rearranging: TMEM
// wants lane = row with the row's codes in order, so the code tile comes in by
// TMA in a 32-byte swizzle and tcgen05.cp puts its 128 x 32 bytes into eight
// columns.  The rank-r adapter runs as dense bf16 MMAs after the int8 ones
// into an fp32 accumulator of its own, and the epilogue joins the two, which
// neither scale could do inside one accumulator.
//
// Roles: warp 0 operand producer, warp 1 TMEM owner and MMA
// issuer, warps 2..5 epilogue, the others load the codes where TMA
// cannot (q8_load_codes).
//
// Persistent clusters of `splits` CTAs; the CTAs of a cluster share each
// tile's sum over K, so that tiles can be handed out evenly whatever their
// number (27648 channels are 216 tiles: two rounds for 148 single CTAs, a
// quarter of the second idle, but three full ones for 74 clusters of two).
// Each CTA finishes its share of the tile's tokens: the others push their
// integer partials of that share into its shared memory (distributed shared
// memory, one buffer per source), then it adds them to its own.  So no
// workspace and no atomics, and launches can overlap; integer sums do not
// depend on the split.  The integer accumulator is double-buffered: the next
// tile's MMAs run beside the epilogue.  Row tiles past the end start at
// M - 128 instead, so that every code the MMA reads is a legal one (a layer of
// 64 channels gets its codes from q8_load_codes); K ends inside a k-tile after
// whole MMAs.
//
// Measured, with adapters: one token on 9216 -> 27648 31 us (80% of the copy
// rate), sixteen on 36864 -> 9216 39.5; sixteen on 20480 -> 5120 19 us with
// clusters of three, 22 with two.  Splits of 1, 2, 3, 4 and 8 are offered:
// resident clusters of 5, 6 and 7 fill 130, 132 and 105 SMs, those of 4 fill 132.
#pragma once
#include <cstdint>
#include <type_traits>
#include "gemm.cuh"
#include "ptx.cuh"
#include "rownorm.cuh"  // pack_bf16x2

namespace slope {

struct Q8Params {
    int M, T, K, r;        // output channels, tokens, dense K, adapter rank
    int m_tiles, num_work;
    int splits;            // CTAs per cluster
    int meta_tma;          // 1: codes by TMA, 0: by the warps from 6 on
    const uint16_t *meta;  // [M x K/16]
    const float *xscale, *wscale;
    uint16_t *Y;           // [T x M]
};

// The columns of a BN-wide tile that the CTAs of a cluster of S finish: CTA u
// takes [first(u), first(u + 1)), in steps of 8, or of 2 where there are fewer
// than S steps of 8.
struct Q8Shares {
    int step, steps, S;
    __host__ __device__ Q8Shares(int bn, int splits) : step(bn >= 8 * splits ? 8 : 2), steps(bn / step), S(splits) {}
    __host__ __device__ int first(int u) const { return steps * u / S * step; }
    __host__ __device__ int most() const { return (steps + S - 1) / S * step; }
};

// Shared memory of a tile kernel for the partials of the other CTAs of its
// cluster: enough for clusters of 1, 2, 3, 4 and 8 (five to seven CTAs were
// measured slower than three or four on every layer tried).
constexpr int q8_red_bytes(int bn) { return bn == 128 ? 57344 : bn == 64 ? 28672 : bn == 32 ? 16384 : 7168; }

template <int BN>
struct Q8Cfg {
    static constexpr int A_BYTES = 16384;     // 128 rows x 128 stored int8
    static constexpr int B_PANEL = BN * 128;  // BN rows x 128 dense int8, 128-byte swizzle
    static constexpr int E_BYTES = 4096;      // 128 rows x 32 bytes of codes, 32-byte swizzle
    static constexpr int STAGE_BYTES = A_BYTES + 2 * B_PANEL + E_BYTES;
    static constexpr int RED_BYTES = q8_red_bytes(BN);
    static constexpr int XS_BYTES = 3 * BN * 4;  // token scales of three tiles
    static constexpr int BAR_BYTES = 256;
    static constexpr int NS_RAW = (232448 - 1024 - BAR_BYTES - XS_BYTES - RED_BYTES) / STAGE_BYTES;
    static constexpr int NS = NS_RAW > 8 ? 8 : NS_RAW;
    static constexpr int CODE_WARPS = NS % 4 == 0 ? 4 : NS % 3 == 0 ? 3 : NS;  // a divisor of NS, see q8_load_codes
    static constexpr int THREADS = 32 * (6 + CODE_WARPS);
    static constexpr int ADP_COL = 2 * BN;    // fp32 adapter accumulator, after the two integer ones
    static constexpr int E_COL = 3 * BN;      // 8 columns per stage
    static constexpr int TMEM_COLS = BN == 128 ? 512 : BN >= 32 ? 256 : 128;
    static constexpr int SMEM_BYTES = NS * STAGE_BYTES + RED_BYTES + XS_BYTES + BAR_BYTES + 1024;
    static_assert(E_COL + 8 * NS <= TMEM_COLS, "TMEM budget");
    static_assert(BAR_BYTES >= 8 * (2 * NS + 6) + 8, "barrier area");
    static_assert(B_PANEL % 1024 == 0 && STAGE_BYTES % 1024 == 0, "swizzle-atom alignment");
    static_assert(NS >= 3 && SMEM_BYTES <= 232448, "shared memory budget");
};

// W token columns of one warp's 32 channels: v holds this lane's channel.
// Neighbouring lanes swap so that each stores a bf16 pair of one token.
template <int W>
__device__ __forceinline__ void q8_store(const float (&v)[W], const Q8Params &p, int t0, int f0, int lane, bool ok) {
    const int odd = lane & 1;
#pragma unroll
    for (int j = 0; j < W; j += 2) {
        const float other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
        const uint32_t pr = odd ? pack_bf16x2(other, v[j + 1]) : pack_bf16x2(v[j], other);
        const int t = t0 + j + odd;
        const int64_t at = (int64_t)t * p.M + f0 + (lane & ~1);
        if (ok && t < p.T && in_bounds(at, 2, (int64_t)p.T * p.M)) *reinterpret_cast<uint32_t *>(p.Y + at) = pr;
    }
}

// The code tiles of a kernel's k-tiles (128 rows x 32 bytes, in the 32-byte
// swizzle), by WARPS warps in turn: for code rows of K/8 bytes that are not a
// multiple of 16, which TMA cannot address, and for layers of 64 channels,
// whose missing rows take positions 0 and 1 (of kept values that TMA reads as
// zero).  Words past the row are zeros that no MMA reads.
//
// A warp has the codes of its next k-tile on their way in registers (8 bytes at
// a time, four lanes to a row) while it waits for the stage.  More than one
// k-tile ahead does not work within a warp, as the fence between its stores and
// the tensor core's reads waits for its loads too: 16 tokens, 9152 -> 27648
// take 38.7 us with four warps, 77 with one that is four ahead, 41 with one
// whose asynchronous copies go into the stage (codes by TMA, 9344: 33).
//
// Work items first, first + step, .. below num_work, each with the k-tiles
// [k0, k1) and `extra` ones without codes; row0(w) is a work item's first row,
// dst(s) the stage's code tile, wait(s, phase) the stage's being free,
// publish(s) the warp's arrival.  False where a wait gave up.  WARPS divides NS,
// so that a stage has one warp, which sees each of its phases: a wait tells only
// a phase's parity.
template <int WARPS, int NS, typename Row0, typename Dst, typename Wait, typename Publish>
__device__ __forceinline__ bool q8_load_codes(const uint16_t *meta, int M, int K, int which, int lane, int first, int step,
                                              int num_work, int k0, int k1, int extra, Row0 row0, Dst dst, Wait wait,
                                              Publish publish) {
    static_assert(NS % WARPS == 0, "one warp per stage");
    const int words = K >> 4;  // of a row; a multiple of 4
    const int c = lane & 3;
    int w = first, kt = k0, s = 0;
    uint32_t ph = 0;
    auto advance = [&](int n) {
        for (kt += n; kt >= k1 + extra && w < num_work; w += step) kt -= k1 + extra - k0;
        for (s += n; s >= NS; ph ^= 1) s -= NS;
    };
    for (advance(which); w < num_work; advance(WARPS)) {
        uint2 v[16];
        if (kt < k1) {
            const bool in = kt * 16 + 4 * c < words;
            const int m0 = row0(w);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = m0 + 8 * i + (lane >> 2);
                const int64_t at = (int64_t)row * words + kt * 16 + 4 * c;
                v[i] = row >= M ? make_uint2(0x44444444u, 0x44444444u) : make_uint2(0, 0);
                if (in && row < M && in_bounds(at, 4, (int64_t)M * words)) v[i] = load_ahead8(meta + at);
            }
        }
        if (!wait(s, ph ^ 1)) return false;
        if (kt < k1) {
            uint8_t *e = dst(s);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = 8 * i + (lane >> 2), x = (row >> 2) & 1;
                *reinterpret_cast<uint2 *>(e + row * 32 + 16 * ((c >> 1) ^ x) + 8 * (c & 1)) = v[i];
            }
            fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) publish(s);
    }
    return true;
}

// A pair's peer tells the leader of each stage whose codes its own warps have
// written (`codes`, this CTA's) by an arrival on the leader's `full`, which
// releases at cluster scope what its wait has acquired from them: the leader's
// tcgen05.cp reads the codes of both CTAs.  The peer's MMA warp does it, which
// has nothing else to do and nothing in flight: a cluster-scope release by the
// loading warps waits for their loads ahead too (512 x 224 tiles: 2458 tokens,
// 27200 -> 5824 294 us against 400; 256 x 256 tiles, whose loaders wait for
// their loads anyway: 6000 tokens, 832 -> 5184 35 against 38, 300 tokens,
// 4160 -> 9216 26 against 25).  False where a wait gave up.
template <int NS>
__device__ __forceinline__ bool q8_relay_codes(uint64_t *codes, uint64_t *full, int lane, int first, int step, int num_work,
                                               int ktiles, volatile int *abort_flag) {
    int s = 0;
    uint32_t ph = 0;
    for (int w = first; w < num_work; w += step)
        for (int kt = 0; kt < ktiles; ++kt) {
            if (!mbar_wait_warp(&codes[s], ph, abort_flag)) return false;
            if (lane == 0) mbar_arrive_cluster_rel(cluster_addr(&full[s], 0));
            if (++s == NS) { s = 0; ph ^= 1; }
        }
    return true;
}

template <int BN>
__global__ void __launch_bounds__(Q8Cfg<BN>::THREADS, 1)
    q8_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmE, const __grid_constant__ CUtensorMap tmR,
                   const __grid_constant__ CUtensorMap tmXL, const __grid_constant__ Q8Params p) {
    using C = Q8Cfg<BN>;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint32_t *red = reinterpret_cast<uint32_t *>(smem + NS * C::STAGE_BYTES);  // [source][token of the share][128 channels]
    float *xs_buf = reinterpret_cast<float *>(smem + NS * C::STAGE_BYTES + C::RED_BYTES);  // [3][BN]
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + NS * C::STAGE_BYTES + C::RED_BYTES + C::XS_BYTES);
    uint64_t *empty = full + NS;
    uint64_t *acc_full = empty + NS;     // [2]
    uint64_t *acc_empty = acc_full + 2;  // [2], 4 arrivals
    uint64_t *red_full = acc_empty + 2;  // every other CTA's four warps have pushed their partials of this CTA's share
    uint64_t *red_empty = red_full + 1;  // every other CTA's four warps have read this CTA's partials
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(red_empty + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int S = p.splits;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    const int cluster = blockIdx.x / S, num_clusters = gridDim.x / S;
    const int kts = (p.K + 255) >> 8;
    const int k0 = (int)((int64_t)kts * rank / S), k1 = (int)((int64_t)kts * (rank + 1) / S);
    const int adp_kts = (p.r + 63) >> 6;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], p.meta_tma ? 1 : 2);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 4);
        }
        mbar_init(red_full, S > 1 ? 4 * (S - 1) : 1);
        mbar_init(red_empty, S > 1 ? 4 * (S - 1) : 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        if (p.meta_tma) tma_prefetch_desc(&tmE);
        if (p.r > 0) {
            tma_prefetch_desc(&tmR);
            tma_prefetch_desc(&tmXL);
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    if (S > 1) cluster_sync();  // the others' barriers are initialised before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    if (warp == 6 && lane == 0 && p.meta_tma) {
        // the first stages' weights on their way to L2 beside the tail of the kernel before (3% at one to sixteen
        // tokens; nothing is read from them before the wait)
        const int pm0 = max(0, min(cluster % p.m_tiles * 128, p.M - 128));
        for (int kt = k0; kt < min(k1, k0 + NS); ++kt) {
            tma_prefetch_2d(&tmA, kt * 128, pm0);
            tma_prefetch_2d(&tmE, kt * 16, pm0);
        }
    }
    grid_dep_wait();
    grid_dep_launch();

    if (warp == 0) {
        // ------------------------------------------------------------ operand producer
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (int w = cluster; w < p.num_work; w += num_clusters) {
                const int mt = w % p.m_tiles, nt = w / p.m_tiles;
                const int m0 = max(0, min(mt * 128, p.M - 128)), n0 = nt * BN;
                for (int kt = k0; kt < k1 + adp_kts; ++kt) {
                    if (!mbar_wait(&empty[s], ph ^ 1, abort_flag)) goto done;
                    uint8_t *a = smem + s * C::STAGE_BYTES;
                    uint8_t *b = a + C::A_BYTES;
                    if (kt < k1) {
                        mbar_arrive_expect_tx(&full[s], C::A_BYTES + 2 * C::B_PANEL + (p.meta_tma ? C::E_BYTES : 0));
                        tma_load_2d(a, &tmA, &full[s], kt * 128, m0);
                        if (p.meta_tma) tma_load_2d(b + 2 * C::B_PANEL, &tmE, &full[s], kt * 16, m0);
                        tma_load_2d(b, &tmB, &full[s], kt * 256, n0);
                        tma_load_2d(b + C::B_PANEL, &tmB, &full[s], kt * 256 + 128, n0);
                    } else {  // adapter: R^T (MN-major, two panels of 64 channels) and XL, 64 of the rank
                        const int j0 = (kt - k1) * 64;
                        mbar_arrive_expect_tx(&full[s], C::A_BYTES + C::B_PANEL);
                        tma_load_2d(a, &tmR, &full[s], m0, j0);
                        tma_load_2d(a + 8192, &tmR, &full[s], m0 + 64, j0);
                        tma_load_2d(b, &tmXL, &full[s], j0, n0);
                    }
                    if (++s == NS) { s = 0; ph ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (the whole warp, one lane elected)
        constexpr uint32_t IDESC_SP = instr_desc_sp_i8(128, BN);
        constexpr uint32_t IDESC_AD = instr_desc(128, BN, 1, 0, 0);
        const uint32_t base = smem_addr(smem);
        const uint64_t a_desc0 = smem_desc(base, 16, 1024, SWZ_128B);
        const uint64_t b_desc0 = smem_desc(base + C::A_BYTES, 16, 1024, SWZ_128B);
        const uint64_t e_desc0 = smem_desc(base + C::A_BYTES + 2 * C::B_PANEL, 16, 256, SWZ_32B);
        const uint64_t a2_desc0 = smem_desc(base, 8192, 1024, SWZ_128B);
        int s = 0, it = 0;
        uint32_t ph = 0;
        for (int w = cluster; w < p.num_work; w += num_clusters, ++it) {
            const uint32_t d = tmem_base + (it & 1) * BN;
            if (!mbar_wait_warp(&acc_empty[it & 1], ((it >> 1) & 1) ^ 1, abort_flag)) goto done;
            tc_fence_after();
            for (int kt = k0; kt < k1; ++kt) {
                if (!mbar_wait_warp(&full[s], ph, abort_flag)) goto done;
                tc_fence_after();
                const uint64_t off = (uint64_t)((s * C::STAGE_BYTES) >> 4);
                // the code columns of stage s: their last readers finished before the stage was refilled
                const uint32_t ecol = tmem_base + C::E_COL + 8 * s;
                elect_cp_128x256b<false>(ecol, e_desc0 + off);
                const int nblk = min(4, (p.K - kt * 256) >> 6);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c < nblk)
                        elect_mma_sp_i8<false>(d, a_desc0 + off + (uint64_t)(2 * c),
                                               b_desc0 + off + (uint64_t)(((c >> 1) * C::B_PANEL + (c & 1) * 64) >> 4),
                                               ecol + 2 * c, IDESC_SP, (kt > k0 || c > 0) ? 1u : 0u);
                elect_commit<false>(&empty[s]);
                if (++s == NS) { s = 0; ph ^= 1; }
            }
            if (adp_kts > 0 && it > 0) {  // the tile before has left the adapter's accumulator
                if (!mbar_wait_warp(&acc_empty[(it - 1) & 1], ((it - 1) >> 1) & 1, abort_flag)) goto done;
                tc_fence_after();
            }
            for (int kt = 0; kt < adp_kts; ++kt) {
                if (!mbar_wait_warp(&full[s], ph, abort_flag)) goto done;
                tc_fence_after();
                const uint64_t off = (uint64_t)((s * C::STAGE_BYTES) >> 4);
                const int nblk = min(4, (p.r - kt * 64 + 15) >> 4);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c < nblk)
                        elect_mma_bf16<false>(tmem_base + C::ADP_COL, a2_desc0 + off + (uint64_t)(128 * c),
                                              b_desc0 + off + (uint64_t)(2 * c), IDESC_AD, (kt > 0 || c > 0) ? 1u : 0u);
                elect_commit<false>(&empty[s]);
                if (++s == NS) { s = 0; ph ^= 1; }
            }
            elect_commit<false>(&acc_full[it & 1]);
        }
    } else if (warp < 6) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        const Q8Shares shares(BN, S);
        const int c_own = shares.first(rank), own = shares.first(rank + 1) - c_own;  // this CTA's columns
        int it = 0;
        for (int w = cluster; w < p.num_work; w += num_clusters, ++it) {
            const int mt = w % p.m_tiles, nt = w / p.m_tiles;
            const int m0 = max(0, min(mt * 128, p.M - 128)), n0 = nt * BN;
            const int cols = min(BN, (p.T - n0 + 1) & ~1);  // columns with tokens
            const int f = m0 + 32 * q + lane;               // this lane's channel
            const bool row_ok = f >= mt * 128 && f < p.M;   // rows the tile before owns are not stored again
            const float ws = f < p.M && in_bounds(f, 1, p.M) ? __ldg(p.wscale + f) : 0.0f;
            // Every warp writes the scales that it reads itself (the four write the same values).  A warp may be here
            // while another is still in the tile before the last: that one's sums must be released before the
            // wait below ends, so three buffers keep them apart.
            float *xs = xs_buf + it % 3 * BN;
            for (int c = lane; c < BN; c += 32) xs[c] = n0 + c < p.T && in_bounds(n0 + c, 1, p.T) ? __ldg(p.xscale + n0 + c) : 0.0f;
            __syncwarp();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + (it & 1) * BN;
            const uint32_t tadp = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + C::ADP_COL;
            if (!mbar_wait_warp(&acc_full[it & 1], (it >> 1) & 1, abort_flag)) break;
            tc_fence_after();
            auto push = [&](auto width, int c, uint32_t dst) {
                constexpr int W = decltype(width)::value;
                uint32_t v[W];
                tmem_ld_32x32_n(taddr + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < W; ++j) st_cluster_u32(dst + j * 512, v[j]);
            };
            auto finish = [&](auto width, int c) {
                constexpr int W = decltype(width)::value;
                uint32_t ai[W], af[W];
                tmem_ld_32x32_n(taddr + c, ai);
                if (p.r > 0) tmem_ld_32x32_n(tadp + c, af);
                tmem_ld_wait();
                for (int u = 0; u < S - 1; ++u) {
                    const uint32_t *src = red + (u * own + c - c_own) * 128 + 32 * q + lane;
#pragma unroll
                    for (int j = 0; j < W; ++j) ai[j] += src[j * 128];
                }
                float v[W];
                // the scales one by one, as their product may leave the range
#pragma unroll
                for (int j = 0; j < W; ++j)
                    v[j] = fmaf((float)(int)ai[j] * ws, xs[c + j], p.r > 0 ? bits_to_f32(af[j]) : 0.0f);
                q8_store(v, p, n0 + c, m0 + 32 * q, lane, row_ok);
            };
            using W8 = std::integral_constant<int, 8>;
            using W2 = std::integral_constant<int, 2>;
            if (S > 1) {
                if (it > 0 && !__all_sync(0xffffffffu, mbar_wait_cluster(red_empty, (it - 1) & 1, abort_flag))) break;
                for (int i = 1; i < S; ++i) {
                    const int u = (rank + i) % S;  // the CTA that finishes columns [c0, c0 + n)
                    const int c0 = shares.first(u), n = shares.first(u + 1) - c0;
                    const uint32_t dst = cluster_addr(red + (rank - (rank > u)) * n * 128 + 32 * q + lane, u);
                    const int c_end = min(c0 + n, cols);
                    if (shares.step == 8) {
#pragma unroll 1
                        for (int c = c0; c < c_end; c += 8) push(W8{}, c, dst + (c - c0) * 512);
                    } else {
#pragma unroll 1
                        for (int c = c0; c < c_end; c += 2) push(W2{}, c, dst + (c - c0) * 512);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_rel(cluster_addr(red_full, u));
                }
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(red_full, it & 1, abort_flag))) break;
            }
            const int c_end = min(c_own + own, cols);
            if (shares.step == 8) {
#pragma unroll 1
                for (int c = c_own; c < c_end; c += 8) finish(W8{}, c);
            } else {
#pragma unroll 1
                for (int c = c_own; c < c_end; c += 2) finish(W2{}, c);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&acc_empty[it & 1]);
                for (int i = 1; i < S; ++i) mbar_arrive_cluster_rel(cluster_addr(red_empty, (rank + i) % S));
            }
        }
    } else if (!p.meta_tma) {
        // ------------------------------------------------------------ code loaders
        if (!q8_load_codes<C::CODE_WARPS, NS>(
                p.meta, p.M, p.K, warp - 6, lane, cluster, num_clusters, p.num_work, k0, k1, adp_kts,
                [&](int w) { return max(0, min(w % p.m_tiles * 128, p.M - 128)); },
                [&](int st) { return smem + st * C::STAGE_BYTES + C::A_BYTES + 2 * C::B_PANEL; },
                [&](int st, uint32_t phase) { return mbar_wait_warp(&empty[st], phase, abort_flag); },
                [&](int st) { mbar_arrive(&full[st]); }))
            goto done;
    }
done:
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (S > 1) cluster_sync();  // no CTA leaves while another may still signal it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace slope
