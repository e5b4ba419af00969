// skinny_q8.cuh -- the int8 2:4 product at a few tokens, on CUDA cores.
//
//   Y[t][o] = xscale[t] wscale[o] sum_j Xq[t][k(o, j)] Wq[o][j] + XL[t] . R[.][o]
//
// With Wq compressed: j runs over the kept values of row o and k(o, j) is
// where the codes place them.  At a few tokens the time is the streaming of
// Wq and its codes (0.625 bytes per dense weight), which a tensor-core tile
// cannot shorten, so the arithmetic only has to keep up: four kept values of
// two groups are one 32-bit word, their codes spread into a byte-permute
// selector that picks the four matching token bytes out of eight, and one
// 4-way dot product adds them.  Sums are exact in 32 bits, so their order
// does not matter.
//
// A CTA stages TB tokens' rows in shared memory (16-byte chunks, even and odd
// ones in two planes, so that a warp's reads of its 32 bytes per lane touch
// consecutive chunks), then its warps take groups of four output channels:
// the four share every token chunk read.  With few channels, `ksplit` warps
// of the CTA share a group, each taking every ksplit-th step of the sum.
//
// Taken at up to four tokens of small layers, where setting up the tensor-core
// tiles costs more than the sum (one token, 1024 -> 4096: 4.3 us against 5.3);
// on large ones the decoding of codes falls behind the loads (one token,
// 9216 -> 27648: the tiles' 31 us are 80% of the copy rate).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"
#include "skinny.cuh"
#include "rownorm.cuh"

namespace slope {

struct SkinnyQ8Params {
    const int8_t *X;        // [T x K]
    const float *xscale;    // [T]
    const int8_t *W;        // [M x K/2] kept values
    const float *wscale;    // [M]
    const uint16_t *meta;   // [M x K/16]
    const uint16_t *XL, *R; // [T x r], [r x M] bf16, or null with r = 0
    uint16_t *Y;            // [T x M]
    int T, K, M, r;
    int ksplit;             // warps that share a group of channels (a power of two up to SQ8_WARPS)
};

constexpr int SQ8_WARPS = 16;
constexpr int SQ8_ROWS = 4;  // output channels of a warp's group

// Selectors of two words of kept values (low and high half) from the 16-bit
// code word that covers them: each 2-bit position becomes a nibble, the
// second group's of a word offset by 4 (the second source of the permute).
__device__ __forceinline__ uint32_t code_selectors(uint32_t c) {
    c = (c | (c << 8)) & 0x00FF00FFu;
    c = (c | (c << 4)) & 0x0F0F0F0Fu;
    return ((c | (c << 2)) & 0x33333333u) | 0x44004400u;
}

template <int TB>
__global__ void __launch_bounds__(32 * SQ8_WARPS) skinny_q8_kernel(const __grid_constant__ SkinnyQ8Params p) {
    extern __shared__ __align__(16) uint8_t sq8_smem[];
    __shared__ int part[SQ8_WARPS][SQ8_ROWS * TB];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.y * TB;
    const int steps = (p.K + 1023) >> 10;       // 1024 dense positions a step, 32 to a lane
    const int chunks = steps * 64;              // 16-byte chunks of a staged row, zero past K
    uint4 *xs = reinterpret_cast<uint4 *>(sq8_smem);  // [TB][2 planes][chunks / 2]
    grid_dep_wait();
    grid_dep_launch();
    for (int i = tid; i < TB * chunks; i += blockDim.x) {
        const int t = i / chunks, c = i - t * chunks;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (t0 + t < p.T && 16 * c < p.K && in_bounds((int64_t)(t0 + t) * p.K + 16 * c, 16, (int64_t)p.T * p.K))
            v = *reinterpret_cast<const uint4 *>(p.X + (int64_t)(t0 + t) * p.K + 16 * c);
        xs[t * chunks + (c & 1) * (chunks >> 1) + (c >> 1)] = v;
    }
    __syncthreads();
    const int gpc = SQ8_WARPS / p.ksplit;       // groups of channels the CTA takes at once
    const int wg = warp / p.ksplit, ks = warp - wg * p.ksplit;
    const int64_t w_ext = (int64_t)p.M * (p.K / 2), m_ext = (int64_t)p.M * (p.K / 16);
    for (int g0 = blockIdx.x * gpc; g0 * SQ8_ROWS < p.M; g0 += gridDim.x * gpc) {
        const int o0 = (g0 + wg) * SQ8_ROWS;    // this warp's channels
        const bool live = o0 < p.M;             // M is a multiple of SQ8_ROWS
        int acc[SQ8_ROWS][TB];
#pragma unroll
        for (int q = 0; q < SQ8_ROWS; ++q)
#pragma unroll
            for (int t = 0; t < TB; ++t) acc[q][t] = 0;
        if (live) {
#pragma unroll 2
            for (int s = ks; s < steps; s += p.ksplit) {
                const int k = s * 1024 + lane * 32;  // dense position; K is a multiple of 64, so all 32 or none
                if (k < p.K) {
                    uint4 w[SQ8_ROWS];
                    uint32_t c[SQ8_ROWS];
#pragma unroll
                    for (int q = 0; q < SQ8_ROWS; ++q) {
                        const int64_t wo = (int64_t)(o0 + q) * (p.K / 2) + k / 2, mo = (int64_t)(o0 + q) * (p.K / 16) + k / 16;
                        w[q] = make_uint4(0, 0, 0, 0);
                        c[q] = 0x44444444u;
                        if (in_bounds(wo, 16, w_ext)) w[q] = __ldcs(reinterpret_cast<const uint4 *>(p.W + wo));
                        if (in_bounds(mo, 2, m_ext)) c[q] = __ldcs(reinterpret_cast<const uint32_t *>(p.meta + mo));
                    }
                    uint32_t sel[SQ8_ROWS][2];
#pragma unroll
                    for (int q = 0; q < SQ8_ROWS; ++q) {
                        sel[q][0] = code_selectors(c[q] & 0xFFFFu);
                        sel[q][1] = code_selectors(c[q] >> 16);
                    }
#pragma unroll
                    for (int t = 0; t < TB; ++t) {
                        const uint4 x0 = xs[t * chunks + (k >> 5)], x1 = xs[t * chunks + (chunks >> 1) + (k >> 5)];
#pragma unroll
                        for (int q = 0; q < SQ8_ROWS; ++q) {
                            int a = acc[q][t];
                            a = __dp4a((int)w[q].x, (int)__byte_perm(x0.x, x0.y, sel[q][0]), a);
                            a = __dp4a((int)w[q].y, (int)__byte_perm(x0.z, x0.w, sel[q][0] >> 16), a);
                            a = __dp4a((int)w[q].z, (int)__byte_perm(x1.x, x1.y, sel[q][1]), a);
                            a = __dp4a((int)w[q].w, (int)__byte_perm(x1.z, x1.w, sel[q][1] >> 16), a);
                            acc[q][t] = a;
                        }
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < SQ8_ROWS; ++q)
#pragma unroll
                for (int t = 0; t < TB; ++t) acc[q][t] = __reduce_add_sync(0xffffffffu, acc[q][t]);
        }
        if (p.ksplit > 1) {
            if (lane == 0) {
#pragma unroll
                for (int q = 0; q < SQ8_ROWS; ++q)
#pragma unroll
                    for (int t = 0; t < TB; ++t) part[warp][q * TB + t] = acc[q][t];
            }
            __syncthreads();
            if (ks == 0) {
#pragma unroll
                for (int q = 0; q < SQ8_ROWS; ++q)
#pragma unroll
                    for (int t = 0; t < TB; ++t) {
                        int a = 0;
                        for (int u = 0; u < p.ksplit; ++u) a += part[warp + u][q * TB + t];
                        acc[q][t] = a;
                    }
            }
            __syncthreads();
        }
        if (!live || ks != 0) continue;
        // the adapter: lanes share the rank
        float ad[SQ8_ROWS][TB];
#pragma unroll
        for (int q = 0; q < SQ8_ROWS; ++q)
#pragma unroll
            for (int t = 0; t < TB; ++t) ad[q][t] = 0.0f;
        if (p.r > 0) {
            for (int j = lane; j < p.r; j += 32) {
                uint2 rv = make_uint2(0, 0);
                if (in_bounds((int64_t)j * p.M + o0, 4, (int64_t)p.r * p.M))
                    rv = *reinterpret_cast<const uint2 *>(p.R + (int64_t)j * p.M + o0);
                const float2 ra = bf16x2_to_float2(rv.x), rb = bf16x2_to_float2(rv.y);
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    if (t0 + t < p.T && in_bounds((int64_t)(t0 + t) * p.r + j, 1, (int64_t)p.T * p.r)) {
                        const float x = __uint_as_float((uint32_t)p.XL[(int64_t)(t0 + t) * p.r + j] << 16);
                        ad[0][t] = fmaf(x, ra.x, ad[0][t]);
                        ad[1][t] = fmaf(x, ra.y, ad[1][t]);
                        ad[2][t] = fmaf(x, rb.x, ad[2][t]);
                        ad[3][t] = fmaf(x, rb.y, ad[3][t]);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < SQ8_ROWS; ++q)
#pragma unroll
                for (int t = 0; t < TB; ++t) ad[q][t] = warp_sum(ad[q][t]);
        }
        if (lane == 0 && in_bounds(o0, SQ8_ROWS, p.M)) {
            const float4 ws = *reinterpret_cast<const float4 *>(p.wscale + o0);
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                if (t0 + t < p.T && in_bounds((int64_t)(t0 + t) * p.M + o0, SQ8_ROWS, (int64_t)p.T * p.M)) {
                    const float x = p.xscale[t0 + t];
                    const uint32_t lo = pack_bf16x2(fmaf((float)acc[0][t] * ws.x, x, ad[0][t]), fmaf((float)acc[1][t] * ws.y, x, ad[1][t]));
                    const uint32_t hi = pack_bf16x2(fmaf((float)acc[2][t] * ws.z, x, ad[2][t]), fmaf((float)acc[3][t] * ws.w, x, ad[3][t]));
                    *reinterpret_cast<uint2 *>(p.Y + (int64_t)(t0 + t) * p.M + o0) = make_uint2(lo, hi);
                }
            }
        }
    }
}

}  // namespace slope
