// rownorm.cuh -- row-wise kernels around the int8 product: root-mean-square
// norm (with the residual's addition and an int8 output), its gradients, and
// the int8 quantiser of rows.
//
// Norm.  For a token row x (and the residual stream's row e, when there is
// one):  h = bf16(x + e),  rstd = (mean h^2 + eps)^(-1/2),
//        y = bf16((h w) rstd),  and in int8  y ~ q s  with
//        p = h w,  q = round(127 p / max|p|),  s = rstd max|p| / 127.
// The factor rstd cancels in q: p is the product of two bf16 numbers, exact in
// binary32 but at the ends of its range (see FAR_MAX), and q is decided exactly
// (quant_exact), so that q does not depend on how the sum of squares was
// ordered or rounded.
//
// Quantiser.  q = round(127 a / max|a|), s = max|a| / 127 for rows a of bf16
// values: the kept weights of an output channel, or tokens no norm produced.
//
// Gradients.  With n = h rstd and g = dY w:
//   dh = rstd (g - n mean(g n)) (+ the gradient arriving along the residual),
//   dw = sum over tokens of dY n.
//
// A row is read once, held in registers as bf16 while its statistics are
// reduced, and written once (but for the gradients of few rows, which read dY
// and H twice, and far_row): HBM bounds it at many rows, except the int8 output
// without a residual, which the instructions per value bound, and a launch's
// latency at few.  A row is one warp's up to 1024 values and one CTA's above,
// NV 16-byte chunks to a thread.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"
#include "skinny.cuh"  // bf16x2_to_float2

namespace slope {

constexpr int ROW_WARPS = 4;            // rows per CTA where a warp takes a row
constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A row's factors for the quantiser.  `f` brings max|p| into a range where
// 127 p and 127 / max|p| neither overflow nor lose bits (a power of two, so
// p f is exact for every p that does not quantise to zero).
struct QuantRow {
    float f, pm, inv;
};
__device__ __forceinline__ QuantRow quant_row(float pmax) {
    QuantRow q;
    q.f = pmax < 0x1p-60f ? 0x1p100f : pmax > 0x1p60f ? 0x1p-100f : 1.0f;
    q.pm = pmax * q.f;
    q.inv = pmax > 0.0f ? __fdividef(127.0f, q.pm) : 0.0f;
    return q;
}

__device__ __forceinline__ uint2 pack_codes(const float2 (&m)[4]) {  // the low bytes
    uint2 r;
    r.x = __byte_perm(__byte_perm(__float_as_uint(m[0].x), __float_as_uint(m[0].y), 0x0040),
                      __byte_perm(__float_as_uint(m[1].x), __float_as_uint(m[1].y), 0x0040), 0x5410);
    r.y = __byte_perm(__byte_perm(__float_as_uint(m[2].x), __float_as_uint(m[2].y), 0x0040),
                      __byte_perm(__float_as_uint(m[3].x), __float_as_uint(m[3].y), 0x0040), 0x5410);
    return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
constexpr float ROUND_MAGIC = 12582912.0f;  // 1.5 2^23: adding it rounds to an integer in the float's low bits

// The largest of |a|, |b|, |c|, or NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// round(127 p / max|p|), ties to even, decided exactly for t = p f: k is the
// rounding of the binary32 quotient, off by at most one beside a border.
// 127 t has at most 23 significant bits and k pm too (7 + 16), and their
// difference d, a multiple of t's last place, fits 24, so d is exact:
// |d| > pm / 2 moves k by one, |d| = pm / 2 is a tie.
__device__ __forceinline__ float quant_exact(float t, float k, float pm) {
    const float d = fmaf(-k, pm, 127.0f * t), a = fabsf(d), half = 0.5f * pm;
    const bool odd = (static_cast<int>(k) & 1) != 0;
    return (a > half || (a == half && odd)) ? k + copysignf(1.0f, d) : k;
}

// Eight products of two bf16 numbers to int8 codes.  The fused p inv is off by
// at most 2^-14 (inv two units of 2^-23 of 127, the difference below half of
// 2^-24); one within 2^-13 of a border (2.4 in 10^4 of them) is decided again
// by quant_exact.
__device__ __forceinline__ uint2 quant8(float2 (&p)[4], const QuantRow &q) {
    if (q.f != 1.0f) {
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = __fmul2_rn(p[k], both(q.f));
    }
    float2 m[4];
    float worst = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m[k] = __ffma2_rn(p[k], both(q.inv), both(ROUND_MAGIC));
        const float2 neg = __ffma2_rn(m[k], both(-1.0f), both(ROUND_MAGIC));  // minus the rounded value
        const float2 d = __ffma2_rn(p[k], both(q.inv), neg);
        worst = max_abs3(worst, d.x, d.y);
    }
    if (worst > 0.5f - 0x1p-13f) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m[k].x = quant_exact(p[k].x, m[k].x - ROUND_MAGIC, q.pm) + ROUND_MAGIC;
            m[k].y = quant_exact(p[k].y, m[k].y - ROUND_MAGIC, q.pm) + ROUND_MAGIC;
        }
    }
    return pack_codes(m);
}

// Eight bf16 values to int8 codes.  With eight significant bits on either
// side, a quotient t = 127 a / max|a| that is not a border k + 1/2 is further
// than t / (254 255) = 1.5 10^-5 t from it, and a inv is off by at most
// 3 10^-7 t: rounding it to 18 bits after the leading one (steps of 2^-18, at
// most 3.8 10^-6 of it) leaves every border exact and moves nothing else
// onto one or across it, and the rounding to an integer then breaks ties to even.
// The rounding is Dekker's split: a inv - g with g about 33 a inv has the last
// place of 32 a inv, which is 2^-18 of a inv's leading one, g is a multiple of
// it, and so g plus the difference is exact.
__device__ __forceinline__ uint2 quant8_rows(float2 (&a)[4], const QuantRow &q) {
    if (q.f != 1.0f) {
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = __fmul2_rn(a[k], both(q.f));
    }
    const float inv33 = q.inv * 33.0f;
    float2 m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 neg = __fmul2_rn(a[k], both(-inv33));               // -g
        const float2 d = __ffma2_rn(a[k], both(q.inv), neg);             // a inv - g
        const float2 t = __ffma2_rn(neg, both(-1.0f), d);                // a inv, split
        m[k] = __fadd2_rn(t, both(ROUND_MAGIC));
    }
    return pack_codes(m);
}

struct RowParams {
    const uint16_t *X;    // [T x D] tokens (or the quantiser's rows)
    const uint16_t *res;  // [T x D] residual stream, or null
    const uint16_t *w;    // [D] norm weight
    uint16_t *H;          // [T x D] bf16(X + res), or null
    uint16_t *Y;          // [T x D] normalised tokens, or null
    int8_t *Q;            // [T x D] int8, or null
    float *qscale;        // [T], with Q
    float *rstd;          // [T], or null
    int64_t T;
    int D;
    float eps;
};

// h = bf16(x + e), eight values.
__device__ __forceinline__ uint4 add_bf16x8(uint4 x, uint4 e) {
    uint32_t a[4] = {x.x, x.y, x.z, x.w};
    const uint32_t b[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 u = bf16x2_to_float2(a[k]), v = bf16x2_to_float2(b[k]);
        a[k] = pack_bf16x2(u.x + v.x, u.y + v.y);
    }
    return make_uint4(a[0], a[1], a[2], a[3]);
}

// Eight values' p = h w (the quantiser: a), and their share of a row's
// statistics.  The norm: the sums of the even and of the odd squares and the largest |p| as a float's
// bits (NaN, larger than any number, if one is).  The quantiser: the largest
// |a| of the even and of the odd values, as two bf16 patterns (an infinity's
// or a NaN's is larger than any number's).
template <bool NORM>
__device__ __forceinline__ void row_stats(uint4 h, uint4 w, float2 (&v)[4], float2 &ss, uint32_t &mx) {
    const uint32_t a[4] = {h.x, h.y, h.z, h.w}, b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[k] = bf16x2_to_float2(a[k]);
        if (NORM) {
            ss = __ffma2_rn(v[k], v[k], ss);
            v[k] = __fmul2_rn(v[k], bf16x2_to_float2(b[k]));
            mx = __float_as_uint(max_abs3(__uint_as_float(mx), v[k].x, v[k].y));
        } else {
            mx = __vmaxu2(mx, a[k] & 0x7FFF7FFFu);
        }
    }
}
// A thread's statistic as the bits of a float, comparable as an integer.
template <bool NORM>
__device__ __forceinline__ uint32_t row_max_bits(uint32_t mx) {
    return NORM ? mx & 0x7FFFFFFFu : max(mx << 16, mx & 0xFFFF0000u);
}

// Rows whose mean square plus eps, m, leaves binary32's normal range (an
// overflow, or with an eps below it) take their squares again, of h f with f a
// power of two; 1 for all others.  An infinity in the row stays one.
__device__ __forceinline__ float square_factor(float m) {
    return __float_as_uint(m) == kInfBits ? 0x1p-80f : m < 0x1p-120f ? 0x1p80f : 1.0f;
}
// Sum of the squares of h f, eight values.
__device__ __forceinline__ float scaled_squares(uint4 h, float f, float s2) {
    const uint32_t a[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 u = bf16x2_to_float2(a[k]);
        s2 = fmaf(u.x * f, u.x * f, fmaf(u.y * f, u.y * f, s2));
    }
    return s2;
}

// Products of two bf16 numbers have 16 significant bits, so binary32, whose
// last place is 2^-149, holds them down to 2^-134.  In a row whose largest
// product is FAR_MAX or more, what it loses below quantises to zero.  In others
// (rows of zeros apart) p is taken in binary64 times 2^200, which is exact and
// in range: products of bf16 numbers start at 2^-266.
// Y takes the products' low bits only where rstd is large enough to bring them
// back above bf16's own smallest values (last place 2^-133): above FAR_RSTD
// y = h w rstd, where it is asked for, is taken in binary64 as well.  So it is in
// a row with a product that is not finite in binary32: y may be.
constexpr float FAR_MAX = 0x1p-110f, FAR_RSTD = 0x1p14f;
__device__ __forceinline__ bool far_candidate(const RowParams &p, uint32_t mx, float rstd) {  // mx: the largest |p| as a float's bits
    const uint32_t least = __float_as_uint(FAR_MAX);
    return mx - least >= kInfBits - least || (rstd > FAR_RSTD && p.Y);
}
__device__ __forceinline__ float2 far_products(uint32_t h, uint32_t w) {
    const float2 x = bf16x2_to_float2(h), y = bf16x2_to_float2(w);
    return make_float2((float)((double)x.x * y.x * 0x1p200), (float)((double)x.y * y.y * 0x1p200));
}
// Whether any of the eight products is not zero.
__device__ __forceinline__ bool any_product(uint4 h, uint4 w) {
    const uint32_t a[4] = {h.x, h.y, h.z, h.w}, b[4] = {w.x, w.y, w.z, w.w};
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) any |= __vminu2(a[k] & 0x7FFF7FFFu, b[k] & 0x7FFF7FFFu);
    return any != 0;
}

// Eight outputs of a row from its p (h w, or the quantiser's values): y = p rstd and the codes of p.
template <bool NORM>
__device__ __forceinline__ void row_outputs(const RowParams &p, int64_t at, float2 (&v)[4], float rstd, const QuantRow &q,
                                            bool finite) {
    if (NORM && p.Y) {
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 t = __fmul2_rn(v[k], both(rstd));
            y[k] = pack_bf16x2(t.x, t.y);
        }
        *reinterpret_cast<uint4 *>(p.Y + at) = make_uint4(y[0], y[1], y[2], y[3]);
    }
    if (p.Q) *reinterpret_cast<uint2 *>(p.Q + at) = !finite ? make_uint2(0, 0) : NORM ? quant8(v, q) : quant8_rows(v, q);
}

// The outputs of a row that takes binary64, by its warp or CTA (`group` threads
// of which this is number gi; s_max: 32 words that nobody reads any more).  A
// call that reads the row again, two values at a time, so that the other rows'
// registers do not pay for it.  `mx`: the row's largest |p| as a float's bits.
template <bool WARP>
__device__ __noinline__ void far_row(const RowParams &p, int64_t row, int gi, int group, float rstd, uint32_t mx, uint32_t *s_max) {
    const int64_t base = row * p.D, total = p.T * p.D;
    const bool tiny = mx < __float_as_uint(FAR_MAX);
    // Values 2 j and 2 j + 1 of this thread's chunks.  H, which it has written, may be the buffer of X or res.
    auto load = [&](int j, uint32_t &h, uint32_t &w) {
        h = w = 0;
        if (!in_bounds(base + 2 * j, 2, total) || !in_bounds(2 * j, 2, p.D)) return;
        w = *reinterpret_cast<const uint32_t *>(p.w + 2 * j);
        h = *reinterpret_cast<const uint32_t *>((p.H ? p.H : p.X) + base + 2 * j);
        if (p.res && !p.H) {
            const float2 x = bf16x2_to_float2(h), e = bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(p.res + base + 2 * j));
            h = pack_bf16x2(x.x + e.x, x.y + e.y);
        }
    };
    if (tiny) {
        float most = 0.0f;
#pragma unroll 1
        for (int c = gi; c < p.D >> 3; c += group)
#pragma unroll 1
            for (int j = 4 * c; j < 4 * c + 4; ++j) {
                uint32_t h, w;
                load(j, h, w);
                const float2 v = far_products(h, w);
                most = fmaxf(most, fmaxf(fabsf(v.x), fabsf(v.y)));
            }
        mx = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
        if (!WARP) {
            if ((gi & 31) == 0) s_max[gi >> 5] = mx;
            __syncthreads();
            mx = __reduce_max_sync(0xffffffffu, (gi & 31) < (group >> 5) ? s_max[gi & 31] : 0u);
        }
    }
    const float pmax = __uint_as_float(mx);
    const QuantRow q = quant_row(pmax);
    const double unit = tiny ? (double)q.f * 0x1p200 : (double)q.f;
    if (p.Q && gi == 0 && in_bounds(row, 1, p.T))
        p.qscale[row] = mx >= kInfBits ? __uint_as_float(0x7FC00000u)
                        : tiny         ? (float)((double)rstd * pmax / 127.0 * 0x1p-200) : rstd * (pmax / 127.0f);
#pragma unroll 1
    for (int c = gi; c < p.D >> 3; c += group)
#pragma unroll 1
        for (int j = 4 * c; j < 4 * c + 4; ++j) {
            uint32_t h, w;
            load(j, h, w);
            if (!in_bounds(base + 2 * j, 2, total)) continue;
            const float2 x = bf16x2_to_float2(h), u = bf16x2_to_float2(w);
            const double px = (double)x.x * u.x, py = (double)x.y * u.y;
            if (p.Y) *reinterpret_cast<uint32_t *>(p.Y + base + 2 * j) = pack_bf16x2((float)(px * rstd), (float)(py * rstd));
            if (p.Q) {
                const float vx = (float)(px * unit), vy = (float)(py * unit);
                const int a = static_cast<int>(quant_exact(vx, rintf(vx * q.inv), q.pm));
                const int b = static_cast<int>(quant_exact(vy, rintf(vy * q.inv), q.pm));
                *reinterpret_cast<uint16_t *>(p.Q + base + 2 * j) = static_cast<uint16_t>(mx < kInfBits ? (a & 0xFF) | (b & 0xFF) << 8 : 0);
            }
        }
}

// NORM: the norm; otherwise the quantiser.  WARP: a warp per row, otherwise a
// CTA per row, held in registers.  H may be the buffer of X or res, and Y that
// of any of them: a thread reads its chunks of a row before it writes those
// same chunks.
template <int NV, bool WARP, bool NORM>
__global__ void __launch_bounds__(WARP ? 32 * ROW_WARPS : 1024) row_kernel(const __grid_constant__ RowParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gsize = WARP ? 32 : blockDim.x, gi = WARP ? lane : threadIdx.x;
    const int64_t row = WARP ? (int64_t)blockIdx.x * ROW_WARPS + warp : (int64_t)blockIdx.x;
    const int nchunk = p.D >> 3;
    const int64_t total = p.T * p.D;
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    grid_dep_wait();
    grid_dep_launch();
    if (WARP && row >= p.T) return;

    uint4 h[NV];
    const float inv_d = 1.0f / (float)p.D;
    const int64_t base = row * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = gi + i * gsize;
        h[i] = make_uint4(0, 0, 0, 0);
        if (c < nchunk && in_bounds(base + 8 * c, 8, total)) h[i] = *reinterpret_cast<const uint4 *>(p.X + base + 8 * c);
    }
    if (NORM && p.res) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = gi + i * gsize;
            if (c < nchunk && in_bounds(base + 8 * c, 8, total)) {
                h[i] = add_bf16x8(h[i], *reinterpret_cast<const uint4 *>(p.res + base + 8 * c));
                if (p.H) *reinterpret_cast<uint4 *>(p.H + base + 8 * c) = h[i];
            }
        }
    }
    auto weight = [&](int c) {
        return NORM && c < nchunk && in_bounds(8 * c, 8, p.D) ? __ldg(reinterpret_cast<const uint4 *>(p.w + 8 * c))
                                                              : make_uint4(0, 0, 0, 0);
    };
    float2 ss2 = make_float2(0.0f, 0.0f);
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float2 v[4];
        row_stats<NORM>(h[i], weight(gi + i * gsize), v, ss2, mx);
    }
    float ss = NORM ? warp_sum(ss2.x + ss2.y) : 0.0f;
    mx = __reduce_max_sync(0xffffffffu, row_max_bits<NORM>(mx));
    if (!WARP) {
        if (lane == 0) {
            s_sum[warp] = ss;
            s_max[warp] = mx;
        }
        __syncthreads();
        const int nw = blockDim.x >> 5;
        ss = warp_sum(lane < nw ? s_sum[lane] : 0.0f);
        mx = __reduce_max_sync(0xffffffffu, lane < nw ? s_max[lane] : 0u);
    }

    float rstd = 1.0f;
    if (NORM) {
        const float m = fmaf(ss, inv_d, p.eps), f = square_factor(m);
        rstd = rsqrtf(m);
        if (f != 1.0f) {  // (an infinity in the row gives rstd = 0, and NaN beside it)
            float s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) s2 = scaled_squares(h[i], f, s2);
            s2 = warp_sum(s2);
            if (!WARP) {
                __syncthreads();  // every thread has read the first sums
                if (lane == 0) s_sum[warp] = s2;
                __syncthreads();
                s2 = warp_sum(lane < (int)(blockDim.x >> 5) ? s_sum[lane] : 0.0f);
            }
            rstd = rsqrtf(fmaf(s2, inv_d, p.eps * f * f)) * f;
        }
        if (p.rstd && gi == 0 && in_bounds(row, 1, p.T)) p.rstd[row] = rstd;
    }
    if (NORM && far_candidate(p, mx, rstd)) {
        bool far = true;
        if (mx < __float_as_uint(FAR_MAX)) {  // not for a row of zeros; in a CTA every thread has read the maxima, then
            bool any = false;
#pragma unroll
            for (int i = 0; i < NV; ++i) any |= any_product(h[i], weight(gi + i * gsize));
            far = WARP ? __any_sync(0xffffffffu, any) : __syncthreads_or(any) != 0;
        }
        if (far) {
            far_row<WARP>(p, row, gi, gsize, rstd, mx, s_max);
            return;
        }
    }
    const bool finite = NORM || mx < kInfBits;
    const float pmax = __uint_as_float(mx);
    const QuantRow q = quant_row(finite ? pmax : 0.0f);
    // without this the compiler keeps the row's p across the reductions: 50 registers for 43 with two chunks a thread
#pragma unroll
    for (int i = 0; i < NV; ++i) asm volatile("" : "+r"(h[i].x), "+r"(h[i].y), "+r"(h[i].z), "+r"(h[i].w));
    if (p.Q && gi == 0 && in_bounds(row, 1, p.T))
        p.qscale[row] = finite ? rstd * (pmax / 127.0f) : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = gi + i * gsize;
        if (c < nchunk && in_bounds(base + 8 * c, 8, total)) {
            float2 v[4], s_unused = make_float2(0.0f, 0.0f);
            uint32_t m_unused = 0;
            row_stats<NORM>(h[i], weight(c), v, s_unused, m_unused);
            row_outputs<NORM>(p, base + 8 * c, v, rstd, q, finite);
        }
    }
}

// The same for many long rows: CTAs that take several rows each, with a ring of
// two rows (X, and res beside it) that bulk copies keep filled, so that the
// load of the next row runs beside the arithmetic and the stores of this one.
// The row and the weight stay in registers between the statistics and the
// outputs.  A CTA's rows take one barrier each: when it falls every thread has
// read its chunks, and the row's stage is refilled.
//
// 8192 x 9216 in a row of calls: with residual and both outputs (9 bytes a
// value) one row per CTA and nothing ahead takes 139 us, one CTA of this per
// SM with four stages 115, with two 109 (fewer reads in flight disturb the
// writes less), and eight rounds of two CTAs per SM 104, 100% of the measured
// copy rate: SMs differ in speed, and rounds let the fast ones take more.
// Without the residual there is less to load per barrier, and the instructions
// (22 a value in int8, of which the reductions and the barrier are about five)
// bound it: 53 us in bf16, 67 in int8.  The quantiser takes 36 (96%).
constexpr int STREAM_STAGES = 2;
constexpr int STREAM_WARPS = 8;  // rows in work at once in a CTA of the gradients' warp form
// Threads at most and CTAs per SM of a form with NV chunks a thread.  Norm:
// 12288 with everything 143 us with two CTAs per SM, 151 with one; 16384 99
// us (4096 rows) with one, 127 with two, which spill.  Quantiser: 9216 36 us
// with four, 38 with two; 12288 50 and 48.  Few chunks to many threads beat more to fewer
// (16384: 99 us with six, 196 with eight, which spill).
constexpr int stream_threads(int nv, bool norm, bool warp) { return warp ? 32 * STREAM_WARPS : nv <= 6 ? 384 : norm ? 512 : 1024; }
constexpr int stream_ctas(int nv, bool norm) { return norm ? (nv <= 2 ? 3 : nv <= 4 ? 2 : 1) : nv <= 3 ? 4 : nv <= 6 ? 2 : 1; }
constexpr int stream_bwd_ctas(int nv, bool warp) { return warp ? (nv <= 2 ? 3 : 2) : nv <= 2 ? 3 : nv == 3 ? 2 : 1; }
template <int NV, bool NORM>
__global__ void __launch_bounds__(stream_threads(NV, NORM, false), stream_ctas(NV, NORM))
    row_stream_kernel(const __grid_constant__ RowParams p) {
    extern __shared__ __align__(16) uint8_t row_smem[];
    __shared__ __align__(8) uint64_t full[STREAM_STAGES];
    __shared__ float s_sum[2][32];
    __shared__ uint32_t s_max[2][32];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int gi = threadIdx.x, gsize = blockDim.x;
    const int nchunk = p.D >> 3;
    const int64_t total = p.T * p.D;
    const uint32_t row_bytes = (uint32_t)p.D * 2;
    const bool has_res = NORM && p.res;
    const uint32_t stage_bytes = has_res ? 2 * row_bytes : row_bytes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STREAM_STAGES; ++i) mbar_init(&full[i], 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row0 = blockIdx.x, step = gridDim.x;
    auto fetch = [&](int64_t row, int s) {  // one thread
        if (row >= p.T || !in_bounds(row * p.D, p.D, total)) return;
        uint8_t *dst = row_smem + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        bulk_load(dst, p.X + row * p.D, row_bytes, &full[s]);
        if (has_res) bulk_load(dst + row_bytes, p.res + row * p.D, row_bytes, &full[s]);
    };
    if (gi == 0)
        for (int s = 0; s < STREAM_STAGES; ++s) fetch(row0 + s * step, s);
    uint4 w[NV];
    auto load_w = [&]() {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = gi + i * gsize;
            w[i] = NORM && c < nchunk && in_bounds(8 * c, 8, p.D) ? __ldg(reinterpret_cast<const uint4 *>(p.w + 8 * c))
                                                                  : make_uint4(0, 0, 0, 0);
        }
    };
    load_w();
    const float inv_d = 1.0f / (float)p.D;
    int s = 0, turn = 0;
    uint32_t ph = 0;
    for (int64_t row = row0; row < p.T; row += step) {
        const int64_t base = row * p.D;
        const uint8_t *src = row_smem + s * stage_bytes;
        auto load_h = [&](int c) {
            uint4 h = *reinterpret_cast<const uint4 *>(src + 16 * c);
            if (has_res) h = add_bf16x8(h, *reinterpret_cast<const uint4 *>(src + row_bytes + 16 * c));
            return h;
        };
        // a copy that does not come gives up after its limit, and the thread works on what is there
        mbar_wait(&full[s], ph, &abort_flag);
        __syncwarp();
        uint4 held[NV];  // h, or the quantiser's row
        float2 v[4], ss2 = make_float2(0.0f, 0.0f);
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = gi + i * gsize;
            uint4 h = make_uint4(0, 0, 0, 0);
            if (c < nchunk) {
                h = load_h(c);
                if (has_res && p.H && in_bounds(base + 8 * c, 8, total)) *reinterpret_cast<uint4 *>(p.H + base + 8 * c) = h;
            }
            row_stats<NORM>(h, w[i], v, ss2, mx);
            held[i] = h;
        }
        float ss = NORM ? warp_sum(ss2.x + ss2.y) : 0.0f;
        mx = __reduce_max_sync(0xffffffffu, row_max_bits<NORM>(mx));
        if (lane == 0) {
            s_sum[turn][warp] = ss;
            s_max[turn][warp] = mx;
        }
        __syncthreads();
        if (NORM) ss = warp_sum(lane < nw ? s_sum[turn][lane] : 0.0f);
        mx = __reduce_max_sync(0xffffffffu, lane < nw ? s_max[turn][lane] : 0u);
        // without this the compiler keeps the row's p and the weight as floats across the barrier, twice the registers
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            asm volatile("" : "+r"(held[i].x), "+r"(held[i].y), "+r"(held[i].z), "+r"(held[i].w));
            if (NORM) asm volatile("" : "+r"(w[i].x), "+r"(w[i].y), "+r"(w[i].z), "+r"(w[i].w));
        }
        float rstd = 1.0f;
        if (NORM) {
            const float m = fmaf(ss, inv_d, p.eps), f = square_factor(m);
            rstd = rsqrtf(m);
            if (f != 1.0f) {
                float s2 = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i) s2 = scaled_squares(held[i], f, s2);
                s2 = warp_sum(s2);
                __syncthreads();
                if (lane == 0) s_sum[turn][warp] = s2;
                __syncthreads();
                s2 = warp_sum(lane < nw ? s_sum[turn][lane] : 0.0f);
                rstd = rsqrtf(fmaf(s2, inv_d, p.eps * f * f)) * f;
            }
        }
        if (gi == 0) {
            // every thread has read the stage
            fetch(row + STREAM_STAGES * step, s);
            if (NORM && p.rstd && in_bounds(row, 1, p.T)) p.rstd[row] = rstd;
        }
        bool far = NORM && far_candidate(p, mx, rstd);
        if (far && mx < __float_as_uint(FAR_MAX)) {  // see row_kernel
            bool any = false;
#pragma unroll
            for (int i = 0; i < NV; ++i) any |= any_product(held[i], w[i]);
            far = __syncthreads_or(any) != 0;
        }
        ph ^= s;
        s ^= 1;
        turn ^= 1;  // the next row's sums go beside this row's, which other warps may still read
        if (far) {
            far_row<false>(p, row, gi, gsize, rstd, mx, s_max[turn ^ 1]);
            load_w();  // rather than hold it across the call
            continue;
        }
        const bool finite = NORM || mx < kInfBits;
        const float pmax = __uint_as_float(mx);
        const QuantRow q = quant_row(finite ? pmax : 0.0f);
        if (p.Q && gi == 0 && in_bounds(row, 1, p.T))
            p.qscale[row] = finite ? rstd * (pmax / 127.0f) : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = gi + i * gsize;
            if (c < nchunk && in_bounds(base + 8 * c, 8, total)) {
                row_stats<NORM>(held[i], w[i], v, ss2, mx);  // p again
                row_outputs<NORM>(p, base + 8 * c, v, rstd, q, finite);
            }
        }
    }
}

struct RowBwdParams {
    const uint16_t *dY, *H, *w;
    const float *rstd;
    const uint16_t *dres;  // or null
    uint16_t *dH;
    float *dw;             // [D], written by row_bwd_once_kernel
    float *part;           // [parts x D] partial sums of dw
    int64_t T;
    int D;
    int parts;             // CTAs of the launch
};

// Both gradients in one launch, without partial sums: dw needs no row's
// statistics but rstd, which is given, so the launch's last CTAs compute it
// from columns while the others compute dH from rows.  They read dY and H once
// more (from L2, where few rows leave them), which costs less than a second
// launch and its scratch up to about a thousand rows: 4.6 against 6.1 us at
// 777 x 1000, but 10.1 against 7.9 at 2048 x 1024.
//
// Row CTAs: one row (a warp's each where they are short) held in registers.
// Column CTAs: 32 columns, 16 bytes to a thread, the rows spread over the
// CTA's groups of four threads and their sums added in a fixed order.
constexpr int BWD_COLS = 32;
template <int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 64 * ROW_WARPS : 1024) row_bwd_once_kernel(const __grid_constant__ RowBwdParams p, int row_ctas) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nchunk = p.D >> 3;
    const int64_t total = p.T * p.D;
    __shared__ float s_sum[32][BWD_COLS];
    grid_dep_wait();
    grid_dep_launch();
    if ((int)blockIdx.x >= row_ctas) {
        const int c = ((int)blockIdx.x - row_ctas) * (BWD_COLS / 8) + (threadIdx.x & 3);  // this thread's 16 bytes of a row
        const int groups = blockDim.x >> 2;
        float acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
        if (c < nchunk) {
#pragma unroll 4
            for (int64_t t = threadIdx.x >> 2; t < p.T; t += groups) {
                const int64_t at = t * p.D + 8 * c;
                if (!in_bounds(at, 8, total) || !in_bounds(t, 1, p.T)) continue;
                const uint4 hv = *reinterpret_cast<const uint4 *>(p.H + at), gv = *reinterpret_cast<const uint4 *>(p.dY + at);
                const float rstd = p.rstd[t];
                const uint32_t a[4] = {hv.x, hv.y, hv.z, hv.w}, b[4] = {gv.x, gv.y, gv.z, gv.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 hh = bf16x2_to_float2(a[k]), gg = bf16x2_to_float2(b[k]);
                    acc[2 * k] = fmaf(gg.x, hh.x * rstd, acc[2 * k]);
                    acc[2 * k + 1] = fmaf(gg.y, hh.y * rstd, acc[2 * k + 1]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
        if (lane < 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) s_sum[warp][8 * lane + j] = acc[j];
        }
        __syncthreads();
        const int d = ((int)blockIdx.x - row_ctas) * BWD_COLS + threadIdx.x;
        if (threadIdx.x < BWD_COLS && d < p.D) {
            float t = s_sum[0][threadIdx.x];
            for (int k = 1; k < (int)(blockDim.x >> 5); ++k) t += s_sum[k][threadIdx.x];
            if (in_bounds(d, 1, p.D)) p.dw[d] = t;
        }
        return;
    }
    const int gsize = WARP ? 32 : blockDim.x, gi = WARP ? lane : threadIdx.x;
    const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : (int64_t)blockIdx.x;
    if (WARP && row >= p.T) return;
    const int64_t base = row * p.D;
    const float rstd = in_bounds(row, 1, p.T) ? p.rstd[row] : 0.0f;
    uint4 h[NV], g[NV];
    float dot = 0.0f;  // sum of g n
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = gi + i * gsize;
        h[i] = g[i] = make_uint4(0, 0, 0, 0);
        if (c < nchunk && in_bounds(base + 8 * c, 8, total)) {
            h[i] = *reinterpret_cast<const uint4 *>(p.H + base + 8 * c);
            g[i] = *reinterpret_cast<const uint4 *>(p.dY + base + 8 * c);
        }
    }
    auto weight = [&](int c) {
        return c < nchunk && in_bounds(8 * c, 8, p.D) ? __ldg(reinterpret_cast<const uint4 *>(p.w + 8 * c)) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint4 wv = weight(gi + i * gsize);
        const uint32_t a[4] = {h[i].x, h[i].y, h[i].z, h[i].w}, b[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
        const uint32_t d[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 hh = bf16x2_to_float2(a[k]), gg = bf16x2_to_float2(b[k]), ww = bf16x2_to_float2(d[k]);
            dot = fmaf(gg.x * ww.x, hh.x * rstd, fmaf(gg.y * ww.y, hh.y * rstd, dot));
        }
    }
    dot = warp_sum(dot);
    if (!WARP) {
        if (lane == 0) s_sum[0][warp] = dot;
        __syncthreads();
        dot = warp_sum(lane < (int)(blockDim.x >> 5) ? s_sum[0][lane] : 0.0f);
    }
    const float mean = dot / (float)p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = gi + i * gsize;
        if (c >= nchunk || !in_bounds(base + 8 * c, 8, total)) continue;
        const uint4 wv = weight(c);
        uint4 ev = make_uint4(0, 0, 0, 0);
        if (p.dres) ev = *reinterpret_cast<const uint4 *>(p.dres + base + 8 * c);
        const uint32_t a[4] = {h[i].x, h[i].y, h[i].z, h[i].w}, b[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
        const uint32_t d[4] = {wv.x, wv.y, wv.z, wv.w}, e[4] = {ev.x, ev.y, ev.z, ev.w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 hh = bf16x2_to_float2(a[k]), gg = bf16x2_to_float2(b[k]), ww = bf16x2_to_float2(d[k]);
            const float2 ee = bf16x2_to_float2(e[k]);
            o[k] = pack_bf16x2(fmaf(rstd, fmaf(-hh.x * rstd, mean, gg.x * ww.x), ee.x),
                               fmaf(rstd, fmaf(-hh.y * rstd, mean, gg.y * ww.y), ee.y));
        }
        *reinterpret_cast<uint4 *>(p.dH + base + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// Many rows: persistent groups (a warp up to 1024 values, a CTA above) with the
// rings of row_stream_kernel.  A group
// keeps its sum of dY n in registers, a CTA writes its groups' sum as one row
// of `part`, and dw_sum_kernel adds those rows in a fixed order.  The second
// pass reads the row again from shared memory, so registers hold only the sums
// and the weight.  A warp refills a stage after its own second pass, a CTA
// after the next row's barrier, when every thread is done with it.  8192 x 5120
// with dres (8 bytes a value): 59 us, 86% of the copy rate.
template <int NV, bool WARP>
__global__ void __launch_bounds__(stream_threads(NV, true, WARP), stream_bwd_ctas(NV, WARP))
    row_bwd_stream_kernel(const __grid_constant__ RowBwdParams p) {
    extern __shared__ __align__(16) uint8_t row_smem[];
    constexpr int GROUPS = WARP ? STREAM_WARPS : 1;
    __shared__ __align__(8) uint64_t s_full[GROUPS][STREAM_STAGES];
    __shared__ float s_sum[2][32];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int gi = WARP ? lane : threadIdx.x, gsize = WARP ? 32 : blockDim.x, group = WARP ? warp : 0;
    const int nchunk = p.D >> 3;
    const int64_t total = p.T * p.D;
    const uint32_t row_bytes = (uint32_t)p.D * 2;
    const uint32_t stage_bytes = (p.dres ? 3 : 2) * row_bytes;
    uint8_t *ring = row_smem + (uint32_t)(group * STREAM_STAGES) * stage_bytes;
    uint64_t *full = s_full[group];
    if (threadIdx.x == 0) {
        for (int i = 0; i < GROUPS * STREAM_STAGES; ++i) mbar_init(&s_full[0][0] + i, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row0 = (int64_t)blockIdx.x * GROUPS + group, step = (int64_t)gridDim.x * GROUPS;
    auto fetch = [&](int64_t row, int s) {  // one thread of the group
        if (row >= p.T || !in_bounds(row * p.D, p.D, total)) return;
        uint8_t *dst = ring + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        bulk_load(dst, p.H + row * p.D, row_bytes, &full[s]);
        bulk_load(dst + row_bytes, p.dY + row * p.D, row_bytes, &full[s]);
        if (p.dres) bulk_load(dst + 2 * row_bytes, p.dres + row * p.D, row_bytes, &full[s]);
    };
    if (gi == 0)
        for (int s = 0; s < STREAM_STAGES; ++s) fetch(row0 + s * step, s);
    uint4 w[NV];
    float acc[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = gi + i * gsize;
        w[i] = c < nchunk && in_bounds(8 * c, 8, p.D) ? __ldg(reinterpret_cast<const uint4 *>(p.w + 8 * c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    }
    const float inv_d = 1.0f / (float)p.D;
    int s = 0, turn = 0;
    uint32_t ph = 0;
    for (int64_t row = row0; row < p.T; row += step) {
        const int64_t base = row * p.D;
        const uint8_t *src = ring + s * stage_bytes;
        const float rstd = in_bounds(row, 1, p.T) ? __ldg(p.rstd + row) : 0.0f;
        mbar_wait(&full[s], ph, &abort_flag);
        __syncwarp();
        float dot = 0.0f;  // sum of g n
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = gi + i * gsize;
            if (c < nchunk) {
                const uint4 hv = *reinterpret_cast<const uint4 *>(src + 16 * c);
                const uint4 gv = *reinterpret_cast<const uint4 *>(src + row_bytes + 16 * c);
                const uint32_t a[4] = {hv.x, hv.y, hv.z, hv.w}, b[4] = {gv.x, gv.y, gv.z, gv.w};
                const uint32_t d[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 hh = bf16x2_to_float2(a[k]), gg = bf16x2_to_float2(b[k]), ww = bf16x2_to_float2(d[k]);
                    const float dnx = gg.x * (hh.x * rstd), dny = gg.y * (hh.y * rstd);  // dY n
                    dot = fmaf(dnx, ww.x, fmaf(dny, ww.y, dot));
                    acc[i][2 * k] += dnx;
                    acc[i][2 * k + 1] += dny;
                }
            }
        }
        dot = warp_sum(dot);
        if (!WARP) {
            if (lane == 0) s_sum[turn][warp] = dot;
            __syncthreads();
            // the stage of the row before: every thread has left its second pass
            if (gi == 0 && row > row0) fetch(row + step, s ^ 1);
            dot = warp_sum(lane < nw ? s_sum[turn][lane] : 0.0f);
            turn ^= 1;
        }
        const float mean = dot * inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = gi + i * gsize;
            if (c < nchunk && in_bounds(base + 8 * c, 8, total)) {
                const uint4 hv = *reinterpret_cast<const uint4 *>(src + 16 * c);
                const uint4 gv = *reinterpret_cast<const uint4 *>(src + row_bytes + 16 * c);
                uint4 ev = make_uint4(0, 0, 0, 0);
                if (p.dres) ev = *reinterpret_cast<const uint4 *>(src + 2 * row_bytes + 16 * c);
                const uint32_t a[4] = {hv.x, hv.y, hv.z, hv.w}, b[4] = {gv.x, gv.y, gv.z, gv.w};
                const uint32_t d[4] = {w[i].x, w[i].y, w[i].z, w[i].w}, e[4] = {ev.x, ev.y, ev.z, ev.w};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 hh = bf16x2_to_float2(a[k]), gg = bf16x2_to_float2(b[k]), ww = bf16x2_to_float2(d[k]);
                    const float2 ee = bf16x2_to_float2(e[k]);
                    o[k] = pack_bf16x2(fmaf(rstd, fmaf(-hh.x * rstd, mean, gg.x * ww.x), ee.x),
                                       fmaf(rstd, fmaf(-hh.y * rstd, mean, gg.y * ww.y), ee.y));
                }
                *reinterpret_cast<uint4 *>(p.dH + base + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        if (WARP) {
            __syncwarp();
            if (gi == 0) fetch(row + STREAM_STAGES * step, s);
        }
        ph ^= s;
        s ^= 1;
    }
    // this CTA's partial row; the warps of the warp form add theirs in warp order, in the rings' memory
    const int64_t pbase = (int64_t)blockIdx.x * p.D, ptotal = (int64_t)p.parts * p.D;
    float *s_dw = reinterpret_cast<float *>(row_smem);  // [STREAM_WARPS][D], no more than the rings' 4 D bytes a stage
    if (WARP) __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = gi + i * gsize;
        if (c < nchunk && (WARP || in_bounds(pbase + 8 * c, 8, ptotal))) {
            float4 *dst = reinterpret_cast<float4 *>((WARP ? s_dw + warp * p.D : p.part + pbase) + 8 * c);
            dst[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            dst[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
        }
    }
    if (WARP) {
        __syncthreads();
        for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
            float t = s_dw[d];
#pragma unroll
            for (int k = 1; k < STREAM_WARPS; ++k) t += s_dw[k * p.D + d];
            if (in_bounds(pbase + d, 1, ptotal)) p.part[pbase + d] = t;
        }
    }
}

// dw[d] = sum over the `parts` rows of part[.][d], in a fixed order: 32
// columns per CTA, DW_WARPS warps over the rows, their sums added in warp
// order.  The gradients of 8192 x 2048 take 31.8 us with 16 warps, 33.3 with 8,
// 35.2 with 32 that have every load in flight: CTAs of that size do not fit
// beside the rings' and start after them.
constexpr int DW_WARPS = 16;
__global__ void __launch_bounds__(32 * DW_WARPS) dw_sum_kernel(const float *part, int parts, int D, float *dw) {
    __shared__ float s[DW_WARPS][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + lane;
    grid_dep_wait();
    grid_dep_launch();
    float a = 0.0f;
    if (d < D) {
#pragma unroll 4
        for (int r = warp; r < parts; r += DW_WARPS)
            if (in_bounds((int64_t)r * D + d, 1, (int64_t)parts * D)) a += __ldcg(part + (int64_t)r * D + d);
    }
    s[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && d < D) {
#pragma unroll
        for (int k = 1; k < DW_WARPS; ++k) a += s[k][lane];
        if (in_bounds(d, 1, D)) dw[d] = a;
    }
}

}  // namespace slope
