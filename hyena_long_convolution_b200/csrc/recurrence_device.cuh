// recurrence_device.cuh -- the token arithmetic of the gated linear recurrence,
// shared by its scan, backward and decode kernels so that they form the same
// bits: gates, the unit's segments, and the carry from one unit to the next.
//
//   a = exp(l), l = log_rate * sigmoid(gate);  w = sqrt(1 - a^2) (normalize) or 1
//   s <- a s + w v,  v = x1 x2;  y = x3 s + Dskip v
//
// Rounding.  Slow channels have l near -1e-4: a rounded to fp32 next to 1 keeps
// only four digits of 1 - a, so that an exponential with a biased last digit
// would be off by that bias times the thousands of tokens a slow channel
// remembers.  For |l| < 1/2 the kernels therefore form expm1(l) (a polynomial,
// accurate relative to l) and round a = 1 + expm1(l) once, to nearest; 1 - a^2
// comes from the same value as (1 - a)(1 + a).  The decay over a segment or a
// unit is formed from the sum of its l, not as a product of rounded a.
#pragma once

#include "layer_device.cuh"
#include "layer_internal.h"

namespace hyena {

constexpr unsigned int kFullMask = 0xffffffffu;

__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float sqrt_approx(float x)
{
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Products that a sum takes are written as one __ffma2_rn below: left apart,
// the compiler contracts __fmul2_rn and __fadd2_rn where the product has no
// other use, so that kernels would differ in the last bit.

// expm1(x) / x for |x| < 1/2: the degree-6 polynomial through the function at
// the Chebyshev nodes of [-1/2, 1/2] (relative error 1.4e-8 with these fp32
// coefficients).  Outside it the value is not used.
__device__ __forceinline__ float2 expm1_over_x(float2 x)
{
    float2 q = __ffma2_rn(bcast2(1.9962176156695932e-4f), x, bcast2(1.399777363985777e-3f));
    q = __ffma2_rn(q, x, bcast2(8.333181962370872e-3f));
    q = __ffma2_rn(q, x, bcast2(4.166530445218086e-2f));
    q = __ffma2_rn(q, x, bcast2(1.666666716337204e-1f));
    q = __ffma2_rn(q, x, bcast2(5.000000596046448e-1f));
    return __ffma2_rn(q, x, bcast2(1.f));
}

constexpr float kLog2e = 1.4426950408889634f;

// e = exp(-gate) and sigmoid(gate) = 1 / (1 + e) of a channel pair: 0 where e
// overflows (gates below -88), NaN for NaN.
__device__ __forceinline__ float2 gate_sigmoid(float2 g, float2 &e)
{
    const float2 t = __fmul2_rn(g, bcast2(-kLog2e));
    e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
    const float2 d = __fadd2_rn(e, bcast2(1.f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

// A rate of -inf counts as the lowest finite one: times a sigmoid of 0 it has to be 0.
__device__ __forceinline__ float2 finite_rate(float2 r)
{
    float2 f;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(f.x) : "f"(r.x), "f"(-3.402823466e38f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(f.y) : "f"(r.y), "f"(-3.402823466e38f));
    return f;
}

// a b + c of two bf16 pairs and an fp32 pair, one rounding (the product of two
// bf16 values is exact).
__device__ __forceinline__ float2 fma_bf16x2(uint32_t a, uint32_t b, float2 c)
{
    float2 r;
    asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %2;\n\tmov.b32 {bl, bh}, %3;\n\t"
        "fma.rn.f32.bf16 %0, al, bl, %4;\n\tfma.rn.f32.bf16 %1, ah, bh, %5;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(a), "r"(b), "f"(c.x), "f"(c.y));
    return r;
}

// v = x1 x2, exact (adding -0 keeps the sign of a zero).
__device__ __forceinline__ float2 product(uint32_t a, uint32_t b) { return fma_bf16x2(a, b, bcast2(-0.f)); }

// a = exp(l) and, with kNorm, w = sqrt(1 - a^2) (0 where a rounds to 1 exactly
// because l = 0; NaN for l > 0).
template <bool kNorm>
__device__ __forceinline__ void decay(float2 l, float2 &a, float2 &w)
{
    const float2 q = expm1_over_x(l);
    const float2 t = __fmul2_rn(l, bcast2(kLog2e));
    const float2 E = make_float2(ex2_approx(t.x), ex2_approx(t.y));
    const float2 near_one = __ffma2_rn(q, l, bcast2(1.f));
    const bool sx = fabsf(l.x) < 0.5f, sy = fabsf(l.y) < 0.5f;
    a = make_float2(sx ? near_one.x : E.x, sy ? near_one.y : E.y);
    if constexpr (kNorm) {
        const float2 m = __fmul2_rn(make_float2(-q.x, -q.y), l);
        const float2 p = make_float2(sx ? m.x : 1.f - E.x, sy ? m.y : 1.f - E.y);  // 1 - a
        const float2 z = __ffma2_rn(p, a, p);
        w = make_float2(sqrt_approx(z.x), sqrt_approx(z.y));
    }
}

// The decay over several tokens from the sum of their l.  A reset among them
// (l = -inf) gives -0: the mark that nothing passes, not even Inf or NaN, which
// an underflowed product (+0) lets through as NaN.
__device__ __forceinline__ float2 decay_over(float2 l)
{
    float2 a, w;
    decay<false>(l, a, w);
    a.x = l.x == -INFINITY ? -0.f : a.x;
    a.y = l.y == -INFINITY ? -0.f : a.y;
    return a;
}

// One carry step, C <- P C + A.  kCut: P may carry the mark of a reset.
template <bool kCut>
__device__ __forceinline__ float2 carry(float2 P, float2 C, float2 A)
{
    const float2 r = __ffma2_rn(P, C, A);
    if constexpr (!kCut) return r;
    return make_float2(__float_as_int(P.x) < 0 ? A.x : r.x, __float_as_int(P.y) < 0 ? A.y : r.y);
}

// Gates of a segment: a, w, the sum l of the tokens' l, and the product P of
// their a (for the steps within the unit only; -0 if a token is a reset).
// `mask` bit i: token i is a reset.
template <bool kNorm, bool kReset, class Row>
__device__ __forceinline__ void segment_gates(float2 (&a)[RSEG], float2 (&w)[RSEG], float2 &l, float2 &P, Row gate,
                                              float2 rate, unsigned int mask)
{
#pragma unroll
    for (int i = 0; i < RSEG; ++i) {
        float2 e;
        const float2 sig = gate_sigmoid(bf16x2_to_float2(gate(i)), e);
        float2 li = __fmul2_rn(rate, sig);
        l = i == 0 ? li : __ffma2_rn(rate, sig, l);
        if (kReset && (mask >> i & 1u)) li = l = bcast2(-INFINITY);  // a = 0, w = 1
        decay<kNorm>(li, a[i], w[i]);
        P = i == 0 ? a[i] : __fmul2_rn(P, a[i]);
    }
    if (kReset && mask) P = bcast2(-0.f);
}

// End state of a segment from a zero start, with u = w v.
template <bool kReset>
__device__ __forceinline__ float2 segment_end(const float2 (&a)[RSEG], const float2 (&u)[RSEG], unsigned int mask)
{
    float2 A = u[0];
#pragma unroll
    for (int i = 1; i < RSEG; ++i) A = kReset && (mask >> i & 1u) ? u[i] : __ffma2_rn(a[i], A, u[i]);
    return A;
}

// The gradient that a segment hands to the token before it, e_t = a_t (r_t +
// e_{t+1}) with r = x3 dy, from a zero e at its right edge.
template <bool kReset, class Row>
__device__ __forceinline__ float2 segment_left(const float2 (&a)[RSEG], Row x3, Row dy, unsigned int mask)
{
    float2 e = bcast2(0.f);
#pragma unroll
    for (int i = RSEG - 1; i >= 0; --i) {
        e = __fmul2_rn(a[i], fma_bf16x2(x3(i), dy(i), e));
        if (kReset && (mask >> i & 1u)) e = bcast2(0.f);
    }
    return e;
}

// Bit i: token t0 + i of row b is a reset (i < n).
__device__ __forceinline__ unsigned int segment_resets(const uint8_t *reset, long long row0, int n, int lane)
{
    const bool r = lane < n && reset[row0 + lane] != 0;
    return __ballot_sync(kFullMask, r);
}

}  // namespace hyena
