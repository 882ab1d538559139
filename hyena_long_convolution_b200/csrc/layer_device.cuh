// layer_device.cuh -- device-side helpers of the layer operators (gated
// recurrence, RMS norm, 8-bit products, feed-forward block) beyond those of
// hyena_device.cuh.
#pragma once

#include <cuda_fp8.h>

#include "hyena_device.cuh"

namespace hyena {

__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Bulk copy of `bytes` (a multiple of 16, both addresses 16-byte aligned) into
// this CTA's shared memory, counted by `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// ---------------------------------------------------------------- e4m3

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100: a zero row keeps a finite scale

__device__ __forceinline__ float2 bcast2(float x) { return make_float2(x, x); }

// The scale of values whose largest magnitude has these bits (NaN, the largest
// bits of all, among them).
__device__ __forceinline__ float scale_of(unsigned int amax_bits)
{
    const float a = __uint_as_float(amax_bits);
    return a < kAmaxFloor ? kAmaxFloor / kE4m3Max : a / kE4m3Max;  // NaN stays
}

// The codes of the fp32 quotients v / scale.  The product with the rounded
// reciprocal is up to two units in the last place off, the other code next to the
// border of two; one step with its remainder v - z scale (Markstein, 1990), which
// one FMA forms, puts every z at, above or below a border as the quotient is: all
// 2^23 significands of a scale, with the 13 values of v around each border, give
// the same.  It costs 2 to 15% (8192 x 4096 with a bf16 residual 52 -> 55 us, 65536 x
// 1024 without one 50 -> 57), division 22% (32768 x 4096 without one 139 -> 169).
// kPairs: in packed arithmetic, which takes 132 us there where one value at a time
// takes 151, but holds registers that cost a CTA an SM with a bf16 residual (8192 x
// 4096 with one scale per row: 61) and with four vectors a thread (65536 x 1024: 61).
template <bool kPairs>
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float scale, float inv)
{
    const bool step = scale < INFINITY;  // else the product: 0, NaN of an Inf, NaN
    unsigned short h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = make_float2(v[2 * i], v[2 * i + 1]);
        float2 z;
        if constexpr (kPairs) {
            z = __fmul2_rn(y, bcast2(inv));
            if (step) z = __ffma2_rn(__ffma2_rn(z, bcast2(-scale), y), bcast2(inv), z);
        } else {
            z = make_float2(y.x * inv, y.y * inv);
            if (step) z.x = __fmaf_rn(__fmaf_rn(z.x, -scale, y.x), inv, z.x);
            if (step) z.y = __fmaf_rn(__fmaf_rn(z.y, -scale, y.y), inv, z.y);
        }
        h[i] = __nv_cvt_float2_to_fp8x2(z, __NV_SATFINITE, __NV_E4M3);
    }
    uint2 q;
    q.x = h[0] | static_cast<uint32_t>(h[1]) << 16;
    q.y = h[2] | static_cast<uint32_t>(h[3]) << 16;
    return q;
}


constexpr float kSmallScale = 0x1p-60f;  // below it a remainder may be subnormal

template <bool kPairs>
__device__ __forceinline__ uint2 e4m3x8(float (&v)[8], float scale)
{
    if (scale < kSmallScale) {  // the same quotients
        scale *= 0x1p+64f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= 0x1p+64f;
    }
    return e4m3x8<kPairs>(v, scale, 1.f / scale);
}

// The same of one value.
__device__ __forceinline__ uint8_t e4m3_code(float v, float scale, float inv)
{
    float z = v * inv;
    if (scale < kSmallScale)
        z = v / scale;
    else if (scale < INFINITY)
        z = __fmaf_rn(__fmaf_rn(z, -scale, v), inv, z);
    return __nv_cvt_float_to_fp8(z, __NV_SATFINITE, __NV_E4M3);
}

template <bool kPairs>
__device__ __forceinline__ void store_e4m3x8(uint8_t *p, float (&v)[8], float scale)
{
    *reinterpret_cast<uint2 *>(p) = e4m3x8<kPairs>(v, scale);
}

}  // namespace hyena
