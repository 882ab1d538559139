// fp8_quantize.cu -- e4m3 codes with scales of a bf16 or fp32 tensor, on sm_100a:
//
//   scale = max(max|x|, 2^-100) / 448 over each group of 128 channels of a row
//   (activations) or of 128 rows x 128 channels (weights);  q = x / scale rounded
//
// One pass: a group sits in registers between its maximum and its codes, so x is
// read once.  HBM-bound, 3 bytes a bf16 value: 32768 x 4096 68 us, 6.0 TB/s (92% of the
// measured copy), 11008 x 4096 by blocks 23.3 us (89%), 32768 x 4096 of fp32 104 us (99%).
#include "product_device.cuh"

namespace hyena {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = kScaleGroup / 8;  // lanes of a group's row, 8 channels each
constexpr int kHalfWarps = kThreads / kLanes;

// 8 values as they are in memory, zeros where there are none.
template <bool kBf16>
struct Eight {
    uint4 q[kBf16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *p, long long o, bool inside)
    {
        const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(p) + o * (kBf16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (kBf16 ? 1 : 2); ++i) q[i] = inside ? __ldcs(from + i) : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        if constexpr (kBf16) {
            const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = bf16x2_to_float2(w[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        } else {
            const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
        }
    }
    // Bits of the largest magnitude (as integers, so that NaN is the largest).
    __device__ __forceinline__ unsigned int largest() const
    {
        if constexpr (kBf16) {
            constexpr unsigned int kMag = 0x7fff7fffu;
            const unsigned int m = __vmaxu2(__vmaxu2(q[0].x & kMag, q[0].y & kMag), __vmaxu2(q[0].z & kMag, q[0].w & kMag));
            return max(m << 16, m & 0xffff0000u);
        } else {
            float v[8];
            values(v);
            unsigned int m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
            return m;
        }
    }
};

// The largest over a half-warp of each of its lanes' kT values: lane l gets that of
// value l % kT.
template <int kT>
__device__ __forceinline__ unsigned int largest_of_turns(unsigned int (&m)[kT], int lane)
{
#pragma unroll
    for (int d = kT / 2; d > 0; d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < d; ++i) {
            const unsigned int mine = up ? m[i + d] : m[i], other = up ? m[i] : m[i + d];
            m[i] = max(mine, __shfl_xor_sync(0xffffffffu, other, d));
        }
    }
#pragma unroll
    for (int d = kT; d < kLanes; d <<= 1) m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], d));
    return m[0];
}

// Groups of 128 channels of one row: a half-warp each, kTurns rows one after
// another with all their loads first; a lane works out the scale of one of them.
// (Every lane each scale, and magnitudes value by value: 128 instructions for a
// thread's 8 values and 84 us for 32768 x 4096 bf16, bound by them.)  Of a CTA's 16 half-warps 1 << wide lie side by
// side in a row and the others below them, so that narrow rows fill it too.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantArgs A, int groups, int wide)
{
    constexpr int kTurns = kBf16 ? 8 : 4;
    wait_for_stream();
    const int lane = threadIdx.x % kLanes, hw = threadIdx.x / kLanes;
    const int grp = (blockIdx.y << wide) + (hw & ((1 << wide) - 1));
    const int below = kHalfWarps >> wide;
    const long long r0 = static_cast<long long>(blockIdx.x) * (below * kTurns) + (hw >> wide);
    const int c = grp * kScaleGroup + lane * 8;
    const bool inside = c < A.D;
    Eight<kBf16> x[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const long long r = r0 + t * below;
        x[t].load(A.x, r * A.ld_x + c, inside && r < A.rows);
    }
    unsigned int m[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) m[t] = x[t].largest();
    const float my_scale = scale_of(largest_of_turns(m, lane)), my_inv = 1.f / my_scale;
    {
        const long long r = r0 + (lane % kTurns) * below;
        if (lane < kTurns && grp < groups && r < A.rows) A.scales[r * groups + grp] = my_scale;
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const long long r = r0 + t * below;
        const float scale = __shfl_sync(0xffffffffu, my_scale, t, kLanes);
        const float inv = __shfl_sync(0xffffffffu, my_inv, t, kLanes);
        if (inside && r < A.rows) {
            float v[8];
            x[t].values(v);
            *reinterpret_cast<uint2 *>(A.q + r * A.ld_q + c) =
                scale < kSmallScale ? e4m3x8<true>(v, scale) : e4m3x8<true>(v, scale, inv);
        }
    }
}

// Blocks of 128 rows x 128 channels: a CTA each, thread t of 256 the rows
// t / 16, t / 16 + 16, ... of 8 channels.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) quantize_blocks_kernel(const QuantArgs A, int groups)
{
    constexpr int kRows = kScaleGroup / kHalfWarps;
    __shared__ unsigned int part[kThreads / 32];
    wait_for_stream();
    const int lane = threadIdx.x % kLanes;
    const long long band = blockIdx.x;
    const int grp = blockIdx.y;
    const int c = grp * kScaleGroup + lane * 8;
    const long long r0 = band * kScaleGroup + threadIdx.x / kLanes;
    Eight<kBf16> x[kRows];
    unsigned int m = 0;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const long long r = r0 + j * kHalfWarps;
        x[j].load(A.x, r * A.ld_x + c, c < A.D && r < A.rows);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) m = max(m, x[j].largest());
    m = __reduce_max_sync(0xffffffffu, m);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, part[i]);
    const float scale = scale_of(m);
    if (threadIdx.x == 0) A.scales[band * groups + grp] = scale;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const long long r = r0 + j * kHalfWarps;
        if (c < A.D && r < A.rows) {
            float v[8];
            x[j].values(v);
            store_e4m3x8<true>(A.q + r * A.ld_q + c, v, scale);
        }
    }
}

}  // namespace

int launch_fp8_quantize(const QuantArgs &a, cudaStream_t st)
{
    const int groups = (a.D + kScaleGroup - 1) / kScaleGroup;
    if (a.block == 1) {
        // side by side as many as leave at most an eighth of them without a group (9
        // groups: 2; 32768 x 1032 bf16 by 16 and 2: 28.1 and 20.5 us)
        int wide = 4;
        while (wide > 0 && (((groups - 1) >> wide) + 1) << (wide + 3) > 9 * groups) --wide;
        const int rows = (kHalfWarps >> wide) * (a.x_bf16 ? 8 : 4);  // of a CTA
        const dim3 grid(static_cast<unsigned int>((a.rows + rows - 1) / rows), (groups + (1 << wide) - 1) >> wide);
        return launch_early(a.x_bf16 ? quantize_rows_kernel<true> : quantize_rows_kernel<false>, grid, kThreads, 0, 1, st,
                            "fp8_quantize launch", a, groups, wide);
    }
    const dim3 grid(static_cast<unsigned int>((a.rows + kScaleGroup - 1) / kScaleGroup), groups);
    return launch_early(a.x_bf16 ? quantize_blocks_kernel<true> : quantize_blocks_kernel<false>, grid, kThreads, 0, 1, st,
                        "fp8_quantize launch", a, groups);
}

}  // namespace hyena
