// fp8_quantize.cu -- e4m3 codes with scales of a bf16 or fp32 tensor, on sm_100a:
//
//   scale = max(max|x|, 2^-100) / 448 over each group of 128 channels of a row
//   (activations) or of 128 rows x 128 channels (weights);  q = x / scale rounded
//
// One pass: a group sits in registers between its maximum and its codes, so x is
// read once.  HBM-bound: 3 bytes a bf16 value.
#include "layer_device.cuh"
#include "product_internal.h"

namespace hyena {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = kScaleGroup / 8;  // lanes of a group's row, 8 channels each
constexpr int kTurns = 4;                // groups a half-warp takes, all loads first

template <bool kBf16>
__device__ __forceinline__ void load8(float (&v)[8], const void *p, long long o)
{
    if constexpr (kBf16) {
        const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + o);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_float2(w[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
        const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + o);
        const float4 a = f[0], b = f[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// Bits of the largest magnitude (as integers, so that NaN is the largest).
__device__ __forceinline__ unsigned int amax8(const float (&v)[8])
{
    unsigned int m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// Groups of 128 channels of one row: a half-warp each.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantArgs A, int groups)
{
    const long long items = A.rows * groups;
    const int lane = threadIdx.x % kLanes;
    const long long first = static_cast<long long>(blockIdx.x) * (kThreads / kLanes) * kTurns + threadIdx.x / kLanes;
    float v[kTurns][8];
    long long row[kTurns];
    int c[kTurns], grp[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const long long i = first + t * (kThreads / kLanes);
        row[t] = i / groups;
        grp[t] = static_cast<int>(i - row[t] * groups);
        c[t] = grp[t] * kScaleGroup + lane * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[t][j] = 0.f;
        if (i >= items) c[t] = A.D;  // nothing to read or write
        if (c[t] < A.D) load8<kBf16>(v[t], A.x, row[t] * A.ld_x + c[t]);
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        unsigned int m = amax8(v[t]);
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float scale = scale_of(m);
        if (c[t] < A.D) {
            store_e4m3x8<true>(A.q + row[t] * A.ld_q + c[t], v[t], scale);
            if (lane == 0) A.scales[row[t] * groups + grp[t]] = scale;
        }
    }
}

// Blocks of 128 rows x 128 channels: a CTA each, thread t of 256 the rows
// t / 16, t / 16 + 16, ... of 8 channels.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) quantize_blocks_kernel(const QuantArgs A, int groups)
{
    constexpr int kRows = kScaleGroup * kLanes / kThreads;
    __shared__ unsigned int part[kThreads / 32];
    const int lane = threadIdx.x % kLanes;
    const long long blk = blockIdx.x;
    const long long band = blk / groups;
    const int grp = static_cast<int>(blk - band * groups);
    const int c = grp * kScaleGroup + lane * 8;
    const long long r0 = band * kScaleGroup + threadIdx.x / kLanes;
    float v[kRows][8];
    unsigned int m = 0;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const long long r = r0 + j * (kThreads / kLanes);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
        if (c < A.D && r < A.rows) load8<kBf16>(v[j], A.x, r * A.ld_x + c);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) m = max(m, amax8(v[j]));
    m = __reduce_max_sync(0xffffffffu, m);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, part[i]);
    const float scale = scale_of(m);
    if (threadIdx.x == 0) A.scales[blk] = scale;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const long long r = r0 + j * (kThreads / kLanes);
        if (c < A.D && r < A.rows) store_e4m3x8<true>(A.q + r * A.ld_q + c, v[j], scale);
    }
}

}  // namespace

int launch_fp8_quantize(const QuantArgs &a, cudaStream_t st)
{
    const int groups = (a.D + kScaleGroup - 1) / kScaleGroup;
    if (a.block == 1) {
        const long long per = (kThreads / kLanes) * kTurns;
        const unsigned int grid = static_cast<unsigned int>((a.rows * groups + per - 1) / per);
        if (a.x_bf16)
            quantize_rows_kernel<true><<<grid, kThreads, 0, st>>>(a, groups);
        else
            quantize_rows_kernel<false><<<grid, kThreads, 0, st>>>(a, groups);
    } else {
        const unsigned int grid = static_cast<unsigned int>((a.rows + kScaleGroup - 1) / kScaleGroup * groups);
        if (a.x_bf16)
            quantize_blocks_kernel<true><<<grid, kThreads, 0, st>>>(a, groups);
        else
            quantize_blocks_kernel<false><<<grid, kThreads, 0, st>>>(a, groups);
    }
    HYENA_TRY(cudaGetLastError(), "fp8_quantize launch");
    return 1;
}

}  // namespace hyena
