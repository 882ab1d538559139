// rms_norm.cu -- root-mean-square norm with the residual's addition, its output
// in bf16 or in 8 bits with scales, and its gradient, on sm_100a.
//
//   h = x + residual, rounded to the residual's type (or h = x)
//   rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd weight
//   bf16: y rounded once.  e4m3: for each row (or each 128 channels of it)
//   scale = max(max|y|, 2^-100) / 448, q = the fp32 quotient y / scale, rounded.
// Gradient, with n = h rstd and t = weight dy:
//   dh = rstd (t - n mean(t n)) + dresidual_out;  dweight = sum over rows dy n
//
// Forward: a CTA a row (up to 256 channels 8 to 32 lanes, up to 1024 without a
// residual a warp, several rows to a CTA) holds it in registers between the
// reduction and the output, so every input is read once; thread i of T owns the
// 8-channel vectors i, i + T, ...  HBM-bound: 32768 rows of 4096 channels with a
// bf16 residual take 168-173 us, 97-99% of the measured copy bandwidth; 8192 rows
// with an fp32 residual and an e4m3 output 66-68 us, 85-87%.
#include "layer_device.cuh"
#include "layer_internal.h"

namespace hyena {

namespace {

constexpr int kNormThreads = 512;  // most threads of a row
constexpr int kNormStages = 6;     // most stages of the gradient's ring
constexpr int kNormSmem = 200 * 1024;
constexpr int kNarrowWidth = 256;    // widest row that lanes of one warp take
constexpr int kNarrowThreads = 256;
constexpr int kNarrowTurns = 3;
constexpr int kNarrowCtas = 2;  // an SM, by its registers
constexpr unsigned int kFullMask = 0xffffffffu;

__device__ __forceinline__ void load_bf16x8(float (&v)[8], const uint16_t *p)
{
    const uint4 q = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_to_float2(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void load_f32x8(float (&v)[8], const float *p)
{
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(p + i);
        v[i] = q.x;
        v[i + 1] = q.y;
        v[i + 2] = q.z;
        v[i + 3] = q.w;
    }
}

__device__ __forceinline__ void store_bf16x8(uint16_t *p, const float (&v)[8])
{
    uint4 q;
    q.x = float2_to_bf16x2(make_float2(v[0], v[1]));
    q.y = float2_to_bf16x2(make_float2(v[2], v[3]));
    q.z = float2_to_bf16x2(make_float2(v[4], v[5]));
    q.w = float2_to_bf16x2(make_float2(v[6], v[7]));
    *reinterpret_cast<uint4 *>(p) = q;
}

__device__ __forceinline__ void store_f32x8(float *p, const float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

// A tensor of type kind R (0 absent, 1 bf16, 2 fp32), 8 values at element o.
template <int R>
__device__ __forceinline__ void load8(float (&v)[8], const void *p, long long o)
{
    if constexpr (R == 2)
        load_f32x8(v, static_cast<const float *>(p) + o);
    else
        load_bf16x8(v, static_cast<const uint16_t *>(p) + o);
}

// The same as it is in memory, and as channel pairs, which the arithmetic takes two
// at a time.
template <int R>
struct Vector {
    uint4 q{0u, 0u, 0u, 0u};
    __device__ __forceinline__ void load(const void *p, long long o)
    {
        q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + o);
    }
    __device__ __forceinline__ void pairs(float2 (&v)[4]) const
    {
        v[0] = bf16x2_to_float2(q.x);
        v[1] = bf16x2_to_float2(q.y);
        v[2] = bf16x2_to_float2(q.z);
        v[3] = bf16x2_to_float2(q.w);
    }
};

template <>
struct Vector<2> {
    float4 a{0.f, 0.f, 0.f, 0.f}, b{0.f, 0.f, 0.f, 0.f};
    __device__ __forceinline__ void load(const void *p, long long o)
    {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + o);
        a = q[0];
        b = q[1];
    }
    __device__ __forceinline__ void pairs(float2 (&v)[4]) const
    {
        v[0] = make_float2(a.x, a.y);
        v[1] = make_float2(a.z, a.w);
        v[2] = make_float2(b.x, b.y);
        v[3] = make_float2(b.z, b.w);
    }
};

template <int R>
__device__ __forceinline__ void load_pairs(float2 (&v)[4], const void *p, long long o)
{
    Vector<R> t;
    t.load(p, o);
    t.pairs(v);
}

__device__ __forceinline__ void store_pairs(float *p, const float2 (&v)[4])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}

__device__ __forceinline__ void store_bf16_pairs(uint16_t *p, const float2 (&v)[4])
{
    uint4 q;
    q.x = float2_to_bf16x2(v[0]);
    q.y = float2_to_bf16x2(v[1]);
    q.z = float2_to_bf16x2(v[2]);
    q.w = float2_to_bf16x2(v[3]);
    *reinterpret_cast<uint4 *>(p) = q;
}

// The weight, fp32 or bf16 (the same for the whole launch).
__device__ __forceinline__ void load_weight(float (&v)[8], const void *p, bool bf16, int c)
{
    if (bf16)
        load_bf16x8(v, static_cast<const uint16_t *>(p) + c);
    else
        load_f32x8(v, static_cast<const float *>(p) + c);
}

// Sum over a row's threads, the blockDim.x of a CTA (or, below 32, of neighbouring
// lanes), the same bits in every thread: by butterfly within the warps and again
// over the warps' sums (16 at most).  `part` is used by one call only.
__device__ __forceinline__ float block_sum(float v, float *part)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        if (d < static_cast<int>(blockDim.x)) v += __shfl_xor_sync(kFullMask, v, d);
    const int warps = blockDim.x >> 5;
    if (warps <= 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    const int w = threadIdx.x & 15;
    v = w < warps ? part[w] : 0.f;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
    return v;
}

// Largest absolute value over a row's threads as its bits: as unsigned numbers the bits
// order as the values, and a NaN's are the largest, so that it shows.
__device__ __forceinline__ unsigned int block_max(unsigned int v, unsigned int *part)
{
    const int warps = blockDim.x >> 5;
    if (warps == 0) {
#pragma unroll
        for (int d = 8; d > 0; d >>= 1)
            if (d < static_cast<int>(blockDim.x)) v = max(v, __shfl_xor_sync(kFullMask, v, d));
        return v;
    }
    v = __reduce_max_sync(kFullMask, v);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
    for (int w = 1; w < warps; ++w) v = max(v, part[w]);
    return v;
}

// R: the residual's type kind.  Q: 0 bf16 output, 1 e4m3 with a scale per row,
// 2 e4m3 with a scale per 128 channels (16 neighbouring threads' vectors).
template <int VPT, int R, int Q>
__global__ void __launch_bounds__(kNormThreads) rms_norm_kernel(const NormArgs A)
{
    __shared__ float sum_part[32];
    __shared__ unsigned int max_part[32];
    const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int T = blockDim.x;
    const int width = row < A.rows ? A.D : 0;  // none for what is over in the last of several rows' CTAs
    const uint16_t *x = A.x + row * A.ld_x;
    float h[VPT][8];
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = 8 * (static_cast<int>(threadIdx.x) + k * T);
        if (c < width) {
            load_bf16x8(h[k], x + c);
            if constexpr (R != 0) {
                float r[8];
                const long long o = row * A.ld_r + c;
                load8<R>(r, A.residual, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[k][i] += r[i];
                if constexpr (R == 1) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 f =
                            bf16x2_to_float2(float2_to_bf16x2(make_float2(h[k][i], h[k][i + 1])));
                        h[k][i] = f.x;
                        h[k][i + 1] = f.y;
                    }
                    if (A.residual_out) store_bf16x8(static_cast<uint16_t *>(A.residual_out) + o, h[k]);
                } else if (A.residual_out) {
                    store_f32x8(static_cast<float *>(A.residual_out) + o, h[k]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[k][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = __fmaf_rn(h[k][i], h[k][i], sq);
    }
    const float rstd = __frsqrt_rn(block_sum(sq, sum_part) / static_cast<float>(A.D) + A.eps);
    if (A.rstd && threadIdx.x == 0 && width) A.rstd[row] = rstd;
    unsigned int amax[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = 8 * (static_cast<int>(threadIdx.x) + k * T);
        float w[8];
        if (c < width) {
            load_weight(w, A.weight, A.weight_bf16, c);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 0.f;
        }
        amax[k] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[k][i] = h[k][i] * rstd * w[i];
            if constexpr (Q != 0) amax[k] = max(amax[k], __float_as_uint(h[k][i]) & 0x7fffffffu);
        }
        if constexpr (Q == 0) {
            if (c < width) store_bf16x8(A.y + row * A.ld_y + c, h[k]);
        }
    }
    if constexpr (Q == 1) {
#pragma unroll
        for (int k = 1; k < VPT; ++k) amax[0] = max(amax[0], amax[k]);
        const float scale = scale_of(block_max(amax[0], max_part));
        if (threadIdx.x == 0 && width) A.scales[row] = scale;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = 8 * (static_cast<int>(threadIdx.x) + k * T);
            if (c < width) store_e4m3x8<VPT <= 2 && R != 1>(A.q + row * A.ld_y + c, h[k], scale);
        }
    } else if constexpr (Q == 2) {
        const int groups = (A.D + 127) / 128;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            unsigned int m = amax[k];
#pragma unroll
            for (int d = 8; d > 0; d >>= 1)
                if (d < T) m = max(m, __shfl_xor_sync(kFullMask, m, d));
            const float scale = scale_of(m);
            const int c = 8 * (static_cast<int>(threadIdx.x) + k * T);
            if (c < width) {
                if ((threadIdx.x & 15) == 0) A.scales[row * groups + c / 128] = scale;
                store_e4m3x8<VPT <= 2 && R != 1>(A.q + row * A.ld_y + c, h[k], scale);
            }
        }
    }
}

// Gradient.  A CTA walks the rows blockIdx.x, blockIdx.x + gridDim.x, ... and
// keeps its channels' weight and part of dweight in registers; the parts go to
// `partial` [gridDim.x][D].  HBM-bound (8 bytes an element with a bf16
// residual): rows come through a ring of A.stages stages of shared memory, a
// bulk copy a tensor, and are read from there on both sides of the row's
// reduction (holding the next row in registers instead kept 49 KB an SM under
// way and reached 75% of the copy bandwidth).  The arithmetic takes channel pairs:
// one channel at a time it was the limit, 105 us for 16384 x 4096 against 84, and
// 5 for the parts' sum (84 is the copy bandwidth).
template <int VPT, int R>
__global__ void __launch_bounds__(kNormThreads) rms_norm_backward_kernel(const NormArgs A)
{
    constexpr int kSize = R == 2 ? 4 : 2;  // of h and dresidual_out
    extern __shared__ __align__(128) unsigned char stages[];
    __shared__ float part[2][32];
    __shared__ uint64_t full[kNormStages];
    const int T = blockDim.x;
    const int S = A.stages;
    const uint32_t dy_bytes = 2u * A.D, h_bytes = kSize * static_cast<uint32_t>(A.D);
    const bool copy_dres = A.dres_out != nullptr && A.stage_dres;
    const uint32_t stage_bytes = dy_bytes + h_bytes * (1 + copy_dres);
    const auto request = [&](long long row, int s) {  // one thread
        unsigned char *to = stages + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        bulk_load(to, A.dy + row * A.ld_y, dy_bytes, &full[s]);
        bulk_load(to + dy_bytes, static_cast<const char *>(A.h) + row * A.ld_h * kSize, h_bytes, &full[s]);
        if (copy_dres)
            bulk_load(to + dy_bytes + h_bytes, static_cast<const char *>(A.dres_out) + row * A.ld_r * kSize, h_bytes,
                      &full[s]);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
        for (int s = 0; s < S; ++s) {
            const long long row = blockIdx.x + static_cast<long long>(s) * gridDim.x;
            if (row < A.rows) request(row, s);
        }
    }
    float2 dw[VPT][4], w[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = 8 * (static_cast<int>(threadIdx.x) + k * T);
        if (c < A.D) {
            if (A.weight_bf16)
                load_pairs<1>(w[k], A.weight, c);
            else
                load_pairs<2>(w[k], A.weight, c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[k][i] = bcast2(0.f);
    }
    const float per_channel = 1.f / static_cast<float>(A.D);
    __syncthreads();
    int s = 0, turn = 0;  // stage, and how often the ring has gone round
    long long behind = blockIdx.x + static_cast<long long>(S - 1) * gridDim.x;  // the newest row asked for
    // A copy that does not come within the wait's limit: no result is passed off from
    // there on.  One thread's NaN reaches all of a row by its sum.
    bool lost = false;
    for (long long row = blockIdx.x, i = 0; row < A.rows; row += gridDim.x, ++i) {
        float rstd = A.rstd_in[row];
        if (lost || !mbar_wait_bounded(&full[s], turn & 1)) {
            lost = true;
            rstd = __int_as_float(0x7fffffff);
        }
        const unsigned char *st = stages + s * stage_bytes;
        const uint16_t *dy = reinterpret_cast<const uint16_t *>(st);
        const unsigned char *h = st + dy_bytes;
        float2 dot = bcast2(0.f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = 8 * (static_cast<int>(threadIdx.x) + k * T);
            if (c < A.D) {
                float2 n[4], d[4];
                load_pairs<R>(n, h, c);
                load_pairs<1>(d, dy, c);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[j] = __fmul2_rn(n[j], bcast2(rstd));
                    dw[k][j] = __ffma2_rn(d[j], n[j], dw[k][j]);
                    dot = __ffma2_rn(__fmul2_rn(d[j], w[k][j]), n[j], dot);
                }
            }
        }
        const float mean = block_sum(dot.x + dot.y, part[i & 1]) * per_channel;
        // behind the reduction every thread is through with the row before
        if (i > 0) {
            behind += gridDim.x;
            if (threadIdx.x == 0 && !lost && behind < A.rows) request(behind, s == 0 ? S - 1 : s - 1);
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = 8 * (static_cast<int>(threadIdx.x) + k * T);
            if (c < A.D) {
                float2 n[4], d[4], r[4];
                load_pairs<R>(n, h, c);
                load_pairs<1>(d, dy, c);
                if (copy_dres) {
                    load_pairs<R>(r, h + h_bytes, c);
                } else if (A.dres_out) {
                    load_pairs<R>(r, A.dres_out, row * A.ld_r + c);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) r[j] = bcast2(0.f);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[j] = __fmul2_rn(n[j], bcast2(rstd));
                    const float2 t = __ffma2_rn(n[j], bcast2(-mean), __fmul2_rn(d[j], w[k][j]));
                    r[j] = __ffma2_rn(bcast2(rstd), t, r[j]);
                }
                if (A.dx) store_bf16_pairs(A.dx + row * A.ld_x + c, r);
                if constexpr (R == 2) {
                    if (A.dres) store_pairs(A.dres + row * A.ld_dr + c, r);
                }
            }
        }
        if (++s == S) {
            s = 0;
            ++turn;
        }
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = 8 * (static_cast<int>(threadIdx.x) + k * T);
        if (c < A.D) store_pairs(A.partial + static_cast<long long>(blockIdx.x) * A.D + c, dw[k]);
    }
}

// Gradient of short rows (of heads, say): G lanes a row, 8 channels each, 32 / G
// rows a warp, and kNarrowTurns rows' loads of a lane under way together, from
// global memory; no row needs the CTA's other warps.  90 us for 524288 x 128 and
// for 262144 x 256 (83 at the copy bandwidth); by the kernel above, where a short
// row leaves most lanes idle, 103 and 130.  Registers for three CTAs an SM spill
// (116 us for 524288 x 128), those for two 24 bytes at most where G is 8 or 16; two
// turns instead of three take 95 and 99.
template <int G, int R>
__global__ void __launch_bounds__(kNarrowThreads, kNarrowCtas) rms_norm_backward_narrow_kernel(const NormArgs A)
{
    constexpr int kRows = 32 / G;
    constexpr int kTurns = kNarrowTurns;
    __shared__ __align__(16) float part[kNarrowThreads / 32][8 * G];  // stored four at a time
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / G, c = 8 * (lane % G);
    const bool live = c < A.D;
    const float per_channel = 1.f / static_cast<float>(A.D);
    float2 w[4], dw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = dw[j] = bcast2(0.f);
    if (live) {
        if (A.weight_bf16)
            load_pairs<1>(w, A.weight, c);
        else
            load_pairs<2>(w, A.weight, c);
    }
    const long long step = static_cast<long long>(gridDim.x) * (kNarrowThreads / 32) * kRows;
    long long base = (static_cast<long long>(blockIdx.x) * (kNarrowThreads / 32) + warp) * kRows;
    for (; base < A.rows; base += step * kTurns) {
        Vector<R> h[kTurns], dres[kTurns];
        Vector<1> dy[kTurns];
        float rstd[kTurns];
#pragma unroll
        for (int u = 0; u < kTurns; ++u) {
            const long long row = base + u * step + sub;
            rstd[u] = 0.f;
            h[u] = dres[u] = Vector<R>();
            dy[u] = Vector<1>();
            if (live && row < A.rows) {
                rstd[u] = A.rstd_in[row];
                h[u].load(A.h, row * A.ld_h + c);
                dy[u].load(A.dy, row * A.ld_y + c);
                if (A.dres_out) dres[u].load(A.dres_out, row * A.ld_r + c);
            }
        }
#pragma unroll
        for (int u = 0; u < kTurns; ++u) {
            const long long row = base + u * step + sub;
            float2 n[4], d[4], r[4], dot = bcast2(0.f);
            h[u].pairs(n);
            dy[u].pairs(d);
            dres[u].pairs(r);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                n[j] = __fmul2_rn(n[j], bcast2(rstd[u]));
                dw[j] = __ffma2_rn(d[j], n[j], dw[j]);
                d[j] = __fmul2_rn(d[j], w[j]);
                dot = __ffma2_rn(d[j], n[j], dot);
            }
            float mean = dot.x + dot.y;
#pragma unroll
            for (int k = G / 2; k > 0; k >>= 1) mean += __shfl_xor_sync(kFullMask, mean, k);
            mean *= per_channel;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[j] = __ffma2_rn(bcast2(rstd[u]), __ffma2_rn(n[j], bcast2(-mean), d[j]), r[j]);
            if (live && row < A.rows) {
                if (A.dx) store_bf16_pairs(A.dx + row * A.ld_x + c, r);
                if constexpr (R == 2) {
                    if (A.dres) store_pairs(A.dres + row * A.ld_dr + c, r);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int k = G; k < 32; k <<= 1) {
            dw[j].x += __shfl_xor_sync(kFullMask, dw[j].x, k);
            dw[j].y += __shfl_xor_sync(kFullMask, dw[j].y, k);
        }
    }
    if (sub == 0) store_pairs(&part[warp][c], dw);
    __syncthreads();
    if (threadIdx.x < A.D) {
        float s = 0.f;
        for (int k = 0; k < kNarrowThreads / 32; ++k) s += part[k][threadIdx.x];
        A.partial[static_cast<long long>(blockIdx.x) * A.D + threadIdx.x] = s;
    }
}

// dweight: the CTAs' parts summed in double, in a fixed order: a CTA takes 32
// channels, eight lanes four each, and a warp's four groups of lanes every 128th
// part; then the groups and the warps by butterfly.  Latency-bound, so that a
// thread's loads go out together (592 parts of 1032 channels: 5.8 us, one load at a time 8.4).
__global__ void __launch_bounds__(1024) norm_weight_sum_kernel(const float *partial, int parts, int D, float *dweight)
{
    __shared__ double sum[32][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + 4 * (lane & 7);
    double s[4] = {0., 0., 0., 0.};
    if (c < D) {
#pragma unroll 8
        for (int p = 4 * warp + (lane >> 3); p < parts; p += 128) {
            const float4 v = *reinterpret_cast<const float4 *>(partial + static_cast<long long>(p) * D + c);
            s[0] += v.x;
            s[1] += v.y;
            s[2] += v.z;
            s[3] += v.w;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s[i] += __shfl_xor_sync(kFullMask, s[i], 8);
        s[i] += __shfl_xor_sync(kFullMask, s[i], 16);
        if (lane < 8) sum[warp][4 * lane + i] = s[i];
    }
    __syncthreads();
    double v = sum[lane][warp];  // the warp's channel, a lane a warp's sum
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
    const int out = blockIdx.x * 32 + warp;
    if (lane == 0 && out < D) dweight[out] = static_cast<float>(v);
}

// Threads of a row of up to kNarrowWidth channels.
int narrow_lanes(int D) { return D <= 64 ? 8 : (D <= 128 ? 16 : 32); }

// Vectors per thread and threads of a row of D channels.  Without a residual a
// row's own loads are few, and up to 1024 channels a warp a row, eight to a CTA,
// hides them better (131072 x 512 72 -> 47 us, 65536 x 1024 57 -> 47); with one the
// warps' registers then hold too much (65536 x 1024 82 -> 97).
struct NormShape {
    int vpt, threads;
};

NormShape norm_shape(int D, bool residual)
{
    const int v = D / 8;
    const int vpt = v <= 256 ? 1 : (v <= 2 * kNormThreads ? 2 : 4);
    if (D <= kNarrowWidth) return {1, narrow_lanes(D)};
    if (!residual && D <= 1024) return {D <= 512 ? 2 : 4, 32};
    return {vpt, ((v + vpt - 1) / vpt + 31) / 32 * 32};
}

template <int VPT, int Q>
void forward_r(const NormArgs &a, int threads, cudaStream_t st)
{
    // Short rows go as many to a CTA as fill 256 threads where there are enough of
    // them, else as fill a warp
    const unsigned int most = threads <= 32 ? 256 / threads : 1, least = threads < 32 ? 32 / threads : 1;
    const unsigned int per = a.rows >= 148ll * most ? most : least;
    const unsigned int grid = static_cast<unsigned int>((a.rows + per - 1) / per);
    const dim3 block(threads, per);
    switch (a.residual ? a.res_kind : 0) {
        case 0: rms_norm_kernel<VPT, 0, Q><<<grid, block, 0, st>>>(a); break;
        case 1: rms_norm_kernel<VPT, 1, Q><<<grid, block, 0, st>>>(a); break;
        default: rms_norm_kernel<VPT, 2, Q><<<grid, block, 0, st>>>(a); break;
    }
}

template <int VPT>
void forward_q(const NormArgs &a, int threads, cudaStream_t st)
{
    if (!a.q)
        forward_r<VPT, 0>(a, threads, st);
    else if (a.group == 0)
        forward_r<VPT, 1>(a, threads, st);
    else
        forward_r<VPT, 2>(a, threads, st);
}

// CTAs of the gradient an SM, what it holds with a bf16 h by their registers and 200 KB
// of stages (for 16384 x 4096 two took 105 us where three, which do not fit at once,
// took 119).  With an fp32 h and dresidual_out two of more than 5120 channels do not
// fit either and go one after the other: 8192 x 8192 takes 182 us, 92% of the copy
// bandwidth (16384 x 4096, where two fit, 167 us, 100%).
int gradient_ctas(int D)
{
    if (D <= kNarrowWidth) return kNarrowCtas;
    return D <= 512 ? 16 : (D <= 1024 ? 8 : (D <= 2048 ? 4 : (D <= 8192 ? 2 : 1)));
}

// More threads than the forward takes, and with them more CTAs' work hidden.
NormShape gradient_shape(int D)
{
    const int v = D / 8;
    const int vpt = v <= kNormThreads ? 1 : (v <= 2 * kNormThreads ? 2 : 4);
    return {vpt, ((v + vpt - 1) / vpt + 31) / 32 * 32};
}

template <int G>
void launch_narrow(const NormArgs &a, int parts, cudaStream_t st)
{
    if (a.res_kind == 2)
        rms_norm_backward_narrow_kernel<G, 2><<<parts, kNarrowThreads, 0, st>>>(a);
    else
        rms_norm_backward_narrow_kernel<G, 1><<<parts, kNarrowThreads, 0, st>>>(a);
}

// The ring of a gradient CTA: as many stages as its part of an SM's shared memory
// holds, two at least; without dresidual_out where two with it exceed an SM's shared
// memory (an fp32 one of more than 10240 channels).
template <int VPT, int R>
int launch_gradient(NormArgs a, int parts, int threads, cudaStream_t st)
{
    thread_local int configured_device = -1;
    int dev = 0;
    HYENA_TRY(cudaGetDevice(&dev), "rms norm gradient: current device");
    auto kernel = rms_norm_backward_kernel<VPT, R>;
    if (configured_device != dev) {
        HYENA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem),
                  "rms norm gradient: set max dynamic shared memory");
        configured_device = dev;
    }
    const int size = R == 2 ? 4 : 2;
    int bytes = a.D * (2 + 2 * size);
    a.stage_dres = 2 * bytes <= kNormSmem;
    if (!a.stage_dres || !a.dres_out) bytes = a.D * (2 + size);
    a.stages = kNormSmem / gradient_ctas(a.D) / bytes;
    a.stages = a.stages < 2 ? 2 : (a.stages > kNormStages ? kNormStages : a.stages);
    kernel<<<parts, threads, a.stages * bytes, st>>>(a);
    return 0;
}

template <int VPT>
int backward_r(const NormArgs &a, int parts, int threads, cudaStream_t st)
{
    return a.res_kind == 2 ? launch_gradient<VPT, 2>(a, parts, threads, st)
                           : launch_gradient<VPT, 1>(a, parts, threads, st);
}

}  // namespace

int launch_rms_norm(const NormArgs &a, cudaStream_t st)
{
    const NormShape s = norm_shape(a.D, a.residual != nullptr);
    if (s.vpt == 1)
        forward_q<1>(a, s.threads, st);
    else if (s.vpt == 2)
        forward_q<2>(a, s.threads, st);
    else
        forward_q<4>(a, s.threads, st);
    HYENA_TRY(cudaGetLastError(), "rms norm launch");
    return 1;
}

int norm_parts(long long rows, int D)
{
    const int most = 148 * gradient_ctas(D);  // the SMs of the one target: the size is asked for without a device
    const int per = D <= kNarrowWidth ? kNarrowThreads / narrow_lanes(D) : 1;  // rows a CTA takes at a time
    rows = (rows + per - 1) / per;
    return static_cast<int>(rows < most ? rows : most);
}

int launch_rms_norm_backward(const NormArgs &a, cudaStream_t st)
{
    const NormShape s = gradient_shape(a.D);
    const int parts = norm_parts(a.rows, a.D);
    int rc = 0;
    if (a.D > kNarrowWidth)
        rc = s.vpt == 1   ? backward_r<1>(a, parts, s.threads, st)
             : s.vpt == 2 ? backward_r<2>(a, parts, s.threads, st)
                          : backward_r<4>(a, parts, s.threads, st);
    else if (narrow_lanes(a.D) == 8)
        launch_narrow<8>(a, parts, st);
    else if (narrow_lanes(a.D) == 16)
        launch_narrow<16>(a, parts, st);
    else
        launch_narrow<32>(a, parts, st);
    if (rc < 0) return rc;
    norm_weight_sum_kernel<<<(a.D + 31) / 32, 1024, 0, st>>>(a.partial, parts, a.D, a.dweight);
    HYENA_TRY(cudaGetLastError(), "rms norm gradient launch");
    return 2;
}

}  // namespace hyena
