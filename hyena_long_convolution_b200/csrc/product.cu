// product.cu -- products of the 8-bit projections and of the gated feed-forward
// block, and its gradient: the simplest form, FP32 FMAs over shared-memory tiles.
//
//   y[m, n] = sum_k x[m, k] w[n, k] (times scales per 128 channels of codes)
//   y = act(g) u with g = x Wg^T, u = x Wu^T
//   dg = dy u act'(g), du = dy act(g); dx = dg Wg + du Wu; dWg = dg^T x, dWu = du^T x
#include "product_device.cuh"

namespace hyena {

namespace {

constexpr int TM = 32, TN = 128, TK = 16;  // tile of a CTA of 256 threads: row t / 8, columns t % 8 + 8 j

template <bool kF8>
__device__ __forceinline__ float value(const void *p, long long i)
{
    if constexpr (kF8) {
        __nv_fp8_e4m3 e;
        e.__x = static_cast<const uint8_t *>(p)[i];
        return static_cast<float>(e);
    } else {
        return bf16_value(static_cast<const uint16_t *>(p)[i]);
    }
}

// acc[j] += sum over k < K of A(m, k) B(n, k), n = n0 + t % 8 + 8 j, with element
// strides (am, ak), (bn, bk).
template <bool kF8>
__device__ void accumulate(float (&acc)[16], const void *a, long long am, long long ak, const void *b, long long bn,
                           long long bk, long long m0, long long M, long long n0, long long N, long long k0,
                           long long K, float *sa, float *sb)
{
    const int t = threadIdx.x;
    for (long long k = k0; k < K; k += TK) {
        for (int i = t; i < TM * TK; i += 256) {
            const int r = i / TK, c = i % TK;
            sa[r * (TK + 1) + c] = (m0 + r < M && k + c < K) ? value<kF8>(a, (m0 + r) * am + (k + c) * ak) : 0.f;
        }
        for (int i = t; i < TN * TK; i += 256) {
            const int r = i / TK, c = i % TK;
            sb[r * (TK + 1) + c] = (n0 + r < N && k + c < K) ? value<kF8>(b, (n0 + r) * bn + (k + c) * bk) : 0.f;
        }
        __syncthreads();
        for (int c = 0; c < TK; ++c) {
            const float x = sa[(t / 8) * (TK + 1) + c];
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[j] = fmaf(x, sb[(t % 8 + 8 * j) * (TK + 1) + c], acc[j]);
        }
        __syncthreads();
    }
}

template <bool kF8, int kAct, bool kGated>
__global__ void __launch_bounds__(256) product_kernel(const ProductArgs A)
{
    __shared__ float sa[TM * (TK + 1)], sb[TN * (TK + 1)];
    const int tiles = (A.N + TN - 1) / TN, groups = (A.K + kScaleGroup - 1) / kScaleGroup;
    const int nb = blockIdx.x % tiles;
    const long long m0 = static_cast<long long>(blockIdx.x / tiles) * TM, n0 = static_cast<long long>(nb) * TN;
    const long long m = m0 + threadIdx.x / 8;
    float acc[2][16] = {};
    for (int w = 0; w < (kGated ? 2 : 1); ++w) {
        const void *b = w ? A.w2 : A.w1;
        if constexpr (kF8) {
            for (int g = 0; g < groups; ++g) {
                float d[16] = {};
                const long long k0 = static_cast<long long>(g) * kScaleGroup;
                const long long k1 = k0 + kScaleGroup < A.K ? k0 + kScaleGroup : A.K;
                accumulate<true>(d, A.x, A.ld_x, 1, b, A.ld_w, 1, m0, A.M, n0, A.N, k0, k1, sa, sb);
                const float s = m < A.M ? A.sx[m * A.sx_row + static_cast<long long>(g) * A.sx_step] *
                                              (w ? A.sw2 : A.sw1)[static_cast<long long>(nb) * groups + g]
                                        : 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[w][j] = fmaf(d[j], s, acc[w][j]);
            }
        } else {
            accumulate<false>(acc[w], A.x, A.ld_x, 1, b, A.ld_w, 1, m0, A.M, n0, A.N, 0, A.K, sa, sb);
        }
    }
    float v[16];
    unsigned int mx = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        v[j] = kGated ? activation<kAct>(acc[0][j]) * acc[1][j] : acc[0][j];
        mx = max(mx, __float_as_uint(v[j]) & 0x7fffffffu);
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    if (m >= A.M) return;
    const float scale = scale_of(mx);
    if (A.q && threadIdx.x % 8 == 0) A.scales[m * tiles + nb] = scale;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const long long n = n0 + threadIdx.x % 8 + 8 * j;
        if (n >= A.N) continue;
        if (A.q) {
            A.q[m * A.ld_q + n] = __nv_cvt_float_to_fp8(v[j] / scale, __NV_SATFINITE, __NV_E4M3);
        } else if (A.y_f32) {
            static_cast<float *>(A.y)[m * A.ld_y + n] = v[j];
        } else {
            static_cast<uint16_t *>(A.y)[m * A.ld_y + n] = bf16_bits(v[j]);
        }
        if (A.g) {
            if (A.g_f32) {
                static_cast<float *>(A.g)[m * A.ld_g + n] = acc[0][j];
                static_cast<float *>(A.u)[m * A.ld_g + n] = acc[1][j];
            } else {
                static_cast<uint16_t *>(A.g)[m * A.ld_g + n] = bf16_bits(acc[0][j]);
                static_cast<uint16_t *>(A.u)[m * A.ld_g + n] = bf16_bits(acc[1][j]);
            }
        }
    }
}

template <int kAct>
__global__ void __launch_bounds__(256) slopes_kernel(const FfnBackArgs A, uint16_t *dg, uint16_t *du)
{
    const long long n = A.M * A.F;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const long long m = i / A.F, f = i - m * A.F;
        const long long k = m * A.ld_g + f;
        const float g = A.g_f32 ? static_cast<const float *>(A.g)[k] : bf16_value(static_cast<const uint16_t *>(A.g)[k]);
        const float u = A.g_f32 ? static_cast<const float *>(A.u)[k] : bf16_value(static_cast<const uint16_t *>(A.u)[k]);
        const float dy = bf16_value(A.dy[m * A.ld_dy + f]);
        const float2 a = activation_slope<kAct>(g);
        dg[i] = bf16_bits(dy * u * a.y);
        du[i] = bf16_bits(dy * a.x);
    }
}

// C[m, n] = sum_k A1(m, k) B1(n, k) + sum_k A2(m, k) B2(n, k)
__global__ void __launch_bounds__(256)
    gradient_kernel(const uint16_t *a1, const uint16_t *a2, long long am, long long ak, const uint16_t *b1,
                    const uint16_t *b2, long long bn, long long bk, uint16_t *c, long long ld_c, long long M, int N,
                    long long K)
{
    __shared__ float sa[TM * (TK + 1)], sb[TN * (TK + 1)];
    const int tiles = (N + TN - 1) / TN;
    const long long m0 = static_cast<long long>(blockIdx.x / tiles) * TM;
    const long long n0 = static_cast<long long>(blockIdx.x % tiles) * TN;
    float acc[16] = {};
    accumulate<false>(acc, a1, am, ak, b1, bn, bk, m0, M, n0, N, 0, K, sa, sb);
    if (a2) accumulate<false>(acc, a2, am, ak, b2, bn, bk, m0, M, n0, N, 0, K, sa, sb);
    const long long m = m0 + threadIdx.x / 8;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const long long n = n0 + threadIdx.x % 8 + 8 * j;
        if (m < M && n < N) c[m * ld_c + n] = bf16_bits(acc[j]);
    }
}

template <bool kF8, int kAct>
void start_product(const ProductArgs &a, cudaStream_t st)
{
    const unsigned int grid = static_cast<unsigned int>((a.M + TM - 1) / TM * ((a.N + TN - 1) / TN));
    if (a.gated)
        product_kernel<kF8, kAct, true><<<grid, 256, 0, st>>>(a);
    else
        product_kernel<kF8, HYENA_ACT_IDENTITY, false><<<grid, 256, 0, st>>>(a);
}

template <int kAct>
void start_by_type(const ProductArgs &a, cudaStream_t st)
{
    if (a.fp8)
        start_product<true, kAct>(a, st);
    else
        start_product<false, kAct>(a, st);
}

}  // namespace

size_t product_workspace(long long, int, int, bool, bool) { return 256; }
size_t ffn_backward_workspace(long long M, int, int F) { return 256 + static_cast<size_t>(M) * F * 4; }

int launch_product(const ProductArgs &a, cudaStream_t st)
{
    switch (a.act) {
        case HYENA_ACT_SILU: start_by_type<HYENA_ACT_SILU>(a, st); break;
        case HYENA_ACT_GELU: start_by_type<HYENA_ACT_GELU>(a, st); break;
        case HYENA_ACT_GELU_TANH: start_by_type<HYENA_ACT_GELU_TANH>(a, st); break;
        default: start_by_type<HYENA_ACT_IDENTITY>(a, st); break;
    }
    HYENA_TRY(cudaGetLastError(), "product launch");
    return 1;
}

int launch_ffn_backward(const FfnBackArgs &a, cudaStream_t st)
{
    uint16_t *dg = reinterpret_cast<uint16_t *>(static_cast<unsigned char *>(a.workspace) + 256);
    uint16_t *du = dg + a.M * a.F;
    switch (a.act) {
        case HYENA_ACT_SILU: slopes_kernel<HYENA_ACT_SILU><<<1184, 256, 0, st>>>(a, dg, du); break;
        case HYENA_ACT_GELU: slopes_kernel<HYENA_ACT_GELU><<<1184, 256, 0, st>>>(a, dg, du); break;
        case HYENA_ACT_GELU_TANH: slopes_kernel<HYENA_ACT_GELU_TANH><<<1184, 256, 0, st>>>(a, dg, du); break;
        default: slopes_kernel<HYENA_ACT_IDENTITY><<<1184, 256, 0, st>>>(a, dg, du); break;
    }
    HYENA_TRY(cudaGetLastError(), "ffn slopes launch");
    const auto grid = [](long long M, int N) {
        return static_cast<unsigned int>((M + TM - 1) / TM * ((N + TN - 1) / TN));
    };
    gradient_kernel<<<grid(a.M, a.D), 256, 0, st>>>(dg, du, a.F, 1, a.w1, a.w2, 1, a.ld_w, a.dx, a.ld_dx, a.M, a.D,
                                                    a.F);
    HYENA_TRY(cudaGetLastError(), "ffn dx launch");
    gradient_kernel<<<grid(a.F, a.D), 256, 0, st>>>(dg, nullptr, 1, a.F, a.x, nullptr, 1, a.ld_x, a.dw1, a.ld_dw, a.F,
                                                    a.D, a.M);
    HYENA_TRY(cudaGetLastError(), "ffn dWg launch");
    gradient_kernel<<<grid(a.F, a.D), 256, 0, st>>>(du, nullptr, 1, a.F, a.x, nullptr, 1, a.ld_x, a.dw2, a.ld_dw, a.F,
                                                    a.D, a.M);
    HYENA_TRY(cudaGetLastError(), "ffn dWu launch");
    return 4;
}

}  // namespace hyena
