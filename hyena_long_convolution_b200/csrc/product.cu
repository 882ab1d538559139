// product.cu -- host side of the products (tensor maps, workspace, which kernel)
// and the element-wise part of the feed-forward block's gradient:
//
//   dg = dy u act'(g), du = dy act(g), rounded to bf16: they are operands of the
//   tensor cores.  That adds 1.7e-3 of rounding to the gradients' own 1.7e-3; g and u
//   kept in bf16 add as much again (3.0e-3 in all), kept in fp32 nothing.
//
// HBM-bound: 14 bytes an element with fp32 products, 193 us for 8192 x 11008, 6.5 TB/s.
#include <cudaTypedefs.h>

#include <mutex>

#include "product_device.cuh"
#include "product_kernel.cuh"

namespace hyena {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

void resolve_encode()
{
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

// dg = dy u act'(g), du = dy act(g), 8 values a thread at a time.
template <int kAct, bool kF32>
__global__ void __launch_bounds__(256) slopes_kernel(const FfnBackArgs A, uint16_t *dg, uint16_t *du)
{
    wait_for_stream();
    const long long per = A.F / 8, n = A.M * per;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const long long m = i / per, f = (i - m * per) * 8;
        float g[8], u[8], d[8], a[8], b[8];
        if constexpr (kF32) {
            load8_f32(g, static_cast<const float *>(A.g) + m * A.ld_g + f);
            load8_f32(u, static_cast<const float *>(A.u) + m * A.ld_g + f);
        } else {
            load8_bf16(g, static_cast<const uint16_t *>(A.g) + m * A.ld_g + f);
            load8_bf16(u, static_cast<const uint16_t *>(A.u) + m * A.ld_g + f);
        }
        load8_bf16(d, A.dy + m * A.ld_dy + f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float2 slope;
            const float2 y = activation_slope2<kAct>(make_float2(g[j], g[j + 1]), slope);
            const float2 dy = make_float2(d[j], d[j + 1]);
            const float2 dgate = __fmul2_rn(__fmul2_rn(dy, make_float2(u[j], u[j + 1])), slope), dup = __fmul2_rn(dy, y);
            a[j] = dgate.x, a[j + 1] = dgate.y;
            b[j] = dup.x, b[j + 1] = dup.y;
        }
        *reinterpret_cast<uint4 *>(dg + i * 8) = pack_bf16(a);
        *reinterpret_cast<uint4 *>(du + i * 8) = pack_bf16(b);
    }
}

template <int kAct>
int start_slopes(const FfnBackArgs &a, uint16_t *dg, uint16_t *du, int grid, cudaStream_t st)
{
    return launch_early(a.g_f32 ? slopes_kernel<kAct, true> : slopes_kernel<kAct, false>, dim3(grid), 256, 0, 1, st,
                        "ffn slopes launch", a, dg, du);
}

// Parts of shared tiles: fp32 sums of 128 x 256 for each CTA.
size_t part_bytes()
{
    const int sms = product_sms();
    return static_cast<size_t>(sms > 0 ? sms : 148) * 128 * 256 * 4;
}

}  // namespace

bool encode_matrix(CUtensorMap *m, const void *p, int size, long long rows, int cols, long long ld, int box_rows)
{
    std::call_once(g_encode_once, resolve_encode);
    if (g_encode == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * size};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kRowBytes / size), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1u, 1u};
    const CUtensorMapDataType type = size == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    return g_encode(m, type, 2, const_cast<void *>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int product_sms()
{
    static int sms = [] {  // the same on every device that the library is built for
        int dev = 0, n = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        return n;
    }();
    return sms;
}

int allow_shared(const void *kernel, int bytes, std::atomic<unsigned long long> &done)
{
    int dev = 0;
    HYENA_TRY(cudaGetDevice(&dev), "current device");
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return 0;
    HYENA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes), "product attribute");
    if (dev < 64) done.fetch_or(bit, std::memory_order_release);
    return 0;
}

// The narrow kernel reads the weights at the rate of HBM, where the wide one has most of
// its rows empty (32 rows, 4096 -> 4096 x 11008: in e4m3 13 and 23 us, in bf16 34 and
// 38).  Its smaller tiles pay
//
//   up to 32 rows always, so that a workspace of so few needs no parts.  With one weight
//   in codes and a little more than a tile an SM that costs 17 to 32 rows something
//   (4096 -> 19200: 24.9-25.5 and 20.8-22.6 us; 22016: 25.5-26.0 and 21.7-25.0), with
//   more it saves (38016: 38-39 and 42-43);
//
//   up to 64 rows, for one weight in codes up to a tile an SM (4096 -> 18944: 19.4 and
//   21.4 us; 22016: 33 and 22), for two in bf16 always (19200: 75 and 78);
//   beyond, and for two weights in codes, while they leave SMs to share a tile's k
//   (4096 -> 8192, 64 rows, two weights in codes 21.0 and 22.4, 9728: 29 and 23; 128
//   rows in bf16 32.5 and 35, 41 and 37; 256 rows of 1024 x 4096 in e4m3 12 and 18, 74
//   tiles and more 21 and 20); of two in bf16 with more than 128 rows half as many
//   (4096 x 2048, 256 rows: 64 tiles 18 and 16 us).
bool product_is_narrow(long long M, int N, bool fp8, bool gated)
{
    if (!product_has_parts(M)) return true;
    const int nt = narrow_tokens(M, fp8 && gated), sms = product_sms();
    const long long tiles = (M + nt - 1) / nt * ((N + 127) / 128);
    if (M <= 64 && !(fp8 && gated)) return !fp8 || tiles <= sms;
    return tiles <= (fp8 || M <= 128 ? sms / 2 : sms / 4);
}

// dx of few rows likewise, by the weights' columns (steps, 1 row: 1032 -> 2760 38 and 24 us,
// 4096 -> 11008 126 and 107; 128 rows 50 and 38, 139 and 126), and of more rows while two
// CTAs to a tile leave some SMs to dW beside it: 256 rows of 512 -> 1408 (8 tiles) 35 and
// 25, of 2048 -> 4096 (32) 66 and 56, 700 of 1032 -> 2760 (54) 62 and 60, 200 of 4096 ->
// 11008 (64) 163 and 165; but 1000 of 1032 -> 2760 (72) 71.5 and 74.6.  The gradient
// alone, pairs and columns: 256 rows of 2048 -> 4096 47 and 37, 4096 -> 4096 (64) 57 and
// 52, 4096 -> 11008 (64) 118 and 119, 700 of 1032 -> 2760 41.5 and 43.
bool ffn_dx_is_narrow(long long M, int D)
{
    return M <= 128 || 2 * ((M + 127) / 128) * ((D + 127) / 128) <= product_sms() - 16;
}

size_t product_workspace(long long M) { return kProductHeader + (product_has_parts(M) ? part_bytes() : 0); }

size_t ffn_backward_workspace(long long M, int F)
{
    return kProductHeader + part_bytes() + static_cast<size_t>(M) * F * 4;
}

int launch_product(const ProductArgs &a, cudaStream_t st)
{
    return product_is_narrow(a.M, a.N, a.fp8, a.gated) ? launch_product_narrow(a, st) : launch_product_wide(a, st);
}

int launch_ffn_backward(const FfnBackArgs &a, cudaStream_t st)
{
    const int sms = product_sms();
    if (sms < 1) return -1;
    uint16_t *dg = reinterpret_cast<uint16_t *>(static_cast<unsigned char *>(a.workspace) + kProductHeader +
                                                part_bytes());
    uint16_t *du = dg + a.M * a.F;
    const long long ctas = (a.M * (a.F / 8) + 255) / 256;
    const int grid = ctas < sms * 8ll ? static_cast<int>(ctas) : sms * 8;
    int n = 0;
    switch (a.act) {
        case HYENA_ACT_SILU: n = start_slopes<HYENA_ACT_SILU>(a, dg, du, grid, st); break;
        case HYENA_ACT_GELU: n = start_slopes<HYENA_ACT_GELU>(a, dg, du, grid, st); break;
        case HYENA_ACT_GELU_TANH: n = start_slopes<HYENA_ACT_GELU_TANH>(a, dg, du, grid, st); break;
        default: n = start_slopes<HYENA_ACT_IDENTITY>(a, dg, du, grid, st); break;
    }
    if (n < 0) return -1;
    const int k = launch_ffn_gradients(a, dg, du, st);
    return k < 0 ? -1 : n + k;
}

}  // namespace hyena
