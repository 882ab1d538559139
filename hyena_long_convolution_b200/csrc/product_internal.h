// product_internal.h -- host-side declarations of the 8-bit products and the
// feed-forward block, shared by their entry points and launchers (not part of
// the public interface).
#pragma once

#include <atomic>

#include "layer_internal.h"

namespace hyena {

constexpr int kScaleGroup = 128;  // channels (and weight rows) per scale

struct QuantArgs {
    const void *x;
    long long ld_x;
    bool x_bf16;
    uint8_t *q;
    long long ld_q;
    float *scales;
    int block;
    long long rows;
    int D;
};

int launch_fp8_quantize(const QuantArgs &a, cudaStream_t st);

// y = x w1^T, or act(x w1^T) (x w2^T): forward products of either operand type.
struct ProductArgs {
    const void *x, *w1, *w2;  // bf16, or e4m3 codes
    long long ld_x, ld_w;
    bool fp8;
    const float *sx, *sw1, *sw2;  // scales of codes
    int sx_row, sx_step;          // scale of (row m, group j): sx[m sx_row + j sx_step]
    bool gated;                   // two weights and the activation between them
    int act;
    void *y;                      // bf16 or fp32, or
    bool y_f32;
    long long ld_y;
    uint8_t *q;                   // e4m3 codes with scales
    long long ld_q;
    float *scales;
    void *g, *u;                  // kept products or null
    long long ld_g;
    bool g_f32;
    long long M;
    int N, K;
    void *workspace;
};

int launch_product(const ProductArgs &a, cudaStream_t st);

struct FfnBackArgs {
    const uint16_t *dy, *x, *w1, *w2;
    long long ld_dy, ld_x, ld_w;
    const void *g, *u;
    long long ld_g;
    bool g_f32;
    int act;
    uint16_t *dx, *dw1, *dw2;
    long long ld_dx, ld_dw;
    long long M;
    int D, F;
    void *workspace;
};

int launch_ffn_backward(const FfnBackArgs &a, cudaStream_t st);

// The narrow kernel's tokens: the smallest of 16, 32, 64 or (not with two weights in
// codes, whose sums would fill the registers) 128 that holds the rows, or several of
// the largest.
inline int narrow_tokens(long long M, bool fp8_gated)
{
    return M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 || fp8_gated ? 64 : 128));
}
// Whether the workspace of a call has room for the wide kernel's parts: without it the call is
// narrow.  One condition for both, so that no part is written where there is no room.
inline bool product_has_parts(long long M) { return M > 32; }
bool product_is_narrow(long long M, int N, bool fp8, bool gated);

int launch_product_narrow(const ProductArgs &a, cudaStream_t st);
int launch_product_wide(const ProductArgs &a, cudaStream_t st);
int launch_ffn_dx_narrow(const FfnBackArgs &a, const uint16_t *dg, const uint16_t *du, bool beside, cudaStream_t st);
bool ffn_dx_is_narrow(long long M, int D);
int launch_ffn_gradients(const FfnBackArgs &a, const uint16_t *dg, const uint16_t *du, cudaStream_t st);

// Map of a [rows, cols] matrix of codes, bf16 or fp32 (size 1, 2, 4) with boxes of 128 bytes of a row
// times box_rows rows, laid out with the 128-byte swizzle.
bool encode_matrix(CUtensorMap *m, const void *p, int size, long long rows, int cols, long long ld, int box_rows);
int product_sms();

// Header and, where the wide kernel may share a tile's k, the parts; of the gradient dg
// and du too.
size_t product_workspace(long long M);
size_t ffn_backward_workspace(long long M, int F);

// Lets a kernel have `bytes` of shared memory, once a device (`done`: a bit each).
int allow_shared(const void *kernel, int bytes, std::atomic<unsigned long long> &done);

// Launches a kernel that waits for the stream itself (wait_for_stream), so that its
// launch and its setup overlap the end of the kernel before it.
template <class... P, class... Q>
int launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st,
                 const char *what, const Q &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    HYENA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...), what);
    return 1;
}

}  // namespace hyena
