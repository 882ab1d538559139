// product_api.cu -- the extern "C" entry points of the 8-bit products and the
// feed-forward block: argument checks and dispatch.  Nothing here computes any
// part of an operator.
#include "product_internal.h"

namespace hyena {

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool is_dtype(int t) { return t == HYENA_BF16 || t == HYENA_F32; }
bool is_act(int a) { return a >= HYENA_ACT_SILU && a <= HYENA_ACT_IDENTITY; }

// A tensor of `rows` rows of `width` elements of `size` bytes, row stride ld in
// elements, a multiple of `step` (rows == 0: not looked at).
hyena_status_t check_tensor(const void *p, int64_t ld, int64_t rows, int width, int step, int size)
{
    if (rows == 0) return HYENA_OK;
    if (!p || ld < width) return HYENA_ERR_INVALID_ARG;
    if (ld % step || !aligned16(p)) return HYENA_ERR_ALIGNMENT;
    // element offsets in 64 bits, tensor maps' strides in 40
    if (ld >= (1ll << 38) / size || rows > (1ll << 46) / ld / size) return HYENA_ERR_UNSUPPORTED;
    return HYENA_OK;
}

hyena_status_t check_sizes(int64_t rows, int a, int b)
{
    if (rows < 0 || a < 1 || b < 1) return HYENA_ERR_INVALID_ARG;
    if (a % 8 || b % 8) return HYENA_ERR_ALIGNMENT;
    if (rows >= (1ll << 31) || a > HYENA_MAX_WIDTH || b > HYENA_MAX_WIDTH) return HYENA_ERR_UNSUPPORTED;
    // tiles of 256 rows x 128 columns are counted in 31 bits
    if (((rows + 255) / 256) * ((a > b ? a : b) / 128 + 1) >= (1ll << 31)) return HYENA_ERR_UNSUPPORTED;
    return HYENA_OK;
}

// fp32 scales: only their presence and word alignment matter.
hyena_status_t check_scales(const float *s)
{
    if (!s) return HYENA_ERR_INVALID_ARG;
    return (reinterpret_cast<uintptr_t>(s) & 3u) ? HYENA_ERR_ALIGNMENT : HYENA_OK;
}

hyena_status_t check_workspace(const void *ws, size_t bytes, size_t need)
{
    if (!ws || bytes < need) return HYENA_ERR_WORKSPACE;
    return aligned16(ws) ? HYENA_OK : HYENA_ERR_ALIGNMENT;
}

hyena_status_t check_group(int group)
{
    if (group == 0 || group == kScaleGroup) return HYENA_OK;
    return group < 0 ? HYENA_ERR_INVALID_ARG : HYENA_ERR_UNSUPPORTED;
}

// An output at the address of one of the others would be written while that is read.
// (Extents are not compared: columns of one matrix may lie between each other.)
template <typename... T>
bool clash(const void *out, const T *...others)
{
    return out != nullptr && ((out == static_cast<const void *>(others)) || ...);
}

int scale_groups(int n) { return (n + kScaleGroup - 1) / kScaleGroup; }

hyena_status_t product(const ProductArgs &a, void *stream)
{
    const int n = launch_product(a, static_cast<cudaStream_t>(stream));
    if (n < 0) return HYENA_ERR_CUDA;
    set_last_launches(n);
    return HYENA_OK;
}

}  // namespace

}  // namespace hyena

using namespace hyena;

extern "C" {

hyena_status_t hyena_fp8_quantize(const void *x, int64_t ld_x, hyena_dtype_t x_type, uint8_t *q, int64_t ld_q,
                                  float *scales, int block, int64_t rows, int D, void *stream)
{
    hyena_status_t st = check_sizes(rows, D, 8);
    if (st != HYENA_OK) return st;
    if (!is_dtype(x_type)) return HYENA_ERR_INVALID_ARG;
    if (block != 1 && block != kScaleGroup) return block < 1 ? HYENA_ERR_INVALID_ARG : HYENA_ERR_UNSUPPORTED;
    st = check_tensor(x, ld_x, rows, D, 8, x_type == HYENA_BF16 ? 2 : 4);
    if (st == HYENA_OK) st = check_tensor(q, ld_q, rows, D, 8, 1);
    if (st == HYENA_OK && rows > 0) st = check_scales(scales);
    if (st != HYENA_OK) return st;
    set_last_launches(0);
    if (rows == 0) return HYENA_OK;
    if (clash(q, x, scales) || clash(scales, x)) return HYENA_ERR_INVALID_ARG;
    QuantArgs a{};
    a.x = x;
    a.ld_x = ld_x;
    a.x_bf16 = x_type == HYENA_BF16;
    a.q = q;
    a.ld_q = ld_q;
    a.scales = scales;
    a.block = block;
    a.rows = rows;
    a.D = D;
    const int n = launch_fp8_quantize(a, static_cast<cudaStream_t>(stream));
    if (n < 0) return HYENA_ERR_CUDA;
    set_last_launches(n);
    return HYENA_OK;
}

size_t hyena_fp8_matmul_workspace_size(int64_t M, int N, int K)
{
    return check_sizes(M, N, K) == HYENA_OK ? product_workspace(M) : 0;
}

hyena_status_t hyena_fp8_matmul(const uint8_t *x, int64_t ld_x, const float *x_scales, int x_group, const uint8_t *w,
                                int64_t ld_w, const float *w_scales, void *y, int64_t ld_y, hyena_dtype_t y_type,
                                int64_t M, int N, int K, void *workspace, size_t workspace_bytes, void *stream)
{
    hyena_status_t st = check_sizes(M, N, K);
    if (st == HYENA_OK) st = check_group(x_group);
    if (st != HYENA_OK) return st;
    if (!is_dtype(y_type)) return HYENA_ERR_INVALID_ARG;
    st = check_tensor(x, ld_x, M, K, 16, 1);
    if (st == HYENA_OK) st = check_tensor(w, ld_w, N, K, 16, 1);
    if (st == HYENA_OK) st = check_tensor(y, ld_y, M, N, 8, y_type == HYENA_BF16 ? 2 : 4);
    if (st == HYENA_OK && M > 0) st = check_scales(x_scales);
    if (st == HYENA_OK) st = check_scales(w_scales);
    if (st != HYENA_OK) return st;
    set_last_launches(0);
    if (M == 0) return HYENA_OK;
    st = check_workspace(workspace, workspace_bytes, product_workspace(M));
    if (st != HYENA_OK) return st;
    if (clash(y, x, w, x_scales, w_scales, workspace)) return HYENA_ERR_INVALID_ARG;
    ProductArgs a{};
    a.x = x;
    a.w1 = w;
    a.ld_x = ld_x;
    a.ld_w = ld_w;
    a.fp8 = true;
    a.sx = x_scales;
    a.sw1 = w_scales;
    a.sx_row = x_group ? scale_groups(K) : 1;
    a.sx_step = x_group ? 1 : 0;
    a.y = y;
    a.y_f32 = y_type == HYENA_F32;
    a.ld_y = ld_y;
    a.M = M;
    a.N = N;
    a.K = K;
    a.workspace = workspace;
    return product(a, stream);
}

size_t hyena_gated_ffn_workspace_size(int64_t M, int D, int F, int backward)
{
    if (check_sizes(M, D, F) != HYENA_OK) return 0;
    return backward ? ffn_backward_workspace(M, F) : product_workspace(M);
}

hyena_status_t hyena_gated_ffn(const hyena_bf16_t *x, int64_t ld_x, const hyena_bf16_t *gate_w,
                               const hyena_bf16_t *up_w, int64_t ld_w, hyena_activation_t act, hyena_bf16_t *y,
                               int64_t ld_y, void *gate_out, void *up_out, int64_t ld_g, hyena_dtype_t keep_type,
                               int64_t M, int D, int F, void *workspace, size_t workspace_bytes, void *stream)
{
    hyena_status_t st = check_sizes(M, D, F);
    if (st != HYENA_OK) return st;
    if (!is_act(act) || (gate_out == nullptr) != (up_out == nullptr)) return HYENA_ERR_INVALID_ARG;
    st = check_tensor(x, ld_x, M, D, 8, 2);
    if (st == HYENA_OK) st = check_tensor(gate_w, ld_w, F, D, 8, 2);
    if (st == HYENA_OK) st = check_tensor(up_w, ld_w, F, D, 8, 2);
    if (st == HYENA_OK) st = check_tensor(y, ld_y, M, F, 8, 2);
    if (st == HYENA_OK && gate_out) {
        if (!is_dtype(keep_type)) return HYENA_ERR_INVALID_ARG;
        const int size = keep_type == HYENA_BF16 ? 2 : 4;
        st = check_tensor(gate_out, ld_g, M, F, 8, size);
        if (st == HYENA_OK) st = check_tensor(up_out, ld_g, M, F, 8, size);
    }
    if (st != HYENA_OK) return st;
    set_last_launches(0);
    if (M == 0) return HYENA_OK;
    st = check_workspace(workspace, workspace_bytes, product_workspace(M));
    if (st != HYENA_OK) return st;
    if (clash(y, x, gate_w, up_w, gate_out, up_out, workspace) || clash(gate_out, x, gate_w, up_w, up_out, workspace) ||
        clash(up_out, x, gate_w, up_w, workspace))
        return HYENA_ERR_INVALID_ARG;
    ProductArgs a{};
    a.x = x;
    a.w1 = gate_w;
    a.w2 = up_w;
    a.ld_x = ld_x;
    a.ld_w = ld_w;
    a.gated = true;
    a.act = act;
    a.y = y;
    a.ld_y = ld_y;
    a.g = gate_out;
    a.u = up_out;
    a.ld_g = ld_g;
    a.g_f32 = keep_type == HYENA_F32;
    a.M = M;
    a.N = F;
    a.K = D;
    a.workspace = workspace;
    return product(a, stream);
}

hyena_status_t hyena_gated_ffn_fp8(const uint8_t *x, int64_t ld_x, const float *x_scales, int x_group,
                                   const uint8_t *gate_w, const float *gate_scales, const uint8_t *up_w,
                                   const float *up_scales, int64_t ld_w, hyena_activation_t act, hyena_bf16_t *y,
                                   int64_t ld_y, uint8_t *q, int64_t ld_q, float *scales, int64_t M, int D, int F,
                                   void *workspace, size_t workspace_bytes, void *stream)
{
    hyena_status_t st = check_sizes(M, D, F);
    if (st == HYENA_OK) st = check_group(x_group);
    if (st != HYENA_OK) return st;
    if (!is_act(act) || (M > 0 && (y == nullptr) == (q == nullptr))) return HYENA_ERR_INVALID_ARG;
    st = check_tensor(x, ld_x, M, D, 16, 1);
    if (st == HYENA_OK) st = check_tensor(gate_w, ld_w, F, D, 16, 1);
    if (st == HYENA_OK) st = check_tensor(up_w, ld_w, F, D, 16, 1);
    if (st == HYENA_OK && y) st = check_tensor(y, ld_y, M, F, 8, 2);
    if (st == HYENA_OK && q) st = check_tensor(q, ld_q, M, F, 16, 1);
    if (st == HYENA_OK && q) st = check_scales(scales);
    if (st == HYENA_OK && M > 0) st = check_scales(x_scales);
    if (st == HYENA_OK) st = check_scales(gate_scales);
    if (st == HYENA_OK) st = check_scales(up_scales);
    if (st != HYENA_OK) return st;
    set_last_launches(0);
    if (M == 0) return HYENA_OK;
    st = check_workspace(workspace, workspace_bytes, product_workspace(M));
    if (st != HYENA_OK) return st;
    for (const void *out : {static_cast<const void *>(y), static_cast<const void *>(q), static_cast<const void *>(scales)})
        if (clash(out, x, x_scales, gate_w, gate_scales, up_w, up_scales, workspace)) return HYENA_ERR_INVALID_ARG;
    if (clash(q, scales)) return HYENA_ERR_INVALID_ARG;
    ProductArgs a{};
    a.x = x;
    a.w1 = gate_w;
    a.w2 = up_w;
    a.ld_x = ld_x;
    a.ld_w = ld_w;
    a.fp8 = true;
    a.sx = x_scales;
    a.sw1 = gate_scales;
    a.sw2 = up_scales;
    a.sx_row = x_group ? scale_groups(D) : 1;
    a.sx_step = x_group ? 1 : 0;
    a.gated = true;
    a.act = act;
    a.y = y;
    a.ld_y = ld_y;
    a.q = q;
    a.ld_q = ld_q;
    a.scales = scales;
    a.M = M;
    a.N = F;
    a.K = D;
    a.workspace = workspace;
    return product(a, stream);
}

hyena_status_t hyena_gated_ffn_backward(const hyena_bf16_t *dy, int64_t ld_dy, const hyena_bf16_t *x, int64_t ld_x,
                                        const hyena_bf16_t *gate_w, const hyena_bf16_t *up_w, int64_t ld_w,
                                        const void *gate, const void *up, int64_t ld_g, hyena_dtype_t keep_type,
                                        hyena_activation_t act, hyena_bf16_t *dx, int64_t ld_dx,
                                        hyena_bf16_t *dgate_w, hyena_bf16_t *dup_w, int64_t ld_dw, int64_t M, int D,
                                        int F, void *workspace, size_t workspace_bytes, void *stream)
{
    hyena_status_t st = check_sizes(M, D, F);
    if (st != HYENA_OK) return st;
    if (!is_act(act) || !is_dtype(keep_type)) return HYENA_ERR_INVALID_ARG;
    const int size = keep_type == HYENA_BF16 ? 2 : 4;
    st = check_tensor(dy, ld_dy, M, F, 8, 2);
    if (st == HYENA_OK) st = check_tensor(x, ld_x, M, D, 8, 2);
    if (st == HYENA_OK) st = check_tensor(gate_w, ld_w, F, D, 8, 2);
    if (st == HYENA_OK) st = check_tensor(up_w, ld_w, F, D, 8, 2);
    if (st == HYENA_OK) st = check_tensor(gate, ld_g, M, F, 8, size);
    if (st == HYENA_OK) st = check_tensor(up, ld_g, M, F, 8, size);
    if (st == HYENA_OK) st = check_tensor(dx, ld_dx, M, D, 8, 2);
    if (st == HYENA_OK) st = check_tensor(dgate_w, ld_dw, F, D, 8, 2);
    if (st == HYENA_OK) st = check_tensor(dup_w, ld_dw, F, D, 8, 2);
    if (st != HYENA_OK) return st;
    set_last_launches(0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {
        for (hyena_bf16_t *dw : {dgate_w, dup_w})
            if (cudaMemset2DAsync(dw, static_cast<size_t>(ld_dw) * 2, 0, static_cast<size_t>(D) * 2, F, s) !=
                cudaSuccess)
                return HYENA_ERR_CUDA;
        set_last_launches(2);
        return HYENA_OK;
    }
    st = check_workspace(workspace, workspace_bytes, ffn_backward_workspace(M, F));
    if (st != HYENA_OK) return st;
    for (const void *out : {dx, dgate_w, dup_w})
        if (clash(out, dy, x, gate_w, up_w, gate, up, workspace)) return HYENA_ERR_INVALID_ARG;
    if (clash(dx, dgate_w, dup_w) || clash(dgate_w, dup_w)) return HYENA_ERR_INVALID_ARG;
    FfnBackArgs a{};
    a.dy = dy;
    a.x = x;
    a.w1 = gate_w;
    a.w2 = up_w;
    a.ld_dy = ld_dy;
    a.ld_x = ld_x;
    a.ld_w = ld_w;
    a.g = gate;
    a.u = up;
    a.ld_g = ld_g;
    a.g_f32 = keep_type == HYENA_F32;
    a.act = act;
    a.dx = dx;
    a.dw1 = dgate_w;
    a.dw2 = dup_w;
    a.ld_dx = ld_dx;
    a.ld_dw = ld_dw;
    a.M = M;
    a.D = D;
    a.F = F;
    a.workspace = workspace;
    const int n = launch_ffn_backward(a, s);
    if (n < 0) return HYENA_ERR_CUDA;
    set_last_launches(n);
    return HYENA_OK;
}

}  // extern "C"
