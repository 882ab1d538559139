// product_narrow.cu -- forward products with few rows (generated tokens) on the
// tensor cores of sm_100a.
//
// The weights are the operand with 128 rows and the tokens the one with kNT <= 128:
// a CTA's tile is 2 x 128 weight rows (128 of the gate's and the same of the up
// projection's, or 256 in a row) times all tokens.  Every weight is read once,
// through a ring of TMA stages as deep as shared memory allows; which is all the
// time there is to spend, so k is split until every SM reads the same share.
#include "product_kernel.cuh"

namespace hyena {

namespace {

constexpr int kTile = 128;
constexpr int kOperand = kTile * kRowBytes;  // 16 KB

template <int kNT>
struct Narrow {
    static constexpr int kStages = kNT <= 32 ? 6 : (kNT == 64 ? 5 : 4);
    static constexpr int kStage = 2 * kOperand + kNT * kRowBytes;
    static constexpr int kSmem = kStages * kStage + 1024;
    static constexpr int kH = kNT / 2;                // tokens of a thread
    static constexpr int kC = kH < 16 ? kH : 16;      // of them at a time
};

struct NarrowArgs {
    Plan plan;
    int tile_cols;
    ProductArgs a;
    unsigned int *hdr;
};

__device__ __forceinline__ void store_one(void *p, bool f32, long long at, float v)
{
    if (f32)
        static_cast<float *>(p)[at] = v;
    else
        static_cast<uint16_t *>(p)[at] = bf16_bits(v);
}

template <int kNT, bool kF8>
__global__ void __launch_bounds__(kThreadsProduct, 1)
    product_narrow_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap m1,
                          const __grid_constant__ CUtensorMap m2, const __grid_constant__ NarrowArgs A)
{
    using T = Narrow<kNT>;
    constexpr int kStages = T::kStages, kStage = T::kStage, kH = T::kH, kC = T::kC;
    constexpr int kBlock = kF8 ? 128 : 64;  // k of a block
    extern __shared__ unsigned char raw[];
    __shared__ ProductShared<kStages> sh;
    __shared__ float token_scale[kEpiWarps][kH];
    __shared__ unsigned int token_max[kEpiWarps][kH];
    unsigned char *stages = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~1023ull);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x;
    const Plan &P = A.plan;
    volatile unsigned int *dead = &sh.dead;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(sh.full + i, 1);
            mbar_init(sh.empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sh.tfull + i, 1);
            mbar_init(sh.tempty + i, kEpiWarps);
        }
        sh.dead = 0u;
        fence_mbar_init();
    }
    if (warp == kEpiWarps + 1) tmem_alloc<1>(&sh.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp >= kEpiWarps) {
        fewer_registers();
        if (warp == kEpiWarps) {  // ----------------------------------- TMA
            int s = 0;
            uint32_t ph = 1;
            bool ok = true;
            for (Walk w(P, unit); ok && w.next();) {
                const int tn = w.tile / P.tiles_m, tm = w.tile - tn * P.tiles_m;
                const int n = tn * A.tile_cols;
                for (int kb = w.k0; kb < w.k1; ++kb) {
                    if (!(ok = warp_wait(sh.empty + s, ph, dead))) break;
                    if (elect_one()) {
                        unsigned char *p = stages + s * kStage;
                        mbar_arrive_expect_tx(sh.full + s, kStage);
                        tma_load_2d(p, &m1, sh.full + s, kb * kBlock, n);
                        tma_load_2d(p + kOperand, A.a.gated ? &m2 : &m1, sh.full + s, kb * kBlock,
                                    A.a.gated ? n : n + kTile);
                        tma_load_2d(p + 2 * kOperand, &mx, sh.full + s, kb * kBlock, tm * kNT);
                    }
                    __syncwarp();
                    if (++s == kStages) s = 0, ph ^= 1;
                }
            }
            if (!ok) let_land();
        } else if (warp == kEpiWarps + 1) {  // ----------------------- MMA
            constexpr uint32_t idesc = instruction_desc(kF8, kTile, kNT, false, false);
            const uint32_t base = smem_u32(stages);
            int s = 0, buf = 0;
            uint32_t ph = 0, tph = 1;
            bool ok = true;
            for (Walk w(P, unit); ok && w.next();) {
                for (int kb = w.k0; kb < w.k1; ++kb) {
                    const bool fresh = kF8 || kb == w.k0;
                    if (fresh && !(ok = warp_wait(sh.tempty + buf, tph, dead))) break;
                    if (!(ok = warp_wait(sh.full + s, ph, dead))) break;
                    tc_fence_after();
                    const uint64_t dw = operand_desc(base + s * kStage, 16);
                    const uint64_t dx = operand_desc(base + s * kStage + 2 * kOperand, 16);
                    const bool last = kF8 || kb + 1 == w.k1;
                    if (elect_one()) {
#pragma unroll
                        for (int g = 0; g < 2; ++g)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma<1, kF8>(tmem + buf * 256 + g * kTile, dw + (g * kOperand + i * 32) / 16, dx + i * 2,
                                            idesc, !(fresh && i == 0));
                        mma_commit_to<1>(sh.empty + s);
                        if (last) mma_commit_to<1>(sh.tfull + buf);
                    }
                    __syncwarp();
                    if (last) {
                        buf ^= 1;
                        if (buf == 0) tph ^= 1;
                    }
                    if (++s == kStages) s = 0, ph ^= 1;
                }
            }
            if (!ok) let_land();
        }
        __syncwarp();
    } else {  // ------------------------------------------------- sums, outputs
        more_registers();
        const int hh = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + hh * kH;
        const int groups = P.blocks;  // of codes: one a k-block
        int buf = 0;
        uint32_t tph = 0;
        bool ok = true;
        for (Walk w(P, unit); w.next();) {
            const int tn = w.tile / P.tiles_m, tm = w.tile - tn * P.tiles_m;
            const long long m = static_cast<long long>(tm) * kNT + hh * kH;  // this thread's first token
            float v[2 * kH];
            auto done_reading = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sh.tempty + buf);
                buf ^= 1;
                if (buf == 0) tph ^= 1;
            };
            if constexpr (kF8) {
#pragma unroll
                for (int i = 0; i < 2 * kH; ++i) v[i] = 0.f;
                const int gated = A.a.gated, tn1 = gated ? tn : 2 * tn;
                const bool two = gated || tn * A.tile_cols + kTile < A.a.N;
                const float *s1 = A.a.sw1 + static_cast<long long>(tn1) * groups;
                const float *s2 = gated ? A.a.sw2 + static_cast<long long>(tn) * groups : s1 + (two ? groups : 0);
                // the scales of the warp's tokens, a token a lane, one k-block ahead
                const float *sx0 = m + lane < A.a.M && lane < kH ? A.a.sx + (m + lane) * A.a.sx_row : nullptr;
                const float *sx1 = kH > 32 && m + 32 + lane < A.a.M ? A.a.sx + (m + 32 + lane) * A.a.sx_row : nullptr;
                const auto scale_at = [&](const float *p, int kb) {
                    return p ? __ldg(p + static_cast<long long>(kb) * A.a.sx_step) : 0.f;
                };
                float x0 = scale_at(sx0, w.k0), x1 = scale_at(sx1, w.k0);
                float f1 = __ldg(s1 + w.k0), f2 = __ldg(s2 + w.k0);
                for (int kb = w.k0; kb < w.k1; ++kb) {
                    __syncwarp();
                    if (lane < kH) token_scale[warp][lane] = x0;
                    if constexpr (kH > 32) token_scale[warp][lane + 32] = x1;
                    const float2 c1 = bcast2(f1), c2 = bcast2(f2);
                    if (kb + 1 < w.k1) {
                        x0 = scale_at(sx0, kb + 1);
                        x1 = scale_at(sx1, kb + 1);
                        f1 = __ldg(s1 + kb + 1);
                        f2 = __ldg(s2 + kb + 1);
                    }
                    if (ok) ok = wait_phase(sh.tfull + buf, tph, dead);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = lanes + buf * 256;
                    constexpr int kChunks = kH / kC;
                    float d[2][kC];
                    tmem_ld(d[0], at);
#pragma unroll
                    for (int i = 0; i < 2 * kChunks; ++i) {
                        tmem_wait(d[i & 1]);
                        if (i + 1 < 2 * kChunks)
                            tmem_ld(d[(i + 1) & 1], at + (i + 1) / kChunks * kTile + (i + 1) % kChunks * kC);
#pragma unroll
                        for (int j = 0; j < kC; j += 2) {
                            const float2 x = *reinterpret_cast<const float2 *>(&token_scale[warp][i % kChunks * kC + j]);
                            const float2 r =
                                __ffma2_rn(make_float2(d[i & 1][j], d[i & 1][j + 1]),
                                           __fmul2_rn(x, i < kChunks ? c1 : c2),
                                           make_float2(v[i * kC + j], v[i * kC + j + 1]));
                            v[i * kC + j] = r.x;
                            v[i * kC + j + 1] = r.y;
                        }
                    }
                    done_reading();
                }
            } else {
                if (ok) ok = wait_phase(sh.tfull + buf, tph, dead);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 2 * kH / kC; ++i) {
                        float d[kC];
                        tmem_ld(d, lanes + buf * 256 + i / (kH / kC) * kTile + i % (kH / kC) * kC);
                        tmem_wait(d);
#pragma unroll
                        for (int j = 0; j < kC; ++j) v[i * kC + j] = d[j];
                    }
                    done_reading();
                }
            }
            if (!ok) {
#pragma unroll
                for (int i = 0; i < 2 * kH; ++i) v[i] = __uint_as_float(0x7fffffffu);
            }
            if (w.k1 - w.k0 < P.blocks &&
                !join_parts<1>(v, P, unit, 0, w.tile, w.k0, tid, reinterpret_cast<unsigned char *>(A.hdr), &sh.flag))
                continue;
            const int n = tn * A.tile_cols + row;
            const int tokens = static_cast<int>(A.a.M - m < kH ? A.a.M - m : kH);  // may be negative
            if (!A.a.gated) {
#pragma unroll
                for (int j = 0; j < kH; ++j) {
                    if (j >= tokens) break;
                    if (n < A.a.N) store_one(A.a.y, A.a.y_f32, (m + j) * A.a.ld_y + n, v[j]);
                    if (n + kTile < A.a.N) store_one(A.a.y, A.a.y_f32, (m + j) * A.a.ld_y + n + kTile, v[kH + j]);
                }
                continue;
            }
            if (A.a.g && n < A.a.N) {
#pragma unroll
                for (int j = 0; j < kH; ++j) {
                    if (j >= tokens) break;
                    store_one(A.a.g, A.a.g_f32, (m + j) * A.a.ld_g + n, v[j]);
                    store_one(A.a.u, A.a.g_f32, (m + j) * A.a.ld_g + n, v[kH + j]);
                }
            }
            gate<kH>(v, A.a.act);
            if (kF8 && A.a.q) {
                // the largest of each token's 128 values: four warps' lanes
#pragma unroll
                for (int j = 0; j < kH; ++j) {
                    const unsigned int b = n < A.a.N ? __float_as_uint(v[j]) & 0x7fffffffu : 0u;
                    const unsigned int mx = __reduce_max_sync(0xffffffffu, b);
                    if (lane == 0) token_max[warp][j] = mx;
                }
                named_sync(2 + hh, kEpiThreads / 2);
#pragma unroll
                for (int j = 0; j < kH; ++j) {
                    if (j >= tokens) break;
                    unsigned int mx = token_max[4 * hh][j];
#pragma unroll
                    for (int i = 1; i < 4; ++i) mx = max(mx, token_max[4 * hh + i][j]);
                    const float scale = scale_of(mx);
                    if (n < A.a.N)
                        A.a.q[(m + j) * A.a.ld_q + n] = __nv_cvt_float_to_fp8(v[j] / scale, __NV_SATFINITE, __NV_E4M3);
                    if (row == 0) A.a.scales[(m + j) * P.tiles_n + tn] = scale;
                }
                named_sync(2 + hh, kEpiThreads / 2);
            } else if (n < A.a.N) {
#pragma unroll
                for (int j = 0; j < kH; ++j) {
                    if (j >= tokens) break;
                    static_cast<uint16_t *>(A.a.y)[(m + j) * A.a.ld_y + n] = bf16_bits(v[j]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kEpiWarps + 1) tmem_dealloc<1>(tmem);
    if (tid == 0 && sh.dead != 0u) atomicOr(A.hdr + 2, kErrLocalTimeout);
}

template <int kNT, bool kF8>
int start(const CUtensorMap &x, const CUtensorMap &w1, const CUtensorMap &w2, const NarrowArgs &w, cudaStream_t st)
{
    HYENA_TRY(cudaFuncSetAttribute(product_narrow_kernel<kNT, kF8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   Narrow<kNT>::kSmem),
              "product (narrow) attribute");
    product_narrow_kernel<kNT, kF8><<<w.plan.units, kThreadsProduct, Narrow<kNT>::kSmem, st>>>(x, w1, w2, w);
    HYENA_TRY(cudaGetLastError(), "product (narrow) launch");
    return 1;
}

template <bool kF8>
int start_by_tokens(int nt, const CUtensorMap &x, const CUtensorMap &w1, const CUtensorMap &w2, const NarrowArgs &w,
                    cudaStream_t st)
{
    switch (nt) {
        case 16: return start<16, kF8>(x, w1, w2, w, st);
        case 32: return start<32, kF8>(x, w1, w2, w, st);
        case 64: return start<64, kF8>(x, w1, w2, w, st);
        default: return start<128, kF8>(x, w1, w2, w, st);
    }
}

}  // namespace

int launch_product_narrow(const ProductArgs &a, cudaStream_t st)
{
    const int u = product_sms();
    if (u < 1) return -1;
    const int nt = narrow_tokens(a.M);
    const int kb = a.fp8 ? 128 : 64;
    CUtensorMap x, w1, w2;
    if (!encode_matrix(&x, a.x, a.fp8, a.M, a.K, a.ld_x, nt) ||
        !encode_matrix(&w1, a.w1, a.fp8, a.N, a.K, a.ld_w, kTile) ||
        !encode_matrix(&w2, a.gated ? a.w2 : a.w1, a.fp8, a.N, a.K, a.ld_w, kTile))
        return -1;
    NarrowArgs w{};
    w.tile_cols = a.gated ? kTile : 2 * kTile;
    Plan &p = w.plan;
    p.tiles_m = static_cast<int>((a.M + nt - 1) / nt);
    p.tiles_n = (a.N + w.tile_cols - 1) / w.tile_cols;
    p.tiles = p.tiles_m * p.tiles_n;
    p.blocks = (a.K + kb - 1) / kb;
    const long long all = static_cast<long long>(p.tiles) * p.blocks;
    p.units = all / 2 < u ? static_cast<int>(all / 2 > 0 ? all / 2 : 1) : u;
    p.split = p.tiles <= p.units ? p.tiles : p.tiles % p.units + p.units;
    w.a = a;
    w.hdr = static_cast<unsigned int *>(a.workspace);
    return a.fp8 ? start_by_tokens<true>(nt, x, w1, w2, w, st) : start_by_tokens<false>(nt, x, w1, w2, w, st);
}

}  // namespace hyena
