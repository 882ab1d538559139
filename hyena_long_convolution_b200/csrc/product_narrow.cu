// product_narrow.cu -- products with few rows (generated tokens; dx of the feed-forward
// block's gradient) on the tensor cores of sm_100a.
//
// The weights are the operand with 128 rows and the tokens the one with kNT <= 128:
// a CTA's tile is 128 weight rows (128 of the gate's and the same of the up
// projection's) times all tokens, read through a ring of TMA stages as deep as shared
// memory allows.  With few tokens reading the weights is all the time there is to
// spend, and some 80 CTAs with 200 KB under way each are enough to do it at the rate
// of HBM.  With fewer tiles than that a cluster of CTAs shares a tile's k and joins its
// sums through their shared memory, in the order of k.  The sums leave through shared
// memory in any case: a warp then has a token's 128 values, four a lane, for wide
// stores and the maximum that codes need.
//
// Bound by HBM and by what comes before and after the stream: launch, first data 2.5 us
// after, sums and outputs 1 to 3.  On the device, weights from HBM: one token through
// 4096 -> 2 x 11008 in bf16 31-32 us (5.7 TB/s, 87% of the measured copy), through 4096
// -> 12288 in e4m3 12 us (4.2 TB/s); 16 through 4096 -> 2 x 11008 in e4m3, codes out,
// 18.7 (4.8 TB/s); 64 through 11008 -> 4096 in e4m3 15.8, by clusters of four.  Parts in
// global memory, added up by the last CTA to arrive, took 22 and 40 us where clusters
// take 15 and 17; the outputs straight from the registers, 64 times the same code, 40 us
// for 128 tokens' codes.
#include "product_kernel.cuh"

namespace hyena {

namespace {

constexpr int kTile = 128;
constexpr int kOperand = kTile * kRowBytes;  // 16 KB
constexpr int kRing = 217 * 1024;            // shared memory for stages, at most

template <int kNT, bool kGated>
struct Narrow {
    static constexpr int kG = kGated ? 2 : 1;  // weights
    static constexpr int kStage = kG * kOperand + kNT * kRowBytes;
    static constexpr int kStages = kRing / kStage;
    static constexpr int kSmem = kStages * kStage + 1024;
    static constexpr int kH = kNT / 2;            // tokens of a thread
    static constexpr int kC = kH < 16 ? kH : 16;  // of them at a time
    // Parts of tensor memory that sums alternate between.  Codes' sums go to registers
    // after each 128 k, and a turn through both takes longer than the MMAs between.
    static constexpr int kBufs = 512 / (kG * kNT) < 8 ? 512 / (kG * kNT) : 8;
    static_assert(kG * kNT * kTile * 4 <= kStages * kStage, "a tile's sums fit the stages");
};

struct NarrowArgs {
    int tiles_m; // tiles of tokens
    int blocks;  // k-blocks
    int share;   // CTAs of a cluster, which share a tile's k
    int blocks1; // dx: k-blocks of the first pair of operands
    bool beside; // dx: dW may start beside it
    ProductArgs a;
    unsigned int *hdr;
};

__device__ __forceinline__ void store_four(void *p, bool f32, long long at, float2 lo, float2 hi)
{
    if (f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + at) = make_float4(lo.x, lo.y, hi.x, hi.y);
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + at) =
            make_uint2(float2_to_bf16x2(lo), float2_to_bf16x2(hi));
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ float2 activate(float2 g, int act)
{
    switch (act) {
        case HYENA_ACT_SILU: return activation2<HYENA_ACT_SILU>(g);
        case HYENA_ACT_GELU: return activation2<HYENA_ACT_GELU>(g);
        case HYENA_ACT_GELU_TANH: return activation2<HYENA_ACT_GELU_TANH>(g);
        default: return g;
    }
}

template <int kNT, bool kF8, bool kGated, bool kDx>
__global__ void __launch_bounds__(kThreadsProduct, 1)
    product_narrow_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mx2,
                          const __grid_constant__ CUtensorMap m1, const __grid_constant__ CUtensorMap m2,
                          const __grid_constant__ NarrowArgs A)
{
    using T = Narrow<kNT, kGated>;
    constexpr int kStages = T::kStages, kStage = T::kStage, kH = T::kH, kC = T::kC, kG = T::kG, kBufs = T::kBufs;
    constexpr int kBlock = kF8 ? 128 : 64;  // k of a block
    extern __shared__ unsigned char raw[];
    __shared__ ProductShared<kStages> sh;
    __shared__ __align__(16) float token_scale[kEpiWarps][2][kH];
    unsigned char *stages = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~1023ull);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int share = A.share, rank = share > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int tn = blockIdx.x / share / A.tiles_m, m0 = (blockIdx.x / share - tn * A.tiles_m) * kNT;
    const int k0 = A.blocks * rank / share, k1 = A.blocks * (rank + 1) / share;
    volatile unsigned int *dead = &sh.dead;

    if (tid == kEpiThreads) {
        prefetch_map(&m1);
        prefetch_map(&mx);
        if (kGated || kDx) prefetch_map(&m2);
        if (kDx) prefetch_map(&mx2);
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(sh.full + i, 1);
            mbar_init(sh.empty + i, 1);
        }
        for (int i = 0; i < kBufs; ++i) {
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
    wait_for_stream();
    if (kDx && A.beside) let_next_start();
    const uint32_t tmem = sh.tmem;

    if (warp >= kEpiWarps) {
        fewer_registers();
        const uint32_t on = elected_lane();
        int s = 0;
        bool ok = true;
        if (warp == kEpiWarps) {  // ----------------------------------- TMA
            uint32_t ph = 1;
            for (int kb = k0; kb < k1; ++kb) {
                if (!(ok = warp_wait(sh.empty + s, ph, dead))) break;
                unsigned char *p = stages + s * kStage;
                const uint32_t bar = smem_u32(sh.full + s);
                expect_tx(on, sh.full + s, kStage);
                if constexpr (kDx) {  // k is not the weights' contiguous axis: boxes of 64 columns x 64 k
                    const bool up = kb >= A.blocks1;
                    const int k = (up ? kb - A.blocks1 : kb) * kBlock;
                    load_box<1>(on, p, up ? &m2 : &m1, bar, tn * kTile, k);
                    load_box<1>(on, p + kOperand / 2, up ? &m2 : &m1, bar, tn * kTile + 64, k);
                    load_box<1>(on, p + kOperand, up ? &mx2 : &mx, bar, k, m0);
                } else {
                    load_box<1>(on, p, &m1, bar, kb * kBlock, tn * kTile);
                    if (kGated) load_box<1>(on, p + kOperand, &m2, bar, kb * kBlock, tn * kTile);
                    load_box<1>(on, p + kG * kOperand, &mx, bar, kb * kBlock, m0);
                }
                if (++s == kStages) s = 0, ph ^= 1;
            }
            if (!ok) let_land();
        } else if (warp == kEpiWarps + 1) {  // ----------------------- MMA
            constexpr uint32_t idesc = instruction_desc(kF8, kTile, kNT, kDx, false);
            constexpr int kStepW = kDx ? 2048 : 32;  // bytes from one instruction's weights to the next one's
            const uint32_t base = smem_u32(stages);
            int buf = 0;
            uint32_t ph = 0, tph = 1;
            bool stage_full = false, part_free = false;  // seen while the MMAs before were issued
            for (int kb = k0; kb < k1; ++kb) {
                const bool fresh = kF8 || kb == k0, last = kF8 || kb + 1 == k1;
                if (!stage_full && !(ok = warp_wait(sh.full + s, ph, dead))) break;
                if (fresh && !part_free && !(ok = warp_wait(sh.tempty + buf, tph, dead))) break;
                tc_fence_after();
                const uint64_t dw = operand_desc(base + s * kStage, kDx ? kOperand / 2 : 16);
                const uint64_t dx = operand_desc(base + s * kStage + kG * kOperand, 16);
                const uint32_t d = tmem + buf * (kG * kNT);
                uint64_t *const empty = sh.empty + s, *const tfull = sh.tfull + buf;
                if (++s == kStages) s = 0, ph ^= 1;
                if (last && ++buf == kBufs) buf = 0, tph ^= 1;
                const bool f = mbar_test_wait(sh.full + s, ph), e = mbar_test_wait(sh.tempty + buf, tph);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int g = 0; g < kG; ++g)
                        mma<1, kF8>(on, d + g * kNT, dw + (g * kOperand + i * kStepW) / 16, dx + i * 2, idesc,
                                    fresh && i == 0 ? 0u : 1u);
                mma_commit_to<1>(on, empty);
                if (last) mma_commit_to<1>(on, tfull);
                stage_full = __all_sync(0xffffffffu, f);
                part_free = __all_sync(0xffffffffu, e);
            }
            if (!ok) let_land();
        }
        __syncwarp();
        if (share > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {  // ------------------------------------------------- sums, outputs
        more_registers();
        const int hh = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + hh * kH;
        const int groups = A.blocks;  // of codes: one a k-block
        int buf = 0;
        uint32_t tph = 0;
        bool ok = true;
        const int m = m0 + hh * kH;  // this thread's first token
        float v[kG * kH];
        auto done_reading = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sh.tempty + buf);
            if (++buf == kBufs) buf = 0, tph ^= 1;
        };
        if constexpr (kF8) {
#pragma unroll
            for (int i = 0; i < kG * kH; ++i) v[i] = 0.f;
            const float *s1 = A.a.sw1 + static_cast<long long>(tn) * groups;
            const float *s2 = kGated ? A.a.sw2 + static_cast<long long>(tn) * groups : s1;
            // the scales of the warp's tokens, a token a lane, one k-block ahead
            const float *sx0 = m + lane < A.a.M && lane < kH ? A.a.sx + (m + lane) * static_cast<long long>(A.a.sx_row) : nullptr;
            const float *sx1 = kH > 32 && m + 32 + lane < A.a.M
                                   ? A.a.sx + (m + 32 + lane) * static_cast<long long>(A.a.sx_row)
                                   : nullptr;
            const auto scale_at = [&](const float *p, int kb) {
                return p ? load_here(p + static_cast<long long>(kb) * A.a.sx_step) : 0.f;
            };
            float x0 = scale_at(sx0, k0), x1 = scale_at(sx1, k0);
            float f1 = load_here(s1 + k0), f2 = load_here(s2 + k0);
            for (int kb = k0; kb < k1; ++kb) {
                __syncwarp();
                // a token's scale times each weight's
#pragma unroll
                for (int g = 0; g < kG; ++g) {
                    if (lane < kH) token_scale[warp][g][lane] = x0 * (g ? f2 : f1);
                    if constexpr (kH > 32) token_scale[warp][g][lane + 32] = x1 * (g ? f2 : f1);
                }
                if (kb + 1 < k1) {
                    x0 = scale_at(sx0, kb + 1);
                    x1 = scale_at(sx1, kb + 1);
                    f1 = load_here(s1 + kb + 1);
                    f2 = load_here(s2 + kb + 1);
                }
                ok = ok && warp_wait(sh.tfull + buf, tph, dead);
                if (!ok) break;
                tc_fence_after();
                __syncwarp();
                const uint32_t at = lanes + buf * (kG * kNT);
                constexpr int kChunks = kH / kC;
                float d[2][kC];
                tmem_ld(d[0], at);
#pragma unroll
                for (int i = 0; i < kG * kChunks; ++i) {
                    const int g = i / kChunks, first = i % kChunks * kC;
                    tmem_wait(d[i & 1]);
                    if (i + 1 < kG * kChunks)
                        tmem_ld(d[(i + 1) & 1], at + (i + 1) / kChunks * kNT + (i + 1) % kChunks * kC);
#pragma unroll
                    for (int j = 0; j < kC; j += 4) {
                        const float4 c = *reinterpret_cast<const float4 *>(&token_scale[warp][g][first + j]);
                        float *t = v + g * kH + first + j;
                        const float2 lo = __ffma2_rn(make_float2(d[i & 1][j], d[i & 1][j + 1]), make_float2(c.x, c.y),
                                                     make_float2(t[0], t[1]));
                        const float2 hi = __ffma2_rn(make_float2(d[i & 1][j + 2], d[i & 1][j + 3]),
                                                     make_float2(c.z, c.w), make_float2(t[2], t[3]));
                        t[0] = lo.x, t[1] = lo.y, t[2] = hi.x, t[3] = hi.y;
                    }
                }
                done_reading();
            }
        } else {
            ok = ok && warp_wait(sh.tfull + buf, tph, dead);
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < kG * kH / kC; ++i) {
                    float d[kC];
                    tmem_ld(d, lanes + (buf * kG + i / (kH / kC)) * kNT + i % (kH / kC) * kC);
                    tmem_wait(d);
#pragma unroll
                    for (int j = 0; j < kC; ++j) v[i * kC + j] = d[j];
                }
                done_reading();
            }
        }
        if (!ok) {
#pragma unroll
            for (int i = 0; i < kG * kH; ++i) v[i] = __uint_as_float(0x7fffffffu);
        }
        // the sums as [weight][token][row], in place of the stages
        float *red = reinterpret_cast<float *>(stages);
#pragma unroll
        for (int i = 0; i < kG * kH; ++i) red[(i / kH * kNT + hh * kH + i % kH) * kTile + row] = v[i];
        if (share > 1)
            cluster_sync();
        else
            named_sync(1, kEpiThreads);
        // this CTA's share of the tokens, a warp each in turn, four rows of the weights a lane
        const int n = tn * kTile + 4 * lane;
        const bool inside = n < A.a.N;
        const int first = rank * (kNT / share);
        const int tokens = static_cast<int>(A.a.M - m0 < kNT ? A.a.M - m0 : kNT);
        const int end = min(tokens, first + kNT / share);
#pragma unroll 1
        for (int t = first + warp; t < end; t += kEpiWarps) {
            float2 lo[kG], hi[kG];
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                const uint32_t at = smem_u32(red + (g * kNT + t) * kTile + 4 * lane);
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int r = 0; r < 8; ++r) {  // in the order of k
                    if (r >= share) break;
                    const float4 f = share > 1 ? ld_cluster(cluster_addr_of(at, r)) : ld_cluster(at);
                    sum = make_float4(sum.x + f.x, sum.y + f.y, sum.z + f.z, sum.w + f.w);
                }
                lo[g] = make_float2(sum.x, sum.y);
                hi[g] = make_float2(sum.z, sum.w);
            }
            const long long row_y = (m0 + static_cast<long long>(t)) * A.a.ld_y + n;
            if constexpr (kGated) {
                if (A.a.g && inside) {
                    const long long row_g = (m0 + static_cast<long long>(t)) * A.a.ld_g + n;
                    store_four(A.a.g, A.a.g_f32, row_g, lo[0], hi[0]);
                    store_four(A.a.u, A.a.g_f32, row_g, lo[1], hi[1]);
                }
                lo[0] = __fmul2_rn(activate(lo[0], A.a.act), lo[1]);
                hi[0] = __fmul2_rn(activate(hi[0], A.a.act), hi[1]);
                if (kF8 && A.a.q) {
                    constexpr unsigned int kMag = 0x7fffffffu;
                    unsigned int mx = max(max(__float_as_uint(lo[0].x) & kMag, __float_as_uint(lo[0].y) & kMag),
                                          max(__float_as_uint(hi[0].x) & kMag, __float_as_uint(hi[0].y) & kMag));
                    const float scale = scale_of(__reduce_max_sync(0xffffffffu, inside ? mx : 0u)), inv = 1.f / scale;
                    const uint32_t code = e4m3_code(lo[0].x, scale, inv) | e4m3_code(lo[0].y, scale, inv) << 8 |
                                          e4m3_code(hi[0].x, scale, inv) << 16 |
                                          static_cast<uint32_t>(e4m3_code(hi[0].y, scale, inv)) << 24;
                    if (inside) *reinterpret_cast<uint32_t *>(A.a.q + (m0 + static_cast<long long>(t)) * A.a.ld_q + n) = code;
                    if (lane == 0) A.a.scales[(m0 + static_cast<long long>(t)) * ((A.a.N + kTile - 1) / kTile) + tn] = scale;
                    continue;
                }
            }
            if (inside) store_four(A.a.y, A.a.y_f32, row_y, lo[0], hi[0]);
        }
        if (share > 1) cluster_sync();  // the others have read this CTA's sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kEpiWarps + 1) tmem_dealloc<1>(tmem);
    if (tid == 0 && sh.dead != 0u) atomicOr(A.hdr + 2, kErrLocalTimeout);
}

struct Maps {
    CUtensorMap x, x2, w1, w2;
};

template <int kNT, bool kF8, bool kGated, bool kDx>
int start(const Maps &m, const NarrowArgs &w, int tiles, cudaStream_t st)
{
    const auto kernel = product_narrow_kernel<kNT, kF8, kGated, kDx>;
    constexpr int kSmem = Narrow<kNT, kGated>::kSmem;
    static std::atomic<unsigned long long> done{0};
    if (allow_shared(reinterpret_cast<const void *>(kernel), kSmem, done) < 0) return -1;
    return launch_early(kernel, dim3(tiles * w.share), kThreadsProduct, kSmem, w.share, st, "product (narrow) launch",
                        m.x, m.x2, m.w1, m.w2, w);
}

template <bool kF8, bool kGated, bool kDx>
int start_by_tokens(int nt, const Maps &m, const NarrowArgs &w, int tiles, cudaStream_t st)
{
    switch (nt) {
        case 16: return start<16, kF8, kGated, kDx>(m, w, tiles, st);
        case 32: return start<32, kF8, kGated, kDx>(m, w, tiles, st);
        case 64: return start<64, kF8, kGated, kDx>(m, w, tiles, st);
        default:
            if constexpr (kF8 && kGated)
                return -1;  // not asked for
            else
                return start<128, kF8, kGated, kDx>(m, w, tiles, st);
    }
}

// CTAs to a tile: clusters of up to 8 while all fit at once (a GPU of 148 SMs holds 74
// of two CTAs of this size, 33 of four, 15 of eight) and each CTA keeps 4 k-blocks.
int share_of(int tiles, int blocks, int sms)
{
    if (tiles <= (sms - 28) / 8 && blocks >= 32) return 8;
    if (tiles <= (sms - 16) / 4 && blocks >= 16) return 4;
    return tiles <= sms / 2 && blocks >= 8 ? 2 : 1;
}

}  // namespace

int launch_product_narrow(const ProductArgs &a, cudaStream_t st)
{
    const int sms = product_sms();
    if (sms < 1) return -1;
    const int nt = narrow_tokens(a.M, a.fp8 && a.gated);
    const int kb = a.fp8 ? 128 : 64, size = a.fp8 ? 1 : 2;
    Maps m;
    if (!encode_matrix(&m.x, a.x, size, a.M, a.K, a.ld_x, nt) ||
        !encode_matrix(&m.w1, a.w1, size, a.N, a.K, a.ld_w, kTile))
        return -1;
    m.x2 = m.x;
    if (!a.gated)
        m.w2 = m.w1;
    else if (!encode_matrix(&m.w2, a.w2, size, a.N, a.K, a.ld_w, kTile))
        return -1;
    NarrowArgs w{};
    w.tiles_m = static_cast<int>((a.M + nt - 1) / nt);
    const int tiles = w.tiles_m * ((a.N + kTile - 1) / kTile);
    w.blocks = (a.K + kb - 1) / kb;
    w.share = share_of(tiles, w.blocks, sms);
    w.a = a;
    w.hdr = static_cast<unsigned int *>(a.workspace);
    if (!a.gated) return start_by_tokens<true, false, false>(nt, m, w, tiles, st);
    return a.fp8 ? start_by_tokens<true, true, false>(nt, m, w, tiles, st)
                 : start_by_tokens<false, true, false>(nt, m, w, tiles, st);
}

// dx = dg Wg + du Wu as a product with few rows: the weights' columns are the tile's 128
// rows, and k runs through F twice.
int launch_ffn_dx_narrow(const FfnBackArgs &a, const uint16_t *dg, const uint16_t *du, bool beside, cudaStream_t st)
{
    const int sms = product_sms();
    if (sms < 1) return -1;
    const int nt = narrow_tokens(a.M, false);
    Maps m;
    if (!encode_matrix(&m.x, dg, 2, a.M, a.F, a.F, nt) || !encode_matrix(&m.x2, du, 2, a.M, a.F, a.F, nt) ||
        !encode_matrix(&m.w1, a.w1, 2, a.F, a.D, a.ld_w, 64) || !encode_matrix(&m.w2, a.w2, 2, a.F, a.D, a.ld_w, 64))
        return -1;
    NarrowArgs w{};
    w.tiles_m = static_cast<int>((a.M + nt - 1) / nt);
    const int tiles = w.tiles_m * ((a.D + kTile - 1) / kTile);
    w.blocks1 = (a.F + 63) / 64;
    w.blocks = 2 * w.blocks1;
    w.share = share_of(tiles, w.blocks, sms);
    w.beside = beside;
    w.a.y = a.dx;
    w.a.ld_y = a.ld_dx;
    w.a.M = a.M;
    w.a.N = a.D;
    w.hdr = static_cast<unsigned int *>(a.workspace);
    return start_by_tokens<false, false, true>(nt, m, w, tiles, st);
}

}  // namespace hyena
