// product_wide.cu -- products with many rows on the tensor cores of sm_100a, a
// pair of CTAs to a tile of 256 x 256 sums:
//
//   forward   y = x w^T, or act(x Wg^T) (x Wu^T): the pair's 256 columns are 128 of
//             the gate's and the same 128 of the up projection's
//   dx        dg Wg + du Wu: k runs through F twice
//   dW        dg^T x, du^T x: k runs through the tokens
//
// A TMA warp fills a ring of stages (128 rows x 128 bytes of each operand a CTA; where
// k is not the contiguous axis, boxes of 64 columns x 64 k, which the MMA takes as they
// are), one warp of the pair issues the MMAs, eight warps a CTA read tensor memory.
// The pair halves what each SM fetches of the second operand: a k-block is 32 KB for
// 512 cycles of MMAs.  Of the forward products there is also a form with one CTA to a
// tile of 128 x 256, four stages of 48 KB, for few rows and for tiles that come out in
// fewer waves that way (see ctas_of).
//
// bf16: sums stay in tensor memory over the whole of k, in one of two halves, so that a
// tile's outputs are worked out while the next one's MMAs run.  Bound by the tensor
// cores (86% of cycles active in 2048 x 4096 -> 11008) and, in long runs, by power: 8192
// x 4096 -> 11008 with silu 928-963 us, 1.53-1.59 PFLOP/s, where the measured library
// product does 1.62.
//
// e4m3 codes: the sums over each 128 k go times their scales into registers (128 a
// thread), since the scales are any fp32 numbers; the two halves of tensor memory then
// change places every k-block.  8192 x 4096 -> 12288: 389-393 us in calls with pauses between
// them, 2.1 PFLOP/s, 51% of cycles active; 440-460 back to back, by power.  Of a tile's 31000 cycles 27000 go to 32 k-blocks of 840, which is the
// way round of a half, 1700, over two halves: 165 to issue its MMAs, 330 more until
// warps that wait see them done (660 in the two warps that share a scheduler with the
// MMA warp, whatever that scheduler is, since MMAs that wait for the tensor core hold
// up what else is issued there), 400 to read, 60 to say so, 160 until the MMA warp
// knows, 512 the MMAs themselves; the rest to the outputs, which the MMAs run ahead of
// by two k-blocks only.  With sums read once a tile only, which is what the MMAs alone
// could do, 268 us, by power at 1.39 GHz instead of 1.59.  As fast: the MMAs of a
// k-block 60 to 160 cycles apart, or by a warp for each half; 32 columns a load instead
// of 16.  Slower: each group of 128 columns by MMAs and barriers of its own, four parts
// of tensor memory (460 us); polling (686); tiles of one CTA (410).
#include "product_kernel.cuh"

namespace hyena {

namespace {

constexpr int kTile = 128;                       // rows of a CTA's operands
constexpr int kOperand = kTile * kRowBytes;      // 16 KB
constexpr int kHalf = 64;                        // columns of each group of 128 a thread has

// kCtas: 2, a pair with half of the second operand each, or 1, which has all of it.
template <int kCtas>
struct Wide {
    static constexpr int kStage = (kCtas == 2 ? 2 : 3) * kOperand;
    static constexpr int kStages = kCtas == 2 ? 5 : 4;
    static constexpr int kPatches = kCtas == 2 ? 2 : 1;  // of a warp
    static constexpr int kSmem = kStages * kStage + kEpiWarps * kPatches * kPatch + 1024;
    static constexpr int kRows = kCtas * kTile;  // of a tile
};

enum { kForward = 0, kDx = 1, kDw = 2 };

struct WideArgs {
    Plan plan;
    long long rows;      // of the output
    int cols;
    int blocks1;         // dx: k-blocks of the first pair of operands
    int tile_cols;       // output columns of a tile
    ProductArgs a;       // forward
    unsigned int *hdr;
    bool beside;         // dx lets dW start beside it, and dW does not wait for it before its end
};

template <int kMode, bool kF8, int kCtas>
__global__ void __launch_bounds__(kThreadsProduct, 1)
    product_wide_kernel(const __grid_constant__ CUtensorMap a1, const __grid_constant__ CUtensorMap a2,
                        const __grid_constant__ CUtensorMap b1, const __grid_constant__ CUtensorMap b2,
                        const __grid_constant__ CUtensorMap c1, const __grid_constant__ CUtensorMap c2,
                        const __grid_constant__ CUtensorMap c3, const __grid_constant__ WideArgs A)
{
    constexpr bool kAmn = kMode == kDw, kBmn = kMode != kForward;
    constexpr int kBlock = kF8 ? 128 : 64;  // k of a block
    constexpr int kStage = Wide<kCtas>::kStage, kStages = Wide<kCtas>::kStages, kPatches = Wide<kCtas>::kPatches;
    constexpr int kRows = Wide<kCtas>::kRows;
    extern __shared__ unsigned char raw[];
    __shared__ ProductShared<kStages> sh;
    unsigned char *stages = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~1023ull);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kCtas == 2 ? static_cast<int>(cluster_rank()) : 0, unit = blockIdx.x / kCtas;
    const Plan &P = A.plan;
    volatile unsigned int *dead = &sh.dead;

    if (tid == kEpiThreads) {
        prefetch_map(&a1);
        prefetch_map(&b1);
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(sh.full + i, 1);
            mbar_init(sh.empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sh.tfull + i, 1);
            mbar_init(sh.tempty + i, kCtas * kEpiWarps);
        }
        sh.dead = 0u;
        fence_mbar_init();
    }
    if (warp == kEpiWarps + 1) tmem_alloc<kCtas>(&sh.tmem);
    tc_fence_before();
    all_sync<kCtas>();
    tc_fence_after();
    // dW reads dg, du and x, which were complete when dx passed its own wait
    if (kMode != kDw || !A.beside) wait_for_stream();
    if (kMode == kDx && A.beside) let_next_start();
    const uint32_t tmem = sh.tmem;

    // tile -> (tile row, tile column): bands of kBand tile rows, columns within
    auto place = [&](int tile, int &tm, int &tn) {
        const int band = P.by_band(tile), r = tile - band * (kBand * P.tiles_n);
        const int rows = P.tiles_m - band * kBand;
        if (rows >= kBand) {
            tn = r / kBand;
            tm = band * kBand + r % kBand;
        } else {
            tn = P.by_last(r);
            tm = band * kBand + (r - tn * rows);
        }
    };

    if (warp >= kEpiWarps) {
        fewer_registers();
        const uint32_t on = elected_lane();
        int s = 0;
        bool ok = true;
        if (warp == kEpiWarps) {  // ----------------------------------- TMA
            const uint32_t full0 = kCtas == 2 ? cluster_addr(sh.full, 0) : smem_u32(sh.full);
            const uint32_t first = rank == 0 ? on : 0u;
            uint32_t ph = 1;
            for (Walk w(P, unit); ok && w.next();) {
                int tm, tn;
                place(w.tile, tm, tn);
                const CUtensorMap *ma = &a1;
                int m = tm * kRows + rank * kTile;
                if (kMode == kDw && tm >= P.tiles_m / 2) {
                    ma = &a2;
                    m -= P.tiles_m / 2 * 256;
                }
                const bool gated = kMode == kForward && A.a.gated;
                const int n = tn * A.tile_cols + (gated ? 0 : rank * kTile);
                const CUtensorMap *mb = gated && rank ? &b2 : &b1;
                for (int kb = w.k0; kb < w.k1; ++kb) {
                    if (!(ok = warp_wait(sh.empty + s, ph, dead))) break;
                    expect_tx(first, sh.full + s, kCtas * kStage);
                    const uint32_t bar = full0 + 8 * s;
                    unsigned char *pa = stages + s * kStage, *pb = pa + kOperand;
                    int k = kb * kBlock;
                    if (kMode == kDx && kb >= A.blocks1) {
                        k -= A.blocks1 * kBlock;
                        ma = &a2;
                        mb = &b2;
                    }
                    if constexpr (kAmn) {
                        load_box<kCtas>(on, pa, ma, bar, m, k);
                        load_box<kCtas>(on, pa + kOperand / 2, ma, bar, m + 64, k);
                    } else {
                        load_box<kCtas>(on, pa, ma, bar, k, m);
                    }
                    if constexpr (kBmn) {
                        load_box<kCtas>(on, pb, mb, bar, n, k);
                        load_box<kCtas>(on, pb + kOperand / 2, mb, bar, n + 64, k);
                    } else {
                        load_box<kCtas>(on, pb, mb, bar, k, n);
                        if (kCtas == 1)
                            load_box<kCtas>(on, pb + kOperand, gated ? &b2 : &b1, bar, k, gated ? n : n + kTile);
                    }
                    if (++s == kStages) s = 0, ph ^= 1;
                }
            }
            if (!ok) let_land();
        } else if (warp == kEpiWarps + 1 && rank == 0) {  // ---------- MMA
            constexpr uint32_t idesc = instruction_desc(kF8, kRows, 256, kAmn, kBmn);
            constexpr uint64_t kStepA = (kAmn ? 2048 : 32) >> 4, kStepB = (kBmn ? 2048 : 32) >> 4;
            const uint32_t base = smem_u32(stages);
            int buf = 0;
            uint32_t ph = 0, tph = 1;
            bool stage_full = false, part_free = false;  // seen while the MMAs before were issued
            for (Walk w(P, unit); ok && w.next();) {
                for (int kb = w.k0; kb < w.k1; ++kb) {
                    const bool fresh = kF8 || kb == w.k0, last = kF8 || kb + 1 == w.k1;
                    if (!stage_full && !(ok = warp_wait(sh.full + s, ph, dead))) break;
                    const uint64_t da = operand_desc(base + s * kStage, kOperand / 2);
                    const uint64_t db = operand_desc(base + s * kStage + kOperand, kOperand / 2);
                    const uint32_t d = tmem + buf * 256;
                    if (fresh && !part_free && !(ok = warp_wait(sh.tempty + buf, tph, dead))) break;
                    tc_fence_after();
                    uint64_t *const empty = sh.empty + s, *const tfull = sh.tfull + buf;
                    if (++s == kStages) s = 0, ph ^= 1;
                    if (last) {
                        buf ^= 1;
                        if (buf == 0) tph ^= 1;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma<kCtas, kF8>(on, d, da + i * kStepA, db + i * kStepB, idesc, fresh && i == 0 ? 0u : 1u);
                    if (last) mma_commit_to<kCtas>(on, tfull);
                    mma_commit_to<kCtas>(on, empty);
                    const bool f = mbar_test_wait(sh.full + s, ph), e = mbar_test_wait(sh.tempty + buf, tph);
                    stage_full = __all_sync(0xffffffffu, f);
                    part_free = __all_sync(0xffffffffu, e);
                }
            }
            if (!ok) let_land();
        }
        __syncwarp();
    } else {  // ------------------------------------------------- sums, outputs
        more_registers();
        const int hh = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + hh * kHalf;
        const uint32_t tempty = kCtas == 2 ? cluster_addr(sh.tempty, 0) : smem_u32(sh.tempty);
        const int groups = P.blocks;  // of codes: one a k-block
        unsigned char *patch = stages + kStages * kStage + warp * (kPatches * kPatch);
        RowStore<kPatches> out(patch, lane);
        int buf = 0;
        uint32_t tph = 0;
        bool ok = true;
        Walk w(P, unit);
        int tm = 0, tn = 0;
        const float *sx = nullptr, *s1 = nullptr, *s2 = nullptr;
        float x = 0.f, f1 = 0.f, f2 = 0.f;
        bool live = false;
        // The next tile and, of codes, the scales of its first k-block: asked for before
        // the outputs of the tile in hand are written.
        auto advance = [&] {
            if (!w.next()) return false;
            place(w.tile, tm, tn);
            if constexpr (kF8) {
                const long long m = static_cast<long long>(tm) * kRows + rank * kTile + row;
                live = m < A.rows;
                sx = A.a.sx + (live ? m * A.a.sx_row + static_cast<long long>(w.k0) * A.a.sx_step : 0);
                const int n1 = A.a.gated ? tn : 2 * tn;
                // the second group of 128 columns may lie outside
                const int n2 = n1 + (!A.a.gated && tn * A.tile_cols + kTile < A.cols ? 1 : 0);
                s1 = A.a.sw1 + static_cast<long long>(n1) * groups + w.k0;
                s2 = (A.a.gated ? A.a.sw2 : A.a.sw1) + static_cast<long long>(n2) * groups + w.k0;
                x = live ? load_here(sx) : 0.f;
                f1 = load_here(s1);
                f2 = load_here(s2);
            }
            return true;
        };
        for (bool more = advance(); more;) {
            const int tile = w.tile, k0 = w.k0, k1 = w.k1, row0 = tm, col0 = tn;
            float v[2 * kHalf];
            auto done_reading = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(tempty + 8 * buf);
                buf ^= 1;
                if (buf == 0) tph ^= 1;
            };
            if constexpr (kF8) {
#pragma unroll
                for (int i = 0; i < 2 * kHalf; ++i) v[i] = 0.f;
                for (int kb = k0; kb < k1; ++kb) {
                    const float2 c1 = bcast2(x * f1), c2 = bcast2(x * f2);
                    if (kb + 1 < k1) {  // the next k-block's scales while this one's sums come in
                        sx += A.a.sx_step;
                        x = live ? load_here(sx) : 0.f;
                        f1 = load_here(++s1);
                        f2 = load_here(++s2);
                    }
                    ok = ok && warp_wait(sh.tfull + buf, tph, dead);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = lanes + buf * 256;
                    float d[2][16];
                    tmem_ld(d[0], at);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        tmem_wait(d[i & 1]);
                        if (i < 7)
                            tmem_ld(d[(i + 1) & 1], at + (i + 1) / 4 * kTile + (i + 1) % 4 * 16);
                        else
                            done_reading();
                        const float2 c = i < 4 ? c1 : c2;
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float2 r = __ffma2_rn(make_float2(d[i & 1][j], d[i & 1][j + 1]), c,
                                                        make_float2(v[i * 16 + j], v[i * 16 + j + 1]));
                            v[i * 16 + j] = r.x;
                            v[i * 16 + j + 1] = r.y;
                        }
                    }
                }
            } else {
                ok = ok && warp_wait(sh.tfull + buf, tph, dead);
                if (ok) {
                    tc_fence_after();
                    const uint32_t at = lanes + buf * 256;
                    float d[4][32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld(d[i], at + i / 2 * kTile + i % 2 * 32);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        tmem_wait(d[i]);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[i * 32 + j] = d[i][j];
                    }
                    done_reading();
                }
            }
            if (!ok) {
#pragma unroll
                for (int i = 0; i < 2 * kHalf; ++i) v[i] = __uint_as_float(0x7fffffffu);
            }
            more = advance();
            if (P.share > 1 &&
                !join_parts<kCtas>(v, P, unit, rank, tile, tid, reinterpret_cast<unsigned char *>(A.hdr), &sh.flag))
                continue;
            const long long m = static_cast<long long>(row0) * kRows + rank * kTile + row;
            const int n = col0 * A.tile_cols + hh * kHalf;
            const int left = A.cols - n;
            // the warp's first row; none of its rows may lie inside
            const int m0 = static_cast<int>(m) - lane;
            if constexpr (kMode != kForward) {
                // dW: the tile rows of the gate's, then those of the up projection's
                const bool second = kMode == kDw && row0 >= P.tiles_m / 2;
                const int r = second ? m0 - P.tiles_m / 2 * 256 : m0;
                if (r < A.rows) {
                    out.values(second ? &c2 : &c1, false, n, r, v, left);
                    out.values(second ? &c2 : &c1, false, n + kTile, r, v + kHalf, left - kTile);
                }
            } else if (!A.a.gated) {
                if (m0 < A.rows) {
                    out.values(&c1, A.a.y_f32, n, m0, v, left);
                    out.values(&c1, A.a.y_f32, n + kTile, m0, v + kHalf, left - kTile);
                }
            } else {
                if (A.a.g && m0 < A.rows) {
                    out.values(&c2, A.a.g_f32, n, m0, v, left);
                    out.values(&c3, A.a.g_f32, n, m0, v + kHalf, left);
                }
                gate<kHalf>(v, A.a.act);
                if (kF8 && A.a.q) {
                    // the largest of the row's 128 values: this half's and the other's
                    unsigned int mx = 0;
                    if (left >= kHalf) {
#pragma unroll
                        for (int i = 0; i < kHalf; ++i) mx = max(mx, __float_as_uint(v[i]) & 0x7fffffffu);
                    } else {
#pragma unroll
                        for (int i = 0; i < kHalf; ++i)
                            if (i < left) mx = max(mx, __float_as_uint(v[i]) & 0x7fffffffu);
                    }
                    sh.amax[tid] = mx;
                    named_sync(1, kEpiThreads);
                    mx = max(mx, sh.amax[tid ^ kTile]);
                    named_sync(1, kEpiThreads);
                    const float scale = scale_of(mx);
                    const bool small = scale < kSmallScale;
                    const float by = small ? scale * 0x1p+64f : scale, inv = 1.f / by;
                    if (small) {  // the same quotients
#pragma unroll
                        for (int i = 0; i < kHalf; ++i) v[i] *= 0x1p+64f;
                    }
                    const int rows = static_cast<int>(A.rows - m0 < 32 ? A.rows - m0 : 32);
                    store_codes(patch, lane, A.a.q + static_cast<long long>(m0) * A.a.ld_q + n, A.a.ld_q, left, rows, [&](int c) {
                        const uint2 lo = e4m3x8<true>(reinterpret_cast<const float(&)[8]>(v[16 * c]), by, inv);
                        const uint2 hi = e4m3x8<true>(reinterpret_cast<const float(&)[8]>(v[16 * c + 8]), by, inv);
                        return make_uint4(lo.x, lo.y, hi.x, hi.y);
                    });
                    if (hh == 0 && m < A.rows) A.a.scales[m * P.tiles_n + col0] = scale;
                } else if (m0 < A.rows) {
                    out.values(&c1, false, n, m0, v, left);
                }
            }
        }
        out.finish();
    }
    tc_fence_before();
    all_sync<kCtas>();  // the other CTA may still tell this one's barriers
    if (warp == kEpiWarps + 1) tmem_dealloc<kCtas>(tmem);
    if (tid == 0 && sh.dead != 0u) atomicOr(A.hdr + 2, kErrLocalTimeout);
    if (kMode == kDw && A.beside) wait_for_stream();  // dx, for whoever comes next
}

}  // namespace

// ---------------------------------------------------------------- host

namespace {

// Units to a tile, where that takes kJoin k-blocks off a unit's run, which is about
// what the joining costs.
constexpr int kJoin = 16;

void make_plan(Plan &p, int ctas, int units, int tiles_m, int tiles_n, int blocks)
{
    const int most = ctas == 2 ? kMostParts : kMostParts - 1;
    p.tiles_m = tiles_m;
    p.tiles_n = tiles_n;
    p.tiles = tiles_m * tiles_n;
    p.by_band.set(kBand * tiles_n);
    p.by_last.set(tiles_m % kBand ? tiles_m % kBand : 1);
    p.blocks = blocks;
    p.share = units / p.tiles < most ? units / p.tiles : most;
    if (p.share < 2 || blocks - blocks / p.share <= kJoin) p.share = 1;
    p.units = p.share > 1 ? p.tiles * p.share : (p.tiles < units ? p.tiles : units);
}

struct Maps {
    CUtensorMap a1, a2, b1, b2, c1, c2, c3;
};

// Outputs leave in boxes of 128 bytes of each of 32 rows.
bool encode_output(CUtensorMap *m, const void *p, bool f32, long long rows, int cols, long long ld)
{
    return encode_matrix(m, p, f32 ? 4 : 2, rows, cols, ld, 32);
}

template <int kMode, bool kF8, int kCtas>
int start(const Maps &m, const WideArgs &w, cudaStream_t st)
{
    static std::atomic<unsigned long long> done{0};
    const auto kernel = product_wide_kernel<kMode, kF8, kCtas>;
    if (allow_shared(reinterpret_cast<const void *>(kernel), Wide<kCtas>::kSmem, done) < 0) return -1;
    return launch_early(kernel, dim3(kCtas * w.plan.units), kThreadsProduct, Wide<kCtas>::kSmem, kCtas, st,
                        "product (wide) launch", m.a1, m.a2, m.b1, m.b2, m.c1, m.c2, m.c3, w);
}

// CTAs to a tile.  Tiles of one, half as many rows, are taken where they make fewer
// waves, since a wave of them takes 1.0 (codes) to 1.3 (bf16, which they feed 48 KB a
// k-block instead of 32) of a pair's time: codes from 11 : 10 on, which is up to ten
// waves, bf16 from 4 : 3.  4096 -> 11008 with silu, pairs and single ones: 300 rows (3
// waves and 2) in codes 59 and 42 us, in bf16 71 and 61; 1664 rows (9 and 8) 168 and
// 160, 211 and 225.  -> 14336, 640 rows (5 and 4) 98 and 82, 125 and 118, but -> 8192,
// 1152 rows (5 and 4) in bf16 117 and 120.  Up to 128 rows a pair has one half empty:
// with as many waves 23.5 and 22 us (4096 -> 18944 in codes), 22.8 and 24.1 (4096 ->
// 6144 x 2), with fewer 41 and 25 (11008 x 2).
int ctas_of(const ProductArgs &a, int sms, int tile_cols)
{
    if (a.M <= kTile) return 1;
    const long long across = (a.N + tile_cols - 1) / tile_cols;
    const long long one = ((a.M + kTile - 1) / kTile * across + sms - 1) / sms;
    const long long two = ((a.M + 2 * kTile - 1) / (2 * kTile) * across + sms / 2 - 1) / (sms / 2);
    return (a.fp8 ? 10 * two >= 11 * one : 3 * two >= 4 * one) ? 1 : 2;
}

}  // namespace

int launch_product_wide(const ProductArgs &a, cudaStream_t st)
{
    const int sms = product_sms();
    if (sms < 2) return -1;
    WideArgs w{};
    w.tile_cols = a.gated ? kTile : 2 * kTile;
    const int ctas = ctas_of(a, sms, w.tile_cols), rows = ctas * kTile;
    const int kb = a.fp8 ? 128 : 64, size = a.fp8 ? 1 : 2;
    Maps m;
    bool ok = encode_matrix(&m.a1, a.x, size, a.M, a.K, a.ld_x, kTile) &&
              encode_matrix(&m.b1, a.w1, size, a.N, a.K, a.ld_w, kTile) &&
              (!a.gated || encode_matrix(&m.b2, a.w2, size, a.N, a.K, a.ld_w, kTile)) &&
              (!a.y || encode_output(&m.c1, a.y, a.y_f32, a.M, a.N, a.ld_y)) &&
              (!a.g || (encode_output(&m.c2, a.g, a.g_f32, a.M, a.N, a.ld_g) &&
                        encode_output(&m.c3, a.u, a.g_f32, a.M, a.N, a.ld_g)));
    if (!ok) return -1;
    m.a2 = m.a1;
    if (!a.gated) m.b2 = m.b1;
    if (!a.y) m.c1 = m.a1;  // not read
    if (!a.g) m.c2 = m.c3 = m.c1;
    make_plan(w.plan, ctas, sms / ctas, static_cast<int>((a.M + rows - 1) / rows),
              (a.N + w.tile_cols - 1) / w.tile_cols, (a.K + kb - 1) / kb);
    w.rows = a.M;
    w.cols = a.N;
    w.a = a;
    w.hdr = static_cast<unsigned int *>(a.workspace);
    if (ctas == 1) return a.fp8 ? start<kForward, true, 1>(m, w, st) : start<kForward, false, 1>(m, w, st);
    return a.fp8 ? start<kForward, true, 2>(m, w, st) : start<kForward, false, 2>(m, w, st);
}

int launch_ffn_gradients(const FfnBackArgs &a, const uint16_t *dg, const uint16_t *du, cudaStream_t st)
{
    const int u = product_sms() / 2;
    if (u < 1) return -1;
    const bool narrow = ffn_dx_is_narrow(a.M, a.D);
    Maps x{}, w;  // of dx and of dW
    if (!narrow &&
        (!encode_matrix(&x.a1, dg, 2, a.M, a.F, a.F, kTile) || !encode_matrix(&x.a2, du, 2, a.M, a.F, a.F, kTile) ||
         !encode_matrix(&x.b1, a.w1, 2, a.F, a.D, a.ld_w, 64) || !encode_matrix(&x.b2, a.w2, 2, a.F, a.D, a.ld_w, 64) ||
         !encode_output(&x.c1, a.dx, false, a.M, a.D, a.ld_dx)))
        return -1;
    if (!encode_matrix(&w.a1, dg, 2, a.M, a.F, a.F, 64) || !encode_matrix(&w.a2, du, 2, a.M, a.F, a.F, 64) ||
        !encode_matrix(&w.b1, a.x, 2, a.M, a.D, a.ld_x, 64) ||
        !encode_output(&w.c1, a.dw1, false, a.F, a.D, a.ld_dw) || !encode_output(&w.c2, a.dw2, false, a.F, a.D, a.ld_dw))
        return -1;
    x.c2 = x.c3 = x.c1;
    w.b2 = w.b1;
    w.c3 = w.c1;
    WideArgs p{}, q{};
    p.tile_cols = q.tile_cols = 2 * kTile;
    p.blocks1 = (a.F + 63) / 64;
    make_plan(p.plan, 2, u, static_cast<int>((a.M + 255) / 256), (a.D + 255) / 256, 2 * p.blocks1);
    make_plan(q.plan, 2, u, 2 * ((a.F + 255) / 256), (a.D + 255) / 256, static_cast<int>((a.M + 63) / 64));
    p.rows = a.M;
    q.rows = a.F;
    p.cols = q.cols = a.D;
    p.hdr = q.hdr = static_cast<unsigned int *>(a.workspace);
    // Side by side, so that dW's units begin where dx leaves room (step of 1000 x 1032 ->
    // 2760: 80 us one after the other, 72), unless both put parts in the workspace.
    p.beside = q.beside = narrow || p.plan.share == 1 || q.plan.share == 1;
    const int n = narrow ? launch_ffn_dx_narrow(a, dg, du, p.beside, st) : start<kDx, false, 2>(x, p, st);
    if (n < 0) return -1;
    const int k = start<kDw, false, 2>(w, q, st);
    return k < 0 ? -1 : n + k;
}

}  // namespace hyena
