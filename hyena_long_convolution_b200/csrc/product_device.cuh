// product_device.cuh -- device-side helpers of the products and the
// feed-forward block: tcgen05 (tensor cores, tensor memory), clusters of two
// CTAs, bounded waits, activations.  Hand-written inline PTX; no library code.
#pragma once

#include "layer_device.cuh"
#include "product_internal.h"

namespace hyena {

// ---------------------------------------------------------------- waits

// Waits for the phase with the given parity, at most four seconds of the time
// that the CTA runs (a look that comes late, after the CTA was suspended, counts
// as 10 ms).  `dead` is the CTA's: once one wait ran out, the others end too.
__device__ __forceinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile unsigned int *dead)
{
    unsigned long long last = global_timer_ns(), spent = 0;
    while (*dead == 0u) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        const unsigned long long now = global_timer_ns();
        const unsigned long long step = now - last;
        spent += step < 10000000ull ? step : 10000000ull;
        last = now;
        if (spent > 4 * kWaitLimitNs) *dead = 1u;
    }
    return false;
}

__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile unsigned int *dead)
{
    if (mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, dead);
}

// 1 in one lane of a whole warp.  The loops that feed TMA and the tensor cores are
// run by all lanes of a warp, and only the instructions themselves by this one, by
// predicate: operands stay in uniform registers and the warp never parts.  (A
// k-block's turn of the MMA warp, by a branch around them: 770 cycles, of which the
// MMAs take 120.)
__device__ __forceinline__ uint32_t elected_lane()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}

// wait_phase by all lanes of a warp, which agree on the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile unsigned int *dead)
{
    return __all_sync(0xffffffffu, wait_phase(bar, parity, dead)) != 0;
}

// A read-only load that is issued where it stands: left to the compiler, a value that is
// asked for early may be loaded where it is used.
__device__ __forceinline__ float load_here(const float *p)
{
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// ---------------------------------------------------------------- launches

// The kernels here are launched while the one ahead of them in the stream ends
// (launch_early): what comes before this reads and writes no global memory.  They do
// not let the next one start early (griddepcontrol.launch_dependents), since one that
// reads its inputs before it waits, as the modal scan's short passes do, would read
// outputs that are not written yet.  The one exception is dx, which lets dW start beside
// it: dW reads nothing of dx's and waits for it before it ends, so that what follows dW
// finds both written.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// The address of shared memory (of `p`) in CTA `rank` of this cluster.
__device__ __forceinline__ uint32_t cluster_addr_of(uint32_t addr, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank)
{
    return cluster_addr_of(smem_u32(p), rank);
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// All threads of the CTA, or of the cluster.
template <int kCtas>
__device__ __forceinline__ void all_sync()
{
    if constexpr (kCtas > 1)
        cluster_sync();
    else
        __syncthreads();
}

// Tells a barrier of a CTA of this cluster that tensor memory has been read: the
// reads are complete (tmem_wait), so that nothing has to be released at cluster
// scope, whose fence took 4.6 of the 17 cycles that an instruction waited.
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Brings a tensor map close, before the first load that needs it.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// The lane with `on` != 0 ...
// ... arrives at a barrier and adds to the bytes that it waits for;
__device__ __forceinline__ void expect_tx(uint32_t on, uint64_t *bar, uint32_t bytes)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%1], "
        "%2;\n\t}" ::"r"(on),
        "r"(smem_u32(bar)), "r"(bytes)
        : "memory");
}

// ... loads a box of a matrix into this CTA's shared memory, counted by its barrier,
// or, of a pair of CTAs, by a barrier of either.
template <int kCtas>
__device__ __forceinline__ void load_box(uint32_t on, void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1)
{
    if constexpr (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%1], [%2, {%3, %4}], [%5];\n\t}" ::"r"(on),
            "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%1], [%2, {%3, %4}], [%5];\n\t}" ::"r"(on),
            "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

constexpr uint32_t kTmemAll = 512;  // columns

template <int kCtas>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot)
{
    if constexpr (kCtas == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                     "r"(kTmemAll)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                     "r"(kTmemAll)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}

template <int kCtas>
__device__ __forceinline__ void tmem_dealloc(uint32_t base)
{
    if constexpr (kCtas == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(kTmemAll));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(kTmemAll));
}

// Shared-memory operand of 128-byte rows as TMA's 128-byte swizzle leaves them,
// tile at a 1024-byte boundary.  K-major (rows of the operand's M or N, 128 bytes
// of k each): groups of 8 rows 1024 bytes apart; the next MMA's k is 32 bytes on.
// MN-major (a row for each k, 64 bf16 of M or N each): groups of 8 k 1024 bytes
// apart, the next 64 of M or N `lbo` bytes on; the next MMA's k is 2048 bytes on.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>((lbo >> 4) & 0x3fffu) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// fp32 accumulators; bf16 (kind::f16) or e4m3 (kind::f8f6f4) operands.
__host__ __device__ constexpr uint32_t instruction_desc(bool f8, int m, int n, bool a_mn, bool b_mn)
{
    return (1u << 4) | ((f8 ? 0u : 1u) << 7) | ((f8 ? 0u : 1u) << 10) | (static_cast<uint32_t>(a_mn) << 15) |
           (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// The lane with `on` != 0: D (tensor memory) (+)= A B.
template <int kCtas, bool kF8>
__device__ __forceinline__ void mma(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
#define HYENA_MMA(group, kind)                                                                                       \
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"                       \
                 "@q tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),         \
                 "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(on)                                                       \
                 : "memory")
    if constexpr (kCtas == 2) {
        if constexpr (kF8)
            HYENA_MMA("2", "f8f6f4");
        else
            HYENA_MMA("2", "f16");
    } else {
        if constexpr (kF8)
            HYENA_MMA("1", "f8f6f4");
        else
            HYENA_MMA("1", "f16");
    }
#undef HYENA_MMA
}

// The lane with `on` != 0 has `bar` (of both CTAs of a pair) told when the MMAs that
// it issued so far are done.
template <int kCtas>
__device__ __forceinline__ void mma_commit_to(uint32_t on, uint64_t *bar)
{
    if constexpr (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
            "%1;\n\t}" ::"r"(smem_u32(bar)),
            "h"(static_cast<uint16_t>(3)), "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
            "r"(on)
            : "memory");
}

// Consecutive fp32 columns of the warp's 32 lanes of tensor memory, a lane a
// thread; complete after tmem_wait, through which the values go so that nothing
// reads them before.
#define HYENA_R8(v, o)                                                                                             \
    "=f"(v[o]), "=f"(v[o + 1]), "=f"(v[o + 2]), "=f"(v[o + 3]), "=f"(v[o + 4]), "=f"(v[o + 5]), "=f"(v[o + 6]),     \
        "=f"(v[o + 7])
__device__ __forceinline__ void tmem_ld(float (&v)[8], uint32_t a)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : HYENA_R8(v, 0) : "r"(a));
}
__device__ __forceinline__ void tmem_ld(float (&v)[16], uint32_t a)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : HYENA_R8(v, 0), HYENA_R8(v, 8)
        : "r"(a));
}
__device__ __forceinline__ void tmem_ld(float (&v)[32], uint32_t a)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : HYENA_R8(v, 0), HYENA_R8(v, 8), HYENA_R8(v, 16), HYENA_R8(v, 24)
        : "r"(a));
}
#undef HYENA_R8
#define HYENA_W8(v, o)                                                                                             \
    "+f"(v[o]), "+f"(v[o + 1]), "+f"(v[o + 2]), "+f"(v[o + 3]), "+f"(v[o + 4]), "+f"(v[o + 5]), "+f"(v[o + 6]),     \
        "+f"(v[o + 7])
__device__ __forceinline__ void tmem_wait(float (&v)[8])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : HYENA_W8(v, 0)::"memory");
}
__device__ __forceinline__ void tmem_wait(float (&v)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : HYENA_W8(v, 0), HYENA_W8(v, 8)::"memory");
}
__device__ __forceinline__ void tmem_wait(float (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : HYENA_W8(v, 0), HYENA_W8(v, 8), HYENA_W8(v, 16), HYENA_W8(v, 24)::"memory");
}
#undef HYENA_W8

// ---------------------------------------------------------------- activations

// Two values at a time, in packed arithmetic.  With n = 2^-24: 2^x is the hardware's
// approximation, 4 n off, and 1 / x likewise, 2 n; each rounding on the way to an
// exponential's argument z moves e^z by n |z|.  There are two for silu (its constant,
// the product), three for gelu (the square too) and eight for gelu_tanh (four in the
// cubic, three in its constant), so that e^z is (2, 3, 8 |z| + 4) n off, and the
// sigmoid, 1 - s of that and 3 n.  Below 2^-126 either is zero.
__device__ __forceinline__ float2 exp2_2(float2 x)
{
    float2 r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(x.y));
    return r;
}
__device__ __forceinline__ float2 reciprocal2(float2 x)
{
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(x.y));
    return r;
}

constexpr float kLog2E = 1.44269504088896341f;

// 1 / (1 + e^(-c x)), zero where the exponential passes 2^126.
__device__ __forceinline__ float2 sigmoid2(float2 x, float c)
{
    const float2 e = exp2_2(__fmul2_rn(x, bcast2(-c * kLog2E)));
    return reciprocal2(__fadd2_rn(e, bcast2(1.f)));
}

// The normal distribution's Phi(g), and e^{-g^2 / 2} in e.  Phi(-|g|) = t p(t)
// e^{-g^2 / 2} with t = 1 / (1 + 0.3 |g|) and p of degree 7 fitted to the function in
// the relative maximum norm for |g| <= 14.5 (1.9e-7 with the coefficients in fp32;
// with the arithmetic 30 half steps of fp32 and those of the exponential), which keeps
// the digits that 1 + erf loses where g is negative.  Beyond 13.2 the exponential, and
// Phi(-|g|), is zero.
__device__ __forceinline__ float2 normal_cdf2(float2 g, float2 &e)
{
    const float2 a = make_float2(fabsf(g.x), fabsf(g.y));
    const float2 t = reciprocal2(__ffma2_rn(a, bcast2(0.3f), bcast2(1.f)));
    float2 p = bcast2(0.03542377054691315f);
    p = __ffma2_rn(p, t, bcast2(-0.15615858137607574f));
    p = __ffma2_rn(p, t, bcast2(0.20455701649188995f));
    p = __ffma2_rn(p, t, bcast2(-0.05203420668840408f));
    p = __ffma2_rn(p, t, bcast2(0.1276918649673462f));
    p = __ffma2_rn(p, t, bcast2(0.10017592459917068f));
    p = __ffma2_rn(p, t, bcast2(0.12071213871240616f));
    p = __ffma2_rn(p, t, bcast2(0.11963200569152832f));
    e = exp2_2(__fmul2_rn(__fmul2_rn(g, g), bcast2(-0.5f * kLog2E)));
    const float2 tail = __fmul2_rn(__fmul2_rn(p, t), e);
    const float2 rest = __ffma2_rn(tail, bcast2(-1.f), bcast2(1.f));
    return make_float2(g.x < 0.f ? tail.x : rest.x, g.y < 0.f ? tail.y : rest.y);
}

constexpr float kGeluTanh = 1.59576912160573072f;  // 2 sqrt(2 / pi): (1 + tanh z) / 2 = sigmoid(2 z)

// act(g) of the gated block (HYENA_ACT_*).
template <int kAct>
__device__ __forceinline__ float2 activation2(float2 g)
{
    if constexpr (kAct == HYENA_ACT_SILU) {
        return __fmul2_rn(g, sigmoid2(g, 1.f));
    } else if constexpr (kAct == HYENA_ACT_GELU) {
        float2 e;
        return __fmul2_rn(g, normal_cdf2(g, e));
    } else if constexpr (kAct == HYENA_ACT_GELU_TANH) {
        const float2 z = __ffma2_rn(__fmul2_rn(__fmul2_rn(g, g), bcast2(0.044715f)), g, g);
        return __fmul2_rn(g, sigmoid2(z, kGeluTanh));
    } else {
        return g;
    }
}

// act(g), and act'(g) in d.
template <int kAct>
__device__ __forceinline__ float2 activation_slope2(float2 g, float2 &d)
{
    if constexpr (kAct == HYENA_ACT_SILU) {
        const float2 s = sigmoid2(g, 1.f), rest = __ffma2_rn(s, bcast2(-1.f), bcast2(1.f));
        d = __fmul2_rn(s, __ffma2_rn(g, rest, bcast2(1.f)));
        return __fmul2_rn(g, s);
    } else if constexpr (kAct == HYENA_ACT_GELU) {
        float2 e;
        const float2 c = normal_cdf2(g, e);
        d = __ffma2_rn(g, __fmul2_rn(e, bcast2(0.39894228040143268f)), c);
        return __fmul2_rn(g, c);
    } else if constexpr (kAct == HYENA_ACT_GELU_TANH) {
        // g^2 at most 2^64, beyond which (1 - s) is 0 or y is: times an infinite `in` that is NaN
        const float2 sq = __fmul2_rn(g, g), g2 = make_float2(fminf(sq.x, 0x1p+64f), fminf(sq.y, 0x1p+64f));
        const float2 s = sigmoid2(__ffma2_rn(__fmul2_rn(g2, bcast2(0.044715f)), g, g), kGeluTanh);
        const float2 in = __ffma2_rn(g2, bcast2(3.f * 0.044715f * kGeluTanh), bcast2(kGeluTanh));
        const float2 y = __fmul2_rn(g, s);
        d = __ffma2_rn(__fmul2_rn(y, __ffma2_rn(s, bcast2(-1.f), bcast2(1.f))), in, s);
        return y;
    } else {
        d = bcast2(1.f);
        return g;
    }
}

}  // namespace hyena
