// product_kernel.cuh -- what the two tensor-core product kernels share: the
// division of their work, the joining of partial sums, the outputs.
#pragma once

#include "product_device.cuh"

namespace hyena {

constexpr int kEpiWarps = 8;                      // read tensor memory: warp w lanes 32 (w % 4) .. + 31
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kThreadsProduct = kEpiThreads + 128; // + a TMA warp, an MMA warp and two that only end
// Registers: the reading warps hold 128 sums a thread.  256 x 208 + 128 x 88 = 384 x
// 168, what the kernels are launched with.
constexpr int kRegsEpi = 208, kRegsAux = 88;
constexpr int kRowBytes = 128;                    // of a k-block: 64 bf16 or 128 codes
constexpr size_t kProductHeader = HYENA_PRODUCT_HEADER; // 256 bytes of header, then a counter for each split tile

// Quotients by a number that the host knows, of 0 <= n < 2^31: the high part of a
// product (m = ceil(2^(31 + s) / d), 2^s >= d).  An integer division takes 150 cycles,
// of which a tile's place needs two.
struct Divide {
    unsigned int m;
    int s;
    void set(int d)
    {
        s = 0;
        while ((1ll << s) < d) ++s;
        m = static_cast<unsigned int>(((1ull << (31 + s)) + d - 1) / d);
    }
    __device__ __forceinline__ int operator()(int n) const
    {
        return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned int>(n)) * m) >> (31 + s));
    }
};

constexpr int kBand = 8;  // tile rows that are walked together, so that L2 holds what they share

// How a product is divided: tiles of the output, k-blocks of a tile, units (pairs of
// CTAs).  A unit takes whole tiles one after another; or, with few tiles, `share`
// units take an even part of a tile's k-blocks each and the parts are joined.
// (Sharing out what is left of many tiles after whole waves costs more than it saves,
// at every number of tiles from 76 to 1376; runs that cross from one tile into the
// next have two joins to wait for.)
struct Plan {
    int tiles_m, tiles_n, tiles;
    Divide by_band, by_last;  // by the tiles of a band of kBand tile rows, and by the rows of the last, smaller one
    int blocks;               // k-blocks of a tile
    int units, share;
};

struct Walk {
    int tile, k0, k1, step, end;
    __device__ __forceinline__ Walk(const Plan &p, int unit)
    {
        const int part = unit % p.share;
        step = p.share > 1 ? p.tiles : p.units;  // a part: one tile
        tile = unit / p.share - step;
        end = p.tiles;
        k0 = static_cast<int>(static_cast<long long>(p.blocks) * part / p.share);
        k1 = static_cast<int>(static_cast<long long>(p.blocks) * (part + 1) / p.share);
    }
    __device__ __forceinline__ bool next() { return (tile += step) < end; }
};

constexpr int kMostParts = 4;  // of a pair's tile; of a single CTA's, never so few, 3

// v = the parts' sums, in order.  Written out for each number of parts, so that many
// loads are under way: part by part, 2.8 us each.
template <int kParts, int kCtas, int kV>
__device__ __forceinline__ void add_parts(float (&v)[kV], const float4 *parts)
{
    constexpr size_t kNext = static_cast<size_t>(kCtas) * (kV / 4) * kEpiThreads;  // the next unit's slot of the same rows
#pragma unroll
    for (int i = 0; i < kV / 4; ++i) {
        float4 f = __ldcg(parts + i * kEpiThreads);
#pragma unroll
        for (int u = 1; u < kParts; ++u) {
            const float4 g = __ldcg(parts + u * kNext + i * kEpiThreads);
            f = make_float4(f.x + g.x, f.y + g.y, f.z + g.z, f.w + g.w);
        }
        v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
}

// The sums of a part of a tile go to memory, and the CTA whose part is the last to
// arrive adds them up in the order of k, so that the result does not depend on
// which that was.  The two CTAs of a pair each have their own half of the tile.
// v: this thread's sums, kept as float4 [i][thread] of its part's slot.  True in the
// CTA that holds the tile's sums.
template <int kCtas, int kV>
__device__ __forceinline__ bool join_parts(float (&v)[kV], const Plan &p, int unit, int rank, int tile, int t,
                                           unsigned char *workspace, unsigned int *flag)
{
    constexpr size_t kSlot = static_cast<size_t>(kV / 4) * kEpiThreads;
    float4 *slots = reinterpret_cast<float4 *>(workspace + kProductHeader) + t;
    float4 *own = slots + (static_cast<long long>(kCtas) * unit + rank) * kSlot;
#pragma unroll
    for (int i = 0; i < kV / 4; ++i)
        own[i * kEpiThreads] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    named_sync(1, kEpiThreads);
    if (t == 0) {
        __threadfence();  // the stores of all, which the barrier has ordered before it
        unsigned int *count = reinterpret_cast<unsigned int *>(workspace + 256) + kCtas * tile + rank;
        const bool last = atomicAdd(count, 1u) + 1 == static_cast<unsigned int>(p.share);
        if (last) *count = 0u;  // for the next call
        __threadfence();
        *flag = last ? 1u : 0u;
    }
    named_sync(1, kEpiThreads);
    if (*flag == 0u) return false;
    const float4 *parts = slots + (static_cast<long long>(kCtas) * tile * p.share + rank) * kSlot;
    if (p.share == 2)
        add_parts<2, kCtas, kV>(v, parts);
    else if (kCtas == 1 || p.share == 3)
        add_parts<3, kCtas, kV>(v, parts);
    else
        add_parts<kCtas == 1 ? 3 : kMostParts, kCtas, kV>(v, parts);
    return true;
}

// g[i] <- act(g[i]) u[i] of kV each.
template <int kAct, int kV>
__device__ __forceinline__ void gate(float (&v)[2 * kV])
{
#pragma unroll
    for (int i = 0; i < kV; i += 2) {
        const float2 y = __fmul2_rn(activation2<kAct>(make_float2(v[i], v[i + 1])),
                                    make_float2(v[kV + i], v[kV + i + 1]));
        v[i] = y.x;
        v[i + 1] = y.y;
    }
}

template <int kV>
__device__ __forceinline__ void gate(float (&v)[2 * kV], int act)
{
    switch (act) {
        case HYENA_ACT_SILU: gate<HYENA_ACT_SILU, kV>(v); break;
        case HYENA_ACT_GELU: gate<HYENA_ACT_GELU, kV>(v); break;
        case HYENA_ACT_GELU_TANH: gate<HYENA_ACT_GELU_TANH, kV>(v); break;
        default: gate<HYENA_ACT_IDENTITY, kV>(v); break;
    }
}

__device__ __forceinline__ void load8_bf16(float (&v)[8], const uint16_t *p)
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

__device__ __forceinline__ void load8_f32(float (&v)[8], const float *p)
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// 8 values to 16 bytes of bf16.
__device__ __forceinline__ uint4 pack_bf16(const float *v)
{
    uint4 q;
    q.x = float2_to_bf16x2(make_float2(v[0], v[1]));
    q.y = float2_to_bf16x2(make_float2(v[2], v[3]));
    q.z = float2_to_bf16x2(make_float2(v[4], v[5]));
    q.w = float2_to_bf16x2(make_float2(v[6], v[7]));
    return q;
}

// A warp's 32 rows of outputs, a row a lane in registers, go through 4 KB of shared
// memory, in rows of 128 bytes whose 16-byte chunks are permuted by the row (chunk c
// of row r at c ^ (r % 8)): free of bank conflicts, and TMA's 128-byte swizzle.
// Straight from the registers a store touches 32 rows, 16 bytes of each: 8000 cycles
// for a CTA's 128 x 256 sums; from the patch by the lanes 2800.
constexpr int kPatch = 4096;

// Codes, 64 bytes a row, are written by the lanes: `chunk(c)` gives a lane's 16 bytes,
// row r goes to p + r * pitch, `left` bytes (a multiple of 8) of it, `rows` rows.
template <class F>
__device__ __forceinline__ void store_codes(unsigned char *patch, int lane, unsigned char *p, long long pitch, int left,
                                            int rows, F chunk)
{
    constexpr int kChunks = 4, kRows = 32 / kChunks;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
        *reinterpret_cast<uint4 *>(patch + lane * 128 + ((c ^ (lane & 7)) << 4)) = chunk(c);
    __syncwarp();
    const int c = lane % kChunks;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int r = i * kRows + lane / kChunks;
        const uint4 q = *reinterpret_cast<const uint4 *>(patch + r * 128 + ((c ^ (r & 7)) << 4));
        unsigned char *to = p + r * pitch + c * 16;
        if (r >= rows || c * 16 >= left) continue;
        if (c * 16 + 16 <= left)
            *reinterpret_cast<uint4 *>(to) = q;
        else
            *reinterpret_cast<uint2 *>(to) = make_uint2(q.x, q.y);
    }
}

// Values go by TMA, which leaves out what lies outside the matrix.
// kPatches of a warp: with two, one is filled while TMA reads the other.
template <int kPatches>
struct RowStore {
    unsigned char *patches;
    int lane, next;
    __device__ __forceinline__ RowStore(unsigned char *p, int l) : patches(p), lane(l), next(0) {}

    // 128 bytes of each row at (column, row) of the matrix
    template <class F>
    __device__ __forceinline__ void put(const CUtensorMap *map, int column, int row, F chunk)
    {
        unsigned char *patch = patches + next * kPatch;
        next ^= kPatches - 1;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPatches - 1) : "memory");
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4 *>(patch + lane * 128 + ((c ^ (lane & 7)) << 4)) = chunk(c);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
                "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
                "r"(column), "r"(row), "r"(smem_u32(patch))
                : "memory");
    }

    // 64 values as bf16 or fp32; `left` columns of the matrix from there on (maybe none)
    __device__ __forceinline__ void values(const CUtensorMap *map, bool f32, int column, int row, const float *v, int left)
    {
        if (left <= 0) return;
        if (!f32) {
            put(map, column, row, [&](int c) { return pack_bf16(v + 8 * c); });
            return;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (left <= 32 * h) return;
            put(map, column + 32 * h, row, [&](int c) {
                const float *f = v + 32 * h + 4 * c;
                return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                  __float_as_uint(f[3]));
            });
        }
    }

    // before the CTA ends: everything written
    __device__ __forceinline__ void finish()
    {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
};

__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi)); }
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsAux)); }

// Shared memory of a CTA beside its stages.
template <int kStages>
struct ProductShared {
    uint64_t full[kStages];   // a stage's operands arrived
    uint64_t empty[kStages];  // the MMAs that read a stage are done
    uint64_t tfull[8];        // a part of tensor memory holds sums
    uint64_t tempty[8];       // it has been read
    uint32_t tmem;
    unsigned int dead;        // a wait ran out
    unsigned int flag;
    unsigned int amax[kEpiThreads];
};

// What a CTA whose wait ran out does before it ends: its copies and MMAs under
// way land within microseconds or not at all; 20 ms are given them.
__device__ __forceinline__ void let_land()
{
    const unsigned long long t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 20000000ull) {
    }
}

}  // namespace hyena
